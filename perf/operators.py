"""Cases of the sequence operators: causal depthwise convolution, selective
state space scan, and norms with gate and residual scale.

`run` makes one pass through an operator: as elementary torch operations in
32 bits where `own` is false, through the package's entry points where it is
true.  `exact` computes the same outputs in 64 bits from the definitions,
token by token.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # a batch of prompts through the convolution of a wide block; x is the first half of a projection's output
        dict(name="causal_prompt", op="causal_forward", io="bf16", B=4, T=4096, C=4096, k=4, halves=True, state=False, ragged=False),
        # a few odd-sized requests that continue from their own states, padded to the longest
        dict(name="causal_continued", op="causal_forward", io="f32", B=3, T=517, C=390, k=3, halves=False, state=True, ragged=True),
        # its gradients in a training step
        dict(name="causal_grad", op="causal_backward", io="bf16", B=8, T=2048, C=2048, k=4, halves=False, state=False, ragged=False),
        # one token of each of a batch of requests being answered
        dict(name="causal_token", op="causal_step", io="bf16", B=32, C=2048, k=4, ragged=False),
        # one long prompt
        dict(name="scan_long_prompt", op="scan_forward", io="bf16", B=1, T=8192, C=2048, N=16, G=1, halves=True, state=False, ragged=False),
        # the forward pass of a training step
        dict(name="scan_train", op="scan_forward", io="bf16", B=8, T=2048, C=2048, N=16, G=1, halves=True, state=False, ragged=False),
        # the backward pass of a training step
        dict(name="scan_grad", op="scan_backward", io="bf16", B=8, T=1024, C=2048, N=16, G=1, halves=True, state=False, ragged=False),
        # gradients through padded rows of odd lengths, cut from longer texts: states come in and their gradients go out
        dict(name="scan_grad_continued", op="scan_backward", io="f32", B=2, T=301, C=384, N=12, G=2, halves=False, state=True, ragged=True),
        # one token of each of a batch of requests being answered
        dict(name="scan_token", op="scan_step", io="bf16", B=64, C=4096, N=16, G=1, ragged=False),
        # gated norm after a block, residual scale and the next block's norm, over a training batch
        dict(name="norm_block", op="norm_forward", io="bf16", res="f32", B=8, T=2048, C=2048, post=True, ragged=False),
        # its gradients
        dict(name="norm_block_grad", op="norm_backward", io="bf16", res="f32", B=8, T=2048, C=2048, post=True, ragged=False),
        # residual and norm for one token of each of a few requests
        dict(name="norm_token", op="norm_forward", io="bf16", res="bf16", B=16, T=1, C=4096, post=False, ragged=False),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["causal_forward", "causal_backward", "causal_step", "scan_forward", "scan_forward", "scan_backward",
                     "scan_backward", "scan_step", "norm_forward", "norm_backward"])
    io = rng.choice(["f32", "bf16"])
    ragged = rng.random() < 0.4
    if op in ("causal_step", "scan_step"):
        c = dict(op=op, io=io, B=_spread(rng, 1, 256), C=_spread(rng, 96, 8192), ragged=ragged)
        if op == "causal_step":
            return dict(c, k=rng.randint(2, 7))
        N = rng.choice([4, 8, 16, 16, 32, 64])
        return dict(c, B=max(1, min(c["B"], (1 << 24) // (c["C"] * N))), N=N, G=1)
    most = 1 << 25
    C = _spread(rng, 96, 4096)
    T = _spread(rng, 1, 8192)
    B = _spread(rng, 1, 16)
    if op.startswith("norm"):
        most >>= 1
        B = max(1, min(B, most // (T * C)))
        return dict(op=op, io=io, res=rng.choice([io, "f32"]), B=B, T=T, C=C, post=rng.random() < 0.5, ragged=ragged)
    both = dict(halves=rng.random() < 0.5, state=rng.random() < 0.5, ragged=ragged)
    if op.startswith("causal"):
        B = max(1, min(B, most // (T * C)))
        return dict(op=op, io=io, B=B, T=T, C=C, k=rng.randint(2, 7), **both)
    N = rng.choice([4, 8, 13, 16, 16, 24, 32])
    if op == "scan_backward":
        most >>= 1
        T = min(T, 4096)
    G = rng.choice([1, 1, 2])
    C -= C % G
    while B > 1 and B * T * C * N > most * 16:
        B -= 1
    T = max(1, min(T, most * 16 // (B * C * N)))
    return dict(op=op, io=io, B=B, T=T, C=C, N=N, G=G, **both)


class _Draws:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, *shape, dtype=torch.float32):
        return torch.randn(*shape, generator=self.g, device="cuda").to(dtype)

    def uniform(self, *shape):
        return torch.rand(*shape, generator=self.g, device="cuda")

    def lengths(self, B, T):
        """Rows of all lengths up to T, the last one whole and, of several, the first one empty."""
        n = (self.uniform(B) * (T + 1)).to(torch.int32).clamp(0, T)
        if B > 1:
            n[0] = 0
        n[-1] = T
        return n


def _tokens(d, case, dt):
    """[B][T][C] activations: on their own, or as one half of a projection's output."""
    B, T, C = case["B"], case["T"], case["C"]
    if case["halves"]:
        both = d.normal(B, T, 2 * C, dtype=dt)
        return both[..., :C], both[..., C:]
    return d.normal(B, T, C, dtype=dt), d.normal(B, T, C, dtype=dt)


def prepare(case, seed):
    d = _Draws(seed)
    op, dt, C = case["op"], DTYPES[case["io"]], case["C"]
    B, T = case["B"], case.get("T", 1)
    s = {"op": op}
    if op.startswith("causal"):
        k = case["k"]
        s["w"] = (d.uniform(C, k) * 2 - 1) / math.sqrt(k)
        s["b"] = (d.uniform(C) * 2 - 1) / math.sqrt(k)
        if op == "causal_step":
            s["x"], s["state"] = d.normal(B, C, dtype=dt), d.normal(B, k - 1, C, dtype=dt)
            s["active"] = (d.uniform(B) < 0.7).to(torch.int32) if case["ragged"] else None
            return s
        s["x"] = _tokens(d, case, dt)[0]
        s["state"] = d.normal(B, k - 1, C, dtype=dt) if case["state"] else None
        s["lengths"] = d.lengths(B, T) if case["ragged"] else None
        if op == "causal_backward":
            s["dy"] = d.normal(B, T, C, dtype=dt)
            s["dstate"] = d.normal(B, k - 1, C, dtype=dt) if case["state"] else None
        return s
    if op.startswith("scan"):
        N, G = case["N"], case["G"]
        # decay rates spread around 1..N, step sizes softplus(dt + dt_bias) of 1e-3 to 1e-1
        s["a"] = -torch.arange(1, N + 1, device="cuda", dtype=torch.float32) * torch.exp(0.1 * d.normal(C, N))
        step = torch.exp(d.uniform(C) * math.log(100.0) + math.log(1e-3))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        s["d"] = 1 + 0.1 * d.normal(C)
        if op == "scan_step":
            s["x"], s["dt"], s["z"] = d.normal(B, C, dtype=dt), (0.5 * d.normal(B, C)).to(dt), d.normal(B, C, dtype=dt)
            bc = d.normal(B, 2 * N, dtype=dt)
            s["b"], s["c"] = bc[:, :N], bc[:, N:]
            s["state"] = d.normal(B, C, N)
            s["active"] = (d.uniform(B) < 0.7).to(torch.int32) if case["ragged"] else None
            return s
        s["x"], s["z"] = _tokens(d, case, dt)
        s["dt"] = (0.5 * d.normal(B, T, C)).to(dt)
        bc = d.normal(B, T, 2 * G * N, dtype=dt)
        s["b"], s["c"] = bc[..., : G * N].unflatten(-1, (G, N)), bc[..., G * N:].unflatten(-1, (G, N))
        s["state"] = d.normal(B, C, N) if case["state"] else None
        s["lengths"] = d.lengths(B, T) if case["ragged"] else None
        if op == "scan_backward":
            s["dy"] = d.normal(B, T, C, dtype=dt)
            s["dstate"] = d.normal(B, C, N) if case["state"] else None
        return s
    res = DTYPES[case["res"]]
    s["x"], s["res"] = d.normal(B, T, C, dtype=dt), (4 * d.normal(B, T, C)).to(res)
    s["gate"] = d.normal(B, T, C, dtype=dt) if case["post"] else None
    s["w"] = 1 + 0.1 * d.normal(C) if case["post"] else None
    s["scale"], s["w_res"] = 0.5 + 0.1 * d.normal(C), 1 + 0.1 * d.normal(C)
    s["lengths"] = d.lengths(B, T) if case["ragged"] else None
    if op == "norm_backward":
        s["dy"], s["dres"] = d.normal(B, T, C, dtype=dt), d.normal(B, T, C).to(res)
    return s


def run(s):
    if own:
        return _RUN_OWN[s["op"]](s)
    return _RUN_PLAIN[s["op"]](s)


# ------------------------------------------------ the package's entry points
def _own_causal_forward(s):
    import depthwise_convolution_wtconv_b200 as wt
    y, state = wt.causal_forward(s["x"], s["w"], s["b"], state=s["state"], lengths=s["lengths"])
    return dict(y=y, state=state)


def _own_causal_backward(s):
    import depthwise_convolution_wtconv_b200 as wt
    dx, g = wt.causal_backward(s["x"], s["dy"], s["w"], s["b"], state=s["state"], lengths=s["lengths"], dstate=s["dstate"])
    return dict(dx=dx, dw=g["dw"], db=g["db"], dstate=g["dstate"])


def _own_causal_step(s):
    import depthwise_convolution_wtconv_b200 as wt
    y = wt.causal_step(s["x"], s["state"], s["w"], s["b"], active=s["active"])
    return dict(y=y, state=s["state"])


def _own_scan_forward(s):
    import depthwise_convolution_wtconv_b200 as wt
    y, state = wt.scan_forward(s["x"], s["dt"], s["a"], s["b"], s["c"], s["d"], s["z"], s["dt_bias"], state=s["state"], lengths=s["lengths"])
    return dict(y=y, state=state)


def _own_scan_backward(s):
    import depthwise_convolution_wtconv_b200 as wt
    return wt.scan_backward(s["x"], s["dt"], s["a"], s["b"], s["c"], s["dy"], s["d"], s["z"], s["dt_bias"], state=s["state"],
                            lengths=s["lengths"], dstate=s["dstate"])


def _own_scan_step(s):
    import depthwise_convolution_wtconv_b200 as wt
    y = wt.scan_step(s["x"], s["dt"], s["state"], s["a"], s["b"], s["c"], s["d"], s["z"], s["dt_bias"], active=s["active"])
    return dict(y=y, state=s["state"])


def _own_norm_forward(s):
    import depthwise_convolution_wtconv_b200 as wt
    y, res = wt.norm_forward(s["x"], s["w"], gate=s["gate"], res=s["res"], scale=s["scale"], w_res=s["w_res"], lengths=s["lengths"])
    return dict(y=y, res=res)


def _own_norm_backward(s):
    import depthwise_convolution_wtconv_b200 as wt
    return wt.norm_backward(s["x"], s["dy"], s["w"], gate=s["gate"], res=s["res"], scale=s["scale"], w_res=s["w_res"], dres=s["dres"],
                            lengths=s["lengths"])


_RUN_OWN = dict(causal_forward=_own_causal_forward, causal_backward=_own_causal_backward, causal_step=_own_causal_step,
                scan_forward=_own_scan_forward, scan_backward=_own_scan_backward, scan_step=_own_scan_step,
                norm_forward=_own_norm_forward, norm_backward=_own_norm_backward)


# ------------------------------------------------------------ the plain forms
def _sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def _dsilu(v):
    g = _sigmoid(v)
    return g * (1 + v * (1 - g))


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _valid(s):
    """[B][T][1] truth values of the tokens within their row's length, or None."""
    if s["lengths"] is None:
        return None
    return (torch.arange(s["x"].shape[1], device="cuda") < s["lengths"][:, None])[..., None]


def _kept(v, valid):
    """v in 32 bits, zero behind the lengths."""
    return v.float() if valid is None else torch.where(valid, v.float(), 0.0)


def _tail(s, T, k):
    """[B][k-1][1] positions, in the inputs with the state before them, of what the state after the pass holds."""
    n = torch.full((s["x"].shape[0],), T, device="cuda") if s["lengths"] is None else s["lengths"].long()
    return (n[:, None] + torch.arange(k - 1, device="cuda"))[..., None]


def _joined(s, valid):
    x = _kept(s["x"], valid)
    k = s["w"].shape[1]
    before = x.new_zeros(x.shape[0], k - 1, x.shape[2]) if s["state"] is None else s["state"].float()
    return torch.cat([before, x], 1)


def _plain_causal_forward(s):
    T, k, dt = s["x"].shape[1], s["w"].shape[1], s["x"].dtype
    valid = _valid(s)
    joined = _joined(s, valid)
    p = (joined.unfold(1, k, 1) * s["w"]).sum(-1) + s["b"]
    y = _kept(p * _sigmoid(p), valid)
    state = torch.gather(joined, 1, _tail(s, T, k).expand(-1, -1, joined.shape[2]))
    return dict(y=y.to(dt), state=state.to(dt))


def _plain_causal_backward(s):
    T, k, dt = s["x"].shape[1], s["w"].shape[1], s["x"].dtype
    valid = _valid(s)
    joined = _joined(s, valid)
    taps = joined.unfold(1, k, 1)
    p = (taps * s["w"]).sum(-1) + s["b"]
    g = _kept(s["dy"], valid) * _dsilu(p)
    zeros = g.new_zeros(g.shape[0], k - 1, g.shape[2])
    djoined = (torch.cat([zeros, g, zeros], 1).unfold(1, k, 1) * s["w"].flip(1)).sum(-1)
    if s["dstate"] is not None:
        djoined.scatter_add_(1, _tail(s, T, k).expand(-1, -1, g.shape[2]), s["dstate"].float())
    return dict(dx=djoined[:, k - 1:].to(dt), dw=(taps * g[..., None]).sum((0, 1)), db=g.sum((0, 1)),
                dstate=None if s["state"] is None else djoined[:, : k - 1].to(dt))


def _plain_causal_step(s):
    joined = torch.cat([s["state"], s["x"][:, None]], 1)
    p = (joined.float() * s["w"].t()).sum(1) + s["b"]
    y, state = p * _sigmoid(p), joined[:, 1:]
    if s["active"] is not None:
        on = (s["active"] != 0)[:, None]
        y, state = torch.where(on, y, 0.0), torch.where(on[..., None], state, s["state"])
    s["state"].copy_(state.contiguous())
    return dict(y=y.to(s["x"].dtype), state=s["state"])


def _recurrence(a, b, first):
    """h_t = a_t h_{t-1} + b_t along dim 1 by doubling: after each turn, a and b are those of twice as many steps at once.
    Overwrites a and b."""
    if first is not None:
        b[:, 0] += a[:, 0] * first
    n = 1
    while n < b.shape[1]:
        b[:, n:] += a[:, n:] * b[:, :-n]
        a[:, n:] *= a[:, :-n].clone()
        n *= 2
    return b


def _scan_parts(s):
    """delta, x in 32 bits (delta is zero behind the lengths, which leaves the state as it is), and B, C of each channel's group."""
    valid = _valid(s)
    v = s["dt"].float() + s["dt_bias"]
    delta = _kept(_softplus(v), valid)
    x = _kept(s["x"], valid)
    per = x.shape[2] // s["b"].shape[2]
    b, c = (_kept(s[m].flatten(2), valid).unflatten(-1, s["b"].shape[2:]).repeat_interleave(per, 2) for m in "bc")
    return valid, v, delta, x, b, c


def _plain_scan_forward(s):
    dt = s["x"].dtype
    valid, _, delta, x, b, c = _scan_parts(s)
    h = _recurrence(torch.exp(delta[..., None] * s["a"]), (delta * x)[..., None] * b, s["state"])
    z = _kept(s["z"], valid)
    y = ((h * c).sum(-1) + s["d"] * x) * (z * _sigmoid(z))
    return dict(y=y.to(dt), state=h[:, -1].clone())


def _plain_scan_backward(s):
    dt = s["x"].dtype
    valid, v, delta, x, b, c = _scan_parts(s)
    a = torch.exp(delta[..., None] * s["a"])
    h = _recurrence(a.clone(), (delta * x)[..., None] * b, s["state"])
    z, dy = _kept(s["z"], valid), _kept(s["dy"], valid)
    p = (h * c).sum(-1) + s["d"] * x
    dp, dz = dy * z * _sigmoid(z), dy * p * _dsilu(z)
    # the adjoint runs backwards: e_t = c_t dp_t + a_{t+1} e_{t+1}
    after = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    e = _recurrence(after.flip(1), (dp[..., None] * c).flip(1), s["dstate"]).flip(1)
    del after
    B, T, C, N = h.shape
    G = s["b"].shape[2]
    db = (e * (delta * x)[..., None]).view(B, T, G, C // G, N).sum(3)
    dc = (h * dp[..., None]).view(B, T, G, C // G, N).sum(3)
    before = torch.cat([torch.zeros_like(h[:, :1]) if s["state"] is None else s["state"][:, None], h[:, :-1]], 1)
    ah = a * before  # the state that each token kept
    del before, h
    eb = (e * b).sum(-1)
    ddt = ((e * ah * s["a"]).sum(-1) + x * eb) * _sigmoid(v)
    ddt = _kept(ddt, valid)
    da = (e * ah * delta[..., None]).sum((0, 1))
    return dict(dx=(s["d"] * dp + delta * eb).to(dt), ddt=ddt.to(dt), da=da, db=db.to(dt), dc=dc.to(dt), dd=(dp * x).sum((0, 1)),
                dz=dz.to(dt), ddt_bias=ddt.sum((0, 1)), dstate=None if s["state"] is None else a[:, 0] * e[:, 0])


def _plain_scan_step(s):
    x, z = s["x"].float(), s["z"].float()
    delta = _softplus(s["dt"].float() + s["dt_bias"])
    h = torch.exp(delta[..., None] * s["a"]) * s["state"] + (delta * x)[..., None] * s["b"].float()[:, None]
    y = ((h * s["c"].float()[:, None]).sum(-1) + s["d"] * x) * (z * _sigmoid(z))
    if s["active"] is not None:
        on = (s["active"] != 0)[:, None]
        y, h = torch.where(on, y, 0.0), torch.where(on[..., None], h, s["state"])
    s["state"].copy_(h)
    return dict(y=y.to(s["x"].dtype), state=s["state"])


EPS = 1e-6


def _norm_parts(s):
    valid = _valid(s)
    x = _kept(s["x"], valid)
    u, v, n1 = x, x, None
    if s["gate"] is not None:
        g = _kept(s["gate"], valid)
        u = v = x * g * _sigmoid(g)
    if s["w"] is not None:
        n1 = torch.rsqrt((u * u).mean(-1, keepdim=True) + EPS)
        v = u * n1 * s["w"]
    r = _kept(s["res"], valid) + s["scale"] * v
    n2 = torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS)
    return valid, x, u, v, n1, r, n2


def _plain_norm_forward(s):
    _, _, _, _, _, r, n2 = _norm_parts(s)
    return dict(y=(r * n2 * s["w_res"]).to(s["x"].dtype), res=r.to(s["res"].dtype))


def _plain_norm_backward(s):
    valid, x, u, v, n1, r, n2 = _norm_parts(s)
    dt = s["x"].dtype
    dy = _kept(s["dy"], valid)
    t = dy * s["w_res"]
    dr = _kept(s["dres"], valid) + n2 * t - r * n2 ** 3 * (r * t).mean(-1, keepdim=True)
    out = dict(dw_res=(dy * r * n2).sum((0, 1)), dscale=(dr * v).sum((0, 1)), dres=dr.to(s["res"].dtype), dw=None, dgate=None)
    du = dr * s["scale"]
    if s["w"] is not None:
        out["dw"] = (du * u * n1).sum((0, 1))
        t = du * s["w"]
        du = n1 * t - u * n1 ** 3 * (u * t).mean(-1, keepdim=True)
    if s["gate"] is not None:
        g = _kept(s["gate"], valid)
        out["dgate"] = (du * x * _dsilu(g)).to(dt)
        du = du * g * _sigmoid(g)
    out["dx"] = du.to(dt)
    return out


_RUN_PLAIN = dict(causal_forward=_plain_causal_forward, causal_backward=_plain_causal_backward, causal_step=_plain_causal_step,
                  scan_forward=_plain_scan_forward, scan_backward=_plain_scan_backward, scan_step=_plain_scan_step,
                  norm_forward=_plain_norm_forward, norm_backward=_plain_norm_backward)


# --------------------------------------------------------------- what it takes
def work(case):
    """Inputs once, outputs once; a multiply-add is two operations, exp, division and the like one each."""
    op, C, B, T = case["op"], case["C"], case["B"], case.get("T", 1)
    E = 4 if case["io"] == "f32" else 2
    M = B * T
    if op.startswith("causal"):
        k = case["k"]
        params = 4 * C * (k + 1)
        state = E * B * (k - 1) * C
        if op == "causal_step":
            return dict(bytes=2 * E * M * C + 2 * state + params, flops=M * C * (2 * k + 4))
        if op == "causal_forward":
            return dict(bytes=2 * E * M * C + params + state * (1 + case["state"]), flops=M * C * (2 * k + 4))
        return dict(bytes=3 * E * M * C + 2 * params + 3 * state * case["state"], flops=M * C * (6 * k + 10))
    if op.startswith("scan"):
        N, G = case["N"], case["G"]
        state, params = 4 * B * C * N, 4 * C * (N + 2)
        if op in ("scan_forward", "scan_step"):
            return dict(bytes=E * M * (4 * C + 2 * G * N) + params + state * (2 if op == "scan_step" else 1 + case["state"]),
                        flops=M * C * (7 * N + 12))
        return dict(bytes=E * M * (7 * C + 4 * G * N) + 2 * params + 3 * state * case["state"], flops=M * C * (20 * N + 30))
    R = 4 if case["res"] == "f32" else 2
    gate, post = int(case["post"]), int(case["post"])
    if op == "norm_forward":
        return dict(bytes=M * C * (E * (2 + gate) + 2 * R) + 4 * C * (2 + post), flops=M * C * (8 + 9 * gate))
    return dict(bytes=M * C * (E * (3 + 2 * gate) + 3 * R) + 8 * C * (2 + post), flops=M * C * (22 + 24 * gate))


# ------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    s = {n: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for n, v in s.items()}
    B = s["x"].shape[0]
    T = s["x"].shape[1] if s["x"].dim() == 3 else 1
    if "lengths" in s:
        n = [T] * B if s["lengths"] is None else s["lengths"].tolist()
    else:
        n = [1] * B if s["active"] is None else [int(v != 0) for v in s["active"].tolist()]
        s["x"] = s["x"][:, None]
        if s["op"] == "scan_step":
            s.update({m: s[m][:, None] for m in ("dt", "z")} | {m: s[m][:, None, None] for m in ("b", "c")})
    return _EXACT[s["op"].split("_")[0]](s, n)


def _exact_causal(s, n):
    """Row by row: the row's inputs behind its state, then a sum over the taps."""
    x, w = s["x"], s["w"]
    B, T, C = x.shape
    k = w.shape[1]
    y, state = torch.zeros_like(x), x.new_zeros(B, k - 1, C)
    back = s["op"] == "causal_backward"
    dx, dstate, dw, db = torch.zeros_like(x), x.new_zeros(B, k - 1, C), torch.zeros_like(w), torch.zeros_like(s["b"])
    for i in range(B):
        before = s["state"][i] if s["state"] is not None else x.new_zeros(k - 1, C)
        row = torch.cat([before, x[i, : n[i]]])
        p = s["b"].repeat(n[i], 1)
        for j in range(k):
            p += w[:, j] * row[j: j + n[i]]
        gate = torch.sigmoid(p)
        y[i, : n[i]] = p * gate
        state[i] = row[n[i]:]
        if back:
            g = s["dy"][i, : n[i]] * (gate + p * gate * (1 - gate))
            drow = torch.zeros_like(row)
            for j in range(k):
                drow[j: j + n[i]] += w[:, j] * g
                dw[:, j] += (g * row[j: j + n[i]]).sum(0)
            if s["dstate"] is not None:
                drow[n[i]:] += s["dstate"][i]
            db += g.sum(0)
            dstate[i], dx[i, : n[i]] = drow[: k - 1], drow[k - 1:]
    if back:
        return dict(dx=dx, dw=dw, db=db, dstate=None if s["state"] is None else dstate)
    if s["op"] == "causal_step":
        off = [i for i in range(B) if n[i] == 0]
        state[off] = s["state"][off]
        return dict(y=y[:, 0], state=state)
    return dict(y=y, state=state)


def _exact_scan(s, n):
    """Token by token through the definition; the gradients token by token back, over the kept states."""
    x, a = s["x"], s["a"]
    B, T, C = x.shape
    N, G = a.shape[1], s["b"].shape[2]
    n = torch.tensor(n, device=x.device)
    live = torch.arange(T, device=x.device)[None] < n[:, None]
    back = s["op"] == "scan_backward"
    h = s["state"].clone() if s["state"] is not None else x.new_zeros(B, C, N)
    y = torch.zeros_like(x)
    kept = x.new_empty(T + 1, B, C, N) if back else None
    if back:
        kept[0] = h
    pre = torch.zeros_like(x)

    def at(t):
        on = live[:, t, None]
        step = torch.where(on, torch.nn.functional.softplus(s["dt"][:, t] + s["dt_bias"], threshold=60), 0.0)
        xt = torch.where(on, x[:, t], 0.0)
        b, c = (torch.where(on[..., None], s[m][:, t], 0.0).repeat_interleave(C // G, 1) for m in "bc")
        return on, step, xt, b, c

    for t in range(T):
        on, step, xt, b, c = at(t)
        h = torch.exp(step[..., None] * a) * h + (step * xt)[..., None] * b
        pre[:, t] = (h * c).sum(-1) + s["d"] * xt
        zt = torch.where(on, s["z"][:, t], 0.0)
        y[:, t] = pre[:, t] * zt * torch.sigmoid(zt)
        if back:
            kept[t + 1] = h
    if not back:
        return dict(y=y[:, 0] if s["op"] == "scan_step" else y, state=h)
    dx, ddt, dz = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    db, dc = x.new_zeros(B, T, G, N), x.new_zeros(B, T, G, N)
    da, dd, dbias = torch.zeros_like(a), torch.zeros_like(s["d"]), torch.zeros_like(s["d"])
    e = s["dstate"].clone() if s["dstate"] is not None else torch.zeros_like(h)
    for t in reversed(range(T)):
        on, step, xt, b, c = at(t)
        zt, g = torch.where(on, s["z"][:, t], 0.0), torch.where(on, s["dy"][:, t], 0.0)
        gate = torch.sigmoid(zt)
        dp = g * zt * gate
        dz[:, t] = g * pre[:, t] * (gate + zt * gate * (1 - gate))
        e = e + dp[..., None] * c
        dc[:, t] = (dp[..., None] * kept[t + 1]).view(B, G, C // G, N).sum(2)
        db[:, t] = (e * (step * xt)[..., None]).view(B, G, C // G, N).sum(2)
        decay = torch.exp(step[..., None] * a)
        dlog = e * decay * kept[t]
        da += (dlog * step[..., None]).sum(0)
        eb = (e * b).sum(-1)
        dv = torch.where(on, ((dlog * a).sum(-1) + eb * xt) * torch.sigmoid(s["dt"][:, t] + s["dt_bias"]), 0.0)
        ddt[:, t] = dv
        dbias += dv.sum(0)
        dd += (dp * xt).sum(0)
        dx[:, t] = s["d"] * dp + step * eb
        e = decay * e
    return dict(dx=dx, ddt=ddt, da=da, db=db, dc=dc, dd=dd, dz=dz, ddt_bias=dbias, dstate=None if s["state"] is None else e)


def _exact_norm(s, n):
    """The forward formulas on the rows within their lengths, and their gradients by differentiation."""
    x = s["x"]
    B, T, C = x.shape
    live = (torch.arange(T, device=x.device)[None] < torch.tensor(n, device=x.device)[:, None]).reshape(-1)
    names = [m for m in ("x", "gate", "res") if s[m] is not None]
    rows = {m: s[m].reshape(-1, C)[live].requires_grad_() for m in names}
    par = {m: s[m].clone().requires_grad_() for m in ("w", "scale", "w_res") if s[m] is not None}

    def whole(v):
        out = x.new_zeros(B * T, C)
        out[live] = v
        return out.view(B, T, C)

    with torch.enable_grad():
        u = rows["x"]
        if "gate" in rows:
            u = u * rows["gate"] * torch.sigmoid(rows["gate"])
        if "w" in par:
            u = par["w"] * u / torch.sqrt(u.square().mean(-1, keepdim=True) + EPS)
        r = rows["res"] + par["scale"] * u
        y = par["w_res"] * r / torch.sqrt(r.square().mean(-1, keepdim=True) + EPS)
        if s["op"] == "norm_forward":
            return dict(y=whole(y.detach()), res=whole(r.detach()))
        total = (y * s["dy"].reshape(-1, C)[live]).sum() + (r * s["dres"].reshape(-1, C)[live]).sum()
        total.backward()
    out = dict(dgate=None, dw=None, **{"d" + m: whole(v.grad) for m, v in rows.items() if m != "gate"})
    out.update({"d" + m: v.grad for m, v in par.items()})
    if "gate" in rows:
        out["dgate"] = whole(rows["gate"].grad)
    return out


_EXACT = dict(causal=_exact_causal, scan=_exact_scan, norm=_exact_norm)
