"""The sequence operators on the GPU against the float64 oracle.

Every value is held to the rounding of its type plus, for the operations in
the longest chain behind it, one 32-bit error each relative to the sum of its
terms' absolute values (tests/seq_cases.py)."""
import pytest
import torch

import depthwise_convolution_wtconv_b200 as wt
import seq_cases as sc
from seq_cases import causal_case, causal_oracle, check, cuda, norm_case, norm_oracle, scan_case, scan_ops, scan_oracle

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ causal
# strips are 16 tokens at these sizes, gradient blocks 128; vectors 4, 2 or 1 channels (longer strips: test_seq_edges_gpu.py)
CAUSAL = [
    dict(B=1, T=1, C=8, k=4, io="f32"),
    dict(B=2, T=2, C=16, k=4, io="bf16"),                      # shorter than the taps
    dict(B=3, T=33, C=7, k=3, io="bf16", ragged=True),         # odd channels, one token in the last strip
    dict(B=4, T=31, C=20, k=2, io="f32", ragged=True, state=False),
    dict(B=2, T=64, C=136, k=5, io="bf16", state=False),
    dict(B=2, T=65, C=260, k=8, io="f32", ragged=True),
    dict(B=1, T=300, C=36, k=7, io="bf16", bias=False),        # a second gradient block, no bias
    dict(B=5, T=257, C=3, k=6, io="f32", ragged=True),
    dict(B=2, T=40, C=24, k=1, io="f32", ragged=True),         # no state at all
]


def _name(c):
    return "-".join(f"{k}{v}" for k, v in c.items())


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("case", CAUSAL, ids=_name)
def test_causal_forward(cuda_ok, case, silu):
    s = causal_case(**case)
    d = cuda(s)
    y, state = wt.causal_forward(d["x"], d["w"], d["b"], silu=silu, state=d["state"], lengths=d["lengths"])
    want, size = causal_oracle(s, silu), causal_oracle(s, silu, mag=True)
    check(y, want["y"], size["y"], case["k"] + 8, "y")
    assert torch.equal(state.double().cpu(), torch.from_numpy(want["state"]))


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("case", CAUSAL, ids=_name)
def test_causal_backward(cuda_ok, case, silu):
    s = causal_case(**case)
    d = cuda(s)
    dx, g = wt.causal_backward(d["x"], d["dy"], d["w"], d["b"], silu=silu, state=d["state"], lengths=d["lengths"],
                               dstate=d["dstate"])
    want, size = causal_oracle(s, silu, True), causal_oracle(s, silu, True, mag=True)
    k, n = case["k"], case["B"] * case["T"]
    check(dx, want["dx"], size["dx"], 2 * k + 10, "dx")
    check(g["dw"], want["dw"], size["dw"], k + 10 + n / 8, "dw")
    check(g["db"], None if s["b"] is None else want["db"], size["db"], k + 10 + n / 8, "db")
    check(g["dstate"], None if s["state"] is None else want["dstate"], size["dstate"], 2 * k + 10, "dstate")


@pytest.mark.parametrize("io,B,C,k", [("f32", 1, 8, 4), ("bf16", 5, 36, 4), ("bf16", 3, 7, 3), ("f32", 2, 130, 8), ("f32", 2, 4, 1)])
def test_causal_step_equals_the_prompt(cuda_ok, io, B, C, k):
    """Token by token gives the outputs and states of the whole prompt, bit for bit; rows that are not active keep theirs."""
    T = 9
    d = cuda(causal_case(B, T, C, k, io, seed=2))
    y, state = wt.causal_forward(d["x"], d["w"], d["b"], state=d["state"])
    s = d["state"].clone()
    for t in range(T):
        assert torch.equal(wt.causal_step(d["x"][:, t], s, d["w"], d["b"]), y[:, t])
    assert torch.equal(s, state)
    before = s.clone()
    active = (torch.arange(B, device="cuda") % 2).to(torch.int32)
    out = wt.causal_step(d["x"][:, 0], s, d["w"], d["b"], active=active)
    on = active.bool()
    assert not out[~on].any() and torch.equal(s[~on], before[~on])
    if k > 1:
        assert torch.equal(s[on][:, -1], d["x"][:, 0][on])


def test_causal_prompt_in_pieces(cuda_ok):
    """A prompt cut into pieces, the state handed on in place, gives the same outputs."""
    d = cuda(causal_case(2, 100, 24, 4, "bf16", seed=5))
    y, state = wt.causal_forward(d["x"], d["w"], d["b"], state=d["state"])
    s, t = d["state"].clone(), 0
    for n in (1, 2, 34, 0, 63):
        if n:
            piece, _ = wt.causal_forward(d["x"][:, t:t + n], d["w"], d["b"], state=s, state_out=s)
            assert torch.equal(piece, y[:, t:t + n])
        t += n
    assert torch.equal(s, state)


# -------------------------------------------------------------------- scan
# tiles are 16 tokens, blocks 32 channels
SCAN = [
    dict(B=1, T=1, C=8, N=4, io="f32"),
    dict(B=2, T=3, C=33, N=16, io="bf16"),                              # one channel in the second block
    dict(B=3, T=17, C=64, N=16, io="f32", ragged=True),
    dict(B=4, T=48, C=30, N=13, io="bf16", ragged=True, G=2),            # two groups of 15 channels, odd states
    dict(B=2, T=37, C=96, N=1, io="f32", G=3, state=False),
    dict(B=1, T=130, C=40, N=64, io="f32", z=False),
    dict(B=2, T=64, C=32, N=16, io="bf16", d=False, bias=False, state=False),
    dict(B=3, T=300, C=20, N=5, io="f32", ragged=True),
    dict(B=1, T=600, C=34, N=8, io="f32", slow=True),                   # states that hardly decay
    dict(B=5, T=50, C=2, N=3, io="bf16", ragged=True, G=2, z=False, d=False),
    dict(B=1, T=1100, C=16, N=16, io="bf16"),
]


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("case", SCAN, ids=_name)
def test_scan_forward(cuda_ok, case, softplus):
    s = _scan_inputs(case, softplus)
    d = cuda(s)
    y, state = wt.scan_forward(d["x"], d["dt"], d["a"], d["b"], d["c"], d["d"], d["z"], d["dt_bias"], softplus=softplus,
                               state=d["state"], lengths=d["lengths"])
    want, size = scan_oracle(s, softplus), scan_oracle(s, softplus, mag=True)
    ops = scan_ops(case["B"], case["T"], case["C"], case["N"])
    check(y, want["y"], size["y"], ops, "y")
    check(state, want["state"], size["state"], ops, "state")


def _scan_inputs(case, softplus):
    s = scan_case(**case)
    if not softplus:  # step sizes as they are: positive, and small without the bias too
        s["dt"] = (0.05 * s["dt"].abs()).to(s["dt"].dtype)
        s["dt_bias"] = None if s["dt_bias"] is None else 0.01 * s["dt_bias"].abs()
    return s


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("case", SCAN, ids=_name)
def test_scan_backward(cuda_ok, case, softplus):
    s = _scan_inputs(case, softplus)
    d = cuda(s)
    g = wt.scan_backward(d["x"], d["dt"], d["a"], d["b"], d["c"], d["dy"], d["d"], d["z"], d["dt_bias"], softplus=softplus,
                         state=d["state"], lengths=d["lengths"], dstate=d["dstate"])
    want, size = scan_oracle(s, softplus, True), scan_oracle(s, softplus, True, mag=True)
    ops = 2 * scan_ops(case["B"], case["T"], case["C"], case["N"])  # there and back
    given = dict(dd=s["d"], dz=s["z"], ddt_bias=s["dt_bias"], dstate=s["state"])
    for m in ("dx", "ddt", "da", "db", "dc", "dd", "dz", "ddt_bias", "dstate"):
        check(g[m], None if m in given and given[m] is None else want.get(m), size.get(m), ops, m)


@pytest.mark.parametrize("io,B,C,N,G", [("f32", 1, 8, 16, 1), ("bf16", 5, 36, 16, 2), ("bf16", 3, 7, 5, 1), ("f32", 2, 130, 64, 1),
                                        ("f32", 3, 6, 1, 3)])
def test_scan_step(cuda_ok, io, B, C, N, G):
    """Steps against the oracle's pass over the same tokens; rows that are not active keep their state."""
    T = 5
    s = scan_case(B, T, C, N, io, G=G, seed=4)
    d = cuda(s)
    state = d["state"].clone()
    ys = [wt.scan_step(d["x"][:, t], d["dt"][:, t], state, d["a"], d["b"][:, t], d["c"][:, t], d["d"], d["z"][:, t], d["dt_bias"])
          for t in range(T)]
    want, size = scan_oracle(s), scan_oracle(s, mag=True)
    ops = scan_ops(B, T, C, N)
    check(torch.stack(ys, 1), want["y"], size["y"], ops, "y")
    check(state, want["state"], size["state"], ops, "state")
    before = state.clone()
    active = (torch.arange(B, device="cuda") % 2).to(torch.int32)
    out = wt.scan_step(d["x"][:, 0], d["dt"][:, 0], state, d["a"], d["b"][:, 0], d["c"][:, 0], d["d"], d["z"][:, 0], d["dt_bias"],
                       active=active)
    off = ~active.bool()
    assert not out[off].any() and torch.equal(state[off], before[off])
    assert B == 1 or not torch.equal(state[~off], before[~off])


def test_scan_prompt_in_pieces(cuda_ok):
    """A prompt in pieces, the state handed on in place: the pieces' last state is the prompt's, and so are the outputs."""
    s = scan_case(2, 150, 40, 16, "f32", seed=6)
    d = cuda(s)
    st, t, ys = d["state"].clone(), 0, []
    for n in (1, 16, 50, 83):
        cut = {m: d[m][:, t:t + n] for m in ("x", "dt", "b", "c", "z")}
        y, _ = wt.scan_forward(cut["x"], cut["dt"], d["a"], cut["b"], cut["c"], d["d"], cut["z"], d["dt_bias"], state=st, state_out=st)
        ys.append(y)
        t += n
    want, size = scan_oracle(s), scan_oracle(s, mag=True)
    check(torch.cat(ys, 1), want["y"], size["y"], scan_ops(2, 150, 40, 16), "y")
    check(st, want["state"], size["state"], scan_ops(2, 150, 40, 16), "state")


# -------------------------------------------------------------------- norm
NORM = [
    dict(B=1, T=1, C=1, io="f32"),
    dict(B=2, T=3, C=7, io="bf16", res="bf16"),
    dict(B=3, T=5, C=64, io="bf16", res="f32", ragged=True),
    dict(B=1, T=4, C=2048, io="bf16", res="f32"),
    dict(B=2, T=2, C=2056, io="bf16", res="bf16"),              # one chunk a thread, one thread in the last warp
    dict(B=1, T=3, C=8200, io="f32", res="f32"),
    dict(B=1, T=2, C=16384, io="bf16", res="f32"),              # the longest row
    dict(B=1, T=2, C=16383, io="bf16", res="bf16"),             # the longest odd row
    dict(B=2, T=350, C=40, io="f32", res="bf16", ragged=True),   # many rows, one a block (more: test_seq_edges_gpu.py)
    dict(B=2, T=3, C=100, io="f32", gate=False),
    dict(B=2, T=3, C=100, io="bf16", w=False),
    dict(B=2, T=3, C=100, io="bf16", res="f32", gate=False, w=False),
    dict(B=2, T=3, C=100, io="f32", res="f32", scale=False, gate=False),
    dict(B=2, T=3, C=100, io="f32", res="f32", w_res=False, ragged=True),
]


@pytest.mark.parametrize("case", NORM, ids=_name)
def test_norm_forward(cuda_ok, case):
    s = norm_case(**case)
    d = cuda(s)
    y, res = wt.norm_forward(d["x"], d["w"], d["gate"], d["res"], d["scale"], d["w_res"], lengths=d["lengths"])
    want, size = norm_oracle(s), norm_oracle(s, mag=True)
    ops = 24 + case["C"] / 8
    check(y, want["y"], size["y"], ops, "y")
    check(res, want["res"], size["res"], ops, "res")


@pytest.mark.parametrize("case", NORM, ids=_name)
def test_norm_backward(cuda_ok, case):
    s = norm_case(**case)
    d = cuda(s)
    g = wt.norm_backward(d["x"], d["dy"], d["w"], d["gate"], d["res"], d["scale"], d["w_res"], dres=d["dres"], lengths=d["lengths"])
    want, size = norm_oracle(s, True), norm_oracle(s, True, mag=True)
    ops = 2 * (24 + case["C"] / 8) + case["B"] * case["T"] / 8
    given = dict(dgate=s["gate"], dw=s["w"], dres=s["res"], dscale=s["scale"], dw_res=s["w_res"])
    for m in ("dx", "dgate", "dw", "dres", "dscale", "dw_res"):
        check(g[m], None if m in given and given[m] is None else want.get(m), size.get(m), ops, m)


def test_norm_of_single_tokens(cuda_ok):
    """[B, C] inputs are rows of one token."""
    s = norm_case(7, 1, 96, "bf16", res="f32", seed=3)
    d = cuda(s)
    flat = {m: d[m][:, 0] for m in ("x", "gate", "res", "dy", "dres")}
    y, res = wt.norm_forward(d["x"], d["w"], d["gate"], d["res"], d["scale"], d["w_res"])
    y2, res2 = wt.norm_forward(flat["x"], d["w"], flat["gate"], flat["res"], d["scale"], d["w_res"])
    assert torch.equal(y[:, 0], y2) and torch.equal(res[:, 0], res2)


def test_norm_without_dres(cuda_ok):
    """No gradient for res_out is a zero gradient."""
    d = cuda(norm_case(2, 3, 24, "f32", res="f32"))
    args = (d["x"], d["dy"], d["w"], d["gate"], d["res"], d["scale"], d["w_res"])
    a, b = wt.norm_backward(*args), wt.norm_backward(*args, dres=torch.zeros_like(d["dres"]))
    for m in a:
        assert torch.equal(a[m], b[m]), m


# ------------------------------------------------- shared by the operators
def _calls(io, C=24, T=50, B=3, view=lambda t: t):
    """Every call with fixed inputs, as functions that give all their outputs; `view` lays out the activations."""
    a, s, n = causal_case(B, T, C, 4, io), scan_case(B, T, C, 8, io, G=2), norm_case(B, T, C, io, res="f32")
    c, s, n = cuda(a), cuda(s), cuda(n)
    lens = torch.tensor([T, 0, T // 2], dtype=torch.int32, device="cuda")
    for d in (c, s, n):
        for m in ("x", "dt", "z", "b", "c", "dy", "gate", "res", "dres"):
            if isinstance(d.get(m), torch.Tensor) and d[m].dim() >= 3:
                d[m] = view(d[m])
    flat = lambda r: [t for p in r for t in (p.values() if isinstance(p, dict) else [p]) if t is not None]
    step = lambda d, ms: {m: d[m][:, 0] for m in ms}
    st, sx = step(c, "x"), step(s, ("x", "dt", "b", "c", "z"))

    def causal_step(**k):
        held = c["state"].clone()
        return [wt.causal_step(st["x"], held, c["w"], c["b"], **k), held]

    def scan_step(**k):
        held = s["state"].clone()
        return [wt.scan_step(sx["x"], sx["dt"], held, s["a"], sx["b"], sx["c"], s["d"], sx["z"], s["dt_bias"], **k), held]
    ins = (s["x"], s["dt"], s["a"], s["b"], s["c"])
    return dict(
        causal_forward=lambda **k: flat(wt.causal_forward(c["x"], c["w"], c["b"], state=c["state"], lengths=lens, **k)),
        causal_backward=lambda **k: flat(wt.causal_backward(c["x"], c["dy"], c["w"], c["b"], state=c["state"], lengths=lens,
                                                            dstate=c["dstate"], **k)),
        causal_step=causal_step, scan_step=scan_step,
        scan_forward=lambda **k: flat(wt.scan_forward(*ins, s["d"], s["z"], s["dt_bias"], state=s["state"], lengths=lens, **k)),
        scan_backward=lambda **k: flat([wt.scan_backward(*ins, s["dy"], s["d"], s["z"], s["dt_bias"], state=s["state"], lengths=lens,
                                                         dstate=s["dstate"], **k)]),
        norm_forward=lambda **k: flat(wt.norm_forward(n["x"], n["w"], n["gate"], n["res"], n["scale"], n["w_res"], lengths=lens, **k)),
        norm_backward=lambda **k: flat([wt.norm_backward(n["x"], n["dy"], n["w"], n["gate"], n["res"], n["scale"], n["w_res"],
                                                         dres=n["dres"], lengths=lens, **k)]),
    )


OPS = ("causal_forward", "causal_backward", "causal_step", "scan_forward", "scan_backward", "scan_step", "norm_forward",
       "norm_backward")


def _half(t):
    """The values of t as the first part of wider rows."""
    wide = torch.zeros(*t.shape[:2], t[0, 0].numel() * 2 + 8, dtype=t.dtype, device=t.device)
    part = wide[..., : t[0, 0].numel()]
    part.copy_(t.flatten(2))
    return part.unflatten(-1, t.shape[2:])


def _odd(t):
    """... as rows that begin at odd addresses."""
    wide = torch.zeros(*t.shape[:2], t[0, 0].numel() + 3, dtype=t.dtype, device=t.device)
    part = wide[..., 1: 1 + t[0, 0].numel()]
    part.copy_(t.flatten(2))
    return part.unflatten(-1, t.shape[2:])


def _token_major(t):
    """... with the batch inside the tokens."""
    return t.transpose(0, 1).contiguous().transpose(0, 1)


@pytest.mark.parametrize("view", [_half, _odd, _token_major], ids=["half", "odd", "token_major"])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("op", OPS)
def test_strided_inputs_give_the_same(cuda_ok, op, io, view):
    """The layout of the inputs changes no result beyond the order of a sum."""
    want, got = _calls(io)[op](), _calls(io, view=view)[op]()
    for a, b in zip(want, got):
        tol = 2 * sc.HALF[a.dtype] + 2.0 ** -18
        assert torch.allclose(a.double(), b.double(), rtol=tol, atol=tol * float(a.double().abs().max() + 1e-30))


def test_strided_outputs(cuda_ok):
    """Outputs go into halves of wider rows and leave the rest of them alone."""
    d = cuda(causal_case(2, 40, 16, 4, "bf16"))
    want, _ = wt.causal_forward(d["x"], d["w"], d["b"])
    wide = torch.full((2, 40, 48), 7.0, dtype=torch.bfloat16, device="cuda")
    wt.causal_forward(d["x"], d["w"], d["b"], y=wide[..., 16:32])
    assert torch.equal(wide[..., 16:32], want) and (wide[..., :16] == 7).all() and (wide[..., 32:] == 7).all()
    s = cuda(scan_case(2, 40, 16, 8, "f32"))
    args = (s["x"], s["dt"], s["a"], s["b"], s["c"], s["dy"], s["d"], s["z"], s["dt_bias"])
    g = wt.scan_backward(*args)
    wide = torch.full((2, 40, 80), 7.0, device="cuda")  # ddt, db and dc as one projection's output gradient
    h = dict(dx=torch.empty_like(g["dx"]), ddt=wide[..., :16], da=torch.empty_like(g["da"]), db=wide[..., 16:24].unflatten(-1, (1, 8)),
             dc=wide[..., 24:32].unflatten(-1, (1, 8)), dd=torch.empty_like(g["dd"]), dz=wide[..., 64:], ddt_bias=torch.empty_like(g["dd"]),
             dstate=None)
    wt.scan_backward(*args, grads=h)
    for m in ("dx", "ddt", "da", "db", "dc", "dd", "dz", "ddt_bias"):
        assert torch.equal(g[m], h[m]), m
    assert (wide[..., 32:64] == 7).all()


@pytest.mark.parametrize("op", OPS)
def test_repeats_streams_and_graphs(cuda_ok, op):
    """The same bits again, on another stream, and from a captured graph that is replayed."""
    call = _calls("bf16", C=72, T=130)[op]
    want = call()
    for a, b in zip(want, call()):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=side)
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    for t in held:
        t.fill_(9)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, held):
        assert torch.equal(a, b)


def test_two_captured_graphs_with_one_workspace(cuda_ok):
    """A workspace carries nothing from call to call: two graphs may share one, replayed in turn on one stream."""
    cases = [cuda(scan_case(2, 70, 48, 8, "f32", seed=i)) for i in range(2)]
    call = lambda s, ws: wt.scan_backward(s["x"], s["dt"], s["a"], s["b"], s["c"], s["dy"], s["d"], s["z"], s["dt_bias"], ws=ws)
    want = [call(s, None) for s in cases]
    from depthwise_convolution_wtconv_b200 import _seq
    ws = torch.empty(wt.load_seq().wtconv_scan_workspace_size(_seq.ScanDesc(2, 70, 48, 8, 1, 0, 1), 1), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in cases:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(call(s, ws))
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        for m in w:
            assert w[m] is None and o[m] is None or torch.equal(w[m], o[m]), m


def test_binding_refusals(cuda_ok):
    x, w = torch.zeros(2, 4, 8, device="cuda"), torch.zeros(8, 4, device="cuda")
    with pytest.raises(TypeError):
        wt.causal_forward(x.half(), w)
    with pytest.raises(ValueError, match="shape"):
        wt.causal_forward(x, w[:4])
    with pytest.raises(ValueError, match="contiguous"):
        wt.causal_forward(x.transpose(1, 2).contiguous().transpose(1, 2), w)
    with pytest.raises(TypeError, match="lengths"):
        wt.causal_forward(x, w, lengths=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="state"):
        wt.causal_forward(x, w, state=torch.zeros(2, 4, 8, device="cuda"))
    with pytest.raises(wt.WTConvError, match="ARG"):
        wt.causal_forward(x, w, y=x[:, :1].expand(2, 4, 8).detach())
    with pytest.raises(wt.WTConvError, match="UNSUPPORTED"):
        wt.causal_forward(x, torch.zeros(8, 9, device="cuda"))
    b = torch.zeros(2, 4, 16, device="cuda")
    a = torch.zeros(8, 16, device="cuda")
    with pytest.raises(ValueError, match="c must have shape"):
        wt.scan_forward(x, x, a, b, b[..., :8])
    with pytest.raises(wt.WTConvError, match="ARG"):
        wt.scan_forward(x, x, a, b.view(2, 4, 1, 16).expand(2, 4, 3, 16).contiguous(), b.view(2, 4, 1, 16).expand(2, 4, 3, 16).contiguous())
    with pytest.raises(wt.WTConvError, match="WORKSPACE"):
        wt.scan_backward(x, x, a, b, b, x, ws=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(wt.WTConvError, match="ARG"):
        wt.norm_forward(x)
    with pytest.raises(wt.WTConvError, match="ARG"):
        wt.norm_backward(x, None, torch.ones(8, device="cuda"))


@pytest.mark.parametrize("T", [16, 129, 2000])
def test_scan_state_updated_in_place(cuda_ok, T):
    """The state after the pass may take the place of the one before it, also where rows are cut into chunks."""
    d = cuda(scan_case(2, T, 64, 16, "bf16", seed=8))
    args = (d["x"], d["dt"], d["a"], d["b"], d["c"], d["d"], d["z"], d["dt_bias"])
    lengths = torch.tensor([T, T // 3], dtype=torch.int32, device="cuda")
    y, state = wt.scan_forward(*args, state=d["state"], lengths=lengths)
    for _ in range(5):
        s = d["state"].clone()
        y2, _ = wt.scan_forward(*args, state=s, state_out=s, lengths=lengths)
        assert torch.equal(y, y2) and torch.equal(s, state)


# -------------------------------------------------------- a block of all three
def _block(g, C, E, N, R):
    """Parameters of a gated state space block of C channels, E inside, on the CPU."""
    r = lambda *s: torch.randn(*s, generator=g)
    step = torch.exp(torch.rand(E, generator=g) * 4.6 - 6.9)
    return dict(w_in=r(2 * E, C) / C ** 0.5, conv=r(E, 4) / 2, conv_b=0.1 * r(E), w_x=r(R + 2 * N, E) / E ** 0.5,
                w_dt=r(E, R) / R ** 0.5, dt_bias=step + torch.log(-torch.expm1(-step)),
                a=-torch.arange(1, N + 1, dtype=torch.float32).repeat(E, 1), d=1 + 0.1 * r(E), w=1 + 0.1 * r(E),
                w_out=r(C, E) / E ** 0.5, scale=0.5 + 0.1 * r(C), w_res=1 + 0.1 * r(C))


def _split(p, proj, N, R):
    return proj[..., :R] @ p["w_dt"].t(), proj[..., R: R + N], proj[..., R + N:]


def _prompt(p, u, res, N, R, lengths=None, states=(None, None)):
    """The block over a prompt: its outputs and every tensor its gradients need."""
    E = p["d"].shape[0]
    xz = u @ p["w_in"].t()
    x, z = xz[..., :E], xz[..., E:]
    xc, s1 = wt.causal_forward(x, p["conv"], p["conv_b"], state=states[0], lengths=lengths)
    dt, b, c = _split(p, xc @ p["w_x"].t(), N, R)
    y, s2 = wt.scan_forward(xc, dt, p["a"], b, c, p["d"], None, p["dt_bias"], state=states[1], lengths=lengths)
    v, _ = wt.norm_forward(y, p["w"], gate=z, lengths=lengths)
    o = v @ p["w_out"].t()
    out, res2 = wt.norm_forward(o, None, res=res, scale=p["scale"], w_res=p["w_res"], lengths=lengths)
    return out, res2, (s1, s2), (x, z, xc, dt, b, c, y, v, o)


def _reference_block(p, u, res, N, R):
    """The same block in float64 torch, token by token, differentiable."""
    E = p["d"].shape[0]
    xz = u @ p["w_in"].t()
    x, z = xz[..., :E], xz[..., E:]
    pad = torch.nn.functional.pad(x, (0, 0, 3, 0))
    xc = torch.nn.functional.silu((pad.unfold(1, 4, 1) * p["conv"]).sum(-1) + p["conv_b"])
    dt, b, c = _split(p, xc @ p["w_x"].t(), N, R)
    step = torch.nn.functional.softplus(dt + p["dt_bias"])
    h, ys = torch.zeros(u.shape[0], E, N, dtype=u.dtype), []
    for t in range(u.shape[1]):
        h = torch.exp(step[:, t, :, None] * p["a"]) * h + (step[:, t] * xc[:, t])[..., None] * b[:, t, None]
        ys.append((h * c[:, t, None]).sum(-1) + p["d"] * xc[:, t])
    g = torch.stack(ys, 1) * torch.nn.functional.silu(z)
    v = g * torch.rsqrt(g.square().mean(-1, keepdim=True) + 1e-6) * p["w"]
    r = res + p["scale"] * (v @ p["w_out"].t())
    return r * torch.rsqrt(r.square().mean(-1, keepdim=True) + 1e-6) * p["w_res"], r


def test_block_for_training(cuda_ok):
    """norm, convolution, scan and gate together in fp32: outputs and the gradients of the inputs and of every parameter
    against float64 differentiation.  Tolerance 2e-4 of each tensor's norm: about 3 T + E + C = 300 operations of 2^-21 in
    a row, each at most its share of the norm."""
    torch.backends.cuda.matmul.allow_tf32 = False
    B, T, C, E, N, R = 2, 40, 48, 96, 16, 6
    g = torch.Generator().manual_seed(11)
    p = _block(g, C, E, N, R)
    u, res = torch.randn(B, T, C, generator=g), torch.randn(B, T, C, generator=g)
    dout, dres = torch.randn(B, T, C, generator=g), torch.randn(B, T, C, generator=g)
    q = {k: v.double().requires_grad_() for k, v in p.items()}
    u64, r64 = u.double().requires_grad_(), res.double().requires_grad_()
    want, want_res = _reference_block(q, u64, r64, N, R)
    ((want * dout).sum() + (want_res * dres).sum()).backward()

    P = {k: v.cuda() for k, v in p.items()}
    ud, rd = u.cuda(), res.cuda()
    out, res2, _, (x, z, xc, dt, b, c, y, v, o) = _prompt(P, ud, rd, N, R)
    got = {}
    n2 = wt.norm_backward(o, dout.cuda(), res=rd, scale=P["scale"], w_res=P["w_res"], dres=dres.cuda())
    got.update(scale=n2["dscale"], w_res=n2["dw_res"], res=n2["dres"])
    do = n2["dx"]
    got["w_out"] = torch.einsum("btc,bte->ce", do, v)
    n1 = wt.norm_backward(y, do @ P["w_out"], P["w"], gate=z)
    got["w"] = n1["dw"]
    s = wt.scan_backward(xc, dt, P["a"], b, c, n1["dx"], P["d"], None, P["dt_bias"])
    got.update(a=s["da"], d=s["dd"], dt_bias=s["ddt_bias"])
    proj = xc @ P["w_x"].t()
    dproj = torch.cat([s["ddt"] @ P["w_dt"], s["db"], s["dc"]], -1)
    got["w_dt"] = torch.einsum("bte,btr->er", s["ddt"], proj[..., :R])
    got["w_x"] = torch.einsum("btr,bte->re", dproj, xc)
    dx, gc = wt.causal_backward(x, s["dx"] + dproj @ P["w_x"], P["conv"], P["conv_b"])
    got.update(conv=gc["dw"], conv_b=gc["db"])
    dxz = torch.cat([dx, n1["dgate"]], -1)
    got["w_in"] = torch.einsum("bte,btc->ec", dxz, ud)
    got["u"] = dxz @ P["w_in"]
    ref = {**{k: t.grad for k, t in q.items()}, "u": u64.grad, "res": r64.grad}
    pairs = [("out", out, want), ("res", res2, want_res)] + [("d" + k, got[k], ref[k]) for k in ref]
    for name, a, w in pairs:
        err = (a.double().cpu() - w.detach()).norm() / w.detach().norm()
        assert err < 2e-4, (name, float(err))


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_block_for_serving(cuda_ok, io):
    """A padded batch of prompts, then single tokens from the states it left, in a captured graph that is replayed: the same
    as one longer prompt.  bf16: each of the five activations behind an output is rounded by 2^-8, 2^-5 in all."""
    torch.backends.cuda.matmul.allow_tf32 = False
    B, T, more, C, E, N, R = 3, 33, 6, 32, 64, 16, 4
    g = torch.Generator().manual_seed(12)
    dt_ = sc.DT[io]
    P = {k: v.cuda() if k in ("conv", "conv_b", "dt_bias", "a", "d", "w", "scale", "w_res") else v.to(dt_).cuda()
         for k, v in _block(g, C, E, N, R).items()}
    n = [33, 1, 20]
    lengths = torch.tensor(n, dtype=torch.int32, device="cuda")
    u, res = (torch.randn(B, T + more, C, generator=g).to(dt_).cuda() for _ in range(2))
    # row i of the batch: its first n[i] tokens as the prompt (NaN behind), the next ones singly
    pu, pr = u[:, :T].clone(), res[:, :T].clone()
    for i, k in enumerate(n):
        pu[i, k:], pr[i, k:] = float("nan"), float("nan")
    _, _, (s1, s2), _ = _prompt(P, pu, pr, N, R, lengths)
    tok_u, tok_r = torch.empty(B, C, dtype=dt_, device="cuda"), torch.empty(B, C, dtype=dt_, device="cuda")

    def token():
        xz = tok_u @ P["w_in"].t()
        xc = wt.causal_step(xz[:, :E], s1, P["conv"], P["conv_b"])
        dt, b, c = _split(P, xc @ P["w_x"].t(), N, R)
        y = wt.scan_step(xc, dt, s2, P["a"], b, c, P["d"], None, P["dt_bias"])
        v, _ = wt.norm_forward(y, P["w"], gate=xz[:, E:])
        return wt.norm_forward(v @ P["w_out"].t(), None, res=tok_r, scale=P["scale"], w_res=P["w_res"])
    tok_u.zero_(), tok_r.zero_()
    keep = s1.clone(), s2.clone()
    token()  # the library's first use, and the matrix products', outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, res2 = token()
    s1.copy_(keep[0]), s2.copy_(keep[1])
    got = []
    for j in range(more):
        tok_u.copy_(torch.stack([u[i, n[i] + j] for i in range(B)]))
        tok_r.copy_(torch.stack([res[i, n[i] + j] for i in range(B)]))
        graph.replay()
        got.append((out.clone(), res2.clone()))
    whole = torch.tensor([k + more for k in n], dtype=torch.int32, device="cuda")
    want, want_res, states, _ = _prompt(P, u, res, N, R, whole)
    tol = 1e-4 if io == "f32" else 2.0 ** -5
    rel = lambda a, b: float((a.double() - b.double()).norm() / b.double().norm())
    for i in range(B):
        assert rel(torch.stack([o[i] for o, _ in got]), want[i, n[i]: n[i] + more]) < tol
        assert rel(torch.stack([r[i] for _, r in got]), want_res[i, n[i]: n[i] + more]) < tol
    assert rel(s1, states[0]) < tol and rel(s2, states[1]) < tol


def _far(t):
    """... in a batch whose rows lie so far apart that the last one begins behind 2^31 elements."""
    row = t[0].numel()
    buf = torch.empty(2 * ((1 << 30) + 8) + row, dtype=t.dtype, device=t.device)
    far = buf.as_strided((3, *t.shape[1:]), ((1 << 30) + 8, *t.stride()[1:]))
    far.copy_(t)
    return far


@pytest.mark.parametrize("op", OPS)
def test_offsets_beyond_32_bits(cuda_ok, op):
    """Inputs whose last batch row begins behind 2^31 elements give what dense ones give."""
    want, got = _calls("bf16", C=16, T=20)[op](), _calls("bf16", C=16, T=20, view=lambda t: _far(t.contiguous()))[op]()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_token_strides_beyond_32_bits_in_all(cuda_ok):
    """Tokens 2^29 elements apart: the fifth begins at 2^31."""
    x = sc.normal(sc.gen(3), 1, 5, 40, dt=torch.bfloat16).cuda()
    buf = torch.empty(4 * (1 << 29) + 40, dtype=torch.bfloat16, device="cuda")
    far = buf.as_strided((1, 5, 40), (0, 1 << 29, 1))
    far.copy_(x)
    w = sc.normal(sc.gen(4), 40, 4).cuda()
    out = torch.empty_like(buf).as_strided((1, 5, 40), (0, 1 << 29, 1))
    y, _ = wt.causal_forward(x, w)
    wt.causal_forward(far, w, y=out)
    assert torch.equal(y, out)
    a, bc = -torch.ones(40, 8, device="cuda"), sc.normal(sc.gen(5), 1, 5, 8, dt=torch.bfloat16).cuda()
    y, _ = wt.scan_forward(x, x, a, bc, bc)
    wt.scan_forward(far, far, a, bc, bc, y=out)
    assert torch.equal(y, out)
    ones = torch.ones(40, device="cuda")
    y, _ = wt.norm_forward(x, ones)
    wt.norm_forward(far, ones, y=out)
    assert torch.equal(y, out)


@pytest.mark.parametrize("T", [300, 2500])
@pytest.mark.parametrize("C,G,N,io", [(30, 2, 13, "bf16"), (64, 1, 16, "f32"), (33, 1, 4, "bf16")])
def test_scan_gradients_of_cut_rows(cuda_ok, T, C, G, N, io):
    """Rows cut into chunks, an empty one, a whole one and one that ends inside: the gradients of each row are those of the
    row on its own, in a batch large enough not to be cut."""
    B = 3
    s = scan_case(B, T, C, N, io, G=G, seed=9)
    n = torch.tensor([T, 0, T // 3 + 5], dtype=torch.int32)
    d = cuda({**s, "lengths": n})
    names = ("x", "dt", "b", "c", "z", "dy", "state", "dstate")
    run = lambda d: wt.scan_backward(d["x"], d["dt"], d["a"], d["b"], d["c"], d["dy"], d["d"], d["z"], d["dt_bias"], state=d["state"],
                                     lengths=d["lengths"], dstate=d["dstate"])
    cut = run(d)
    many = 300  # copies of the batch: more rows than would be cut
    big = run({**d, **{m: d[m].repeat(many, *[1] * (d[m].dim() - 1)) for m in names}, "lengths": d["lengths"].repeat(many)})
    for m in ("dx", "ddt", "db", "dc", "dz", "dstate"):
        a, b = cut[m].double(), big[m][:B].double()
        tol = 2 * sc.HALF[cut[m].dtype] + 2.0 ** -14  # 2^-21 for each of the about 100 tokens that a state lasts
        assert torch.allclose(a, b, rtol=tol, atol=tol * float(b.abs().max())), m
    for m in ("da", "dd", "ddt_bias"):
        a, b = cut[m].double(), big[m].double() / many
        assert float((a - b).norm() / b.norm()) < 2.0 ** -14, m


@pytest.mark.parametrize("parts", [dict(gate=False), dict(w=False, gate=False, res="f32")], ids=["post", "pre"])
def test_norm_of_rows_between_empty_ones(cuda_ok, parts):
    """Many short rows, most of them empty, through blocks that go on from row to row with one sum over the block each."""
    B, T, C = 900, 4, 2048
    s = norm_case(B, T, C, "bf16", **parts, seed=2)
    s["lengths"] = torch.tensor([(0, 1, 0, 4, 0, 0, 2)[i % 7] for i in range(B)], dtype=torch.int32)
    d = cuda(s)
    args = (d["x"], d["w"], d["gate"], d["res"], d["scale"], d["w_res"])
    y, _ = wt.norm_forward(*args, lengths=d["lengths"])
    whole, _ = wt.norm_forward(*args)
    live = (torch.arange(T, device="cuda") < d["lengths"][:, None])[..., None]
    assert torch.equal(y, torch.where(live, whole, 0))
    g = wt.norm_backward(d["x"], d["dy"], d["w"], d["gate"], d["res"], d["scale"], d["w_res"], dres=d["dres"], lengths=d["lengths"])
    h = wt.norm_backward(d["x"], d["dy"], d["w"], d["gate"], d["res"], d["scale"], d["w_res"], dres=d["dres"])
    assert torch.equal(g["dx"], torch.where(live, h["dx"], 0))


# blocks of 1, 2, 4, 8 and 16 warps (a warp per four states, and up to four where blocks are few), tokens shared out among them
SCAN_WARPS = [
    dict(B=40, T=20, C=480, N=4, io="bf16"),                             # 600 blocks of one warp
    dict(B=20, T=21, C=480, N=7, io="f32", ragged=True),                 # 300 of two, states copied to eight
    dict(B=2, T=35, C=40, N=24, io="bf16", ragged=True),                 # eight warps, six with states
    dict(B=2, T=35, C=40, N=32, io="f32"),
    dict(B=2, T=50, C=24, N=33, io="bf16", G=3, z=False),                # sixteen, 36 states after the copy
    dict(B=1, T=4100, C=8, N=16, io="f32", ragged=False),                # as many chunks as there may be
]


@pytest.mark.parametrize("case", SCAN_WARPS, ids=_name)
def test_scan_in_blocks_of_all_sizes(cuda_ok, case):
    s = scan_case(**case, seed=21)
    d = cuda(s)
    args = (d["x"], d["dt"], d["a"], d["b"], d["c"])
    y, state = wt.scan_forward(*args, d["d"], d["z"], d["dt_bias"], state=d["state"], lengths=d["lengths"])
    g = wt.scan_backward(*args, d["dy"], d["d"], d["z"], d["dt_bias"], state=d["state"], lengths=d["lengths"], dstate=d["dstate"])
    want, size = scan_oracle(s, grads=True), scan_oracle(s, grads=True, mag=True)
    ops = scan_ops(case["B"], min(case["T"], 600), case["C"], case["N"]) + case["T"] / 8  # a state outlasts 600 tokens by less than that
    check(y, want["y"], size["y"], ops, "y")
    check(state, want["state"], size["state"], ops, "state")
    for m in ("dx", "ddt", "da", "db", "dc", "dd", "dz", "ddt_bias", "dstate"):
        check(g[m], None if m == "dz" and s["z"] is None else want[m], size[m], 2 * ops, m)


@pytest.mark.parametrize("N", [4, 8, 24, 64])
def test_scan_step_of_many_rows(cuda_ok, N):
    """More rows than blocks along them, some switched off: the same as one token of the forward pass."""
    s = scan_case(500, 1, 100, N, "bf16", seed=22)
    d = cuda(s)
    active = (torch.arange(500, device="cuda") % 3 != 0).to(torch.int32)
    want, after = wt.scan_forward(d["x"], d["dt"], d["a"], d["b"], d["c"], d["d"], d["z"], d["dt_bias"], state=d["state"],
                                  lengths=active)
    held = d["state"].clone()
    one = lambda m: d[m][:, 0]
    y = wt.scan_step(one("x"), one("dt"), held, d["a"], one("b"), one("c"), d["d"], one("z"), d["dt_bias"], active=active)
    assert torch.allclose(y.float(), want[:, 0].float(), rtol=2.0 ** -7, atol=1e-6 * float(want.abs().max()))  # a step of bf16
    assert torch.allclose(held, after, rtol=2.0 ** -20, atol=2.0 ** -20 * float(after.abs().max()))
    off = ~active.bool()
    assert torch.equal(held[off], d["state"][off]) and not y[off].any()


@pytest.mark.parametrize("op", OPS)
def test_two_calls_at_once(cuda_ok, op):
    """The same call on two streams at the same time, each with workspaces of its own."""
    call = _calls("f32", C=96, T=400)[op]
    want = call()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [call(stream=streams[k % 2]) for k in range(6)]
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(want, g):
            assert torch.equal(a, b)
