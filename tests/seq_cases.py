"""Inputs of the sequence operators' tests and the comparison with the float64
oracle."""
import numpy as np
import torch

from oracle import seq_oracle as so

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
# half a step of the output's type, relative to the value
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
# one 32-bit operation, the approximate exponential and quotient among them,
# is off by less than this, relative to the size of its terms
UNIT = 2.0 ** -21


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, dt=torch.float32):
    return torch.randn(*shape, generator=g).to(dt)


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def cuda(d):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in d.items()}


def check(got, want, size, ops, what):
    """|got - want| <= rounding of the output + ops * UNIT * size, elementwise.
    `ops`: operations in the longest chain behind a value; `size`: the oracle's
    sums over absolute values."""
    if want is None:
        assert got is None, what
        return
    assert got is not None, what
    assert tuple(got.shape) == want.shape, (what, got.shape, want.shape)
    half = HALF[got.dtype]
    got = np64(got)
    assert np.isfinite(got).all(), what
    bound = half * np.abs(want) + ops * UNIT * size + 1e-37
    bad = np.abs(got - want) > bound
    if bad.any():
        i = np.unravel_index(np.argmax(np.abs(got - want) / bound), want.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {want.size} off, worst at {i}: {got[i]} for {want[i]} (bound {bound[i]:.3g})")


def lengths_of(kind, B, T, g):
    """None, or lengths with an empty row, a row of one token and a whole row."""
    if kind is None:
        return None
    n = torch.randint(0, T + 1, (B,), generator=g, dtype=torch.int32)
    n[0] = 0
    if B > 1:
        n[1] = T
    if B > 2:
        n[2] = 1
    return n


def poison(t, lengths):
    """NaN in the tokens behind the lengths (they must not be used)."""
    if t is None or lengths is None:
        return t
    t = t.clone()
    for i, n in enumerate(lengths.tolist()):
        t[i, n:] = float("nan")
    return t


def clean(t, lengths):
    return None if t is None else torch.nan_to_num(t, nan=0.0) if lengths is not None else t


# ------------------------------------------------------------------ causal
def causal_case(B, T, C, k, io, state=True, ragged=False, bias=True, seed=0):
    g = gen(seed)
    dt = DT[io]
    n = lengths_of("x" if ragged else None, B, T, g)
    return dict(x=poison(normal(g, B, T, C, dt=dt), n), w=normal(g, C, k) / k ** 0.5, b=normal(g, C) * 0.3 if bias else None,
                state=normal(g, B, k - 1, C, dt=dt) if state else None, lengths=n, dy=poison(normal(g, B, T, C, dt=dt), n),
                dstate=normal(g, B, k - 1, C, dt=dt) if state else None)


def causal_oracle(s, silu=True, grads=False, mag=False):
    n = s["lengths"]
    more = dict(dy=np64(clean(s["dy"], n)), dstate=np64(s["dstate"])) if grads else {}
    return so.causal(np64(clean(s["x"], n)), np64(s["w"]), np64(s["b"]), np64(s["state"]), None if n is None else n.tolist(),
                     silu, mag=mag, **more)


# -------------------------------------------------------------------- scan
def scan_case(B, T, C, N, io, G=1, state=True, ragged=False, z=True, d=True, bias=True, seed=0, slow=False):
    g = gen(seed)
    dt = DT[io]
    n = lengths_of("x" if ragged else None, B, T, g)
    a = -torch.arange(1, N + 1, dtype=torch.float32) * torch.exp(0.2 * normal(g, C, N))
    step = torch.exp(torch.rand(C, generator=g) * np.log(100.0) + np.log(1e-4 if slow else 1e-2))
    dt_bias = step + torch.log(-torch.expm1(-step))
    return dict(x=poison(normal(g, B, T, C, dt=dt), n), dt=poison((0.5 * normal(g, B, T, C)).to(dt), n), a=a,
                b=poison(normal(g, B, T, G, N, dt=dt), n), c=poison(normal(g, B, T, G, N, dt=dt), n),
                d=normal(g, C) if d else None, z=poison(normal(g, B, T, C, dt=dt), n) if z else None,
                dt_bias=dt_bias if bias else None, state=normal(g, B, C, N) if state else None, lengths=n,
                dy=poison(normal(g, B, T, C, dt=dt), n), dstate=normal(g, B, C, N) if state else None)


def scan_oracle(s, softplus=True, grads=False, mag=False):
    n = s["lengths"]
    c = lambda m: np64(clean(s[m], n))
    more = dict(dy=c("dy"), dstate=np64(s["dstate"])) if grads else {}
    return so.scan(c("x"), c("dt"), np64(s["a"]), c("b"), c("c"), np64(s["d"]), c("z"), np64(s["dt_bias"]), np64(s["state"]),
                   None if n is None else n.tolist(), softplus, mag=mag, **more)


def scan_ops(B, T, C, N):
    """Steps of the recurrence, then sums over states, tokens and channels."""
    return 24 + 2 * T + N + (B * T + C) / 8


# -------------------------------------------------------------------- norm
def norm_case(B, T, C, io, res=None, w=True, gate=True, scale=True, w_res=True, ragged=False, seed=0):
    g = gen(seed)
    dt, rt = DT[io], DT[res or io]
    n = lengths_of("x" if ragged else None, B, T, g)
    p = lambda t: poison(t, n)
    return dict(x=p(normal(g, B, T, C, dt=dt)), w=1 + 0.2 * normal(g, C) if w else None,
                gate=p(normal(g, B, T, C, dt=dt)) if gate else None, res=p((3 * normal(g, B, T, C)).to(rt)) if res else None,
                scale=1 + 0.2 * normal(g, C) if scale and res else None, w_res=1 + 0.2 * normal(g, C) if w_res and res else None,
                lengths=n, dy=p(normal(g, B, T, C, dt=dt)) if not res or w_res else None,
                dres=p(normal(g, B, T, C).to(rt)) if res else None)


def norm_oracle(s, grads=False, mag=False, eps=1e-6):
    n = s["lengths"]
    c = lambda m: np64(clean(s[m], n))
    more = dict(dy=c("dy"), dres=c("dres")) if grads else {}
    return so.norm(c("x"), np64(s["w"]), c("gate"), c("res"), np64(s["scale"]), np64(s["w_res"]), eps,
                   None if n is None else n.tolist(), mag=mag, **more)
