"""The sequence operators on the GPU at the edges of their layouts, sizes and
variants, against the float64 oracle (tests/seq_cases.py) or against the same
call on plain inputs."""
import pytest
import torch

import depthwise_convolution_wtconv_b200 as wt
import seq_cases as sc
from depthwise_convolution_wtconv_b200 import _seq
from seq_cases import check, cuda, scan_case, scan_ops, scan_oracle

pytestmark = pytest.mark.gpu


# ------------------------------------------------- rows of one token
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,C,N", [(1, 64, 16), (3, 40, 12)])
def test_scan_of_one_token_of_rows_at_odd_strides(cuda_ok, io, B, C, N):
    """One token of longer rows whose token stride is no multiple of an access: the stride of a single token does not matter."""
    s = scan_case(B, 1, C, N, io, seed=31)
    d = cuda(s)

    def slices(t):
        n, w = t[0, 0].numel(), t[0, 0].numel() + 1  # rows of an odd width, three to a batch row of an aligned one
        buf = torch.zeros(B, (3 * w + 15) // 16 * 16, dtype=t.dtype, device="cuda")
        part = buf.as_strided((B, 1, n), (buf.shape[1], w, 1))
        part.copy_(t.flatten(2))
        return part.unflatten(-1, t.shape[2:])
    o = {**d, **{m: slices(d[m]) for m in ("x", "dt", "b", "c", "z", "dy")}}
    outs = []
    for q in (d, o):
        args = (q["x"], q["dt"], q["a"], q["b"], q["c"])
        y, state = wt.scan_forward(*args, q["d"], q["z"], q["dt_bias"], state=q["state"])
        g = wt.scan_backward(*args, q["dy"], q["d"], q["z"], q["dt_bias"], state=q["state"], dstate=q["dstate"])
        outs.append(dict(g, y=y, state=state))
    for m in outs[0]:
        assert torch.equal(outs[0][m], outs[1][m]), m


# ------------------------------------------- calls from two host threads
def test_scans_of_different_states_from_two_host_threads(cuda_ok):
    """Four and sixteen states run in the same kernels with shared memory of different sizes; calls from two host threads
    at once must not take it from one another.  Entries called as the binding calls them, with arguments made ready, so
    that the threads are inside the library at the same time (the interpreter's lock is not held there)."""
    import threading
    B, T, C = 1, 4, 32
    entry, rows, f32 = _seq._entry("wtconv_scan_forward"), lambda t: _seq._rows(t, "", t.shape, t.dtype, 0), torch.float32
    calls, kept = [], []
    for N in (4, 16):
        d = cuda(scan_case(B, T, C, N, "f32", seed=32))
        y, st = torch.zeros(B, T, C, device="cuda"), torch.cuda.Stream()
        b, c = d["b"][:, :, 0], d["c"][:, :, 0]
        calls.append((_seq._pack_scan(B, T, C, N, 1, 0, 1), rows(d["x"]), rows(d["dt"]), d["a"].data_ptr(), rows(b), rows(c), None,
                      None, None, None, None, rows(y), None, None, 0, st.cuda_stream))
        kept.append((d, y, st, wt.scan_forward(d["x"], d["dt"], d["a"], d["b"], d["c"])[0]))
    torch.cuda.synchronize()
    answers = [set(), set()]
    start = threading.Barrier(2)

    def run(i):
        start.wait()
        for _ in range(40000):
            answers[i].add(entry(*calls[i]))
    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert answers == [{0}, {0}]
    for _, y, _, want in kept:
        assert torch.equal(y, want)


# ------------------------------------- chunks over which a state grows
def _growing(T, dt):
    """Rows cut into chunks (one row of 8 channels), a > 0, step sizes `dt` as they are; x and dy of one everywhere."""
    one = lambda *s: torch.ones(*s)
    return dict(x=one(1, T, 8), dt=dt.reshape(1, T, 1).repeat(1, 1, 8), a=one(8, 4), b=one(1, T, 1, 4), c=one(1, T, 1, 4), d=None, z=None,
                dt_bias=None, state=None, lengths=None, dy=one(1, T, 8), dstate=None)


def _check_scan(s, names):
    d = cuda(s)
    args = (d["x"], d["dt"], d["a"], d["b"], d["c"])
    y, state = wt.scan_forward(*args, softplus=False, state=d["state"])
    got = dict(wt.scan_backward(*args, d["dy"], softplus=False, state=d["state"], dstate=d["dstate"]), y=y, state=state)
    want, size = scan_oracle(s, False, True), scan_oracle(s, False, True, mag=True)
    for m in names:
        check(got[m], want[m], size[m], 2 * scan_ops(1, s["x"].shape[1], 8, 4), m)


def test_scan_state_of_zero_under_growth_beyond_fp32(cuda_ok):
    """Nothing goes in before the last 20 tokens and no gradient comes from behind the first 20: what stays zero over a
    chunk stays so, though the chunk's growth, exp(160), is beyond fp32."""
    s = _growing(2000, torch.full((2000,), 2.0))
    s["x"][:, :-20] = 0
    s["dy"][:, 20:] = 0
    _check_scan(s, ("y", "state", "dx", "ddt", "da", "db", "dc"))


def test_scan_growth_beyond_fp32_of_a_small_state(cuda_ok):
    """A state of 1e-30 grows by exp(100) over the first 80 tokens, and a gradient of 1e-30 by as much on its way back: both
    are ordinary numbers then.  The exponent is a sum of 80 steps, off by at most 80 roundings of 2^7, 4e-4 in all; the
    bound is 4e-3."""
    dt = torch.zeros(2000)
    dt[:80] = 1.25
    s = _growing(2000, dt)
    s["x"].zero_()
    s["state"] = torch.full((1, 8, 4), 1e-30)
    s["dy"].zero_()
    s["dy"][:, -1] = 1e-30
    _check_scan(s, ("y", "state", "dstate"))


def test_scan_decay_beyond_fp32_of_a_large_state(cuda_ok):
    """... and a state of 1e30 shrinks by exp(-100) to 4e-14."""
    dt = torch.zeros(2000)
    dt[:80] = 1.25
    s = _growing(2000, dt)
    s["a"] = -s["a"]
    s["x"].zero_()
    s["state"] = torch.full((1, 8, 4), 1e30)
    s["dy"].zero_()
    s["dy"][:, -1] = 1e30
    _check_scan(s, ("y", "state", "dstate"))


# ------------------------------------- what may share memory
def test_steps_and_norms_where_their_inputs_lie(cuda_ok):
    """Every value is read by the thread that writes there: with the same rows, outputs in place of inputs are the same."""
    s = cuda(scan_case(5, 1, 72, 16, "bf16", seed=33))
    one = {m: s[m][:, 0] for m in ("x", "dt", "b", "c", "z")}

    def scan(at=None):
        q = {m: t.clone() for m, t in one.items()}
        held = s["state"].clone()
        y = wt.scan_step(q["x"], q["dt"], held, s["a"], q["b"], q["c"], s["d"], q["z"], s["dt_bias"], y=at and q[at])
        return y, held
    want = scan()
    for m in ("x", "dt", "z"):
        got = scan(m)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), m
    c = cuda(sc.causal_case(5, 1, 72, 4, "bf16", seed=34))
    x, h1, h2 = c["x"][:, 0].clone(), c["state"].clone(), c["state"].clone()
    want = wt.causal_step(x, h1, c["w"], c["b"])
    assert torch.equal(wt.causal_step(x, h2, c["w"], c["b"], y=x), want) and torch.equal(h1, h2)
    for C in (64, 4104, 8200):  # 8, 16 and 32 values a thread
        n = cuda(sc.norm_case(3, 120, C, "f32", res="f32", ragged=True, seed=35))
        q = {m: n[m].clone() for m in ("x", "gate", "res", "dy", "dres")}
        args = lambda d: (d["x"], n["w"], d["gate"], d["res"], n["scale"], n["w_res"])
        want = wt.norm_forward(*args(n), lengths=n["lengths"])
        got = wt.norm_forward(*args(q), lengths=n["lengths"], y=q["x"], res_out=q["res"])
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        back = lambda d, g: wt.norm_backward(d["x"], d["dy"], n["w"], d["gate"], d["res"], n["scale"], n["w_res"], dres=d["dres"],
                                             lengths=n["lengths"], grads=g)
        q = {m: n[m].clone() for m in q}
        want = back(n, None)
        got = back(q, dict(want, dx=q["x"], dgate=q["gate"], dres=q["dres"], dw=want["dw"].clone(), dscale=want["dscale"].clone(),
                           dw_res=want["dw_res"].clone()))
        for m in want:
            assert torch.equal(got[m], want[m]), m


@pytest.mark.parametrize("T", [20, 1000])
def test_gradient_of_the_state_in_place_of_the_state(cuda_ok, T):
    s = cuda(scan_case(2, T, 64, 16, "f32", seed=36))
    call = lambda state, g: wt.scan_backward(s["x"], s["dt"], s["a"], s["b"], s["c"], s["dy"], s["d"], s["z"], s["dt_bias"], state=state,
                                             dstate=s["dstate"], grads=g)
    want = call(s["state"], None)
    held = s["state"].clone()
    got = call(held, {m: held if m == "dstate" else torch.empty_like(t) for m, t in want.items()})
    for m in want:
        assert torch.equal(got[m], want[m]), m
    c = cuda(sc.causal_case(2, T, 64, 4, "f32", seed=37))
    call = lambda state, g: wt.causal_backward(c["x"], c["dy"], c["w"], c["b"], state=state, dstate=c["dstate"], grads=g)
    dx, want = call(c["state"], None)
    held = c["state"].clone()
    dx2, got = call(held, {m: held if m == "dstate" else torch.empty_like(t) for m, t in want.items()})
    assert torch.equal(dx, dx2) and all(torch.equal(got[m], want[m]) for m in want)


# ------------------------------------- every variant against the oracle
# Norms: rows of 8, 16 and 32 values a thread (up to 4096, 8192 and 16384 channels), wide and odd, more rows than blocks, so
# that blocks go on from row to row and the parameters' gradients are sums over rows within a block and over blocks.
PARTS = [dict(), dict(gate=False, w=False), dict(w_res=False, scale=False)]
NORM = [dict(B=2, T=(T if rows else 1), C=C, io=io, res=None if alone else res, ragged=bool(rows and i % 2), **({} if alone else PARTS[i % 3]))
        for i, (C, T) in enumerate([(2048, 170), (2047, 170), (4097, 80), (5120, 80), (5119, 80), (8192, 80), (8201, 80), (16384, 75),
                                    (16383, 75)])
        for io, res, alone, rows in [("f32", "f32", False, True), ("bf16", "f32", False, True), ("bf16", "bf16", True, True),
                                     ("f32", "bf16", False, False), ("bf16", "bf16", False, False)]]


def _name(c):
    return "-".join(f"{k}{v}" for k, v in c.items())


@pytest.mark.parametrize("case", NORM, ids=_name)
def test_norm_of_every_width(cuda_ok, case):
    """The longest chain behind a value: 32 values a thread and the sums over the block (24 + C / 8 covers both), twice on the
    way back; for the parameters also the rows of a block and the blocks, at most B T / 8 in a row."""
    s = sc.norm_case(**case, seed=41)
    d = cuda(s)
    args = (d["w"], d["gate"], d["res"], d["scale"], d["w_res"])
    y, res = wt.norm_forward(d["x"], *args, lengths=d["lengths"])
    g = wt.norm_backward(d["x"], d["dy"], *args, dres=d["dres"], lengths=d["lengths"])
    want, size = sc.norm_oracle(s, True), sc.norm_oracle(s, True, mag=True)
    ops = 24 + case["C"] / 8
    check(y, want["y"], size["y"], ops, "y")
    check(res, want["res"], size["res"], ops, "res")
    given = dict(dgate=s["gate"], dw=s["w"], dres=s["res"], dscale=s["scale"], dw_res=s["w_res"])
    for m in ("dx", "dgate", "dw", "dres", "dscale", "dw_res"):
        check(g[m], None if m in given and given[m] is None else want.get(m), size.get(m), 2 * ops + 4 + case["B"] * case["T"] / 8, m)


def _check_causal(s, k, strip):
    d = cuda(s)
    y, state = wt.causal_forward(d["x"], d["w"], d["b"], state=d["state"], lengths=d["lengths"])
    dx, g = wt.causal_backward(d["x"], d["dy"], d["w"], d["b"], state=d["state"], lengths=d["lengths"], dstate=d["dstate"])
    want, size = sc.causal_oracle(s, grads=True), sc.causal_oracle(s, grads=True, mag=True)
    check(y, want["y"], size["y"], k + 8, "y")
    assert torch.equal(state.double().cpu(), torch.from_numpy(want["state"]))
    check(dx, want["dx"], size["dx"], 2 * k + 10, "dx")
    check(g["dstate"], want["dstate"], size["dstate"], 2 * k + 10, "dstate")
    # in a row: a strip's tokens, the 8 strips of a block, a slice of the blocks and the slices
    ops = k + 10 + strip + 8 + 32 + 32
    check(g["dw"], want["dw"], size["dw"], ops, "dw")
    check(g["db"], want["db"], size["db"], ops, "db")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("k", range(1, 9))
def test_causal_by_two_channels(cuda_ok, k, io):
    """Channel counts that are even and no multiple of four."""
    _check_causal(sc.causal_case(4, 37, 66, k, io, ragged=True, seed=42), k, 16)


@pytest.mark.parametrize("T,C,k,io", [(2433, 4096, 5, "bf16"), (2433, 4096, 7, "f32"), (2433, 4098, 3, "bf16"), (1217, 4096, 3, "f32"),
                                      (1217, 4099, 4, "bf16")])
def test_causal_in_long_strips(cuda_ok, T, C, k, io):
    """Enough threads for strips of 64 tokens (gradients 128), and of 32 (64): T one past a strip, rows that end within
    one and one past one, taps that do not divide it, states in and out."""
    s = sc.causal_case(3, T, C, k, io, seed=43)
    s["lengths"] = torch.tensor([T, T - 255, T // 3 + 1], dtype=torch.int32)
    s["x"], s["dy"] = sc.poison(s["x"], s["lengths"]), sc.poison(s["dy"], s["lengths"])
    _check_causal(s, k, 128)


@pytest.mark.parametrize("T", [16, 40, 700])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_scan_tokens_that_do_not_move_a_state(cuda_ok, T, io):
    """A step of zero leaves a state as it is, to the bit, and so do the tokens behind a length, which are steps of zero in
    the kernel: within a tile of 16 tokens, behind it, and over chunks."""
    s = scan_case(4, T, 40, 16, io, bias=False, seed=44)
    s["dt"] = (0.05 * s["dt"].abs()).to(s["dt"].dtype)
    n = torch.tensor([1, 5, 15, 0], dtype=torch.int32) + (T - 16)
    live = (torch.arange(T) < n[:, None])[..., None]
    d = cuda(dict(s, dt=torch.where(live, s["dt"], 0), dy=torch.where(live, s["dy"], 0)))
    args = lambda q: (q["x"], q["dt"], q["a"], q["b"], q["c"])
    run = lambda q, n: (wt.scan_forward(*args(q), q["d"], q["z"], softplus=False, state=q["state"], lengths=n),
                        wt.scan_backward(*args(q), q["dy"], q["d"], q["z"], softplus=False, state=q["state"], lengths=n,
                                         dstate=q["dstate"]))
    cut = {m: sc.poison(d[m], n) if m in ("x", "dt", "b", "c", "z", "dy") else d[m] for m in d}
    (y, state), g = run(d, None)
    (y2, state2), g2 = run(cut, n.cuda())
    live = live.cuda()
    assert torch.equal(state, state2) and torch.equal(torch.where(live, y, 0), y2)
    assert torch.equal(g["dstate"], g2["dstate"]) and torch.equal(torch.where(live, g["dx"], 0), g2["dx"])
    still = dict(d, dt=torch.zeros_like(d["dt"]), dy=torch.zeros_like(d["dy"]))
    (_, state), g = run(still, None)
    assert torch.equal(state, d["state"]) and torch.equal(g["dstate"], d["dstate"])
