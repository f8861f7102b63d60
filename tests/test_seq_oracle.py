"""The float64 oracle of the sequence operators: hand-computed values, and its
gradients against central differences of its own forward pass."""
import numpy as np
import pytest

from oracle import seq_oracle as so

R = np.random.default_rng(3)


def _check_grads(value, inputs, grads, names):
    """d value / d input against central differences in a few random directions
    (step 1e-5: truncation ~1e-10, rounding ~1e-11, relative)."""
    for name in names:
        for _ in range(3):
            v = R.standard_normal(inputs[name].shape)
            h = 1e-5
            up = value({**inputs, name: inputs[name] + h * v})
            down = value({**inputs, name: inputs[name] - h * v})
            want = (up - down) / (2 * h)
            got = (grads[name] * v).sum()
            assert abs(got - want) <= 1e-6 * max(1.0, abs(want)), name


def test_causal_by_hand():
    x = np.array([[[1.0], [2.0], [3.0]]])
    out = so.causal(x, np.array([[10.0, 1.0]]), np.array([0.5]), np.array([[[4.0]]]), act=False)
    assert out["y"].ravel().tolist() == [41.5, 12.5, 23.5]
    assert out["state"].ravel().tolist() == [3.0]
    cut = so.causal(x, np.array([[10.0, 1.0]]), None, np.array([[[4.0]]]), lengths=[0], act=False)
    assert cut["y"].ravel().tolist() == [0, 0, 0] and cut["state"].ravel().tolist() == [4.0]


def test_scan_by_hand():
    one = np.ones((1, 2, 1))
    out = so.scan(2 * one, one, np.array([[-np.log(2.0)]]), np.ones((1, 2, 1, 1)), 3 * np.ones((1, 2, 1, 1)), d=np.array([1.0]),
                  state=np.array([[[4.0]]]), sp=False)
    # h = 4/2 + 2 = 4, then 4/2 + 2 = 4; y = 3 h + x = 14
    assert np.allclose(out["y"].ravel(), [14, 14]) and np.allclose(out["state"], 4.0)


@pytest.mark.parametrize("act", [True, False])
@pytest.mark.parametrize("lengths", [None, [0, 3, 7]])
def test_causal_gradients(act, lengths):
    B, T, C, k = 3, 7, 2, 4
    i = dict(x=R.standard_normal((B, T, C)), w=R.standard_normal((C, k)), bias=R.standard_normal(C),
             state=R.standard_normal((B, k - 1, C)))
    dy, ds = R.standard_normal((B, T, C)), R.standard_normal((B, k - 1, C))

    def value(i):
        o = so.causal(i["x"], i["w"], i["bias"], i["state"], lengths, act)
        return (o["y"] * dy).sum() + (o["state"] * ds).sum()
    o = so.causal(i["x"], i["w"], i["bias"], i["state"], lengths, act, dy, ds)
    _check_grads(value, i, dict(x=o["dx"], w=o["dw"], bias=o["db"], state=o["dstate"]), i)


@pytest.mark.parametrize("sp", [True, False])
@pytest.mark.parametrize("lengths", [None, [0, 4, 6]])
def test_scan_gradients(sp, lengths):
    B, T, C, N, G = 3, 6, 4, 3, 2
    r = R.standard_normal
    i = dict(x=r((B, T, C)), dt=0.3 + 0.2 * r((B, T, C)), a=-np.exp(r((C, N))), b=r((B, T, G, N)), c=r((B, T, G, N)), d=r(C),
             z=r((B, T, C)), dt_bias=0.1 * r(C), state=r((B, C, N)))
    dy, ds = r((B, T, C)), r((B, C, N))

    def value(i):
        o = so.scan(**i, lengths=lengths, sp=sp)
        return (o["y"] * dy).sum() + (o["state"] * ds).sum()
    o = so.scan(**i, lengths=lengths, sp=sp, dy=dy, dstate=ds)
    _check_grads(value, i, {m: o["d" + m] if m != "dt_bias" else o["ddt_bias"] for m in i}, i)


@pytest.mark.parametrize("parts", [("gate", "w", "res", "scale", "w_res"), ("gate", "w"), ("w",), ("gate",), ("res", "w_res"),
                                   ("res", "scale"), ("w", "res")])
def test_norm_gradients(parts):
    B, T, C = 2, 3, 5
    r = R.standard_normal
    i = dict(x=r((B, T, C)), gate=r((B, T, C)), res=r((B, T, C)), w=r(C), scale=r(C), w_res=r(C))
    i = {m: v for m, v in i.items() if m == "x" or m in parts}
    dy, dr = r((B, T, C)), r((B, T, C))
    lengths = [3, 1]

    def value(i):
        o = so.norm(**i, eps=1e-3, lengths=lengths)
        return (0 if o["y"] is None else (o["y"] * dy).sum()) + (0 if o["res"] is None else (o["res"] * dr).sum())
    o = so.norm(**i, eps=1e-3, lengths=lengths, dy=dy, dres=dr if "res" in parts else None)
    _check_grads(value, i, {m: o["d" + m] for m in i}, i)


def test_sizes_bound_the_values():
    """The sums over absolute values are at least the values themselves."""
    r = R.standard_normal
    B, T, C, N = 2, 5, 3, 2
    args = (r((B, T, C)), r((B, T, C)), -np.exp(r((C, N))), r((B, T, 1, N)), r((B, T, 1, N)), r(C), r((B, T, C)))
    kw = dict(dy=r((B, T, C)), dstate=r((B, C, N)), state=r((B, C, N)))
    v, m = so.scan(*args, **kw), so.scan(*args, **kw, mag=True)
    for k in v:
        assert (np.abs(v[k]) <= m[k] * (1 + 1e-12)).all(), k
