"""Float64 oracle of the sequence operators: token by token, straight from the
definitions in include/wtconv_seq.h, with the gradients written out by hand.

Every function takes `mag`: with it, the same sums are formed over the
absolute values of their terms (inputs, factors and differences alike).  That
is the size against which the rounding errors of a 32-bit computation of the
same sums are to be measured, however much the terms cancel.
"""
import numpy as np


def sigmoid(v):
    return 0.5 * (1.0 + np.tanh(0.5 * np.asarray(v, dtype=np.float64)))


def silu(v):
    return v * sigmoid(v)


def dsilu(v, mag=False):
    s = sigmoid(v)
    return s * (1.0 + np.abs(v) * (1.0 - s)) if mag else s * (1.0 + v * (1.0 - s))


def softplus(v):
    return np.logaddexp(0.0, v)


def _lengths(n, B, T):
    return [T] * B if n is None else [max(0, min(int(v), T)) for v in n]


def _abs(mag, *arrays):
    return [a if a is None or not mag else np.abs(a) for a in arrays]


def causal(x, w, bias, state=None, lengths=None, act=True, dy=None, dstate=None, mag=False):
    """x [B,T,C], w [C,k]: dict y, state; with dy also dx, dw, db, dstate."""
    B, T, C = x.shape
    k = w.shape[1]
    n = _lengths(lengths, B, T)
    m = (lambda v: np.abs(v)) if mag else (lambda v: v)
    out = dict(y=np.zeros((B, T, C)), state=np.zeros((B, k - 1, C)))
    if dy is not None:
        out.update(dx=np.zeros((B, T, C)), dw=np.zeros((C, k)), db=np.zeros(C), dstate=np.zeros((B, k - 1, C)))
    for i in range(B):
        before = np.zeros((k - 1, C)) if state is None else state[i]
        row = np.concatenate([before, x[i, :n[i]]])
        drow = np.zeros_like(row)
        for t in range(n[i]):
            win = row[t:t + k]
            p = (win * w.T).sum(0) + (0.0 if bias is None else bias)
            size = (m(win) * m(w.T)).sum(0) + (0.0 if bias is None else m(bias))
            out["y"][i, t] = (size if mag else silu(p)) if act else (size if mag else p)
            if dy is not None:
                # the error of p reaches dy silu'(p) through silu'' (at most 1/2)
                g = m(dy[i, t]) * ((dsilu(p, mag) + (0.5 * size if mag else 0.0)) if act else 1.0)
                drow[t:t + k] += m(w.T) * g
                out["dw"] += (m(win) * g).T
                out["db"] += g
        out["state"][i] = row[n[i]:]
        if dy is not None:
            if dstate is not None:
                drow[n[i]:] += m(dstate[i])
            out["dstate"][i], out["dx"][i, :n[i]] = drow[:k - 1], drow[k - 1:]
    return out


def scan(x, dt, a, b, c, d=None, z=None, dt_bias=None, state=None, lengths=None, sp=True, dy=None, dstate=None, mag=False):
    """x, dt, z [B,T,C], a [C,N], b, c [B,T,G,N], state [B,C,N]: dict y, state;
    with dy also dx, ddt, da, db, dc, dd, dz, ddt_bias, dstate."""
    B, T, C = x.shape
    N, G = a.shape[1], b.shape[2]
    n = _lengths(lengths, B, T)
    v = dt + (0.0 if dt_bias is None else dt_bias)
    step = softplus(v) if sp else v
    slope = sigmoid(v) if sp else np.ones_like(v)
    decay_rate = a
    x, b, c, d, state, dy, dstate = _abs(mag, x, b, c, d, state, dy, dstate)
    if mag:
        step_m, a = np.abs(step), np.abs(a)
    else:
        step_m = step
    gate = np.ones_like(x) if z is None else silu(z)
    dgate = np.zeros_like(x) if z is None else dsilu(z, mag)
    gate, = _abs(mag, gate)
    out = dict(y=np.zeros((B, T, C)), state=np.zeros((B, C, N)))
    if dy is not None:
        out.update({m: np.zeros((B, T, C)) for m in ("dx", "ddt", "dz")}, da=np.zeros((C, N)), db=np.zeros((B, T, G, N)),
                   dc=np.zeros((B, T, G, N)), dd=np.zeros(C), ddt_bias=np.zeros(C), dstate=np.zeros((B, C, N)))
    skip = np.zeros(C) if d is None else d
    for i in range(B):
        h = np.zeros((C, N)) if state is None else state[i].copy()
        kept, decays, pre = [h], [], []
        for t in range(n[i]):
            bt, ct = b[i, t].repeat(C // G, 0), c[i, t].repeat(C // G, 0)
            decay = np.exp(step[i, t][:, None] * decay_rate)
            h = decay * h + (step_m[i, t] * x[i, t])[:, None] * bt
            p = (ct * h).sum(1) + skip * x[i, t]
            out["y"][i, t] = p * gate[i, t]
            kept.append(h)
            decays.append(decay)
            pre.append(p)
        out["state"][i] = h
        if dy is None:
            continue
        e = np.zeros((C, N)) if dstate is None else dstate[i].copy()
        for t in reversed(range(n[i])):
            bt, ct = b[i, t].repeat(C // G, 0), c[i, t].repeat(C // G, 0)
            dp = dy[i, t] * gate[i, t]
            out["dz"][i, t] = dy[i, t] * pre[t] * dgate[i, t]
            e = e + dp[:, None] * ct
            out["dc"][i, t] = (dp[:, None] * kept[t + 1]).reshape(G, C // G, N).sum(1)
            out["db"][i, t] = (e * (step_m[i, t] * x[i, t])[:, None]).reshape(G, C // G, N).sum(1)
            ek = e * decays[t] * kept[t]
            out["da"] += ek * step_m[i, t][:, None]
            eb = (e * bt).sum(1)
            dv = ((ek * a).sum(1) + x[i, t] * eb) * slope[i, t]
            out["ddt"][i, t] = dv
            out["ddt_bias"] += dv
            out["dd"] += dp * x[i, t]
            out["dx"][i, t] = skip * dp + step_m[i, t] * eb
            e = decays[t] * e
        out["dstate"][i] = e
    return out


def norm(x, w=None, gate=None, res=None, scale=None, w_res=None, eps=1e-6, lengths=None, dy=None, dres=None, mag=False):
    """x, gate, res [B,T,C]: dict y, res; with dy or dres also the gradients
    dx, dgate, dw, dres, dscale, dw_res."""
    B, T, C = x.shape
    live = np.arange(T)[None, :, None] < np.array(_lengths(lengths, B, T))[:, None, None]
    keep = lambda v: None if v is None else np.where(live, v, 0.0)
    x, gate, res, dy, dres = keep(x), keep(gate), keep(res), keep(dy), keep(dres)
    one = np.ones(C)
    s, w_, wr = (one if v is None else v for v in (scale, w, w_res))
    act = 1.0 if gate is None else silu(gate)
    inv = lambda q: 1.0 / np.sqrt((q * q).mean(-1, keepdims=True) + eps)
    u = x * act
    n1 = np.ones((B, T, 1)) if w is None else inv(u)
    v = u * n1 * w_
    r = None if res is None else res + s * v
    n2 = None if res is None else inv(r)
    if mag:  # the same sums over absolute values, under the true norms
        x, res, dy, dres, s, w_, wr, act = _abs(mag, x, res, dy, dres, s, w_, wr, act)
        u, v = np.abs(u), np.abs(v)
        r = None if res is None else res + s * v
    out = dict(y=v if res is None else (None if w_res is None else r * n2 * wr), res=r)
    if dy is None and dres is None:
        return out
    minus = 1.0 if mag else -1.0
    if res is not None:
        g = np.zeros_like(r) if dres is None else dres
        out["dw_res"] = None
        if w_res is not None:
            t = dy * wr
            g = g + n2 * t + minus * r * n2 ** 3 * (r * t).mean(-1, keepdims=True)
            out["dw_res"] = (dy * r * n2).sum((0, 1))
        g = np.where(live, g, 0.0)
        out["dres"], out["dscale"] = g, (g * v).sum((0, 1))
        q = g * s
    else:
        q = dy
    out["dw"] = None
    if w is not None:
        out["dw"] = (q * u * n1).sum((0, 1))
        t = q * w_
        q = n1 * t + minus * u * n1 ** 3 * (u * t).mean(-1, keepdims=True)
    out["dgate"] = None if gate is None else np.where(live, q * x * dsilu(gate, mag), 0.0)
    out["dx"] = np.where(live, q * act, 0.0)
    return out
