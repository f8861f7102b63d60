"""ctypes binding of the sequence operators of libwtconv.so (argument
checks and marshalling only): the causal depthwise convolution, the selective
state space scan and the norms with gate and residual scale.

Activations are CUDA tensors [B, T, C] (fp32 or bf16) whose last dimension is
contiguous; the other strides are free.  Parameters and the scan's state are
fp32.  `lengths` (int32 [B]) gives the tokens of each row of a padded batch:
the rest is not used, and outputs and gradients there are zero.  Outputs may
be passed in; `stream` selects the stream (default: the current one of the
inputs' device), on which outputs and workspace are then allocated too.
"""
import ctypes
import struct

import torch

from ._lib import BF16, F32, _check, load

# The current stream's address and the current device's index, without the
# objects around them.  A torch built without CUDA has neither; no call gets as
# far there, since its tensors are refused before.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)

# every symbol include/wtconv_seq.h declares
EXPORTS_SEQ = ("wtconv_causal_forward", "wtconv_causal_backward", "wtconv_causal_step", "wtconv_causal_workspace_size",
               "wtconv_scan_forward", "wtconv_scan_backward", "wtconv_scan_step", "wtconv_scan_workspace_size",
               "wtconv_norm_forward", "wtconv_norm_backward", "wtconv_norm_workspace_size")

_Tensor = torch.Tensor
_TYPES = {torch.float32: F32, torch.bfloat16: BF16}
_i = ctypes.c_int


class Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_longlong), ("token_stride", ctypes.c_longlong)]


class CausalDesc(ctypes.Structure):
    _fields_ = [("B", _i), ("T", _i), ("C", _i), ("k", _i), ("io", _i), ("silu", _i)]


class ScanDesc(ctypes.Structure):
    _fields_ = [("B", _i), ("T", _i), ("C", _i), ("N", _i), ("G", _i), ("io", _i), ("softplus", _i)]


class NormDesc(ctypes.Structure):
    _fields_ = [("B", _i), ("T", _i), ("C", _i), ("io", _i), ("res", _i), ("eps", ctypes.c_float)]


_bound = None
_call = {}  # entries that take descriptors and rows as packed bytes, which are quicker to make than structures


def load_seq():
    """The library with the sequence operators' signatures set."""
    global _bound
    if _bound is not None:
        return _bound
    lib = load()
    vp, rp, sz = ctypes.c_void_p, ctypes.POINTER(Rows), ctypes.c_size_t
    cd, sd, nd = (ctypes.POINTER(d) for d in (CausalDesc, ScanDesc, NormDesc))
    args = {
        "wtconv_causal_forward": [cd, rp, vp, vp, vp, vp, rp, vp, vp],
        "wtconv_causal_backward": [cd, rp, rp, vp, vp, vp, vp, vp, rp, vp, vp, vp, vp, sz, vp],
        "wtconv_causal_step": [cd, rp, vp, vp, vp, rp, vp, vp],
        "wtconv_scan_forward": [sd, rp, rp, vp, rp, rp, vp, rp, vp, vp, vp, rp, vp, vp, sz, vp],
        "wtconv_scan_backward": [sd, rp, rp, vp, rp, rp, vp, rp, vp, vp, vp, rp, vp, rp, rp, vp, rp, rp, vp, rp, vp, vp, vp, sz, vp],
        "wtconv_scan_step": [sd, rp, rp, vp, rp, rp, vp, rp, vp, vp, rp, vp, vp],
        "wtconv_norm_forward": [nd, rp, rp, vp, rp, vp, vp, vp, rp, rp, vp],
        "wtconv_norm_backward": [nd, rp, rp, vp, rp, vp, vp, vp, rp, rp, rp, rp, vp, rp, vp, vp, vp, sz, vp],
        "wtconv_causal_workspace_size": [cd], "wtconv_scan_workspace_size": [sd, _i], "wtconv_norm_workspace_size": [nd],
    }
    for name, types in args.items():
        f = getattr(lib, name)
        f.argtypes, f.restype = types, sz if name.endswith("size") else ctypes.c_int
        _call[name] = g = lib[name]
        g.argtypes, g.restype = [t if t in (sz, _i) else vp for t in types], f.restype
    _bound = lib
    return lib


def _entry(name):
    if _bound is None:
        load_seq()
    return _call[name]


def _elsewhere(x, stream):
    """The context of a call on another stream than the current one, or on
    another device than the current one (a launch goes to the current device):
    what is allocated then belongs to that stream too."""
    if stream is None:
        return torch.cuda.device(x.device)
    if stream.device != x.device:
        raise ValueError("stream must be on the inputs' device")
    return torch.cuda.stream(stream)


def _activation(x, name):
    """The device of an activation, and the code of its type."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if x.dtype not in _TYPES:
        raise TypeError(f"{name} must be torch.float32 or torch.bfloat16")
    return x.get_device(), _TYPES[x.dtype]


def _refuse(t, name, shape, dtype, dev):
    """Says what is wrong with a tensor that is not of this shape and type on this device."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the inputs' device")
    raise ValueError(f"{name} must be contiguous")


def _dense(t, name, shape, dtype, dev):
    """The address of a contiguous tensor (None: NULL)."""
    if t is None:
        return None
    if not isinstance(t, _Tensor) or t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        _refuse(t, name, shape, dtype, dev)
    return t.data_ptr()


_pack_rows = struct.Struct("Pqq").pack


def _rows(t, name, shape, dtype, dev, inner=1):
    """A [B, T, ...] or (single token) [B, ...] tensor as the library's rows;
    `inner`: the number of last dimensions that make up a row."""
    if t is None:
        return None
    if not isinstance(t, _Tensor) or t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        _refuse(t, name, shape, dtype, dev)
    s = t.stride()
    if s[-1] != 1 and shape[-1] != 1 or inner == 2 and s[-2] != shape[-1] and shape[-2] != 1:
        raise ValueError(f"{name} must be contiguous along its last dimension" + ("s" if inner == 2 else ""))
    return _pack_rows(t.data_ptr(), s[0], s[1] if len(s) > inner + 1 else 0)


_CONTIGUOUS = torch.contiguous_format


def _like(t):
    """A new contiguous tensor of t's shape, type and device (a third of the time that torch.empty takes)."""
    return torch.empty_like(t, memory_format=_CONTIGUOUS)


def _workspace(need, ws, like):
    if ws is None:
        ws = like.new_empty(need, dtype=torch.uint8)
    elif not ws.is_cuda or not ws.is_contiguous() or ws.device != like.device:
        raise ValueError("ws must be a contiguous tensor on the inputs' device")
    return ws, ws.numel() * ws.element_size()


# ---------------------------------------------------------- causal convolution
_pack_causal = struct.Struct("6i").pack


def _causal(x, w, silu, T, io):
    """The descriptor, the taps and the shape of the state."""
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w must have shape [C, k]")
    B, C = x.shape[0], x.shape[-1]
    k = w.shape[1]
    return _pack_causal(B, T, C, k, io, bool(silu)), k, (B, k - 1, C)


def causal_forward(x, w, b=None, silu=True, state=None, lengths=None, y=None, state_out=None, stream=None):
    """Causal depthwise convolution over tokens: (y, state_out).

    y[t] = silu(b + sum_j w[:, j] x[t - (k-1) + j]); x [B, T, C], w [C, k], b [C];
    state [B, k-1, C]: the inputs before the first token (None: zeros);
    state_out: the last k-1 inputs, to go on from (may be `state` itself)."""
    dev, code = _activation(x, "x")
    if stream is not None or dev != _current_device():
        with _elsewhere(x, stream):
            return causal_forward(x, w, b, silu, state, lengths, y, state_out)
    if x.dim() != 3:
        raise ValueError("x must have shape [B, T, C]")
    desc, k, held = _causal(x, w, silu, x.shape[1], code)
    f32, io, C = torch.float32, x.dtype, x.shape[2]
    y = _like(x) if y is None else y
    if state_out is None:
        state_out = x.new_empty(held) if state is None else _like(state)
    _check(_entry("wtconv_causal_forward")(desc, _rows(x, "x", x.shape, io, dev), _dense(w, "w", (C, k), f32, dev),
                                     _dense(b, "b", (C,), f32, dev), _dense(state, "state", held, io, dev),
                                     _dense(lengths, "lengths", (x.shape[0],), torch.int32, dev), _rows(y, "y", x.shape, io, dev),
                                     _dense(state_out, "state_out", held, io, dev), _raw_stream(dev)), "wtconv_causal_forward")
    return y, state_out


def causal_backward(x, dy, w, b=None, silu=True, state=None, lengths=None, dstate=None, dx=None, grads=None, ws=None,
                    stream=None):
    """Gradients of <y, dy> + <state_out, dstate>: (dx, dict dw, db, dstate).

    grads["dstate"] is that of the state before the pass (None without one);
    grads["db"] is None without a bias."""
    dev, code = _activation(x, "x")
    if stream is not None or dev != _current_device():
        with _elsewhere(x, stream):
            return causal_backward(x, dy, w, b, silu, state, lengths, dstate, dx, grads, ws)
    if x.dim() != 3:
        raise ValueError("x must have shape [B, T, C]")
    desc, k, held = _causal(x, w, silu, x.shape[1], code)
    f32, io, C = torch.float32, x.dtype, x.shape[2]
    dx = _like(x) if dx is None else dx
    g = grads if grads is not None else dict(dw=_like(w), db=None if b is None else _like(b),
                                             dstate=None if state is None else _like(state))
    ws, nws = _workspace(_entry("wtconv_causal_workspace_size")(desc), ws, x)
    _check(_entry("wtconv_causal_backward")(desc, _rows(x, "x", x.shape, io, dev), _rows(dy, "dy", x.shape, io, dev),
                                      _dense(w, "w", (C, k), f32, dev), _dense(b, "b", (C,), f32, dev),
                                      _dense(state, "state", held, io, dev),
                                      _dense(lengths, "lengths", (x.shape[0],), torch.int32, dev),
                                      _dense(dstate, "dstate", held, io, dev), _rows(dx, "dx", x.shape, io, dev),
                                      _dense(g["dw"], "dw", (C, k), f32, dev), _dense(g["db"], "db", (C,), f32, dev),
                                      _dense(g["dstate"], "grads['dstate']", held, io, dev), ws.data_ptr(), nws, _raw_stream(dev)),
           "wtconv_causal_backward")
    return dx, g


def causal_step(x, state, w, b=None, silu=True, active=None, y=None, stream=None):
    """One token of every row, y [B, C] of x [B, C]; state [B, k-1, C] is moved
    on in place.  active (int32 [B]): 0 leaves a row's state as it is and its
    output zero."""
    dev, code = _activation(x, "x")
    if stream is not None or dev != _current_device():
        with _elsewhere(x, stream):
            return causal_step(x, state, w, b, silu, active, y)
    if x.dim() != 2:
        raise ValueError("x must have shape [B, C]")
    desc, k, held = _causal(x, w, silu, 1, code)
    f32, io, C = torch.float32, x.dtype, x.shape[1]
    y = _like(x) if y is None else y
    _check(_entry("wtconv_causal_step")(desc, _rows(x, "x", x.shape, io, dev), _dense(w, "w", (C, k), f32, dev),
                                  _dense(b, "b", (C,), f32, dev), _dense(active, "active", (x.shape[0],), torch.int32, dev),
                                  _rows(y, "y", x.shape, io, dev), _dense(state, "state", held, io, dev), _raw_stream(dev)),
           "wtconv_causal_step")
    return y


# ------------------------------------------------------------------------ scan
_pack_scan = struct.Struct("7i").pack


def _scan(x, a, b, softplus, T, io):
    """The descriptor, the states and the shape of b and c (groups may be left out)."""
    if not isinstance(a, torch.Tensor) or a.dim() != 2:
        raise ValueError("a must have shape [C, N]")
    lead = x.dim() - 1
    if not isinstance(b, torch.Tensor) or b.dim() not in (lead + 1, lead + 2):
        raise ValueError("b must have the shape of x with [N] or [G, N] in place of the channels")
    N = a.shape[1]
    G = b.shape[-2] if b.dim() == lead + 2 else 1
    inner = (G, N) if b.dim() == lead + 2 else (N,)
    return _pack_scan(x.shape[0], T, x.shape[-1], N, G, io, bool(softplus)), N, x.shape[:lead] + inner


def scan_forward(x, dt, a, b, c, d=None, z=None, dt_bias=None, softplus=True, state=None, lengths=None, y=None,
                 state_out=None, ws=None, stream=None):
    """Selective state space scan: (y, state_out).

    delta = softplus(dt + dt_bias);  h = exp(delta a) h + delta x b;
    y = (c . h + d x) silu(z).  x, dt, z [B, T, C]; a [C, N] fp32; b, c
    [B, T, N], or [B, T, G, N] for G groups of channels; d, dt_bias [C] fp32;
    state, state_out [B, C, N] fp32 (state_out may be `state` itself)."""
    dev, code = _activation(x, "x")
    if stream is not None or dev != _current_device():
        with _elsewhere(x, stream):
            return scan_forward(x, dt, a, b, c, d, z, dt_bias, softplus, state, lengths, y, state_out, ws)
    if x.dim() != 3:
        raise ValueError("x must have shape [B, T, C]")
    desc, N, bc = _scan(x, a, b, softplus, x.shape[1], code)
    f32, io, S, C, inner = torch.float32, x.dtype, x.shape, x.shape[2], len(bc) - 2
    held = (x.shape[0], C, N)
    y = _like(x) if y is None else y
    if state_out is None:
        state_out = x.new_empty(held, dtype=f32) if state is None else _like(state)
    need = _entry("wtconv_scan_workspace_size")(desc, 0)
    ws, nws = _workspace(need, ws, x) if need or ws is not None else (None, 0)
    _check(_entry("wtconv_scan_forward")(desc, _rows(x, "x", S, io, dev), _rows(dt, "dt", S, io, dev),
                                   _dense(a, "a", (C, N), f32, dev), _rows(b, "b", bc, io, dev, inner),
                                   _rows(c, "c", bc, io, dev, inner), _dense(d, "d", (C,), f32, dev),
                                   _rows(z, "z", S, io, dev), _dense(dt_bias, "dt_bias", (C,), f32, dev),
                                   _dense(state, "state", held, f32, dev),
                                   _dense(lengths, "lengths", (x.shape[0],), torch.int32, dev), _rows(y, "y", S, io, dev),
                                   _dense(state_out, "state_out", held, f32, dev), None if ws is None else ws.data_ptr(),
                                   nws, _raw_stream(dev)), "wtconv_scan_forward")
    return y, state_out


def scan_backward(x, dt, a, b, c, dy, d=None, z=None, dt_bias=None, softplus=True, state=None, lengths=None, dstate=None,
                  grads=None, ws=None, stream=None):
    """Gradients of <y, dy> + <state_out, dstate>: dict dx, ddt, da, db, dc, dd,
    dz, ddt_bias, dstate (the last for the state before the pass), None for
    inputs that are not given."""
    dev, code = _activation(x, "x")
    if stream is not None or dev != _current_device():
        with _elsewhere(x, stream):
            return scan_backward(x, dt, a, b, c, dy, d, z, dt_bias, softplus, state, lengths, dstate, grads, ws)
    if x.dim() != 3:
        raise ValueError("x must have shape [B, T, C]")
    desc, N, bc = _scan(x, a, b, softplus, x.shape[1], code)
    f32, io, S, C, inner = torch.float32, x.dtype, x.shape, x.shape[2], len(bc) - 2
    held = (x.shape[0], C, N)
    g = grads
    if g is None:
        new = lambda t: None if t is None else _like(t)
        g = dict(dx=_like(x), ddt=_like(x), da=_like(a), db=_like(b), dc=_like(b), dd=new(d), dz=new(z), ddt_bias=new(dt_bias),
                 dstate=new(state))
    ws, nws = _workspace(_entry("wtconv_scan_workspace_size")(desc, 1), ws, x)
    _check(_entry("wtconv_scan_backward")(desc, _rows(x, "x", S, io, dev), _rows(dt, "dt", S, io, dev),
                                    _dense(a, "a", (C, N), f32, dev), _rows(b, "b", bc, io, dev, inner),
                                    _rows(c, "c", bc, io, dev, inner), _dense(d, "d", (C,), f32, dev),
                                    _rows(z, "z", S, io, dev), _dense(dt_bias, "dt_bias", (C,), f32, dev),
                                    _dense(state, "state", held, f32, dev),
                                    _dense(lengths, "lengths", (x.shape[0],), torch.int32, dev),
                                    _rows(dy, "dy", S, io, dev), _dense(dstate, "dstate", held, f32, dev),
                                    _rows(g["dx"], "dx", S, io, dev), _rows(g["ddt"], "ddt", S, io, dev),
                                    _dense(g["da"], "da", (C, N), f32, dev), _rows(g["db"], "db", bc, io, dev, inner),
                                    _rows(g["dc"], "dc", bc, io, dev, inner), _dense(g["dd"], "dd", (C,), f32, dev),
                                    _rows(g["dz"], "dz", S, io, dev), _dense(g["ddt_bias"], "ddt_bias", (C,), f32, dev),
                                    _dense(g["dstate"], "grads['dstate']", held, f32, dev), ws.data_ptr(), nws, _raw_stream(dev)),
           "wtconv_scan_backward")
    return g


def scan_step(x, dt, state, a, b, c, d=None, z=None, dt_bias=None, softplus=True, active=None, y=None, stream=None):
    """One token of every row, y [B, C] of x, dt, z [B, C] and b, c [B, N] or
    [B, G, N]; state [B, C, N] fp32 is moved on in place.  active (int32 [B]):
    0 leaves a row's state as it is and its output zero."""
    dev, code = _activation(x, "x")
    if stream is not None or dev != _current_device():
        with _elsewhere(x, stream):
            return scan_step(x, dt, state, a, b, c, d, z, dt_bias, softplus, active, y)
    if x.dim() != 2:
        raise ValueError("x must have shape [B, C]")
    desc, N, bc = _scan(x, a, b, softplus, 1, code)
    f32, io, S, C, inner = torch.float32, x.dtype, x.shape, x.shape[1], len(bc) - 1
    y = _like(x) if y is None else y
    _check(_entry("wtconv_scan_step")(desc, _rows(x, "x", S, io, dev), _rows(dt, "dt", S, io, dev),
                                _dense(a, "a", (C, N), f32, dev), _rows(b, "b", bc, io, dev, inner),
                                _rows(c, "c", bc, io, dev, inner), _dense(d, "d", (C,), f32, dev), _rows(z, "z", S, io, dev),
                                _dense(dt_bias, "dt_bias", (C,), f32, dev),
                                _dense(active, "active", (x.shape[0],), torch.int32, dev), _rows(y, "y", S, io, dev),
                                _dense(state, "state", (x.shape[0], C, N), f32, dev), _raw_stream(dev)), "wtconv_scan_step")
    return y


# ------------------------------------------------------------------------ norm
_pack_norm = struct.Struct("5if").pack


def _norm(x, res, eps, io):
    """The descriptor and the residual's type."""
    if x.dim() not in (2, 3):
        raise ValueError("x must have shape [B, T, C] or [B, C]")
    res_io = io if res is None else _activation(res, "res")[1]
    T = x.shape[1] if x.dim() == 3 else 1
    rt = x.dtype if res is None else res.dtype
    return _pack_norm(x.shape[0], T, x.shape[-1], io, res_io, eps), rt


def norm_forward(x, w=None, gate=None, res=None, scale=None, w_res=None, eps=1e-6, lengths=None, y=None, res_out=None,
                 stream=None):
    """Norm after a block, gate, residual scale and norm before the next block,
    in one pass: (y, res_out).

    u = x silu(gate);  v = u w / sqrt(mean(u^2) + eps);  res_out = res + scale v;
    y = res_out w_res / sqrt(mean(res_out^2) + eps).  Each of gate, w and scale
    may be left out; without res y = v and res_out is None, without w_res y is
    None.  x, gate [B, T, C] or [B, C]; res in fp32 or bf16, whatever x is;
    w, scale, w_res [C] fp32."""
    dev, code = _activation(x, "x")
    if stream is not None or dev != _current_device():
        with _elsewhere(x, stream):
            return norm_forward(x, w, gate, res, scale, w_res, eps, lengths, y, res_out)
    desc, rt = _norm(x, res, eps, code)
    f32, io, S, V = torch.float32, x.dtype, x.shape, (x.shape[-1],)
    if y is None and (res is None or w_res is not None):
        y = _like(x)
    if res_out is None and res is not None:
        res_out = _like(res)
    _check(_entry("wtconv_norm_forward")(desc, _rows(x, "x", S, io, dev), _rows(gate, "gate", S, io, dev), _dense(w, "w", V, f32, dev),
                                   _rows(res, "res", S, rt, dev), _dense(scale, "scale", V, f32, dev),
                                   _dense(w_res, "w_res", V, f32, dev),
                                   _dense(lengths, "lengths", (x.shape[0],), torch.int32, dev), _rows(y, "y", S, io, dev),
                                   _rows(res_out, "res_out", S, rt, dev), _raw_stream(dev)), "wtconv_norm_forward")
    return y, res_out


def norm_backward(x, dy=None, w=None, gate=None, res=None, scale=None, w_res=None, dres=None, eps=1e-6, lengths=None,
                  grads=None, ws=None, stream=None):
    """Gradients of <y, dy> + <res_out, dres>: dict dx, dgate, dw, dres (of the
    residual that came in), dscale, dw_res, None for inputs that are not given.
    dy is None exactly where the forward pass gives no y; dres None is zero."""
    dev, code = _activation(x, "x")
    if stream is not None or dev != _current_device():
        with _elsewhere(x, stream):
            return norm_backward(x, dy, w, gate, res, scale, w_res, dres, eps, lengths, grads, ws)
    desc, rt = _norm(x, res, eps, code)
    f32, io, S, V = torch.float32, x.dtype, x.shape, (x.shape[-1],)
    g = grads
    if g is None:
        new = lambda t: None if t is None else _like(t)
        g = dict(dx=_like(x), dgate=new(gate), dw=new(w), dres=new(res), dscale=new(scale), dw_res=new(w_res))
    ws, nws = _workspace(_entry("wtconv_norm_workspace_size")(desc), ws, x)
    _check(_entry("wtconv_norm_backward")(desc, _rows(x, "x", S, io, dev), _rows(gate, "gate", S, io, dev),
                                    _dense(w, "w", V, f32, dev), _rows(res, "res", S, rt, dev),
                                    _dense(scale, "scale", V, f32, dev), _dense(w_res, "w_res", V, f32, dev),
                                    _dense(lengths, "lengths", (x.shape[0],), torch.int32, dev), _rows(dy, "dy", S, io, dev),
                                    _rows(dres, "dres", S, rt, dev), _rows(g["dx"], "dx", S, io, dev),
                                    _rows(g["dgate"], "dgate", S, io, dev), _dense(g["dw"], "dw", V, f32, dev),
                                    _rows(g["dres"], "dres", S, rt, dev), _dense(g["dscale"], "dscale", V, f32, dev),
                                    _dense(g["dw_res"], "dw_res", V, f32, dev), ws.data_ptr(), nws, _raw_stream(dev)),
           "wtconv_norm_backward")
    return g
