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

import torch

from ._lib import BF16, F32, _check, load

# every symbol include/wtconv_seq.h declares
EXPORTS_SEQ = ("wtconv_causal_forward", "wtconv_causal_backward", "wtconv_causal_step", "wtconv_causal_workspace_size",
               "wtconv_scan_forward", "wtconv_scan_backward", "wtconv_scan_step", "wtconv_scan_workspace_size",
               "wtconv_norm_forward", "wtconv_norm_backward", "wtconv_norm_workspace_size")

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
    }
    for name, types in args.items():
        f = getattr(lib, name)
        f.argtypes, f.restype = types, ctypes.c_int
    for name, types in (("wtconv_causal_workspace_size", [cd]), ("wtconv_scan_workspace_size", [sd, _i]),
                        ("wtconv_norm_workspace_size", [nd])):
        f = getattr(lib, name)
        f.argtypes, f.restype = types, sz
    _bound = lib
    return lib


class _on:
    """The stream of a call, on the inputs' device, which is made the current
    one (a launch goes to the current device); a stream that was passed in is
    made current too, so that what is allocated belongs to it."""
    __slots__ = ("device", "stream", "inside")

    def __init__(self, x, stream):
        self.device, self.stream, self.inside = x.device, stream, None

    def __enter__(self):
        if self.stream is not None:
            if self.stream.device != self.device:
                raise ValueError("stream must be on the inputs' device")
            self.inside = torch.cuda.stream(self.stream)
            self.inside.__enter__()
            return self.stream.cuda_stream
        if self.device.index != torch.cuda.current_device():
            self.inside = torch.cuda.device(self.device)
            self.inside.__enter__()
        return torch.cuda.current_stream(self.device).cuda_stream

    def __exit__(self, *e):
        if self.inside is not None:
            self.inside.__exit__(*e)


def _activation(x, name):
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if x.dtype not in _TYPES:
        raise TypeError(f"{name} must be torch.float32 or torch.bfloat16")


def _tensor(t, name, shape, dtype, like):
    """t, which has to be a tensor of this shape and type on like's device."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.device != like.device:
        raise ValueError(f"{name} must be on the inputs' device")
    return t


def _dense(t, name, shape, dtype, like):
    """The address of a contiguous tensor (None: NULL)."""
    if t is None:
        return None
    if not _tensor(t, name, shape, dtype, like).is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t, name, shape, dtype, like, inner=1):
    """A [B, T, ...] or (single token) [B, ...] tensor as the library's rows;
    `inner`: the number of last dimensions that make up a row."""
    if t is None:
        return None
    _tensor(t, name, shape, dtype, like)
    s = t.stride()
    if s[-1] != 1 and shape[-1] != 1 or inner == 2 and s[-2] != shape[-1] and shape[-2] != 1:
        raise ValueError(f"{name} must be contiguous along its last dimension" + ("s" if inner == 2 else ""))
    return Rows(t.data_ptr(), s[0], s[1] if len(s) > inner + 1 else 0)


def _empty(shape, dtype, like):
    return torch.empty(shape, dtype=dtype, device=like.device)


def _workspace(need, ws, like):
    if ws is None:
        ws = torch.empty(need, dtype=torch.uint8, device=like.device)
    elif not ws.is_cuda or not ws.is_contiguous() or ws.device != like.device:
        raise ValueError("ws must be a contiguous tensor on the inputs' device")
    return ws, ws.numel() * ws.element_size()


# ---------------------------------------------------------- causal convolution
def _causal(x, w, silu, T):
    _activation(x, "x")
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w must have shape [C, k]")
    B, C = x.shape[0], x.shape[-1]
    k = w.shape[1]
    return CausalDesc(B, T, C, k, _TYPES[x.dtype], int(bool(silu))), (B, k - 1, C)


def causal_forward(x, w, b=None, silu=True, state=None, lengths=None, y=None, state_out=None, stream=None):
    """Causal depthwise convolution over tokens: (y, state_out).

    y[t] = silu(b + sum_j w[:, j] x[t - (k-1) + j]); x [B, T, C], w [C, k], b [C];
    state [B, k-1, C]: the inputs before the first token (None: zeros);
    state_out: the last k-1 inputs, to go on from (may be `state` itself)."""
    lib = load_seq()
    if x.dim() != 3:
        raise ValueError("x must have shape [B, T, C]")
    desc, held = _causal(x, w, silu, x.shape[1])
    f32, io, C = torch.float32, x.dtype, x.shape[2]
    with _on(x, stream) as st:
        y = _empty(x.shape, io, x) if y is None else y
        state_out = _empty(held, io, x) if state_out is None else state_out
        _check(lib.wtconv_causal_forward(desc, _rows(x, "x", x.shape, io, x), _dense(w, "w", (C, desc.k), f32, x),
                                         _dense(b, "b", (C,), f32, x), _dense(state, "state", held, io, x),
                                         _dense(lengths, "lengths", (desc.B,), torch.int32, x), _rows(y, "y", x.shape, io, x),
                                         _dense(state_out, "state_out", held, io, x), st), "wtconv_causal_forward")
    return y, state_out


def causal_backward(x, dy, w, b=None, silu=True, state=None, lengths=None, dstate=None, dx=None, grads=None, ws=None,
                    stream=None):
    """Gradients of <y, dy> + <state_out, dstate>: (dx, dict dw, db, dstate).

    grads["dstate"] is that of the state before the pass (None without one);
    grads["db"] is None without a bias."""
    lib = load_seq()
    if x.dim() != 3:
        raise ValueError("x must have shape [B, T, C]")
    desc, held = _causal(x, w, silu, x.shape[1])
    f32, io, C = torch.float32, x.dtype, x.shape[2]
    with _on(x, stream) as st:
        dx = _empty(x.shape, io, x) if dx is None else dx
        g = grads if grads is not None else dict(dw=torch.empty_like(w), db=None if b is None else torch.empty_like(b),
                                                 dstate=None if state is None else torch.empty_like(state))
        ws, nws = _workspace(lib.wtconv_causal_workspace_size(desc), ws, x)
        _check(lib.wtconv_causal_backward(desc, _rows(x, "x", x.shape, io, x), _rows(dy, "dy", x.shape, io, x),
                                          _dense(w, "w", (C, desc.k), f32, x), _dense(b, "b", (C,), f32, x),
                                          _dense(state, "state", held, io, x),
                                          _dense(lengths, "lengths", (desc.B,), torch.int32, x),
                                          _dense(dstate, "dstate", held, io, x), _rows(dx, "dx", x.shape, io, x),
                                          _dense(g["dw"], "dw", (C, desc.k), f32, x), _dense(g["db"], "db", (C,), f32, x),
                                          _dense(g["dstate"], "grads['dstate']", held, io, x), ws.data_ptr(), nws, st),
               "wtconv_causal_backward")
    return dx, g


def causal_step(x, state, w, b=None, silu=True, active=None, y=None, stream=None):
    """One token of every row, y [B, C] of x [B, C]; state [B, k-1, C] is moved
    on in place.  active (int32 [B]): 0 leaves a row's state as it is and its
    output zero."""
    lib = load_seq()
    if x.dim() != 2:
        raise ValueError("x must have shape [B, C]")
    desc, held = _causal(x, w, silu, 1)
    f32, io, C = torch.float32, x.dtype, x.shape[1]
    with _on(x, stream) as st:
        y = _empty(x.shape, io, x) if y is None else y
        _check(lib.wtconv_causal_step(desc, _rows(x, "x", x.shape, io, x), _dense(w, "w", (C, desc.k), f32, x),
                                      _dense(b, "b", (C,), f32, x), _dense(active, "active", (desc.B,), torch.int32, x),
                                      _rows(y, "y", x.shape, io, x), _dense(state, "state", held, io, x), st),
               "wtconv_causal_step")
    return y


# ------------------------------------------------------------------------ scan
def _scan(x, a, b, softplus, T):
    """The descriptor and the shape of b and c (groups may be left out)."""
    _activation(x, "x")
    if not isinstance(a, torch.Tensor) or a.dim() != 2:
        raise ValueError("a must have shape [C, N]")
    lead = x.dim() - 1
    if not isinstance(b, torch.Tensor) or b.dim() not in (lead + 1, lead + 2):
        raise ValueError("b must have the shape of x with [N] or [G, N] in place of the channels")
    N = a.shape[1]
    G = b.shape[-2] if b.dim() == lead + 2 else 1
    inner = (G, N) if b.dim() == lead + 2 else (N,)
    return ScanDesc(x.shape[0], T, x.shape[-1], N, G, _TYPES[x.dtype], int(bool(softplus))), x.shape[:lead] + inner


def scan_forward(x, dt, a, b, c, d=None, z=None, dt_bias=None, softplus=True, state=None, lengths=None, y=None,
                 state_out=None, ws=None, stream=None):
    """Selective state space scan: (y, state_out).

    delta = softplus(dt + dt_bias);  h = exp(delta a) h + delta x b;
    y = (c . h + d x) silu(z).  x, dt, z [B, T, C]; a [C, N] fp32; b, c
    [B, T, N], or [B, T, G, N] for G groups of channels; d, dt_bias [C] fp32;
    state, state_out [B, C, N] fp32 (state_out may be `state` itself)."""
    lib = load_seq()
    if x.dim() != 3:
        raise ValueError("x must have shape [B, T, C]")
    desc, bc = _scan(x, a, b, softplus, x.shape[1])
    f32, io, S, C, inner = torch.float32, x.dtype, x.shape, x.shape[2], len(bc) - 2
    held = (desc.B, C, desc.N)
    with _on(x, stream) as st:
        y = _empty(S, io, x) if y is None else y
        state_out = _empty(held, f32, x) if state_out is None else state_out
        need = lib.wtconv_scan_workspace_size(desc, 0)
        ws, nws = _workspace(need, ws, x) if need or ws is not None else (None, 0)
        _check(lib.wtconv_scan_forward(desc, _rows(x, "x", S, io, x), _rows(dt, "dt", S, io, x),
                                       _dense(a, "a", (C, desc.N), f32, x), _rows(b, "b", bc, io, x, inner),
                                       _rows(c, "c", bc, io, x, inner), _dense(d, "d", (C,), f32, x),
                                       _rows(z, "z", S, io, x), _dense(dt_bias, "dt_bias", (C,), f32, x),
                                       _dense(state, "state", held, f32, x),
                                       _dense(lengths, "lengths", (desc.B,), torch.int32, x), _rows(y, "y", S, io, x),
                                       _dense(state_out, "state_out", held, f32, x), None if ws is None else ws.data_ptr(),
                                       nws, st), "wtconv_scan_forward")
    return y, state_out


def scan_backward(x, dt, a, b, c, dy, d=None, z=None, dt_bias=None, softplus=True, state=None, lengths=None, dstate=None,
                  grads=None, ws=None, stream=None):
    """Gradients of <y, dy> + <state_out, dstate>: dict dx, ddt, da, db, dc, dd,
    dz, ddt_bias, dstate (the last for the state before the pass), None for
    inputs that are not given."""
    lib = load_seq()
    if x.dim() != 3:
        raise ValueError("x must have shape [B, T, C]")
    desc, bc = _scan(x, a, b, softplus, x.shape[1])
    f32, io, S, C, inner = torch.float32, x.dtype, x.shape, x.shape[2], len(bc) - 2
    held = (desc.B, C, desc.N)
    with _on(x, stream) as st:
        g = grads
        if g is None:
            new = lambda t, shape, dtype: None if t is None else _empty(shape, dtype, x)
            g = dict(dx=_empty(S, io, x), ddt=_empty(S, io, x), da=_empty((C, desc.N), f32, x), db=_empty(bc, io, x),
                     dc=_empty(bc, io, x), dd=new(d, (C,), f32), dz=new(z, S, io), ddt_bias=new(dt_bias, (C,), f32),
                     dstate=new(state, held, f32))
        ws, nws = _workspace(lib.wtconv_scan_workspace_size(desc, 1), ws, x)
        _check(lib.wtconv_scan_backward(desc, _rows(x, "x", S, io, x), _rows(dt, "dt", S, io, x),
                                        _dense(a, "a", (C, desc.N), f32, x), _rows(b, "b", bc, io, x, inner),
                                        _rows(c, "c", bc, io, x, inner), _dense(d, "d", (C,), f32, x),
                                        _rows(z, "z", S, io, x), _dense(dt_bias, "dt_bias", (C,), f32, x),
                                        _dense(state, "state", held, f32, x),
                                        _dense(lengths, "lengths", (desc.B,), torch.int32, x),
                                        _rows(dy, "dy", S, io, x), _dense(dstate, "dstate", held, f32, x),
                                        _rows(g["dx"], "dx", S, io, x), _rows(g["ddt"], "ddt", S, io, x),
                                        _dense(g["da"], "da", (C, desc.N), f32, x), _rows(g["db"], "db", bc, io, x, inner),
                                        _rows(g["dc"], "dc", bc, io, x, inner), _dense(g["dd"], "dd", (C,), f32, x),
                                        _rows(g["dz"], "dz", S, io, x), _dense(g["ddt_bias"], "ddt_bias", (C,), f32, x),
                                        _dense(g["dstate"], "grads['dstate']", held, f32, x), ws.data_ptr(), nws, st),
               "wtconv_scan_backward")
    return g


def scan_step(x, dt, state, a, b, c, d=None, z=None, dt_bias=None, softplus=True, active=None, y=None, stream=None):
    """One token of every row, y [B, C] of x, dt, z [B, C] and b, c [B, N] or
    [B, G, N]; state [B, C, N] fp32 is moved on in place.  active (int32 [B]):
    0 leaves a row's state as it is and its output zero."""
    lib = load_seq()
    if x.dim() != 2:
        raise ValueError("x must have shape [B, C]")
    desc, bc = _scan(x, a, b, softplus, 1)
    f32, io, S, C, inner = torch.float32, x.dtype, x.shape, x.shape[1], len(bc) - 1
    with _on(x, stream) as st:
        y = _empty(S, io, x) if y is None else y
        _check(lib.wtconv_scan_step(desc, _rows(x, "x", S, io, x), _rows(dt, "dt", S, io, x),
                                    _dense(a, "a", (C, desc.N), f32, x), _rows(b, "b", bc, io, x, inner),
                                    _rows(c, "c", bc, io, x, inner), _dense(d, "d", (C,), f32, x), _rows(z, "z", S, io, x),
                                    _dense(dt_bias, "dt_bias", (C,), f32, x),
                                    _dense(active, "active", (desc.B,), torch.int32, x), _rows(y, "y", S, io, x),
                                    _dense(state, "state", (desc.B, C, desc.N), f32, x), st), "wtconv_scan_step")
    return y


# ------------------------------------------------------------------------ norm
def _norm(x, res, eps):
    _activation(x, "x")
    if x.dim() not in (2, 3):
        raise ValueError("x must have shape [B, T, C] or [B, C]")
    if res is not None:
        _activation(res, "res")
    T = x.shape[1] if x.dim() == 3 else 1
    rt = x.dtype if res is None else res.dtype
    return NormDesc(x.shape[0], T, x.shape[-1], _TYPES[x.dtype], _TYPES[rt], eps), rt


def norm_forward(x, w=None, gate=None, res=None, scale=None, w_res=None, eps=1e-6, lengths=None, y=None, res_out=None,
                 stream=None):
    """Norm after a block, gate, residual scale and norm before the next block,
    in one pass: (y, res_out).

    u = x silu(gate);  v = u w / sqrt(mean(u^2) + eps);  res_out = res + scale v;
    y = res_out w_res / sqrt(mean(res_out^2) + eps).  Each of gate, w and scale
    may be left out; without res y = v and res_out is None, without w_res y is
    None.  x, gate [B, T, C] or [B, C]; res in fp32 or bf16, whatever x is;
    w, scale, w_res [C] fp32."""
    lib = load_seq()
    desc, rt = _norm(x, res, eps)
    f32, io, S, V = torch.float32, x.dtype, x.shape, (x.shape[-1],)
    with _on(x, stream) as st:
        if y is None and (res is None or w_res is not None):
            y = _empty(S, io, x)
        if res_out is None and res is not None:
            res_out = _empty(S, rt, x)
        _check(lib.wtconv_norm_forward(desc, _rows(x, "x", S, io, x), _rows(gate, "gate", S, io, x), _dense(w, "w", V, f32, x),
                                       _rows(res, "res", S, rt, x), _dense(scale, "scale", V, f32, x),
                                       _dense(w_res, "w_res", V, f32, x),
                                       _dense(lengths, "lengths", (desc.B,), torch.int32, x), _rows(y, "y", S, io, x),
                                       _rows(res_out, "res_out", S, rt, x), st), "wtconv_norm_forward")
    return y, res_out


def norm_backward(x, dy=None, w=None, gate=None, res=None, scale=None, w_res=None, dres=None, eps=1e-6, lengths=None,
                  grads=None, ws=None, stream=None):
    """Gradients of <y, dy> + <res_out, dres>: dict dx, dgate, dw, dres (of the
    residual that came in), dscale, dw_res, None for inputs that are not given.
    dy is None exactly where the forward pass gives no y; dres None is zero."""
    lib = load_seq()
    desc, rt = _norm(x, res, eps)
    f32, io, S, V = torch.float32, x.dtype, x.shape, (x.shape[-1],)
    with _on(x, stream) as st:
        g = grads
        if g is None:
            new = lambda t, shape, dtype: None if t is None else _empty(shape, dtype, x)
            g = dict(dx=_empty(S, io, x), dgate=new(gate, S, io), dw=new(w, V, f32), dres=new(res, S, rt),
                     dscale=new(scale, V, f32), dw_res=new(w_res, V, f32))
        ws, nws = _workspace(lib.wtconv_norm_workspace_size(desc), ws, x)
        _check(lib.wtconv_norm_backward(desc, _rows(x, "x", S, io, x), _rows(gate, "gate", S, io, x),
                                        _dense(w, "w", V, f32, x), _rows(res, "res", S, rt, x),
                                        _dense(scale, "scale", V, f32, x), _dense(w_res, "w_res", V, f32, x),
                                        _dense(lengths, "lengths", (desc.B,), torch.int32, x), _rows(dy, "dy", S, io, x),
                                        _rows(dres, "dres", S, rt, x), _rows(g["dx"], "dx", S, io, x),
                                        _rows(g["dgate"], "dgate", S, io, x), _dense(g["dw"], "dw", V, f32, x),
                                        _rows(g["dres"], "dres", S, rt, x), _dense(g["dscale"], "dscale", V, f32, x),
                                        _dense(g["dw_res"], "dw_res", V, f32, x), ws.data_ptr(), nws, st),
               "wtconv_norm_backward")
    return g
