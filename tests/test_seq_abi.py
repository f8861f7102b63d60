"""The sequence operators' C entries and binding without a GPU: exports, sizes
and refusals, all before any launch."""
import ctypes
import os
import re

import pytest
import torch

import depthwise_convolution_wtconv_b200 as wt
from depthwise_convolution_wtconv_b200 import _seq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, ARG, ALIGN, WS, UNSUPPORTED = 0, 1, 3, 4, 6
FAKE = 0x10000  # aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    return wt.load_seq()


def test_header_declares_the_binding_exports(lib):
    text = open(os.path.join(ROOT, "include", "wtconv_seq.h")).read()
    names = re.findall(r"^(?:size_t|wtconv_status)\s+(wtconv_\w+)\s*\(", text, re.M)
    assert sorted(names) == sorted(wt.EXPORTS_SEQ)
    for n in names:
        assert hasattr(lib, n)


def test_header_is_plain_c(tmp_path):
    import shutil
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    src = tmp_path / "c.c"
    src.write_text('#include "wtconv_seq.h"\nint main(void) { wtconv_norm_desc d = {1, 1, 1, WTCONV_F32, WTCONV_F32, 0.f};\n'
                   "  return wtconv_norm_workspace_size(&d) == 0; }\n")
    pkg = os.path.join(ROOT, "depthwise_convolution_wtconv_b200")
    exe = str(tmp_path / "c")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-I" + os.path.join(ROOT, "include"), str(src), "-L" + pkg,
                    "-lwtconv", "-Wl,-rpath," + pkg, "-o", exe], check=True)
    assert subprocess.run([exe]).returncode == 0


def R(p=FAKE, sb=1 << 16, st=64):
    return _seq.Rows(p, sb, st)


CAUSAL = dict(B=2, T=8, C=64, k=4, io=0, silu=1)
SCAN = dict(B=2, T=8, C=64, N=16, G=1, io=0, softplus=1)
NORM = dict(B=2, T=8, C=64, io=0, res=0, eps=1e-6)


def causal_desc(**kw):
    return _seq.CausalDesc(*{**CAUSAL, **kw}.values())


def scan_desc(**kw):
    return _seq.ScanDesc(*{**SCAN, **kw}.values())


def norm_desc(**kw):
    return _seq.NormDesc(*{**NORM, **kw}.values())


@pytest.mark.parametrize("kw,status", [(dict(B=0), ARG), (dict(T=0), ARG), (dict(C=-1), ARG), (dict(k=0), ARG), (dict(io=2), ARG),
                                       (dict(k=9), UNSUPPORTED)])
def test_causal_descriptors(lib, kw, status):
    d = causal_desc(**kw)
    assert lib.wtconv_causal_forward(d, R(), FAKE, None, None, None, R(), None, None) == status
    assert lib.wtconv_causal_workspace_size(d) == 0


# what every call refuses: an argument in place of a good one, and the answer
def _forward(lib, d=None, x=R(), w=FAKE, bias=FAKE, state=FAKE, lengths=FAKE, y=R(), out=FAKE):
    return lib.wtconv_causal_forward(d or causal_desc(), x, w, bias, state, lengths, y, out, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), ARG), (dict(y=None), ARG), (dict(w=None), ARG), (dict(x=R(None)), ARG), (dict(x=R(sb=-1)), ARG),
    (dict(x=R(st=-64)), ARG), (dict(y=R(st=63)), ARG), (dict(y=R(sb=511)), ARG), (dict(y=R(sb=0)), ARG), (dict(x=R(st=1 << 60)), ARG),
    (dict(x=R(FAKE + 2)), ALIGN), (dict(y=R(FAKE + 1)), ALIGN), (dict(w=FAKE + 2), ALIGN), (dict(bias=FAKE + 1), ALIGN),
    (dict(state=FAKE + 2), ALIGN), (dict(lengths=FAKE + 2), ALIGN), (dict(out=FAKE + 2), ALIGN)])
def test_causal_forward_refusals(lib, kw, status):
    assert _forward(lib, **kw) == status


def test_causal_backward_refusals(lib):
    d = causal_desc()
    need = lib.wtconv_causal_workspace_size(d)
    assert need == 2 * 64 * 5 * 4  # one strip block a row: the sums of 4 taps and the bias of each channel

    def f(x=R(), dy=R(), w=FAKE, bias=FAKE, dx=R(), dw=FAKE, db=FAKE, ws=FAKE, nws=need):
        return lib.wtconv_causal_backward(d, x, dy, w, bias, None, None, None, dx, dw, db, None, ws, nws, None)
    assert f(dy=None) == ARG and f(dx=None) == ARG and f(dw=None) == ARG and f(db=None) == ARG
    assert f(dx=R(st=32)) == ARG
    assert f(ws=None) == WS and f(nws=need - 1) == WS and f(ws=FAKE + 8) == ALIGN


def test_steps_refuse_more_than_one_token(lib):
    assert lib.wtconv_causal_step(causal_desc(), R(), FAKE, None, None, R(), FAKE, None) == ARG
    assert lib.wtconv_causal_step(causal_desc(T=1), R(), FAKE, None, None, R(), None, None) == ARG
    assert lib.wtconv_scan_step(scan_desc(), R(), R(), FAKE, R(), R(), None, None, None, None, R(), FAKE, None) == ARG
    assert lib.wtconv_scan_step(scan_desc(T=1), R(), R(), FAKE, R(), R(), None, None, None, None, R(), None, None) == ARG
    assert lib.wtconv_scan_step(scan_desc(T=1), R(), R(), FAKE, R(), R(), None, None, None, None, R(), FAKE + 2, None) == ALIGN


@pytest.mark.parametrize("kw,status", [(dict(N=0), ARG), (dict(G=0), ARG), (dict(G=3), ARG), (dict(T=0), ARG), (dict(io=-1), ARG),
                                       (dict(N=65), UNSUPPORTED)])
def test_scan_descriptors(lib, kw, status):
    d = scan_desc(**kw)
    assert lib.wtconv_scan_forward(d, R(), R(), FAKE, R(), R(), None, None, None, None, None, R(), None, FAKE, 1 << 40, None) == status
    assert lib.wtconv_scan_workspace_size(d, 1) == 0


@pytest.mark.parametrize("kw,status", [(dict(x=None), ARG), (dict(dt=None), ARG), (dict(a=None), ARG), (dict(b=None), ARG),
                                       (dict(c=R(None)), ARG), (dict(y=None), ARG), (dict(y=R(st=8)), ARG), (dict(z=R(st=-1)), ARG),
                                       (dict(a=FAKE + 2), ALIGN), (dict(state=FAKE + 2), ALIGN), (dict(b=R(FAKE + 2)), ALIGN)])
def test_scan_forward_refusals(lib, kw, status):
    g = {**dict(x=R(), dt=R(), a=FAKE, b=R(), c=R(), d=None, z=None, bias=None, state=None, lengths=None, y=R(), out=None), **kw}
    assert lib.wtconv_scan_forward(scan_desc(), *g.values(), FAKE, 1 << 40, None) == status


def test_scan_backward_refusals(lib):
    d = scan_desc()
    need = lib.wtconv_scan_workspace_size(d, 1)
    assert need > 0 and lib.wtconv_scan_workspace_size(d, 2) == 0 and lib.wtconv_scan_workspace_size(None, 1) == 0

    def f(**kw):
        g = {**dict(x=R(), dt=R(), a=FAKE, b=R(), c=R(), d=FAKE, z=R(), bias=FAKE, state=None, lengths=None, dy=R(), dout=None,
                    dx=R(), ddt=R(), da=FAKE, db=R(), dc=R(), dd=FAKE, dz=R(), dbias=FAKE, dstate=None, ws=FAKE, nws=need), **kw}
        return lib.wtconv_scan_backward(d, *g.values(), None)
    for m in ("dy", "dx", "ddt", "da", "db", "dc", "dd", "dz", "dbias", "d", "z", "bias"):
        assert f(**{m: None}) == ARG, m
    assert f(db=R(st=8)) == ARG and f(ws=None) == WS and f(nws=need - 1) == WS and f(ws=FAKE + 4) == ALIGN


@pytest.mark.parametrize("kw,status", [(dict(C=0), ARG), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG), (dict(res=5), ARG),
                                       (dict(C=16385), UNSUPPORTED)])
def test_norm_descriptors(lib, kw, status):
    d = norm_desc(**kw)
    assert lib.wtconv_norm_forward(d, R(), None, FAKE, None, None, None, None, R(), None, None) == status
    assert lib.wtconv_norm_workspace_size(d) == 0


def test_norm_refusals(lib):
    def f(x=R(), gate=None, w=FAKE, res=None, scale=None, w_res=None, lengths=None, y=R(), out=None):
        return lib.wtconv_norm_forward(norm_desc(), x, gate, w, res, scale, w_res, lengths, y, out, None)
    assert f(w=None) == ARG                                   # nothing to do
    assert f(y=None) == ARG and f(out=R()) == ARG and f(scale=FAKE) == ARG and f(w_res=FAKE) == ARG
    assert f(res=R(), out=R()) == ARG                         # y without w_res
    assert f(res=R(), w_res=FAKE) == ARG                      # no res_out
    assert f(res=R(), w_res=FAKE, out=R(), y=None) == ARG
    assert f(res=R(), w_res=FAKE, out=R(st=1)) == ARG
    assert f(gate=R(FAKE + 2)) == ALIGN and f(w=FAKE + 2) == ALIGN
    d = norm_desc()
    need = lib.wtconv_norm_workspace_size(d)
    assert need == 16 * 3 * 64 * 4                            # a block a row, three sums a channel

    def g(**kw):
        a = {**dict(x=R(), gate=R(), w=FAKE, res=R(), scale=FAKE, w_res=FAKE, lengths=None, dy=R(), dres_out=R(), dx=R(), dgate=R(),
                    dw=FAKE, dres=R(), dscale=FAKE, dw_res=FAKE, ws=FAKE, nws=need), **kw}
        return lib.wtconv_norm_backward(d, *a.values(), None)
    for m in ("dy", "dx", "dgate", "dw", "dres", "dscale", "dw_res", "gate", "w", "scale", "w_res"):
        assert g(**{m: None}) == ARG, m
    assert g(ws=None) == WS and g(nws=need - 16) == WS and g(ws=FAKE + 8) == ALIGN


_X = torch.zeros(1, 2, 8)
_W = torch.zeros(8, 4)
_CALLS = {
    "causal_forward": lambda: wt.causal_forward(_X, _W),
    "causal_backward": lambda: wt.causal_backward(_X, _X, _W),
    "causal_step": lambda: wt.causal_step(_X[0], torch.zeros(2, 3, 8), _W),
    "scan_forward": lambda: wt.scan_forward(_X, _X, _W, _X[..., :4], _X[..., :4]),
    "scan_backward": lambda: wt.scan_backward(_X, _X, _W, _X[..., :4], _X[..., :4], _X),
    "scan_step": lambda: wt.scan_step(_X[0], _X[0], torch.zeros(2, 8, 4), _W, _X[0, :, :4], _X[0, :, :4]),
    "norm_forward": lambda: wt.norm_forward(_X, torch.ones(8)),
    "norm_backward": lambda: wt.norm_backward(_X, _X, torch.ones(8)),
}


@pytest.mark.parametrize("name", sorted(_CALLS))
def test_every_binding_refuses_cpu_tensors(name):
    with pytest.raises(TypeError, match="CUDA tensor"):
        _CALLS[name]()


def test_outputs_in_place_of_inputs_are_refused(lib):
    """A convolution or scan whose output begins where an input does would read what it has written."""
    far = lambda k: R(FAKE + (k << 32))
    d = causal_desc()
    assert lib.wtconv_causal_forward(d, far(1), FAKE, None, None, None, far(1), None, None) == ARG
    need = lib.wtconv_causal_workspace_size(d)
    for dx in (1, 2):
        assert lib.wtconv_causal_backward(d, far(1), far(2), FAKE, None, None, None, None, far(dx), FAKE, None, None, FAKE, need,
                                          None) == ARG
    s = scan_desc()
    for k in range(1, 6):
        assert lib.wtconv_scan_forward(s, far(1), far(2), FAKE, far(3), far(4), None, far(5), None, None, None, far(k), None, FAKE,
                                       1 << 40, None) == ARG
    need = lib.wtconv_scan_workspace_size(s, 1)
    outs = dict(dx=far(11), ddt=far(12), db=far(13), dc=far(14), dz=far(15))
    for m in outs:
        o = {**outs, m: far(6)}
        assert lib.wtconv_scan_backward(s, far(1), far(2), FAKE, far(3), far(4), None, far(5), None, None, None, far(6), None, o["dx"],
                                        o["ddt"], FAKE, o["db"], o["dc"], None, o["dz"], None, None, FAKE, need, None) == ARG
