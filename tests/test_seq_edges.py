"""Refusals and sizes of the sequence operators' C entries, without a GPU: the
addresses are made up, so nothing here may run where a call could be launched."""
import os
import subprocess
import sys

import pytest
import torch

import depthwise_convolution_wtconv_b200 as wt
from depthwise_convolution_wtconv_b200 import _seq

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")

ARG = 1
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def lib():
    return wt.load_seq()


def P(k):
    """Addresses far apart, one for each k."""
    return 0x10000 + (k << 32)


def R(k, sb=1 << 16, st=64):
    return _seq.Rows(P(k), sb, st)


# ------------------------------------- outputs that begin where an input does
CAUSAL = dict(x=1, w=2, bias=3, state=4, lengths=5, y=6, state_out=7)
CAUSAL_BACK = dict(x=1, dy=2, w=3, bias=4, state=5, lengths=6, dstate_out=7, dx=8, dw=9, dbias=10, dstate=11)
CAUSAL_STEP = dict(x=1, w=2, bias=3, active=4, y=5, state=6)
SCAN = dict(x=1, dt=2, a=3, b=4, c=5, d=6, z=7, dt_bias=8, state=9, lengths=10, y=11, state_out=12)
SCAN_BACK = dict(x=1, dt=2, a=3, b=4, c=5, d=6, z=7, dt_bias=8, state=9, lengths=10, dy=11, dstate_out=12, dx=13, ddt=14, da=15, db=16,
                 dc=17, dd=18, dz=19, ddt_bias=20, dstate=21)
SCAN_STEP = dict(x=1, dt=2, a=3, b=4, c=5, d=6, z=7, dt_bias=8, active=9, y=10, state=11)
NORM = dict(x=1, gate=2, w=3, res=4, scale=5, w_res=6, lengths=7, y=8, res_out=9)
NORM_BACK = dict(x=1, gate=2, w=3, res=4, scale=5, w_res=6, lengths=7, dy=8, dres_out=9, dx=10, dgate=11, dw=12, dres=13, dscale=14,
                 dw_res=15)
ROWS = {"x", "y", "dy", "dx", "dt", "b", "c", "z", "ddt", "db", "dc", "dz", "gate", "res", "res_out", "dres_out", "dgate", "dres"}


def call(lib, name, desc, places, strides={}, ws=True):
    args = [R(k, **strides.get(m, {})) if m in ROWS else P(k) for m, k in places.items()]
    return getattr(lib, name)(desc, *args, *([P(90), 1 << 40] if ws else []), None)


def pairs(table, outs, ins):
    return [(o, i) for o in outs for i in ins if o in table and i in table]


@pytest.mark.parametrize("out,at", pairs(CAUSAL, ("y", "state_out"), ("x", "w", "bias", "lengths")) + [("y", "state")])
def test_causal_forward_over_an_input(lib, out, at):
    d = _seq.CausalDesc(2, 8, 64, 4, F32, 1)
    assert call(lib, "wtconv_causal_forward", d, {**CAUSAL, out: CAUSAL[at]}, ws=False) == ARG


@pytest.mark.parametrize("out,at", pairs(CAUSAL_BACK, ("dx", "dstate"), ("x", "dy", "w", "bias", "lengths", "dstate_out")) +
                         [("dx", "state")])
def test_causal_backward_over_an_input(lib, out, at):
    d = _seq.CausalDesc(2, 8, 64, 4, F32, 1)
    assert call(lib, "wtconv_causal_backward", d, {**CAUSAL_BACK, out: CAUSAL_BACK[at]}) == ARG


@pytest.mark.parametrize("out,at", pairs(CAUSAL_STEP, ("y",), ("w", "bias", "active", "state")) +
                         pairs(CAUSAL_STEP, ("state",), ("x", "w", "bias", "active")))
def test_causal_step_over_an_input(lib, out, at):
    d = _seq.CausalDesc(2, 1, 64, 4, F32, 1)
    assert call(lib, "wtconv_causal_step", d, {**CAUSAL_STEP, out: CAUSAL_STEP[at]}, ws=False) == ARG


@pytest.mark.parametrize("out,at", pairs(SCAN, ("y", "state_out"), ("x", "dt", "a", "b", "c", "d", "z", "dt_bias", "lengths")) +
                         [("y", "state")])
def test_scan_forward_over_an_input(lib, out, at):
    d = _seq.ScanDesc(2, 8, 64, 16, 1, F32, 1)
    assert call(lib, "wtconv_scan_forward", d, {**SCAN, out: SCAN[at]}) == ARG


@pytest.mark.parametrize("out,at", pairs(SCAN_BACK, ("dx", "ddt", "db", "dc", "dz", "dstate"),
                                         ("x", "dt", "a", "b", "c", "d", "z", "dt_bias", "lengths", "dy", "dstate_out")) +
                         pairs(SCAN_BACK, ("dx", "ddt", "db", "dc", "dz"), ("state",)))
def test_scan_backward_over_an_input(lib, out, at):
    d = _seq.ScanDesc(2, 8, 64, 16, 1, F32, 1)
    assert call(lib, "wtconv_scan_backward", d, {**SCAN_BACK, out: SCAN_BACK[at]}) == ARG


@pytest.mark.parametrize("out,at", pairs(SCAN_STEP, ("y",), ("a", "b", "c", "d", "dt_bias", "active", "state")) +
                         pairs(SCAN_STEP, ("state",), ("x", "dt", "a", "b", "c", "d", "z", "dt_bias", "active")))
def test_scan_step_over_an_input(lib, out, at):
    d = _seq.ScanDesc(2, 1, 64, 16, 1, F32, 1)
    assert call(lib, "wtconv_scan_step", d, {**SCAN_STEP, out: SCAN_STEP[at]}, ws=False) == ARG


@pytest.mark.parametrize("name,desc,places,at", [("wtconv_causal_step", _seq.CausalDesc(2, 1, 64, 4, F32, 1), CAUSAL_STEP, "x")] +
                         [("wtconv_scan_step", _seq.ScanDesc(2, 1, 64, 16, 1, F32, 1), SCAN_STEP, m) for m in ("x", "dt", "z")])
def test_steps_in_place_of_other_rows(lib, name, desc, places, at):
    """A step may write where its input lies, but not in rows that lie otherwise."""
    assert call(lib, name, desc, {**places, "y": places[at]}, {"y": dict(sb=1 << 17)}, ws=False) == ARG


@pytest.mark.parametrize("out,at", pairs(NORM, ("y", "res_out"), ("x", "gate", "res", "w", "scale", "w_res", "lengths")))
def test_norm_forward_over_an_input(lib, out, at):
    """Refused: parameters, rows that lie otherwise, and rows of another type."""
    d = _seq.NormDesc(2, 8, 64, BF16, F32, 1e-6)
    other_type = (out == "y") != (at in ("x", "gate"))
    for strides in [{}] if at not in ROWS or other_type else [dict(sb=1 << 17), dict(st=128)]:
        assert call(lib, "wtconv_norm_forward", d, {**NORM, out: NORM[at]}, {out: strides}, ws=False) == ARG


@pytest.mark.parametrize("out,at", pairs(NORM_BACK, ("dx", "dgate", "dres"), ("x", "gate", "res", "dy", "dres_out", "w", "scale", "w_res",
                                                                              "lengths")))
def test_norm_backward_over_an_input(lib, out, at):
    d = _seq.NormDesc(2, 8, 64, BF16, F32, 1e-6)
    other_type = (out == "dres") != (at in ("res", "dres_out"))
    for strides in [{}] if at not in ROWS or other_type else [dict(sb=1 << 17), dict(st=128)]:
        assert call(lib, "wtconv_norm_backward", d, {**NORM_BACK, out: NORM_BACK[at]}, {out: strides}) == ARG


# --------------------------------------------- rows beyond 32-bit channels
@pytest.mark.parametrize("C,G,N", [(2 ** 31 - 1, 1, 1), (2 ** 28, 2 ** 28, 4), (2 ** 25, 2 ** 25, 64), (2 ** 25, 2 ** 25, 61)])
def test_scan_rows_of_too_many_elements(lib, C, G, N):
    """Channels (rounded up in each group) and states of a token have to fit 32 bits, also where they are copied to
    rounded-up rows."""
    places = {m: k for m, k in SCAN.items()}
    wide = {m: dict(sb=1 << 40, st=(1 << 31) - 1) for m in ROWS}
    for T in (1, 2):
        d = _seq.ScanDesc(1, T, C, N, G, BF16, 1)
        assert call(lib, "wtconv_scan_forward", d, places, wide) == ARG
        assert lib.wtconv_scan_workspace_size(d, 0) == 0 and lib.wtconv_scan_workspace_size(d, 1) == 0


def test_causal_rows_of_too_many_elements(lib):
    d = _seq.CausalDesc(1, 1, 2 ** 31 - 1, 4, BF16, 1)
    assert call(lib, "wtconv_causal_forward", d, CAUSAL, ws=False) == ARG
    assert lib.wtconv_causal_workspace_size(d) == 0
    assert lib.wtconv_causal_workspace_size(_seq.CausalDesc(1, 1, 2 ** 31 - 4096, 4, BF16, 1)) > 0
    assert lib.wtconv_scan_workspace_size(_seq.ScanDesc(1, 1, 2 ** 31 - 4096, 4, 1, BF16, 1), 1) > 0


# ------------------------------------------------- torch without CUDA
def test_package_without_the_bindings_of_cuda():
    """A torch built without CUDA lacks the calls for the current stream and device: the package still imports, what needs
    no GPU still answers, and tensors are refused as ever."""
    code = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import depthwise_convolution_wtconv_b200 as wt
from depthwise_convolution_wtconv_b200 import _seq
d = wt.make_desc(2, 8, 16, 16, 5, 2, "f32")
assert wt.kernel_launches(d, 3) > 0 and wt.workspace_size(d, 3) >= 0
assert wt.load_seq().wtconv_causal_workspace_size(_seq.CausalDesc(2, 8, 64, 4, 0, 1)) > 0
try:
    wt.causal_forward(torch.zeros(1, 2, 8), torch.zeros(8, 4))
except TypeError as e:
    assert "CUDA tensor" in str(e)
else:
    raise AssertionError("not refused")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


# ------------------------------------------------- the norm's workspace
@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("C", [1, 64, 250, 2048, 2049, 4096, 4097, 5120, 8192, 8200, 16383, 16384])
def test_norm_workspace_is_what_its_blocks_leave(lib, C, io):
    """Three sums a channel of every block; a block is the threads that hold a row, 512 threads on each of 148 SMs."""
    values = next(v for v in (8, 16, 32) if -(-C // v) <= 512)
    threads = -(-C // values // 32) * 32
    for B, T in ((1, 1), (3, 7), (64, 1024)):
        blocks = min(B * T, 148 * max(1, min(16, 512 // threads)))
        assert lib.wtconv_norm_workspace_size(_seq.NormDesc(B, T, C, io, F32, 1e-6)) == (blocks * 3 * C * 4 + 15) // 16 * 16
