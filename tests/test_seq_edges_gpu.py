"""The sequence operators on the GPU at the edges of their layouts, sizes and
variants, against the float64 oracle (tests/seq_cases.py) or against the same
call on plain inputs."""
import pytest
import torch

import depthwise_convolution_wtconv_b200 as wt
import seq_cases as sc
from seq_cases import cuda, scan_case

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
