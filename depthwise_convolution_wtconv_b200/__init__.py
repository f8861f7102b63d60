"""WTConv (multi-level Haar wavelet depthwise convolution) for B200.

The compute path is libwtconv.so (hand-written sm_100a CUDA kernels behind a
C ABI, see include/wtconv.h); `forward`, `backward_data`, `backward_weight`,
`backward`, `fold_weights` and `forward_folded` are thin ctypes wrappers over
it that take CUDA tensors.  Beside the image layer the library holds the
sequence operators (include/wtconv_seq.h): `causal_forward`, `causal_backward`,
`causal_step` (causal depthwise convolution over tokens), `scan_forward`,
`scan_backward`, `scan_step` (selective state space scan) and `norm_forward`,
`norm_backward` (norms with gate and residual scale).
"""
from ._lib import (  # noqa: F401
    forward, backward_data, backward_weight, backward, backward_weight_noalloc, fold_weights, forward_folded,
    workspace_size, kernel_launches, make_desc, load,
    WTConvError, EXPORTS, LIB_PATH,
)
from ._seq import (  # noqa: F401
    causal_forward, causal_backward, causal_step, scan_forward, scan_backward, scan_step,
    norm_forward, norm_backward, load_seq, EXPORTS_SEQ,
)
