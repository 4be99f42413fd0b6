"""Shared pieces of the training operators' GPU tests."""
from __future__ import annotations

import numpy as np
import torch

EPS32 = 2.0 ** -24   # half an ulp of fp32, relative
# unit roundoff of each output type (24 and 8 significant bits)
OUT_EPS = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
TORCH = {"bf16": torch.bfloat16, "fp32": torch.float32}


def rows(values, dtype, pad=0, shift=0):
    """values [N, C] on the GPU as rows of a wider buffer: row stride C + pad, the
    first row `shift` elements into an allocation, NaN around them."""
    v = torch.as_tensor(np.asarray(values, dtype=np.float32)).to(dtype)
    N, C = v.shape
    buf = torch.full((shift + N * (C + pad),), float("nan"), dtype=dtype, device="cuda")
    out = buf[shift:].view(N, C + pad)[:, :C]
    out.copy_(v)
    return out


def wide(t):
    """Exact float64 values of a device tensor."""
    return t.detach().double().cpu().numpy()


def sum_error(V):
    """Relative error of a softmax sum over V values as the kernels form it: each
    term's exponential (2 ulp) and its argument (a difference, a product and the
    rounded factor: 3 roundings of |a|, and |a| 2^-a <= 0.54), at most V / 128 + 16
    sequential additions of positive terms and 16 of a tree."""
    return 4 * 2 * EPS32 + 3 * 0.54 * EPS32 + (V / 128 + 32) * EPS32
