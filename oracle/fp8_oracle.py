"""Plain float64 definitions of the 8-bit projections: rows to e4m3 with a
scale for each 128 columns, and the product with block-scaled weights.

TEST INFRASTRUCTURE: imported only by tests/.  It shares no code with the CUDA
path.

Pins (tests/test_fp8_products.py): a group worked by hand, torch's e4m3 cast.
"""
from __future__ import annotations

import numpy as np

from .smla_oracle import E4M3_TABLE
from .step_oracle import nearest_code


def quantise(x):
    """float64 [M, K] -> (codes uint8 [M, K], scales float32 [M, ceil(K / 128)])."""
    M, K = x.shape
    codes = np.zeros((M, K), dtype=np.uint8)
    scales = np.zeros((M, -(-K // 128)), dtype=np.float32)
    for j in range(scales.shape[1]):
        v = x[:, 128 * j:128 * j + 128]
        good = np.isfinite(v).all(axis=1)
        v = np.where(good[:, None], v, 0)
        s = np.where(good, np.abs(v).max(axis=1) / 448.0, np.nan).astype(np.float32)
        coded = good & (s >= np.float32(2.0 ** -126))
        c = nearest_code(E4M3_TABLE[:127], v / np.where(coded, s, 1).astype(np.float64)[:, None])
        c = c.astype(np.uint8) | np.where(np.signbit(v), 0x80, 0).astype(np.uint8)
        codes[:, 128 * j:128 * j + 128] = np.where(coded[:, None], c, 0)
        scales[:, j] = s
    return codes, scales


def values(codes, scales, block_rows=1):
    """float64 values of codes [M, K] under a scale for block_rows x 128."""
    s = np.repeat(scales.astype(np.float64), 128, axis=1)[:, :codes.shape[1]]
    return E4M3_TABLE[codes] * np.repeat(s, block_rows, axis=0)[:codes.shape[0]]


def matmul(a, a_scales, b, b_scales, out_half_step):
    """(a b^T, its tolerance): codes uint8 [M, K], [N, K].

    The codes' products are exact in fp32.  A group's 128 of them are added by
    the tensor cores, each addition off by at most a step (2^-23) of the sizes
    added; the product of the scales, its product with the group's sum and the
    sum over the groups round once each (2^-24), one more for every group.
    Then the result is rounded (out_half_step, relative)."""
    va, vb = values(a, a_scales), values(b, b_scales, 128)
    out = va @ vb.T
    size = np.abs(va) @ np.abs(vb).T
    groups = a_scales.shape[1]
    tol = size * (128 * 2.0 ** -23 + (groups + 2) * 2.0 ** -24)
    return out, tol + out_half_step * (np.abs(out) + tol) + 2.0 ** -133
