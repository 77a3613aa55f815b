"""Plain float64 definitions of the serving step around the decode: the 4-bit
row format, step maps, the cache write and attention over any set of rows.

TEST INFRASTRUCTURE: imported only by tests/.  It shares no code with the CUDA
path; every definition is written element by element or with whole-array
numpy steps that a reader can check by eye.

Pins (tests/test_step_oracle.py): e2m1 values and rounding against an
exhaustive nearest search, the row parse against rows packed by hand, step
maps against an append simulation, the write's fp8 rows against torch's e4m3
cast.
"""
from __future__ import annotations

import numpy as np

from .smla_oracle import E4M3_TABLE, bf16_bits_to_f64, parse_rows

FP4_ROW_BYTES = 416
E2M1_TABLE = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def parse_fp4_rows(rows):
    """uint8 [n, 416] -> (latent float64 [n, 512], rope float64 [n, 64])."""
    rows = np.ascontiguousarray(rows, dtype=np.uint8)
    assert rows.ndim == 2 and rows.shape[1] == FP4_ROW_BYTES
    nib = np.empty((rows.shape[0], 512), dtype=np.uint8)
    nib[:, 0::2] = rows[:, :256] & 15
    nib[:, 1::2] = rows[:, :256] >> 4
    scales = E4M3_TABLE[rows[:, 256:288]]
    rope = bf16_bits_to_f64(np.ascontiguousarray(rows[:, 288:]).view("<u2"))
    return E2M1_TABLE[nib] * np.repeat(scales, 16, axis=1), rope


def parse(rows):
    """Rows of either format, by their width."""
    return parse_fp4_rows(rows) if rows.shape[1] == FP4_ROW_BYTES else parse_rows(rows)


def nearest_code(magnitudes, x):
    """Index into the ascending table `magnitudes` nearest to |x|, ties to
    the even index, past the end to the last."""
    x = np.abs(np.asarray(x, dtype=np.float64))
    hi = np.clip(np.searchsorted(magnitudes, x), 1, len(magnitudes) - 1)
    lo = hi - 1
    dl, dh = x - magnitudes[lo], magnitudes[hi] - x
    return np.where((dl > dh) | ((dl == dh) & (hi % 2 == 0)), hi, lo)


def quantise_fp8(y):
    """float64 [n, 512] -> (codes uint8 [n, 512], scales float32 [n, 4])."""
    g = y.reshape(-1, 4, 128)
    scale = (np.abs(g).max(axis=2) / 448.0).astype(np.float32)
    s = np.where(scale > 0, scale, 1).astype(np.float64)[:, :, None]
    code = nearest_code(E4M3_TABLE[:127], g / s).astype(np.uint8)
    code |= np.where(np.signbit(g), 0x80, 0).astype(np.uint8)
    code[scale == 0] = 0
    return code.reshape(-1, 512), scale


def quantise_fp4(y):
    """float64 [n, 512] -> (codes uint8 [n, 512] of 4 bits, scale codes uint8 [n, 32])."""
    g = y.reshape(-1, 32, 16)
    sc = nearest_code(E4M3_TABLE[:127], np.abs(g).max(axis=2) / 6.0).astype(np.uint8)
    s = E4M3_TABLE[sc]
    code = nearest_code(E2M1_TABLE[:8], g / np.where(s > 0, s, 1)[:, :, None]).astype(np.uint8)
    code |= np.where(np.signbit(g), 8, 0).astype(np.uint8)
    code[s == 0] = 0
    return code.reshape(-1, 512), sc


def normalise(x, gamma, eps):
    """float64 latent rows after the root-mean-square norm (gamma None: as is)."""
    if gamma is None:
        return x
    return x / np.sqrt((x * x).mean(axis=1, keepdims=True) + np.float64(np.float32(eps))) * gamma


def rotate(z, cos_sin, pairs):
    """float64 rope parts [n, 64] rotated by each row's cos_sin [n, 64]."""
    out = z.copy()
    for j in range(32):
        a, b = (2 * j, 2 * j + 1) if pairs else (j, j + 32)
        c, s = cos_sin[:, j], cos_sin[:, 32 + j]
        out[:, a] = z[:, a] * c - z[:, b] * s
        out[:, b] = z[:, a] * s + z[:, b] * c
    return out


def rank_rows(n, D, rank, I):
    """How many of the first n positions rank holds."""
    return sum(1 for t in range(n) if (t // I) % D == rank)


def step_maps(ctx, q, free, table, T, D, rank, bs, I):
    """Returns the six maps of a step and updates `table` in place."""
    B = len(ctx)
    row_start, req_id, positions, slots, local, taken = [0], [], [], [], [], 0
    for b in range(B):
        lp = rank_rows(int(ctx[b]) - int(q[b]), D, rank, I)  # cached here before the step
        for p in range(int(ctx[b]) - int(q[b]), int(ctx[b])):
            req_id.append(b)
            positions.append(p)
            if (p // I) % D != rank:
                slots.append(-1)
                continue
            if lp % bs == 0:  # opens a block
                table[b, lp // bs] = free[taken]
                taken += 1
            slots.append(int(table[b, lp // bs]) * bs + lp % bs)
            lp += 1
        local.append(lp)
        row_start.append(row_start[-1] + int(q[b]))
    pad = T - len(slots)
    return [np.array(v, dtype=np.int32) for v in
            (row_start, req_id + [0] * pad, positions + [0] * pad, slots + [-1] * pad, local, [taken])]


def window_positions(p, window, sinks):
    """Positions the token at p attends."""
    return [t for t in range(p + 1) if t < sinks or t > p - window]


def attend(q, rows, sm_scale, key_step=0.0):
    """One token: q float64 [H, 576], cache rows uint8 [n, 656 or 416].

    Returns (out, lse, out_tol, lse_tol): the tolerances bound the kernel's
    arithmetic.  A score's products are of an exact q and of keys within
    key_step (relative) of the cache's, summed in fp32 by at most 42 rounded
    (perhaps truncated) additions; p and a split's partial output round to
    fp16 (2^-11 each, and 2^-11 for the peer's p rescaled), out to bf16
    (2^-8); the fp32 steps after the scores are below 2^-19.  Below 2^-14
    fp16's step is 2^-24, so each of those fp16 roundings is off by up to
    2^-25 as well: a p against a sum that is at least 1 (a key's p is 2^0
    when it sets the reference), a key (where key_step is not 0) and a
    partial output.  fp4 rows' codes times scales are exact in fp16; their
    rope values round as other keys do below 2^-14."""
    H = q.shape[0]
    if len(rows) == 0:
        return np.zeros((H, 512)), np.full(H, -np.inf), np.zeros((H, 512)), np.zeros(H)
    lat, rope = parse(rows)
    k = np.concatenate([lat, rope], axis=1)
    s = sm_scale * (q @ k.T)
    m = s.max(axis=1, keepdims=True)
    lse = m[:, 0] + np.log(np.exp(s - m).sum(axis=1))
    p = np.exp(s - lse[:, None])
    size = sm_scale * (np.abs(q) @ np.abs(k).T)
    tiny = 2.0 ** -25
    lse_tol = size.max(axis=1) * (42 * 2.0 ** -23 + key_step) + 2.0 ** -19
    if rows.shape[1] == FP4_ROW_BYTES:
        lse_tol = lse_tol + sm_scale * np.abs(q[:, 512:]).sum(axis=1) * tiny
    if key_step:
        lse_tol = lse_tol + sm_scale * np.abs(q).sum(axis=1) * tiny
    out = p @ lat
    out_tol = 2.0 ** -8 * np.abs(out) + (3 * 2.0 ** -11 + key_step + 2 * lse_tol)[:, None] * (p @ np.abs(lat))
    out_tol = out_tol + tiny * (2 + 2 * np.abs(lat).sum(axis=0))
    return out, lse, out_tol, lse_tol
