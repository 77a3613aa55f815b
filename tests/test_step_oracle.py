"""Pins of oracle/step_oracle.py, independent of its arithmetic."""
import numpy as np
import pytest
import torch

from oracle import step_oracle as so
from oracle.smla_oracle import E4M3_TABLE


def test_e2m1_table_is_sign_two_exponent_bits_and_one_mantissa_bit():
    for code in range(16):
        e, m = (code >> 1) & 3, code & 1
        v = m * 0.5 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1)
        assert so.E2M1_TABLE[code] == (-v if code & 8 else v)


def test_nearest_code_is_nearest_and_ties_go_to_even():
    for table in (so.E2M1_TABLE[:8], E4M3_TABLE[:127]):
        x = np.concatenate([np.linspace(0, 1.1 * table[-1], 4001), (table[:-1] + table[1:]) / 2])
        got = so.nearest_code(table, x)
        dist = np.abs(x[:, None] - table[None])
        assert np.array_equal(dist[np.arange(len(x)), got], dist.min(axis=1))
        mid = so.nearest_code(table, (table[:-1] + table[1:]) / 2)
        assert np.all(mid % 2 == 0)


def test_fp8_rows_agree_with_torch_cast():
    rng = np.random.default_rng(0)
    y = rng.standard_normal((40, 512))
    code, scale = so.quantise_fp8(y)
    v = y.reshape(-1, 4, 128) / scale.astype(np.float64)[:, :, None]
    ref = torch.from_numpy(np.clip(v, -448, 448)).float().to(torch.float8_e4m3fn).view(torch.uint8)
    assert (code != ref.numpy().reshape(-1, 512)).mean() < 1e-3  # fp32 border cases aside
    assert np.allclose(scale, np.abs(y.reshape(-1, 4, 128)).max(axis=2) / 448, rtol=2.0 ** -24)


def test_fp4_row_parse_of_a_row_packed_by_hand():
    row = np.zeros((1, 416), dtype=np.uint8)
    row[0, 0] = 0x2 | (0xF << 4)   # dim 0: 1.0, dim 1: -6.0
    row[0, 255] = 0x9 | (0x3 << 4)  # dim 510: -0.5, dim 511: 1.5
    row[0, 256] = 0x40  # 2.0 for dims 0..15
    row[0, 287] = 0x30  # 0.5 for dims 496..511
    row[0, 414:416] = (0x80, 0xBF)  # bf16 -1.0
    lat, rope = so.parse_fp4_rows(row)
    assert lat[0, 0] == 2.0 and lat[0, 1] == -12.0
    assert lat[0, 510] == -0.25 and lat[0, 511] == 0.75
    assert np.count_nonzero(lat) == 4
    assert rope[0, 63] == -1.0 and np.count_nonzero(rope) == 1


@pytest.mark.parametrize("D,I,bs", [(1, 1, 4), (3, 1, 2), (2, 4, 3), (4, 2, 1)])
def test_step_maps_place_every_position_once(D, I, bs):
    """Steps appended one after the other: each position of each request is
    held by exactly one rank, in a slot no other position has."""
    rng = np.random.default_rng(D * 7 + I)
    B, W = 5, 64
    ctx = np.zeros(B, dtype=np.int64)
    tables = [np.full((B, W), -1, dtype=np.int32) for _ in range(D)]
    free = [list(rng.permutation(400)) for _ in range(D)]
    seen = [dict() for _ in range(D)]
    for _ in range(6):
        q = rng.integers(0, 9, B)
        ctx = ctx + q
        T = int(q.sum()) + 2
        held = np.zeros(T, dtype=int)
        for r in range(D):
            rs, req, pos, slots, local, taken = so.step_maps(ctx, q, free[r], tables[r], T, D, r, bs, I)
            free[r] = free[r][int(taken[0]):]
            for i in range(int(rs[-1])):
                if slots[i] >= 0:
                    held[i] += 1
                    assert slots[i] not in seen[r]
                    seen[r][int(slots[i])] = (int(req[i]), int(pos[i]))
            assert np.all(slots[rs[-1]:] == -1)
        assert np.all(held[:int(q.sum())] == 1)
    assert sum(len(s) for s in seen) == int(ctx.sum())


def test_window_positions():
    assert so.window_positions(5, 2, 0) == [4, 5]
    assert so.window_positions(5, 2, 2) == [0, 1, 4, 5]
    assert so.window_positions(2, 2, 2) == [0, 1, 2]
    assert so.window_positions(0, 1, 0) == [0]
    assert so.window_positions(3, 100, 7) == [0, 1, 2, 3]
