"""Tree attention at the edges of what its queries, calls and buffers may be."""
import numpy as np
import pytest
import torch

from oracle import step_oracle as so
from oracle.smla_oracle import bf16_bits_to_f64
from sparse_mla_decode_dcp_gb300 import capi
from test_tree_decode import FORMATS, SCALE, Case, _err


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("at", [0, 511, 512, 575])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
def test_a_query_that_is_not_finite_is_reported(cuda_device, fmt, at, value):
    """Wherever in the row it is; the other rows are as they were."""
    c = Case(cuda_device, fmt, nodes=[5, 2], ctx=[70, 9], H=16, bs=16, seed=7).upload()
    clean = c.run()
    assert _err() == 0
    c.q[2, 5, at] = value
    c.upload()
    out, lse = c.run()
    assert _err() == capi.DEVERR_RANGE
    assert not lse[2, 5].isfinite() and not out[2, 5].isfinite().any()
    keep = torch.ones(c.T, c.H, dtype=torch.bool)
    keep[2, 5] = False
    assert torch.equal(out[keep], clean[0][keep]) and torch.equal(lse[keep], clean[1][keep])


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("low", [-60, -100, -113, -120, -126])
def test_tiny_latents_beside_an_ordinary_rope_part(cuda_device, fmt, low):
    """Finite scores whatever the sizes of the two parts are."""
    c = Case(cuda_device, fmt, nodes=[5], ctx=[70], H=16, bs=16, seed=7)
    c.q[:, ::2, :512] *= 2.0 ** low
    c.q[:, ::3, 512:] *= 300
    c.upload()
    out, lse = c.run()
    assert _err() == 0
    c.check(out, lse)


@pytest.mark.gpu
def test_latents_of_all_sizes(cuda_device):
    """8-bit rows: nodes whose latents are from 2^-126 to 2^16 of ordinary ones."""
    c = Case(cuda_device, "fp8", nodes=[72], ctx=[70], H=16, bs=16, seed=8, max_nodes=72)
    by = torch.exp2(torch.arange(-126, 18, 2).double())[:, None, None]
    c.q[..., :512] = (c.q[..., :512].double() * by).bfloat16()
    c.upload()
    out, lse = c.run()
    assert _err() == 0
    assert out.isfinite().all() and lse.isfinite().all()
    c.check(out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("ctx", [70, 900])
@pytest.mark.parametrize("fmt,low,high", [("fp8", 12, 100), ("fp4", 4, 12)])
def test_scores_past_the_exponentials_range(cuda_device, fmt, low, high, ctx):
    """Scores from some 2^13 to 2^100: the largest key alone counts, in whole
    tiles and in merged ranges."""
    c = Case(cuda_device, fmt, nodes=[8], ctx=[ctx], H=16, bs=16, seed=9)
    by = torch.exp2(torch.linspace(low, high, 8).floor().double())[:, None, None]
    c.q = (c.q.double() * by).bfloat16()
    if fmt == "fp4":  # groups' scales as large as they may be
        for pool in c.pools:
            pool[:, 256:288] = 0x70
    c.upload()
    out, lse = c.run()
    assert _err() == 0
    assert out.isfinite().all() and lse.isfinite().all()
    q = bf16_bits_to_f64(c.q.view(torch.int16).numpy().astype(np.uint16))
    checked = 0
    for j in range(8):
        lat, rope = so.parse(np.stack([c.pools[d][s] for d, s in c.keys(0, j, -1)]))
        s = SCALE * q[j] @ np.concatenate([lat, rope], axis=1).T
        size = SCALE * (np.abs(q[j]) @ np.abs(np.concatenate([lat, rope], axis=1)).T).max(axis=1)
        first, second = np.argmax(s, axis=1), np.sort(s, axis=1)[:, -2]
        tol = size * 2.0 ** -17  # 42 steps of 2^-23 of the products' sum, as so.attend has it, and the keys' rope in fp16
        assert np.all(np.abs(lse[j].cpu().double().numpy() - s.max(axis=1)) <= tol + np.log(ctx + 8))
        for h in range(16):
            if s[h].max() - second[h] > 2 * tol[h] + 20:  # another key's weight is below e^-20
                want = lat[first[h]]
                assert np.all(np.abs(out[j, h].cpu().double().numpy() - want) <= 2.0 ** -7 * np.abs(want) + 2.0 ** -12)
                checked += 1
    assert checked > 60
