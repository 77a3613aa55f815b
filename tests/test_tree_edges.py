"""Tree attention at the edges of what its queries, calls and buffers may be."""
import numpy as np
import pytest
import torch

from sparse_mla_decode_dcp_gb300 import capi
from test_tree_decode import FORMATS, Case, _err


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
