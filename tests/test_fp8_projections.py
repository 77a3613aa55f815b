"""Calls of the 8-bit projections that are refused before anything runs."""
import pytest
import torch

from sparse_mla_decode_dcp_gb300 import capi
from sparse_mla_decode_dcp_gb300.pipeline import Fp8Projections


def _weight(*shape):
    *batch, R, K = shape
    rows = capi.alloc_fp8_rows(shape, "cpu").codes
    return capi.Fp8Rows(rows, torch.ones((*batch, -(-R // 128), -(-K // 128))))


@pytest.mark.parametrize("positions", [None, torch.zeros(1, dtype=torch.int32), torch.zeros(4, dtype=torch.int32),
                                       torch.zeros((3, 1), dtype=torch.int32)])
def test_rotation_needs_a_position_for_each_row(positions):
    """One position would be taken for all rows."""
    p = Fp8Projections(_weight(2 * (16 + 64), 64), _weight(2, 512, 16), _weight(2, 16, 512), _weight(8, 32), 5,
                       cos_sin=torch.zeros((9, 64)))
    with pytest.raises(ValueError, match="a position for each of the 3 rows"):
        p.query(torch.zeros((3, 64), dtype=torch.bfloat16), positions)
