"""Attention over the 4-bit cache with numbers at the ends of their ranges: NaN keys
beside weights that pass every bound, scores so large that fp32 has no place for
anything beside them."""
import pytest
import torch

from test_gpu_attend4 import make, run
from test_gpu_attend4_lanes import FORMS, crowd, places

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("later", [133, 5 + 128 * 4])
@pytest.mark.parametrize("dim, rows", FORMS)
def test_nan_stays_beside_a_weight_that_passes_the_range(dim, rows, later):
    """A NaN key in the first tile, and in a later one, at the same place, a key whose score in base 2 is some 200 above all
    others: rows that see both are NaN, in out and in lse."""
    c = make(**crowd(700, 600), group=rows // 4, dim=dim, seed=5)
    c["q"] = torch.ones_like(c["q"])
    c["cache"].k_scale.mul_(1e-3)
    page, off = places(c, 0, [later])
    c["cache"].k[page, 0, off] = 0x77  # 6 twice
    c["cache"].k_group[page, 0, off] = torch.ones(1, dim // 16, device="cuda").to(torch.float8_e4m3fn)
    c["cache"].k_scale[page, 0, off] = 140 / (6 * dim * c["scale"])
    clean, clean_lse, status = run(c)
    assert status == 0 and not bool(torch.isnan(clean_lse).any())
    page, off = places(c, 0, [5])
    c["cache"].k_scale[page, 0, off] = float("nan")
    out, lse, status = run(c)
    assert status == 0 and bool(torch.isnan(out[:4]).all()) and bool(torch.isnan(lse[:4]).all())
    assert torch.equal(out[4:], clean[4:]) and torch.equal(lse[4:], clean_lse[4:])
