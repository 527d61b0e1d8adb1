"""Attention over the 4-bit cache where neighbouring lanes of a warp go different
ways: keys whose value scale is no number beside others, pages outside the cache,
maxima that rise tile after tile.  Every form of the kernel's tiles (16, 32 and 64
rows, head_dim 64 and 128); tolerances as in test_gpu_attend4."""
import pytest
import torch

import speculative_decoding_token_rejection_gb300 as sv
from test_gpu_attend4 import check, make, reference, run

pytestmark = pytest.mark.gpu

FORMS = [(dim, rows) for dim in (64, 128) for rows in (16, 32, 64)]


def places(c, i, keys):
    """Pages and offsets of keys of request i."""
    t = torch.as_tensor(keys, device="cuda")
    return c["table"][i].long()[t // c["cache"].block_size], t % c["cache"].block_size


def crowd(*lens):
    """Lengths of a batch so large that a request's keys are one CTA's work, tile after tile."""
    return dict(gammas=[3] * 320, lens=[*lens] + [4] * (320 - len(lens)), kv_heads=1, uniform=True)


@pytest.mark.parametrize("dim, rows", FORMS)
def test_every_third_value_scale_is_no_number(dim, rows):
    c = make([3, 3, 0], [700, 300, 50], kv_heads=2, group=rows // 4, dim=dim, seed=rows)
    page, off = places(c, 0, range(1, 690, 3))
    c["cache"].v_scale[page, 1, off] = float("inf")
    out, lse, status = run(c)
    ref, rlse, tol, ltol = reference(c)
    assert status == 0 and bool(((lse.double() - rlse).abs() <= ltol).all())
    gone = torch.zeros(out.shape[:2], dtype=torch.bool, device="cuda")
    gone[:4, c["group"]:] = True
    assert bool(torch.isnan(out[gone]).all())
    assert bool(((out.double() - ref).abs() <= tol)[~gone].all())


@pytest.mark.parametrize("dim, rows", FORMS)
def test_every_other_page_is_outside(dim, rows):
    """Pages of 3 tokens: the lanes' keys are there and not by turns."""
    c = make([3, 0], [390, 200], kv_heads=1, group=rows // 4, dim=dim, block=3, fmt="int4", seed=rows + 1)
    # the same without those keys; the verify tokens are in pages that stay
    keep = [x for x in range(130) if x % 2 == 0 or x > 125]
    short = dict(c, table=torch.zeros_like(c["table"]), lens=[3 * len(keep), 200])
    short["table"][0, :len(keep)] = c["table"][0, torch.tensor(keep, device="cuda")]
    short["table"][1] = c["table"][1]
    c["table"][0, [x for x in range(130) if x not in keep]] = c["cache"].num_blocks
    out, lse, status = run(c)
    ref, rlse, tol, ltol = reference(short)
    assert status == sv.DATA_STATUS_BITS["BAD_SLOT"]
    assert bool(((lse.double() - rlse).abs() <= ltol).all()) and bool(((out.double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("dim, rows", FORMS)
def test_maxima_that_rise_tile_after_tile(dim, rows):
    """Some rows' maxima rise in every tile, others' fall (queries of both signs)."""
    c = make(**crowd(1100, 513), group=rows // 4, dim=dim, seed=rows + 2)
    c["q"] = c["q"].abs().clone()
    c["q"][1::2] *= -1
    c["cache"].k &= 0x77
    for i, n in enumerate(c["lens"][:2]):
        page, off = places(c, i, range(n))
        c["cache"].k_scale[page, 0, off] = 0.02 * torch.exp2(torch.arange(n, device="cuda") / 128)
    check(c)
