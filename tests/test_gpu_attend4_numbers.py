"""Attention over the 4-bit cache with numbers at the ends of their ranges: NaN keys
beside weights that pass every bound, scores so large that fp32 has no place for
anything beside them."""
import math

import pytest
import torch

import test_gpu_attend as eight
from test_gpu_attend4 import make, numbers, run
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


def ties(lens, *, score, prefix=0, dim=128, fmt="int4", **kw):
    """A batch in which all scores of a row are the same number, of about `score` in size (base e) and never a product that
    fp32 holds exactly, and value scales change by fours and sixteens from 128 keys to the next."""
    c = make([kw.pop("G", 0)] * len(lens), lens, prefix=prefix, dim=dim, fmt=fmt, uniform=True, seed=len(lens), **kw)
    c["q"] = torch.ones_like(c["q"])
    c["q"][:, 1::2] *= -1  # (every other query head has scores of the other sign)
    cache = c["cache"]
    cache.k.fill_(0x33 if fmt == "int4" else 0x55)  # 3, twice
    cache.k_group.copy_(torch.ones(cache.k_group.shape))
    cache.k_scale.fill_(1.0)
    c["scale"] = 1.0001 * score / (3 * dim)
    cache.v_scale.fill_(1 / 64)
    for i, n in enumerate(lens):
        t = torch.arange(prefix if i else 0, n, device="cuda")
        page, off = c["table"][i].long()[t // cache.block_size], t % cache.block_size
        cache.v_scale[page, :, off] = (torch.exp2((t // 128 * 5 % 8).float()) / 64)[:, None].expand(-1, cache.num_kv_heads)
    return c


def check_averages(c):
    """out is the average of the values that a row sees: bf16 (2^-8 of it), and weights of 11 bits, their exponentials and
    sums (2^-10 of the average size).  lse is its score plus ln of the number of keys, off by the
    roundings of the scale, its factors, the product, the maximum and the way back to base e: seven of 2^-24 at most."""
    out, lse, status = run(c)
    cache, b, G = c["cache"], c["cache"].block_size, c["G"]
    assert status == 0
    for i, n in enumerate(c["lens"]):
        t = torch.arange(n, device="cuda")
        page, off = c["table"][i].long()[t // b], t % b
        raw = cache.v_group.view(torch.uint8)[page, :, off].view(torch.float8_e4m3fn)
        v = numbers(cache.v[page, :, off], raw, cache.format) * cache.v_scale[page, :, off].double()[..., None]
        for j in range(G + 1):
            see, row = n - G + j, i * (G + 1) + j
            mean = v[:see].mean(0).repeat_interleave(c["group"], 0)
            size = v[:see].abs().mean(0).repeat_interleave(c["group"], 0)
            assert bool(((out[row].double() - mean).abs() <= 2.0 ** -8 * mean.abs() + 2.0 ** -10 * size).all())
            score = c["q"][row, :, 0].double() * 3 * cache.head_dim * c["scale"]
            assert bool(((lse[row].double() - score - math.log(see)).abs() <= 2.0 ** -21 * (score.abs() + 20)).all())


SCORES = [1.0, 2000.0, 3e4, 3e5, 3e6, 2.0 ** 24 + 2, 3.0 * 2 ** 25, 2.0 ** 28, 3.3 * 2 ** 30, 1.1e20, 1.9e38]


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("dim, fmt, group", [(128, "int4", 4), (64, "e2m1", 4), (128, "e2m1", 20)])
def test_ties_over_several_chunks(dim, fmt, group, score):
    check_averages(ties([1000, 300, 128, 129], score=score, dim=dim, fmt=fmt, group=group))
    check_averages(ties([3000], score=score, dim=dim, fmt=fmt, group=group, G=1))
    # many tiles a chunk
    check_averages(ties([1000, 520, 300] + [4] * 317, score=score, dim=dim, fmt=fmt, group=group, G=3, kv_heads=1))


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("dim, fmt, G, group", [(128, "int4", 4, 4), (64, "e2m1", 4, 4), (128, "e2m1", 0, 1)])
def test_ties_behind_a_shared_prefix(dim, fmt, G, group, score):
    """More than one CTA of the prefix for a row, and several chunks behind it."""
    lens = [7168 + 100 * i for i in range(1, 8)] + [7168, 7169 + G] + [7232] * 71
    check_averages(ties(lens, score=score, dim=dim, fmt=fmt, prefix=7168, G=G, group=group, kv_heads=2))
    lens = [16400 + i for i in range(80)]
    check_averages(ties(lens, score=score, dim=dim, fmt=fmt, prefix=16384, group=1, kv_heads=1))


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_ties_behind_a_shared_prefix_of_eight_bits(fmt, score):
    """The 8-bit cache's prefix is the same kernel's work."""
    lens = [7168 + 100 * i for i in range(1, 8)] + [7232] * 73
    c = eight.make([4] * len(lens), lens, prefix=7168, kv_heads=2, fmt=fmt, uniform=True, seed=1)
    c["q"] = torch.ones_like(c["q"])
    c["q"][:, 1::2] *= -1
    cache, b = c["cache"], c["cache"].block_size
    cache.k.copy_(torch.full(cache.k.shape, 3.0))
    cache.k_scale.fill_(1.0)
    c["scale"] = 1.0001 * score / (3 * cache.head_dim)
    for i, n in enumerate(lens):
        page, off = places(c, i, range(7168 if i else 0, n))
        step = torch.arange(7168 if i else 0, n, device="cuda") // 128 * 5 % 8
        cache.v_scale[page, :, off] = (torch.exp2(step.float()) / 64)[:, None].expand(-1, 2)
    out, lse, status = eight.run(c)
    assert status == 0
    for i, n in enumerate(lens[:8]):
        page, off = places(c, i, range(n))
        v = cache.v[page, :, off].double() * cache.v_scale[page, :, off].double()[..., None]
        for j in range(5):
            see, row = n - 4 + j, i * 5 + j
            mean = v[:see].mean(0).repeat_interleave(c["group"], 0)
            size = v[:see].abs().mean(0).repeat_interleave(c["group"], 0)
            assert bool(((out[row].double() - mean).abs() <= 2.0 ** -8 * mean.abs() + 2.0 ** -10 * size).all())
            exact = c["q"][row, :, 0].double() * 3 * cache.head_dim * c["scale"]
            assert bool(((lse[row].double() - exact - math.log(see)).abs() <= 2.0 ** -21 * (exact.abs() + 20)).all())
