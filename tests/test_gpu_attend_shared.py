"""Attention with a prefix that is shared by the batch -- unpacked once, met by
every request's rows on the tensor cores, joined with the private keys -- in
the ways a call may be made: launch modes, streams, graphs, workspaces, and bad
data.  Each case takes the shortest prefix that a call of its sizes shares."""
import pytest
import torch

import speculative_decoding_token_rejection_gb300 as sv
from test_gpu_attend import check, make, run
from test_gpu_attend_scales import shared, shared_prefix

pytestmark = pytest.mark.gpu

BITS = sv.DATA_STATUS_BITS


@pytest.mark.parametrize("entry, value", [(9, 140), (14, 2), (19, 0), (19, -5), (29, 160)])
def test_a_bad_range_leaves_the_others_right(entry, value):
    """Requests whose own range is in order get their result, whatever stands in the entries of others."""
    N, G = 40, 4
    c = shared([G] * N, [5 + i for i in range(N)], seed=23)
    ws = torch.full((1 << 26,), 0xFF, dtype=torch.uint8, device="cuda")
    want, want_lse, _ = run(c, workspace=ws)
    assert c["cu"][entry] == G * (entry + 1)
    c["cu"][entry] = value
    ws.fill_(0xFF)
    out, lse, status = run(c, workspace=ws)
    assert status == BITS["BAD_CU"]
    for i in range(N):
        if i not in (entry, entry + 1):
            rows = slice(i * (G + 1), (i + 1) * (G + 1))
            assert torch.equal(out[rows], want[rows]) and torch.equal(lse[rows], want_lse[rows]), i


@pytest.mark.parametrize("many", [True, False])
def test_bytes_behind_every_length_may_be_anything(many):
    """Pages of the prefix that no request's tokens reach yet: NaN scales and bytes."""
    if many:
        c = shared([4] * 40, [-60 - i for i in range(40)], uniform=True, fmt="e4m3", seed=24)
    else:
        c = make([1, 0], [1500, 1421], prefix=2400, group=2, fmt="e4m3", seed=24)
    cache, b, last = c["cache"], c["cache"].block_size, max(c["lens"])
    for t in range(last, c["prefix"]):
        page, off = int(c["table"][0, t // b]), t % b
        for data, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
            scale[page, :, off] = float("nan")
            data.view(torch.uint8)[page, :, off] = 0x7F if t % 2 else 0xFF
    check(c)


@pytest.mark.parametrize("kw, least, most", [
    (dict(gammas=[3] * 8, kv_heads=8), 16384, 16400), (dict(gammas=[4] * 64, kv_heads=8), 1024, 4096),
    (dict(gammas=[7] * 512, kv_heads=8), 512, 1024), (dict(gammas=[0] * 512, kv_heads=8), 256, 640),
    (dict(gammas=[3] * 64, kv_heads=1, group=8), 8192, 16400), (dict(gammas=[3] * 64, kv_heads=8, dim=64), 1024, 4096)])
def test_a_prefix_is_shared_from_where_that_pays(kw, least, most):
    """Between two lengths at which the two ways were measured: at the first reading by each request won, at the other
    sharing did (or it is the first above all that were measured)."""
    assert least < shared_prefix(**kw) <= most
