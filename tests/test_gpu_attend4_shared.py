"""Attention over the 4-bit cache with a prefix that is shared by the batch (each
case takes the shortest one that a call of its sizes shares), and with scales that
kv_write would not have written.  What holds over the 8-bit cache holds here: its
tests run on 4-bit caches, against the formula of test_gpu_attend4 with its
tolerances."""
import math

import pytest
import torch

import speculative_decoding_token_rejection_gb300 as sv
import test_gpu_attend4 as four
import test_gpu_attend_scales as scales
from test_gpu_attend4 import BOTH, FORMATS, check, make, poison, reference, run, verifier
from test_gpu_attend_shared import SIZES

pytestmark = pytest.mark.gpu


def shared_prefix(gammas, *, kv_heads=2, group=4, dim=128, block=16, **_):
    """The shortest prefix that a call of these sizes computes once for all requests.  (One that every request reads for
    itself needs the workspace of a call without a prefix.)"""
    N, G, rows = len(gammas), max(gammas), sum(gammas) + len(gammas)
    cache = make([0], [1], kv_heads=kv_heads, dim=dim)["cache"]

    def size(prefix, most):
        return sv.spec_verify_attend_workspace_size(verifier().handle, cache=cache, num_reqs=N, max_spec_len=G,
                                                    num_q_heads=kv_heads * group, max_seq_len=most,
                                                    shared_prefix_len=prefix, num_tokens=rows)

    for prefix in range(128 // block * block, 1 << 16, block):
        if size(prefix, prefix + 4096) != size(0, prefix + 4096):
            return prefix
    raise AssertionError("no prefix is shared")


def shared(gammas, own, **kw):
    """A call with a prefix that is shared; `own`: tokens behind it (before its end if negative; None: no tokens at all)."""
    prefix = shared_prefix(gammas, **kw)
    return make(gammas, [0 if n is None else prefix + n for n in own], prefix=prefix, **kw)


def grown(gammas, lens, *, prefix=0, **kw):
    """A call whose prefix, if it has one, is lengthened to one that is shared."""
    longer = max(0, shared_prefix(gammas, **kw) - prefix) if prefix else 0
    return make(gammas, [n + longer for n in lens], prefix=prefix + longer, **kw)


def check_scales(c):
    """As check; rows that see a value scale that is no number have NaN outputs, and what they would have else is that of a
    scale of 0."""
    out, lse, status = run(c)
    cache, b = c["cache"], c["cache"].block_size
    given, odd = cache.v_scale.clone(), ~torch.isfinite(cache.v_scale)
    cache.v_scale[odd] = 0.0
    ref, rlse, tol, ltol = reference(c)
    cache.v_scale.copy_(given)
    nan, at = torch.zeros(lse.shape, dtype=torch.bool, device="cuda"), 0
    for i, (g, n) in enumerate(zip(c["gammas"], c["lens"])):
        t = torch.arange(n, device="cuda")
        seen = odd[c["table"][i].long()[t // b], :, t % b].long().cumsum(0)
        for j in range(g + 1):
            if n - g + j > 0:
                nan[at + j] = (seen[n - g + j - 1] > 0).repeat_interleave(c["group"])
        at += g + 1
    assert status == 0 and torch.equal(torch.isinf(lse), torch.isinf(rlse)) and not bool(torch.isnan(lse).any())
    live = ~torch.isinf(rlse)
    assert bool(((lse.double() - rlse).abs() <= ltol)[live].all())
    assert torch.equal(torch.isnan(out), nan[..., None].expand(out.shape))
    assert bool((out.double() - ref).abs().le(tol)[~nan].all())
    return out, lse


@pytest.mark.parametrize("name", SIZES)
def test_against_the_formula(name):
    check(poison(shared(seed=1, **SIZES[name])))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kw", [dict(kv_heads=1, group=1), dict(kv_heads=4, group=3, dim=64), dict(kv_heads=2, group=20)])
def test_groups_of_query_heads(kw, fmt):
    check(poison(shared([2] * 30, [40 + 7 * i for i in range(30)], uniform=True, fmt=fmt, seed=2, **kw)))


@pytest.mark.parametrize("name", SIZES)
def test_serial_launch_and_repeats_give_the_same(name):
    c = shared(seed=3, **SIZES[name])
    want = run(c)
    for flags in (0, 0, sv.SV_FLAG_SERIAL_LAUNCH):
        got = run(c, flags=flags)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("fmt", FORMATS)
def test_bytes_behind_every_length_may_be_anything(fmt):
    """Pages of the prefix that no request's tokens reach yet: scales and group scales that are no numbers, any nibbles."""
    c = shared([4] * 40, [-60 - i for i in range(40)], uniform=True, fmt=fmt, seed=24)
    cache, b = c["cache"], c["cache"].block_size
    for t in range(max(c["lens"]), c["prefix"]):
        page, off = int(c["table"][0, t // b]), t % b
        for data, group, scale in ((cache.k, cache.k_group, cache.k_scale), (cache.v, cache.v_group, cache.v_scale)):
            scale[page, :, off] = float("nan") if t % 3 else float("inf")
            group.view(torch.uint8)[page, :, off] = 0x7F if t % 2 else 0xFF
            data[page, :, off] = t % 256
    check(c)


def test_nan_key_reaches_only_the_rows_that_see_it():
    c = shared([3] * 40, [3 - i for i in range(40)], uniform=True, seed=11)  # all requests but the first end inside
    clean, clean_lse, _ = run(c)
    page = int(c["table"][0, (c["prefix"] - 1) // 16])  # the prefix's last key: position prefix - 1
    c["cache"].k_scale[page, 0, 15] = float("nan")
    out, lse, _ = run(c)
    see = torch.tensor([[n - 4 + j >= c["prefix"] - 1 for j in range(4)] for n in c["lens"]]).reshape(-1).cuda()
    assert 0 < int(see.sum()) < see.numel() // 4
    hit = torch.zeros(out.shape[:2], dtype=torch.bool, device="cuda")
    hit[see, :c["group"]] = True
    assert bool(torch.isnan(out[hit]).all()) and bool(torch.isnan(lse[hit]).all())
    assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], clean_lse[~hit])


def test_calls_of_other_sizes_share_a_workspace():
    calls = [shared(seed=19, **SIZES[name]) for name in SIZES]
    calls += [make([2, 0, 5], [3000, 20, 900], seed=20), make([1, 0], [2500, 2421], prefix=2400, group=2, seed=21)]
    want = [run(c) for c in calls]
    ws = torch.full((1 << 27,), 0xFF, dtype=torch.uint8, device="cuda")
    for i in (0, 4, 1, 5, 2, 3, 0, 1, 3, 2):
        got = run(calls[i], workspace=ws)
        assert torch.equal(got[0], want[i][0]) and torch.equal(got[1], want[i][1])


def test_in_a_graph():
    c = shared(seed=16, **SIZES["uniform"])
    want, want_lse, _ = run(c)
    out, lse, ver, most = torch.zeros_like(want), torch.zeros_like(want_lse), verifier(), max(c["lens"])
    ws = ver.attend_workspace(cache=c["cache"], num_reqs=40, max_spec_len=4, num_q_heads=8, max_seq_len=most,
                              shared_prefix_len=c["prefix"], num_tokens=200)
    side, q = torch.cuda.Stream(), c["q"].clone()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ver.attend(q=q, cache=c["cache"], block_tables=c["table"], seq_lens=c["seq_lens"], max_seq_len=most, max_spec_len=4,
                   scale=c["scale"], out=out, lse=lse, shared_prefix_len=c["prefix"], workspace=ws)
    for _ in range(2):
        out.zero_()
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("test, args", [
    (four.test_small_and_large_queries, (1e-3, "e2m1")), (four.test_small_and_large_queries, (30.0, "int4")),
    (four.test_small_and_large_queries, (3000.0, "e2m1")), (four.test_value_scales_of_many_sizes, (BOTH[1],)),
    (four.test_value_scales_that_count_as_zero, (BOTH[1], 0.0)),
    (four.test_value_scales_that_count_as_zero, (BOTH[1], 2.0 ** -70)),
    (four.test_value_scales_that_are_no_numbers, (BOTH[1], math.nan)),
    (four.test_nan_in_a_row_of_q_stays_in_it, (BOTH[1],)), (four.test_rows_of_very_different_sizes, (BOTH[1],)),
    (four.test_strided_and_unaligned_queries_and_outputs, (BOTH[1],)), (four.test_bad_page_in_a_shared_prefix, (60,)),
    (four.test_only_the_first_row_names_the_prefix_pages, (2240, "int4"))], ids=lambda x: getattr(x, "__name__", None))
def test_the_same_with_shared_prefixes(test, args, monkeypatch):
    monkeypatch.setattr(four, "make", grown)
    test(*args)


@pytest.mark.parametrize("test, args", [
    (scales.test_value_scales_of_zero, (0.02, "int8")), (scales.test_value_scales_of_zero, (1.0, "e4m3")),
    (scales.test_a_zero_value_scale_at_the_row_s_best_key, ()), (scales.test_negative_value_scales, ()),
    (scales.test_value_scales_that_are_no_numbers, (math.nan,)), (scales.test_value_scales_that_are_no_numbers, (math.inf,)),
    (scales.test_value_scales_below_the_writer_s_smallest, ()), (scales.test_zero_rows_before_large_ones, ()),
    (scales.test_tiny_queries_and_huge_keys, ())], ids=lambda x: getattr(x, "__name__", None))
@pytest.mark.parametrize("form", scales.FORMS)
def test_scales_that_the_writer_does_not_give(form, test, args, monkeypatch):
    monkeypatch.setattr(scales, "make", make)
    monkeypatch.setattr(scales, "shared", shared)
    monkeypatch.setattr(scales, "check", check_scales)
    test(form, *args)


# (requests, G, kv heads, query heads a kv head): more than 32 rows a request; on both sides of four CTAs an SM
@pytest.mark.parametrize("N, G, kv_heads, group", [(33, 7, 2, 8), (33, 7, 2, 20), (160, 5, 4, 8), (9, 8, 1, 16)])
@pytest.mark.parametrize("prefix", [True, False])
def test_a_workspace_holds_for_fewer_draft_tokens(N, G, kv_heads, group, prefix):
    """Fewer tokens change the tiles of the private part, too: of 32 rows where requests have few on average, else of 64."""
    kw = dict(kv_heads=kv_heads, group=group, dim=64)
    prefix, own = shared_prefix([G] * N, **kw) if prefix else 0, 600
    ver, cache = verifier(), make([0], [5], **kw)["cache"]

    def size(tokens):
        return sv.spec_verify_attend_workspace_size(ver.handle, cache=cache, num_reqs=N, max_spec_len=G,
                                                    num_q_heads=kv_heads * group, max_seq_len=prefix + own,
                                                    shared_prefix_len=prefix, num_tokens=tokens)

    ws = torch.empty(max(16, size(N * (G + 1))), dtype=torch.uint8, device="cuda")
    lens = [prefix + own] + [prefix + max(G + 1, 7 * i % own) for i in range(N - 1)]
    for few in (0, 1, 2, 3, G):  # one request with G drafts, the others with `few`
        c = make([G] + [few] * (N - 1), lens, prefix=prefix, seed=few, **kw)
        want, got = run(c), run(c, workspace=ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    check(c)
