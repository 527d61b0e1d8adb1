"""Attention with a prefix that is shared by the batch -- unpacked once, met by
every request's rows on the tensor cores, joined with the private keys -- in
the ways a call may be made: launch modes, streams, graphs, workspaces, and bad
data.  Each case takes the shortest prefix that a call of its sizes shares."""
import pytest
import torch

import speculative_decoding_token_rejection_gb300 as sv
import test_gpu_attend
from test_gpu_attend import CASES, check, make, poison, reference, run, verifier
from test_gpu_attend_scales import shared, shared_prefix

pytestmark = pytest.mark.gpu

BITS = sv.DATA_STATUS_BITS
SIZES = {
    "uniform": dict(gammas=[4] * 40, own=[10 + i for i in range(40)], uniform=True),
    "ragged, token-major": dict(gammas=[i % 6 for i in range(70)], own=[4 + 3 * i for i in range(70)], block=8, fmt="e4m3",
                                nhd=True, group=8),
    "narrow heads, some inside it": dict(gammas=[3] * 64, own=[200 - 4 * i for i in range(64)], kv_heads=1, dim=64),
    "many heads, idle requests": dict(gammas=[1] * 200, own=[None if i % 3 == 1 else 2 * i for i in range(200)], kv_heads=8,
                                      group=2, block=32),
}


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


@pytest.mark.parametrize("name", SIZES)
def test_against_the_formula(name):
    check(poison(shared(seed=1, **SIZES[name])))


@pytest.mark.parametrize("name", SIZES)
def test_serial_launch_and_repeats_give_the_same(name):
    c = shared(seed=3, **SIZES[name])
    want = run(c)
    for flags in (0, 0, sv.SV_FLAG_SERIAL_LAUNCH):
        got = run(c, flags=flags)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("flags", [0, sv.SV_FLAG_SERIAL_LAUNCH])
def test_on_another_stream_and_in_a_graph(flags):
    c = shared(seed=16, **SIZES["uniform"])
    want, want_lse, _ = run(c)
    prefix, most = c["prefix"], max(c["lens"])
    ver = verifier(flags)
    out, lse = torch.zeros_like(want), torch.zeros_like(want_lse)
    ws = ver.attend_workspace(num_reqs=40, max_spec_len=4, num_q_heads=8, num_kv_heads=2, head_dim=128, max_seq_len=most,
                              shared_prefix_len=prefix, num_tokens=200)
    ws.fill_(0xFF)  # NaN throughout: what a workspace holds before a call does not matter
    q = c["q"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def call(stream=None):
        ver.attend(q=q, cache=c["cache"], block_tables=c["table"], seq_lens=c["seq_lens"], max_seq_len=most,
                   max_spec_len=4, scale=c["scale"], out=out, lse=lse, shared_prefix_len=prefix, workspace=ws,
                   stream=stream)

    call(side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for _ in range(2):
        out.zero_()
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    q.mul_(0.5)  # the graph reads its inputs anew
    graph.replay()
    torch.cuda.synchronize()
    half = run(dict(c, q=q))
    assert torch.equal(out, half[0]) and torch.equal(lse, half[1]) and not torch.equal(out, want)


def test_calls_of_other_sizes_share_a_workspace():
    calls = [shared(seed=19, **SIZES[name]) for name in SIZES]
    calls += [make([2, 0, 5], [3000, 20, 900], seed=20), make([1, 0], [2500, 2421], prefix=2400, group=2, seed=21)]
    want = [run(c) for c in calls]
    ws = torch.full((1 << 27,), 0xFF, dtype=torch.uint8, device="cuda")
    for i in (0, 4, 1, 5, 2, 3, 0, 1, 3, 2):
        got = run(calls[i], workspace=ws)
        assert torch.equal(got[0], want[i][0]) and torch.equal(got[1], want[i][1])


def test_a_small_workspace_is_refused():
    for c, kw in ((shared(seed=17, **SIZES["uniform"]), {}), (make([1, 0], [2500, 2421], prefix=2400, seed=17), {})):
        N = len(c["gammas"])
        need = sv.spec_verify_attend_workspace_size(
            verifier().handle, num_reqs=N, max_spec_len=c["G"], num_q_heads=8, num_kv_heads=2, head_dim=128,
            max_seq_len=max(c["lens"]), shared_prefix_len=c["prefix"], num_tokens=c["q"].shape[0])
        assert need > 16
        want = run(c)
        got = run(c, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        for n in (16, 1024):
            with pytest.raises(sv.SpecVerifyError) as ei:
                run(c, workspace=torch.empty(n, dtype=torch.uint8, device="cuda"))
            assert ei.value.code == sv.SV_ERR_CAPACITY


def test_nan_key_reaches_only_the_rows_that_see_it():
    c = shared([3] * 40, [3 - i for i in range(40)], uniform=True, seed=11)  # all requests but the first end inside
    clean, clean_lse, _ = run(c)
    page, off = int(c["table"][0, (c["prefix"] - 1) // 16]), 15  # the prefix's last key: position prefix - 1
    c["cache"].k_scale[page, 0, off] = float("nan")
    out, lse, _ = run(c)
    see = torch.tensor([[n - 4 + j >= c["prefix"] - 1 for j in range(4)] for n in c["lens"]]).reshape(-1).cuda()
    assert 0 < int(see.sum()) < see.numel() // 4
    hit = torch.zeros(out.shape[:2], dtype=torch.bool, device="cuda")
    hit[see, :c["group"]] = True
    assert bool(torch.isnan(out[hit]).all()) and bool(torch.isnan(lse[hit]).all())
    assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], clean_lse[~hit])


def grown(gammas, lens, *, prefix=0, **kw):
    """A call whose prefix, if it has one and rows enough, is lengthened to one that is shared."""
    longer = 0
    if prefix and (sum(gammas) + len(gammas)) * kw.get("group", 4) >= 96:
        longer = max(0, shared_prefix(gammas, **kw) - prefix)
    return make(gammas, [n + longer for n in lens], prefix=prefix + longer, **kw)


@pytest.mark.parametrize("name", [n for n, kw in CASES.items() if kw.get("prefix") and
                                  (sum(kw["gammas"]) + len(kw["gammas"])) * kw.get("group", 4) >= 96])
def test_the_formula_s_cases_with_shared_prefixes(name):
    kw = CASES[name]
    check(poison(grown(seed=len(name), **kw)))


@pytest.mark.parametrize("test, args", [
    (test_gpu_attend.test_small_and_large_queries, (1e-3, "int8")),
    (test_gpu_attend.test_small_and_large_queries, (30.0, "e4m3")),
    (test_gpu_attend.test_small_and_large_queries, (3000.0, "int8")),
    (test_gpu_attend.test_value_scales_of_many_sizes, ()), (test_gpu_attend.test_nan_in_a_row_of_q_stays_in_it, ()),
    (test_gpu_attend.test_rows_of_very_different_sizes, ()),
    (test_gpu_attend.test_strided_and_unaligned_queries_and_outputs, ())], ids=lambda x: getattr(x, "__name__", str(x)))
def test_the_same_with_shared_prefixes(test, args, monkeypatch):
    monkeypatch.setattr(test_gpu_attend, "make", grown)
    test(*args)


def test_bad_page_in_a_shared_prefix():
    """Its keys are left out of every row."""
    c = shared([4] * 60, [4 + i for i in range(60)], uniform=True, seed=18)
    cut = dict(c, table=torch.cat([c["table"][:, :5], c["table"][:, 6:]], 1), lens=[n - 16 for n in c["lens"]],
               prefix=c["prefix"] - 16, seq_lens=c["seq_lens"] - 16)
    ref, rlse, tol, ltol = reference(cut)
    c["table"][:, 5] = c["cache"].num_blocks
    out, lse, status = run(c)
    assert status == BITS["BAD_SLOT"]
    assert bool(((out.double() - ref).abs() <= tol).all()) and bool(((lse - rlse).abs() <= ltol).all())


@pytest.mark.parametrize("kv_heads, group", [(1, 4), (2, 4), (1, 16)])
def test_a_workspace_holds_for_fewer_draft_tokens(kv_heads, group):
    N, G = 33, 7
    prefix = shared_prefix([G] * N, kv_heads=kv_heads, group=group, dim=64)
    ver = verifier()

    def size(tokens):
        return sv.spec_verify_attend_workspace_size(ver.handle, num_reqs=N, max_spec_len=G, num_q_heads=kv_heads * group,
                                                    num_kv_heads=kv_heads, head_dim=64, max_seq_len=prefix + 70,
                                                    shared_prefix_len=prefix, num_tokens=tokens)

    sizes = [size(n) for n in range(N, N * (G + 1) + 1)]
    assert sizes == sorted(sizes)
    ws = torch.empty(sizes[-1], dtype=torch.uint8, device="cuda")
    lens = [prefix + 70] + [prefix + i for i in range(N - 1)]
    for few in (0, 2, 6):  # one request with G drafts, the others with `few`
        c = make([G] + [few] * (N - 1), lens, prefix=prefix, kv_heads=kv_heads, group=group, dim=64, seed=few)
        want, got = run(c), run(c, workspace=ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("name", ["private", "shared"])
def test_pages_far_apart(name):
    """One layer's pages of a cache that holds many layers' side by side: 72 GB from the first to the last."""
    c = make([1, 0, 2], [200, 40, 135], block=64, seed=14) if name == "private" else \
        shared([1] * 200, [5 + i % 9 for i in range(200)], kv_heads=8, group=2, block=128, seed=14)
    old = c["cache"]
    n, h, b, d = old.k.shape
    stride = (72 << 30) // n // 128 * 128
    room = torch.empty((n - 1) * stride + 2 * h * b * d, dtype=torch.int8, device="cuda")
    k, v = (room[at:].as_strided((n, h, b, d), (stride, b * d, d, 1)) for at in (0, h * b * d))
    k.copy_(old.k)
    v.copy_(old.v)
    want = run(c)
    got = run(dict(c, cache=sv.KVCache(k=k, v=v, k_scale=old.k_scale, v_scale=old.v_scale)))
    assert got[2] == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
