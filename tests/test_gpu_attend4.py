"""The verify tokens' attention over the paged 4-bit cache against the formula in
64 bits.

Tolerances, from the arithmetic, are those of the 8-bit cache (test_gpu_attend):
a nibble times its group scale is an exact 16-bit operand, as a byte's number is
there.  A score is a sum of D exact products in fp32, off by at most e = 2^-24 *
(D + 32) * max_k scale * sum_d |q_d k_d|; weights are off by 2 e relative, plus
2^-20 for the exponential and the sums, and rounded to 11 bits before they meet
the values; the bf16 output adds half a step.  A weight that underflows 16 bits
loses 2^-25 of the largest product of a weight and its value's scale (a scale's
size enters the exponent as 2^-64 at least), times the value's number without it.  |lse - exact| <= e + 2^-20 * (1 + |exact|)."""
import math

import pytest
import torch

import speculative_decoding_token_rejection_gb300 as sv
import test_gpu_attend as eight
from test_gpu_kv4_cache import E2M1, FORMATS

pytestmark = pytest.mark.gpu

verifier = eight.verifier
CASES = eight.CASES


def random_side4(gen, shape, fmt, nhd):
    """Nibbles of all codes, group scales over a hundredfold range, rows of different sizes."""
    n, h, b, d = shape
    data = torch.randint(0, 256, (n, h, b, d // 2), generator=gen, device="cuda", dtype=torch.uint8)
    group = torch.exp(1.2 * torch.randn(n, h, b, d // 16, generator=gen, device="cuda")).clamp(0.02, 50)
    group = (group * 8).to(torch.float8_e4m3fn)
    scale = torch.exp(0.5 * torch.randn(n, h, b, generator=gen, device="cuda")) / 30
    if nhd:
        data = data.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
        group = group.view(torch.uint8).permute(0, 2, 1, 3).contiguous().view(torch.float8_e4m3fn).permute(0, 2, 1, 3)
        scale = scale.permute(0, 2, 1).contiguous().permute(0, 2, 1)
    return data, group, scale


def make(gammas, lens, *, prefix=0, kv_heads=2, group=4, dim=128, block=16, fmt="e2m1", nhd=False, uniform=False,
         q_gain=1.0, seed=0):
    fmt = {"int8": "int4", "e4m3": "e2m1"}.get(fmt, fmt)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    N = len(gammas)
    need = [max(0, -(-(n - prefix) // block)) for n in lens]
    pre = prefix // block
    blocks = pre + sum(need) + 2
    order = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32).cpu()
    table = torch.full((N, pre + max(need + [1])), 0, dtype=torch.int32)
    at = pre
    for i in range(N):
        table[i, :pre] = order[:pre]
        table[i, pre:pre + need[i]] = order[at:at + need[i]]
        at += need[i]
    k, kg, ks = random_side4(gen, (blocks, kv_heads, block, dim), fmt, nhd)
    v, vg, vs = random_side4(gen, (blocks, kv_heads, block, dim), fmt, nhd)
    rows = sum(gammas) + N
    qkv = torch.randn(rows, kv_heads * group + 3, dim, generator=gen, device="cuda") * q_gain
    return dict(gammas=gammas, lens=lens, prefix=prefix, group=group, table=table.cuda(),
                seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), q=qkv.to(torch.bfloat16)[:, 1:-2],
                cache=sv.KVCache4(k=k, v=v, k_group=kg, v_group=vg, k_scale=ks, v_scale=vs, format=fmt),
                scale=dim ** -0.5, cu=None if uniform else torch.tensor(gammas, device="cuda").cumsum(0).to(torch.int32),
                G=max(gammas + [0]))


def poison(c):
    """Everything that no row may see becomes NaN: pages in no table, and the tails of the last pages."""
    cache, block, pre = c["cache"], c["cache"].block_size, c["prefix"] // c["cache"].block_size
    used = torch.zeros(cache.num_blocks, block, dtype=torch.bool)
    table = c["table"].cpu()
    used[table[0, :pre].long()] = True
    for i, n in enumerate(c["lens"]):
        for t in range(c["prefix"], max(n, 0), block):
            used[table[i, t // block], :min(block, n - t)] = True
    gone = ~used.cuda()[:, None, :].expand(-1, cache.num_kv_heads, -1)
    for group, scale in ((cache.k_group, cache.k_scale), (cache.v_group, cache.v_scale)):
        scale[gone] = float("nan")
        group.view(torch.uint8)[gone] = 0x7F
    return c


run = eight.run


def numbers(data, group, fmt):
    """Nibbles times group scales in 64 bits."""
    code = torch.stack([data & 15, data >> 4], -1).flatten(-2).long()
    if fmt == "int4":
        x = ((code ^ 8) - 8).double()
    else:
        x = E2M1.to(data.device).double()[code & 7] * torch.where(code > 7, -1.0, 1.0)
    return (x.unflatten(-1, (-1, 16)) * group.double()[..., None]).flatten(-2)


def reference(c):
    """(out, lse, tolerance of out, tolerance of lse), in 64 bits."""
    cache, grp = c["cache"], c["group"]
    h, d, b = cache.num_kv_heads, cache.head_dim, cache.block_size
    rows = c["q"].shape[0]
    out = torch.zeros(rows, h, grp, d, dtype=torch.float64, device="cuda")
    lse = torch.full((rows, h, grp), -math.inf, dtype=torch.float64, device="cuda")
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    at = 0
    for i, (g, n) in enumerate(zip(c["gammas"], c["lens"])):
        if n > 0:
            t = torch.arange(n, device="cuda")
            page, off = c["table"][i].long()[t // b], t % b

            def side(data, group, scale):
                raw = group.view(torch.uint8)[page, :, off].view(torch.float8_e4m3fn)
                num = numbers(data[page, :, off], raw, cache.format).permute(1, 0, 2)
                return num, scale[page, :, off].double().t()

            kn, ks = side(cache.k, cache.k_group, cache.k_scale)
            vn, vs = side(cache.v, cache.v_group, cache.v_scale)
            vs = torch.where(vs.abs() < 2.0 ** -64, torch.zeros_like(vs), vs)  # (counts as zero, by definition)
            k, v = kn * ks[..., None], vn * vs[..., None]
            q = c["q"][at:at + g + 1].double().reshape(g + 1, h, grp, d).permute(1, 0, 2, 3).reshape(h, -1, d)
            a = torch.matmul(q, k.transpose(1, 2)) * c["scale"]
            big = (torch.matmul(q.abs(), k.abs().transpose(1, 2)) * abs(c["scale"])).amax(-1)
            pos = n - (g + 1) + torch.arange(g + 1, device="cuda").repeat_interleave(grp)
            a = a.masked_fill(t[None, :] > pos[:, None], -math.inf)
            z = torch.logsumexp(a, -1)
            p = torch.exp(a - torch.where(torch.isinf(z), torch.zeros_like(z), z)[..., None])
            o, e = torch.matmul(p, v), 2.0 ** -24 * (d + 32) * big
            w = (2 * e + 2.0 ** -20 + 2.0 ** -11)[..., None] * torch.matmul(p, v.abs()) + 2.0 ** -8 * o.abs()
            most = (p * vs.abs().clamp_min(2.0 ** -64)[:, None, :]).amax(-1, keepdim=True)
            w = w + 2.0 ** -25 * most * torch.matmul((a > -math.inf).double(), vn.abs())
            y = e + 2.0 ** -20 * (1 + torch.where(torch.isinf(z), torch.zeros_like(z), z).abs())
            for dst, src in ((out, o), (tol, w)):
                dst[at:at + g + 1] = src.reshape(h, g + 1, grp, d).permute(1, 0, 2, 3)
            for dst, src in ((lse, z), (ltol, y)):
                dst[at:at + g + 1] = src.reshape(h, g + 1, grp).permute(1, 0, 2)
        at += g + 1
    return out.reshape(rows, -1, d), lse.reshape(rows, -1), tol.reshape(rows, -1, d), ltol.reshape(rows, -1)


def check(c, status=0, **kw):
    out, lse, got = run(c, **kw)
    ref, rlse, tol, ltol = reference(c)
    assert got == status
    assert torch.equal(torch.isinf(lse), torch.isinf(rlse)) and not bool(torch.isnan(lse).any())
    live = ~torch.isinf(rlse)
    assert bool(((lse.double() - rlse).abs() <= ltol)[live].all())
    assert bool((out.double() - ref).abs().le(tol).all())
    return out, lse


# (as for the 8-bit cache, with row tiles of their own sizes; int8 cases take whole numbers, e4m3 ones E2M1)
MORE = {
    "rows of one tile and of two": dict(gammas=[7, 8, 15, 16, 0], lens=[130, 131, 260, 1000, 9], kv_heads=1, group=8),
    "seventy-two rows": dict(gammas=[8] * 3, lens=[700, 9, 128], kv_heads=2, group=8, fmt="int4", uniform=True),
    "chunks that end inside pages": dict(gammas=[2], lens=[40007], kv_heads=1, group=2, block=24, fmt="int4", dim=64),
    "one request, many keys": dict(gammas=[0], lens=[100001], kv_heads=8, group=1, block=64),
}


@pytest.mark.parametrize("name", [*CASES, *MORE])
def test_against_the_formula(name):
    check(poison(make(seed=len(name), **{**CASES, **MORE}[name])))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", [1, 3, 8, 20])
def test_groups_of_query_heads(group, dim, fmt):
    check(poison(make([0, 3, 1], [300, 77, 128], group=group, dim=dim, fmt=fmt, kv_heads=2, seed=group)))


def test_lengths_around_tiles():
    """Every length from 0 to 260 keys, of one and of several tokens."""
    check(poison(make([0] * 130, list(range(0, 260, 2)), kv_heads=1, group=2, dim=64, seed=2)))
    check(poison(make([i % 4 for i in range(130)], list(range(1, 261, 2)), kv_heads=1, group=2, block=7, seed=3)))


@pytest.mark.parametrize("name", ["ragged, token-major", "prefix, many rows", "prefix, idle requests"])
def test_serial_launch_gives_the_same(name):
    c = make(seed=3, **CASES[name])
    a, b = run(c), run(c, flags=sv.SV_FLAG_SERIAL_LAUNCH)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("name", ["many drafts", "prefix, many rows", "prefix, many rows, e4m3", "long"])
def test_repeats_are_bitwise_equal(name):
    c = make(seed=4, **CASES[name])
    a = run(c)
    for _ in range(3):
        b = run(c)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("gain", [1e-3, 30.0, 3000.0])
@pytest.mark.parametrize("fmt", FORMATS)
def test_small_and_large_queries(gain, fmt):
    check(make([4] * 40, [2300 + i for i in range(40)], prefix=2240, q_gain=gain, fmt=fmt, uniform=True, seed=6))
    check(make([2, 0], [77, 500], q_gain=gain, fmt=fmt, seed=7))


BOTH = [dict(gammas=[3, 1], lens=[400, 90]), dict(gammas=[4] * 40, lens=[2330] * 40, prefix=2240, uniform=True)]


@pytest.mark.parametrize("kw", BOTH)
def test_value_scales_of_many_sizes(kw):
    """Value rows 2^-40 to 2^40 in size, the writer's smallest scale and negative ones among them."""
    c = make(seed=9, **kw)
    s = c["cache"].v_scale
    gen = torch.Generator(device="cuda").manual_seed(1)
    s.mul_(torch.exp2(torch.randint(-40, 41, s.shape, generator=gen, device="cuda").float()))
    s.mul_(torch.where(torch.rand(s.shape, generator=gen, device="cuda") < 0.3, -1.0, 1.0))
    zero = torch.rand(s.shape, generator=gen, device="cuda") < 0.2
    s[zero] = 2.0 ** -64
    c["cache"].v[zero] = 0
    check(c)


@pytest.mark.parametrize("kw", BOTH)
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -70])
def test_value_scales_that_count_as_zero(kw, scale):
    """The key counts in lse and in the weights' sum, its value does not."""
    c = make(seed=22, **kw)
    gen = torch.Generator(device="cuda").manual_seed(2)
    gone = torch.rand(c["cache"].v_scale.shape, generator=gen, device="cuda") < 0.3
    c["cache"].v_scale[gone] = scale
    check(c)


@pytest.mark.parametrize("kw", BOTH)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_value_scales_that_are_no_numbers(kw, bad):
    """out is NaN in the rows that see the key, for its head; lse is not."""
    c = make(seed=23, **kw)
    clean, clean_lse, _ = run(c)
    block = c["cache"].block_size
    at = c["lens"][0] - 2  # seen by all of request 0's rows but the last but one's predecessors
    page, off = int(c["table"][0, at // block]), at % block
    c["cache"].v_scale[page, 1, off] = bad
    out, lse, status = run(c)
    assert status == 0 and torch.equal(lse, clean_lse)
    see = torch.zeros(clean.shape[:2], dtype=torch.bool, device="cuda")
    g = c["gammas"][0]
    see[g - 1:g + 1, c["group"]:] = True
    assert bool(torch.isnan(out[see]).all())
    assert torch.equal(out[~see], clean[~see])


@pytest.mark.parametrize("kw", BOTH)
def test_nan_in_a_row_of_q_stays_in_it(kw):
    c = make(seed=10, **kw)
    clean, _, _ = run(c)
    c["q"] = c["q"].clone()
    c["q"][1, 2, 5] = float("nan")
    out, lse, _ = run(c)
    assert bool(torch.isnan(out[1, 2]).all()) and bool(torch.isnan(lse[1, 2]))
    out[1, 2] = clean[1, 2]
    assert torch.equal(out, clean)


@pytest.mark.parametrize("kw", [dict(gammas=[3, 1, 2], lens=[100, 90, 40]), BOTH[1]])
def test_rows_of_very_different_sizes(kw):
    c = make(seed=21, **kw)
    c["q"] = c["q"].clone()
    c["q"][1, 2] *= 1e30
    c["q"][2] *= 1e-30
    c["q"][3, 1] *= 3e5
    c["q"][4] = 0
    c["q"][5, 0] = 3.3e38
    c["scale"] = 1e-3
    c["cache"].k_scale.mul_(0.01)
    check(c)


def test_nan_key_reaches_only_the_rows_that_see_it():
    c = make([3, 3], [100, 90], block=16, seed=11)
    clean, _, _ = run(c)
    page, off = int(c["table"][0, 98 // 16]), 98 % 16  # seen by verify tokens 2 and 3 of request 0
    c["cache"].k_scale[page, 0, off] = float("nan")
    c["cache"].v_scale[page, 1, off] = float("nan")
    out, lse, _ = run(c)
    assert bool(torch.isnan(out[2:4]).all())
    assert bool(torch.isnan(lse[2:4, :c["group"]]).all())
    out[2:4] = clean[2:4]
    assert torch.equal(out, clean)


def test_all_scores_at_the_lowest_value():
    """Scores of about -2e38 (times log2 e still a float) are numbers, not masks: the row is an average."""
    c = make([0, 1], [50, 40], fmt="int4", kv_heads=1, seed=12)
    c["q"] = torch.ones_like(c["q"])
    c["cache"].k.fill_(0x99)  # -7 twice
    c["cache"].k_group.copy_(torch.full(c["cache"].k_group.shape, 16.0))
    c["cache"].k_scale.fill_(1.0)
    c["scale"] = 1.5e34  # -112 * 128 * 1.5e34 = -2.15e38
    out, lse, status = run(c)
    assert status == 0 and bool(torch.isfinite(lse).all())
    for row, (i, see) in enumerate([(0, 50), (1, 39), (1, 40)]):
        t = torch.arange(see, device="cuda")
        page, off = c["table"][i].long()[t // 16], t % 16
        raw = c["cache"].v_group.view(torch.uint8)[page, 0, off].view(torch.float8_e4m3fn)
        v = numbers(c["cache"].v[page, 0, off], raw, "int4") * c["cache"].v_scale[page, 0, off].double()[:, None]
        assert bool(((out[row].double() - v.mean(0)).abs() <= 2.0 ** -8 * v.mean(0).abs() + 2.0 ** -10 * v.abs().mean(0)).all())


def test_bad_pages_lengths_and_ranges():
    bits = sv.DATA_STATUS_BITS
    c = make([1, 2, 0], [40, 50, 30], seed=13)
    clean, clean_lse, _ = run(c)
    c["table"][1, 1] = c["cache"].num_blocks
    out, lse, status = run(c)
    assert status == bits["BAD_SLOT"]
    assert torch.equal(out[:2], clean[:2]) and torch.equal(out[5:], clean[5:])
    cut = dict(c, table=c["table"].clone(), lens=[40, 34, 30],
               seq_lens=torch.tensor([40, 34, 30], dtype=torch.int32, device="cuda"))
    cut["table"][1, 1], cut["table"][1, 2] = c["table"][1, 2], c["table"][1, 3]
    ref, rlse, tol, ltol = reference(cut)
    assert bool(((out.double() - ref).abs() <= tol)[2:5].all()) and bool(((lse - rlse).abs() <= ltol)[2:5].all())
    c["table"][1, 1] = -7
    assert run(c)[2] == bits["BAD_SLOT"]
    c = make([1, 2, 0], [40, 50, 30], seed=13)
    for bad in (51, -1):
        c["seq_lens"][2] = bad
        out, lse, status = run(c)
        assert status == bits["BAD_PARAM"]
        assert torch.equal(out[:5], clean[:5]) and bool((out[5] == 0).all()) and bool((lse[5] == -math.inf).all())
    c["seq_lens"][2] = 30
    for bad in (9, 0):
        c["cu"][1] = bad
        out, lse, status = run(c)
        assert status & bits["BAD_CU"] and torch.equal(out[:2], clean[:2])


@pytest.mark.parametrize("N", [3, 60])
def test_bad_page_in_a_shared_prefix(N):
    c = make([4] * N, [2500 + i for i in range(N)], prefix=2496, uniform=True, seed=18)
    cut = dict(c, table=torch.cat([c["table"][:, :5], c["table"][:, 6:]], 1), lens=[n - 16 for n in c["lens"]],
               prefix=2480, seq_lens=c["seq_lens"] - 16)
    ref, rlse, tol, ltol = reference(cut)
    c["table"][:, 5] = c["cache"].num_blocks
    out, lse, status = run(c)
    assert status == sv.DATA_STATUS_BITS["BAD_SLOT"]
    assert bool(((out.double() - ref).abs() <= tol).all()) and bool(((lse - rlse).abs() <= ltol).all())


def test_calls_of_other_sizes_share_a_workspace():
    a = make([4] * 60, [2700 + i for i in range(60)], prefix=2640, uniform=True, seed=19)
    b = make([2, 0, 5], [3000, 20, 900], seed=20)
    want_a, want_b = run(a), run(b)
    ws = torch.empty(1 << 27, dtype=torch.uint8, device="cuda")
    for c, want in ((a, want_a), (b, want_b), (a, want_a)):
        got = run(c, workspace=ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_offsets_beyond_32_bits():
    c = make([1, 0], [70, 40], kv_heads=8, block=64, group=1, seed=14)
    old = c["cache"]
    blocks = (1 << 32) // (8 * 64 * 64) + 8
    sides = []
    for data, group, scale in ((old.k, old.k_group, old.k_scale), (old.v, old.v_group, old.v_scale)):
        d = torch.zeros(blocks, 8, 64, 64, dtype=torch.uint8, device="cuda")
        g = torch.zeros(blocks, 8, 64, 8, dtype=torch.uint8, device="cuda")
        s = torch.ones(blocks, 8, 64, device="cuda")
        d[-old.num_blocks:], g[-old.num_blocks:], s[-old.num_blocks:] = data, group.view(torch.uint8), scale
        sides.append((d, g.view(torch.float8_e4m3fn), s))
    (k, kg, ks), (v, vg, vs) = sides
    c["cache"] = sv.KVCache4(k=k, v=v, k_group=kg, v_group=vg, k_scale=ks, v_scale=vs, format="e2m1")
    c["table"] += blocks - old.num_blocks
    # (only the pages of the tables are gathered for the formula)
    check(c)


@pytest.mark.parametrize("kw", BOTH)
def test_strided_and_unaligned_queries_and_outputs(kw):
    c = make(seed=15, **kw)
    clean, _, _ = run(c)
    rows, hq, d = c["q"].shape
    q = torch.zeros(hq, rows, d + 3, dtype=torch.bfloat16, device="cuda").permute(1, 0, 2)[..., 1:d + 1]
    q.copy_(c["q"])
    out = torch.full((hq, rows, d + 3), 5.0, dtype=torch.bfloat16, device="cuda")
    verifier().attend(q=q, cache=c["cache"], block_tables=c["table"], seq_lens=c["seq_lens"],
                      max_seq_len=max(c["lens"]), max_spec_len=c["G"], scale=c["scale"],
                      out=out.permute(1, 0, 2)[..., 3:], cu_num_draft_tokens=c["cu"], shared_prefix_len=c["prefix"])
    assert torch.equal(out.permute(1, 0, 2)[..., 3:], clean)
    assert bool((out[..., :3] == 5.0).all())


def test_rows_of_the_cache_in_wider_memory():
    """Strides between rows and heads that leave gaps."""
    c = make([3, 1], [100, 90], seed=24)
    want = run(c)
    old, sides = c["cache"], []
    for data, group, scale in ((old.k, old.k_group, old.k_scale), (old.v, old.v_group, old.v_scale)):
        n, h, b, d = data.shape
        wide = torch.full((n, h + 1, b, d + 32), 0x7F, dtype=torch.uint8, device="cuda")[:, 1:, :, 32:]
        wide.copy_(data)
        g = torch.full((n, h, b + 2, 2 * group.shape[3]), 0x7F, dtype=torch.uint8, device="cuda")[:, :, 1:-1, :group.shape[3]]
        g.copy_(group.view(torch.uint8))
        s = torch.full((n, b, h, 3), float("nan"), device="cuda")[..., 1].permute(0, 2, 1)
        s.copy_(scale)
        sides.append((wide, g.view(torch.float8_e4m3fn), s))
    (k, kg, ks), (v, vg, vs) = sides
    c["cache"] = sv.KVCache4(k=k, v=v, k_group=kg, v_group=vg, k_scale=ks, v_scale=vs, format=old.format)
    got = run(c)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_on_another_stream_and_in_a_graph():
    c = make([4] * 40, [2330] * 40, prefix=2240, uniform=True, seed=16)
    want, want_lse, _ = run(c)
    ver = verifier()
    out, lse = torch.zeros_like(want), torch.zeros_like(want_lse)
    ws = ver.attend_workspace(cache=c["cache"], num_reqs=40, max_spec_len=4, num_q_heads=8, max_seq_len=2330,
                              shared_prefix_len=2240, num_tokens=200)
    ws.fill_(0xFF)
    q = c["q"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def call(stream=None):
        ver.attend(q=q, cache=c["cache"], block_tables=c["table"], seq_lens=c["seq_lens"], max_seq_len=2330,
                   max_spec_len=4, scale=c["scale"], out=out, lse=lse, shared_prefix_len=2240, workspace=ws,
                   stream=stream)

    call(side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_no_lse_and_small_workspace():
    c = make([2, 1], [5000, 70], seed=17)
    assert torch.equal(run(c, want_lse=False)[0], run(c)[0])
    ver = verifier()
    need = sv.spec_verify_attend_workspace_size(ver.handle, cache=c["cache"], num_reqs=2, max_spec_len=2, num_q_heads=8,
                                                max_seq_len=5000, num_tokens=5)
    assert need > 16
    with pytest.raises(sv.SpecVerifyError) as ei:
        run(c, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert ei.value.code == sv.SV_ERR_CAPACITY


@pytest.mark.parametrize("prefix", [16, 112, 2240])
@pytest.mark.parametrize("fmt", FORMATS)
def test_only_the_first_row_names_the_prefix_pages(prefix, fmt):
    gammas = [2, 0, 4, 1, 3] * (8 if prefix > 2000 else 1)
    c = make(gammas, [prefix + x for x in [40, 0, 3, 300, -5] * (len(gammas) // 5)], prefix=prefix, fmt=fmt, seed=33)
    want = run(c)
    c["table"][1:, :prefix // 16] = torch.tensor([-7, 1 << 30], dtype=torch.int32, device="cuda").repeat(
        prefix // 16)[:prefix // 16]
    got = run(c)
    assert got[2] == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("kv_heads, group, gamma", [(1, 1, 0), (2, 4, 3), (1, 16, 2), (8, 1, 0)])
def test_prefixes_around_the_choice(kv_heads, group, gamma):
    """Shared or read by each request, a prefix gives the same result."""
    N = 30
    for prefix in (96, 128, 480, 1024, 2048):
        check(make([gamma] * N, [prefix + 5 * i for i in range(N)], prefix=prefix, kv_heads=kv_heads, group=group,
                   uniform=True, seed=prefix))


def test_a_workspace_holds_for_fewer_draft_tokens():
    N, G, prefix, kv_heads, group = 33, 7, 4096, 2, 4
    ver, caches = verifier(), make([0], [5], kv_heads=kv_heads, group=group, dim=64)["cache"]

    def size(tokens):
        return sv.spec_verify_attend_workspace_size(ver.handle, cache=caches, num_reqs=N, max_spec_len=G,
                                                    num_q_heads=kv_heads * group, max_seq_len=prefix + 70,
                                                    shared_prefix_len=prefix, num_tokens=tokens)

    sizes = [size(n) for n in range(N, N * (G + 1) + 1)]
    assert sizes == sorted(sizes)
    ws = torch.empty(sizes[-1], dtype=torch.uint8, device="cuda")
    lens = [prefix + 70] + [prefix + i for i in range(N - 1)]
    for few in (0, 1, 2, 6):  # one request with G drafts, the others with `few`
        c = make([G] + [few] * (N - 1), lens, prefix=prefix, kv_heads=kv_heads, group=group, dim=64, seed=few)
        want, got = run(c), run(c, workspace=ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kw,G", [
    (dict(gammas=[0] * 16, lens=[16384 + i for i in range(16)], prefix=16384, kv_heads=8), 0),
    (dict(gammas=[0] * 20, lens=[70000 + 40 * i for i in range(20)], prefix=70000, kv_heads=1, group=1, dim=64), 0),
    # ragged batches: there may be rows enough to share it, but few are there
    (dict(gammas=[0] * 40, lens=[16400 + i for i in range(40)], prefix=16400, group=1), 4),
    (dict(gammas=[0] * 30 + [3], lens=[0] * 20 + [16400] * 10 + [16403], prefix=16400, group=2, dim=64), 8),
])
def test_a_prefix_that_few_rows_share(kw, G, fmt):
    c = make(seed=25, fmt=fmt, **kw)
    c["G"] = max(G, c["G"])
    check(poison(c))


@pytest.mark.parametrize("gammas", [[8] + [0] * 9, [15, 3, 0, 0, 0, 1], [40] + [0] * 20, [5] * 4 + [8]])
def test_ragged_batches_with_a_few_long_requests(gammas):
    """Tiles of fewer rows than the longest request has, or not."""
    check(poison(make(gammas, [700 + 50 * i for i in range(len(gammas))], group=4, kv_heads=1, seed=26)))


def test_workspace_size_refuses_what_the_call_does():
    import ctypes
    lib, n = sv.load_library(), ctypes.c_int64()

    def size(**kw):
        a = sv.SpecVerifyAttend4Args()
        a.num_reqs, a.max_spec_len, a.num_q_heads, a.max_seq_len, a.num_draft_tokens_total = 3, 2, 8, 100, 6
        a.cache.num_kv_heads, a.cache.head_dim = 2, 128
        for name, value in kw.items():
            setattr(a.cache if hasattr(a.cache, name) else a, name, value)
        return lib.spec_verify_attend4_workspace_size(verifier().handle, ctypes.byref(a), ctypes.byref(n))

    assert size() == 0
    for kw in (dict(num_kv_heads=0), dict(num_kv_heads=3), dict(num_reqs=-1), dict(max_seq_len=-1), dict(head_dim=0)):
        assert size(**kw) != 0
    assert size(num_reqs=0, num_draft_tokens_total=0, num_kv_heads=1) == 0 and n.value == 0
