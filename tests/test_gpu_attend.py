"""The verify tokens' attention over the paged 8-bit cache against the formula
in 64 bits.

Tolerances, from the arithmetic.  A score is a sum of D exact products in
fp32: its error is at most e = 2^-24 * (D + 32) * max_k scale * sum_d |q_d k_d|
(the 32 for the scale factors, the subtraction of the maximum and the base-2
exponent).  Weights are off by 2 e relative, plus 2^-20 for the exponential and
the sums, and are rounded to 11 bits before they meet the values (2^-11); so
|out - exact| <= (2 e + 2^-20 + 2^-11) * sum_k p_k |v_k| + 2^-8 |exact|, the last
term for the bf16 output.  The 16-bit weights have steps of 2^-24 of the
largest product of a weight and its value's scale, w: with b_k the value bytes'
numbers, 2^-25 * w * sum_k |b_k| more where weights underflow.  |lse - exact| <= e + 2^-20 * (1 + |exact|)."""
import math

import pytest
import torch

import speculative_decoding_token_rejection_gb300 as sv
from test_gpu_kv_cache import DTYPES, QMAX

pytestmark = pytest.mark.gpu

VER = {}


def verifier(flags=0):
    if flags not in VER:
        VER[flags] = sv.Verifier(1 << 16, sv.SV_MAX_SPEC_LEN, 8, flags=flags)
    return VER[flags]


def random_side(gen, shape, fmt, nhd):
    """Cache bytes and scales; the rows' sizes differ widely."""
    n, h, b, d = shape
    x = torch.randn(n, h, b, d, generator=gen, device="cuda")
    top = x.abs().amax(-1) / QMAX[fmt]
    y = x / top[..., None]
    data = y.round().to(torch.int8) if fmt == "int8" else y.to(torch.float8_e4m3fn)
    scale = top * torch.exp(0.5 * torch.randn(n, h, b, generator=gen, device="cuda"))
    if nhd:
        raw = data.view(torch.uint8).permute(0, 2, 1, 3).contiguous().view(DTYPES[fmt])
        return raw.permute(0, 2, 1, 3), scale.permute(0, 2, 1).contiguous().permute(0, 2, 1)
    return data, scale


def make(gammas, lens, *, prefix=0, kv_heads=2, group=4, dim=128, block=16, fmt="int8", nhd=False, uniform=False,
         q_gain=1.0, seed=0):
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
    k, ks = random_side(gen, (blocks, kv_heads, block, dim), fmt, nhd)
    v, vs = random_side(gen, (blocks, kv_heads, block, dim), fmt, nhd)
    rows = sum(gammas) + N
    qkv = torch.randn(rows, kv_heads * group + 3, dim, generator=gen, device="cuda") * q_gain
    return dict(gammas=gammas, lens=lens, prefix=prefix, group=group, table=table.cuda(),
                seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), q=qkv.to(torch.bfloat16)[:, 1:-2],
                cache=sv.KVCache(k=k, v=v, k_scale=ks, v_scale=vs), scale=dim ** -0.5,
                cu=None if uniform else torch.tensor(gammas, device="cuda").cumsum(0).to(torch.int32),
                G=max(gammas + [0]))


def poison(c):
    """Everything that no row may see becomes NaN (scales; bytes too in e4m3):
    pages in no table, and the tails of the last pages."""
    cache, block, pre = c["cache"], c["cache"].block_size, c["prefix"] // c["cache"].block_size
    used = torch.zeros(cache.num_blocks, block, dtype=torch.bool)
    table = c["table"].cpu()
    used[table[0, :pre].long()] = True
    for i, n in enumerate(c["lens"]):
        for t in range(c["prefix"], max(n, 0), block):
            used[table[i, t // block], :min(block, n - t)] = True
    gone = ~used.cuda()[:, None, :].expand(-1, cache.num_kv_heads, -1)
    for data, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        scale[gone] = float("nan")
        raw = data.view(torch.uint8) if data.dtype != torch.int8 else data
        raw[gone] = 0x7F
    return c


def run(c, *, flags=0, stream=None, want_lse=True, workspace=None):
    ver = verifier(flags)
    rows, hq = c["q"].shape[:2]
    out = torch.full((rows, hq, c["cache"].head_dim), 777.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((rows, hq), 777.0, device="cuda") if want_lse else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ver.attend(q=c["q"], cache=c["cache"], block_tables=c["table"], seq_lens=c["seq_lens"],
               max_seq_len=max(max(c["lens"] + [0]), c["prefix"]), max_spec_len=c["G"], scale=c["scale"], out=out,
               cu_num_draft_tokens=c["cu"], shared_prefix_len=c["prefix"], lse=lse, status=status, stream=stream,
               workspace=workspace)
    torch.cuda.synchronize()
    return out, lse, int(status.item())


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

            def side(data, scale):
                raw = (data if data.dtype == torch.int8 else data.view(torch.uint8))[page, :, off]
                x = raw.double() if data.dtype == torch.int8 else raw.view(torch.float8_e4m3fn).double()
                return (x * scale[page, :, off].double()[..., None]).permute(1, 0, 2)

            k, v = side(cache.k, cache.k_scale), side(cache.v, cache.v_scale)
            q = c["q"][at:at + g + 1].double().reshape(g + 1, h, grp, d).permute(1, 0, 2, 3).reshape(h, -1, d)
            a = torch.matmul(q, k.transpose(1, 2)) * c["scale"]
            big = (torch.matmul(q.abs(), k.abs().transpose(1, 2)) * abs(c["scale"])).amax(-1)
            pos = n - (g + 1) + torch.arange(g + 1, device="cuda").repeat_interleave(grp)
            a = a.masked_fill(t[None, :] > pos[:, None], -math.inf)
            z = torch.logsumexp(a, -1)
            p = torch.exp(a - torch.where(torch.isinf(z), torch.zeros_like(z), z)[..., None])
            o, e = torch.matmul(p, v), 2.0 ** -24 * (d + 32) * big
            w = (2 * e + 2.0 ** -20 + 2.0 ** -11)[..., None] * torch.matmul(p, v.abs()) + 2.0 ** -8 * o.abs()
            vs = cache.v_scale[page, :, off].double().t()[:, None, :]
            most = (p * vs).amax(-1, keepdim=True)
            w = w + 2.0 ** -25 * most * torch.matmul((a > -math.inf).double(), v.abs() / vs.transpose(1, 2))
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


CASES = {
    "one token, one key": dict(gammas=[0], lens=[1]),
    "one token, a thousand keys": dict(gammas=[0], lens=[1000], kv_heads=8),
    "no keys": dict(gammas=[0, 2], lens=[0, 0]),
    "rows before the first key": dict(gammas=[5, 3, 0], lens=[3, 1, 2], group=3),
    "around a tile": dict(gammas=[1, 2, 3, 4, 5], lens=[15, 16, 17, 63, 64], block=7, fmt="e4m3"),
    "around larger tiles": dict(gammas=[4] * 6, lens=[127, 128, 129, 255, 256, 257], uniform=True, dim=64, fmt="e4m3"),
    "ragged, token-major": dict(gammas=[0, 8, 3, 1], lens=[700, 33, 1, 2051], nhd=True, group=1, kv_heads=3, block=24),
    "group of seven": dict(gammas=[3, 0, 7], lens=[100, 300, 17], group=7, kv_heads=1),
    "group of sixteen": dict(gammas=[7, 2], lens=[400, 90], group=16, kv_heads=1, dim=64),
    "many drafts": dict(gammas=[40, 3], lens=[600, 70], group=4, kv_heads=1, fmt="e4m3"),
    "the longest draft": dict(gammas=[256], lens=[257], group=2, kv_heads=1, dim=64),
    "page of one token": dict(gammas=[2, 1], lens=[50, 9], block=1),
    "large pages": dict(gammas=[2, 1], lens=[300, 900], block=512, nhd=True),
    "long": dict(gammas=[4, 0], lens=[20011, 12345], kv_heads=1, group=8),
    "many requests": dict(gammas=[1] * 200, lens=[1 + 13 * (i % 40) for i in range(200)], kv_heads=1, dim=64),
    "prefix alone": dict(gammas=[0, 0], lens=[32, 32], prefix=32),
    "prefix, some shorter than it": dict(gammas=[3, 3, 3], lens=[40, 34, 66], prefix=64, block=16),
    "prefix, idle requests": dict(gammas=[2, 0, 0, 1], lens=[70, 0, 65, 64], prefix=64, fmt="e4m3"),
    "prefix of one page": dict(gammas=[4] * 40, lens=[24 + i for i in range(40)], prefix=16, uniform=True),
    "prefix, small batch": dict(gammas=[4] * 6, lens=[1100 + 7 * i for i in range(6)], prefix=1056, block=24, dim=64),
    "prefix, many rows": dict(gammas=[4] * 50, lens=[1030 + 3 * i for i in range(50)], prefix=1024, uniform=True),
    "prefix, many rows, e4m3": dict(gammas=[i % 6 for i in range(70)], lens=[2100 + 3 * i for i in range(70)],
                                    prefix=2096, block=8, fmt="e4m3", nhd=True, group=8),
    "prefix, many rows, narrow heads": dict(gammas=[7] * 33, lens=[510 + i for i in range(33)], prefix=480, block=32,
                                            dim=64, fmt="e4m3", group=5),
    "prefix, many rows, one tile and a bit": dict(gammas=[0] * 300, lens=[145 + (i % 3) for i in range(300)],
                                                  prefix=144, uniform=True, kv_heads=1, group=3),
    "prefix, many rows, some inside it": dict(gammas=[3] * 64, lens=[300 - 4 * i for i in range(64)], prefix=272,
                                              group=4, kv_heads=1),
    "prefix, one row tile": dict(gammas=[0] * 25, lens=[400 + i for i in range(25)], prefix=384, kv_heads=3, group=4,
                                 uniform=True),
    "prefix, a last row tile of its own": dict(gammas=[0] * 75, lens=[25730 + i % 5 for i in range(75)], prefix=25728,
                                               kv_heads=1, group=4, dim=64, fmt="e4m3", uniform=True),
    "prefix, long": dict(gammas=[7] * 32, lens=[9000 + i for i in range(32)], prefix=8992, kv_heads=1, group=8,
                         uniform=True),
}


@pytest.mark.parametrize("name", CASES)
def test_against_the_formula(name):
    check(poison(make(seed=len(name), **CASES[name])))


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
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_small_and_large_queries(gain, fmt):
    """Flat and one-hot softmaxes; 3000 passes the range of 16-bit floats inside a row."""
    check(make([4] * 40, [200 + i for i in range(40)], prefix=192, q_gain=gain, fmt=fmt, uniform=True, seed=6))
    check(make([2, 0], [77, 500], q_gain=gain, fmt=fmt, seed=7))


def test_value_scales_of_many_sizes():
    """Value rows 2^-40 to 2^40 in size, zero rows (the writer's smallest scale) among them."""
    for kw in (dict(gammas=[3, 1], lens=[400, 90]),
               dict(gammas=[4] * 40, lens=[330] * 40, prefix=320, uniform=True)):
        c = make(seed=9, **kw)
        s = c["cache"].v_scale
        gen = torch.Generator(device="cuda").manual_seed(1)
        s.mul_(torch.exp2(torch.randint(-40, 41, s.shape, generator=gen, device="cuda").float()))
        zero = torch.rand(s.shape, generator=gen, device="cuda") < 0.2
        s[zero] = 2.0 ** -64
        c["cache"].v[zero] = 0
        check(c)


def test_nan_in_a_row_of_q_stays_in_it():
    for kw in (dict(gammas=[3, 1], lens=[100, 90]),
               dict(gammas=[4] * 40, lens=[330] * 40, prefix=320, uniform=True)):
        c = make(seed=10, **kw)
        clean, _, _ = run(c)
        c["q"] = c["q"].clone()
        c["q"][1, 2, 5] = float("nan")
        out, lse, _ = run(c)
        assert bool(torch.isnan(out[1, 2]).all()) and bool(torch.isnan(lse[1, 2]))
        out[1, 2] = clean[1, 2]
        assert torch.equal(out, clean)


def test_rows_of_very_different_sizes():
    """Every row has its own range: one of 1e30 (an idle request's left-overs, say) takes nothing from its neighbours."""
    for kw in (dict(gammas=[3, 1, 2], lens=[100, 90, 40]),
               dict(gammas=[4] * 40, lens=[330] * 40, prefix=320, uniform=True)):
        c = make(seed=21, **kw)
        c["q"] = c["q"].clone()
        c["q"][1, 2] *= 1e30
        c["q"][2] *= 1e-30
        c["q"][3, 1] *= 3e5
        c["q"][4] = 0
        c["q"][5, 0] = 3.3e38
        c["scale"] = 1e-3
        check(c)


def test_nan_key_reaches_only_the_rows_that_see_it():
    for kw in (dict(gammas=[3, 3], lens=[100, 90], block=16),
               dict(gammas=[3] * 40, lens=[100] * 40, prefix=64, uniform=True, block=16)):
        c = make(seed=11, **kw)
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
    """Scores of -2e38 (times log2 e still a float) are numbers, not masks: the row is an average."""
    c = make([0, 1], [50, 40], fmt="int8", kv_heads=1, seed=12)
    c["q"] = torch.ones_like(c["q"])
    c["cache"].k.fill_(-100)
    c["cache"].k_scale.fill_(1.0)
    c["scale"] = 1.7e34  # -100 * 128 * 1.7e34 = -2.2e38
    out, lse, status = run(c)
    assert status == 0 and bool(torch.isfinite(lse).all())
    # every weight of a row is the same: the mean of the values (bf16, and 11-bit weights)
    for row, (i, see) in enumerate([(0, 50), (1, 39), (1, 40)]):
        t = torch.arange(see, device="cuda")
        page, off = c["table"][i].long()[t // 16], t % 16
        v = c["cache"].v[page, 0, off].double() * c["cache"].v_scale[page, 0, off].double()[:, None]
        assert bool(((out[row].double() - v.mean(0)).abs() <= 2.0 ** -8 * v.mean(0).abs() + 2.0 ** -10 * v.abs().mean(0)).all())


def test_bad_pages_lengths_and_ranges():
    bits = sv.DATA_STATUS_BITS
    c = make([1, 2, 0], [40, 50, 30], seed=13)
    clean, clean_lse, _ = run(c)
    # a page outside the cache: its keys are left out
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
    # a length outside [0, max_seq_len]
    c = make([1, 2, 0], [40, 50, 30], seed=13)
    for bad in (51, -1):
        c["seq_lens"][2] = bad
        out, lse, status = run(c)
        assert status == bits["BAD_PARAM"]
        assert torch.equal(out[:5], clean[:5]) and bool((out[5] == 0).all()) and bool((lse[5] == -math.inf).all())
    c["seq_lens"][2] = 30
    # prefix sums that do not fit: the request's rows are left alone
    c["cu"][1] = 9
    out, lse, status = run(c)
    assert status & bits["BAD_CU"]
    assert torch.equal(out[:2], clean[:2])
    c["cu"][1] = 0
    out, lse, status = run(c)
    assert status & bits["BAD_CU"] and torch.equal(out[:2], clean[:2])


def test_bad_page_in_a_shared_prefix():
    """Its keys are left out of every row, in both ways of reading a prefix."""
    for N in (3, 60):
        c = make([4] * N, [400 + i for i in range(N)], prefix=384, uniform=True, seed=18)
        cut = dict(c, table=torch.cat([c["table"][:, :5], c["table"][:, 6:]], 1), lens=[n - 16 for n in c["lens"]],
                   prefix=368, seq_lens=c["seq_lens"] - 16)
        ref, rlse, tol, ltol = reference(cut)
        c["table"][:, 5] = c["cache"].num_blocks
        out, lse, status = run(c)
        assert status == sv.DATA_STATUS_BITS["BAD_SLOT"]
        assert bool(((out.double() - ref).abs() <= tol).all()) and bool(((lse - rlse).abs() <= ltol).all())


def test_calls_of_other_sizes_share_a_workspace():
    a = make([4] * 60, [700 + i for i in range(60)], prefix=640, uniform=True, seed=19)
    b = make([2, 0, 5], [3000, 20, 900], seed=20)
    want_a, want_b = run(a), run(b)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    for c, want in ((a, want_a), (b, want_b), (a, want_a)):
        got = run(c, workspace=ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_offsets_beyond_32_bits():
    c = make([1, 0], [70, 40], kv_heads=8, block=64, group=1, seed=14)
    old = c["cache"]
    blocks = (1 << 32) // (8 * 64 * 128) + 8
    sides = []
    for data, scale in ((old.k, old.k_scale), (old.v, old.v_scale)):
        d = torch.zeros(blocks, 8, 64, 128, dtype=torch.int8, device="cuda")
        s = torch.ones(blocks, 8, 64, device="cuda")
        d[-old.num_blocks:], s[-old.num_blocks:] = data, scale
        sides += [d, s]
    c["cache"] = sv.KVCache(k=sides[0], v=sides[2], k_scale=sides[1], v_scale=sides[3])
    c["table"] += blocks - old.num_blocks
    check(c)


def test_strided_and_unaligned_queries_and_outputs():
    for kw in (dict(gammas=[3, 1], lens=[100, 90]),
               dict(gammas=[4] * 40, lens=[330] * 40, prefix=320, uniform=True)):
        c = make(seed=15, **kw)
        clean, _, _ = run(c)
        rows, hq, d = c["q"].shape
        q = torch.zeros(hq, rows, d + 3, dtype=torch.bfloat16, device="cuda").permute(1, 0, 2)[..., 1:d + 1]
        q.copy_(c["q"])
        out = torch.full((hq, rows, d + 3), 5.0, dtype=torch.bfloat16, device="cuda")
        verifier().attend(q=q, cache=c["cache"], block_tables=c["table"], seq_lens=c["seq_lens"],
                          max_seq_len=max(c["lens"]), max_spec_len=c["G"], scale=c["scale"],
                          out=out.permute(1, 0, 2)[..., 3:], cu_num_draft_tokens=c["cu"],
                          shared_prefix_len=c["prefix"])
        assert torch.equal(out.permute(1, 0, 2)[..., 3:], clean)
        assert bool((out[..., :3] == 5.0).all())


def test_on_another_stream_and_in_a_graph():
    c = make([4] * 40, [330] * 40, prefix=320, uniform=True, seed=16)
    want, want_lse, _ = run(c)
    ver = verifier()
    out, lse = torch.zeros_like(want), torch.zeros_like(want_lse)
    ws = ver.attend_workspace(num_reqs=40, max_spec_len=4, num_q_heads=8, num_kv_heads=2, head_dim=128,
                              max_seq_len=330, shared_prefix_len=320, num_tokens=200)
    ws.fill_(0xFF)  # what a workspace holds before a call does not matter
    q = c["q"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def call(stream=None):
        ver.attend(q=q, cache=c["cache"], block_tables=c["table"], seq_lens=c["seq_lens"], max_seq_len=330,
                   max_spec_len=4, scale=c["scale"], out=out, lse=lse, shared_prefix_len=320, workspace=ws,
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
    c = make([2, 1], [50, 70], prefix=32, seed=17)
    assert torch.equal(run(c, want_lse=False)[0], run(c)[0])
    ver = verifier()
    need = sv.spec_verify_attend_workspace_size(ver.handle, num_reqs=2, max_spec_len=2, num_q_heads=8, num_kv_heads=2,
                                                head_dim=128, max_seq_len=70, shared_prefix_len=32, num_tokens=5)
    if need > 16:
        with pytest.raises(sv.SpecVerifyError) as ei:
            run(c, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
        assert ei.value.code == sv.SV_ERR_CAPACITY


@pytest.mark.parametrize("prefix", [16, 48, 112, 320])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_only_the_first_row_names_the_prefix_pages(prefix, fmt):
    c = make([2, 0, 4, 1, 3], [prefix + 40, prefix, prefix + 3, prefix + 300, prefix - 5], prefix=prefix, fmt=fmt, seed=33)
    want = run(c)
    c["table"][1:, :prefix // 16] = torch.tensor([-7, 1 << 30], dtype=torch.int32, device="cuda").repeat(
        prefix // 16)[:prefix // 16]
    got = run(c)
    assert got[2] == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    check(poison(make([2, 0, 4, 1, 3], c["lens"], prefix=prefix, fmt=fmt, seed=33)))


# Short prefixes are read by each request for itself: the same with prefixes that are shared at these sizes.
LONGER = 2112  # a multiple of every block size here


def long_make(gammas, lens, *, prefix=0, **kw):
    more = LONGER if prefix else 0
    return make(gammas, [n + more for n in lens], prefix=prefix + more, **kw)


@pytest.mark.parametrize("name", [n for n in CASES if 0 < CASES[n].get("prefix", 0) < 2048])
def test_longer_prefixes(name):
    check(poison(long_make(seed=len(name), **CASES[name])))


@pytest.mark.parametrize("test, args", [
    (test_small_and_large_queries, (1e-3, "int8")), (test_small_and_large_queries, (30.0, "e4m3")),
    (test_small_and_large_queries, (3000.0, "int8")), (test_value_scales_of_many_sizes, ()),
    (test_nan_in_a_row_of_q_stays_in_it, ()), (test_rows_of_very_different_sizes, ()),
    (test_strided_and_unaligned_queries_and_outputs, ())], ids=lambda x: getattr(x, "__name__", str(x)))
def test_the_same_with_longer_prefixes(test, args, monkeypatch):
    short = make
    monkeypatch.setitem(globals(), "make", lambda gammas, lens, *, prefix=0, **kw: short(
        gammas, [n + (LONGER if prefix else 0) for n in lens], prefix=prefix + (LONGER if prefix else 0), **kw))
    test(*args)


def test_bad_page_in_a_longer_prefix():
    for N in (3, 60):
        c = make([4] * N, [2500 + i for i in range(N)], prefix=2496, uniform=True, seed=18)
        cut = dict(c, table=torch.cat([c["table"][:, :5], c["table"][:, 6:]], 1), lens=[n - 16 for n in c["lens"]],
                   prefix=2480, seq_lens=c["seq_lens"] - 16)
        ref, rlse, tol, ltol = reference(cut)
        c["table"][:, 5] = c["cache"].num_blocks
        out, lse, status = run(c)
        assert status == sv.DATA_STATUS_BITS["BAD_SLOT"]
        assert bool(((out.double() - ref).abs() <= tol).all()) and bool(((lse - rlse).abs() <= ltol).all())


@pytest.mark.parametrize("kv_heads, group, gamma", [(1, 1, 0), (2, 4, 3), (1, 16, 2), (8, 1, 0)])
def test_prefixes_around_the_choice(kv_heads, group, gamma):
    """Shared or read by each request, a prefix gives the same result."""
    N = 30
    for prefix in (96, 128, 256, 480, 1024, 2032, 2048):
        check(make([gamma] * N, [prefix + 5 * i for i in range(N)], prefix=prefix, kv_heads=kv_heads, group=group,
                   uniform=True, seed=prefix))


@pytest.mark.parametrize("kv_heads, group", [(1, 4), (2, 4), (1, 16)])
def test_a_workspace_holds_for_fewer_draft_tokens(kv_heads, group):
    N, G, prefix = 33, 7, 4096
    ver = verifier()

    def size(tokens):
        return sv.spec_verify_attend_workspace_size(ver.handle, num_reqs=N, max_spec_len=G, num_q_heads=kv_heads * group,
                                                    num_kv_heads=kv_heads, head_dim=64, max_seq_len=prefix + 70,
                                                    shared_prefix_len=prefix, num_tokens=tokens)

    sizes = [size(n) for n in range(N, N * (G + 1) + 1)]
    assert sizes == sorted(sizes)
    ws = torch.empty(sizes[-1], dtype=torch.uint8, device="cuda")
    lens = [prefix + 70] + [prefix + i for i in range(N - 1)]
    for few in (0, 1, 2, 3, 6):  # one request with G drafts, the others with `few`
        c = make([G] + [few] * (N - 1), lens, prefix=prefix, kv_heads=kv_heads, group=group, dim=64, seed=few)
        want, got = run(c), run(c, workspace=ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
