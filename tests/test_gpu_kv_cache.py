"""The paged 8-bit KV cache on the GPU: quantised writes and reads against the
definition, computed on the CPU with IEEE divisions.  Bytes, scales and read
values have to be equal: every step of the definition is one rounding."""
import numpy as np
import pytest
import torch

import speculative_decoding_token_rejection_gb300 as sv

pytestmark = pytest.mark.gpu

QMAX = {"int8": 127.0, "e4m3": 448.0}
DTYPES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def make_cache(blocks, heads, block, dim, fmt, nhd=False, dev="cuda", fill=0):
    """A cache whose bytes are `fill`, its scales `fill` as well (NaN for 0x7F)."""
    shape = (blocks, block, heads, dim) if nhd else (blocks, heads, block, dim)
    sides = []
    for _ in range(2):
        data = torch.full(shape, fill, dtype=torch.uint8, device=dev).view(DTYPES[fmt])
        scale = torch.full(shape[:-1], float("nan") if fill else 1.0, device=dev)
        sides += [data.permute(0, 2, 1, 3), scale.permute(0, 2, 1)] if nhd else [data, scale]
    return sv.KVCache(k=sides[0], v=sides[2], k_scale=sides[1], v_scale=sides[3])


def quantise(x, fmt):
    """(numbers of the bytes, scales) of fp32 rows [..., D], on the CPU."""
    x = x.cpu()
    finite = torch.isfinite(x).all(-1)
    top = torch.where(finite, x.abs().amax(-1), torch.zeros(()))
    scale = (top / torch.full_like(top, QMAX[fmt])).clamp_min(2.0 ** -64)
    y = torch.where(finite[..., None], x, torch.zeros(())) / scale[..., None]
    y = y.round().clamp(-127, 127) if fmt == "int8" else y.to(torch.float8_e4m3fn).float()
    return y, torch.where(finite, scale, torch.full_like(scale, float("nan")))


def numbers(t):
    raw = (t if t.dtype == torch.int8 else t.view(torch.uint8)).cpu().contiguous()
    return raw.float() if t.dtype == torch.int8 else raw.view(torch.float8_e4m3fn).float()


def same(a, b):
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))


@pytest.fixture(scope="module")
def ver():
    v = sv.Verifier(64, 8, 1000)
    yield v
    v.close()


CASES = [  # tokens, heads, block, dim, layout token-major, rows aligned
    (1, 1, 1, 64, False, True), (1, 8, 16, 128, False, True), (37, 3, 5, 64, True, True), (64, 2, 16, 128, True, False),
    (333, 5, 24, 128, False, False), (250, 1, 7, 64, False, False), (2048, 8, 32, 128, False, True),
]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,heads,block,dim,nhd,aligned", CASES)
def test_write_then_read(ver, T, heads, block, dim, nhd, aligned, dtype, fmt):
    gen = torch.Generator().manual_seed(T * 7 + heads)
    blocks = -(-T // block) + 2
    pad = 0 if aligned else 1
    x = torch.randn(2, T, heads, dim + pad, generator=gen) * torch.exp(3 * torch.randn(2, T, heads, 1, generator=gen))
    x[0, 0, 0] = 0.0  # a zero row
    x[1, T // 2, heads - 1] *= 1e-30  # below the smallest scale
    x[0, T - 1, 0] *= 1e30
    dev = x.to(dtype).cuda()
    key, value = dev[0, :, :, pad:], dev[1, :, :, pad:]
    slots = torch.randperm(blocks * block, generator=gen)[:T]
    gone = torch.rand(T, generator=gen) < 0.25
    slots = torch.where(gone, torch.full_like(slots, -1), slots)
    cache = make_cache(blocks, heads, block, dim, fmt, nhd, fill=1)
    before = [numbers(t).clone() if t.dim() == 4 else t.cpu().clone() for t in (cache.k, cache.v)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ver.kv_write(cache=cache, key=key, value=value, slot_mapping=slots.cuda(), status=status)
    keep = slots >= 0
    page, off = slots[keep] // block, slots[keep] % block
    for x_, data, scale, old in ((key, cache.k, cache.k_scale, before[0]), (value, cache.v, cache.v_scale, before[1])):
        num, sc = quantise(x_.float(), fmt)
        want, want_scale = old.clone(), torch.full(scale.shape, float("nan"))
        want[page, :, off] = num[keep]
        want_scale[page, :, off] = sc[keep]
        assert torch.equal(numbers(data), want)  # the other slots as they were
        assert same(scale.cpu(), want_scale)
        for out_dtype in (torch.bfloat16, torch.float32):
            wide = torch.full((2, T, heads, dim + pad), 7.0, dtype=out_dtype, device="cuda")
            ver.kv_read(cache=cache, slot_mapping=slots.cuda(), key_out=wide[0, :, :, pad:],
                        value_out=wide[1, :, :, pad:], status=status)
            got = wide[0 if x_ is key else 1, :, :, pad:].cpu()
            back = torch.where(keep[:, None, None], num * sc[..., None], torch.zeros(())).to(out_dtype)
            assert torch.equal(got, back)
            assert pad == 0 or bool((wide[..., :pad] == 7.0).all())
    assert int(status.item()) == 0


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_non_finite_rows_read_back_as_nan(ver, fmt):
    x = torch.randn(6, 2, 64, generator=torch.Generator().manual_seed(1))
    x[1, 0, 5], x[2, 1, 63], x[4, 0, 0] = float("nan"), float("inf"), -float("inf")
    slots = torch.arange(6, device="cuda")
    cache = make_cache(2, 2, 4, 64, fmt)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ver.kv_write(cache=cache, key=x.cuda(), value=(-x).cuda(), slot_mapping=slots, status=status)
    assert int(status.item()) == sv.DATA_STATUS_BITS["BAD_VALUES"]
    key, value = ver.kv_read(cache=cache, slot_mapping=slots, dtype=torch.float32)
    num, sc = quantise(x, fmt)
    assert same(key.cpu(), num * sc[..., None])
    assert same(value.cpu(), -num * sc[..., None])
    assert int(torch.isnan(key).sum()) == 3 * 64


def test_bad_slots_are_skipped_and_reported(ver):
    x = torch.randn(5, 1, 64, generator=torch.Generator().manual_seed(2)).cuda()
    slots = torch.tensor([0, 8, -2, 1 << 40, -1], device="cuda")  # the cache has slots 0 .. 7
    cache = make_cache(2, 1, 4, 64, "int8")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ver.kv_write(cache=cache, key=x, value=x, slot_mapping=slots, status=status)
    assert int(status.item()) == sv.DATA_STATUS_BITS["BAD_SLOT"]
    assert int((numbers(cache.k) != 0).any(-1).sum()) == 1
    status.zero_()
    key, _ = ver.kv_read(cache=cache, slot_mapping=slots, status=status)
    assert int(status.item()) == sv.DATA_STATUS_BITS["BAD_SLOT"]
    assert bool((key[1:] == 0).all()) and bool((key[0] != 0).any())
    status.zero_()
    ver.kv_write(cache=cache, key=x, value=x, slot_mapping=torch.full((5,), -1, device="cuda"), status=status)
    assert int(status.item()) == 0


def test_no_tokens(ver):
    cache = make_cache(2, 1, 4, 64, "int8")
    none = torch.empty(0, 1, 64, device="cuda")
    ver.kv_write(cache=cache, key=none, value=none, slot_mapping=torch.empty(0, dtype=torch.int64, device="cuda"))
    torch.cuda.synchronize()


def test_offsets_beyond_32_bits(ver):
    """Pages behind the first 2^32 bytes of a cache."""
    heads, block, dim = 8, 64, 128
    blocks = (1 << 32) // (heads * block * dim) + 3
    k = torch.zeros(blocks, heads, block, dim, dtype=torch.int8, device="cuda")
    scale = torch.ones(blocks, heads, block, device="cuda")
    cache = sv.KVCache(k=k, v=k, k_scale=scale, v_scale=scale)  # one tensor for both sides: equal rows go in
    x = torch.randn(4, heads, dim, generator=torch.Generator().manual_seed(3)).cuda()
    last = blocks * block - 1
    slots = torch.tensor([last, last - 64, 0, 65], device="cuda")
    ver.kv_write(cache=cache, key=x, value=x, slot_mapping=slots)
    num, sc = quantise(x, "int8")
    for t, s in enumerate(slots.tolist()):
        assert torch.equal(k[s // block, :, s % block].cpu().float(), num[t])
    key, _ = ver.kv_read(cache=cache, slot_mapping=slots, dtype=torch.float32)
    assert torch.equal(key.cpu(), num * sc[..., None])


def test_on_another_stream_and_in_a_graph(ver):
    x = torch.randn(40, 2, 128, generator=torch.Generator().manual_seed(4)).cuda()
    cache = make_cache(4, 2, 16, 128, "e4m3")
    slots = torch.arange(40, device="cuda")
    out = torch.empty(2, 40, 2, 128, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ver.kv_write(cache=cache, key=x, value=x, slot_mapping=slots, stream=side)  # (warm-up outside the capture)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ver.kv_write(cache=cache, key=x, value=x, slot_mapping=slots)
        ver.kv_read(cache=cache, slot_mapping=slots, key_out=out[0], value_out=out[1])
    for seed in (5, 6):
        x.copy_(torch.randn(40, 2, 128, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        num, sc = quantise(x, "e4m3")
        assert torch.equal(out[0].cpu(), num * sc[..., None]) and torch.equal(out[0], out[1])


def test_the_verifiers_rollback_keeps_rejected_drafts_out(ver):
    """slot_mapping as spec_verify_run leaves it: rejected drafts' tokens are not written."""
    N, G, V = 3, 4, 50
    gen = torch.Generator().manual_seed(8)
    target = torch.softmax(torch.randn(N * (G + 1), V, generator=gen), -1).cuda()
    draft = torch.softmax(torch.randn(N * G, V, generator=gen), -1).cuda()
    ids = torch.randint(0, V, (N * G,), generator=gen, dtype=torch.int32).cuda()
    slots = torch.arange(N * (G + 1), device="cuda")
    res = ver.verify(entry="probs", draft_ids=ids, target=target, draft=draft, max_spec_len=G, num_reqs=N, seed=1,
                     slot_mapping=slots)
    cache = make_cache(2, 1, 16, 64, "int8")
    x = torch.randn(N * (G + 1), 1, 64, generator=gen).cuda()
    ver.kv_write(cache=cache, key=x, value=x, slot_mapping=slots)
    written = (numbers(cache.k) != 0).any(-1).reshape(-1)[:N * (G + 1)].reshape(N, G + 1)
    keep = torch.arange(G + 1) <= res.num_accepted.cpu()[:, None]
    assert torch.equal(written, keep) and not bool(keep.all())


def test_rows_that_share_a_scale_are_read_not_written(ver):
    """One scale for all tokens of a page and head, expanded: a write would have its tokens race for it."""
    full = make_cache(3, 2, 16, 64, "int8")
    full.k.copy_(torch.randint(-127, 128, full.k.shape, dtype=torch.int8))
    one = torch.tensor([0.5, 0.25, 2.0, 1.0, 3.0, 0.125], device="cuda").view(3, 2, 1)
    slots, x = torch.arange(48, device="cuda"), torch.ones(48, 2, 64, device="cuda")
    for scale in (one.expand(3, 2, 16), one[:, :1].expand(3, 2, 16), torch.ones(1, 1, 1, device="cuda").expand(3, 2, 16)):
        cache = sv.KVCache(k=full.k, v=full.v, k_scale=scale, v_scale=scale)
        key, _ = ver.kv_read(cache=cache, slot_mapping=slots, dtype=torch.float32)
        want = (full.k.float() * scale[..., None]).permute(0, 2, 1, 3).reshape(48, 2, 64)
        assert torch.equal(key, want)
        with pytest.raises(sv.SpecVerifyError) as ei:
            ver.kv_write(cache=cache, key=x, value=x, slot_mapping=slots)
        assert ei.value.code == sv.SV_ERR_INVALID_ARG
        none = torch.empty(0, 2, 64, device="cuda")
        ver.kv_write(cache=cache, key=none, value=none, slot_mapping=slots[:0])
