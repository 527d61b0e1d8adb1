"""The paged 4-bit KV cache on the GPU: quantised writes and reads against the
definition, computed on the CPU with IEEE divisions.  Nibbles, group scales, row
scales and read values have to be equal: every step of the definition is one
rounding."""
import pytest
import torch

import speculative_decoding_token_rejection_gb300 as sv

pytestmark = pytest.mark.gpu

Q = {"e2m1": 6.0, "int4": 7.0}
E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
FORMATS = ["e2m1", "int4"]


def make_cache4(blocks, heads, block, dim, fmt, nhd=False, dev="cuda", fill=0):
    """A cache whose bytes are `fill` (scales 1, or NaN for a fill)."""
    lead = (blocks, block, heads) if nhd else (blocks, heads, block)
    sides = []
    for _ in range(2):
        data = torch.full(lead + (dim // 2,), fill, dtype=torch.uint8, device=dev)
        group = torch.full(lead + (dim // 16,), fill, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)
        scale = torch.full(lead, float("nan") if fill else 1.0, device=dev)
        if nhd:
            data, group, scale = data.permute(0, 2, 1, 3), group.permute(0, 2, 1, 3), scale.permute(0, 2, 1)
        sides.append((data, group, scale))
    (k, kg, ks), (v, vg, vs) = sides
    return sv.KVCache4(k=k, v=v, k_group=kg, v_group=vg, k_scale=ks, v_scale=vs, format=fmt)


def codes_of(z, fmt):
    """Nibbles of quotients: to the nearest number of the format, ties to the even code."""
    if fmt == "int4":
        return (z.round().clamp(-7, 7).to(torch.int32) & 15).to(torch.uint8)
    a, code = z.abs(), torch.zeros_like(z, dtype=torch.uint8)
    for i in range(7):
        mid = (E2M1[i] + E2M1[i + 1]) / 2
        code += (a >= mid if i % 2 else a > mid).to(torch.uint8)
    return code | (torch.signbit(z).to(torch.uint8) << 3)


def numbers_of(codes, fmt):
    c = codes.long()
    if fmt == "int4":
        return ((c ^ 8) - 8).float()
    return E2M1[c & 7] * torch.where(c > 7, -1.0, 1.0)


def quantise4(x, fmt):
    """(nibbles, group scales, row scales) of fp32 rows [..., D], on the CPU."""
    x = x.cpu()
    finite = torch.isfinite(x).all(-1)
    x = torch.where(finite[..., None], x, torch.zeros(()))
    top = x.abs().amax(-1)
    scale = (top / torch.full_like(top, 448 * Q[fmt])).clamp_min(2.0 ** -64)
    y = x.unflatten(-1, (-1, 16))
    group = (y.abs().amax(-1) / (scale * Q[fmt])[..., None]).to(torch.float8_e4m3fn)
    unit = (group.float() * scale[..., None])[..., None]
    z = torch.where(unit > 0, y / unit, torch.zeros(())).flatten(-2)
    return codes_of(z, fmt), group, torch.where(finite, scale, torch.full_like(scale, float("nan")))


def values4(codes, group, scale, fmt):
    x = numbers_of(codes, fmt).unflatten(-1, (-1, 16)) * group.float()[..., None]
    return x.flatten(-2) * scale[..., None]


def unpack(data):
    """Nibbles [..., D] of bytes."""
    data = data.cpu()
    return torch.stack([data & 15, data >> 4], -1).flatten(-2)


def plain_zero(codes, fmt):
    """Codes with one zero (the sign of a zero is not part of the definition)."""
    return torch.where(codes == 8, torch.zeros_like(codes), codes) if fmt == "e2m1" else codes


def same(a, b):
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))


def raw(t):
    return t.view(torch.uint8).cpu()


@pytest.fixture(scope="module")
def ver():
    v = sv.Verifier(64, 8, 1000)
    yield v
    v.close()


CASES = [  # tokens, heads, block, dim, layout token-major, rows aligned
    (1, 1, 1, 64, False, True), (1, 8, 16, 128, False, True), (37, 3, 5, 64, True, True), (64, 2, 16, 128, True, False),
    (333, 5, 24, 128, False, False), (250, 1, 7, 64, False, False), (2048, 8, 32, 128, False, True),
]


@pytest.mark.parametrize("fmt", FORMATS)
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
    x[1, 0, 0, 16 + pad:32 + pad] *= 1e-9  # a group whose scale rounds to zero beside the others
    dev = x.to(dtype).cuda()
    key, value = dev[0, :, :, pad:], dev[1, :, :, pad:]
    slots = torch.randperm(blocks * block, generator=gen)[:T]
    gone = torch.rand(T, generator=gen) < 0.25
    slots = torch.where(gone, torch.full_like(slots, -1), slots)
    cache = make_cache4(blocks, heads, block, dim, fmt, nhd, fill=1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ver.kv_write(cache=cache, key=key, value=value, slot_mapping=slots.cuda(), status=status)
    keep = slots >= 0
    page, off = slots[keep] // block, slots[keep] % block
    for side, x_, data, group, scale in ((0, key, cache.k, cache.k_group, cache.k_scale),
                                         (1, value, cache.v, cache.v_group, cache.v_scale)):
        code, g, sc = quantise4(x_.float(), fmt)
        want = torch.ones(data.shape, dtype=torch.uint8)
        want = unpack(want)
        want_group, want_scale = torch.ones(group.shape, dtype=torch.uint8), torch.full(scale.shape, float("nan"))
        want[page, :, off] = code[keep]
        want_group[page, :, off] = g.view(torch.uint8)[keep]
        want_scale[page, :, off] = sc[keep]
        assert torch.equal(plain_zero(unpack(data), fmt), plain_zero(want, fmt))  # the other slots as they were
        assert torch.equal(raw(group), want_group)
        assert same(scale.cpu(), want_scale)
        for out_dtype in (torch.bfloat16, torch.float32):
            wide = torch.full((2, T, heads, dim + pad), 7.0, dtype=out_dtype, device="cuda")
            ver.kv_read(cache=cache, slot_mapping=slots.cuda(), key_out=wide[0, :, :, pad:],
                        value_out=wide[1, :, :, pad:], status=status)
            back = torch.where(keep[:, None, None], values4(code, g, sc, fmt), torch.zeros(())).to(out_dtype)
            assert torch.equal(wide[side, :, :, pad:].cpu(), back)
            assert pad == 0 or bool((wide[..., :pad] == 7.0).all())
    assert int(status.item()) == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_every_code_and_group_scale_is_read_exactly(ver, fmt):
    """All 16 nibbles under all 254 e4m3 scales that are numbers, negative ones too."""
    bytes_ = torch.tensor([b for b in range(256) if b & 127 != 127], dtype=torch.uint8)
    cache = make_cache4(len(bytes_), 1, 1, 64, fmt)
    codes = torch.arange(16, dtype=torch.uint8).repeat(4)
    for data, group in ((cache.k, cache.k_group), (cache.v, cache.v_group)):
        data.copy_((codes[0::2] | codes[1::2] << 4).expand(data.shape))
        group.view(torch.uint8).copy_(bytes_.view(-1, 1, 1, 1).expand(group.shape))
    key, value = ver.kv_read(cache=cache, slot_mapping=torch.arange(len(bytes_), device="cuda"), dtype=torch.float32)
    want = values4(codes.expand(len(bytes_), 1, 64), bytes_.view(-1, 1, 1).expand(-1, 1, 4).contiguous().view(
        torch.float8_e4m3fn), torch.ones(len(bytes_), 1), fmt)
    assert torch.equal(key.cpu(), want) and torch.equal(value.cpu(), want)


@pytest.mark.parametrize("fmt", FORMATS)
def test_ties_go_to_the_even_code(ver, fmt):
    """Quotients halfway between two numbers: the row's largest makes the group scale 448 and the row's 1."""
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] if fmt == "e2m1" else [0.5, 1.5, 2.5, 3.5, 4.5, 5.5, 6.5, 7.0]
    row = torch.tensor(ties + [-t for t in ties]).repeat(4) * 448
    cache = make_cache4(1, 1, 1, 64, fmt)
    x = row.view(1, 1, 64).cuda()
    ver.kv_write(cache=cache, key=x, value=x, slot_mapping=torch.zeros(1, dtype=torch.int64, device="cuda"))
    assert float(cache.k_scale) == 1.0 and bool((cache.k_group.float() == 448).all())
    want = [0, 2, 2, 4, 4, 6, 6, 7] if fmt == "e2m1" else [0, 2, 2, 4, 4, 6, 6, 7]
    got = numbers_of(unpack(cache.k), fmt)[0, 0, 0, :8].tolist()
    assert got == [float(E2M1[i]) if fmt == "e2m1" else float(i) for i in want]


@pytest.mark.parametrize("fmt", FORMATS)
def test_non_finite_rows_read_back_as_nan(ver, fmt):
    x = torch.randn(6, 2, 64, generator=torch.Generator().manual_seed(1))
    x[1, 0, 5], x[2, 1, 63], x[4, 0, 0] = float("nan"), float("inf"), -float("inf")
    slots = torch.arange(6, device="cuda")
    cache = make_cache4(2, 2, 4, 64, fmt)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ver.kv_write(cache=cache, key=x.cuda(), value=x.cuda(), slot_mapping=slots, status=status)
    assert int(status.item()) == sv.DATA_STATUS_BITS["BAD_VALUES"]
    key, value = ver.kv_read(cache=cache, slot_mapping=slots, dtype=torch.float32)
    want = values4(*quantise4(x, fmt), fmt)
    assert same(key.cpu(), want) and same(value.cpu(), want)
    assert int(torch.isnan(key).sum()) == 3 * 64


def test_the_largest_rows(ver):
    """Elements next to the largest float: neither the scales nor the quotients overflow."""
    x = torch.randn(4, 1, 128, generator=torch.Generator().manual_seed(2))
    x = x / x.abs().amax(-1, keepdim=True) * torch.finfo(torch.float32).max
    for fmt in FORMATS:
        cache = make_cache4(1, 1, 4, 128, fmt)
        ver.kv_write(cache=cache, key=x.cuda(), value=x.cuda(), slot_mapping=torch.arange(4, device="cuda"))
        code, g, sc = quantise4(x, fmt)
        assert torch.equal(plain_zero(unpack(cache.k)[0, 0], fmt), plain_zero(code[:, 0], fmt))
        assert torch.equal(raw(cache.k_group)[0, 0], g.view(torch.uint8)[:, 0])
        assert torch.equal(cache.k_scale.cpu()[0, 0], sc[:, 0])


def test_bad_slots_are_skipped_and_reported(ver):
    x = torch.randn(5, 1, 64, generator=torch.Generator().manual_seed(2)).cuda()
    slots = torch.tensor([0, 8, -2, 1 << 40, -1], device="cuda")  # the cache has slots 0 .. 7
    cache = make_cache4(2, 1, 4, 64, "e2m1")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ver.kv_write(cache=cache, key=x, value=x, slot_mapping=slots, status=status)
    assert int(status.item()) == sv.DATA_STATUS_BITS["BAD_SLOT"]
    assert int((cache.k != 0).any(-1).sum()) == 1
    status.zero_()
    key, _ = ver.kv_read(cache=cache, slot_mapping=slots, status=status)
    assert int(status.item()) == sv.DATA_STATUS_BITS["BAD_SLOT"]
    assert bool((key[1:] == 0).all()) and bool((key[0] != 0).any())


def test_no_tokens(ver):
    cache = make_cache4(2, 1, 4, 64, "int4")
    none = torch.empty(0, 1, 64, device="cuda")
    slots = torch.empty(0, dtype=torch.int64, device="cuda")
    ver.kv_write(cache=cache, key=none, value=none, slot_mapping=slots)
    assert ver.kv_read(cache=cache, slot_mapping=slots)[0].shape == (0, 1, 64)
    torch.cuda.synchronize()


def test_offsets_beyond_32_bits(ver):
    """Pages behind the first 2^32 bytes of a cache."""
    heads, block, dim = 8, 64, 128
    blocks = (1 << 32) // (heads * block * dim // 2) + 3
    k = torch.zeros(blocks, heads, block, dim // 2, dtype=torch.uint8, device="cuda")
    group = torch.zeros(blocks, heads, block, dim // 16, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scale = torch.ones(blocks, heads, block, device="cuda")
    # (one tensor for both sides: equal rows go in)
    cache = sv.KVCache4(k=k, v=k, k_group=group, v_group=group, k_scale=scale, v_scale=scale, format="int4")
    x = torch.randn(4, heads, dim, generator=torch.Generator().manual_seed(3)).cuda()
    last = blocks * block - 1
    slots = torch.tensor([last, last - 64, 0, 65], device="cuda")
    ver.kv_write(cache=cache, key=x, value=x, slot_mapping=slots)
    code, g, sc = quantise4(x, "int4")
    for t, s in enumerate(slots.tolist()):
        assert torch.equal(unpack(k[s // block, :, s % block]), code[t])
    key, _ = ver.kv_read(cache=cache, slot_mapping=slots, dtype=torch.float32)
    assert torch.equal(key.cpu(), values4(code, g, sc, "int4"))


def test_on_another_stream_and_in_a_graph(ver):
    x = torch.randn(40, 2, 128, generator=torch.Generator().manual_seed(4)).cuda()
    cache = make_cache4(4, 2, 16, 128, "e2m1")
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
        assert torch.equal(out[0].cpu(), values4(*quantise4(x, "e2m1"), "e2m1")) and torch.equal(out[0], out[1])


def test_rows_that_share_a_scale_are_read_not_written(ver):
    full = make_cache4(3, 2, 16, 64, "int4")
    full.k.copy_(torch.randint(0, 256, full.k.shape, dtype=torch.uint8))
    full.k_group.copy_(torch.ones(full.k_group.shape))
    one = torch.tensor([0.5, 0.25, 2.0, 1.0, 3.0, 0.125], device="cuda").view(3, 2, 1)
    slots, x = torch.arange(48, device="cuda"), torch.ones(48, 2, 64, device="cuda")
    group = full.k_group[:, :, :1].expand(3, 2, 16, 4)
    for g, s in ((full.k_group, one.expand(3, 2, 16)), (group, full.k_scale), (group, one[:, :1].expand(3, 2, 16))):
        cache = sv.KVCache4(k=full.k, v=full.v, k_group=g, v_group=g, k_scale=s, v_scale=s, format="int4")
        key, _ = ver.kv_read(cache=cache, slot_mapping=slots, dtype=torch.float32)
        want = numbers_of(unpack(full.k), "int4") * s.cpu()[..., None]
        assert torch.equal(key.cpu(), want.permute(0, 2, 1, 3).reshape(48, 2, 64))
        with pytest.raises(sv.SpecVerifyError) as ei:
            ver.kv_write(cache=cache, key=x, value=x, slot_mapping=slots)
        assert ei.value.code == sv.SV_ERR_INVALID_ARG
