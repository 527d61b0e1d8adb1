"""Host-side refusals of what leads up to a verification step: the library's
checks of sizes, strides and pointers (nothing is enqueued), and the binding's
checks of tensors (on the CPU)."""
import math

import pytest
import torch

import speculative_decoding_token_rejection_gb300 as sv
from test_ops_host import CAPACITY, FAKE, INVALID, OK, UNSUPPORTED, cfg, put


@pytest.fixture(scope="module", autouse=True)
def lib():
    from speculative_decoding_token_rejection_gb300 import _build
    _build.build()
    return sv.load_library()


def cache_struct():
    c = sv.SpecVerifyKv4Cache()
    c.k = c.v = c.k_group = c.v_group = c.k_scale = c.v_scale = FAKE
    c.num_blocks, c.block_size, c.num_kv_heads, c.head_dim, c.format = 10, 16, 2, 128, sv.SV_CACHE_E2M1
    c.token_stride, c.head_stride, c.block_stride = 64, 1024, 2048
    c.group_token_stride, c.group_head_stride, c.group_block_stride = 8, 128, 256
    c.scale_token_stride, c.scale_head_stride, c.scale_block_stride = 1, 16, 32
    return c


CACHE_CHANGES = [
    ("format", sv.SV_CACHE_INT4, OK), ("format", sv.SV_CACHE_INT8, INVALID), ("format", 18, INVALID),
    ("num_kv_heads", 0, INVALID), ("head_dim", 0, INVALID), ("head_dim", 96, UNSUPPORTED), ("num_blocks", 0, INVALID),
    ("block_size", 0, INVALID), ("num_blocks", 1 << 28, UNSUPPORTED), ("k", None, INVALID), ("v", None, INVALID),
    ("k_group", None, INVALID), ("v_group", None, INVALID), ("k_scale", None, INVALID), ("v_scale", None, INVALID),
    ("token_stride", -64, INVALID), ("group_token_stride", -8, INVALID), ("scale_token_stride", -1, INVALID),
    ("k", FAKE + 16, UNSUPPORTED), ("v", FAKE + 1, UNSUPPORTED), ("token_stride", 80, UNSUPPORTED),
    ("k_group", FAKE + 4, UNSUPPORTED), ("group_head_stride", 132, UNSUPPORTED), ("group_token_stride", 16, OK),
    ("token_stride", 32, INVALID), ("head_stride", 0, INVALID), ("block_stride", 0, INVALID), ("block_size", 7, OK),
]


def kv_args():
    a = sv.SpecVerifyKv4Args()
    a.num_tokens, a.dtype, a.cache = 5, sv.SV_BF16, cache_struct()
    a.key = a.value = a.slot_mapping = FAKE
    a.key_token_stride = a.value_token_stride = 256
    a.key_head_stride = a.value_head_stride = 128
    return a


@pytest.mark.parametrize("path,value,code", [("cache." + p, v, c) for p, v, c in CACHE_CHANGES] + [
    ("num_tokens", 5, OK), ("num_tokens", -1, INVALID), ("num_tokens", 1 << 40, UNSUPPORTED), ("num_tokens", 0, OK),
    ("dtype", 2, INVALID), ("reserved", 1, INVALID), ("key", None, INVALID), ("value", None, INVALID),
    ("slot_mapping", None, INVALID), ("key_token_stride", -1, INVALID), ("value_head_stride", -1, INVALID),
    ("key_token_stride", 257, OK), ("key", FAKE + 2, OK)])
def test_check_kv4_args(path, value, code):
    a = kv_args()
    put(path, value)(a)
    assert sv.spec_verify_check_kv4_args(cfg(), a) == code


def attend_args():
    a = sv.SpecVerifyAttend4Args()
    a.num_reqs, a.max_spec_len, a.num_q_heads, a.max_seq_len, a.shared_prefix_len = 3, 2, 8, 100, 32
    a.num_draft_tokens_total, a.cache = 6, cache_struct()
    a.q = a.out = a.block_tables = a.seq_lens = FAKE
    a.q_token_stride = a.out_token_stride = 1024
    a.q_head_stride = a.out_head_stride = 128
    a.block_table_stride, a.scale = 7, 0.1
    return a


@pytest.mark.parametrize("path,value,code", [("cache." + p, v, c) for p, v, c in CACHE_CHANGES
                                             if p not in ("num_kv_heads", "head_dim", "block_size")] + [
    ("num_reqs", 3, OK), ("num_reqs", -1, INVALID), ("num_reqs", 9, CAPACITY), ("max_spec_len", 5, CAPACITY),
    ("num_draft_tokens_total", 5, INVALID), ("num_q_heads", 7, INVALID), ("cache.num_kv_heads", 3, INVALID),
    ("cache.head_dim", 96, UNSUPPORTED), ("max_seq_len", -1, INVALID), ("max_seq_len", (1 << 30) + 1, UNSUPPORTED),
    ("block_table_stride", 1, INVALID), ("shared_prefix_len", 33, INVALID), ("shared_prefix_len", 0, OK),
    ("reserved", 1, INVALID), ("test_flags", sv.SV_TEST_EXPIRE_PRODUCT_WAIT, OK), ("test_flags", 1, INVALID),
    ("q", None, INVALID), ("out", None, INVALID), ("seq_lens", None, INVALID), ("block_tables", None, INVALID),
    ("cache.block_stride", 1 << 35, UNSUPPORTED), ("cache.token_stride", 1 << 32, UNSUPPORTED),
    ("cache.group_block_stride", 1 << 32, UNSUPPORTED), ("cache.scale_block_stride", 1 << 30, UNSUPPORTED),
    ("cache.scale_token_stride", (1 << 30) - 1, OK), ("cache.block_stride", (1 << 32) - 32, OK), ("scale", float("nan"), INVALID), ("scale", -1.0, OK),
    ("workspace_bytes", -1, INVALID), ("workspace", FAKE + 4, INVALID)])
def test_check_attend4_args(path, value, code):
    a = attend_args()
    put(path, value)(a)
    assert sv.spec_verify_check_attend4_args(cfg(), a) == code


def test_check_attend4_args_of_an_empty_batch():
    a = sv.SpecVerifyAttend4Args()
    a.num_q_heads, a.cache.num_kv_heads, a.cache.head_dim = 4, 2, 64
    assert sv.spec_verify_check_attend4_args(cfg(), a) == OK


def plan_args():
    a = sv.SpecVerifyPlanArgs()
    a.num_reqs, a.block_size, a.table_width, a.num_rows = 3, 16, 7, 20
    a.block_table_stride, a.free_capacity = 7, 100
    for name in ("num_new_tokens", "num_computed_tokens", "block_tables", "held_pages", "held_pages_out", "free_pages",
                 "free_range", "free_range_out", "positions", "slot_mapping", "seq_lens", "workspace"):
        setattr(a, name, FAKE)
    a.workspace_bytes = 1 << 20
    return a


@pytest.mark.parametrize("path,value,code", [
    ("num_reqs", 3, OK), ("num_reqs", -1, INVALID), ("num_reqs", 9, CAPACITY), ("num_reqs", 0, OK),
    ("block_size", 0, INVALID), ("block_size", 1, OK), ("table_width", -1, INVALID), ("table_width", 8, INVALID),
    ("table_width", 0, OK), ("num_shared_pages", -1, INVALID), ("num_shared_pages", 7, OK),
    ("num_shared_pages", 8, INVALID), ("num_rows", -1, INVALID), ("num_rows", 0, OK),
    ("num_rows", 1 << 31, UNSUPPORTED), ("free_capacity", 0, INVALID), ("free_capacity", 1 << 31, UNSUPPORTED),
    ("workspace_bytes", -1, INVALID), ("workspace", FAKE + 8, INVALID), ("cu_num_draft_tokens", FAKE, OK)] + [
        (name, None, INVALID) for name in ("num_new_tokens", "num_computed_tokens", "block_tables", "held_pages",
                                           "held_pages_out", "free_pages", "free_range", "free_range_out", "positions",
                                           "slot_mapping", "seq_lens")])
def test_check_plan_args(path, value, code):
    a = plan_args()
    put(path, value)(a)
    assert sv.spec_verify_check_plan_args(cfg(), a) == code


def rotate_args():
    a = sv.SpecVerifyRotateArgs()
    a.num_tokens, a.dtype, a.head_dim, a.rotary_dim, a.num_q_heads, a.num_k_heads = 5, sv.SV_BF16, 128, 64, 8, 2
    for name in ("q", "q_out", "key", "key_out", "positions", "turns"):
        setattr(a, name, FAKE)
    a.magnitude, a.eps = 1.0, 1e-6
    return a


@pytest.mark.parametrize("path,value,code", [
    ("num_tokens", 5, OK), ("num_tokens", -1, INVALID), ("num_tokens", 0, OK), ("num_tokens", 1 << 40, UNSUPPORTED),
    ("dtype", 2, INVALID), ("head_dim", 0, INVALID), ("head_dim", 513, UNSUPPORTED), ("head_dim", 512, OK),
    ("rotary_dim", 63, INVALID), ("rotary_dim", 130, INVALID), ("rotary_dim", -2, INVALID), ("rotary_dim", 0, OK),
    ("num_q_heads", -1, INVALID), ("num_q_heads", 0, OK), ("num_q_heads", 1 << 20, UNSUPPORTED),
    ("num_k_heads", -1, INVALID), ("num_k_heads", 0, OK), ("flags", 2, INVALID), ("flags", 1, OK),
    ("magnitude", float("inf"), INVALID), ("magnitude", -1.0, OK), ("eps", -1e-6, INVALID), ("eps", float("nan"), INVALID),
    ("eps", 0.0, OK), ("q", None, INVALID), ("q_out", None, INVALID), ("key", None, INVALID), ("key_out", None, INVALID),
    ("positions", None, INVALID), ("turns", None, INVALID), ("q_weight", FAKE, OK), ("q_token_stride", -1, INVALID),
    ("key_out_head_stride", -1, INVALID), ("q_token_stride", 3, OK)])
def test_check_rotate_args(path, value, code):
    a = rotate_args()
    put(path, value)(a)
    assert sv.spec_verify_check_rotate_args(cfg(), a) == code


def test_null_handles_and_args(lib):
    for name, a in (("kv4_write", kv_args()), ("kv4_read", kv_args()), ("attend4", attend_args()),
                    ("plan_step", plan_args()), ("rotate", rotate_args())):
        assert getattr(lib, f"spec_verify_{name}")(None, a, None) == INVALID
    for name in ("kv4", "attend4", "plan", "rotate"):
        assert getattr(lib, f"spec_verify_check_{name}_args")(None, None) == INVALID
        assert getattr(lib, f"spec_verify_check_{name}_args")(cfg(), None) == INVALID


def tensors(nhd=False):
    lead = (4, 16, 2) if nhd else (4, 2, 16)
    k = torch.zeros(*lead, 32, dtype=torch.uint8)
    g = torch.zeros(*lead, 4, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.ones(lead)
    if nhd:
        k, g, s = k.permute(0, 2, 1, 3), g.permute(0, 2, 1, 3), s.permute(0, 2, 1)
    return dict(k=k, v=k, k_group=g, v_group=g, k_scale=s, v_scale=s, format="e2m1")


def test_cache_description():
    c = sv.KVCache4(**tensors()).struct
    assert (c.block_stride, c.head_stride, c.token_stride, c.head_dim) == (1024, 512, 32, 64)
    assert (c.group_block_stride, c.group_head_stride, c.group_token_stride) == (128, 64, 4)
    assert (c.scale_block_stride, c.scale_head_stride, c.scale_token_stride) == (32, 16, 1)
    c = sv.KVCache4(**{**tensors(nhd=True), "format": "int4"}).struct
    assert (c.block_stride, c.head_stride, c.token_stride, c.format) == (1024, 32, 64, sv.SV_CACHE_INT4)
    assert (c.group_head_stride, c.group_token_stride, c.scale_head_stride) == (4, 8, 1)


@pytest.mark.parametrize("change,error", [
    (dict(format="int8"), ValueError), (dict(k=torch.zeros(4, 2, 16, 32)), TypeError),
    (dict(k=torch.zeros(4, 2, 16, dtype=torch.uint8)), ValueError),
    (dict(v=torch.zeros(4, 2, 16, 64, dtype=torch.uint8)), ValueError),
    (dict(k_group=torch.zeros(4, 2, 16, 4)), TypeError), (dict(v_scale=torch.ones(4, 2, 8)), ValueError),
    (dict(k_scale=torch.ones(4, 2, 16, dtype=torch.float64)), TypeError),
    (dict(v=torch.zeros(4, 16, 2, 32, dtype=torch.uint8).permute(0, 2, 1, 3)), ValueError),
    (dict(v_scale=torch.ones(4, 16, 2).permute(0, 2, 1)), ValueError),
    (dict(k=torch.zeros(4, 2, 32, 16, dtype=torch.uint8).transpose(2, 3)), ValueError)])
def test_cache_refusals(change, error):
    with pytest.raises(error):
        sv.KVCache4(**{**tensors(), **change})


def test_kv_and_attention_calls_take_either_cache():
    cache, slots, x = sv.KVCache4(**tensors()), torch.zeros(3, dtype=torch.int64), torch.zeros(3, 2, 64)
    assert isinstance(sv.build_kv_args(cache=cache, key=x, value=x, slot_mapping=slots), sv.SpecVerifyKv4Args)
    with pytest.raises(ValueError):
        sv.build_kv_args(cache=cache, key=x[..., :32], value=x, slot_mapping=slots)
    q = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    good = dict(q=q, out=torch.zeros_like(q), cache=cache, block_tables=torch.zeros(2, 3, dtype=torch.int32),
                seq_lens=torch.zeros(2, dtype=torch.int32), max_seq_len=40, max_spec_len=2, scale=1.0,
                cu_num_draft_tokens=torch.tensor([1, 3], dtype=torch.int32), lse=torch.zeros(5, 4))
    a = sv.build_attend_args(**good)
    assert isinstance(a, sv.SpecVerifyAttend4Args) and a.cache.k_group == cache.k_group.data_ptr()
    with pytest.raises(TypeError):
        sv.build_attend_args(**{**good, "q": q.float()})


def plan_tensors(N=3, R=10):
    i32 = dict(dtype=torch.int32)
    return dict(num_new_tokens=torch.ones(N, **i32), num_computed_tokens=torch.zeros(N, **i32),
                block_tables=torch.zeros(N, 4, **i32), held_pages=torch.zeros(N, **i32), held_pages_out=torch.zeros(N, **i32),
                free_pages=torch.arange(9, **i32), free_range=torch.tensor([0, 9]), free_range_out=torch.zeros(2).long(),
                block_size=16, num_rows=R, positions=torch.zeros(R, **i32), slot_mapping=torch.zeros(R).long(),
                seq_lens=torch.zeros(N, **i32), workspace=torch.zeros(64, dtype=torch.uint8))


def test_plan_refusals():
    a = sv.build_plan_args(**plan_tensors())
    assert (a.num_reqs, a.table_width, a.block_table_stride, a.free_capacity, a.num_rows) == (3, 4, 4, 9, 10)
    for kw, error in ((dict(block_tables=torch.zeros(2, 4).int()), ValueError), (dict(block_tables=torch.zeros(3, 4)), ValueError),
                      (dict(block_tables=torch.zeros(1, 4).int().expand(3, -1)), ValueError),
                      (dict(block_tables=torch.zeros(4, 3).int().t()), ValueError), (dict(num_rows=11), ValueError),
                      (dict(slot_mapping=torch.zeros(10).int()), TypeError), (dict(free_range=torch.tensor([0])), ValueError),
                      (dict(held_pages=torch.zeros(3)), TypeError), (dict(seq_lens=torch.zeros(2).int()), ValueError),
                      (dict(workspace=torch.zeros(8)), TypeError)):
        with pytest.raises(error):
            sv.build_plan_args(**{**plan_tensors(), **kw})


def test_rotate_refusals():
    f = sv.RotaryFrequencies(64, device="cpu")
    q, key = torch.zeros(5, 4, 64), torch.zeros(5, 2, 64)
    good = dict(q=q, key=key, q_out=q, key_out=key, positions=torch.zeros(5).int(), frequencies=f,
                q_weight=torch.ones(64))
    a = sv.build_rotate_args(**good)
    assert (a.num_tokens, a.num_q_heads, a.num_k_heads, a.rotary_dim, a.q_token_stride) == (5, 4, 2, 64, 256)
    assert sv.build_rotate_args(**{**good, "key": None, "key_out": None}).num_k_heads == 0
    for kw, error in ((dict(q=None, key=None), ValueError), (dict(q=q.half()), TypeError), (dict(key=key.bfloat16()), TypeError),
                      (dict(key=torch.zeros(4, 2, 64)), ValueError), (dict(q=torch.zeros(5, 256)), ValueError),
                      (dict(q_out=q.bfloat16()), TypeError), (dict(q_out=torch.zeros(1, 4, 64).expand(5, 4, 64)), ValueError),
                      (dict(q_out=torch.zeros(5, 4, 32)), ValueError), (dict(positions=torch.zeros(5)), TypeError),
                      (dict(positions=torch.zeros(4).int()), ValueError), (dict(q_weight=torch.ones(64).double()), TypeError),
                      (dict(key_weight=torch.ones(32)), ValueError), (dict(q=q.transpose(1, 2)[:, :4, :4]), ValueError),
                      (dict(q_out=q.view(5, 2, 2, 64).transpose(1, 2).flatten(1, 2).view(-1).as_strided(
                          (5, 4, 64), (256, 64, 1))), None)):
        if error is None:
            sv.build_rotate_args(**{**good, **kw})
            continue
        with pytest.raises(error):
            sv.build_rotate_args(**{**good, **kw})
    with pytest.raises(ValueError):  # the same memory with other strides
        sv.build_rotate_args(**{**good, "q_out": q.as_strided((5, 4, 64), (64, 320, 1))})


def test_frequencies():
    f = sv.RotaryFrequencies(64, device="cpu")
    assert f.inverse[0] == 1.0 and f.magnitude == 1.0
    # whole 2^-64 of a turn: half of one, and the comparison's three roundings (pi, the quotient, the word) of 2^-53 each
    for w, inv in zip(f.turns.tolist(), f.inverse):
        turn = inv / (2 * math.pi)
        assert abs((w % (1 << 64)) / 2.0 ** 64 - turn) <= 3 * 2.0 ** -53 * turn + 2.0 ** -65
    assert sv.RotaryFrequencies(64, scaling="linear", factor=4.0, device="cpu").inverse[3] == f.inverse[3] / 4
    ntk = sv.RotaryFrequencies(64, scaling="ntk", factor=4.0, device="cpu")
    assert ntk.inverse[0] == 1.0 and ntk.inverse[31] == pytest.approx(f.inverse[31] / 4, rel=1e-12)
    yarn = sv.RotaryFrequencies(64, scaling="yarn", factor=16.0, trained_len=4096, device="cpu")
    assert yarn.inverse[0] == f.inverse[0] and yarn.inverse[31] == pytest.approx(f.inverse[31] / 16, rel=1e-12)
    assert yarn.magnitude == pytest.approx(0.1 * math.log(16) + 1)
    assert all(b <= a for a, b in zip(yarn.inverse, yarn.inverse[1:]))
    assert sv.RotaryFrequencies(4, inverse=[0.5, 0.25], magnitude=2.0, device="cpu").inverse == (0.5, 0.25)
    assert sv.RotaryFrequencies(0, device="cpu").turns.numel() == 0
    for bad in (dict(rotary_dim=63), dict(rotary_dim=-2), dict(scaling="cubic"), dict(base=0.5), dict(factor=0.0),
                dict(scaling="yarn", factor=4.0), dict(rotary_dim=2, scaling="ntk"), dict(inverse=[1.0]),
                dict(inverse=[1.0] * 32, scaling="linear"), dict(inverse=[math.nan] * 32)):
        with pytest.raises(ValueError):
            sv.RotaryFrequencies(**{"rotary_dim": 64, "device": "cpu", **bad})
