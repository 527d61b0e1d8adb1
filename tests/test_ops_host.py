"""Host-side refusals of the operators around the verifier: the library's
checks of sizes, strides and pointers (nothing is enqueued), and the binding's
checks of tensors (on the CPU)."""
import pytest
import torch

import speculative_decoding_token_rejection_gb300 as sv

FAKE = 0x10000  # never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    from speculative_decoding_token_rejection_gb300 import _build
    _build.build()
    return sv.load_library()


def cfg(**kw):
    return sv.make_config(**{**dict(max_num_reqs=8, max_spec_len=4, vocab_size=2000), **kw})


def cache_struct():
    c = sv.SpecVerifyKvCache()
    c.k = c.v = c.k_scale = c.v_scale = FAKE
    c.num_blocks, c.block_size, c.num_kv_heads, c.head_dim, c.format = 10, 16, 2, 128, sv.SV_CACHE_E4M3
    c.token_stride, c.head_stride, c.block_stride = 128, 2048, 4096
    c.scale_token_stride, c.scale_head_stride, c.scale_block_stride = 1, 16, 32
    return c


def kv_args():
    a = sv.SpecVerifyKvArgs()
    a.num_tokens, a.dtype, a.cache = 5, sv.SV_BF16, cache_struct()
    a.key = a.value = a.slot_mapping = FAKE
    a.key_token_stride = a.value_token_stride = 256
    a.key_head_stride = a.value_head_stride = 128
    return a


def put(path, value):
    def change(a):
        names = path.split(".")
        for n in names[:-1]:
            a = getattr(a, n)
        setattr(a, names[-1], value)
    return change


OK, INVALID, UNSUPPORTED, CAPACITY = sv.SV_OK, sv.SV_ERR_INVALID_ARG, sv.SV_ERR_UNSUPPORTED, sv.SV_ERR_CAPACITY

CACHE_CHANGES = [
    ("format", 2, INVALID), ("num_kv_heads", 0, INVALID), ("head_dim", 0, INVALID), ("head_dim", 96, UNSUPPORTED),
    ("head_dim", 256, UNSUPPORTED), ("num_blocks", 0, INVALID), ("block_size", 0, INVALID),
    ("num_blocks", 1 << 28, UNSUPPORTED), ("k", None, INVALID), ("v", None, INVALID), ("k_scale", None, INVALID),
    ("v_scale", None, INVALID), ("token_stride", -128, INVALID), ("scale_token_stride", -1, INVALID),
    ("k", FAKE + 8, UNSUPPORTED), ("v", FAKE + 1, UNSUPPORTED), ("token_stride", 136, UNSUPPORTED),
    ("token_stride", 64, INVALID), ("head_stride", 0, INVALID), ("block_stride", 0, INVALID),
]


@pytest.mark.parametrize("path,value,code", [("cache." + p, v, c) for p, v, c in CACHE_CHANGES] + [
    ("num_tokens", 5, OK), ("num_tokens", -1, INVALID), ("num_tokens", 1 << 40, UNSUPPORTED), ("num_tokens", 0, OK),
    ("dtype", 2, INVALID), ("reserved", 1, INVALID), ("key", None, INVALID), ("value", None, INVALID),
    ("slot_mapping", None, INVALID), ("key_token_stride", -1, INVALID), ("value_head_stride", -1, INVALID),
    ("key_token_stride", 257, OK), ("key", FAKE + 2, OK), ("cache.block_size", 7, OK)])
def test_check_kv_args(path, value, code):
    a = kv_args()
    put(path, value)(a)
    assert sv.spec_verify_check_kv_args(cfg(), a) == code


def attend_args():
    a = sv.SpecVerifyAttendArgs()
    a.num_reqs, a.max_spec_len, a.num_q_heads, a.max_seq_len, a.shared_prefix_len = 3, 2, 8, 100, 32
    a.num_draft_tokens_total, a.cache = 6, cache_struct()
    a.q = a.out = a.block_tables = a.seq_lens = FAKE
    a.q_token_stride = a.out_token_stride = 1024
    a.q_head_stride = a.out_head_stride = 128
    a.block_table_stride, a.scale = 7, 0.1
    return a


@pytest.mark.parametrize("path,value,code", [("cache." + p, v, c) for p, v, c in CACHE_CHANGES
                                             if p not in ("num_kv_heads", "head_dim")] + [
    ("num_reqs", 3, OK), ("num_reqs", -1, INVALID), ("num_reqs", 9, CAPACITY), ("max_spec_len", 5, CAPACITY),
    ("max_spec_len", -1, INVALID), ("num_draft_tokens_total", 5, INVALID), ("num_draft_tokens_total", -1, INVALID),
    ("num_q_heads", 7, INVALID), ("num_q_heads", 0, INVALID), ("cache.num_kv_heads", 0, INVALID),
    ("cache.num_kv_heads", 3, INVALID), ("cache.head_dim", 96, UNSUPPORTED), ("max_seq_len", -1, INVALID),
    ("max_seq_len", 112, OK), ("max_seq_len", 113, OK), ("max_seq_len", 1 << 30, OK), ("max_seq_len", (1 << 30) + 1, UNSUPPORTED), ("block_table_stride", -1, INVALID), ("block_table_stride", 1, INVALID), ("shared_prefix_len", 33, INVALID),
    ("shared_prefix_len", -16, INVALID), ("shared_prefix_len", 112, INVALID), ("shared_prefix_len", 0, OK),
    ("reserved", 1, INVALID), ("reserved2", 1, INVALID), ("q", None, INVALID), ("out", None, INVALID),
    ("seq_lens", None, INVALID), ("block_tables", None, INVALID), ("cache.block_stride", 1 << 35, UNSUPPORTED), ("scale", float("nan"), INVALID),
    ("scale", float("inf"), INVALID), ("scale", -1.0, OK), ("q_head_stride", -1, INVALID),
    ("workspace_bytes", -1, INVALID), ("workspace", FAKE + 4, INVALID)])
def test_check_attend_args(path, value, code):
    a = attend_args()
    put(path, value)(a)
    assert sv.spec_verify_check_attend_args(cfg(), a) == code


def test_check_attend_args_of_an_empty_batch():
    a = sv.SpecVerifyAttendArgs()
    a.num_q_heads, a.cache.num_kv_heads, a.cache.head_dim = 4, 2, 64
    assert sv.spec_verify_check_attend_args(cfg(), a) == OK
    a.cu_num_draft_tokens, a.num_draft_tokens_total = FAKE, 1
    assert sv.spec_verify_check_attend_args(cfg(), a) == INVALID


def logprobs_args():
    a = sv.SpecVerifyLogprobsArgs()
    a.num_reqs, a.max_spec_len, a.vocab_size, a.dtype, a.num_top = 3, 2, 1000, sv.SV_F32, 4
    a.num_draft_tokens_total, a.row_stride = 6, 1000
    a.logits = a.out_tokens = a.logprobs = a.top_ids = a.top_logprobs = FAKE
    return a


@pytest.mark.parametrize("path,value,code", [
    ("num_reqs", 3, OK), ("num_reqs", -1, INVALID), ("num_reqs", 9, CAPACITY), ("max_spec_len", 5, CAPACITY),
    ("num_draft_tokens_total", 7, INVALID), ("vocab_size", 0, INVALID), ("vocab_size", 2001, CAPACITY),
    ("dtype", 3, INVALID), ("reserved", 1, INVALID), ("num_top", -1, INVALID), ("num_top", 33, UNSUPPORTED),
    ("num_top", 1001, INVALID), ("num_top", 0, OK), ("row_stride", 999, INVALID), ("row_stride", 1001, OK),
    ("logits", None, INVALID), ("logits", FAKE + 4, OK), ("out_tokens", None, INVALID), ("logprobs", None, INVALID),
    ("top_ids", None, INVALID), ("top_logprobs", None, INVALID), ("ranks", None, OK), ("entropy", None, OK)])
def test_check_logprobs_args(path, value, code):
    a = logprobs_args()
    put(path, value)(a)
    assert sv.spec_verify_check_logprobs_args(cfg(), a) == code


def test_null_handles_and_args(lib):
    for name, a in (("kv_write", kv_args()), ("kv_read", kv_args()), ("attend", attend_args()),
                    ("logprobs", logprobs_args())):
        assert getattr(lib, f"spec_verify_{name}")(None, a, None) == INVALID
    c = cfg()
    for name in ("kv", "attend", "logprobs"):
        assert getattr(lib, f"spec_verify_check_{name}_args")(None, None) == INVALID
        assert getattr(lib, f"spec_verify_check_{name}_args")(c, None) == INVALID


def tensors(nhd=False, fmt=torch.int8):
    k = torch.zeros(4, 2, 16, 64, dtype=torch.uint8).view(fmt)
    s = torch.ones(4, 2, 16)
    if nhd:
        k = torch.zeros(4, 16, 2, 64, dtype=torch.uint8).view(fmt).permute(0, 2, 1, 3)
        s = torch.ones(4, 16, 2).permute(0, 2, 1)
    return dict(k=k, v=k.clone() if not nhd else k, k_scale=s, v_scale=s)


def test_cache_description():
    c = sv.KVCache(**tensors()).struct
    assert (c.block_stride, c.head_stride, c.token_stride) == (2048, 1024, 64)
    assert (c.scale_block_stride, c.scale_head_stride, c.scale_token_stride) == (32, 16, 1)
    c = sv.KVCache(**tensors(nhd=True, fmt=torch.float8_e4m3fn)).struct
    assert (c.block_stride, c.head_stride, c.token_stride, c.format) == (2048, 64, 128, sv.SV_CACHE_E4M3)


@pytest.mark.parametrize("change,error", [
    (dict(k=torch.zeros(4, 2, 16, 64)), TypeError), (dict(v=torch.zeros(4, 2, 16, 64, dtype=torch.uint8)), TypeError),
    (dict(v=torch.zeros(4, 2, 8, 64, dtype=torch.int8)), ValueError), (dict(k_scale=torch.ones(4, 2, 8)), ValueError),
    (dict(v_scale=torch.ones(4, 2, 16, dtype=torch.float64)), TypeError),
    (dict(v=torch.zeros(4, 16, 2, 64, dtype=torch.int8).permute(0, 2, 1, 3)), ValueError),
    (dict(v_scale=torch.ones(4, 16, 2).permute(0, 2, 1)), ValueError),
    (dict(k=torch.zeros(4, 2, 64, 16, dtype=torch.int8).transpose(2, 3)), ValueError)])
def test_cache_refusals(change, error):
    with pytest.raises(error):
        sv.KVCache(**{**tensors(), **change})


def test_binding_refusals():
    cache = sv.KVCache(**tensors())
    slots = torch.zeros(3, dtype=torch.int64)
    x = torch.zeros(3, 2, 64)
    sv.build_kv_args(cache=cache, key=x, value=x, slot_mapping=slots)
    for kw, error in ((dict(key=torch.zeros(2, 2, 64)), ValueError), (dict(value=x.bfloat16()), TypeError),
                      (dict(key=x.double()), TypeError), (dict(slot_mapping=slots.int()), TypeError),
                      (dict(value=torch.zeros(3, 64, 2).transpose(1, 2)), ValueError)):
        with pytest.raises(error):
            sv.build_kv_args(**{**dict(cache=cache, key=x, value=x, slot_mapping=slots), **kw})
    q = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    good = dict(q=q, out=torch.zeros_like(q), cache=cache, block_tables=torch.zeros(2, 3, dtype=torch.int32),
                seq_lens=torch.zeros(2, dtype=torch.int32), max_seq_len=40, max_spec_len=2, scale=1.0,
                cu_num_draft_tokens=torch.tensor([1, 3], dtype=torch.int32), lse=torch.zeros(5, 4))
    assert sv.spec_verify_check_attend_args(cfg(), sv.build_attend_args(**good)) == OK
    for kw, error in ((dict(q=q.float()), TypeError), (dict(out=torch.zeros(5, 4, 32)), ValueError),
                      (dict(block_tables=torch.zeros(2, 3)), TypeError), (dict(seq_lens=torch.zeros(3).int()), ValueError),
                      (dict(lse=torch.zeros(5, 3)), ValueError),
                      (dict(out=q[:1].expand(5, 4, 64)), ValueError),
                      (dict(cu_num_draft_tokens=torch.tensor([3], dtype=torch.int32)), ValueError)):
        with pytest.raises(error):
            sv.build_attend_args(**{**good, **kw})
    good = dict(logits=torch.zeros(6, 100), out_tokens=torch.zeros(3, 2, dtype=torch.int32),
                logprobs=torch.zeros(3, 2), num_top=2, top_ids=torch.zeros(3, 2, 2, dtype=torch.int32),
                top_logprobs=torch.zeros(3, 2, 2))
    assert sv.spec_verify_check_logprobs_args(cfg(), sv.build_logprobs_args(**good)) == OK
    for kw, error in ((dict(logits=torch.zeros(6, 100).half()), TypeError), (dict(logprobs=torch.zeros(3)), ValueError),
                      (dict(out_tokens=torch.zeros(3, 2)), TypeError), (dict(out_tokens=torch.zeros(6).int()), ValueError),
                      (dict(top_ids=torch.zeros(3, 2, 2)), TypeError),
                      (dict(logits=torch.zeros(100, 6).t()), ValueError)):
        with pytest.raises(error):
            sv.build_logprobs_args(**{**good, **kw})


@pytest.mark.parametrize("value,code", [(0, OK), (sv.SV_TEST_EXPIRE_PRODUCT_WAIT, OK), (sv.SV_TEST_EXPIRE_COPY_WAIT, INVALID),
                                        (3, INVALID), (4, INVALID)])
def test_attend_test_flags(value, code):
    a = attend_args()
    a.test_flags = value
    assert sv.spec_verify_check_attend_args(cfg(), a) == code


def test_expanded_block_tables_are_refused():
    q = torch.zeros(6, 4, 64, dtype=torch.bfloat16)
    good = dict(q=q, out=torch.zeros_like(q), cache=sv.KVCache(**tensors()), seq_lens=torch.zeros(3, dtype=torch.int32),
                max_seq_len=40, max_spec_len=1, scale=1.0)
    table = torch.zeros(1, 3, dtype=torch.int32)
    for bad in (table.expand(3, -1), torch.zeros(20, dtype=torch.int32).as_strided((3, 3), (2, 1))):
        with pytest.raises(ValueError, match="overlap"):
            sv.build_attend_args(**good, block_tables=bad)
    for fine in (table.expand(3, -1).contiguous(), torch.zeros(3, 5, dtype=torch.int32)[:, :3], torch.zeros(3, 0, dtype=torch.int32)):
        a = sv.build_attend_args(**good, block_tables=fine)
        assert a.block_table_stride >= fine.shape[1]
    one = sv.build_attend_args(**{**good, "q": q[:2], "out": good["out"][:2], "seq_lens": good["seq_lens"][:1]},
                               block_tables=table.expand(1, -1))
    assert one.block_table_stride == 3


@pytest.mark.parametrize("strides,code", [
    (dict(block_stride=1 << 34), OK),  # nine pages of 16 GB
    (dict(block_stride=1 << 34, token_stride=144), UNSUPPORTED),  # only 16 divides both: 64 GB at most
    (dict(block_stride=1 << 32, token_stride=144), OK), (dict(block_stride=(1 << 34) + 64), OK),
    (dict(block_stride=(1 << 34) + 16), UNSUPPORTED), (dict(block_stride=1 << 60), UNSUPPORTED),
    (dict(head_stride=1 << 37), OK), (dict(head_stride=1 << 38), UNSUPPORTED)])
def test_spans_of_a_cache(strides, code):
    a = attend_args()
    for name, value in strides.items():
        setattr(a.cache, name, value)
    assert sv.spec_verify_check_attend_args(cfg(), a) == code
