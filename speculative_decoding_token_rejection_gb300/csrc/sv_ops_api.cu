// sv_ops_api.cu -- the C entries of the operators around the verifier: the
// paged 8-bit KV cache, the verify tokens' attention over it and the
// log-probabilities of the committed tokens.  Host-side validation and kernel
// dispatch; no allocation, no host sync.
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdio>

#include "sv_internal.h"

namespace {

template <typename... A>
sv_status fail(sv_status s, const char *fmt, A... a) {
  sv::set_last_error(fmt, a...);
  return s;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A cache's description; with `pointers` false only its sizes.
sv_status check_cache(const spec_verify_kv_cache &c) {
  if (c.format != SV_CACHE_INT8 && c.format != SV_CACHE_E4M3) return fail(SV_ERR_INVALID_ARG, "bad cache format");
  if (c.num_kv_heads < 1) return fail(SV_ERR_INVALID_ARG, "num_kv_heads < 1");
  if (c.head_dim < 1) return fail(SV_ERR_INVALID_ARG, "head_dim < 1");
  if (c.head_dim != 64 && c.head_dim != 128)
    return fail(SV_ERR_UNSUPPORTED, "head_dim %d is not 64 or 128", c.head_dim);
  if (c.num_blocks < 1 || c.block_size < 1) return fail(SV_ERR_INVALID_ARG, "num_blocks or block_size < 1");
  if (c.num_blocks > INT_MAX / c.block_size)
    return fail(SV_ERR_UNSUPPORTED, "a cache of more than 2^31 - 1 slots");
  if (!c.k || !c.v || !c.k_scale || !c.v_scale) return fail(SV_ERR_INVALID_ARG, "a cache pointer is NULL");
  if (c.block_stride < 0 || c.head_stride < 0 || c.token_stride < 0 || c.scale_block_stride < 0 ||
      c.scale_head_stride < 0 || c.scale_token_stride < 0)
    return fail(SV_ERR_INVALID_ARG, "a cache stride < 0");
  if (!aligned16(c.k) || !aligned16(c.v) || c.block_stride % 16 || c.head_stride % 16 || c.token_stride % 16)
    return fail(SV_ERR_UNSUPPORTED, "cache rows must start on 16-byte boundaries");
  if ((c.block_size > 1 && c.token_stride < c.head_dim) || (c.num_kv_heads > 1 && c.head_stride < c.head_dim) ||
      (c.num_blocks > 1 && c.block_stride < c.head_dim))
    return fail(SV_ERR_INVALID_ARG, "cache rows overlap");
  return SV_OK;
}

// Ragged layout shared by the calls (as in spec_verify_check_args).
sv_status check_layout(const spec_verify_config *c, int32_t N, int32_t G, int64_t T, const int32_t *cu) {
  if (N < 0) return fail(SV_ERR_INVALID_ARG, "num_reqs < 0");
  if (G < 0) return fail(SV_ERR_INVALID_ARG, "max_spec_len < 0");
  if (N > c->max_num_reqs) return fail(SV_ERR_CAPACITY, "num_reqs %d > handle max %d", N, c->max_num_reqs);
  if (G > c->max_spec_len) return fail(SV_ERR_CAPACITY, "max_spec_len %d > handle max %d", G, c->max_spec_len);
  if (T < 0) return fail(SV_ERR_INVALID_ARG, "num_draft_tokens_total < 0");
  if (T > static_cast<int64_t>(N) * G) return fail(SV_ERR_INVALID_ARG, "T exceeds num_reqs * max_spec_len");
  if (!cu && T != static_cast<int64_t>(N) * G)
    return fail(SV_ERR_INVALID_ARG, "without cu_num_draft_tokens, T must be num_reqs * max_spec_len");
  return SV_OK;
}

sv_status run_kv(spec_verify_t h, const spec_verify_kv_args *a, void *stream, bool write) {
  if (!h) return fail(SV_ERR_INVALID_ARG, "handle is NULL");
  const sv_status st = spec_verify_check_kv_args(&h->cfg, a);
  if (st != SV_OK) return st;
  if (a->num_tokens == 0) return SV_OK;
  const spec_verify_kv_cache &c = a->cache;
  if (write && ((c.num_blocks > 1 && c.scale_block_stride == 0) || (c.num_kv_heads > 1 && c.scale_head_stride == 0) ||
                (c.block_size > 1 && c.scale_token_stride == 0)))
    return fail(SV_ERR_INVALID_ARG, "rows that share a scale (a scale stride of 0) can be read, not written");
  sv::KvParams p{};
  p.T = a->num_tokens;
  p.c = a->cache;
  p.key = a->key;
  p.value = a->value;
  p.key_token = a->key_token_stride;
  p.key_head = a->key_head_stride;
  p.value_token = a->value_token_stride;
  p.value_head = a->value_head_stride;
  p.slots = a->slot_mapping;
  p.status = a->status;
  p.pdl = !(h->cfg.flags & SV_FLAG_SERIAL_LAUNCH);
  const bool bf16 = a->dtype == SV_BF16;
  const int per32 = bf16 ? 16 : 8;
  const bool vec = ((reinterpret_cast<uintptr_t>(a->key) | reinterpret_cast<uintptr_t>(a->value)) & 31u) == 0 &&
                   a->key_token_stride % per32 == 0 && a->key_head_stride % per32 == 0 &&
                   a->value_token_stride % per32 == 0 && a->value_head_stride % per32 == 0;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = write ? sv::launch_kv_write(p, bf16, vec, s) : sv::launch_kv_read(p, bf16, vec, s);
  if (e != cudaSuccess) return fail(SV_ERR_CUDA, "KV cache launch: %s", cudaGetErrorString(e));
  return SV_OK;
}

}  // namespace

namespace sv {

sv_status check_attend_sizes(const spec_verify_config *c, const spec_verify_attend_args *a) {
  const sv_status st = check_layout(c, a->num_reqs, a->max_spec_len, a->num_draft_tokens_total,
                                    a->cu_num_draft_tokens);
  if (st != SV_OK) return st;
  if (a->cache.num_kv_heads < 1 || a->num_q_heads < 1 || a->num_q_heads % a->cache.num_kv_heads)
    return fail(SV_ERR_INVALID_ARG, "num_q_heads must be a positive multiple of num_kv_heads");
  if (a->cache.head_dim != 64 && a->cache.head_dim != 128)
    return fail(SV_ERR_UNSUPPORTED, "head_dim %d is not 64 or 128", a->cache.head_dim);
  if (a->cache.num_kv_heads > 65535 || a->num_q_heads > 65535)
    return fail(SV_ERR_UNSUPPORTED, "more than 65535 heads");
  if (a->max_seq_len < 0) return fail(SV_ERR_INVALID_ARG, "max_seq_len < 0");
  if (a->max_seq_len > (1 << 30)) return fail(SV_ERR_UNSUPPORTED, "max_seq_len %d > 2^30", a->max_seq_len);
  if (a->shared_prefix_len < 0 || a->shared_prefix_len > a->max_seq_len)
    return fail(SV_ERR_INVALID_ARG, "shared_prefix_len must be in [0, max_seq_len]");
  const int64_t rows = (a->num_draft_tokens_total + a->num_reqs) * static_cast<int64_t>(a->num_q_heads);
  if (rows > INT_MAX / 2) return fail(SV_ERR_UNSUPPORTED, "too many (token, query head) rows for one call");
  return SV_OK;
}

AttendParams attend_params(const spec_verify_t h, const spec_verify_attend_args *a) {
  AttendParams p{};
  p.N = a->num_reqs;
  p.G = a->max_spec_len;
  p.Hq = a->num_q_heads;
  p.group = a->num_q_heads / a->cache.num_kv_heads;
  p.max_seq = a->max_seq_len;
  p.prefix = a->shared_prefix_len;
  p.T = a->num_draft_tokens_total;
  p.cu = a->cu_num_draft_tokens;
  p.c = a->cache;
  p.q = static_cast<const uint16_t *>(a->q);
  p.q_token = a->q_token_stride;
  p.q_head = a->q_head_stride;
  p.tables = a->block_tables;
  // (what the tables hold bounds the lengths too; sizes alone, without a cache, know no tables)
  if (a->cache.block_size > 0 && a->block_tables) {
    const int64_t held = a->block_table_stride * static_cast<int64_t>(a->cache.block_size);
    if (held < p.max_seq) p.max_seq = static_cast<int32_t>(held);
  }
  p.table_stride = a->block_table_stride;
  p.seq_lens = a->seq_lens;
  p.scale = a->scale;
  p.expire = (a->test_flags & SV_TEST_EXPIRE_PRODUCT_WAIT) != 0;
  p.out = static_cast<uint16_t *>(a->out);
  p.out_token = a->out_token_stride;
  p.out_head = a->out_head_stride;
  p.lse = a->lse;
  p.workspace = a->workspace;
  p.status = a->status;
  p.pdl = !(h->cfg.flags & SV_FLAG_SERIAL_LAUNCH);
  return p;
}

// Of the arguments behind the sizes and the cache's description.
sv_status check_attend_call(const spec_verify_attend_args *a) {
  if (a->reserved) return fail(SV_ERR_INVALID_ARG, "reserved must be 0");
  if (a->test_flags & ~SV_TEST_EXPIRE_PRODUCT_WAIT)
    return fail(SV_ERR_INVALID_ARG, "unknown test_flags 0x%x", a->test_flags);
  if (a->num_reqs == 0) return SV_OK;
  const spec_verify_kv_cache &c8 = a->cache;
  const double span = static_cast<double>(c8.num_blocks - 1) * c8.block_stride +
                      static_cast<double>(c8.block_size - 1) * c8.token_stride;
  if (span + static_cast<double>(c8.num_kv_heads - 1) * c8.head_stride >= 0x1p38 || span >= 0x1p32 * cache_unit(c8))
    return fail(SV_ERR_UNSUPPORTED, "a side of the cache spans more than 256 GB, or 2^32 units of %u bytes",
                cache_unit(c8));
  if (a->shared_prefix_len % a->cache.block_size)
    return fail(SV_ERR_INVALID_ARG, "shared_prefix_len must be a multiple of block_size");
  if (a->block_table_stride < 0 ||
      a->shared_prefix_len > a->block_table_stride * static_cast<int64_t>(a->cache.block_size))
    return fail(SV_ERR_INVALID_ARG, "shared_prefix_len exceeds block_table_stride * block_size");
  if (a->max_seq_len > 0 && !a->block_tables) return fail(SV_ERR_INVALID_ARG, "block_tables is NULL");
  if (!a->seq_lens) return fail(SV_ERR_INVALID_ARG, "seq_lens is NULL");
  if (!a->q || !a->out) return fail(SV_ERR_INVALID_ARG, "q or out is NULL");
  if (a->q_token_stride < 0 || a->q_head_stride < 0 || a->out_token_stride < 0 || a->out_head_stride < 0)
    return fail(SV_ERR_INVALID_ARG, "a q or out stride < 0");
  if (!std::isfinite(a->scale)) return fail(SV_ERR_INVALID_ARG, "scale is not finite");
  if (a->workspace_bytes < 0) return fail(SV_ERR_INVALID_ARG, "workspace_bytes < 0");
  if (a->workspace && !aligned16(a->workspace)) return fail(SV_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
  return SV_OK;
}

sv_status run_attend(spec_verify_t h, const AttendParams &p, int64_t workspace_bytes, void *stream) {
  const int64_t need = attend_workspace_bytes(p, h->num_sms, false);
  if (need > 0 && (!p.workspace || workspace_bytes < need))
    return fail(SV_ERR_CAPACITY, "workspace of %lld bytes, the call needs %lld", static_cast<long long>(workspace_bytes),
                static_cast<long long>(need));
  const cudaError_t e = launch_attend(p, h->num_sms, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(SV_ERR_CUDA, "attention launch: %s", cudaGetErrorString(e));
  return SV_OK;
}

}  // namespace sv

extern "C" {

size_t spec_verify_sizeof_kv_args(void) { return sizeof(spec_verify_kv_args); }
size_t spec_verify_sizeof_attend_args(void) { return sizeof(spec_verify_attend_args); }
size_t spec_verify_sizeof_logprobs_args(void) { return sizeof(spec_verify_logprobs_args); }

sv_status spec_verify_check_kv_args(const spec_verify_config *c, const spec_verify_kv_args *a) {
  sv_status st = sv::check_config(c);
  if (st != SV_OK) return st;
  if (!a) return fail(SV_ERR_INVALID_ARG, "args is NULL");
  if (a->num_tokens < 0) return fail(SV_ERR_INVALID_ARG, "num_tokens < 0");
  if (a->dtype != SV_F32 && a->dtype != SV_BF16) return fail(SV_ERR_INVALID_ARG, "bad dtype");
  if (a->reserved) return fail(SV_ERR_INVALID_ARG, "reserved must be 0");
  if ((st = check_cache(a->cache)) != SV_OK) return st;
  if (a->num_tokens > INT_MAX / a->cache.num_kv_heads / 16)  // (two sides of up to eight threads a row)
    return fail(SV_ERR_UNSUPPORTED, "too many tokens for one call");
  if (a->num_tokens == 0) return SV_OK;
  if (!a->key || !a->value) return fail(SV_ERR_INVALID_ARG, "key or value is NULL");
  if (!a->slot_mapping) return fail(SV_ERR_INVALID_ARG, "slot_mapping is NULL");
  if (a->key_token_stride < 0 || a->key_head_stride < 0 || a->value_token_stride < 0 || a->value_head_stride < 0)
    return fail(SV_ERR_INVALID_ARG, "a key or value stride < 0");
  return SV_OK;
}

sv_status spec_verify_kv_write(spec_verify_t h, const spec_verify_kv_args *a, void *stream) {
  return run_kv(h, a, stream, true);
}

sv_status spec_verify_kv_read(spec_verify_t h, const spec_verify_kv_args *a, void *stream) {
  return run_kv(h, a, stream, false);
}

sv_status spec_verify_check_attend_args(const spec_verify_config *c, const spec_verify_attend_args *a) {
  sv_status st = sv::check_config(c);
  if (st != SV_OK) return st;
  if (!a) return fail(SV_ERR_INVALID_ARG, "args is NULL");
  if ((st = sv::check_attend_sizes(c, a)) != SV_OK) return st;
  if (a->num_reqs > 0 && (st = check_cache(a->cache)) != SV_OK) return st;
  return sv::check_attend_call(a);
}

sv_status spec_verify_attend_workspace_size(spec_verify_t h, const spec_verify_attend_args *a, int64_t *bytes) {
  if (!h) return fail(SV_ERR_INVALID_ARG, "handle is NULL");
  if (!a || !bytes) return fail(SV_ERR_INVALID_ARG, "args or bytes is NULL");
  // (a ragged call's T is known without cu, so its check is not the one that forbids a missing cu)
  spec_verify_attend_args b = *a;
  static const int32_t any = 0;
  b.cu_num_draft_tokens = &any;
  const sv_status st = sv::check_attend_sizes(&h->cfg, &b);
  if (st != SV_OK) return st;
  *bytes = a->num_reqs == 0 ? 0 : sv::attend_workspace_bytes(sv::attend_params(h, a), h->num_sms, true);
  return SV_OK;
}

sv_status spec_verify_attend(spec_verify_t h, const spec_verify_attend_args *a, void *stream) {
  if (!h) return fail(SV_ERR_INVALID_ARG, "handle is NULL");
  const sv_status st = spec_verify_check_attend_args(&h->cfg, a);
  if (st != SV_OK) return st;
  if (a->num_reqs == 0) return SV_OK;
  return sv::run_attend(h, sv::attend_params(h, a), a->workspace_bytes, stream);
}

sv_status spec_verify_check_logprobs_args(const spec_verify_config *c, const spec_verify_logprobs_args *a) {
  sv_status st = sv::check_config(c);
  if (st != SV_OK) return st;
  if (!a) return fail(SV_ERR_INVALID_ARG, "args is NULL");
  if ((st = check_layout(c, a->num_reqs, a->max_spec_len, a->num_draft_tokens_total, a->cu_num_draft_tokens)) != SV_OK)
    return st;
  if (a->vocab_size < 1) return fail(SV_ERR_INVALID_ARG, "vocab_size < 1");
  if (a->vocab_size > c->vocab_size)
    return fail(SV_ERR_CAPACITY, "vocab_size %d > handle max %d", a->vocab_size, c->vocab_size);
  if (a->dtype != SV_F32 && a->dtype != SV_BF16) return fail(SV_ERR_INVALID_ARG, "bad dtype");
  if (a->reserved) return fail(SV_ERR_INVALID_ARG, "reserved must be 0");
  if (a->num_top < 0 || a->num_top > a->vocab_size)
    return fail(SV_ERR_INVALID_ARG, "num_top must be in [0, vocab_size]");
  if (a->num_top > SV_MAX_TOP_LOGPROBS)
    return fail(SV_ERR_UNSUPPORTED, "num_top %d > %d", a->num_top, SV_MAX_TOP_LOGPROBS);
  if (static_cast<int64_t>(a->num_reqs) * (a->max_spec_len + 1LL) > INT_MAX / 16)
    return fail(SV_ERR_UNSUPPORTED, "too many token places for one grid");
  if (a->num_reqs == 0) return SV_OK;
  if (!a->logits) return fail(SV_ERR_INVALID_ARG, "logits is NULL");
  if (a->row_stride < a->vocab_size) return fail(SV_ERR_INVALID_ARG, "row_stride < vocab_size");
  if (!a->out_tokens) return fail(SV_ERR_INVALID_ARG, "out_tokens is NULL");
  if (!a->logprobs) return fail(SV_ERR_INVALID_ARG, "logprobs is NULL");
  if (a->num_top > 0 && (!a->top_ids || !a->top_logprobs))
    return fail(SV_ERR_INVALID_ARG, "top_ids / top_logprobs is NULL");
  return SV_OK;
}

sv_status spec_verify_logprobs(spec_verify_t h, const spec_verify_logprobs_args *a, void *stream) {
  if (!h) return fail(SV_ERR_INVALID_ARG, "handle is NULL");
  const sv_status st = spec_verify_check_logprobs_args(&h->cfg, a);
  if (st != SV_OK) return st;
  if (a->num_reqs == 0) return SV_OK;
  sv::LogprobsParams p{};
  p.N = a->num_reqs;
  p.G = a->max_spec_len;
  p.V = a->vocab_size;
  p.K = a->num_top;
  p.T = a->num_draft_tokens_total;
  p.cu = a->cu_num_draft_tokens;
  p.logits = a->logits;
  p.row_stride = a->row_stride;
  p.temperature = a->temperature;
  p.tokens = a->out_tokens;
  p.logprobs = a->logprobs;
  p.ranks = a->ranks;
  p.entropy = a->entropy;
  p.top_ids = a->top_ids;
  p.top_logprobs = a->top_logprobs;
  p.status = a->status;
  p.pdl = !(h->cfg.flags & SV_FLAG_SERIAL_LAUNCH);
  const cudaError_t e = sv::launch_logprobs(p, a->dtype == SV_BF16, h->num_sms, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(SV_ERR_CUDA, "log-probabilities launch: %s", cudaGetErrorString(e));
  return SV_OK;
}

}  // extern "C"
