// sv_step_api.cu -- the C entries of what leads up to a verification step: block
// tables and slots from request lengths, rotary positions, the paged 4-bit KV
// cache and the verify tokens' attention over it.  Host-side validation and
// kernel dispatch; no allocation, no host sync.
#include <climits>
#include <cmath>
#include <cstdint>

#include "sv_internal.h"

namespace {

template <typename... A>
sv_status fail(sv_status s, const char *fmt, A... a) {
  sv::set_last_error(fmt, a...);
  return s;
}

bool aligned(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

sv_status check_cache4(const spec_verify_kv4_cache &c) {
  if (c.format != SV_CACHE_E2M1 && c.format != SV_CACHE_INT4) return fail(SV_ERR_INVALID_ARG, "bad cache format");
  if (c.num_kv_heads < 1) return fail(SV_ERR_INVALID_ARG, "num_kv_heads < 1");
  if (c.head_dim < 1) return fail(SV_ERR_INVALID_ARG, "head_dim < 1");
  if (c.head_dim != 64 && c.head_dim != 128)
    return fail(SV_ERR_UNSUPPORTED, "head_dim %d is not 64 or 128", c.head_dim);
  if (c.num_blocks < 1 || c.block_size < 1) return fail(SV_ERR_INVALID_ARG, "num_blocks or block_size < 1");
  if (c.num_blocks > INT_MAX / c.block_size)
    return fail(SV_ERR_UNSUPPORTED, "a cache of more than 2^31 - 1 slots");
  if (!c.k || !c.v || !c.k_group || !c.v_group || !c.k_scale || !c.v_scale)
    return fail(SV_ERR_INVALID_ARG, "a cache pointer is NULL");
  if (c.block_stride < 0 || c.head_stride < 0 || c.token_stride < 0 || c.group_block_stride < 0 ||
      c.group_head_stride < 0 || c.group_token_stride < 0 || c.scale_block_stride < 0 || c.scale_head_stride < 0 ||
      c.scale_token_stride < 0)
    return fail(SV_ERR_INVALID_ARG, "a cache stride < 0");
  if (!aligned(c.k, 32) || !aligned(c.v, 32) || c.block_stride % 32 || c.head_stride % 32 || c.token_stride % 32)
    return fail(SV_ERR_UNSUPPORTED, "cache rows must start on 32-byte boundaries");
  const int groups = c.head_dim / 16, bytes = c.head_dim / 2;
  if (!aligned(c.k_group, groups) || !aligned(c.v_group, groups) || c.group_block_stride % groups ||
      c.group_head_stride % groups || c.group_token_stride % groups)
    return fail(SV_ERR_UNSUPPORTED, "a row's group scales must start on boundaries of %d bytes", groups);
  if ((c.block_size > 1 && c.token_stride < bytes) || (c.num_kv_heads > 1 && c.head_stride < bytes) ||
      (c.num_blocks > 1 && c.block_stride < bytes))
    return fail(SV_ERR_INVALID_ARG, "cache rows overlap");
  return SV_OK;
}

// What a 4-bit cache has in common with an 8-bit one.
spec_verify_kv_cache common(const spec_verify_kv4_cache &c) {
  spec_verify_kv_cache r{};
  r.k = c.k;
  r.v = c.v;
  r.k_scale = c.k_scale;
  r.v_scale = c.v_scale;
  r.num_blocks = c.num_blocks;
  r.block_size = c.block_size;
  r.num_kv_heads = c.num_kv_heads;
  r.head_dim = c.head_dim;
  r.format = c.format;
  r.block_stride = c.block_stride;
  r.head_stride = c.head_stride;
  r.token_stride = c.token_stride;
  r.scale_block_stride = c.scale_block_stride;
  r.scale_head_stride = c.scale_head_stride;
  r.scale_token_stride = c.scale_token_stride;
  return r;
}
// An attention call's arguments but for its cache's group scales, as those of the 8-bit call.
spec_verify_attend_args common(const spec_verify_attend4_args &a) {
  spec_verify_attend_args r{};
  r.num_reqs = a.num_reqs;
  r.max_spec_len = a.max_spec_len;
  r.num_q_heads = a.num_q_heads;
  r.max_seq_len = a.max_seq_len;
  r.shared_prefix_len = a.shared_prefix_len;
  r.reserved = a.reserved;
  r.num_draft_tokens_total = a.num_draft_tokens_total;
  r.cu_num_draft_tokens = a.cu_num_draft_tokens;
  r.cache = common(a.cache);
  r.q = a.q;
  r.q_token_stride = a.q_token_stride;
  r.q_head_stride = a.q_head_stride;
  r.block_tables = a.block_tables;
  r.block_table_stride = a.block_table_stride;
  r.seq_lens = a.seq_lens;
  r.scale = a.scale;
  r.test_flags = a.test_flags;
  r.out = a.out;
  r.out_token_stride = a.out_token_stride;
  r.out_head_stride = a.out_head_stride;
  r.lse = a.lse;
  r.workspace = a.workspace;
  r.workspace_bytes = a.workspace_bytes;
  r.status = a.status;
  return r;
}

sv::AttendParams attend4_params(const spec_verify_t h, const spec_verify_attend4_args *a) {
  const spec_verify_attend_args b = common(*a);
  sv::AttendParams p = sv::attend_params(h, &b);
  p.k_group = static_cast<const uint8_t *>(a->cache.k_group);
  p.v_group = static_cast<const uint8_t *>(a->cache.v_group);
  p.group_block = a->cache.group_block_stride;
  p.group_head = a->cache.group_head_stride;
  p.group_token = a->cache.group_token_stride;
  return p;
}

sv_status run_kv4(spec_verify_t h, const spec_verify_kv4_args *a, void *stream, bool write) {
  if (!h) return fail(SV_ERR_INVALID_ARG, "handle is NULL");
  const sv_status st = spec_verify_check_kv4_args(&h->cfg, a);
  if (st != SV_OK) return st;
  if (a->num_tokens == 0) return SV_OK;
  const spec_verify_kv4_cache &c = a->cache;
  if (write && ((c.num_blocks > 1 && (c.scale_block_stride == 0 || c.group_block_stride == 0)) ||
                (c.num_kv_heads > 1 && (c.scale_head_stride == 0 || c.group_head_stride == 0)) ||
                (c.block_size > 1 && (c.scale_token_stride == 0 || c.group_token_stride == 0))))
    return fail(SV_ERR_INVALID_ARG, "rows that share a scale (a scale or group stride of 0) can be read, not written");
  sv::Kv4Params p{};
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
  const bool vec = aligned(a->key, 32) && aligned(a->value, 32) && a->key_token_stride % per32 == 0 &&
                   a->key_head_stride % per32 == 0 && a->value_token_stride % per32 == 0 &&
                   a->value_head_stride % per32 == 0;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = write ? sv::launch_kv4_write(p, bf16, vec, s) : sv::launch_kv4_read(p, bf16, vec, s);
  if (e != cudaSuccess) return fail(SV_ERR_CUDA, "4-bit KV cache launch: %s", cudaGetErrorString(e));
  return SV_OK;
}

}  // namespace

extern "C" {

size_t spec_verify_sizeof_kv4_args(void) { return sizeof(spec_verify_kv4_args); }
size_t spec_verify_sizeof_attend4_args(void) { return sizeof(spec_verify_attend4_args); }
size_t spec_verify_sizeof_plan_args(void) { return sizeof(spec_verify_plan_args); }
size_t spec_verify_sizeof_rotate_args(void) { return sizeof(spec_verify_rotate_args); }

sv_status spec_verify_check_kv4_args(const spec_verify_config *c, const spec_verify_kv4_args *a) {
  sv_status st = sv::check_config(c);
  if (st != SV_OK) return st;
  if (!a) return fail(SV_ERR_INVALID_ARG, "args is NULL");
  if (a->num_tokens < 0) return fail(SV_ERR_INVALID_ARG, "num_tokens < 0");
  if (a->dtype != SV_F32 && a->dtype != SV_BF16) return fail(SV_ERR_INVALID_ARG, "bad dtype");
  if (a->reserved) return fail(SV_ERR_INVALID_ARG, "reserved must be 0");
  if ((st = check_cache4(a->cache)) != SV_OK) return st;
  if (a->num_tokens > INT_MAX / a->cache.num_kv_heads / 16)  // (two sides of up to eight threads a row)
    return fail(SV_ERR_UNSUPPORTED, "too many tokens for one call");
  if (a->num_tokens == 0) return SV_OK;
  if (!a->key || !a->value) return fail(SV_ERR_INVALID_ARG, "key or value is NULL");
  if (!a->slot_mapping) return fail(SV_ERR_INVALID_ARG, "slot_mapping is NULL");
  if (a->key_token_stride < 0 || a->key_head_stride < 0 || a->value_token_stride < 0 || a->value_head_stride < 0)
    return fail(SV_ERR_INVALID_ARG, "a key or value stride < 0");
  return SV_OK;
}

sv_status spec_verify_kv4_write(spec_verify_t h, const spec_verify_kv4_args *a, void *stream) {
  return run_kv4(h, a, stream, true);
}

sv_status spec_verify_kv4_read(spec_verify_t h, const spec_verify_kv4_args *a, void *stream) {
  return run_kv4(h, a, stream, false);
}

sv_status spec_verify_check_attend4_args(const spec_verify_config *c, const spec_verify_attend4_args *a) {
  sv_status st = sv::check_config(c);
  if (st != SV_OK) return st;
  if (!a) return fail(SV_ERR_INVALID_ARG, "args is NULL");
  const spec_verify_attend_args b = common(*a);
  if ((st = sv::check_attend_sizes(c, &b)) != SV_OK) return st;
  if (a->num_reqs > 0 && (st = check_cache4(a->cache)) != SV_OK) return st;
  const spec_verify_kv4_cache &c4 = a->cache;
  if (a->num_reqs > 0 && (c4.block_stride > UINT32_MAX || c4.token_stride > UINT32_MAX ||
                          c4.group_block_stride > UINT32_MAX || c4.group_token_stride > UINT32_MAX ||
                          c4.scale_block_stride > UINT32_MAX / 4 || c4.scale_token_stride > UINT32_MAX / 4))
    return fail(SV_ERR_UNSUPPORTED, "a stride between a cache's pages or tokens is 4 GB or more");
  return sv::check_attend_call(&b);
}

sv_status spec_verify_attend4_workspace_size(spec_verify_t h, const spec_verify_attend4_args *a, int64_t *bytes) {
  if (!h) return fail(SV_ERR_INVALID_ARG, "handle is NULL");
  if (!a || !bytes) return fail(SV_ERR_INVALID_ARG, "args or bytes is NULL");
  spec_verify_attend4_args any = *a;
  any.cache.format = SV_CACHE_E2M1;  // (the formats need the same)
  spec_verify_attend_args b = common(any);
  static const int32_t cu = 0;  // (a ragged call's T is known without its prefix sums)
  b.cu_num_draft_tokens = &cu;
  const sv_status st = sv::check_attend_sizes(&h->cfg, &b);
  if (st != SV_OK) return st;
  *bytes = a->num_reqs == 0 ? 0 : sv::attend_workspace_bytes(attend4_params(h, &any), h->num_sms, true);
  return SV_OK;
}

sv_status spec_verify_attend4(spec_verify_t h, const spec_verify_attend4_args *a, void *stream) {
  if (!h) return fail(SV_ERR_INVALID_ARG, "handle is NULL");
  const sv_status st = spec_verify_check_attend4_args(&h->cfg, a);
  if (st != SV_OK) return st;
  if (a->num_reqs == 0) return SV_OK;
  return sv::run_attend(h, attend4_params(h, a), a->workspace_bytes, stream);
}

sv_status spec_verify_check_plan_args(const spec_verify_config *c, const spec_verify_plan_args *a) {
  const sv_status st = sv::check_config(c);
  if (st != SV_OK) return st;
  if (!a) return fail(SV_ERR_INVALID_ARG, "args is NULL");
  if (a->num_reqs < 0) return fail(SV_ERR_INVALID_ARG, "num_reqs < 0");
  if (a->num_reqs > c->max_num_reqs)
    return fail(SV_ERR_CAPACITY, "num_reqs %d > handle max %d", a->num_reqs, c->max_num_reqs);
  if (a->block_size < 1) return fail(SV_ERR_INVALID_ARG, "block_size < 1");
  if (a->table_width < 0) return fail(SV_ERR_INVALID_ARG, "table_width < 0");
  if (a->num_shared_pages < 0 || a->num_shared_pages > a->table_width)
    return fail(SV_ERR_INVALID_ARG, "num_shared_pages must be in [0, table_width]");
  if (a->num_rows < 0) return fail(SV_ERR_INVALID_ARG, "num_rows < 0");
  if (a->num_rows > INT_MAX - 65536) return fail(SV_ERR_UNSUPPORTED, "too many rows for one call");
  if (a->block_table_stride < a->table_width)
    return fail(SV_ERR_INVALID_ARG, "block_table_stride must be at least table_width");
  if (a->free_capacity < 1) return fail(SV_ERR_INVALID_ARG, "free_capacity < 1");
  if (a->free_capacity > INT_MAX) return fail(SV_ERR_UNSUPPORTED, "free_capacity > 2^31 - 1");
  if (!a->free_pages || !a->free_range || !a->free_range_out)
    return fail(SV_ERR_INVALID_ARG, "free_pages, free_range or free_range_out is NULL");
  if (a->num_rows > 0 && (!a->positions || !a->slot_mapping))
    return fail(SV_ERR_INVALID_ARG, "positions or slot_mapping is NULL");
  if (a->workspace_bytes < 0) return fail(SV_ERR_INVALID_ARG, "workspace_bytes < 0");
  if (a->workspace && !aligned(a->workspace, 16)) return fail(SV_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
  if (a->num_reqs == 0) return SV_OK;
  if (!a->num_new_tokens || !a->num_computed_tokens || !a->held_pages)
    return fail(SV_ERR_INVALID_ARG, "num_new_tokens, num_computed_tokens or held_pages is NULL");
  if (!a->held_pages_out || !a->seq_lens) return fail(SV_ERR_INVALID_ARG, "held_pages_out or seq_lens is NULL");
  if (a->table_width > 0 && !a->block_tables) return fail(SV_ERR_INVALID_ARG, "block_tables is NULL");
  return SV_OK;
}

sv_status spec_verify_plan_workspace_size(spec_verify_t h, int32_t num_reqs, int64_t *bytes) {
  if (!h) return fail(SV_ERR_INVALID_ARG, "handle is NULL");
  if (!bytes) return fail(SV_ERR_INVALID_ARG, "bytes is NULL");
  if (num_reqs < 0) return fail(SV_ERR_INVALID_ARG, "num_reqs < 0");
  if (num_reqs > h->cfg.max_num_reqs)
    return fail(SV_ERR_CAPACITY, "num_reqs %d > handle max %d", num_reqs, h->cfg.max_num_reqs);
  *bytes = sv::plan_workspace_bytes(num_reqs);
  return SV_OK;
}

sv_status spec_verify_plan_step(spec_verify_t h, const spec_verify_plan_args *a, void *stream) {
  if (!h) return fail(SV_ERR_INVALID_ARG, "handle is NULL");
  const sv_status st = spec_verify_check_plan_args(&h->cfg, a);
  if (st != SV_OK) return st;
  const int64_t need = sv::plan_workspace_bytes(a->num_reqs);
  if (!a->workspace || a->workspace_bytes < need)
    return fail(SV_ERR_CAPACITY, "workspace of %lld bytes, the call needs %lld",
                static_cast<long long>(a->workspace ? a->workspace_bytes : 0), static_cast<long long>(need));
  sv::PlanParams p{};
  p.N = a->num_reqs;
  p.block = a->block_size;
  p.width = a->table_width;
  p.shared = a->num_shared_pages;
  p.page = sv::fast_div(a->block_size);
  p.R = a->num_rows;
  p.fresh = a->num_new_tokens;
  p.computed = a->num_computed_tokens;
  p.tables = a->block_tables;
  p.table_stride = a->block_table_stride;
  p.held = a->held_pages;
  p.held_out = a->held_pages_out;
  p.ring = a->free_pages;
  p.capacity = a->free_capacity;
  p.range = a->free_range;
  p.range_out = a->free_range_out;
  p.positions = a->positions;
  p.slots = a->slot_mapping;
  p.seq_lens = a->seq_lens;
  p.cu = a->cu_num_draft_tokens;
  p.workspace = a->workspace;
  p.status = a->status;
  p.pdl = !(h->cfg.flags & SV_FLAG_SERIAL_LAUNCH);
  const cudaError_t e = sv::launch_plan(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(SV_ERR_CUDA, "plan launch: %s", cudaGetErrorString(e));
  return SV_OK;
}

sv_status spec_verify_check_rotate_args(const spec_verify_config *c, const spec_verify_rotate_args *a) {
  const sv_status st = sv::check_config(c);
  if (st != SV_OK) return st;
  if (!a) return fail(SV_ERR_INVALID_ARG, "args is NULL");
  if (a->num_tokens < 0) return fail(SV_ERR_INVALID_ARG, "num_tokens < 0");
  if (a->dtype != SV_F32 && a->dtype != SV_BF16) return fail(SV_ERR_INVALID_ARG, "bad dtype");
  if (a->head_dim < 1) return fail(SV_ERR_INVALID_ARG, "head_dim < 1");
  if (a->head_dim > SV_MAX_ROTATE_HEAD_DIM)
    return fail(SV_ERR_UNSUPPORTED, "head_dim %d > %d", a->head_dim, SV_MAX_ROTATE_HEAD_DIM);
  if (a->rotary_dim < 0 || a->rotary_dim > a->head_dim || a->rotary_dim % 2)
    return fail(SV_ERR_INVALID_ARG, "rotary_dim must be even and in [0, head_dim]");
  if (a->num_q_heads < 0 || a->num_k_heads < 0) return fail(SV_ERR_INVALID_ARG, "num_q_heads or num_k_heads < 0");
  if (a->num_q_heads > 65535 || a->num_k_heads > 65535) return fail(SV_ERR_UNSUPPORTED, "more than 65535 heads");
  if (a->flags & ~SV_ROTATE_INTERLEAVED) return fail(SV_ERR_INVALID_ARG, "unknown flags 0x%x", a->flags);
  if (!std::isfinite(a->magnitude)) return fail(SV_ERR_INVALID_ARG, "magnitude is not finite");
  if (!(a->eps >= 0.0f) || !std::isfinite(a->eps)) return fail(SV_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (a->num_tokens > INT_MAX / 64) return fail(SV_ERR_UNSUPPORTED, "too many tokens for one call");
  if (a->num_tokens == 0 || a->num_q_heads + a->num_k_heads == 0) return SV_OK;
  if (!a->positions) return fail(SV_ERR_INVALID_ARG, "positions is NULL");
  if (a->rotary_dim > 0 && !a->turns) return fail(SV_ERR_INVALID_ARG, "turns is NULL");
  if (a->num_q_heads > 0 && (!a->q || !a->q_out)) return fail(SV_ERR_INVALID_ARG, "q or q_out is NULL");
  if (a->num_k_heads > 0 && (!a->key || !a->key_out)) return fail(SV_ERR_INVALID_ARG, "key or key_out is NULL");
  if (a->q_token_stride < 0 || a->q_head_stride < 0 || a->q_out_token_stride < 0 || a->q_out_head_stride < 0 ||
      a->key_token_stride < 0 || a->key_head_stride < 0 || a->key_out_token_stride < 0 || a->key_out_head_stride < 0)
    return fail(SV_ERR_INVALID_ARG, "a stride < 0");
  return SV_OK;
}

sv_status spec_verify_rotate(spec_verify_t h, const spec_verify_rotate_args *a, void *stream) {
  if (!h) return fail(SV_ERR_INVALID_ARG, "handle is NULL");
  const sv_status st = spec_verify_check_rotate_args(&h->cfg, a);
  if (st != SV_OK) return st;
  if (a->num_tokens == 0 || a->num_q_heads + a->num_k_heads == 0) return SV_OK;
  sv::RotateParams p{};
  p.T = a->num_tokens;
  p.D = a->head_dim;
  p.rotary = a->rotary_dim;
  p.Hq = a->num_q_heads;
  p.Hk = a->num_k_heads;
  p.interleaved = (a->flags & SV_ROTATE_INTERLEAVED) != 0;
  p.q = sv::RotateSide{a->q, a->q_out, a->q_weight, a->q_token_stride, a->q_head_stride, a->q_out_token_stride,
                       a->q_out_head_stride};
  p.k = sv::RotateSide{a->key, a->key_out, a->key_weight, a->key_token_stride, a->key_head_stride,
                       a->key_out_token_stride, a->key_out_head_stride};
  p.positions = a->positions;
  p.turns = a->turns;
  p.magnitude = a->magnitude;
  p.eps = a->eps;
  p.pdl = !(h->cfg.flags & SV_FLAG_SERIAL_LAUNCH);
  const cudaError_t e = sv::launch_rotate(p, a->dtype == SV_BF16, h->num_sms, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(SV_ERR_CUDA, "rotary launch: %s", cudaGetErrorString(e));
  return SV_OK;
}

}  // extern "C"
