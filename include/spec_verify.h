/*
 * spec_verify.h -- C ABI of the batched speculative-decoding verifier
 * (rejection sampler) for NVIDIA GB300 (sm_103a).
 *
 * What it computes (page titles and sections of the sources it follows):
 *  - "Speculative Decoding: propose, verify, accept", section 02: per request
 *    draft ids [gamma], draft distributions q [gamma, V] and target
 *    distributions p [gamma+1, V]; section 04: draft y is accepted iff
 *    u < min(1, p(y)/q(y)), evaluated here as fl32(u * q(y)) < p(y); the first
 *    rejection is replaced by a draw from max(0, p - q) renormalised;
 *    section 06: keep the accepted prefix, stop at the first rejection, draw a
 *    bonus token from p[gamma] when every draft is accepted; section 03:
 *    temperature 0 compares the draft with the target argmax.
 *  - "vLLM source walk-through (10): speculative decoding", section
 *    "SpecDecodeMetadata": flattened drafts with cu_num_draft_tokens (inclusive
 *    prefix sums) and max_spec_len; section "Rejection sampling: the two
 *    branches of RejectionSampler": identical temperature/top-k/top-p on the
 *    target and draft sides, output [batch, max_spec_len + 1] filled with
 *    PLACEHOLDER_TOKEN_ID = -1; section "Random kernel": categorical draws by
 *    an exponential race (argmax of weight / exponential draw); section
 *    "Scheduler and KV": rejected draft KV slots become PADDING_SLOT_ID = -1.
 *  - "How speculative decoding interacts with the KV cache", section 3.1:
 *    num_computed_tokens -= gamma - A when it is > 0.
 *
 * Memory and execution model: every pointer in spec_verify_args is a DEVICE
 * pointer on the handle's device, owned by the caller (the library allocates
 * nothing per call).  For the probability entry, target/draft/exponentials may
 * also point into pinned host memory mapped into the device address space
 * (unified addressing): the kernel then reads only the rows a call needs over
 * the host link (NVLink-C2C on GB300).  The logits entry needs device rows.  spec_verify_run only validates on the host and enqueues
 * kernels on the caller's stream; it never synchronises.  Errors visible on
 * the host are returned before anything is enqueued.  Errors in the data are
 * reported through the optional device word `status` (bitwise OR of
 * SV_DATA_* bits; the caller zeroes it) and never trap: a request with invalid
 * data emits nothing (its output row stays -1, num_accepted 0, KV bookkeeping
 * untouched).  One handle may be used from one host thread at a time; calls on
 * different streams must not share output buffers.
 */
#ifndef SPEC_VERIFY_H_
#define SPEC_VERIFY_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SPEC_VERIFY_ABI_VERSION 8u
#define SV_PLACEHOLDER_TOKEN_ID (-1)
#define SV_PADDING_SLOT_ID (-1)
#define SV_MAX_SPEC_LEN 256 /* largest max_spec_len a handle accepts */
#define SV_MAX_NGRAM 64     /* largest max_ngram of the n-gram proposer */

/* Host-visible result codes. */
typedef enum sv_status {
  SV_OK = 0,
  SV_ERR_INVALID_ARG = 1, /* a null, negative, out-of-range or inconsistent argument */
  SV_ERR_UNSUPPORTED = 2, /* a combination this build does not implement (e.g. probs + bf16) */
  SV_ERR_CUDA = 3,        /* a CUDA runtime call failed; see spec_verify_last_error() */
  SV_ERR_CAPACITY = 4     /* the call exceeds the limits the handle was created with */
} sv_status;

/* Input kinds. */
enum sv_entry {
  SV_ENTRY_PROBS = 0, /* target/draft rows are fp32 probabilities, already transformed */
  SV_ENTRY_LOGITS = 1 /* target/draft rows are logits; temperature/top-k/top-p applied here */
};
enum sv_dtype { SV_F32 = 0, SV_BF16 = 1 };

/* Device status bits (bitwise OR into *status). */
enum sv_data_status {
  SV_DATA_BAD_CU = 1,             /* cu_num_draft_tokens not a valid range for this request */
  SV_DATA_BAD_DRAFT_ID = 2,       /* draft id outside [0, V) at an examined position */
  SV_DATA_BAD_EXPONENTIAL = 4,    /* test-mode E <= 0 or NaN where a key needed it (key taken as 0) */
  SV_DATA_EMPTY_DISTRIBUTION = 8, /* a draw found no positive key; token 0 emitted */
  SV_DATA_BAD_VALUES = 16,        /* NaN (greedy) or NaN/+inf/no finite logit (random logits) in a read row,
                                     or a kept set left empty by banned tokens */
  SV_DATA_BAD_PARAM = 32,         /* temperature < 0/NaN/inf/subnormal, or top_p <= 0/NaN */
  SV_DATA_MISSING_DRAFT = 64,     /* draft == NULL but a random request needs draft rows */
  SV_DATA_COPY_TIMEOUT = 128,     /* a bulk row copy did not complete within its wait limit (request
                                     emits nothing); never expected on a healthy GPU */
  SV_DATA_BAD_LIST = 256,         /* a penalty, banned or stop list range of the request is invalid */
  SV_DATA_BAD_SLOT = 512,         /* a KV slot or a block-table entry outside the cache (the token is left out) */
  SV_DATA_NO_PAGES = 1024         /* the free pages do not suffice for a request (it gets none) */
};

/* Handle flags.  SV_FLAG_RESIDENT_ROWS: the logits entry copies both the
 * target and the draft row chunk of a position into shared memory (two CTAs
 * per SM), and the sampler its row chunk.  By default aligned rows are read
 * in place after an L2 prefetch (four CTAs per SM); unaligned rows are always
 * copied.  Results are identical. */
#define SV_FLAG_RESIDENT_ROWS 1u
/* SV_FLAG_ONE_CTA_PER_REQUEST: logits-entry and sampler calls with aligned
 * rows (with or without logits processors), in a handle without
 * SV_FLAG_RESIDENT_ROWS, always take the
 * one-CTA-per-request (per-row) form (see SV_HINT_SMALL_TOP_K); by default
 * the library takes it only for hinted calls with at least two requests
 * (rows) per SM.  Without processors the two forms' results are identical;
 * with processors both stay within the tolerance of the exact definition
 * (the one-CTA form sums the processed kept set afresh, the cluster form
 * corrects the raw sum). */
#define SV_FLAG_ONE_CTA_PER_REQUEST 2u
/* SV_FLAG_SERIAL_LAUNCH: launch the handle's kernels in plain stream order.
 * By default every kernel is launched with programmatic stream serialization
 * (CUDA's programmatic dependent launch): it may be scheduled onto the SMs
 * while the previous kernel in the stream is still running, and its first
 * instruction waits until that kernel has completed and all of its memory
 * writes are visible.  Nothing is read or written earlier than in plain stream
 * order, so results are identical; only the gap between back-to-back kernels
 * shrinks.  Work that is not a kernel (copies, event records, host callbacks)
 * orders the stream as usual. */
#define SV_FLAG_SERIAL_LAUNCH 4u

/* Call hints (the hints field of spec_verify_args and spec_verify_sample_args;
 * they never change a result).  SV_HINT_SMALL_TOP_K: the caller states that
 * every random request (row) of the call has 1 <= top_k <= SV_SMALL_TOP_K_MAX.
 * For such a batch, large enough to give every request its own CTA at once,
 * the sampler samples each row with one CTA the same way, and the logits entry verifies
 * each request with one CTA that reads a position's two rows once (keeping
 * the largest key of every 128-byte block), reads again the few blocks that
 * can hold the top-k set, and derives the threshold, the top-p cut, the
 * normaliser and the race from those candidates; a request outside the
 * statement is still verified exactly, by a slower multi-pass path. */
#define SV_HINT_SMALL_TOP_K 1u
#define SV_SMALL_TOP_K_MAX 256

/* Call flags for tests (the test_flags field of the argument structs; 0 in
 * normal use).  SV_TEST_EXPIRE_COPY_WAIT: the first wait for every bulk row
 * copy into shared memory gives up at once, as if the copy had not completed
 * within its limit; the copy still gets the ordinary second wait, so it lands
 * before the CTA moves on.  The requests that copied rows then report
 * SV_DATA_COPY_TIMEOUT and emit nothing.  Only calls whose rows are copied
 * (SV_FLAG_RESIDENT_ROWS, or unaligned rows) are affected. */
#define SV_TEST_EXPIRE_COPY_WAIT 1u
/* SV_TEST_EXPIRE_PRODUCT_WAIT (attention calls): where a shared prefix is met
 * by the tensor cores, the first wait for a tile's weights gives up at once, as
 * if they had not come within its limit.  What is in flight still ends before
 * the CTA does. */
#define SV_TEST_EXPIRE_PRODUCT_WAIT 2u

typedef struct spec_verify_ctx *spec_verify_t;

/* Limits fixed at creation. */
typedef struct spec_verify_config {
  int32_t max_num_reqs; /* largest num_reqs of any call (>= 1) */
  int32_t max_spec_len; /* largest max_spec_len of any call (0 .. SV_MAX_SPEC_LEN) */
  int32_t vocab_size;   /* largest vocab_size of any call (>= 1) */
  int32_t device;       /* CUDA device ordinal the handle's calls run on */
  int32_t cluster_ctas; /* CTAs cooperating on one request: 0 = automatic, else 1, 2, 4, 8 or 16 */
  uint32_t flags;       /* 0, or SV_FLAG_* bits */
} spec_verify_config;

/* One verification call.  N = num_reqs, G = max_spec_len, V = vocab_size,
 * T = num_draft_tokens_total.  Request i owns draft rows [s_i, s_i + gamma_i)
 * and target rows [s_i + i, s_i + i + gamma_i] (its last target row is the
 * bonus row), where s_i = cu[i-1] (0 for i = 0) and gamma_i = cu[i] - s_i. */
typedef struct spec_verify_args {
  int32_t num_reqs;     /* N >= 0 (N = 0 is a no-op) */
  int32_t max_spec_len; /* G: output row length is G + 1; every gamma_i <= G */
  int32_t vocab_size;   /* V >= 1 */
  int32_t entry;        /* SV_ENTRY_PROBS or SV_ENTRY_LOGITS */
  int32_t dtype;        /* SV_F32 (both entries) or SV_BF16 (logits entry only) */
  uint32_t hints;       /* 0, or SV_HINT_* bits */
  int64_t num_draft_tokens_total; /* T = cu[N-1]; must equal N*G when cu == NULL */

  const int32_t *draft_ids;           /* [T] draft token ids, request-major */
  const int32_t *cu_num_draft_tokens; /* [N] inclusive prefix sums, or NULL: every gamma_i = G */
  const void *target;                 /* [T+N rows, target_row_stride] p rows or target logits */
  int64_t target_row_stride;          /* elements between target rows (>= V) */
  const void *draft;                  /* [T rows, draft_row_stride] q rows or draft logits; may be NULL
                                         when no random request has drafts */
  int64_t draft_row_stride;           /* elements between draft rows (>= V) */

  const float *temperature; /* [N]; 0 selects the greedy path; NULL = 1 for every request */
  const int32_t *top_k;     /* [N] or NULL; <= 0 or >= V disables (logits entry only) */
  const float *top_p;       /* [N] or NULL; >= 1 disables; must be > 0 (logits entry only) */

  /* Randomness.  Test mode: exponentials set (and uniforms, unless T = 0);
   * u [T] in [0, 1) and E [N rows, exponentials_row_stride] > 0 are read as
   * given.  Production mode: both NULL; u and E come from Philox4x32-10 (Salmon et al., SC'11) with key
   * (seed) and counters (j/4, 2r+1, offset) for u_j and (x/4, 2r, offset) for
   * E(x), r = rng_request_base + i; u = (w >> 8) 2^-24, E = -ln((2(w >> 9)+1) 2^-24). */
  const float *uniforms;
  const float *exponentials;
  int64_t exponentials_row_stride;
  uint64_t seed;
  uint64_t offset;
  uint32_t rng_request_base;
  uint32_t test_flags; /* 0, or SV_TEST_EXPIRE_COPY_WAIT (tests only) */

  /* Outputs. */
  int32_t *out_tokens;          /* [N, G+1] committed tokens, -1 after the last one */
  int32_t *num_accepted;        /* [N] accepted draft count A */
  int32_t *num_computed_tokens; /* [N] in/out or NULL: -= gamma_i - A when > 0 */
  int64_t *slot_mapping;        /* [T+N] in/out or NULL: verify tokens j in (A, gamma_i] -> -1 */
  float *dbg_py;                /* [T] or NULL: p_j(y_j) at examined positions j <= min(A, gamma_i - 1) */
  float *dbg_qy;                /* [T] or NULL: q_j(y_j) at the same positions */
  int32_t *status;              /* [1] or NULL: SV_DATA_* bits OR-ed in */

  /* Synthetic acceptance ("vLLM source walk-through (10)", section "About
   * synthetic / block verification": preset per-position rates, non-increasing,
   * accept with "uniform < rate" instead of the probability test).  [G] device
   * array in [0, 1], or NULL for the ordinary test.  Only the decision changes:
   * rows before the stopping position are never read, the replacement or bonus
   * draw there is the ordinary one, and dbg_py/dbg_qy are not written.  Rates
   * outside [0, 1] or increasing over a request's positions: SV_DATA_BAD_PARAM. */
  const float *synthetic_acceptance_rates;

  /* Logits processors, logits entry only ("Speculative Decoding: propose,
   * verify, accept", section 06: the same banned tokens and repetition penalty
   * on p and q at a position, after temperature, top-k and top-p; "vLLM
   * source walk-through (10)", section "Rejection sampling: the two branches
   * of RejectionSampler", step 2: the sampling constraints first, then the
   * processors).  Lists are per request, like cu_num_draft_tokens: request i
   * owns entries [cu[i-1], cu[i]) (cu[-1] = 0) of the id array; ids outside
   * [0, V) are ignored and repeats count once.  A banned token's logit
   * becomes -inf.  With repetition_penalty, every distinct token of the
   * request's penalty list, plus the drafts y_0 .. y_{j-1} when position j is
   * verified, has its logit l replaced by l / theta if l > 0, else l * theta
   * (fp32 arithmetic, rounded to the logits' type), on the target and the
   * draft row alike; banned tokens are not penalised.  On a random row the
   * kept set is placed on the raw logits (temperature, top-k, top-p); the
   * processed values then replace the kept logits and the kept set is
   * renormalised (an entry the cuts dropped stays dropped; a kept set whose
   * every entry is banned is SV_DATA_BAD_VALUES).  A greedy row takes the
   * argmax of the whole processed row.  Theta must be > 0 and finite (else
   * SV_DATA_BAD_PARAM).  The probability entry rejects these fields (its rows
   * are already transformed). */
  const float *repetition_penalty;    /* [N] theta, or NULL: no penalty */
  const int64_t *penalty_cu;          /* [N] or NULL */
  const int32_t *penalty_token_ids;   /* [penalty_total] */
  int64_t penalty_total;
  const int64_t *banned_cu;           /* [N] or NULL */
  const int32_t *banned_token_ids;    /* [banned_total] */
  int64_t banned_total;

  /* Stop tokens, both entries ("Speculative Decoding: propose, verify,
   * accept", sections 13-14: stop rules are checked on the committed prefix
   * only, token by token).  If a committed token c_m (m <= A) is in the
   * request's stop list, the commit ends at the first such m: out row
   * c_0 .. c_m, num_accepted = m, and the KV rollback follows (gamma_i - m
   * tokens, slots of verify tokens m+1 .. gamma_i). */
  const int64_t *stop_cu;             /* [N] or NULL */
  const int32_t *stop_token_ids;      /* [stop_total] */
  int64_t stop_total;
} spec_verify_args;

/* Draft-side sampler ("vLLM source walk-through (10)", section "propose()
 * multi-step loop": each draft step samples its token from the draft model's
 * distribution and keeps that distribution for the rejection sampler).  One
 * token per logits row: the row goes through the verifier's own transform
 * (temperature, top-k, softmax, top-p) and the token is drawn by the same
 * exponential race; temperature 0 takes the argmax (lowest index).  The
 * transformed fp32 row can be written out, ready to be the q input of the
 * probability entry.  R = num_rows, V = vocab_size.  Production draws use the
 * verifier's E counters under the key (seed_lo, seed_hi ^ 0x53414D50), so a
 * sampler call and a verifier call with the same seed never share a stream. */
typedef struct spec_verify_sample_args {
  int32_t num_rows;   /* R >= 0 (0 is a no-op); at most the handle's max_num_reqs */
  int32_t vocab_size; /* V, at most the handle's vocab_size */
  int32_t dtype;      /* SV_F32 or SV_BF16 logits */
  uint32_t hints;     /* 0, or SV_HINT_* bits */
  const void *logits; /* [R rows, row_stride] */
  int64_t row_stride; /* elements between rows (>= V) */
  const float *temperature; /* [R] or NULL (= 1) */
  const int32_t *top_k;     /* [R] or NULL */
  const float *top_p;       /* [R] or NULL */
  const float *exponentials; /* test mode: [R rows, exponentials_row_stride] E > 0; NULL = Philox */
  int64_t exponentials_row_stride;
  uint64_t seed;
  uint64_t offset;
  uint32_t rng_row_base; /* stream of row r: rng_row_base + r */
  uint32_t test_flags;   /* 0, or SV_TEST_EXPIRE_COPY_WAIT (tests only) */
  int32_t *tokens;       /* [R] out: sampled token, -1 for an invalid row */
  float *probs;          /* [R rows, probs_row_stride] out or NULL: the transformed row (random rows only) */
  int64_t probs_row_stride;
  int32_t *status;       /* [1] or NULL: SV_DATA_* bits OR-ed in */

  /* Logits processors per row, as in spec_verify_args (row r = request r;
   * no drafts are added implicitly: a row's penalty list holds its whole
   * context, drafts sampled before it included), so that the sampled q is the
   * q the verifier rebuilds. */
  const float *repetition_penalty;    /* [R] theta, or NULL */
  const int64_t *penalty_cu;          /* [R] or NULL */
  const int32_t *penalty_token_ids;
  int64_t penalty_total;
  const int64_t *banned_cu;           /* [R] or NULL */
  const int32_t *banned_token_ids;
  int64_t banned_total;
} spec_verify_sample_args;

sv_status spec_verify_sample(spec_verify_t handle, const spec_verify_sample_args *args, void *stream);

/* Host-only validation of sampler arguments against `config`. */
sv_status spec_verify_check_sample_args(const spec_verify_config *config, const spec_verify_sample_args *args);

/* Batched n-gram proposer ("vLLM source walk-through (10)", section
 * "NgramProposer": no draft model; the tail of a request's token history is
 * looked up earlier in the history -- the history read backwards, match
 * lengths capped at max_ngram -- and the longest match with a length in
 * [min_ngram, max_ngram] proposes the tokens that followed it).  Exactly: for
 * every end position E <= L - 2 of a request's history t[0 .. L), l(E) is the
 * number of j = 0, 1, ... with t[E - j] == t[L - 1 - j], capped at max_ngram
 * and at E + 1.  The proposal follows the E with the largest l(E), the latest
 * such E on ties (the most recent occurrence), if that l is at least
 * min_ngram: draft = t[E + 1 .. E + 1 + k'), k' = min(k, max_model_len - L,
 * L - 1 - E).  Otherwise nothing is proposed.  R = num_reqs; one CTA per
 * request reads its history once from HBM. */
typedef struct spec_verify_ngram_args {
  int32_t num_reqs;        /* R >= 0 (0 is a no-op); at most the handle's max_num_reqs */
  int32_t min_ngram;       /* 1 <= min_ngram <= max_ngram */
  int32_t max_ngram;       /* max_ngram <= SV_MAX_NGRAM */
  int32_t num_spec_tokens; /* k: 0 .. the handle's max_spec_len */
  int64_t max_model_len;   /* >= 1: a history of L tokens gets at most max_model_len - L */
  int64_t num_tokens_total;              /* length of token_ids (>= 0) */
  const int32_t *token_ids;              /* [num_tokens_total] histories, request after request */
  const int64_t *cu_num_tokens;          /* [R] inclusive prefix sums: request q owns [cu[q-1], cu[q]), cu[-1] = 0 */
  int32_t *draft_token_ids;              /* [R, k] out: the proposal, then -1 (may be NULL when k == 0) */
  int32_t *num_draft_tokens;             /* [R] out: k' (0 when nothing is proposed or the range is bad) */
  int32_t *status;                       /* [1] or NULL: SV_DATA_BAD_CU OR-ed in for a bad range */
} spec_verify_ngram_args;

sv_status spec_verify_ngram_propose(spec_verify_t handle, const spec_verify_ngram_args *args, void *stream);

/* Host-only validation of n-gram proposer arguments against `config`. */
sv_status spec_verify_check_ngram_args(const spec_verify_config *config, const spec_verify_ngram_args *args);

/* ---------------------------------------------------------------------------
 * The paged 8-bit KV cache, and the verify tokens' attention over it.
 *
 * A cache is num_blocks pages of block_size tokens.  The K (V) row of token
 * offset t of page b and kv head h is head_dim bytes at
 * k (v) + b * block_stride + h * head_stride + t * token_stride, and its scale
 * is the float at b * scale_block_stride + h * scale_head_stride +
 * t * scale_token_stride: byte x stands for x * scale.  Head-major and
 * token-major pages are both strides.  Slot s (the framework's slot_mapping,
 * "How speculative decoding interacts with the KV cache", section 3.2) is page
 * s / block_size, offset s % block_size.
 *
 * Quantising a row x: scale = max(max_d |x_d| / Q, 2^-64) with Q = 127 (int8)
 * or 448 (e4m3), byte = x / scale rounded to nearest even (IEEE division).
 * 2^-64 keeps the scale of a zero row positive.  A row that holds a NaN or an
 * infinity gets scale NaN and zero bytes (it reads back as NaN) and raises
 * SV_DATA_BAD_VALUES.
 */
enum sv_cache_format { SV_CACHE_INT8 = 0, SV_CACHE_E4M3 = 1 };

typedef struct spec_verify_kv_cache {
  void *k, *v;              /* 16-byte aligned; strides in bytes, multiples of 16 */
  float *k_scale, *v_scale; /* strides in elements */
  int64_t num_blocks;       /* >= 1; num_blocks * block_size <= 2^31 - 1 pages' tokens */
  int32_t block_size;       /* >= 1 (any: a power of two is not needed) */
  int32_t num_kv_heads;     /* >= 1 */
  int32_t head_dim;         /* 64 or 128 */
  int32_t format;           /* SV_CACHE_* */
  int64_t block_stride, head_stride, token_stride;
  int64_t scale_block_stride, scale_head_stride, scale_token_stride;
} spec_verify_kv_cache;

/* Writing tokens to the cache, and reading them back.  Row (t, h) of key
 * (value) is head_dim elements of `dtype` at element t * token_stride +
 * h * head_stride.  slot_mapping[t] = SV_PADDING_SLOT_ID (-1), as the verifier
 * leaves it for rejected drafts: a write skips the token, a read gives zeros.
 * Any other slot outside the cache does the same and raises SV_DATA_BAD_SLOT.
 * Two tokens of one call must not share a slot.  Rows that share a scale (a
 * scale stride of 0 along more than one element) can be read, not written. */
typedef struct spec_verify_kv_args {
  int64_t num_tokens; /* T >= 0 (0 is a no-op) */
  int32_t dtype;      /* SV_F32 or SV_BF16: the elements of key and value */
  uint32_t reserved;  /* 0 */
  spec_verify_kv_cache cache;
  void *key;   /* read by spec_verify_kv_write, written by spec_verify_kv_read */
  int64_t key_token_stride, key_head_stride;
  void *value;
  int64_t value_token_stride, value_head_stride;
  const int64_t *slot_mapping; /* [T] */
  int32_t *status;             /* [1] or NULL: SV_DATA_* bits OR-ed in */
} spec_verify_kv_args;

sv_status spec_verify_kv_write(spec_verify_t handle, const spec_verify_kv_args *args, void *stream);
sv_status spec_verify_kv_read(spec_verify_t handle, const spec_verify_kv_args *args, void *stream);

/* Host-only validation of the arguments of either call against `config`. */
sv_status spec_verify_check_kv_args(const spec_verify_config *config, const spec_verify_kv_args *args);

/* Attention of the verify tokens over the cache, whose sides may each span 256
 * GB from the first page to the last (but no more than 2^32 times the largest
 * power of two that divides the block and token strides).  The tokens are laid
 * out as the target rows of spec_verify_args: request i owns rows s_i + i ..
 * s_i + i + gamma_i of q, out and lse.  seq_lens[i] = L counts the request's
 * keys, its own gamma_i + 1 verify tokens (already written) included; row j is
 * at position L - (gamma_i + 1) + j and sees the keys 0 .. position.  Query
 * head x reads kv head x / (num_q_heads / num_kv_heads).
 *   s_k = scale * q . key_k;  lse = ln sum_k exp s_k;
 *   out = sum_k exp(s_k - lse) value_k
 * A row that sees no key (L = 0, say) gives out = 0 and lse = -infinity.
 * Key k of request i is at page block_tables[i, k / block_size], offset
 * k % block_size.  The first shared_prefix_len tokens (a multiple of
 * block_size) are the same pages for every request -- entries
 * 0 .. shared_prefix_len / block_size - 1 of row 0 of block_tables stand for
 * all -- and are read once for the whole batch where that pays.  A page outside the cache
 * leaves its keys out and raises SV_DATA_BAD_SLOT; a seq_len outside
 * [0, max_seq_len] or past its block table raises SV_DATA_BAD_PARAM and gives the request's rows
 * out = 0, lse = -infinity; a bad cu range raises SV_DATA_BAD_CU and leaves
 * the rows unwritten.  A NaN score makes its row NaN; nothing of a key that a
 * row does not see reaches it, whatever its scales are (in an e4m3 cache its
 * bytes are numbers, as spec_verify_kv_write leaves them; behind seq_len they
 * may be anything).  Scales may be any floats: a value scale of 0 or below is
 * taken as it stands, one of less than 2^-64, the writer's smallest, as 0, and
 * one that is NaN or infinite makes out NaN, not lse, in the rows that see its
 * key (for the heads that read it).  A key whose value scale is less than
 * 2^-100 of the largest that a row sees may drop out of the row's lse.
 * A key scale times `scale` may be 2^96 in size; with a larger one a row of q
 * below 2^-1 may become NaN though its scores are numbers.
 * SV_DATA_COPY_TIMEOUT: a wait inside a kernel ran out and out and lse are NaN
 * in the rows it was for; never expected on a healthy GPU.
 *
 * The products take 16-bit operands (f16).  The cache's numbers are exact in
 * them.  So is q, times a power of two of its row's own, but for elements below
 * 2^-13 of the row's largest, which may be off by 2^-24 of it.  The softmax's weights
 * are rounded to 11 bits, in steps of 2^-24 of the largest product of a weight
 * and its value's scale.  Exponentials are the GPU's fast ones (relative error
 * 2^-22).  Scores, sums and outputs are fp32 until out is rounded to bf16. */
typedef struct spec_verify_attend_args {
  int32_t num_reqs;     /* N >= 0 (0 is a no-op) */
  int32_t max_spec_len; /* G: every gamma_i <= G */
  int32_t num_q_heads;  /* a multiple of num_kv_heads */
  int32_t max_seq_len;  /* 0 .. 2^30; bounds every seq_len, as block_table_stride * block_size does */
  int32_t shared_prefix_len; /* 0 .. either bound, a multiple of block_size */
  uint32_t reserved;         /* 0 */
  int64_t num_draft_tokens_total; /* T = cu[N-1]; must equal N*G when cu == NULL */
  const int32_t *cu_num_draft_tokens; /* [N] inclusive prefix sums, or NULL: every gamma_i = G */
  spec_verify_kv_cache cache;
  const void *q; /* [T+N, num_q_heads, head_dim] bf16, any element strides, unit stride within a head */
  int64_t q_token_stride, q_head_stride;
  const int32_t *block_tables; /* [N, block_table_stride] */
  int64_t block_table_stride;
  const int32_t *seq_lens; /* [N] */
  float scale;             /* finite */
  uint32_t test_flags;     /* 0, or SV_TEST_EXPIRE_PRODUCT_WAIT (tests only) */
  void *out; /* [T+N, num_q_heads, head_dim] bf16 */
  int64_t out_token_stride, out_head_stride;
  float *lse;      /* [T+N, num_q_heads] contiguous, or NULL */
  void *workspace; /* 16-byte aligned device scratch of spec_verify_attend_workspace_size bytes (0 for many calls
                      without a shared prefix); contents need no initialisation and mean nothing after the call.
                      Calls that may run at the same time need one each. */
  int64_t workspace_bytes;
  int32_t *status; /* [1] or NULL: SV_DATA_* bits OR-ed in */
} spec_verify_attend_args;

sv_status spec_verify_attend(spec_verify_t handle, const spec_verify_attend_args *args, void *stream);

/* Bytes of workspace that calls of these sizes need, and such with fewer draft
 * tokens or a smaller max_seq_len (pointers are not looked at:
 * num_reqs, max_spec_len, num_q_heads, max_seq_len, shared_prefix_len,
 * num_draft_tokens_total, cache.num_kv_heads and cache.head_dim are). */
sv_status spec_verify_attend_workspace_size(spec_verify_t handle, const spec_verify_attend_args *args, int64_t *bytes);

/* Host-only validation of attention arguments against `config` (the workspace's size aside). */
sv_status spec_verify_check_attend_args(const spec_verify_config *config, const spec_verify_attend_args *args);

/* ---------------------------------------------------------------------------
 * The same cache in 4 bits, and attention over it.
 *
 * Every 16 elements of a row share an e4m3 scale, and the row has a float scale
 * besides: nibble x of group j stands for x * group_j * scale.  The nibbles are
 * E2M1 numbers (a sign, 0, 0.5, 1, 1.5, 2, 3, 4 or 6) or signed whole numbers
 * (-8 .. 7, of which the writer gives -7 .. 7).  Element 2i is the low half of
 * byte i, element 2i + 1 the high one.  The K (V) row of token offset t of page
 * b and kv head h is head_dim / 2 bytes at k (v) + b * block_stride +
 * h * head_stride + t * token_stride, its head_dim / 16 group scales are at
 * k_group (v_group) + b * group_block_stride + ..., and its scale as in the
 * 8-bit cache.  A row of head_dim 128 takes 76 bytes, against 132.
 *
 * Quantising a row x, all in fp32 with IEEE divisions: scale = max(max_d |x_d| /
 * (448 Q), 2^-64) with Q = 6 (E2M1) or 7 (whole numbers); group_j =
 * max_(d in j) |x_d| / (Q * scale) rounded to e4m3; nibble = x_d / (group_j *
 * scale) rounded to the nearest number of the format (ties to the even code,
 * at most Q in size), 0 where group_j is 0.  A row that holds a NaN or an
 * infinity gets scale NaN and zero bytes (it reads back as NaN) and raises
 * SV_DATA_BAD_VALUES.
 */
enum sv_cache4_format { SV_CACHE_E2M1 = 16, SV_CACHE_INT4 = 17 };

typedef struct spec_verify_kv4_cache {
  void *k, *v;              /* rows on 32-byte boundaries; strides in bytes, multiples of 32 */
  void *k_group, *v_group;  /* rows on boundaries of head_dim / 16 bytes; strides in bytes, multiples of that */
  float *k_scale, *v_scale; /* strides in elements */
  int64_t num_blocks;       /* >= 1; num_blocks * block_size <= 2^31 - 1 pages' tokens */
  int32_t block_size;       /* >= 1 (any: a power of two is not needed) */
  int32_t num_kv_heads;     /* >= 1 */
  int32_t head_dim;         /* 64 or 128 */
  int32_t format;           /* SV_CACHE_E2M1 or SV_CACHE_INT4 */
  int64_t block_stride, head_stride, token_stride;
  int64_t group_block_stride, group_head_stride, group_token_stride;
  int64_t scale_block_stride, scale_head_stride, scale_token_stride;
} spec_verify_kv4_cache;

/* As spec_verify_kv_args.  (A scale or group stride of 0 along more than one
 * element: such rows can be read, not written.  Where two tokens are written to
 * one slot, each part of the row is of either.) */
typedef struct spec_verify_kv4_args {
  int64_t num_tokens; /* T >= 0 (0 is a no-op) */
  int32_t dtype;      /* SV_F32 or SV_BF16: the elements of key and value */
  uint32_t reserved;  /* 0 */
  spec_verify_kv4_cache cache;
  void *key; /* read by spec_verify_kv4_write, written by spec_verify_kv4_read */
  int64_t key_token_stride, key_head_stride;
  void *value;
  int64_t value_token_stride, value_head_stride;
  const int64_t *slot_mapping; /* [T] */
  int32_t *status;             /* [1] or NULL: SV_DATA_* bits OR-ed in */
} spec_verify_kv4_args;

sv_status spec_verify_kv4_write(spec_verify_t handle, const spec_verify_kv4_args *args, void *stream);
sv_status spec_verify_kv4_read(spec_verify_t handle, const spec_verify_kv4_args *args, void *stream);

/* Host-only validation of the arguments of either call against `config`. */
sv_status spec_verify_check_kv4_args(const spec_verify_config *config, const spec_verify_kv4_args *args);

/* Attention of the verify tokens over the 4-bit cache: layout, masks, errors
 * and outputs are those of spec_verify_attend.  Group scales are numbers, as
 * spec_verify_kv4_write leaves them (those of keys at or behind seq_len may be
 * anything); the rows' scales may be any floats, as there.  Strides between
 * pages and between tokens are below 4 GB.  A nibble times its
 * group scale is exact in the 16-bit products' operands, so what that call
 * rounds to fewer bits is what this one does.  SV_TEST_EXPIRE_PRODUCT_WAIT makes
 * the private keys' first wait for a product give up too. */
typedef struct spec_verify_attend4_args {
  int32_t num_reqs;
  int32_t max_spec_len;
  int32_t num_q_heads;
  int32_t max_seq_len;
  int32_t shared_prefix_len;
  uint32_t reserved; /* 0 */
  int64_t num_draft_tokens_total;
  const int32_t *cu_num_draft_tokens;
  spec_verify_kv4_cache cache;
  const void *q;
  int64_t q_token_stride, q_head_stride;
  const int32_t *block_tables;
  int64_t block_table_stride;
  const int32_t *seq_lens;
  float scale;
  uint32_t test_flags; /* 0, or SV_TEST_EXPIRE_PRODUCT_WAIT (tests only) */
  void *out;
  int64_t out_token_stride, out_head_stride;
  float *lse;
  void *workspace; /* of spec_verify_attend4_workspace_size bytes */
  int64_t workspace_bytes;
  int32_t *status;
} spec_verify_attend4_args;

sv_status spec_verify_attend4(spec_verify_t handle, const spec_verify_attend4_args *args, void *stream);

/* As spec_verify_attend_workspace_size. */
sv_status spec_verify_attend4_workspace_size(spec_verify_t handle, const spec_verify_attend4_args *args,
                                             int64_t *bytes);

/* Host-only validation of attention arguments against `config` (the workspace's size aside). */
sv_status spec_verify_check_attend4_args(const spec_verify_config *config, const spec_verify_attend4_args *args);

/* ---------------------------------------------------------------------------
 * Block tables and slot maps from request lengths.
 *
 * Request i has n = num_new_tokens[i] tokens for this step behind the
 * p = num_computed_tokens[i] whose keys are in the cache; its rows follow those
 * of request i - 1 (for n = gamma_i + 1 this is the verify tokens' layout of the
 * other calls).  It needs ceil((p + n) / block_size) pages.  Those it holds are
 * entries 0 .. held_pages[i] - 1 of its block table (they must hold its computed
 * tokens; pages that a rejection left over stay with it), and missing ones
 * come from the free pages, a ring: with free_range = (head, tail) they are
 * free_pages[x % free_capacity] for x = head .. tail - 1.  Requests take pages
 * from the head in their order; where the pages wanted by the requests up to i
 * are more than there are, request i takes none and raises SV_DATA_NO_PAGES.
 * p < 0: the request is done (or the place is idle).  The pages it held go to the
 * tail, in order, free from the next call on, and its rows are idle.  The first
 * num_shared_pages entries of every table (a prefix that the batch shares) are
 * nobody's own: they stay, and count as held.  Any other page is in one table.
 *   seq_lens = p + n, positions = p .. p + n - 1 and slot_mapping their slots.
 * Idle rows -- of requests that are done or got no pages, and behind the last
 * request's -- have position and slot -1, and their requests seq_lens 0.
 * n < 0 (taken as 0), held_pages outside [0, table_width] or, with p >= 0, too
 * few for p or fewer than num_shared_pages, or a length that needs more than
 * table_width pages (or passes 2^31 - 1) raise SV_DATA_BAD_PARAM, and rows that
 * pass num_rows SV_DATA_BAD_CU; such a request is treated as one that got no
 * pages and does not count among those wanted.
 * With a free_range that is negative or wider than free_capacity, no page is
 * given or taken back (SV_DATA_BAD_PARAM).  Where the pages that the requests up
 * to i give back are more than the places of free_pages that are not free pages
 * already (books that are wrong, or a ring too small), request i's stay with it
 * (SV_DATA_BAD_PARAM): no free page is overwritten.
 * held_pages_out may be held_pages, free_range_out free_range and seq_lens
 * num_computed_tokens.  Nothing depends on the order in which threads run. */
typedef struct spec_verify_plan_args {
  int32_t num_reqs;    /* N >= 0 (0: only idle rows); at most the handle's max_num_reqs */
  int32_t block_size;  /* >= 1 */
  int32_t table_width; /* pages in a row of block_tables, >= 0 */
  int32_t num_shared_pages; /* 0 .. table_width */
  int64_t num_rows;    /* R: 0 .. 2^31 - 1 - 65536 */
  const int32_t *num_new_tokens;      /* [N] */
  const int32_t *num_computed_tokens; /* [N] */
  int32_t *block_tables;              /* [N, block_table_stride] in/out */
  int64_t block_table_stride;         /* >= table_width */
  const int32_t *held_pages;          /* [N] */
  int32_t *held_pages_out;            /* [N] */
  int32_t *free_pages;                /* [free_capacity] in/out */
  int64_t free_capacity;              /* 1 .. 2^31 - 1: no fewer than there are pages */
  const int64_t *free_range;          /* [2]: head, tail */
  int64_t *free_range_out;            /* [2] */
  int32_t *positions;                 /* [R] out */
  int64_t *slot_mapping;              /* [R] out */
  int32_t *seq_lens;                  /* [N] out */
  int32_t *cu_num_draft_tokens;       /* [N] out or NULL: prefix sums of n - 1 (2^31 - 1 at most), for calls on
                                         batches without n = 0 */
  void *workspace; /* 16-byte aligned device scratch of spec_verify_plan_workspace_size bytes; contents need no
                      initialisation.  Calls that may run at the same time need one each. */
  int64_t workspace_bytes;
  int32_t *status; /* [1] or NULL: SV_DATA_* bits OR-ed in */
} spec_verify_plan_args;

sv_status spec_verify_plan_step(spec_verify_t handle, const spec_verify_plan_args *args, void *stream);
sv_status spec_verify_plan_workspace_size(spec_verify_t handle, int32_t num_reqs, int64_t *bytes);

/* Host-only validation of the arguments against `config` (the workspace's size aside). */
sv_status spec_verify_check_plan_args(const spec_verify_config *config, const spec_verify_plan_args *args);

/* ---------------------------------------------------------------------------
 * Rotary positions of queries and keys, with a norm of each head before it.
 *
 * With a weight w, a head's row x becomes x / sqrt(mean x^2 + eps) * w first.
 * Pair i < rotary_dim / 2 of its elements (a, b) then becomes
 * magnitude * (a cos t - b sin t, b cos t + a sin t), t = position * f_i, and
 * elements from rotary_dim on stay as they are.  The pair is (i, i + rotary_dim
 * / 2), or (2i, 2i + 1) with SV_ROTATE_INTERLEAVED.  Frequencies are given as
 * turns[i] = f_i / (2 pi) * 2^64, rounded: the product with a position, modulo
 * 2^64, is the angle as a fraction of a turn, exact however far the position is.
 * Scalings for long contexts are a matter of these numbers and of `magnitude`.
 * The arithmetic is fp32, rounded once at the end.  (With a norm, a row whose sum
 * of squares passes the range of fp32 becomes zeros, and NaN where an element or
 * its pair's other one is not finite.)  Rows of a negative position
 * (idle ones) are neither read nor written.  Outputs may be the inputs
 * themselves (same strides); other overlaps are not allowed. */
#define SV_ROTATE_INTERLEAVED 1u
#define SV_MAX_ROTATE_HEAD_DIM 512
typedef struct spec_verify_rotate_args {
  int64_t num_tokens;  /* T >= 0 (0 is a no-op) */
  int32_t dtype;       /* SV_F32 or SV_BF16: the elements of every row and of the weights */
  int32_t head_dim;    /* 1 .. SV_MAX_ROTATE_HEAD_DIM */
  int32_t rotary_dim;  /* even, 0 .. head_dim */
  int32_t num_q_heads; /* >= 0; q is not looked at when 0 */
  int32_t num_k_heads; /* >= 0; key is not looked at when 0 */
  uint32_t flags;      /* 0 or SV_ROTATE_INTERLEAVED */
  const void *q;       /* [T, num_q_heads, head_dim], strides in elements, unit stride within a head */
  int64_t q_token_stride, q_head_stride;
  void *q_out;
  int64_t q_out_token_stride, q_out_head_stride;
  const void *key; /* [T, num_k_heads, head_dim] */
  int64_t key_token_stride, key_head_stride;
  void *key_out;
  int64_t key_out_token_stride, key_out_head_stride;
  const int32_t *positions;     /* [T] */
  const uint64_t *turns;        /* [rotary_dim / 2] */
  const void *q_weight;         /* [head_dim] or NULL: no norm */
  const void *key_weight;       /* [head_dim] or NULL */
  float magnitude;              /* finite */
  float eps;                    /* >= 0, finite */
} spec_verify_rotate_args;

sv_status spec_verify_rotate(spec_verify_t handle, const spec_verify_rotate_args *args, void *stream);

/* Host-only validation of the arguments against `config`. */
sv_status spec_verify_check_rotate_args(const spec_verify_config *config, const spec_verify_rotate_args *args);

/* Log-probabilities of the committed tokens, as a server returns them with the
 * text.  Logits rows and out_tokens are those of spec_verify_run: token
 * out_tokens[i, m] belongs to logits row s_i + i + m.  Entries of -1 (past the
 * commit) are skipped: their rows are not read, and they give 0 in the float
 * outputs and -1 in ranks and top_ids.  For the others, with x = the row
 * divided by the request's temperature (0 counts as 1: a greedy request has
 * the untempered distribution):
 *   logprobs = x[token] - ln sum exp x;  ranks = 1 + #{logits > logit[token]};
 *   entropy = -sum p ln p;  top_ids / top_logprobs = the num_top largest
 *   logits, the lowest index first among equal ones.
 * To score given tokens, pass max_spec_len = 0 and one token per row.  A -inf
 * logit has probability 0.  A row with a NaN, a +inf or no finite logit raises
 * SV_DATA_BAD_VALUES and gives NaN, ranks and top_ids -1; so do a temperature
 * that is negative, subnormal or not finite (SV_DATA_BAD_PARAM) and a token
 * outside [0, V) (SV_DATA_BAD_DRAFT_ID); a bad cu range (SV_DATA_BAD_CU)
 * gives the request's outputs as for -1. */
#define SV_MAX_TOP_LOGPROBS 32
typedef struct spec_verify_logprobs_args {
  int32_t num_reqs;     /* N >= 0 (0 is a no-op) */
  int32_t max_spec_len; /* G: out_tokens has G + 1 columns */
  int32_t vocab_size;   /* V >= 1 */
  int32_t dtype;        /* SV_F32 or SV_BF16 logits */
  int32_t num_top;      /* K: 0 .. min(V, SV_MAX_TOP_LOGPROBS) */
  uint32_t reserved;    /* 0 */
  int64_t num_draft_tokens_total;     /* T = cu[N-1]; must equal N*G when cu == NULL */
  const int32_t *cu_num_draft_tokens; /* [N] inclusive prefix sums, or NULL: every gamma_i = G */
  const void *logits;                 /* [T+N rows, row_stride], any alignment of the rows */
  int64_t row_stride;                 /* elements between rows (>= V) */
  const float *temperature;           /* [N] or NULL (= 1) */
  const int32_t *out_tokens;          /* [N, G+1] */
  float *logprobs;                    /* [N, G+1] out */
  int32_t *ranks;                     /* [N, G+1] out or NULL */
  float *entropy;                     /* [N, G+1] out or NULL */
  int32_t *top_ids;                   /* [N, G+1, K] out (NULL only when K = 0) */
  float *top_logprobs;                /* [N, G+1, K] out (NULL only when K = 0) */
  int32_t *status;                    /* [1] or NULL: SV_DATA_* bits OR-ed in */
} spec_verify_logprobs_args;

sv_status spec_verify_logprobs(spec_verify_t handle, const spec_verify_logprobs_args *args, void *stream);

/* Host-only validation of log-probability arguments against `config`. */
sv_status spec_verify_check_logprobs_args(const spec_verify_config *config, const spec_verify_logprobs_args *args);

/* Create a handle.  Queries the device and sets kernel attributes on it
 * (temporarily making `device` current).  *out is set only on SV_OK. */
sv_status spec_verify_create(const spec_verify_config *config, spec_verify_t *out);

/* Enqueue one verification on `stream` (a cudaStream_t, NULL = legacy default
 * stream of the current device, which must be the handle's device). */
sv_status spec_verify_run(spec_verify_t handle, const spec_verify_args *args, void *stream);

/* Release a handle (no device memory is held).  NULL is accepted. */
sv_status spec_verify_destroy(spec_verify_t handle);

/* Host-only validation of `args` against `config`: the checks spec_verify_run
 * performs before enqueueing anything.  Touches no device and no pointer target. */
sv_status spec_verify_check_args(const spec_verify_config *config, const spec_verify_args *args);

/* Static name of a status code. */
const char *spec_verify_status_string(sv_status status);

/* Message of the last error raised on the calling thread ("" if none). */
const char *spec_verify_last_error(void);

/* ABI self-description, for bindings that mirror the structs. */
uint32_t spec_verify_abi_version(void);
size_t spec_verify_sizeof_config(void);
size_t spec_verify_sizeof_args(void);
size_t spec_verify_sizeof_sample_args(void);
size_t spec_verify_sizeof_ngram_args(void);
size_t spec_verify_sizeof_kv_args(void);
size_t spec_verify_sizeof_attend_args(void);
size_t spec_verify_sizeof_logprobs_args(void);
size_t spec_verify_sizeof_kv4_args(void);
size_t spec_verify_sizeof_attend4_args(void);
size_t spec_verify_sizeof_plan_args(void);
size_t spec_verify_sizeof_rotate_args(void);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_VERIFY_H_ */
