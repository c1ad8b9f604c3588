/*
 * paged_attn.h -- C ABI of the GB300 (sm_103a) paged-KV attention library.
 *
 * The operation is attention read through a block-paged KV cache, as the
 * inference-server pages describe it:
 *   - "Block-paged KV cache with refcounted blocks, window-aware sliding
 *     layers" and "Triton paged decode and prefill kernels reading K/V
 *     through block tables; split-K decode variant" (inference-server README,
 *     engine feature list);
 *   - "Block-paged per-layer KV with refcounted blocks, lazy allocation, and
 *     SDPA gather -- vLLM/PagedAttention layout" (github README, "What's
 *     inside", Paged KV cache row);
 *   - "GQA with QK/V-norm + KV sharing ... softcapping" (github README,
 *     "What's inside", Custom Gemma 4 forward row);
 *   - mixed-batch chunked prefill, "Needs custom attention path" (architecture
 *     page, "Phase status" table).
 *
 * Definitions shared by every entry point
 * ---------------------------------------
 *  B       requests; Hq / Hkv query / KV heads, G = Hq / Hkv in {1,2,4,8};
 *  D       head_dim in {128, 256}; bs = block_size = 16.
 *  KV pool bf16 [num_blocks][Hkv][bs][D] for K and for V (one pool per layer;
 *          "KV sharing" between layers is the same pool passed twice).  Each
 *          (block, head) tile is one contiguous bs*D*2-byte run.
 *  block_tables  int32 [B][max_blocks], device.  Token t of request b is in
 *          block block_tables[b][t / bs], slot t % bs.  Entries at
 *          j >= ceil(seq_len/bs), and entries of blocks that lie wholly
 *          before every query's sliding window, are never dereferenced (they
 *          may be -1 or point at freed blocks).  Shared prefix blocks are the
 *          same id in several rows; the library only reads them.
 *  seq_lens int32 [B], device: context length including the new tokens.
 *  Query i of request b (n_b new tokens) sits at position p = L_b - n_b + i
 *          and sees key t iff t <= p and (window <= 0 or t > p - window).
 *  Logit   s = scale * q.k; if softcap > 0, s = softcap * tanh(s / softcap).
 *  GQA     query head h reads KV head h / G.
 *  Output  softmax(s) . V over the visible keys, fp32 accumulation, stored
 *          bf16 (round to nearest even).  No visible key -> output 0.
 *
 * Ownership and threading: the caller owns every buffer (device memory unless
 * stated); the library allocates nothing, never synchronises, keeps no state
 * between calls except cached device attributes, and launches on the given
 * stream (a cudaStream_t passed as void*; NULL = legacy default stream).
 * Calls are asynchronous and may be captured in CUDA graphs.
 *
 * Errors: every entry point returns a pka_status.  Argument errors are found
 * on the host before any launch (nothing is written).  PKA_ERR_CUDA means a
 * launch failed; read cudaGetLastError() for the cause.  Kernels never fault
 * on a bad table entry: an id outside [0, num_blocks) is replaced by block 0
 * and bit PKA_DEVERR_BAD_TABLE is OR-ed into *params->err (when non-NULL);
 * a bounded wait that runs out sets PKA_DEVERR_TIMEOUT and the CTA returns.
 */
#ifndef PAGED_ATTN_H_
#define PAGED_ATTN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  PKA_OK = 0,
  PKA_ERR_NULL = -1,        /* a required pointer is NULL */
  PKA_ERR_SHAPE = -2,       /* inconsistent sizes (Hq % Hkv, negative sizes, ...) */
  PKA_ERR_ALIGN = -3,       /* q/out/pool pointer not 16-byte aligned */
  PKA_ERR_UNSUPPORTED = -4, /* head_dim, block_size or G outside the supported set */
  PKA_ERR_WORKSPACE = -5,   /* workspace too small (partials, slots or counters) */
  PKA_ERR_BAD_TABLE = -6,   /* (host view of PKA_DEVERR_BAD_TABLE) */
  PKA_ERR_TIMEOUT = -7,     /* (host view of PKA_DEVERR_TIMEOUT) */
  PKA_ERR_CUDA = -8         /* a CUDA runtime call or launch failed */
} pka_status;

/* Bits OR-ed into the optional device error word (pka_attn_params.err). */
#define PKA_DEVERR_BAD_TABLE 1  /* a table id was outside [0, num_blocks) */
#define PKA_DEVERR_TIMEOUT 2    /* a bounded mbarrier wait ran out */
#define PKA_DEVERR_SEQ_LEN 4    /* seq_len beyond max_blocks*bs or the split cover */
#define PKA_DEVERR_QUERY_LOC 8  /* query_start_loc span outside [0, total_q], negative,
                                   or longer than max_query_len (request skipped) */
#define PKA_DEVERR_REFCOUNT 16  /* a block's reference count fell below zero */
#define PKA_DEVERR_TREE 32      /* a drafted token's parent is not a token before it */

/* One layer's K/V block pool.  k and v are device pointers, 16-byte aligned,
 * bf16 [num_blocks][num_kv_heads][block_size][head_dim]. */
typedef struct {
  const void* k;
  const void* v;
  int32_t num_blocks;
  int32_t num_kv_heads;
  int32_t block_size;
  int32_t head_dim;
} pka_kv_pool;

/* Attention parameters.  scale multiplies q.k and may be any finite value
 * (zero or negative included; NaN or infinite: PKA_ERR_SHAPE); softcap <= 0
 * or above 1e38 (+infinity too) disables the tanh cap (NaN: PKA_ERR_SHAPE);
 * window <= 0 is full (causal) attention, else the W-key sliding window
 * described above.  NaN in a visible key or in a query reaches the outputs that
 * see it, capped or not.  So does NaN in a value; over bf16 pools it also reaches
 * outputs that do not see it but multiply it by a weight of 0: rows of the same
 * prefill tile, and queries whose window starts later in the same block.
 * err: optional device int32 the kernels OR error bits into (never cleared by
 * the library). */
typedef struct {
  float scale;
  float softcap;
  int32_t window;
  int32_t* err;
} pka_attn_params;

/* Library version (major*10000 + minor*100 + patch). */
int pka_version(void);

/* Human-readable name of a pka_status (static string). */
const char* pka_status_string(int status);

/* Decode: one query token per request (engine feature list, "Triton paged
 * decode ... kernels reading K/V through block tables").
 * q   bf16 [B][Hq][D], out bf16 [B][Hq][D] (device, 16-byte aligned).
 * One CTA per (request, KV head) streams that request's visible blocks; use
 * the split-K entry points below when B*Hkv is small next to the SM count. */
int paged_decode_attn(const void* q, void* out, const pka_kv_pool* kv,
                      const int32_t* block_tables, int32_t max_blocks,
                      const int32_t* seq_lens, int32_t B, int32_t Hq,
                      int32_t max_seq_len, const pka_attn_params* params,
                      void* stream);

/* Split-K plan (host only, makes no CUDA call): the workspace shape of a
 * split-K launch for requests of at most max_seq_len tokens.
 *   split_blocks (C): the smallest chunk of 16-key tiles one CTA streams;
 *   num_splits (S):   partial slots per (request, query head),
 *                     ceil(T / C) + 1 for T = most visible blocks of a query.
 * sm_count is accepted for compatibility and not needed: the partition
 * adapts to the GPU it runs on. */
int paged_decode_splitk_plan(int32_t B, int32_t Hkv, int32_t max_seq_len,
                             int32_t block_size, int32_t window, int32_t sm_count,
                             int32_t* num_splits, int32_t* split_blocks);

/* Bytes of fp32 partials a split-K launch writes: B*Hq*S*(D+1)*4. */
size_t paged_decode_splitk_workspace_bytes(int32_t B, int32_t Hq, int32_t D,
                                           int32_t num_splits);

/* Split-K decode ("split-K decode variant", engine feature list).
 * Work partition: a segment is one (request, KV head) with n_b visible
 * blocks ("tiles", blocks [jlo_b, jlo_b + n_b), jlo_b = block of the first
 * visible key).  Segments are laid end to end in (request, head) order on a
 * line of work units: a segment with n_b > 0 takes P = 4 units (the fixed
 * cost of one partial) followed by one unit per tile, an empty segment none.
 * The T units of the line are cut into chunks of q = max(C, ceil(T / grid))
 * units, grid = twice the GPU's SM count, and chunk c is streamed by CTA c.
 * The tiles of a segment whose first tile sits at unit A that fall in chunk
 * c form its piece c - floor(A / q), written to that slot: the piece's
 * softmax-normalised partial output partial_o fp32 [B][Hq][S][D] and its
 * natural-log LSE partial_lse fp32 [B][Hq][S].  Slots a segment does not use
 * get LSE -inf (their partial_o is left untouched).  Needs
 * S >= ceil(T_max / C) + 1 for T_max the visible blocks of max_seq_len (else
 * PKA_ERR_WORKSPACE).  The line's arithmetic is 32-bit: PKA_ERR_SHAPE if
 * B * Hkv * (visible blocks of a table row + 4) exceeds 2^30. */
int paged_decode_splitk(const void* q, float* partial_o, float* partial_lse,
                        const pka_kv_pool* kv, const int32_t* block_tables,
                        int32_t max_blocks, const int32_t* seq_lens, int32_t B,
                        int32_t Hq, int32_t max_seq_len, int32_t num_splits,
                        int32_t split_blocks, const pka_attn_params* params,
                        void* stream);

/* Split-K decode with the log-sum-exp combine fused into the same launch
 * (one launch instead of two).  Same partition and partials as
 * paged_decode_splitk with the plan's (S, C); the CTA that finishes a
 * segment's last piece merges its pieces and writes out bf16 [B][Hq][D].
 * Exception: when the B * Hkv segments (request, KV head) number at most
 * the decode pipelines (twice the GPU's SM count) and none has more than
 * q + 24 units on the split's line (q its chunk), every segment streams
 * whole on its own pipeline and writes its output with no partials and no
 * merge -- the result of paged_decode_attn, bit for bit.
 * workspace: device, 16-byte aligned, at least paged_decode_attn_ws_bytes()
 * bytes: partial outputs fp32 [B][Hq][S][D], partial LSEs [B][Hq][S] (padded
 * to 16 bytes), then B*Hkv int32 arrival counters.  The counters must be
 * zero before the first call (e.g. memset once at allocation); every call
 * that completes leaves them zero again.  After a call that reported
 * PKA_DEVERR_TIMEOUT, zero them before the next call.  Calls sharing one
 * workspace must not overlap on the GPU.  PKA_ERR_SHAPE if
 * B * Hkv * (visible blocks of a table row + 4) exceeds 2^30. */
size_t paged_decode_attn_ws_bytes(int32_t B, int32_t Hq, int32_t Hkv, int32_t D,
                                  int32_t max_seq_len, int32_t window);
int paged_decode_attn_ws(const void* q, void* out, const pka_kv_pool* kv,
                         const int32_t* block_tables, int32_t max_blocks,
                         const int32_t* seq_lens, int32_t B, int32_t Hq,
                         int32_t max_seq_len, const pka_attn_params* params,
                         void* workspace, size_t workspace_bytes, void* stream);

/* Log-sum-exp merge of split partials (the merge a split-K softmax needs):
 * M = max_s LSE_s, w_s = exp(LSE_s - M),
 * out = sum_s w_s*O_s / sum_s w_s (bf16 [B][Hq][D]),
 * lse_out = M + ln sum_s w_s (fp32 [B][Hq], may be NULL).
 * Slots with LSE -inf are skipped without reading their partial_o. */
int paged_decode_splitk_combine(const float* partial_o, const float* partial_lse,
                                int32_t B, int32_t Hq, int32_t D, int32_t num_splits,
                                void* out, float* lse_out, void* stream);

/* Prefill / mixed batch ("Prefill in three modes: monolithic, chunked ...,
 * batched", engine feature list; mixed-batch chunked prefill, architecture
 * page "Phase status").  Varlen: request b owns query rows
 * [query_start_loc[b], query_start_loc[b+1]) of q bf16 [total_q][Hq][D]; rows
 * with one token (decode) and chunks of many tokens may be mixed in one
 * launch.  Causal over cached prefix + chunk.  out bf16 [total_q][Hq][D].
 * max_query_len / max_seq_len are host upper bounds.  query_start_loc is
 * device data: a request whose span is not 0 <= query_start_loc[b] <=
 * query_start_loc[b+1] <= total_q, or is longer than max_query_len, is
 * skipped (its rows are not written) and PKA_DEVERR_QUERY_LOC is OR-ed into
 * the error word; nothing outside out's total_q rows is ever written. */
int paged_prefill_attn(const void* q, void* out, const pka_kv_pool* kv,
                       const int32_t* block_tables, int32_t max_blocks,
                       const int32_t* query_start_loc, const int32_t* seq_lens,
                       int32_t B, int32_t Hq, int32_t total_q, int32_t max_query_len,
                       int32_t max_seq_len, const pka_attn_params* params,
                       void* stream);

/* Mixed batch in one launch with a workspace (mixed-batch chunked prefill,
 * architecture page "Phase status"): same arguments, result and errors as
 * paged_prefill_attn, but requests with exactly one query token (decode rows)
 * go to decode pipelines in the same launch -- split-K over their keys with
 * the log-sum-exp merge fused in, as paged_decode_attn_ws -- instead of
 * filling G of the 128 rows of a tensor-core tile; requests with more tokens
 * run the tensor-core prefill pipeline.  Exception: when the decode rows'
 * B * Hkv segments (request, KV head) number at most the decode pipelines
 * and none has more than q + 24 units on the split's line (q its chunk,
 * the paged_decode_splitk partition over the decode pipelines), every
 * segment streams whole on its own pipeline and writes its output with no
 * partials and no merge.
 * SMs: the prefill side gets P of the GPU's N SMs, the decode pipelines the
 * rest (two per SM).  P shares N in proportion to estimated SM time, from
 * sizes only: prefill E = ceil((total_q - B) / TQ) * Hkv items (TQ = 128/G
 * query tokens per tile) of ceil(K / BN) + 1 key tiles each at 2 us, with
 * K = min(max_seq_len, window + TQ) (max_seq_len without window) and BN = 64
 * at D = 256, 128 at D = 128; decode max(0, B - ceil((total_q - B) /
 * (max_query_len - 1))) rows of Hkv * ceil(K' / 16) blocks at 64 * D bytes
 * per block and 70 GB/s per SM, K' = min(max_seq_len, window).  With
 * share = round(N * prefill / (prefill + decode)), P = share if share >= 2E,
 * else E; then clamped to [1, N - N/4] (P = 0 without prefill rows).
 * Prefill items: one per (request, query tile, KV head) with work, on one
 * CTA each at D = 128; at D = 256 on CTA pairs, two query tiles per pair of
 * SMs, as in paged_prefill_attn (the decode CTAs then number N - P rounded
 * down to even, and the P SMs give S = P / 2 pair slots and 80 piece slots;
 * else S = P slots and 160 piece slots).  When the items are fewer than S
 * (and at most the piece slots; at D = 256 only when also the estimate
 * ceil((total_q - B) / (2 TQ)) * Hkv is below S and at most 80), they are
 * cut along their keys: with theta
 * the smallest piece length >= 4 key tiles for which sum over items of
 * min(8, ceil(tiles / theta)) <= min(S, piece slots), an item of T key
 * tiles runs as p = min(8, ceil(T / theta)) pieces on separate CTAs (CTA
 * pairs), piece k taking tiles [k T / p, (k + 1) T / p); each piece leaves
 * its normalised rows and their LSEs in the workspace (a CTA pair: each CTA
 * its 128 rows in a slot of its own) and the piece that arrives last on the
 * item's counter (at D = 256, each CTA's rows have their own) merges them
 * in piece order (the same result whichever piece merges).
 * workspace: device, 16-byte aligned, at least paged_prefill_attn_ws_bytes()
 * bytes: the layout of paged_decode_attn_ws for B requests, then 160 piece
 * slots of 128 fp32 rows of D columns, their 160 * 128 fp32 LSEs and 160
 * int32 piece counters (padded to 16 bytes).  All counters must be zero
 * before the first call and are left zero by every call that completes
 * (zero them again after a PKA_DEVERR_TIMEOUT).  Calls sharing one
 * workspace must not overlap on the GPU.  PKA_ERR_WORKSPACE if
 * workspace_bytes is too small. */
size_t paged_prefill_attn_ws_bytes(int32_t B, int32_t Hq, int32_t Hkv, int32_t D,
                                   int32_t max_seq_len, int32_t window);
int paged_prefill_attn_ws(const void* q, void* out, const pka_kv_pool* kv,
                          const int32_t* block_tables, int32_t max_blocks,
                          const int32_t* query_start_loc, const int32_t* seq_lens,
                          int32_t B, int32_t Hq, int32_t total_q, int32_t max_query_len,
                          int32_t max_seq_len, const pka_attn_params* params,
                          void* workspace, size_t workspace_bytes, void* stream);

/* Checked mode: validates, on the device, every table entry a call would
 * dereference (j < ceil(seq_len/bs)) against [0, num_blocks), and seq_len
 * against [0, max_blocks*bs]; OR-s PKA_DEVERR_* bits into *err (device int32,
 * required).  Reads only the tables and seq_lens. */
int paged_attn_check_tables(const int32_t* block_tables, int32_t max_blocks,
                            const int32_t* seq_lens, int32_t B, int32_t num_blocks,
                            int32_t block_size, int32_t* err, void* stream);

/* Self-test of the bounded waits.  Launches one CTA whose thread waits, with
 * the wait routine of every kernel in this library, on an mbarrier phase
 * that nothing completes, for budget_cycles SM clock cycles (1 ..
 * 2e9; the kernels' own budget is 2e9, about a second).  The wait runs out,
 * PKA_DEVERR_TIMEOUT is OR-ed into *err (device int32, required) and the
 * kernel returns: a stalled pipeline ends with an error status and a usable
 * context instead of a hang.  PKA_ERR_NULL / PKA_ERR_SHAPE on bad arguments. */
int pka_selftest_bounded_wait(int32_t* err, int64_t budget_cycles, void* stream);

/* H2O attention mass.  The engine's cache offers an H2O eviction policy
 * ("Eviction policies -- Pluggable per-session: LRU, AttentionSink, H2O",
 * github README, "What's inside"; "H2O wiring deferred", architecture page,
 * "Phase status"), which keeps the keys that have drawn the most attention.
 * Two calls give what it needs from a decode step:
 *
 * paged_decode_splitk_logits: paged_decode_splitk that also stores every
 *   visible key's logit: logits fp32 [B][Hq][max_blocks*16] (device, caller
 *   owned), entry [b][h][t] = log2(e) * s_h(t) (s after scale and softcap)
 *   for the keys t query head h of request b sees; other entries are not
 *   written.  Arguments and errors otherwise as paged_decode_splitk.
 * paged_decode_key_mass: after paged_decode_splitk_combine with lse_out
 *   (natural-log LSE [B][Hq]), adds each visible key's attention probability,
 *   summed over the G query heads of its KV head, to key_mass fp32
 *   [B][Hkv][max_blocks*16] (device): key_mass[b][kvh][t] += sum_h
 *   exp(s_h(t) - LSE_h).  Invisible keys are left as they are; a head with
 *   LSE = -inf adds nothing.  Over the visible keys of one (b, kvh) the
 *   added mass sums to G. */
int paged_decode_splitk_logits(const void* q, float* partial_o, float* partial_lse,
                               float* logits, const pka_kv_pool* kv,
                               const int32_t* block_tables, int32_t max_blocks,
                               const int32_t* seq_lens, int32_t B, int32_t Hq,
                               int32_t max_seq_len, int32_t num_splits, int32_t split_blocks,
                               const pka_attn_params* params, void* stream);
int paged_decode_key_mass(const float* logits, const float* lse, const int32_t* seq_lens,
                          int32_t B, int32_t Hq, int32_t num_kv_heads, int32_t max_blocks,
                          int32_t block_size, int32_t window, float* key_mass, void* stream);

/* Append the new tokens' K and V rows to a pool: the cache write that comes
 * before attention on every tick ("Block-paged per-layer KV with refcounted
 * blocks, lazy allocation, and SDPA gather -- vLLM/PagedAttention layout",
 * github README, "What's inside", Paged KV cache row; one new token per
 * active request per tick, architecture page, "How a single request flows
 * through the system", step 7).
 *   k_new, v_new  bf16 [T][Hkv][D], device, contiguous, 16-byte aligned.
 *   k_pool, v_pool  bf16 [num_blocks][Hkv][block_size][D], device, written.
 *   slot_mapping  int32 [T], device: token t goes to slot s = slot_mapping[t]
 *                 = block * block_size + offset, for every KV head; s < 0
 *                 skips the token (padding).  Slots must be distinct (with a
 *                 repeated slot, which token's row lands there is undefined).
 *   err           optional device int32: a slot beyond num_blocks *
 *                 block_size is skipped and ORs PKA_DEVERR_BAD_TABLE into it.
 * Bit-exact copy; T = 0 is a no-op.  D in {128, 256}, block_size 16. */
int paged_kv_append(const void* k_new, const void* v_new, void* k_pool, void* v_pool,
                    int32_t num_blocks, int32_t num_kv_heads, int32_t block_size,
                    int32_t head_dim, const int32_t* slot_mapping, int32_t T, int32_t* err,
                    void* stream);

/* paged_kv_append with the per-head math before attention fused in
 * ("Custom Gemma 4 forward -- Dual-RoPE, GQA with QK/V-norm + KV sharing",
 * github README, "What's inside").  For each token t (position positions[t],
 * slot slot_mapping[t] as in paged_kv_append), in this order:
 *   RMS norm   x <- x / sqrt(mean_c(x_c^2) + eps) * w_c over the D channels of
 *              each head: q with q_norm_weight, k with k_norm_weight (fp32 [D],
 *              device; NULL = no norm for that tensor), v with unit weight when
 *              v_norm != 0;
 *   RoPE       q and k, rotate-half form: with r = rotary_dim and
 *              a_i = positions[t] * rope_theta^(-2i/r), for i < r/2:
 *              (x_i, x_{i+r/2}) <- (x_i cos a_i - x_{i+r/2} sin a_i,
 *                                   x_{i+r/2} cos a_i + x_i sin a_i);
 *              channels >= r unchanged; rotary_dim = 0 turns it off (the two
 *              RoPE variants of a dual scheme are two calls).
 * Then k and v rows go to the pool slots and q (bf16 [T][Hq][D], may be NULL)
 * is overwritten in place; everything is computed in fp32 from the bf16
 * inputs and stored bf16 (round to nearest even).
 * rotary_dim in [0, D], a multiple of 16; rope_theta > 1 when rotary_dim > 0;
 * eps >= 0.  Errors as paged_kv_append. */
int paged_kv_append_rope(void* q, const void* k_new, const void* v_new, void* k_pool,
                         void* v_pool, int32_t num_blocks, int32_t num_q_heads,
                         int32_t num_kv_heads, int32_t block_size, int32_t head_dim,
                         const int32_t* slot_mapping, const int32_t* positions, int32_t T,
                         const float* q_norm_weight, const float* k_norm_weight, int32_t v_norm,
                         float eps, float rope_theta, int32_t rotary_dim, int32_t* err,
                         void* stream);

/* Decode for callers that cannot allocate device memory.  The pages have no
 * counterpart: this is a service of this library.  Some callers cannot call
 * cudaMalloc -- a plugin running while another allocator owns all device
 * memory, code in a region where allocation calls are not allowed -- yet
 * split-K decode needs room for its fp32 partials.  This entry point gives
 * the same result as paged_decode_splitk_plan + paged_decode_splitk +
 * paged_decode_splitk_combine, with the partials in a 16 MiB array compiled
 * into the library, so it allocates nothing; q, out and the pool are the
 * caller's, as for paged_decode_attn.
 * Limit: B*Hq*S*(D+1)*4 bytes <= 16 MiB for the S paged_decode_splitk_plan
 * gives; larger calls return PKA_ERR_WORKSPACE before launching anything.
 * The first call on each device looks up the array's device address (make
 * that first call before any stream capture) and keeps it for the life of
 * the process: after cudaDeviceReset the library's module is loaded again at
 * another address, so a process that resets a device must not call this
 * entry point on that device afterwards.  Every GPU that loads the
 * library holds the array until the process exits.  All calls share the one
 * array: calls that overlap on the GPU (other streams, other threads) race
 * and must be serialised by the caller. */
int paged_decode_attn_noalloc(const void* q, void* out, const pka_kv_pool* kv,
                              const int32_t* block_tables, int32_t max_blocks,
                              const int32_t* seq_lens, int32_t B, int32_t Hq,
                              int32_t max_seq_len, const pka_attn_params* params,
                              void* stream);

/* 4-bit cache.  The pages store the cache in bf16; these entry points keep it
 * in 4 bits (4.5 with the scales), so that the same memory holds 3.6 times the
 * tokens and a decode step reads 3.6 times fewer bytes.
 *
 * Format: a value is stored as e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign)
 * with one e4m3 scale for every 16 channels of a token and KV head, and one
 * fp32 scale per pool: value = pool scale * e4m3 * e2m1.
 *   k, v   device pointers, 16-byte aligned, uint8
 *          [num_blocks][num_kv_heads][head_dim / 128][1152]: units of 16
 *          tokens x 128 channels (paged_kv4_pool_bytes bytes for each of K and V).
 *          K unit: codes [16 tokens][64], channel 2i in the low nibble of
 *          byte i; then scales [16 tokens][8 groups].
 *          V unit: codes [8 groups][16 tokens][8], in the odd groups tokens
 *          8..15 before tokens 0..7; then scales [8 groups][16 tokens].
 *   k_scale, v_scale   > 0 and finite, 6 * scale finite.  A scale of max|x| / 2688
 *          over the values to be stored uses the whole range of the e4m3
 *          scales.
 * Quantisation of a group x of 16 channels, each operation rounded once to
 * fp32: r = max|x| / (6 * pool scale); s = e4m3(min(r, 448)); code =
 * e2m1(x / (s * pool scale)), both to the nearest, ties to even, saturating;
 * s = 0 gives zeros.  A group that holds an infinity or a NaN reads back as
 * NaN in all its 16 channels. */
typedef struct {
  void* k;
  void* v;
  int32_t num_blocks;
  int32_t num_kv_heads;
  int32_t block_size; /* 16 */
  int32_t head_dim;   /* 128 or 256 */
  float k_scale;
  float v_scale;
} pka_kv4_pool;

/* Bytes of one 4-bit pool (K or V): num_blocks * num_kv_heads * 9 * head_dim;
 * 0 for sizes that are not supported. */
size_t paged_kv4_pool_bytes(int32_t num_blocks, int32_t num_kv_heads, int32_t head_dim);

/* paged_kv_append into a 4-bit pool: token t's K and V rows are quantised and
 * written at slot_mapping[t] (< 0 skips the token; a slot past the pool is
 * skipped and ORs PKA_DEVERR_BAD_TABLE into *err; slots must be distinct).
 *   k_new, v_new  bf16 [T][Hkv][D], device, 16-byte aligned; consecutive
 *                 tokens k_stride / v_stride elements apart (at least Hkv * D,
 *                 a multiple of 8: rows may be slices of a wider projection).
 * Other slots of the blocks written are left as they are.  T = 0 is a no-op. */
int paged_kv4_append(const void* k_new, const void* v_new, int64_t k_stride, int64_t v_stride,
                     const pka_kv4_pool* kv, const int32_t* slot_mapping, int32_t T,
                     int32_t* err, void* stream);

/* Blocks of a 4-bit pool as bf16 (rounded to nearest even), for the entry
 * points that read bf16 pools: a prefill chunk over a 4-bit prefix expands its
 * requests' blocks and runs paged_prefill_attn on them.  For i < n, block
 * src_blocks[i] of kv is written to block dst_blocks[i] of dst (dst_blocks
 * NULL: to block i; n at most dst's num_blocks then).  A negative id skips the
 * item, so that rows of a padded block table can be passed as they are; an id
 * past its pool skips it and ORs PKA_DEVERR_BAD_TABLE into *err.  All 16
 * slots are written.  Destinations must be distinct.  The pools agree in KV
 * heads, block size and head_dim. */
int paged_kv4_expand(const pka_kv4_pool* kv, const pka_kv_pool* dst, const int32_t* src_blocks,
                     const int32_t* dst_blocks, int32_t n, int32_t* err, void* stream);

/* Decode over a 4-bit cache: paged_decode_attn_ws on the values the pool
 * holds (arithmetic on them in fp32, or in f16 where that is exact; softmax weights
 * rounded to f16; bf16 out).  Arguments, masks and errors as there; any group
 * of 1 to 8 query heads per KV head; B * Hkv and B * the most blocks a query
 * sees (max_blocks, fewer with a window) at most 2^30, else PKA_ERR_SHAPE.  A
 * table id outside the pool reads as zeros and ORs PKA_DEVERR_BAD_TABLE into
 * params->err.
 * One launch: short segments (request, KV head) stream whole; longer ones are
 * cut into pieces, at most 30 each, whose fp32 partials the last piece to
 * arrive merges in a fixed order (the same bits every time).  max_seq_len
 * sizes the pieces: a segment is cut into pieces of no less than 1/29 of it, so
 * a promise far above the lengths leaves long segments whole and SMs idle (32
 * requests of 512 to 4096 tokens, D = 256: 19.9 us with 4096 promised, 35.0 with
 * 131072); rows that are longer all the same are computed, more slowly.
 * A logit cap rounds the logit by at most 2^-18 of it, whatever the cap.  Logits
 * that are all -infinity give NaN (no visible key: 0).
 * workspace: at least paged_kv4_decode_attn_ws_bytes() bytes, 16-byte
 * aligned: 2048 bytes of arrival counters, then the partials.  The first 2048
 * bytes must be zero before the first call and are left zero by every call, so
 * calls of any sizes can use one workspace (of the largest size) in turn.
 * Calls sharing one workspace must not overlap on the GPU. */
size_t paged_kv4_decode_attn_ws_bytes(int32_t B, int32_t Hq, int32_t Hkv, int32_t D,
                                      int32_t max_seq_len, int32_t window);
int paged_kv4_decode_attn_ws(const void* q, void* out, const pka_kv4_pool* kv,
                             const int32_t* block_tables, int32_t max_blocks,
                             const int32_t* seq_lens, int32_t B, int32_t Hq,
                             int32_t max_seq_len, const pka_attn_params* params,
                             void* workspace, size_t workspace_bytes, void* stream);

/* Pages of a cache ("refcounted blocks, lazy allocation", github README,
 * "What's inside", Paged KV cache row; "repeated or shared-system prompts skip
 * prefill", prefix sharing row).  The reference counts, free lists and tables
 * are the engine's; these entry points do the device side of forking, freeing
 * and compacting.  A pool is any device array of num_blocks blocks of
 * block_bytes bytes (bf16: Hkv*16*D*2 each of K and V; 4-bit: Hkv*9*D).
 *
 * paged_kv_ref_blocks: adds delta to refcounts[id] for every block the B
 *   table rows use (entries j < ceil(seq_len / 16)): +1 when a request is
 *   forked, -1 when it ends.  Negative entries (no block, or one a sliding
 *   layer gave back) are skipped; an id past the pool ORs PKA_DEVERR_BAD_TABLE
 *   into *err, a count that falls below zero PKA_DEVERR_REFCOUNT.  A block that
 *   occurs in several entries counts for each.
 * paged_kv_copy_blocks: block src[i] -> block dst[i] for i < n in each of
 *   num_pools pools (pools: host array of device pointers, 16-byte aligned;
 *   block_bytes a multiple of 16), e.g. the last, partly filled block of a
 *   forked request in every layer.  The destinations must be distinct and
 *   none of them another pair's source (else those blocks' contents are
 *   undefined); src[i] = dst[i] does nothing.  A pair with an id outside the
 *   pool is skipped and ORs PKA_DEVERR_BAD_TABLE into *err.
 * paged_kv_compact: closes a pool up.  With n = the number of live blocks
 *   (refcount > 0), the j-th highest live id at or above n moves to the j-th
 *   lowest free id below n, in each of num_pools pools; afterwards the live
 *   blocks are 0 .. n - 1.  Outputs (device): remap[id] = new id (-1: free);
 *   new_refcounts[new id] (0 from n on; may be refcounts itself); new_tables
 *   = block_tables with the used entries (j < ceil(seq_len / 16)) remapped
 *   (a free block's becomes -1; unused and negative entries are kept; may be
 *   block_tables itself); moves int32 [2 + num_blocks]: [0] the number of
 *   moves, [1] = n, then (old id, new id) for each move, -1 after the last.
 *   A used entry past the pool is kept and ORs PKA_DEVERR_BAD_TABLE into *err.
 *   num_pools = 0 plans only; B = 0 leaves tables out.  Blocks from n on keep
 *   their old contents. */
int paged_kv_ref_blocks(const int32_t* block_tables, int32_t max_blocks, const int32_t* seq_lens,
                        int32_t B, int32_t num_blocks, int32_t delta, int32_t* refcounts,
                        int32_t* err, void* stream);
int paged_kv_copy_blocks(void* const* pools, int32_t num_pools, int32_t num_blocks,
                         int64_t block_bytes, const int32_t* src, const int32_t* dst, int32_t n,
                         int32_t* err, void* stream);
int paged_kv_compact(void* const* pools, int32_t num_pools, int32_t num_blocks,
                     int64_t block_bytes, const int32_t* refcounts, int32_t* new_refcounts,
                     const int32_t* block_tables, int32_t* new_tables, int32_t max_blocks,
                     const int32_t* seq_lens, int32_t B, int32_t* remap, int32_t* moves,
                     int32_t* err, void* stream);

/* Draft trees (speculative decoding).  The pages have no counterpart; these
 * entry points are services of this library beside its prefill, append and page
 * calls.  In a step each request brings n <= 64 drafted tokens that form a tree:
 * token 0 is its root (the last token the model chose, whose K/V are not cached
 * yet), token i > 0 follows token parents[i] < i.  The n tokens take the cache
 * positions L - n .. L - 1 in order (L = seq_lens[b], the drafted tokens
 * included), whatever their depth.  A step is: paged_tree_plan, then per layer
 * paged_kv_append[_rope] with the plan's slots and positions and
 * paged_tree_attn_ws with its masks, then paged_tree_accept.
 * Rows are those of paged_prefill_attn: request b owns rows
 * [query_start_loc[b], query_start_loc[b+1]) of the total_q rows.
 *
 * paged_tree_plan: for each token i of a tree
 *   tree_masks uint64 [total_q]: bit j is set iff token j is i or one of its
 *              ancestors;
 *   positions  int32 [total_q]: T - n + (the number of i's ancestors), for the
 *              rotary embedding; T = total_lens[b] (NULL: L), the length of the
 *              sequence where keys were evicted from its cache;
 *   slots      int32 [total_q]: the pool slot of cache position L - n + i.
 *   Each of the three may be NULL.  parents int32 [total_q]: a token before it in
 *   its tree, -1: none (more than one token may have none); another value ORs
 *   PKA_DEVERR_TREE into *err and counts as -1.  Rows from query_start_loc[B] on
 *   (padding) get mask 0, position 0, slot -1.  A request whose span is not as
 *   in paged_prefill_attn is left out (PKA_DEVERR_QUERY_LOC, its rows unwritten);
 *   one with n > L, n > T or L past its table row gets mask 0, position 0, slot -1
 *   (PKA_DEVERR_SEQ_LEN); a table id outside the pool gives slot -1
 *   (PKA_DEVERR_BAD_TABLE).  max_query_len > 64: PKA_ERR_UNSUPPORTED. */
int paged_tree_plan(const int32_t* parents, const int32_t* query_start_loc,
                    const int32_t* seq_lens, const int32_t* total_lens,
                    const int32_t* block_tables, int32_t max_blocks, int32_t num_blocks, int32_t B,
                    int32_t total_q, int32_t max_query_len, uint64_t* tree_masks,
                    int32_t* positions, int32_t* slots, int32_t* err, void* stream);

/* Attention of drafted tokens: as paged_prefill_attn (arguments, head mapping,
 * scale, cap, table and length errors), but query i of a request sees
 *   - key t < L - n iff window <= 0 or t > p_i - window, with the position
 *     p_i = L - n + max(d_i, 1) - 1, d_i the bits of its mask below n;
 *   - key L - n + j (j < n) iff bit j of tree_masks[row] is set and window <= 0
 *     or d_i - d_j < window.
 * The masks need not come from a tree.  No visible key: output 0; visible
 * logits that are all -infinity: NaN.  Infinities and NaN in K or V reach the
 * queries that see them, at a weight of 0 too, and no others.  Rows of no request
 * are not written.  Logits, maxima and sums are fp32; each weight is rounded
 * to bf16 for its product with V (by 2^-8 of it at most; the sum that divides
 * is of the unrounded ones), as in the other calls over bf16 pools.
 * Keys are cache positions: with a window the cache has to hold the sequence
 * unevicted.
 * One launch, or two: the segments (request, KV head, tile of 128 / G or 64 / G
 * query tokens) are streamed in equal chunks of their keys, one per SM, and what
 * a chunk cuts is merged in key order by the second launch.  Where max_seq_len
 * and the number of segments let none be cut there is no second launch; few of
 * them are shared by two CTAs each.  The same call gives the same bits every
 * time.  max_seq_len is a promise; longer rows are computed all the same, and the
 * nearest one finds the fastest of these forms.
 * The call gathers no key mass (paged_decode_key_mass does, after a plain decode
 * step): tokens that are accepted from trees have mass 0 until a decode step sees
 * them, and are the first that paged_kv_evict gives up once they are not recent.
 * workspace: 16-byte aligned, at least paged_tree_attn_ws_bytes() bytes (which
 * depend on no length and no batch), needs no initialisation.  Calls sharing one
 * workspace must not overlap on the GPU.
 * tree_masks 8-byte aligned.  max_query_len > 64: PKA_ERR_UNSUPPORTED.
 * PKA_ERR_SHAPE if the segments times (visible blocks of a table row + 20) exceed
 * 2^30, max_blocks exceeds 2^26, or num_blocks * Hkv * 16 exceeds 2^31 - 1. */
size_t paged_tree_attn_ws_bytes(int32_t Hq, int32_t Hkv, int32_t D, int32_t max_query_len);
int paged_tree_attn_ws(const void* q, void* out, const pka_kv_pool* kv,
                       const int32_t* block_tables, int32_t max_blocks,
                       const int32_t* query_start_loc, const uint64_t* tree_masks,
                       const int32_t* seq_lens, int32_t B, int32_t Hq, int32_t total_q,
                       int32_t max_query_len, int32_t max_seq_len, const pka_attn_params* params,
                       void* workspace, size_t workspace_bytes, void* stream);

/* Acceptance of drafted tokens.  Walk of each tree: from token 0, while a token
 * c (the lowest) has parents[c] = the current one and tokens[c] = targets[the
 * current one], go to c.  targets int32 [total_q] are the target model's next
 * tokens after each drafted one: its most probable tokens, or samples of its
 * distribution (which makes the accepted text a sample of it, too).
 *   path         int32 [B][max_query_len]: the walk's tokens (indexes within the
 *                tree, the first is 0), -1 after the last;
 *   accepted     int32 [B]: their number (n = 0: 0);
 *   next_tokens  int32 [B]: the target's token after the last one (n = 0: -1),
 *                root of the next step's tree;
 *   new_seq_lens int32 [B]: L - n + accepted (may be seq_lens itself).
 * In each of num_pools bf16 pools (host array; K and V of every layer) the K/V
 * rows of the walk's tokens move to the tree's first slots, so that the cache
 * goes on without a gap: the row at slots[path[k]] to slots[k], both of the
 * request's rows of `slots` (paged_tree_plan); pairs with a negative slot are
 * left out, a slot past the pool ORs PKA_DEVERR_BAD_TABLE into *err.  The slots
 * of all trees must be distinct, and so must the pools (layers that share one
 * name it once; PKA_ERR_SHAPE if two share memory).  num_pools = 0: the walk alone (slots and the
 * pools' sizes are not looked at).  A bad span leaves a request as if n = 0
 * (PKA_DEVERR_QUERY_LOC), and so does n > L (PKA_DEVERR_SEQ_LEN; rows move by the
 * slots alone, which paged_tree_plan makes negative for such a request).
 * num_kv_heads at most 1024. */
int paged_tree_accept(void* const* pools, int32_t num_pools, int32_t num_blocks,
                      int32_t num_kv_heads, int32_t block_size, int32_t head_dim,
                      const int32_t* parents, const int32_t* tokens, const int32_t* targets,
                      const int32_t* slots, const int32_t* query_start_loc,
                      const int32_t* seq_lens, int32_t B, int32_t total_q, int32_t max_query_len,
                      int32_t* path, int32_t* accepted, int32_t* next_tokens,
                      int32_t* new_seq_lens, int32_t* err, void* stream);

/* H2O eviction ("Eviction policies -- Pluggable per-session: LRU, AttentionSink,
 * H2O", github README, "What's inside"): holds the cache of each (layer,
 * request, KV head) to `budget` keys by the mass that paged_decode_key_mass
 * gathers.
 *   key_mass, key_pos  fp32 and int32 [num_layers][B][Hkv][max_blocks * 16]: a
 *            key's mass and its position in the sequence; position -1: a key
 *            appended since the last eviction (key t of L then has position
 *            T - L + t, T = total_lens[b], NULL: L; T >= L).  Before its first
 *            eviction a request's positions are all -1.
 * Of the L keys n = min(L, budget) stay: first the keys at positions below
 * `sinks` or from T - `recent` on, lowest index first, then the others by mass
 * (NaN below everything), ties to the lowest index.  Kept keys with an index of
 * n or more move, with mass and position, to the indexes below n that do not
 * stay: the highest of them to the lowest such index, and so on.  (Their order in
 * the cache does not matter to decode without a window.)  Then
 *   new_mass, new_pos  (may be key_mass, key_pos) hold the kept keys in [0, n)
 *            with their positions, 0 and -1 in [n, L), entries from L on as they
 *            were;
 *   new_seq_lens int32 [B] (may be seq_lens) = n;
 *   pools    (host array of 2 * num_layers distinct bf16 pools: K and V of each
 *            layer; layers that share one evict once; PKA_ERR_SHAPE if two pools
 *            share memory) hold the kept rows; rows from n on keep their contents,
 *            and their blocks can be given back (paged_kv_ref_blocks with the old
 *            lengths and -1, then with the new ones and +1).
 * refcounts (NULL: not looked at) int32 [num_blocks]: a request of whose blocks
 * below n one has a count above 1 is left whole (n = L): it shares them with
 * another request, which would see its rows move (copy them first,
 * paged_kv_copy_blocks).  Without refcounts those blocks must be the request's own.
 * 1 <= budget, sinks + recent <= budget, max_blocks <= 2^26.  A length outside [0, max_blocks * 16]
 * is clamped, T < L taken as L (PKA_DEVERR_SEQ_LEN); a table id outside the pool
 * leaves its rows unmoved (PKA_DEVERR_BAD_TABLE).
 * key_mass, key_pos, new_mass and new_pos 16-byte aligned.
 * workspace: 4-byte aligned, at least paged_kv_evict_ws_bytes() bytes, needs no
 * initialisation; calls sharing one must not overlap on the GPU. */
size_t paged_kv_evict_ws_bytes(int32_t num_layers, int32_t B, int32_t Hkv, int32_t max_blocks,
                               int32_t budget);
int paged_kv_evict(void* const* pools, int32_t num_layers, int32_t num_blocks,
                   int32_t num_kv_heads, int32_t block_size, int32_t head_dim,
                   const int32_t* block_tables, int32_t max_blocks, const int32_t* seq_lens,
                   const int32_t* total_lens, int32_t B, int32_t budget, int32_t sinks,
                   int32_t recent, const float* key_mass, float* new_mass, const int32_t* key_pos,
                   int32_t* new_pos, int32_t* new_seq_lens, const int32_t* refcounts,
                   void* workspace, size_t workspace_bytes, int32_t* err, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGED_ATTN_H_ */
