// C-ABI layer of the 4-bit cache and of the page operations: argument checks
// on the host, then one launch (two for a compaction).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <stdint.h>

#include "kernels.h"
#include "kv4.cuh"
#include "paged_attn.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool good_scale(float s) { return std::isfinite(s) && s > 0.f && std::isfinite(6.f * s); }

int check_kv4_sizes(const pka_kv4_pool* kv) {
  if (kv->num_blocks <= 0 || kv->num_kv_heads <= 0) return PKA_ERR_SHAPE;
  if (kv->block_size != 16) return PKA_ERR_UNSUPPORTED;
  if (kv->head_dim != 128 && kv->head_dim != 256) return PKA_ERR_UNSUPPORTED;
  if (!good_scale(kv->k_scale) || !good_scale(kv->v_scale)) return PKA_ERR_SHAPE;
  return PKA_OK;
}

int check_kv4_pointers(const pka_kv4_pool* kv) {
  if (kv->k == nullptr || kv->v == nullptr) return PKA_ERR_NULL;
  return aligned16(kv->k) && aligned16(kv->v) ? PKA_OK : PKA_ERR_ALIGN;
}

// Workspace of the decode: a fixed area of arrival counters, then partial
// outputs and partial LSEs.  The counters lie in the same place whatever the
// sizes are, so that calls of all sizes can share a workspace in turn.
struct Kv4Layout {
  int32_t S, C;  // partial slots per (request, query head); the plan's shortest piece
  size_t o_bytes, lse_bytes;
  size_t total() const { return pka::kKv4CounterBytes + o_bytes + lse_bytes; }
};

int32_t kv4_max_tiles(int32_t max_seq_len, int32_t window) {
  const int32_t full = max_seq_len / 16 + (max_seq_len % 16 != 0);
  return window > 0 ? std::min(full, (window - 1) / 16 + 2) : full;
}

Kv4Layout kv4_layout(int32_t B, int32_t Hq, int32_t D, int32_t max_seq_len, int32_t window) {
  Kv4Layout L;
  const int32_t T = kv4_max_tiles(max_seq_len, window);
  // at most 30 pieces of a segment, of C tiles or more.  (The plan's own minimum
  // is 16 tiles, so that shorter requests leave some of their slots unused.)
  L.C = std::max(4, (T + 28) / 29);
  L.S = (T + L.C - 1) / L.C + 1;
  L.o_bytes = static_cast<size_t>(B) * Hq * L.S * D * sizeof(float);
  L.lse_bytes = (static_cast<size_t>(B) * Hq * L.S * sizeof(float) + 15) / 16 * 16;
  return L;
}

int check_pools(void* const* pools, int32_t num_pools, int32_t num_blocks, int64_t block_bytes) {
  if (num_pools < 0 || num_blocks <= 0 || block_bytes <= 0) return PKA_ERR_SHAPE;
  if (block_bytes % 16 != 0 || block_bytes > (int64_t(1) << 40)) return PKA_ERR_SHAPE;
  if (num_pools > 0 && pools == nullptr) return PKA_ERR_NULL;
  for (int32_t i = 0; i < num_pools; ++i) {
    if (pools[i] == nullptr) return PKA_ERR_NULL;
    if (!aligned16(pools[i])) return PKA_ERR_ALIGN;
  }
  return PKA_OK;
}

// The copies of `a` in every pool, kMaxCopyPools pools a launch.  The tables
// (if any) go with the first launch.
cudaError_t copy_in_pools(pka::CopyArgs a, void* const* pools, int32_t num_pools, int max_pairs,
                          cudaStream_t stream) {
  const int sms = pka::device_sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  int32_t done = 0;
  do {
    a.num_pools = std::min(num_pools - done, pka::kMaxCopyPools);
    for (int32_t i = 0; i < a.num_pools; ++i) a.pools[i] = pools[done + i];
    const cudaError_t e = pka::launch_copy_blocks(a, max_pairs, sms, stream);
    if (e != cudaSuccess) return e;
    a.tables = nullptr;
    done += a.num_pools;
  } while (done < num_pools);
  return cudaSuccess;
}

}  // namespace

extern "C" {

size_t paged_kv4_pool_bytes(int32_t num_blocks, int32_t num_kv_heads, int32_t head_dim) {
  if (num_blocks <= 0 || num_kv_heads <= 0 || (head_dim != 128 && head_dim != 256)) return 0;
  return static_cast<size_t>(num_blocks) * num_kv_heads * (head_dim / pka::kUnitChannels) *
         pka::kUnitBytes;
}

int paged_kv4_append(const void* k_new, const void* v_new, int64_t k_stride, int64_t v_stride,
                     const pka_kv4_pool* kv, const int32_t* slot_mapping, int32_t T,
                     int32_t* err, void* stream) {
  if (kv == nullptr) return PKA_ERR_NULL;
  int st = check_kv4_sizes(kv);
  if (st != PKA_OK) return st;
  const int64_t row = static_cast<int64_t>(kv->num_kv_heads) * kv->head_dim;
  if (T < 0 || k_stride < row || v_stride < row) return PKA_ERR_SHAPE;
  if (static_cast<int64_t>(kv->num_blocks) * kv->block_size > 0x7fffffffLL) return PKA_ERR_SHAPE;
  if (T == 0) return PKA_OK;
  if (k_new == nullptr || v_new == nullptr || slot_mapping == nullptr) return PKA_ERR_NULL;
  st = check_kv4_pointers(kv);
  if (st != PKA_OK) return st;
  if (!aligned16(k_new) || !aligned16(v_new) || k_stride % 8 != 0 || v_stride % 8 != 0)
    return PKA_ERR_ALIGN;
  pka::Kv4AppendArgs a{};
  a.k_new = static_cast<const uint16_t*>(k_new);
  a.v_new = static_cast<const uint16_t*>(v_new);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.k_pool = static_cast<uint8_t*>(kv->k);
  a.v_pool = static_cast<uint8_t*>(kv->v);
  a.k_scale = kv->k_scale;
  a.v_scale = kv->v_scale;
  a.k_scale6 = 6.f * kv->k_scale;
  a.v_scale6 = 6.f * kv->v_scale;
  a.slot_mapping = slot_mapping;
  a.err = err;
  a.T = T;
  a.Hkv = kv->num_kv_heads;
  a.head_dim = kv->head_dim;
  a.num_blocks = kv->num_blocks;
  const cudaError_t e =
      pka::launch_kv4_append(a, pka::device_sm_count(), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKA_OK : PKA_ERR_CUDA;
}

int paged_kv4_expand(const pka_kv4_pool* kv, const pka_kv_pool* dst, const int32_t* src_blocks,
                     const int32_t* dst_blocks, int32_t n, int32_t* err, void* stream) {
  if (kv == nullptr || dst == nullptr) return PKA_ERR_NULL;
  int st = check_kv4_sizes(kv);
  if (st != PKA_OK) return st;
  if (n < 0 || dst->num_blocks <= 0 || dst->num_kv_heads != kv->num_kv_heads ||
      dst->head_dim != kv->head_dim || dst->block_size != kv->block_size)
    return PKA_ERR_SHAPE;
  if (dst_blocks == nullptr && n > dst->num_blocks) return PKA_ERR_SHAPE;
  if (n == 0) return PKA_OK;
  if (src_blocks == nullptr || dst->k == nullptr || dst->v == nullptr) return PKA_ERR_NULL;
  st = check_kv4_pointers(kv);
  if (st != PKA_OK) return st;
  if (!aligned16(dst->k) || !aligned16(dst->v)) return PKA_ERR_ALIGN;
  pka::Kv4ExpandArgs a{};
  a.k4 = static_cast<const uint8_t*>(kv->k);
  a.v4 = static_cast<const uint8_t*>(kv->v);
  a.k16 = static_cast<uint16_t*>(const_cast<void*>(dst->k));
  a.v16 = static_cast<uint16_t*>(const_cast<void*>(dst->v));
  a.k_scale = kv->k_scale;
  a.v_scale = kv->v_scale;
  a.src_blocks = src_blocks;
  a.dst_blocks = dst_blocks;
  a.err = err;
  a.n = n;
  a.Hkv = kv->num_kv_heads;
  a.head_dim = kv->head_dim;
  a.src_num_blocks = kv->num_blocks;
  a.dst_num_blocks = dst->num_blocks;
  const cudaError_t e =
      pka::launch_kv4_expand(a, pka::device_sm_count(), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKA_OK : PKA_ERR_CUDA;
}

size_t paged_kv4_decode_attn_ws_bytes(int32_t B, int32_t Hq, int32_t Hkv, int32_t D,
                                      int32_t max_seq_len, int32_t window) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || max_seq_len < 0) return 0;
  return kv4_layout(B, Hq, D, max_seq_len, window).total();
}

int paged_kv4_decode_attn_ws(const void* q, void* out, const pka_kv4_pool* kv,
                             const int32_t* block_tables, int32_t max_blocks,
                             const int32_t* seq_lens, int32_t B, int32_t Hq,
                             int32_t max_seq_len, const pka_attn_params* params,
                             void* workspace, size_t workspace_bytes, void* stream) {
  if (kv == nullptr || params == nullptr) return PKA_ERR_NULL;
  int st = check_kv4_sizes(kv);
  if (st != PKA_OK) return st;
  if (B < 0 || Hq <= 0 || max_blocks <= 0 || max_seq_len < 0 || Hq % kv->num_kv_heads != 0)
    return PKA_ERR_SHAPE;
  if (static_cast<int64_t>(max_seq_len) > static_cast<int64_t>(max_blocks) * kv->block_size)
    return PKA_ERR_SHAPE;
  // the kernels clamp lengths to max_blocks * 16 in 32 bits
  if (max_blocks > 0x7fffffff / 16) return PKA_ERR_SHAPE;
  if (Hq / kv->num_kv_heads > 8) return PKA_ERR_UNSUPPORTED;
  if (!std::isfinite(params->scale) || std::isnan(params->softcap)) return PKA_ERR_SHAPE;
  if (B == 0) return PKA_OK;
  if (q == nullptr || out == nullptr || block_tables == nullptr || seq_lens == nullptr ||
      workspace == nullptr)
    return PKA_ERR_NULL;
  st = check_kv4_pointers(kv);
  if (st != PKA_OK) return st;
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace)) return PKA_ERR_ALIGN;
  const Kv4Layout L = kv4_layout(B, Hq, kv->head_dim, max_seq_len, params->window);
  if (workspace_bytes < L.total()) return PKA_ERR_WORKSPACE;
  // what the kernels count in 32 bits: the CTAs (one a segment and some more),
  // and the plan's sum of the requests' visible blocks
  int64_t per = max_blocks;
  if (params->window > 0) per = std::min<int64_t>(per, (params->window - 1) / 16 + 2);
  constexpr int64_t kMost = int64_t(1) << 30;
  if (static_cast<int64_t>(B) * kv->num_kv_heads > kMost || B * per > kMost) return PKA_ERR_SHAPE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  pka::Kv4DecodeArgs a{};
  a.base.q = static_cast<const uint16_t*>(q);
  a.base.out = out;
  a.base.tables = block_tables;
  a.base.seq_lens = seq_lens;
  a.base.err = params->err;
  a.base.batch = B;
  a.base.Hq = Hq;
  a.base.Hkv = kv->num_kv_heads;
  a.base.num_blocks = kv->num_blocks;
  a.base.max_blocks = max_blocks;
  a.base.scale = params->scale;
  a.base.softcap = params->softcap > 1e38f ? 0.f : params->softcap;
  a.base.window = params->window;
  a.base.num_splits = L.S;
  a.base.split_blocks = L.C;
  a.base.seg_counters = reinterpret_cast<int32_t*>(ws);
  a.base.partial_o = reinterpret_cast<float*>(ws + pka::kKv4CounterBytes);
  a.base.partial_lse = reinterpret_cast<float*>(ws + pka::kKv4CounterBytes + L.o_bytes);
  a.k4 = static_cast<const uint8_t*>(kv->k);
  a.v4 = static_cast<const uint8_t*>(kv->v);
  a.k_scale = kv->k_scale;
  a.v_scale = kv->v_scale;
  a.max_tiles = kv4_max_tiles(max_seq_len, params->window);
  const int sms = pka::device_sm_count();
  if (sms <= 0) return PKA_ERR_CUDA;
  const cudaError_t e =
      pka::launch_kv4_decode(a, kv->head_dim, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKA_OK : PKA_ERR_CUDA;
}

int paged_kv_ref_blocks(const int32_t* block_tables, int32_t max_blocks, const int32_t* seq_lens,
                        int32_t B, int32_t num_blocks, int32_t delta, int32_t* refcounts,
                        int32_t* err, void* stream) {
  if (B < 0 || max_blocks <= 0 || max_blocks > 0x7fffffff / 16 || num_blocks <= 0)
    return PKA_ERR_SHAPE;
  if (B == 0) return PKA_OK;
  if (block_tables == nullptr || seq_lens == nullptr || refcounts == nullptr) return PKA_ERR_NULL;
  pka::RefArgs a{};
  a.tables = block_tables;
  a.seq_lens = seq_lens;
  a.refcounts = refcounts;
  a.err = err;
  a.batch = B;
  a.max_blocks = max_blocks;
  a.num_blocks = num_blocks;
  a.delta = delta;
  const cudaError_t e =
      pka::launch_ref_blocks(a, pka::device_sm_count(), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKA_OK : PKA_ERR_CUDA;
}

int paged_kv_copy_blocks(void* const* pools, int32_t num_pools, int32_t num_blocks,
                         int64_t block_bytes, const int32_t* src, const int32_t* dst, int32_t n,
                         int32_t* err, void* stream) {
  const int st = check_pools(pools, num_pools, num_blocks, block_bytes);
  if (st != PKA_OK) return st;
  if (n < 0) return PKA_ERR_SHAPE;
  if (n == 0 || num_pools == 0) return PKA_OK;
  if (src == nullptr || dst == nullptr) return PKA_ERR_NULL;
  pka::CopyArgs a{};
  a.block_bytes = block_bytes;
  a.src = src;
  a.dst = dst;
  a.err = err;
  a.num_blocks = num_blocks;
  a.n = n;
  const cudaError_t e =
      copy_in_pools(a, pools, num_pools, n, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKA_OK : PKA_ERR_CUDA;
}

int paged_kv_compact(void* const* pools, int32_t num_pools, int32_t num_blocks,
                     int64_t block_bytes, const int32_t* refcounts, int32_t* new_refcounts,
                     const int32_t* block_tables, int32_t* new_tables, int32_t max_blocks,
                     const int32_t* seq_lens, int32_t B, int32_t* remap, int32_t* moves,
                     int32_t* err, void* stream) {
  const int st = check_pools(pools, num_pools, num_blocks, num_pools > 0 ? block_bytes : 16);
  if (st != PKA_OK) return st;
  if (B < 0 || num_blocks > (1 << 30)) return PKA_ERR_SHAPE;
  if (B > 0 && (max_blocks <= 0 || max_blocks > 0x7fffffff / 16)) return PKA_ERR_SHAPE;
  if (refcounts == nullptr || new_refcounts == nullptr || remap == nullptr || moves == nullptr)
    return PKA_ERR_NULL;
  if (B > 0 && (block_tables == nullptr || new_tables == nullptr || seq_lens == nullptr))
    return PKA_ERR_NULL;
  pka::PlanArgs p{};
  p.refcounts = refcounts;
  p.new_refcounts = new_refcounts;
  p.remap = remap;
  p.moves = moves;
  p.num_blocks = num_blocks;
  cudaError_t e = pka::launch_compact_plan(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return PKA_ERR_CUDA;
  if (num_pools == 0 && B == 0) return PKA_OK;
  pka::CopyArgs a{};
  a.block_bytes = num_pools > 0 ? block_bytes : 16;
  a.moves = moves;
  a.remap = remap;
  a.err = err;
  a.num_blocks = num_blocks;
  if (B > 0) {
    a.tables = block_tables;
    a.new_tables = new_tables;
    a.seq_lens = seq_lens;
    a.batch = B;
    a.max_blocks = max_blocks;
  }
  e = copy_in_pools(a, pools, num_pools, num_blocks / 2, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKA_OK : PKA_ERR_CUDA;
}

}  // extern "C"
