// C-ABI layer of the draft trees and of the eviction: argument checks on the
// host, then the launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <stdint.h>

#include "kernels.h"
#include "paged_attn.h"

namespace {

constexpr int32_t kMaxTree = 64;  // drafted tokens of a request (bits of a mask)
// Blocks of a table row, where keys are counted in tiles: 2^30 keys, so that no
// tile's end passes 32 bits.
constexpr int32_t kMaxRowBlocks = 1 << 26;
// Bytes of K (and of V) that a segment's moves take at most where the selection
// makes them itself, its CTA beside a second launch over the whole GPU: 2 segments of
// 411 keys cut to 256, D = 128: 11.1 us (12.0 with the second launch), 64 of them 11.9
// (14.1); D = 256: 12.4 (12.4) and 13.2 (15.0).  1000 keys cut to 500: D = 128 15.8
// (14.1) and 17.0 (16.6), D = 256 18.9 (14.5) and 23.9 (20.2).
constexpr int64_t kMovedHere = 64 << 10;

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool aligned16(const void* p) { return aligned(p, 16); }

int check_sizes(int32_t num_blocks, int32_t num_kv_heads, int32_t block_size, int32_t head_dim) {
  if (num_blocks <= 0 || num_kv_heads <= 0) return PKA_ERR_SHAPE;
  if (block_size != 16) return PKA_ERR_UNSUPPORTED;
  if (head_dim != 128 && head_dim != 256) return PKA_ERR_UNSUPPORTED;
  // rows of the pool, and slot numbers, are counted in 32 bits
  if (static_cast<int64_t>(num_blocks) * num_kv_heads * 16 > 0x7fffffffLL) return PKA_ERR_SHAPE;
  return PKA_OK;
}

uint64_t pool_bytes(int32_t num_blocks, int32_t num_kv_heads, int32_t head_dim) {
  return static_cast<uint64_t>(num_blocks) * num_kv_heads * 16 * head_dim * 2;
}

int check_tree(int32_t B, int32_t total_q, int32_t max_query_len) {
  if (B < 0 || B == 0x7fffffff || total_q < 0 || max_query_len < 0) return PKA_ERR_SHAPE;
  return max_query_len > kMaxTree ? PKA_ERR_UNSUPPORTED : PKA_OK;
}

int check_pools(void* const* pools, int32_t n) {
  if (n > 0 && pools == nullptr) return PKA_ERR_NULL;
  for (int32_t i = 0; i < n; ++i) {
    if (pools[i] == nullptr) return PKA_ERR_NULL;
    if (!aligned16(pools[i])) return PKA_ERR_ALIGN;
  }
  return PKA_OK;
}

// Whether two of n pools of so many bytes share memory: rows would move twice.
// Up to 256 pools are sorted by address first (each with each are 8128 comparisons
// for 64 layers).
bool pools_overlap(void* const* pools, int32_t n, uint64_t bytes) {
  auto at = [&](int32_t i) { return reinterpret_cast<uintptr_t>(pools[i]); };
  constexpr int32_t kSorted = 256;
  if (n > kSorted) {
    for (int32_t i = 1; i < n; ++i)
      for (int32_t j = 0; j < i; ++j)
        if ((at(i) > at(j) ? at(i) - at(j) : at(j) - at(i)) < bytes) return true;
    return false;
  }
  uintptr_t sorted[kSorted];
  for (int32_t i = 0; i < n; ++i) sorted[i] = at(i);
  std::sort(sorted, sorted + n);
  for (int32_t i = 1; i < n; ++i)
    if (sorted[i] - sorted[i - 1] < bytes) return true;
  return false;
}

// Workspace of the tree attention: two partial tiles for each chunk of the
// work line, their LSEs and what the chunks cut.
struct TreeLayout {
  size_t o, lse, cuts;
  size_t total() const { return o + lse + cuts; }
};

TreeLayout tree_layout(int32_t group, int32_t D, int32_t max_query_len) {
  const size_t rows = static_cast<size_t>(2) * pka::kTreeMaxCtas *
                      pka::tree_tile_rows(max_query_len, group);
  return TreeLayout{rows * D * sizeof(float), rows * sizeof(float),
                    pka::kTreeMaxCtas * sizeof(int4)};
}

struct EvictLayout {
  int64_t segs, moves;  // segments; moves of one at most
  int64_t words() const { return segs * (1 + 4 * moves); }
};

EvictLayout evict_layout(int32_t layers, int32_t B, int32_t Hkv, int32_t max_blocks,
                         int32_t budget) {
  const int64_t keys = static_cast<int64_t>(max_blocks) * 16;
  return EvictLayout{static_cast<int64_t>(layers) * B * Hkv,
                     std::max<int64_t>(0, std::min<int64_t>(budget, keys - budget))};
}

}  // namespace

extern "C" {

int paged_tree_plan(const int32_t* parents, const int32_t* query_start_loc,
                    const int32_t* seq_lens, const int32_t* total_lens,
                    const int32_t* block_tables, int32_t max_blocks, int32_t num_blocks, int32_t B,
                    int32_t total_q, int32_t max_query_len, uint64_t* tree_masks,
                    int32_t* positions, int32_t* slots, int32_t* err, void* stream) {
  const int st = check_tree(B, total_q, max_query_len);
  if (st != PKA_OK) return st;
  if (max_blocks <= 0 || max_blocks > 0x7fffffff / 16 || num_blocks <= 0 ||
      num_blocks > 0x7fffffff / 16)
    return PKA_ERR_SHAPE;
  if (total_q == 0) return PKA_OK;
  // (without requests every row is padding)
  if (parents == nullptr || query_start_loc == nullptr ||
      (B > 0 && (seq_lens == nullptr || block_tables == nullptr)))
    return PKA_ERR_NULL;
  if (!aligned(tree_masks, 8)) return PKA_ERR_ALIGN;
  pka::TreePlanArgs a{};
  a.parents = parents;
  a.query_start_loc = query_start_loc;
  a.seq_lens = seq_lens;
  a.total_lens = total_lens;
  a.tables = block_tables;
  a.masks = reinterpret_cast<unsigned long long*>(tree_masks);
  a.positions = positions;
  a.slots = slots;
  a.err = err;
  a.batch = B;
  a.num_blocks = num_blocks;
  a.max_blocks = max_blocks;
  a.total_q = total_q;
  a.max_query_len = max_query_len;
  return pka::launch_tree_plan(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PKA_OK
                                                                                    : PKA_ERR_CUDA;
}

size_t paged_tree_attn_ws_bytes(int32_t Hq, int32_t Hkv, int32_t D, int32_t max_query_len) {
  if (Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || D <= 0 || max_query_len < 0 ||
      max_query_len > kMaxTree)
    return 0;
  return tree_layout(Hq / Hkv, D, max_query_len).total();
}

int paged_tree_attn_ws(const void* q, void* out, const pka_kv_pool* kv,
                       const int32_t* block_tables, int32_t max_blocks,
                       const int32_t* query_start_loc, const uint64_t* tree_masks,
                       const int32_t* seq_lens, int32_t B, int32_t Hq, int32_t total_q,
                       int32_t max_query_len, int32_t max_seq_len, const pka_attn_params* params,
                       void* workspace, size_t workspace_bytes, void* stream) {
  if (kv == nullptr || params == nullptr) return PKA_ERR_NULL;
  int st = check_sizes(kv->num_blocks, kv->num_kv_heads, kv->block_size, kv->head_dim);
  if (st != PKA_OK) return st;
  const int32_t Hkv = kv->num_kv_heads;
  if (Hq <= 0 || Hq % Hkv != 0) return PKA_ERR_SHAPE;
  const int32_t G = Hq / Hkv;
  if (G != 1 && G != 2 && G != 4 && G != 8) return PKA_ERR_UNSUPPORTED;
  st = check_tree(B, total_q, max_query_len);
  if (st != PKA_OK) return st;
  if (max_blocks <= 0 || max_blocks > kMaxRowBlocks || max_seq_len < 0 ||
      max_seq_len > static_cast<int64_t>(max_blocks) * 16)
    return PKA_ERR_SHAPE;
  if (!std::isfinite(params->scale) || std::isnan(params->softcap)) return PKA_ERR_SHAPE;
  if (B == 0 || total_q == 0 || max_query_len == 0) return PKA_OK;
  if (q == nullptr || out == nullptr || kv->k == nullptr || kv->v == nullptr ||
      block_tables == nullptr || query_start_loc == nullptr || tree_masks == nullptr ||
      seq_lens == nullptr || workspace == nullptr)
    return PKA_ERR_NULL;
  if (!aligned16(q) || !aligned16(out) || !aligned16(kv->k) || !aligned16(kv->v) ||
      !aligned16(workspace) || !aligned(tree_masks, 8))
    return PKA_ERR_ALIGN;
  const TreeLayout lay = tree_layout(G, kv->head_dim, max_query_len);
  if (workspace_bytes < lay.total()) return PKA_ERR_WORKSPACE;
  // the work line (segments times their blocks and a fixed cost) is counted in 32 bits
  const int64_t tile_rows = pka::tree_tile_rows(max_query_len, G);
  const int64_t segs = static_cast<int64_t>(B) * Hkv * ((max_query_len * G + tile_rows - 1) / tile_rows);
  int64_t per = max_blocks;
  if (params->window > 0) per = std::min<int64_t>(per, (static_cast<int64_t>(params->window) + kMaxTree) / 16 + 2);
  if (segs > (int64_t(1) << 30) / (per + pka::kTreePieceUnits(128))) return PKA_ERR_SHAPE;
  const int sms = pka::device_sm_count();
  if (sms <= 0) return PKA_ERR_CUDA;
  int64_t longest = max_seq_len / 16 + (max_seq_len % 16 != 0);
  if (params->window > 0)
    longest = std::min<int64_t>(longest, (static_cast<int64_t>(params->window) + max_query_len) / 16 + 2);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  pka::TreeArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.out = static_cast<uint16_t*>(out);
  a.k = static_cast<const uint16_t*>(kv->k);
  a.v = static_cast<const uint16_t*>(kv->v);
  a.tables = block_tables;
  a.query_start_loc = query_start_loc;
  a.masks = reinterpret_cast<const unsigned long long*>(tree_masks);
  a.seq_lens = seq_lens;
  a.err = params->err;
  a.partial_o = reinterpret_cast<float*>(ws);
  a.partial_lse = reinterpret_cast<float*>(ws + lay.o);
  a.cuts = reinterpret_cast<int4*>(ws + lay.o + lay.lse);
  a.batch = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.num_blocks = kv->num_blocks;
  a.max_blocks = max_blocks;
  a.total_q = total_q;
  a.max_query_len = max_query_len;
  a.min_chunk = pka::kTreePieceUnits(kv->head_dim) + 8;
  // A merge costs about 6 us, as much as streaming 28 blocks at D = 256.
  a.whole_slack = kv->head_dim == 256 ? 28 : 56;
  const int64_t ctas = std::min(sms, pka::kTreeMaxCtas);
  // Where there are two CTAs for each segment, pairs of them share a segment of
  // more than two tiles and need no merge, up to the length where cutting would
  // gain a merge's worth, the mean length taken as half of the longest.  64
  // segments of 200, 560, 1500 keys, D = 256: pairs 13.1, 16.4, 26.2 us; whole
  // 13.8, 18.8; cut 21.0, 23.9, 31.7.  4 segments of 200, 560, 1000, 1500: pairs
  // 10.8, 13.5, 17.7, 22.9; whole 11.4, 17.3; cut 17.5, 17.4, 18.5, 18.1.  Two tiles
  // (100 keys): pairs 9.3, whole 8.9.  D = 128, 64 segments of 300, 1000, 1500: pairs
  // 10.9, 14.9, 17.4; whole 10.9, 16.7; cut 18.0, 22.6, 24.5.
  const bool pairs = 2 * segs <= ctas && longest > (kv->head_dim == 256 ? 8 : 16) &&
                     longest * (ctas - segs) <= 2 * ctas * a.whole_slack;
  a.pair = pairs ? static_cast<int32_t>(segs) : 0;
  // (100 segments of 34 blocks, D = 256: cut 23.1 us, whole 20.9)
  a.may_cut = !pairs && (segs > ctas || longest + pka::kTreePieceUnits(kv->head_dim) >
                                            a.min_chunk + a.whole_slack);
  a.scale = params->scale;
  a.softcap = params->softcap > 1e38f ? 0.f : params->softcap;
  a.window = params->window;
  return pka::launch_tree_attn(a, kv->head_dim, sms, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? PKA_OK
             : PKA_ERR_CUDA;
}

int paged_tree_accept(void* const* pools, int32_t num_pools, int32_t num_blocks,
                      int32_t num_kv_heads, int32_t block_size, int32_t head_dim,
                      const int32_t* parents, const int32_t* tokens, const int32_t* targets,
                      const int32_t* slots, const int32_t* query_start_loc,
                      const int32_t* seq_lens, int32_t B, int32_t total_q, int32_t max_query_len,
                      int32_t* path, int32_t* accepted, int32_t* next_tokens,
                      int32_t* new_seq_lens, int32_t* err, void* stream) {
  if (num_pools < 0) return PKA_ERR_SHAPE;
  int st = num_pools > 0 ? check_sizes(num_blocks, num_kv_heads, block_size, head_dim) : PKA_OK;
  if (st == PKA_OK) st = check_tree(B, total_q, max_query_len);
  if (st != PKA_OK) return st;
  if (B == 0) return PKA_OK;
  // (without rows every tree is empty)
  if (total_q > 0 && (parents == nullptr || tokens == nullptr || targets == nullptr ||
                      (slots == nullptr && num_pools > 0)))
    return PKA_ERR_NULL;
  if (query_start_loc == nullptr || seq_lens == nullptr || (path == nullptr && max_query_len > 0) ||
      accepted == nullptr || next_tokens == nullptr || new_seq_lens == nullptr)
    return PKA_ERR_NULL;
  st = check_pools(pools, num_pools);
  if (st != PKA_OK) return st;
  // (255 pools a launch, 4 warps a CTA; without pools their sizes are not looked at)
  if (num_pools > 0 && num_kv_heads > 1024) return PKA_ERR_SHAPE;
  if (pools_overlap(pools, num_pools, pool_bytes(num_blocks, num_kv_heads, head_dim)))
    return PKA_ERR_SHAPE;
  pka::TreeAcceptArgs a{};
  a.parents = parents;
  a.tokens = tokens;
  a.targets = targets;
  a.slots = slots;
  a.query_start_loc = query_start_loc;
  a.seq_lens = seq_lens;
  a.path = path;
  a.write_walk = 1;
  a.accepted = accepted;
  a.next_tokens = next_tokens;
  a.new_seq_lens = new_seq_lens;
  a.err = err;
  a.batch = B;
  a.total_q = total_q;
  a.max_query_len = max_query_len;
  a.num_blocks = num_blocks;
  a.Hkv = num_pools > 0 ? num_kv_heads : 1;
  a.head_dim = head_dim;
  int32_t done = 0;
  do {
    // the first launch writes the walk's results, those after it move rows only
    a.num_pools = std::min(num_pools - done, pka::kMaxTreePools);
    for (int32_t i = 0; i < a.num_pools; ++i) a.pools[i] = pools[done + i];
    if (pka::launch_tree_accept(a, static_cast<cudaStream_t>(stream)) != cudaSuccess)
      return PKA_ERR_CUDA;
    a.write_walk = 0;
    done += a.num_pools;
  } while (done < num_pools);
  return PKA_OK;
}

size_t paged_kv_evict_ws_bytes(int32_t num_layers, int32_t B, int32_t Hkv, int32_t max_blocks,
                               int32_t budget) {
  if (num_layers <= 0 || B <= 0 || Hkv <= 0 || max_blocks <= 0 || budget <= 0) return 0;
  const EvictLayout lay = evict_layout(num_layers, B, Hkv, max_blocks, budget);
  return static_cast<size_t>(lay.words() + B) * sizeof(int32_t);
}

int paged_kv_evict(void* const* pools, int32_t num_layers, int32_t num_blocks,
                   int32_t num_kv_heads, int32_t block_size, int32_t head_dim,
                   const int32_t* block_tables, int32_t max_blocks, const int32_t* seq_lens,
                   const int32_t* total_lens, int32_t B, int32_t budget, int32_t sinks,
                   int32_t recent, const float* key_mass, float* new_mass, const int32_t* key_pos,
                   int32_t* new_pos, int32_t* new_seq_lens, const int32_t* refcounts,
                   void* workspace, size_t workspace_bytes, int32_t* err, void* stream) {
  int st = check_sizes(num_blocks, num_kv_heads, block_size, head_dim);
  if (st != PKA_OK) return st;
  if (num_layers <= 0 || B < 0 || max_blocks <= 0 || max_blocks > kMaxRowBlocks)
    return PKA_ERR_SHAPE;
  if (budget <= 0 || sinks < 0 || recent < 0 ||
      static_cast<int64_t>(sinks) + recent > budget)
    return PKA_ERR_SHAPE;
  if (B == 0) return PKA_OK;
  if (block_tables == nullptr || seq_lens == nullptr || key_mass == nullptr ||
      new_mass == nullptr || key_pos == nullptr || new_pos == nullptr || new_seq_lens == nullptr ||
      workspace == nullptr)
    return PKA_ERR_NULL;
  if (num_layers > 0x7fffffff / 2) return PKA_ERR_SHAPE;
  st = check_pools(pools, 2 * num_layers);
  if (st != PKA_OK) return st;
  if (!aligned(workspace, 4) || !aligned16(key_mass) || !aligned16(new_mass) ||
      !aligned16(key_pos) || !aligned16(new_pos))
    return PKA_ERR_ALIGN;
  // a cluster of up to 8 CTAs for each segment
  if (static_cast<int64_t>(num_layers) * B > (1 << 27) / num_kv_heads) return PKA_ERR_SHAPE;
  const EvictLayout lay = evict_layout(num_layers, B, num_kv_heads, max_blocks, budget);
  if (workspace_bytes < static_cast<size_t>(lay.words() + B) * sizeof(int32_t))
    return PKA_ERR_WORKSPACE;
  if (pools_overlap(pools, 2 * num_layers, pool_bytes(num_blocks, num_kv_heads, head_dim)))
    return PKA_ERR_SHAPE;
  const int sms = pka::device_sm_count();
  if (sms <= 0) return PKA_ERR_CUDA;
  pka::EvictMoveArgs m{};
  pka::EvictArgs& a = m.a;
  a.mass = key_mass;
  a.pos = key_pos;
  a.new_mass = new_mass;
  a.new_pos = new_pos;
  a.tables = block_tables;
  a.seq_lens = seq_lens;
  a.total_lens = total_lens;
  a.refcounts = refcounts;
  a.new_seq_lens = new_seq_lens;
  a.err = err;
  const int64_t list = lay.segs * lay.moves;
  a.counts = static_cast<int32_t*>(workspace);
  a.kept = a.counts + lay.segs;
  a.move_src = a.kept + B;
  a.move_dst = a.move_src + list;
  a.move_pos = a.move_dst + list;
  a.move_mass = reinterpret_cast<float*>(a.move_pos + list);
  a.batch = B;
  a.Hkv = num_kv_heads;
  a.num_blocks = num_blocks;
  a.max_blocks = max_blocks;
  a.budget = budget;
  a.sinks = sinks;
  a.recent = recent;
  a.max_moves = static_cast<int32_t>(lay.moves);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  // One launch for few moves of a CTA's segments.  (CTAs of a request read its length
  // at any time: the launch that reads lengths may not write them.)
  auto apart = [&](const int32_t* p) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(new_seq_lens);
    const uintptr_t y = reinterpret_cast<uintptr_t>(p);
    return p == nullptr || (x > y ? x - y : y - x) >= static_cast<uintptr_t>(B) * sizeof(int32_t);
  };
  if (apart(seq_lens) && apart(total_lens) && num_layers <= pka::kMaxEvictLayers &&
      max_blocks <= pka::kEvictCtaKeys / 16 && lay.moves * head_dim * 2 <= kMovedHere) {
    m.here = head_dim;
    m.layers = num_layers;
    for (int32_t i = 0; i < 2 * num_layers; ++i) m.pools[i] = pools[i];
    return pka::launch_evict_select(m, num_layers, s) == cudaSuccess ? PKA_OK : PKA_ERR_CUDA;
  }
  if (pka::launch_evict_select(m, num_layers, s) != cudaSuccess) return PKA_ERR_CUDA;
  for (int32_t done = 0; done < num_layers; done += m.layers) {
    m.first_layer = done;
    m.layers = std::min(num_layers - done, pka::kMaxEvictLayers);
    for (int32_t i = 0; i < 2 * m.layers; ++i) m.pools[i] = pools[2 * done + i];
    if (pka::launch_evict_move(m, head_dim, sms, s) != cudaSuccess) return PKA_ERR_CUDA;
  }
  return PKA_OK;
}

}  // extern "C"
