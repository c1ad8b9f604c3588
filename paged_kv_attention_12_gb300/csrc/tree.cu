// Draft trees of speculative decoding (sm_103a): a step's masks, positions and
// slots from the tokens' parents, and the walk along the target's tokens with
// the move of the accepted tokens' K/V rows.
#include "common.cuh"
#include "kernels.h"
#include "overlap.cuh"

namespace pka {

namespace {

constexpr unsigned kAll = 0xffffffffu;

// Rows [*q0, *q0 + n) of request b, n <= 64; n < 0: a bad span.
__device__ __forceinline__ int tree_span(const int32_t* query_start_loc, int b, int total_q,
                                         int max_query_len, int* q0) {
  const int lo = query_start_loc[b], hi = query_start_loc[b + 1];
  *q0 = lo;
  return lo < 0 || hi < lo || hi > total_q || hi - lo > max_query_len ? -1 : hi - lo;
}

// A value per tree token, two in a lane (tokens lane and lane + 32): that of
// token i (0 <= i < 64).
__device__ __forceinline__ int of_token(int lo, int hi, int i) {
  const int x = __shfl_sync(kAll, lo, i & 31), y = __shfl_sync(kAll, hi, i & 31);
  return i < 32 ? x : y;
}
__device__ __forceinline__ uint64_t of_token(uint64_t lo, uint64_t hi, int i) {
  const uint64_t x = __shfl_sync(kAll, lo, i & 31), y = __shfl_sync(kAll, hi, i & 31);
  return i < 32 ? x : y;
}

// One warp per request.  A token's ancestors by pointer doubling: after s
// steps a mask holds the 2^s nearest of them, and `up` the one that comes next
// (six steps for 64 tokens, fewer for shallow trees).  The last CTA's warps
// past the requests clear the rows that belong to none.
__global__ void __launch_bounds__(128) tree_plan_kernel(const TreePlanArgs a) {
  launch_dependents();
  wait_predecessor();
  const int lane = threadIdx.x & 31;
  const long long gwarp = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) / 32;
  if (gwarp >= a.batch) {
    const int first = a.query_start_loc[a.batch];
    if (first < 0) return;
    const long long others = static_cast<long long>(gridDim.x) * (blockDim.x / 32) - a.batch;
    for (long long r = first + (gwarp - a.batch) * 32 + lane; r < a.total_q; r += others * 32) {
      if (a.masks != nullptr) a.masks[r] = 0;
      if (a.positions != nullptr) a.positions[r] = 0;
      if (a.slots != nullptr) a.slots[r] = -1;
    }
    return;
  }
  const int b = static_cast<int>(gwarp);
  int q0;
  const int n = tree_span(a.query_start_loc, b, a.total_q, a.max_query_len, &q0);
  if (n < 0) {
    if (lane == 0) report(a.err, PKA_DEVERR_QUERY_LOC);
    return;
  }
  const int L = a.seq_lens[b];
  const int T = a.total_lens != nullptr ? a.total_lens[b] : L;
  const bool fits = n <= L && n <= T && L <= a.max_blocks * kBlockSize;
  if (!fits && lane == 0) report(a.err, PKA_DEVERR_SEQ_LEN);
  int up[2];
  uint64_t mask[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = lane + 32 * h;
    up[h] = i < n ? a.parents[q0 + i] : -1;
    if (up[h] < -1 || up[h] >= i) {
      if (i < n && up[h] != -1) report(a.err, PKA_DEVERR_TREE);
      up[h] = -1;
    }
    mask[h] = 1ull << i;
  }
  while (__any_sync(kAll, up[0] >= 0 || up[1] >= 0)) {  // (up falls at every step)
    const uint64_t m0 = mask[0], m1 = mask[1];
    const int u0 = up[0], u1 = up[1];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = max(h == 0 ? u0 : u1, 0);
      const uint64_t m = of_token(m0, m1, at);
      const int u = of_token(u0, u1, at);
      if ((h == 0 ? u0 : u1) >= 0) {
        mask[h] |= m;
        up[h] = u;
      }
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = lane + 32 * h;
    if (i >= n) continue;
    const int r = q0 + i;
    if (a.masks != nullptr) a.masks[r] = fits ? mask[h] : 0;
    if (a.positions != nullptr) a.positions[r] = fits ? T - n + __popcll(mask[h]) - 1 : 0;
    if (a.slots != nullptr) {
      int slot = -1;
      if (fits) {
        const int t = L - n + i;
        const int id = a.tables[static_cast<size_t>(b) * a.max_blocks + t / kBlockSize];
        if (static_cast<unsigned>(id) < static_cast<unsigned>(a.num_blocks))
          slot = id * kBlockSize + t % kBlockSize;
        else
          report(a.err, PKA_DEVERR_BAD_TABLE);
      }
      a.slots[r] = slot;
    }
  }
}

// One warp per (request, pool, KV head).  Every warp walks the tree for itself
// (a few votes per accepted token), so that no warp waits for another; the
// path's k-th row goes to the tree's k-th slot.  As the path's indexes grow,
// p_k >= k: a row's destination is no source of a later row, so batches of
// rows in path order need only load a batch before they store it.
constexpr int kRowBatch = 16;

template <int D>
__global__ void __launch_bounds__(128) tree_accept_kernel(const __grid_constant__ TreeAcceptArgs a) {
  launch_dependents();
  wait_predecessor();
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.x;
  const int item = blockIdx.y * (blockDim.x / 32) + threadIdx.x / 32;  // pool * Hkv + head
  const int items = max(1, a.num_pools * a.Hkv);
  if (item >= items) return;
  const bool writer = item == 0 && a.write_walk != 0;
  // (no other warp may read a length: new_seq_lens may be seq_lens)
  const int L = writer ? a.seq_lens[b] : 0x7fffffff;
  int q0;
  const int n = tree_span(a.query_start_loc, b, a.total_q, a.max_query_len, &q0);
  // What is wrong is reported once, in the end: a branch at each place costs 0.4 us
  // of 5.1 (four layers of wide trees).
  int bad = n < 0 && item == 0 ? PKA_DEVERR_QUERY_LOC : 0;
  // More tokens than keys: none is accepted.  (The plan gave them no slots, so that no
  // warp moves a row.)
  const bool none = max(n, 0) > L;
  if (none) bad |= PKA_DEVERR_SEQ_LEN;
  int parent[2], token[2], target[2], slot[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = lane + 32 * h;
    const bool in = i < n;
    parent[h] = in ? a.parents[q0 + i] : -1;
    token[h] = in ? a.tokens[q0 + i] : 0;
    target[h] = in ? a.targets[q0 + i] : 0;
    slot[h] = in && a.num_pools > 0 ? a.slots[q0 + i] : -1;
    if (in && item == 0 && (parent[h] < -1 || parent[h] >= i)) bad |= PKA_DEVERR_TREE;
  }
  // path[h]: index of the path's token number lane + 32 h
  int path[2] = {-1, -1}, count = 0, next = -1;
  for (int cur = 0; count < n;) {
    if (lane == count) path[0] = cur;
    if (lane + 32 == count) path[1] = cur;
    ++count;
    next = of_token(target[0], target[1], cur);
    const bool c0 = lane > cur && lane < n && parent[0] == cur && token[0] == next;
    const bool c1 = lane + 32 > cur && lane + 32 < n && parent[1] == cur && token[1] == next;
    const unsigned low = __ballot_sync(kAll, c0), high = __ballot_sync(kAll, c1);
    if ((low | high) == 0) break;
    cur = low != 0 ? __ffs(low) - 1 : 31 + __ffs(high);
  }
  if (writer) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (lane + 32 * h < a.max_query_len)
        a.path[static_cast<size_t>(b) * a.max_query_len + lane + 32 * h] = none ? -1 : path[h];
    __syncwarp();  // every lane has read the length
    if (lane == 0) {
      a.accepted[b] = none ? 0 : count;
      a.next_tokens[b] = none ? -1 : next;
      a.new_seq_lens[b] = none ? L : L - max(n, 0) + count;
    }
  }
  if (a.num_pools == 0) {
    if (bad != 0) report(a.err, bad);
    return;
  }
  const int pool = item / a.Hkv, head = item - pool * a.Hkv;
  uint8_t* base = static_cast<uint8_t*>(a.pools[pool]);
  constexpr int kLanes = D / 8;          // lanes of a row, 16 bytes each
  constexpr int kRows = 32 / kLanes;     // rows per instruction
  const int sub = lane / kLanes, part = lane % kLanes;
  for (int k0 = 0; k0 < count; k0 += kRowBatch) {
    uint4 x[kRowBatch / kRows];
    unsigned here = 0;
#pragma unroll
    for (int u = 0; u < kRowBatch / kRows; ++u) {
      const int k = k0 + u * kRows + sub;
      const int p = max(of_token(path[0], path[1], k & 63), 0);
      const int src = of_token(slot[0], slot[1], p), dst = of_token(slot[0], slot[1], k & 63);
      if (k >= count || p == k || src < 0 || dst < 0) continue;
      if (src / kBlockSize >= a.num_blocks || dst / kBlockSize >= a.num_blocks) {
        bad |= PKA_DEVERR_BAD_TABLE;
        continue;
      }
      here |= 1u << u;
      x[u] = *reinterpret_cast<const uint4*>(
          base + ((static_cast<size_t>(src / kBlockSize) * a.Hkv + head) * kBlockSize +
                  src % kBlockSize) * (2 * D) + part * 16);
    }
    __syncwarp();  // the batch's loads before its stores
#pragma unroll
    for (int u = 0; u < kRowBatch / kRows; ++u) {
      const int dst = of_token(slot[0], slot[1], (k0 + u * kRows + sub) & 63);
      if (here >> u & 1)
        *reinterpret_cast<uint4*>(
            base + ((static_cast<size_t>(dst / kBlockSize) * a.Hkv + head) * kBlockSize +
                    dst % kBlockSize) * (2 * D) + part * 16) = x[u];
    }
    __syncwarp();
  }
  if (bad != 0) report(a.err, bad);
}

}  // namespace

cudaError_t launch_tree_plan(const TreePlanArgs& a, cudaStream_t stream) {
  const long long warps = static_cast<long long>(a.batch) + 1;  // one more for the rows of no request
  return launch_overlapped(tree_plan_kernel, dim3(static_cast<unsigned>((warps + 3) / 4)), 128, 0,
                           stream, a);
}

cudaError_t launch_tree_accept(const TreeAcceptArgs& a, cudaStream_t stream) {
  const long long items = static_cast<long long>(a.num_pools) * a.Hkv;
  const dim3 grid(a.batch, static_cast<unsigned>(items < 4 ? 1 : (items + 3) / 4));
  return a.head_dim == 256 ? launch_overlapped(tree_accept_kernel<256>, grid, 128, 0, stream, a)
                           : launch_overlapped(tree_accept_kernel<128>, grid, 128, 0, stream, a);
}

}  // namespace pka
