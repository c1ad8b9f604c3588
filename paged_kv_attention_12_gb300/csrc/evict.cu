// Eviction from a block-paged cache by accumulated attention weight (sm_103a):
// which keys of a (layer, request, KV head) stay, and their move to the front.
//
// Of L keys the n = min(L, budget) first in this order stay: the first and the
// most recent tokens ("held"), lowest index first, then the others by mass,
// ties by index.  Kept keys at n or above move into the holes below n, the
// highest of them into the lowest hole, so that as few rows move as there are
// holes, sources and destinations are disjoint and every key keeps its mass and
// its position beside it.
//
// Two launches: the selection (a cluster per segment: reads 8 bytes a key,
// writes the list of moves), then the moves over all segments (bound by HBM).
#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"
#include "overlap.cuh"

namespace cg = cooperative_groups;

namespace pka {

namespace {

constexpr int kSelWarps = 32;
constexpr int kSelThreads = kSelWarps * 32;
constexpr int kKeep = 16;                 // keys per thread that stay in registers
constexpr int kBins = 2048;
// digits of a 32-bit rank, from the top: 11, 11 and 10 bits
constexpr int kPasses = 3;
__device__ __forceinline__ int digit_shift(int pass) { return pass == 0 ? 21 : pass == 1 ? 10 : 0; }
__device__ __forceinline__ int digit_bits(int pass) { return pass == 2 ? 10 : 11; }

constexpr uint32_t kHeld = 0xffffffffu;   // above every mass

// Masses in their order as unsigned numbers; NaN below all of them.
__device__ __forceinline__ uint32_t rank_of(float mass) {
  if (isnan(mass)) return 0;
  const uint32_t x = __float_as_uint(mass == 0.f ? 0.f : mass);
  return x & 0x80000000u ? ~x : x | 0x80000000u;
}

template <int CTAS>
__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(const EvictArgs a) {
  // hist is read, and totals are written, by the other CTAs of the cluster
  __shared__ int hist[kPasses][kBins];
  __shared__ int totals[4][CTAS];
  __shared__ int warp_sum[kSelWarps];
  __shared__ int found[3];
  __shared__ int shared_block;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = CTAS > 1 ? static_cast<int>(cluster.block_rank()) : 0;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  auto sync = [&]() {
    if constexpr (CTAS > 1)
      cluster.sync();
    else
      __syncthreads();
  };
  for (int i = threadIdx.x; i < kPasses * kBins; i += kSelThreads) hist[0][i] = 0;
  if (threadIdx.x == 0) shared_block = 0;
  launch_dependents();
  wait_predecessor();

  const int seg = blockIdx.x / CTAS;  // (layer * B + request) * Hkv + head
  const int b = seg / a.Hkv % a.batch;
  const bool teller = seg / a.Hkv == b && seg % a.Hkv == 0 && rank == 0 && threadIdx.x == 0;
  const int max_keys = a.max_blocks * kBlockSize;
  int L = a.seq_lens[b];
  int T = a.total_lens != nullptr ? a.total_lens[b] : L;
  if (L < 0 || L > max_keys || T < L) {
    if (teller) report(a.err, PKA_DEVERR_SEQ_LEN);
    L = max(0, min(L, max_keys));
    T = max(T, L);
  }
  int n = min(L, a.budget);
  __syncthreads();
  if (a.refcounts != nullptr && n < L) {
    // a block that would be written and that another request reads too
    const int32_t* row = a.tables + static_cast<size_t>(b) * a.max_blocks;
    bool shared = false;
    for (int j = threadIdx.x; j < (n + kBlockSize - 1) / kBlockSize; j += kSelThreads) {
      const int id = row[j];
      if (static_cast<unsigned>(id) < static_cast<unsigned>(a.num_blocks))
        shared = shared || a.refcounts[id] > 1;
    }
    if (shared) shared_block = 1;
    __syncthreads();
    if (shared_block != 0) n = L;  // (the same in every CTA: all of them look at the whole row)
  }
  if (teller) a.kept[b] = n;
  if (rank == 0 && threadIdx.x == 0 && n == L) a.counts[seg] = 0;

  const size_t first = static_cast<size_t>(seg) * max_keys;
  const float* mass = a.mass + first;
  const int32_t* pos = a.pos + first;
  float* new_mass = a.new_mass + first;
  int32_t* new_pos = a.new_pos + first;
  // keys without a position are the latest ones, in order
  auto position = [&](int t, int p) { return p >= 0 ? p : T - (L - t); };

  // this warp's keys: a run of its own, 32 at a time
  const int per_warp = ((L + CTAS * kSelWarps - 1) / (CTAS * kSelWarps) + 31) / 32 * 32;
  const int lo = min(static_cast<long long>(rank * kSelWarps + warp) * per_warp,
                     static_cast<long long>(L));
  const int hi = min(lo + per_warp, L);
  if (n == L) {
    for (int t = lo + lane; t < hi; t += 32) {
      new_mass[t] = mass[t];
      new_pos[t] = position(t, pos[t]);
    }
    return;  // the whole cluster
  }

  auto rank_at = [&](int t) -> uint32_t {
    const float m = mass[t];
    const int p = position(t, pos[t]);
    return p < a.sinks || p >= T - a.recent ? kHeld : rank_of(m);
  };
  uint32_t keep[kKeep];
#pragma unroll
  for (int k = 0; k < kKeep; ++k) {
    const int t = lo + 32 * k + lane;
    keep[k] = t < hi ? rank_at(t) : 0;
  }
  // f(t, rank, whether the lane has a key) for the warp's keys, in order; a
  // step's lanes hold consecutive keys
  auto each = [&](auto f) {
#pragma unroll
    for (int k = 0; k < kKeep; ++k)
      if (lo + 32 * k < hi) f(lo + 32 * k + lane, keep[k], lo + 32 * k + lane < hi);
    for (int base = lo + 32 * kKeep; base < hi; base += 32) {
      const int t = base + lane;
      f(t, t < hi ? rank_at(t) : 0u, t < hi);
    }
  };

  // ---------------------------------------- the rank of the last key that stays
  uint32_t prefix = 0;
  int need = n, equal = 0;  // keys still to find among those with this prefix
#pragma unroll 1
  for (int pass = 0; pass < kPasses; ++pass) {
    const int shift = digit_shift(pass), bits = digit_bits(pass);
    each([&](int, uint32_t u, bool in) {
      if (in && (pass == 0 || u >> (shift + bits) == prefix))
        atomicAdd(&hist[pass][(u >> shift) & ((1u << bits) - 1)], 1);
    });
    sync();
    // bins from the top, two a thread
    const int bins = 1 << bits;
    int c[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int bin = bins - 1 - (2 * static_cast<int>(threadIdx.x) + e);
      if (bin < 0) continue;
      if constexpr (CTAS > 1) {
#pragma unroll
        for (int r = 0; r < CTAS; ++r) c[e] += *cluster.map_shared_rank(&hist[pass][bin], r);
      } else {
        c[e] = hist[pass][bin];
      }
    }
    int incl = c[0] + c[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int above = incl - c[0] - c[1];
    for (int w = 0; w < warp; ++w) above += warp_sum[w];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (above < need && need <= above + c[e]) {  // exactly one bin
        found[0] = bins - 1 - (2 * static_cast<int>(threadIdx.x) + e);
        found[1] = need - above;
        found[2] = c[e];
      }
      above += c[e];
    }
    __syncthreads();
    prefix = prefix << bits | static_cast<uint32_t>(found[0]);
    need = found[1];
    equal = found[2];
    __syncthreads();
  }
  const uint32_t last = prefix;

  // exclusive count over the cluster's warps in key order; slot: which of the
  // exchanges this is
  auto before_of = [&](int count, int slot, int* total) {
    if (lane == 0) warp_sum[warp] = count;
    __syncthreads();
    int below = 0, all = 0;
    for (int w = 0; w < kSelWarps; ++w) {
      const int v = warp_sum[w];
      if (w < warp) below += v;
      all += v;
    }
    if constexpr (CTAS > 1) {
      if (threadIdx.x < CTAS) *cluster.map_shared_rank(&totals[slot][rank], threadIdx.x) = all;
      cluster.sync();
      all = 0;
#pragma unroll
      for (int r = 0; r < CTAS; ++r) {
        if (r < rank) below += totals[slot][r];
        all += totals[slot][r];
      }
    }
    __syncthreads();
    *total = all;
    return below;
  };

  int total;
  int ties = 0;  // keys of rank `last` before this warp's
  if (need < equal) {
    int count = 0;
    each([&](int, uint32_t u, bool in) {
      count += __popc(__ballot_sync(0xffffffffu, in && u == last));
    });
    ties = before_of(count, 0, &total);
  }
  const unsigned below_me = (1u << lane) - 1u;
  auto stays = [&](uint32_t u, bool in, int& tie) {
    const unsigned same = __ballot_sync(0xffffffffu, in && u == last);
    const bool yes = in && (u > last || (u == last && tie + __popc(same & below_me) < need));
    tie += __popc(same);
    return yes;
  };

  // ------------------------------------------------- holes, movers and lists
  int holes = 0, movers = 0, tie = ties;
  each([&](int t, uint32_t u, bool in) {
    const bool yes = stays(u, in, tie);
    holes += __popc(__ballot_sync(0xffffffffu, in && t < n && !yes));
    movers += __popc(__ballot_sync(0xffffffffu, t >= n && yes));
  });
  int moves;
  int hole = before_of(holes, 1, &moves);
  int mover = before_of(movers, 2, &moves);
  const size_t list = static_cast<size_t>(seg) * a.max_moves;
  if (rank == 0 && threadIdx.x == 0) a.counts[seg] = moves;
  tie = ties;
  each([&](int t, uint32_t u, bool in) {
    const bool yes = stays(u, in, tie);
    const unsigned hm = __ballot_sync(0xffffffffu, in && t < n && !yes);
    const unsigned mm = __ballot_sync(0xffffffffu, t >= n && yes);
    if (in) {
      if (t < n && !yes) {
        a.move_dst[list + hole + __popc(hm & below_me)] = t;
      } else {
        const float m = mass[t];
        const int p = position(t, pos[t]);
        if (t < n) {
          new_mass[t] = m;
          new_pos[t] = p;
        } else {
          if (yes) {  // the highest goes into the lowest hole
            const size_t at = list + (moves - 1 - (mover + __popc(mm & below_me)));
            a.move_src[at] = t;
            a.move_mass[at] = m;
            a.move_pos[at] = p;
          }
          new_mass[t] = 0.f;
          new_pos[t] = -1;
        }
      }
    }
    hole += __popc(hm);
    mover += __popc(mm);
  });
  if constexpr (CTAS > 1) cluster.sync();  // the others may still read this CTA's counts
}

// One warp per 8 moves of a segment: their K and V rows, all loads in flight
// before the stores (sources and destinations are disjoint), and their masses
// and positions.  `layers` segments' pools are in this launch.
constexpr int kMoveBatch = 8;

template <int D>
__global__ void __launch_bounds__(256) evict_move_kernel(const __grid_constant__ EvictMoveArgs m) {
  launch_dependents();
  wait_predecessor();
  const EvictArgs& a = m.a;
  const int lane = threadIdx.x & 31;
  const long long gthread = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (m.first_layer == 0)
    for (long long b = gthread; b < a.batch; b += static_cast<long long>(gridDim.x) * blockDim.x)
      a.new_seq_lens[b] = a.kept[b];
  const int per_seg = (a.max_moves + kMoveBatch - 1) / kMoveBatch;
  const long long units = static_cast<long long>(m.layers) * a.batch * a.Hkv * per_seg;
  const long long stride = static_cast<long long>(gridDim.x) * (blockDim.x / 32);
  constexpr int kRow = D * 2;                 // bytes of a row
  constexpr int kSteps = 2 * kRow / 512;      // warp-wide copies per move: K's row, then V's
  for (long long u = gthread / 32; u < units; u += stride) {
    const int seg = static_cast<int>(u / per_seg);
    const int at = static_cast<int>(u - static_cast<long long>(seg) * per_seg) * kMoveBatch;
    const size_t gseg = static_cast<size_t>(m.first_layer) * a.batch * a.Hkv + seg;
    const int count = min(kMoveBatch, a.counts[gseg] - at);
    if (count <= 0) continue;
    const int layer = seg / (a.batch * a.Hkv);
    const int b = seg / a.Hkv % a.batch, head = seg % a.Hkv;
    const size_t list = gseg * a.max_moves + at;
    // lanes 0..7: sources, 8..15: destinations, as rows of the pools
    long long row = -1;
    if (lane < 2 * kMoveBatch && (lane & 7) < count) {
      const int t = lane < kMoveBatch ? a.move_src[list + lane] : a.move_dst[list + (lane & 7)];
      const int id = a.tables[static_cast<size_t>(b) * a.max_blocks + t / kBlockSize];
      if (static_cast<unsigned>(id) < static_cast<unsigned>(a.num_blocks))
        row = (static_cast<long long>(id) * a.Hkv + head) * kBlockSize + t % kBlockSize;
      else
        report(a.err, PKA_DEVERR_BAD_TABLE);
      if (lane >= kMoveBatch) {
        const size_t key = gseg * (static_cast<size_t>(a.max_blocks) * kBlockSize) + t;
        a.new_mass[key] = a.move_mass[list + (lane & 7)];
        a.new_pos[key] = a.move_pos[list + (lane & 7)];
      }
    }
    uint4 x[kMoveBatch][kSteps];
#pragma unroll
    for (int i = 0; i < kMoveBatch; ++i) {
      const long long src = __shfl_sync(0xffffffffu, row, i);
      if (src < 0) continue;  // uniform
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int off = s * 512 + lane * 16;  // over K's row and V's
        const uint8_t* pool = static_cast<const uint8_t*>(m.pools[2 * layer + off / kRow]);
        x[i][s] = *reinterpret_cast<const uint4*>(pool + src * kRow + off % kRow);
      }
    }
#pragma unroll
    for (int i = 0; i < kMoveBatch; ++i) {
      const long long src = __shfl_sync(0xffffffffu, row, i);
      const long long dst = __shfl_sync(0xffffffffu, row, kMoveBatch + i);
      if (src < 0 || dst < 0) continue;  // uniform
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int off = s * 512 + lane * 16;
        uint8_t* pool = static_cast<uint8_t*>(m.pools[2 * layer + off / kRow]);
        *reinterpret_cast<uint4*>(pool + dst * kRow + off % kRow) = x[i][s];
      }
    }
  }
}

}  // namespace

cudaError_t launch_evict_select(const EvictArgs& a, int layers, cudaStream_t stream) {
  const long long segs = static_cast<long long>(layers) * a.batch * a.Hkv;
  const long long keys = static_cast<long long>(a.max_blocks) * kBlockSize;
  constexpr long long kOne = kSelThreads * kKeep;  // keys that one CTA keeps in registers
  if (keys <= kOne)
    return launch_overlapped(evict_select_kernel<1>, dim3(static_cast<unsigned>(segs)),
                             kSelThreads, 0, stream, a);
  if (keys <= 2 * kOne)
    return launch_overlapped(evict_select_kernel<2>, dim3(static_cast<unsigned>(2 * segs)),
                             kSelThreads, 0, stream, a, 2);
  if (keys <= 4 * kOne)
    return launch_overlapped(evict_select_kernel<4>, dim3(static_cast<unsigned>(4 * segs)),
                             kSelThreads, 0, stream, a, 4);
  return launch_overlapped(evict_select_kernel<8>, dim3(static_cast<unsigned>(8 * segs)),
                           kSelThreads, 0, stream, a, 8);
}

cudaError_t launch_evict_move(const EvictMoveArgs& m, int head_dim, int sm_count,
                              cudaStream_t stream) {
  const long long per_seg = (m.a.max_moves + kMoveBatch - 1) / kMoveBatch;
  const long long warps = static_cast<long long>(m.layers) * m.a.batch * m.a.Hkv * per_seg;
  long long grid = (warps + 7) / 8;
  const long long most = static_cast<long long>(sm_count > 0 ? sm_count : 1) * 16;
  grid = grid < 1 ? 1 : grid < most ? grid : most;
  return head_dim == 256 ? launch_overlapped(evict_move_kernel<256>,
                                             dim3(static_cast<unsigned>(grid)), 256, 0, stream, m)
                         : launch_overlapped(evict_move_kernel<128>,
                                             dim3(static_cast<unsigned>(grid)), 256, 0, stream, m);
}

}  // namespace pka
