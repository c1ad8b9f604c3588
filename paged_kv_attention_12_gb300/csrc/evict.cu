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
// Two launches: the selection (a CTA or cluster per segment: reads 8 bytes a
// key, writes the list of moves), then the moves over all segments (bound by HBM).
// Few moves are made by the selection itself.
// 128 segments of 700 to 4096 keys (two layers, D = 256) cut to 1000: selection
// 11 us, moves 28 us, 5.1 TB/s in rows of 512 bytes.
#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"
#include "overlap.cuh"

namespace cg = cooperative_groups;

namespace pka {

namespace {

constexpr int kSelWarps = 32;
constexpr int kSelThreads = kSelWarps * 32;
constexpr int kGroup = 4;                 // neighbouring keys that a lane takes at once
// The n-th largest rank is found digit by digit, 8 bits from the top.  A lane
// counts in a copy of the histogram of its own (bank = lane): masses share few
// exponents and held keys one rank, and in a single copy the lanes of a warp
// wait for one another.
constexpr int kDigits = 4, kBins = 256;
constexpr int kCtaKeys = kEvictCtaKeys;   // keys of a CTA of a cluster, at most (8 CTAs: more)

constexpr uint32_t kHeld = 0xffffffffu;   // above every mass

// Masses in their order as unsigned numbers; NaN below all of them.
__device__ __forceinline__ uint32_t rank_of(float mass) {
  if (isnan(mass)) return 0;
  const uint32_t x = __float_as_uint(mass == 0.f ? 0.f : mass);
  return x & 0x80000000u ? ~x : x | 0x80000000u;
}

// One warp per 4 moves of a segment: their K and V rows, all loads in flight
// before the stores (sources and destinations are disjoint), and their masses
// and positions (8 moves a warp: 55 us for the call of above instead of 40, at 100
// registers; 2 moves: 43; streaming hints on the loads or the stores: 42).
constexpr int kMoveBatch = 4;

template <int D>
__device__ __forceinline__ void move_batch(const EvictMoveArgs& m, int seg, int at, int lane) {
  const EvictArgs& a = m.a;
  constexpr int kRow = D * 2;                 // bytes of a row
  constexpr int kSteps = 2 * kRow / 512;      // warp-wide copies per move: K's row, then V's
  const size_t gseg = static_cast<size_t>(m.first_layer) * a.batch * a.Hkv + seg;
  const size_t list = gseg * a.max_moves + at;
  // the first lanes: the sources' rows, then the destinations' (the list may be
  // read past its end: it lies in the workspace)
  const int i = lane & (kMoveBatch - 1);
  const bool listed = lane < 2 * kMoveBatch && at + i < a.max_moves;
  int t = -1;
  if (listed) t = lane < kMoveBatch ? a.move_src[list + i] : a.move_dst[list + i];
  const int count = min(kMoveBatch, a.counts[gseg] - at);
  if (count <= 0) return;
  const int layer = seg / (a.batch * a.Hkv);
  const int b = seg / a.Hkv % a.batch, head = seg % a.Hkv;
  int row = i < count ? t : -1;
  if (lane >= kMoveBatch && listed && i < count) {
    const int id = a.tables[static_cast<size_t>(b) * a.max_blocks + t / kBlockSize];
    if (static_cast<unsigned>(id) < static_cast<unsigned>(a.num_blocks)) {
      row = (id * a.Hkv + head) * kBlockSize + t % kBlockSize;
    } else {
      row = -1;
      report(a.err, PKA_DEVERR_BAD_TABLE);
    }
    const size_t key = gseg * (static_cast<size_t>(a.max_blocks) * kBlockSize) + t;
    a.new_mass[key] = a.move_mass[list + i];
    a.new_pos[key] = a.move_pos[list + i];
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

// Ranks of the CTA's keys lie in shared memory (those past a.rank_room are made
// again from mass and position where they are wanted), and every pass over them
// is a short loop: with the ranks in registers the passes were unrolled, and a
// launch fetches its instructions anew (two rows of 411 keys 13.3 us, now 8.9).
// What bounds it: latency for short rows (four digits at 0.6 us, 2.3 with a
// cluster's exchange, and the passes before and after them), issue for long ones.
template <int CTAS>
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(
    const __grid_constant__ EvictMoveArgs job) {
  const EvictArgs& a = job.a;
  extern __shared__ int hist[];          // [kBins][32], then the ranks
  __shared__ int digit[kDigits][kBins];  // read by the other CTAs of the cluster,
  __shared__ int totals[3][CTAS];        // written by them
  __shared__ int sums[kBins];
  __shared__ int warp_sum[kSelWarps];
  __shared__ int found[3];
  __shared__ int shared_block;
  uint32_t* ranks = reinterpret_cast<uint32_t*>(hist + kBins * 32);
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = CTAS > 1 ? static_cast<int>(cluster.block_rank()) : 0;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
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
  const int32_t* table = a.tables + static_cast<size_t>(b) * a.max_blocks;
  if (a.refcounts != nullptr && n < L) {
    // a block that would be written and that another request reads too
    __syncthreads();
    bool shared = false;
    for (int j = threadIdx.x; j < (n + kBlockSize - 1) / kBlockSize; j += kSelThreads) {
      const int id = table[j];
      if (static_cast<unsigned>(id) < static_cast<unsigned>(a.num_blocks))
        shared = shared || a.refcounts[id] > 1;
    }
    if (shared) shared_block = 1;
    __syncthreads();
    if (shared_block != 0) n = L;  // (the same in every CTA: all of them look at the whole row)
  }
  if (teller) {
    a.kept[b] = n;
    if (job.here) a.new_seq_lens[b] = n;
  }
  if (rank == 0 && threadIdx.x == 0 && n == L) a.counts[seg] = 0;

  const size_t first = static_cast<size_t>(seg) * max_keys;
  const float* mass = a.mass + first;
  const int32_t* pos = a.pos + first;
  float* new_mass = a.new_mass + first;
  int32_t* new_pos = a.new_pos + first;
  // keys without a position are the latest ones, in order
  auto position = [&](int t, int p) { return p >= 0 ? p : T - (L - t); };
  auto rank_at = [&](float m, int at) {
    return at < a.sinks || at >= T - a.recent ? kHeld : rank_of(m);
  };

  // this warp's keys [lo, hi): a run of its own
  const int per_warp = ((L + CTAS * kSelWarps - 1) / (CTAS * kSelWarps) + 31) / 32 * 32;
  const int cta_lo = static_cast<int>(
      min(static_cast<long long>(rank) * kSelWarps * per_warp, static_cast<long long>(L)));
  const int lo = static_cast<int>(
      min(static_cast<long long>(rank * kSelWarps + warp) * per_warp, static_cast<long long>(L)));
  const int hi = min(lo + per_warp, L);
  // f(t): the lane's keys t .. t + 3 (t < hi; a row is a multiple of 16 keys, so
  // all four can be read).  Every lane of the warp makes every step.
  auto each = [&](auto f) {
#pragma unroll 1
    for (int g = lo; g < hi; g += 32 * kGroup) f(g + kGroup * lane);
  };
  auto load = [&](int t, float* m, int* p) {
    const float4 x = *reinterpret_cast<const float4*>(mass + t);
    const int4 y = *reinterpret_cast<const int4*>(pos + t);
    m[0] = x.x, m[1] = x.y, m[2] = x.z, m[3] = x.w;
    p[0] = position(t, y.x), p[1] = position(t + 1, y.y);
    p[2] = position(t + 2, y.z), p[3] = position(t + 3, y.w);
  };
  auto store = [&](int t, const float* m, const int* p) {
    *reinterpret_cast<float4*>(new_mass + t) = make_float4(m[0], m[1], m[2], m[3]);
    *reinterpret_cast<int4*>(new_pos + t) = make_int4(p[0], p[1], p[2], p[3]);
  };
  if (n == L) {
    each([&](int t) {
      if (t >= hi) return;
      float m[kGroup];
      int p[kGroup];
      load(t, m, p);
      if (t + kGroup <= hi) {
        store(t, m, p);
      } else {
#pragma unroll
        for (int k = 0; k < kGroup; ++k)
          if (t + k < hi) {
            new_mass[t + k] = m[k];
            new_pos[t + k] = p[k];
          }
      }
    });
    return;  // the whole cluster
  }
  // the four keys' ranks; keys past the warp's end: 0
  auto ranks_of = [&](int t, uint32_t* u) {
    if (t >= hi) {
#pragma unroll
      for (int k = 0; k < kGroup; ++k) u[k] = 0;
      return;
    }
    if (t - cta_lo < a.rank_room) {
      const uint4 x = *reinterpret_cast<const uint4*>(ranks + (t - cta_lo));
      u[0] = x.x, u[1] = x.y, u[2] = x.z, u[3] = x.w;
      return;
    }
    float m[kGroup];
    int p[kGroup];
    load(t, m, p);
#pragma unroll
    for (int k = 0; k < kGroup; ++k) u[k] = t + k < hi ? rank_at(m[k], p[k]) : 0;
  };

  // ---------------------------------------- the rank of the last key that stays
  uint32_t prefix = 0;
  int need = n, equal = 0;  // keys still to find among those with this prefix
#pragma unroll 1
  for (int pass = 0; pass < kDigits; ++pass) {
    const int shift = 24 - 8 * pass;
    for (int i = threadIdx.x; i < kBins * 8; i += kSelThreads)
      reinterpret_cast<int4*>(hist)[i] = make_int4(0, 0, 0, 0);
    __syncthreads();
    if (pass == 0) {
      each([&](int t) {
        if (t >= hi) return;
        float m[kGroup];
        int p[kGroup];
        uint32_t u[kGroup];
        load(t, m, p);
#pragma unroll
        for (int k = 0; k < kGroup; ++k) {
          u[k] = t + k < hi ? rank_at(m[k], p[k]) : 0;
          if (t + k < hi) atomicAdd(&hist[(u[k] >> 24) * 32 + lane], 1);
        }
        if (t - cta_lo < a.rank_room)
          *reinterpret_cast<uint4*>(ranks + (t - cta_lo)) = make_uint4(u[0], u[1], u[2], u[3]);
      });
    } else {
      each([&](int t) {
        uint32_t u[kGroup];
        ranks_of(t, u);
#pragma unroll
        for (int k = 0; k < kGroup; ++k)
          if (t + k < hi && u[k] >> (shift + 8) == prefix)
            atomicAdd(&hist[(u[k] >> shift & 255) * 32 + lane], 1);
      });
    }
    __syncthreads();
    for (int bin = warp; bin < kBins; bin += kSelWarps) {
      const int c = __reduce_add_sync(0xffffffffu, hist[bin * 32 + lane]);
      if (lane == 0) digit[pass][bin] = c;
    }
    const int* all = digit[pass];
    if constexpr (CTAS > 1) {
      cluster.sync();
      if (threadIdx.x < kBins) {
        int c = 0;
#pragma unroll
        for (int r = 0; r < CTAS; ++r)
          c += *cluster.map_shared_rank(&digit[pass][threadIdx.x], r);
        sums[threadIdx.x] = c;
      }
      all = sums;
    }
    __syncthreads();
    if (warp == 0) {  // bins from the top, eight a lane
      int c[8], mine = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        c[e] = all[kBins - 1 - (lane * 8 + e)];
        mine += c[e];
      }
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      int above = incl - mine;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (above < need && need <= above + c[e]) {  // exactly one bin
          found[0] = kBins - 1 - (lane * 8 + e);
          found[1] = need - above;
          found[2] = c[e];
        }
        above += c[e];
      }
    }
    __syncthreads();
    prefix = prefix << 8 | static_cast<uint32_t>(found[0]);
    need = found[1];
    equal = found[2];
  }
  const uint32_t last = prefix;

  // exclusive count over the cluster's warps in key order; slot: which of the
  // exchanges this is
  auto before_of = [&](int count, int slot, int* total) {
    if (lane == 0) warp_sum[warp] = count;
    __syncthreads();
    const int v = lane < kSelWarps ? warp_sum[lane] : 0;
    int below = __reduce_add_sync(0xffffffffu, lane < warp ? v : 0);
    int all = __reduce_add_sync(0xffffffffu, v);
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

  // keys of rank `last`: all of them stay, or the first `need`
  const bool some = need < equal;
  int total;
  int tie = 0;  // those before this warp's
  if (some) {
    int count = 0;
    each([&](int t) {
      uint32_t u[kGroup];
      ranks_of(t, u);
#pragma unroll
      for (int k = 0; k < kGroup; ++k) count += t + k < hi && u[k] == last;
    });
    tie = before_of(__reduce_add_sync(0xffffffffu, count), 0, &total);
  }
  const unsigned below_me = (1u << lane) - 1u;
  // in: a property of the four keys; of all keys before the lane's in the step,
  // how many have it (all: in the step)
  auto before_lane = [&](const bool* in, int* all) {
    int below = 0;
    *all = 0;
#pragma unroll
    for (int k = 0; k < kGroup; ++k) {
      const unsigned m = __ballot_sync(0xffffffffu, in[k]);
      below += __popc(m & below_me);
      *all += __popc(m);
    }
    return below;
  };
  auto stays = [&](int t, const uint32_t* u, bool* yes, int& tie) {
    if (!some) {
#pragma unroll
      for (int k = 0; k < kGroup; ++k) yes[k] = t + k < hi && u[k] >= last;
      return;
    }
    bool same[kGroup];
#pragma unroll
    for (int k = 0; k < kGroup; ++k) same[k] = t + k < hi && u[k] == last;
    int all;
    int at = tie + before_lane(same, &all);
#pragma unroll
    for (int k = 0; k < kGroup; ++k) {
      yes[k] = t + k < hi && (u[k] > last || (same[k] && at < need));
      at += same[k];
    }
    tie += all;
  };

  // ------------------------------------------------- holes, movers and lists
  int holes = 0, movers = 0, tie_now = tie;
  each([&](int t) {
    uint32_t u[kGroup];
    bool yes[kGroup];
    ranks_of(t, u);
    stays(t, u, yes, tie_now);
#pragma unroll
    for (int k = 0; k < kGroup; ++k) {
      holes += t + k < hi && t + k < n && !yes[k];
      movers += t + k >= n && yes[k];
    }
  });
  int moves;
  int hole = before_of(__reduce_add_sync(0xffffffffu, holes), 1, &moves);
  int mover = before_of(__reduce_add_sync(0xffffffffu, movers), 2, &moves);
  const size_t list = static_cast<size_t>(seg) * a.max_moves;
  if (rank == 0 && threadIdx.x == 0) a.counts[seg] = moves;
  each([&](int t) {
    uint32_t u[kGroup];
    bool yes[kGroup], is_hole[kGroup], is_mover[kGroup];
    ranks_of(t, u);
    stays(t, u, yes, tie);
    bool any = false, all_stay = true;
#pragma unroll
    for (int k = 0; k < kGroup; ++k) {
      is_hole[k] = t + k < hi && t + k < n && !yes[k];
      is_mover[k] = t + k >= n && yes[k];
      any = any || yes[k];
      all_stay = all_stay && yes[k] && t + k < n;
    }
    float m[kGroup] = {0.f, 0.f, 0.f, 0.f};
    int p[kGroup] = {-1, -1, -1, -1};
    if (any) load(t, m, p);
    const int step = t - kGroup * lane;  // the warp's first key: holes lie below n, movers above
    if (step < n) {
      int all;
      int h = hole + before_lane(is_hole, &all);
#pragma unroll
      for (int k = 0; k < kGroup; ++k) {
        if (is_hole[k]) a.move_dst[list + h] = t + k;
        h += is_hole[k];
      }
      hole += all;
    }
    if (step + 32 * kGroup > n) {
      const int id = any ? table[t / kBlockSize] : 0;  // (of all four)
      int all;
      int v = mover + before_lane(is_mover, &all);
#pragma unroll
      for (int k = 0; k < kGroup; ++k) {
        if (is_mover[k]) {  // the highest goes into the lowest hole
          const size_t to = list + (moves - 1 - v);
          // its row in the pools (counted in 32 bits), -1: a bad id
          int row = -1;
          if (static_cast<unsigned>(id) < static_cast<unsigned>(a.num_blocks))
            row = (id * a.Hkv + seg % a.Hkv) * kBlockSize + (t + k) % kBlockSize;
          else
            report(a.err, PKA_DEVERR_BAD_TABLE);
          a.move_src[to] = row;
          a.move_mass[to] = m[k];
          a.move_pos[to] = p[k];
        }
        v += is_mover[k];
      }
      mover += all;
    }
    if (t >= hi) return;
    if (t >= n) {
#pragma unroll
      for (int k = 0; k < kGroup; ++k) {
        m[k] = 0.f;
        p[k] = -1;
      }
    }
    if (t + kGroup <= hi && (t >= n || all_stay)) {
      store(t, m, p);
    } else {
#pragma unroll
      for (int k = 0; k < kGroup; ++k) {
        if (t + k >= hi || is_hole[k]) continue;
        new_mass[t + k] = t + k < n ? m[k] : 0.f;
        new_pos[t + k] = t + k < n ? p[k] : -1;
      }
    }
  });
  if constexpr (CTAS > 1) {
    cluster.sync();  // the others may still read this CTA's counts
  } else if (job.here) {
    __syncthreads();
#pragma unroll 1
    for (int at = warp * kMoveBatch; at < moves; at += kSelWarps * kMoveBatch) {
      if (job.here == 256)
        move_batch<256>(job, seg, at, lane);
      else
        move_batch<128>(job, seg, at, lane);
    }
  }
}

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
  for (long long u = gthread / 32; u < units; u += stride) {
    const int seg = static_cast<int>(u / per_seg);
    move_batch<D>(m, seg, static_cast<int>(u - static_cast<long long>(seg) * per_seg) * kMoveBatch,
                  lane);
  }
}

}  // namespace

// Rows of up to 16384 keys take a CTA, longer ones a cluster of two, four or eight
// (16 rows of up to 131072 keys, selection alone: of eight 41 us, although one of
// the clusters has to wait for the others, of four 47).
cudaError_t launch_evict_select(const EvictMoveArgs& args, int layers, cudaStream_t stream) {
  EvictMoveArgs m = args;
  EvictArgs& a = m.a;
  const long long segs = static_cast<long long>(layers) * a.batch * a.Hkv;
  const long long keys = static_cast<long long>(a.max_blocks) * kBlockSize;
  auto launch = [&](auto kernel, int ctas) {
    const long long mine = ((keys + ctas * kSelWarps - 1) / (ctas * kSelWarps) + 31) / 32 * 32 *
                           kSelWarps;
    a.rank_room = static_cast<int32_t>(mine < kCtaKeys ? mine : kCtaKeys);
    const int bytes = (kBins * 32 + a.rank_room) * static_cast<int>(sizeof(int));
    const cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kernel),
                                        (kBins * 32 + kCtaKeys) * static_cast<int>(sizeof(int)));
    if (e != cudaSuccess) return e;
    return launch_overlapped(kernel, dim3(static_cast<unsigned>(ctas * segs)), kSelThreads, bytes,
                             stream, m, ctas);
  };
  if (keys <= kCtaKeys) return launch(evict_select_kernel<1>, 1);
  if (keys <= 2 * kCtaKeys) return launch(evict_select_kernel<2>, 2);
  if (keys <= 4 * kCtaKeys) return launch(evict_select_kernel<4>, 4);
  return launch(evict_select_kernel<8>, 8);
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
