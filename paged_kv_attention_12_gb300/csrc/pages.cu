// Pages of a cache: reference counts, copies of blocks and compaction
// (sm_103a).  The kernels see a block as bytes, so they serve bf16 and 4-bit
// pools alike.
#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"
#include "overlap.cuh"

namespace cg = cooperative_groups;

namespace pka {

namespace {

// ------------------------------------------------------------ block copies
constexpr int kCopyUnroll = 4;
constexpr int kCopyChunk = 32 * 16 * kCopyUnroll;  // bytes a warp copies per item

// One warp per (pair, pool, 2 KB chunk of the block), the chunk's loads in
// flight together.  The pairs come from src / dst, or, for a compaction, from
// its list of moves (whose length only the device knows).  Bound by HBM: 12000
// moves in four pools of 16 KB blocks, 1.57 GB, 240 us with 32 CTAs per SM
// (258 with 8: the hardware evens the SMs out), 6.5 TB/s, 96% of a plain copy.
__global__ void __launch_bounds__(256) copy_blocks_kernel(const __grid_constant__ CopyArgs a) {
  launch_dependents();
  wait_predecessor();
  const int lane = threadIdx.x & 31;
  const long long gthread = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  // the tables of a compaction: entries of a row's used part follow their
  // block; a free block's entry becomes -1
  if (a.tables != nullptr) {
    const long long entries = static_cast<long long>(a.batch) * a.max_blocks;
    for (long long i = gthread; i < entries; i += static_cast<long long>(gridDim.x) * blockDim.x) {
      const int b = static_cast<int>(i / a.max_blocks), j = static_cast<int>(i % a.max_blocks);
      int L = a.seq_lens[b];
      if (L < 0 || L > a.max_blocks * kBlockSize) {
        if (j == 0) report(a.err, PKA_DEVERR_SEQ_LEN);
        L = max(0, min(L, a.max_blocks * kBlockSize));
      }
      int id = a.tables[i];
      if (j < (L + kBlockSize - 1) / kBlockSize && id >= 0) {
        if (id >= a.num_blocks)
          report(a.err, PKA_DEVERR_BAD_TABLE);
        else
          id = a.remap[id];
      }
      a.new_tables[i] = id;
    }
  }
  const int n = a.moves != nullptr ? a.moves[0] : a.n;
  const int chunks = static_cast<int>((a.block_bytes + kCopyChunk - 1) / kCopyChunk);
  const long long items = static_cast<long long>(n) * a.num_pools * chunks;
  const long long wstride = static_cast<long long>(gridDim.x) * (blockDim.x / 32);
  for (long long w = gthread / 32; w < items; w += wstride) {
    const int c = static_cast<int>(w % chunks);
    const long long pp = w / chunks;
    const int pool = static_cast<int>(pp % a.num_pools);
    const int i = static_cast<int>(pp / a.num_pools);
    const int src = a.moves != nullptr ? a.moves[2 + 2 * i] : a.src[i];
    const int dst = a.moves != nullptr ? a.moves[3 + 2 * i] : a.dst[i];
    if (static_cast<unsigned>(src) >= static_cast<unsigned>(a.num_blocks) ||
        static_cast<unsigned>(dst) >= static_cast<unsigned>(a.num_blocks)) {
      if (lane == 0 && c == 0 && pool == 0) report(a.err, PKA_DEVERR_BAD_TABLE);
      continue;
    }
    if (src == dst) continue;
    const uint8_t* from = static_cast<const uint8_t*>(a.pools[pool]) + src * a.block_bytes;
    uint8_t* to = static_cast<uint8_t*>(a.pools[pool]) + dst * a.block_bytes;
    const long long base = static_cast<long long>(c) * kCopyChunk + lane * 16;
    uint4 x[kCopyUnroll];
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u)
      if (base + u * 512 < a.block_bytes)
        x[u] = *reinterpret_cast<const uint4*>(from + base + u * 512);
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u)
      if (base + u * 512 < a.block_bytes) *reinterpret_cast<uint4*>(to + base + u * 512) = x[u];
  }
}

// ------------------------------------------------------- reference counts
// One thread per table entry.  Integer atomics: the counts do not depend on
// their order.
__global__ void __launch_bounds__(256) ref_blocks_kernel(const RefArgs a) {
  launch_dependents();
  wait_predecessor();
  const long long entries = static_cast<long long>(a.batch) * a.max_blocks;
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < entries;
       i += static_cast<long long>(gridDim.x) * blockDim.x) {
    const int b = static_cast<int>(i / a.max_blocks), j = static_cast<int>(i % a.max_blocks);
    int L = a.seq_lens[b];
    if (L < 0 || L > a.max_blocks * kBlockSize) {
      if (j == 0) report(a.err, PKA_DEVERR_SEQ_LEN);
      L = max(0, min(L, a.max_blocks * kBlockSize));
    }
    if (j >= (L + kBlockSize - 1) / kBlockSize) continue;
    const int id = a.tables[i];
    if (id < 0) continue;  // no block here
    if (id >= a.num_blocks) {
      report(a.err, PKA_DEVERR_BAD_TABLE);
      continue;
    }
    const int old = atomicAdd(a.refcounts + id, a.delta);
    if (old + a.delta < 0) report(a.err, PKA_DEVERR_REFCOUNT);
  }
}

// -------------------------------------------------------- compaction plan
// With n live blocks (refcount > 0), the j-th highest live id at or above n
// moves to the j-th lowest free id below n: as many moves as there are holes,
// every source at or above n and every destination below it, so the copies
// cannot overlap.  A live id's place in that order is n - 1 - rank(id) and a
// hole's is id - rank(id), rank(id) the live ids below it: one prefix count
// gives both.
//
// One cluster of CTAS CTAs: the ids are cut into contiguous ranges, one per
// warp; each warp counts its live ids with ballots, the CTAs exchange their
// totals through distributed shared memory, and a second pass over the range
// (the first kKeep steps of it in registers) writes the lists.  Every id is
// read and written by its own warp only until the last phase, so
// new_refcounts may be refcounts.  One CTA does without the cluster's barriers
// and is taken while its registers hold all the ids (one CTA / eight: 2048 ids
// 3.7 / 4.8 us, 65536 ids 42 / 8.2 us, a launch in a stream of them).
constexpr int kPlanWarps = 32;
constexpr int kKeep = 8;
constexpr int kPlanOne = kPlanWarps * 32 * kKeep;  // ids one CTA keeps in registers

template <int CTAS>
__global__ void __launch_bounds__(kPlanWarps * 32, 1) compact_plan_kernel(const PlanArgs a) {
  __shared__ int cta_total[CTAS];  // every CTA's live ids (written by each CTA everywhere)
  __shared__ int warp_total[kPlanWarps];
  __shared__ int moves_total;      // CTA 0's is the cluster's
  cg::cluster_group cluster = cg::this_cluster();
  auto sync = [&]() {
    if constexpr (CTAS > 1)
      cluster.sync();
    else
      __syncthreads();
  };
  auto of = [&](int* p, int rank) {
    if constexpr (CTAS > 1)
      return cluster.map_shared_rank(p, rank);
    else
      return p;
  };
  const int rank = CTAS > 1 ? static_cast<int>(cluster.block_rank()) : 0;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int per_warp =
      ((a.num_blocks + CTAS * kPlanWarps - 1) / (CTAS * kPlanWarps) + 31) / 32 * 32;
  const long long first = static_cast<long long>(rank * kPlanWarps + warp) * per_warp;
  const int lo = static_cast<int>(min(first, static_cast<long long>(a.num_blocks)));
  const int hi = static_cast<int>(min(first + per_warp, static_cast<long long>(a.num_blocks)));
  launch_dependents();
  wait_predecessor();
  if (threadIdx.x == 0) moves_total = 0;

  // a CTA's shared memory may be written by the others once it has started:
  // arrive now, wait before the first such write
  if constexpr (CTAS > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  // the first kKeep steps' counts stay in registers for the second pass
  int ref[kKeep];
  int count = 0;
#pragma unroll
  for (int k = 0; k < kKeep; ++k) {
    const int i = lo + 32 * k + lane;
    ref[k] = i < hi ? a.refcounts[i] : 0;
  }
#pragma unroll
  for (int k = 0; k < kKeep; ++k) count += __popc(__ballot_sync(0xffffffffu, ref[k] > 0));
#pragma unroll 8
  for (int base = lo + 32 * kKeep; base < hi; base += 32) {
    const int i = base + lane;
    count += __popc(__ballot_sync(0xffffffffu, i < hi && a.refcounts[i] > 0));
  }
  if (lane == 0) warp_total[warp] = count;
  __syncthreads();
  if constexpr (CTAS > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (warp == 0) {
    const int v = warp_total[lane];
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    warp_total[lane] = incl - v;
    const int all = __shfl_sync(0xffffffffu, incl, 31);
    // lane r stores this CTA's total into CTA r's array
    if (lane < CTAS) *of(&cta_total[rank], lane) = all;
  }
  sync();
  int live = 0, below = 0;
#pragma unroll
  for (int r = 0; r < CTAS; ++r) {
    if (r < rank) below += cta_total[r];
    live += cta_total[r];
  }
  below += warp_total[warp];

  int movers = 0;
  auto place = [&](int i, int r) {  // r: the refcount of id i, 0 past the end
    const unsigned m = __ballot_sync(0xffffffffu, r > 0);
    const int at = below + __popc(m & ((1u << lane) - 1u));  // live ids below i
    below += __popc(m);
    if (i < hi) {
      if (r > 0 && i < live) {
        a.remap[i] = i;
        a.new_refcounts[i] = r;
      } else if (r > 0) {
        a.moves[2 + 2 * (live - 1 - at)] = i;
      } else {
        a.remap[i] = -1;
        if (i < live)
          a.moves[3 + 2 * (i - at)] = i;
        else
          a.new_refcounts[i] = 0;
      }
    }
    movers += __popc(__ballot_sync(0xffffffffu, r > 0 && i >= live));
  };
#pragma unroll
  for (int k = 0; k < kKeep; ++k)
    if (lo + 32 * k < hi) place(lo + 32 * k + lane, ref[k]);
  for (int base = lo + 32 * kKeep; base < hi; base += 32) {
    const int i = base + lane;
    place(i, i < hi ? a.refcounts[i] : 0);
  }
  if (lane == 0 && movers > 0) atomicAdd(of(&moves_total, 0), movers);
  sync();  // the lists and the count are complete
  const int n = *of(&moves_total, 0);
  const int tid = rank * kPlanWarps * 32 + threadIdx.x;
  for (int j = tid; j < n; j += CTAS * kPlanWarps * 32) {
    const int src = a.moves[2 + 2 * j], dst = a.moves[3 + 2 * j];
    a.remap[src] = dst;
    a.new_refcounts[dst] = a.refcounts[src];
    a.new_refcounts[src] = 0;
  }
  for (int i = 2 + 2 * n + tid; i < 2 + a.num_blocks; i += CTAS * kPlanWarps * 32)
    a.moves[i] = -1;
  if (tid == 0) {
    a.moves[0] = n;
    a.moves[1] = live;
  }
  if constexpr (CTAS > 1)
    cluster.sync();  // CTA 0's shared memory stays until every CTA has read the count
}

int copy_grid(long long warps, int sm_count) {
  const long long want = (warps + 7) / 8;
  const long long cap = static_cast<long long>(sm_count > 0 ? sm_count : 1) * 32;
  return static_cast<int>(want < 1 ? 1 : (want < cap ? want : cap));
}

}  // namespace

cudaError_t launch_copy_blocks(const CopyArgs& a, int max_pairs, int sm_count,
                               cudaStream_t stream) {
  const long long chunks = (a.block_bytes + kCopyChunk - 1) / kCopyChunk;
  long long warps = max_pairs * chunks * a.num_pools;
  if (a.tables != nullptr) {
    const long long tw = (static_cast<long long>(a.batch) * a.max_blocks + 31) / 32;
    if (tw > warps) warps = tw;
  }
  return launch_overlapped(copy_blocks_kernel, copy_grid(warps, sm_count), 256, 0, stream, a);
}

cudaError_t launch_ref_blocks(const RefArgs& a, int sm_count, cudaStream_t stream) {
  const long long entries = static_cast<long long>(a.batch) * a.max_blocks;
  return launch_overlapped(ref_blocks_kernel, copy_grid((entries + 31) / 32, sm_count), 256, 0,
                           stream, a);
}

cudaError_t launch_compact_plan(const PlanArgs& a, cudaStream_t stream) {
  constexpr int kCtas = 8;
  return a.num_blocks <= kPlanOne
             ? launch_overlapped(compact_plan_kernel<1>, 1, kPlanWarps * 32, 0, stream, a)
             : launch_overlapped(compact_plan_kernel<kCtas>, kCtas, kPlanWarps * 32, 0, stream, a,
                                 kCtas);
}

}  // namespace pka
