// Attention of drafted tokens that form a tree over a block-paged cache
// (sm_103a): tcgen05 + TMEM + TMA.
//
// A step of speculative decoding verifies n <= 64 drafted tokens per request.
// Each of them sees the whole cached prefix and, of the drafted tokens, those
// of its mask (itself and its ancestors in the tree).  Every key is read once
// for all n tokens and all G heads of its KV head: n * G rows per 2 * 2 D
// bytes, so HBM bounds the operator up to a few hundred rows.
//
// A row tile packs QR / G tokens x G heads (row = token * G + head) into the
// rows of a 128-row MMA; QR = 64 leaves the room of the upper 64 rows of Q to
// the key stages (the MMA reads them from what follows in shared memory; a
// row's garbage stays in its row).  Work partition: a segment is one (request,
// KV head, row tile) with nb visible blocks; on a line of work units it takes
// kPieceUnits (a piece's fixed cost) and then one unit per block.  The line is
// cut into equal chunks, one per CTA, one CTA per SM.  A segment inside a
// chunk writes its output; the pieces of a cut one leave softmax-normalised
// fp32 rows and their log-sum-exp in the workspace, which the second launch
// merges in key order.  Segments that are no longer than a chunk and what a merge
// costs stay whole, one per CTA, or, where there are two CTAs for each segment,
// half of the tiles for each CTA of a cluster of two: each sends the other half of
// its rows' columns into the other's shared memory and finishes the rest, which
// takes about 2 us instead of the 7 of pieces and merge.
//
// Warps of a CTA: four softmax warps (a row of S and O lies in a TMEM lane; a thread
// owns a row, or with QR = 64 half of its columns), one TMA warp each for K, V and
// Q, and one that issues the MMAs.  The rings of K and V run on over the pieces of a
// chunk, so that the loads do not stop for an epilogue.
//
// Where the time goes (a serving layer: 32 trees of 8 to 16 tokens over 512 to
// 4096 keys, 2 KV heads, D = 256; 154 MB, 38.8 us; global-timer stamps): 0.6 us to
// the chunk, 2 to the first copy, 2.5 to the first S, then 1.4 us for each tile of
// 64 keys, 7.0 TB/s over the SMs (softmax, 0.8 us with its stamps, and MMAs, 0.5, are
// hidden behind the loads), 2 after the last copy has landed, 1.3 for the pieces' rows, and 6 for
// the merge and its launch.  DRAM reads are the keys' bytes.  A sliding layer of
// them (512 keys each, 64 segments on 64 pairs): 17.1 us (19.3 with a CTA each),
// latency.  Four long requests (D = 128, 33 to 131 K keys, 672 MB): 114
// us, 5.9 TB/s.  64 tokens x 4 heads are two row tiles, which read their keys twice,
// the second time from L2: 44.3 us, 1.37 a tile, 7.3 TB/s out of L2.
//
// Measured and dropped: one pass over S with a reference that moves only when the
// weights' sum shows that it must (few instructions, which are cold in every launch:
// the first tile 0.7 us sooner, each later one 0.1 to 0.3 us later; serving 40.6,
// wide trees 45.9), the walk over the pieces out of line (42.0), L2's normal policy for
// K and V (42.4 against 38.9: partial rows leave L2 for HBM and their stores
// wait), a piece's fixed cost of 6 blocks instead of 10 (40.4, and sliding layers 24.5
// instead of 23.1), the pairs' code in the same kernel as the rest (39.1, wide trees
// 45.0).
#include <cuda.h>

#include "common.cuh"
#include "kernels.h"
#include "overlap.cuh"
#include "softmax_math.cuh"
#include "tcgen05.cuh"
#include "tmaps.cuh"

namespace pka {

namespace {

template <int D_, int QR_>
struct TreeShape {
  static constexpr int D = D_, QR = QR_;
  static constexpr int BN = (D == 256) ? 64 : 128;  // keys per key tile
  static constexpr int BPT = BN / kBlockSize;
  static constexpr int DC = D / 64;                 // 128-byte chunks of a row
  static constexpr int kQChunk = QR * 128;
  static constexpr int kQBytes = QR * D * 2;
  static constexpr int kBlockBytes = kBlockSize * D * 2;  // [2 groups][D / 64][8 rows][128 B]
  static constexpr int kStage = BN * D * 2;
  static constexpr int kGroup = DC * 1024;          // stride of the 8-row groups
  static constexpr int KST = 3;
  static constexpr int VST = (kQBytes <= 32768) ? 3 : 2;
  static constexpr int oQ = 0;
  static constexpr int oK = kQBytes;
  static constexpr int oV = oK + KST * kStage;
  static constexpr int oEnd = oV + VST * kStage;
  static constexpr int kSmemBytes = oEnd + 1024;    // slack to align the base to 1 KiB
  // Four softmax warps.  With 128 rows a thread owns a row.  With 64 two threads
  // share one, half of a tile's columns each, in the warps that reach the row's TMEM
  // lanes (warp w: lanes 32 (w % 4) ..): 0 and 4, 1 and 5.
  static constexpr int kSoftmaxWarps = 4;
  static constexpr int kSplit = 128 / QR;
  static constexpr int CN = BN / kSplit;            // columns of a thread
  static constexpr int kWarpK = kSplit == 2 ? 2 : 4, kWarpV = kWarpK + 1, kWarpMma = 6, kWarpQ = 7;
  static constexpr int kThreads = 8 * 32;
  static constexpr int kPieceUnits = kTreePieceUnits(D);
  // TMEM columns: S_j (fp32) in buffer j % 2 at (j % 2) * BN, O at 256, P_j
  // (bf16 pairs) in buffer j % 2 at kTmemP + (j % 2) * BN / 2.
  static constexpr uint32_t kTmemO = 256;
  static constexpr uint32_t kTmemP = (D == 256) ? 2 * BN : 256 + D;
  static constexpr uint32_t kTmemCols = 512;
  static_assert(kTmemP >= 2 * BN && (kTmemP + BN <= kTmemO || kTmemP >= kTmemO + D) &&
                    kTmemP + BN <= kTmemCols && kTmemO + D <= kTmemCols,
                "P buffers clear of S and O");
  static_assert(kSmemBytes + 1536 <= 232448, "shared memory, the static part included");
};

struct TreeLaunch {
  CUtensorMap tm_q, tm_k, tm_v;
  TreeArgs a;
  int32_t q_tokens;   // tokens of a Q box
  int32_t log2_g;
};

// A request as the kernels take it: n query rows from q0 on, L keys (clamped
// to the table); n = 0: nothing to do.
struct Request {
  int n, q0, L;
};

__device__ __forceinline__ Request request_of(const TreeArgs& a, int b, bool tell) {
  Request r;
  r.q0 = a.query_start_loc[b];
  const int hi = a.query_start_loc[b + 1];
  r.L = a.seq_lens[b];
  r.n = 0;
  if (r.q0 < 0 || hi < r.q0 || hi > a.total_q || hi - r.q0 > a.max_query_len) {
    if (tell) report(a.err, PKA_DEVERR_QUERY_LOC);
    return r;
  }
  if (r.L > a.max_blocks * kBlockSize) {
    if (tell) report(a.err, PKA_DEVERR_SEQ_LEN);
    r.L = a.max_blocks * kBlockSize;
  }
  if (hi - r.q0 > r.L) {
    if (tell) report(a.err, PKA_DEVERR_SEQ_LEN);
    return r;
  }
  r.n = hi - r.q0;
  return r;
}

// First block that a query of the request sees (a query's position is at
// least L - n).
__device__ __forceinline__ int first_block(const TreeArgs& a, const Request& r) {
  return a.window > 0 ? max(0, r.L - r.n - a.window + 1) / kBlockSize : 0;
}

template <int QR>
__device__ __forceinline__ int row_tiles(const TreeLaunch& t, const Request& r) {
  return ((r.n << t.log2_g) + QR - 1) / QR;
}

// A request's share of the work line: its units, its segments and the units
// of one of them.
struct Load {
  int units, segs, len;
};

template <typename S>
__device__ __forceinline__ Load load_of(const TreeLaunch& t, const Request& r) {
  if (r.n == 0) return Load{0, 0, 0};
  const int nb = (r.L + kBlockSize - 1) / kBlockSize - first_block(t.a, r);
  const int segs = t.a.Hkv * row_tiles<S::QR>(t, r);
  return Load{segs * (S::kPieceUnits + nb), segs, S::kPieceUnits + nb};
}
template <typename S>
__device__ __forceinline__ Load load_of(const TreeLaunch& t, int b, bool tell) {
  return b < t.a.batch ? load_of<S>(t, request_of(t.a, b, tell)) : Load{0, 0, 0};
}

// Blocks [j0 + lo, j0 + hi) of a segment.
struct Piece {
  int b, kvh, tile;
  int q0, n, L;      // the request
  int j0, blocks;    // first block of the piece, and how many
  int after;         // blocks of the segment after the piece
  bool first;        // it begins with the segment's first block
};

// Walk over the pieces of a chunk; every warp of the CTA makes its own.
struct Walk {
  int b, off, rem;   // request, unit within it, units of the chunk that are left
  Request r;         // request b

  template <typename S>
  __device__ bool next(const TreeLaunch& t, Piece* p) {
    while (rem > 0) {
      const Load load = load_of<S>(t, r);
      if (off >= load.units) {
        if (++b >= t.a.batch) return false;
        off = 0;
        r = request_of(t.a, b, false);
        continue;
      }
      const int item = off / load.len;
      const int at = off - item * load.len;
      const int take = min(load.len - at, rem);
      const int lo = max(at, S::kPieceUnits) - S::kPieceUnits;
      const int hi = at + take - S::kPieceUnits;
      off += take;
      rem -= take;
      if (hi <= lo) continue;
      const int tiles = row_tiles<S::QR>(t, r);
      p->b = b;
      p->kvh = item / tiles;
      p->tile = item - p->kvh * tiles;
      p->q0 = r.q0;
      p->n = r.n;
      p->L = r.L;
      p->j0 = first_block(t.a, r) + lo;
      p->blocks = hi - lo;
      p->after = load.len - S::kPieceUnits - hi;
      p->first = lo == 0;
      return true;
    }
    return false;
  }
};

// Block-wide exclusive scan; every thread gets the total.
template <int NT>
__device__ __forceinline__ int excl_scan(int x, int* warp_sums, int* total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    const int v = warp_sums[w];
    if (w < warp) before += v;
    all += v;
  }
  __syncthreads();
  *total = all;
  return before + incl - x;
}

// 64 columns from column c0 of the words m << at (at may be negative).
__device__ __forceinline__ uint64_t shifted(uint64_t m, int at) {
  if (at >= 64 || at <= -64) return 0;
  return at >= 0 ? m << at : m >> -at;
}
// Bits [lo, hi) of a 64-bit word.
__device__ __forceinline__ uint64_t bit_range(int lo, int hi) {
  lo = max(lo, 0);
  hi = min(hi, 64);
  if (hi <= lo) return 0;
  return (~0ull >> (64 - (hi - lo))) << lo;
}

// Whether a bf16 of the words is an infinity or a NaN (an exponent of ones
// carries into the sign's place).
__device__ __forceinline__ bool wild(const uint4& w) {
  constexpr uint32_t e = 0x7f807f80u, one = 0x00800080u;
  return ((((w.x & e) + one) | ((w.y & e) + one) | ((w.z & e) + one) | ((w.w & e) + one)) &
          0x80008000u) != 0;
}
__device__ __forceinline__ uint32_t tamed(uint32_t w) {
  if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
  if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
  return w;
}

// A V tile's keys [lo, hi) (of the tile, NW warps share them): infinities and
// NaN become zeros; returns whether this lane met one.  A row is a warp's load
// (D = 128: two rows), four in flight.
template <typename S>
__device__ __forceinline__ bool tame_rows(uint8_t* vst, int lo, int hi, int warp, int lane) {
  constexpr int kLanes = S::D / 8, kRows = 32 / kLanes, kStep = S::kSoftmaxWarps * kRows;
  const int part = lane % kLanes;
  uint8_t* col = vst + part / 8 * 1024 + part % 8 * 16;
  auto at = [&](int r) { return reinterpret_cast<uint4*>(col + r / 8 * S::kGroup + r % 8 * 128); };
  bool found = false;
  for (int r = lo + warp * kRows + lane / kLanes; r < hi; r += 4 * kStep) {
    uint4 w[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      w[u] = r + u * kStep < hi ? *at(r + u * kStep) : make_uint4(0u, 0u, 0u, 0u);
    if (wild(w[0]) || wild(w[1]) || wild(w[2]) || wild(w[3])) {
      found = true;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (wild(w[u]))
          *at(r + u * kStep) = make_uint4(tamed(w[u].x), tamed(w[u].y), tamed(w[u].z), tamed(w[u].w));
    }
  }
  return found;
}
// The same keys' rows as zeros.
template <typename S>
__device__ __forceinline__ void clear_rows(uint8_t* vst, int lo, int hi, int warp, int lane) {
  constexpr int kLanes = S::D / 8, kRows = 32 / kLanes;
  const int part = lane % kLanes;
  for (int r = lo + warp * kRows + lane / kLanes; r < hi; r += S::kSoftmaxWarps * kRows)
    *reinterpret_cast<uint4*>(vst + r / 8 * S::kGroup + r % 8 * 128 + part / 8 * 1024 +
                              part % 8 * 16) = make_uint4(0u, 0u, 0u, 0u);
}

// What a query row sees: the prefix from key `kmin` up to `base`, and the
// drafted keys of `mask`.
struct Sight {
  int kmin, base;
  uint64_t mask;

  __device__ __forceinline__ uint64_t columns(int t0) const {  // of keys [t0, t0 + 64)
    return bit_range(kmin - t0, base - t0) | shifted(mask, base - t0);
  }
};

// Adds the infinities and NaN of V's keys [lo, hi) that the row sees to its
// finished output row (the tiles that not every row sees whole go through the
// MMA with such values as zeros, which would reach the other rows as 0 * inf).
// Columns [first, first + N) of them.
template <int N, bool kPartial>
__device__ __noinline__ void add_wild(const TreeArgs& a, const Piece& p, const Sight& see, int lo,
                                      int hi, int first, int D, float* prow, int pstride,
                                      uint16_t* orow) {
  const int32_t* trow = a.tables + static_cast<size_t>(p.b) * a.max_blocks;
  for (int t = lo; t < hi; ++t) {
    if (!(see.columns(t) & 1)) continue;
    const int id = trow[t / kBlockSize];
    if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.num_blocks)) continue;
    const uint16_t* v = a.v + ((static_cast<size_t>(id) * a.Hkv + p.kvh) * kBlockSize +
                               t % kBlockSize) * D;
    for (int d = first; d < first + N; ++d) {
      const uint32_t bits = v[d];
      if ((bits & 0x7f80u) != 0x7f80u) continue;
      const float x = __uint_as_float(bits << 16);
      if (kPartial)
        prow[(d / 4) * pstride + d % 4] += x;
      else
        orow[d] = f32_to_bf16_rn(__uint_as_float(static_cast<uint32_t>(orow[d]) << 16) + x);
    }
  }
}

// Pairs of CTAs (a cluster of two).
__device__ __forceinline__ void pair_sync() {
  __syncwarp();
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
          : "memory");
}
// The address of this CTA's shared variable in the CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t shared_of(const void* p, int rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void store_far(uint32_t to, float x) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(x) : "memory");
}
__device__ __forceinline__ void store_far(uint32_t to, float4 x) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to), "f"(x.x), "f"(x.y),
               "f"(x.z), "f"(x.w)
               : "memory");
}

template <int D, int QR, bool PAIR>
__global__ void __launch_bounds__(TreeShape<D, QR>::kThreads, 1)
    tree_attn_kernel(const __grid_constant__ TreeLaunch t) {
  using S = TreeShape<D, QR>;
  constexpr int BN = S::BN, BPT = S::BPT, DC = S::DC, NW = S::kSoftmaxWarps;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t b_q, b_qfree, b_k[S::KST], b_kfree[S::KST], b_v[S::VST], b_vfree[S::VST],
      b_s[2], b_pv[2], b_p[2], b_pair[2], b_first;
  __shared__ float pair_value[2][2][64];  // [exchange % 2][half][row]
  __shared__ uint32_t tmem_slot;
  __shared__ int failed_flag, wild_piece[2], warp_sums[S::kThreads / 32], longest;
  __shared__ Walk start;  // of the CTA's chunk
  volatile int* failed = &failed_flag;
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* sQ = smem + S::oQ;
  uint8_t* sK = smem + S::oK;
  uint8_t* sV = smem + S::oV;
  const TreeArgs& a = t.a;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  launch_dependents();
  if (threadIdx.x == 0) {
    mbar_init(&b_q, 1);
    mbar_init(&b_qfree, 1);
    mbar_init(&b_first, 1);
    for (int i = 0; i < S::KST; ++i) {
      mbar_init(&b_k[i], 1);
      mbar_init(&b_kfree[i], 1);
    }
    for (int i = 0; i < S::VST; ++i) {
      mbar_init(&b_v[i], 1);
      mbar_init(&b_vfree[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&b_s[i], 1);
      mbar_init(&b_pv[i], 1);
      mbar_init(&b_p[i], NW);
      mbar_init(&b_pair[i], 2);
    }
    failed_flag = 0;
    wild_piece[0] = wild_piece[1] = 0;
    longest = 0;
    mbar_fence_init();
    prefetch_tensormap(&t.tm_q);
    prefetch_tensormap(&t.tm_k);
    prefetch_tensormap(&t.tm_v);
  }
  if (warp == S::kWarpMma) tmem_alloc(&tmem_slot, S::kTmemCols);
  wait_predecessor();

  // ------------------------------------------------------- the CTA's chunk
  // Every CTA sums the requests' units and segments and finds the unit (or,
  // where segments stay whole, the segment) that it begins with.
  constexpr int NT = S::kThreads;
  const int tid = threadIdx.x;
  const int grid = static_cast<int>(gridDim.x);
  Request mine_r{0, 0, 0};
  if (tid < a.batch) mine_r = request_of(a, tid, blockIdx.x == 0);
  const Load mine = load_of<S>(t, mine_r);
  int units = 0, segs = 0;
  Load before{excl_scan<NT>(mine.units, warp_sums, &units),
              excl_scan<NT>(mine.segs, warp_sums, &segs), 0};
  int len = mine.len;
  if (a.batch > NT) {
    Load rest{0, 0, 0};
    for (int b = tid + NT; b < a.batch; b += NT) {
      const Load x = load_of<S>(t, b, blockIdx.x == 0);
      rest.units += x.units;
      rest.segs += x.segs;
      len = max(len, x.len);
    }
    int sum;
    excl_scan<NT>(rest.units, warp_sums, &sum);
    units += sum;
    excl_scan<NT>(rest.segs, warp_sums, &sum);
    segs += sum;
  }
  const int chunk = max(a.min_chunk, (units + grid - 1) / grid);
  len = __reduce_max_sync(0xffffffffu, len);
  if (lane == 0) atomicMax(&longest, len);
  __syncthreads();
  const bool whole = PAIR || !a.may_cut || (segs <= grid && longest <= chunk + a.whole_slack);
  // (where may_cut is false there are no more segments than CTAs)
  const int rank = PAIR ? blockIdx.x & 1 : 0;  // of the CTAs that share a segment
  const long long begin =
      static_cast<long long>(PAIR ? blockIdx.x / 2 : blockIdx.x) * (whole ? 1 : chunk);
  const bool any_work = begin < (whole ? segs : units);
  if (any_work) {
    const int want = static_cast<int>(begin);
    auto look = [&](int b, const Request& r, const Load& x, int at_unit, int at_seg) {
      const int at = whole ? at_seg : at_unit;
      if (want >= at && want < at + (whole ? x.segs : x.units)) {
        start = Walk{b, (want - at) * (whole ? x.len : 1),
                     whole ? x.len : min(chunk, units - want), r};
        if (PAIR) {  // half of the tiles each, the odd one to the first
          const int blocks = x.len - S::kPieceUnits;
          const int half = min(((blocks + BPT - 1) / BPT + 1) / 2 * BPT, blocks);
          if (rank == 1) start.off += S::kPieceUnits + half;
          start.rem = rank == 1 ? blocks - half : S::kPieceUnits + half;
        }
      }
    };
    look(tid, mine_r, mine, before.units, before.segs);
    if (a.batch > NT) {
      int at_unit, at_seg, sum;
      excl_scan<NT>(mine.units, warp_sums, &at_unit);
      excl_scan<NT>(mine.segs, warp_sums, &at_seg);
      for (int base = NT; base < a.batch && (whole ? at_seg : at_unit) <= want; base += NT) {
        Request r{0, 0, 0};
        if (base + tid < a.batch) r = request_of(a, base + tid, false);
        const Load x = load_of<S>(t, r);
        const int u = at_unit + excl_scan<NT>(x.units, warp_sums, &sum);
        at_unit += sum;
        const int s = at_seg + excl_scan<NT>(x.segs, warp_sums, &sum);
        at_seg += sum;
        look(base + tid, r, x, u, s);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  Walk walk{0, 0, 0, {0, 0, 0}};
  if (any_work) walk = start;
  Piece p;

  if (warp == S::kWarpK || warp == S::kWarpV) {
    // ============================ TMA of K, V ============================
    const bool is_k = warp == S::kWarpK;
    const CUtensorMap* map = is_k ? &t.tm_k : &t.tm_v;
    const int nst = is_k ? S::KST : S::VST;
    uint8_t* ring = is_k ? sK : sV;
    uint64_t* full = is_k ? b_k : b_v;
    uint64_t* freed = is_k ? b_kfree : b_vfree;
    const int past = a.num_blocks * a.Hkv * 2;  // a group past the pool: zeros
    const uint64_t policy = policy_evict_first();
    int g = 0;                                  // tiles issued
    // V's first loads wait for K's first tile: what the CTAs ask for at once lands
    // in about 4 us, and S comes first (D = 256: serving layer 40.4 -> 39.5 us, a
    // sliding one 21.1 -> 20.7, 64 pairs over 300 keys 14.0 -> 13.5).  D = 128 gains
    // nothing (four long requests 115.0 us without, 115.2 with it) and a small call
    // loses (8.3 -> 8.9).  They wait for b_first, which the MMA warp arrives at once in
    // a launch, when it has seen K's first tile.  b_k[0] itself will not do: K's
    // stages are refilled without V's help, so its second phase may end before this
    // warp has looked at the first, whose parity it then never sees.
    const bool late = D == 256 && !is_k && (PAIR || walk.rem > S::kPieceUnits + 4 * BPT);
    bool ok = true;
    while (ok && walk.next<S>(t, &p)) {
      const int32_t* trow = a.tables + static_cast<size_t>(p.b) * a.max_blocks + p.j0;
      // the piece's blocks, 32 at a time (one per lane), read 32 ahead
      auto load_groups = [&](int base) -> int {
        int at = past;
        if (base + lane < p.blocks) {
          const int id = trow[base + lane];
          if (static_cast<unsigned>(id) < static_cast<unsigned>(a.num_blocks))
            at = (id * a.Hkv + p.kvh) * 2;
          else
            report(a.err, PKA_DEVERR_BAD_TABLE);
        }
        return at;
      };
      static_assert(32 % BPT == 0, "a tile's blocks lie in one window of 32");
      int now = load_groups(0), next = load_groups(32);
      for (int j = 0; j < p.blocks; j += BPT, ++g) {
        if (j > 0 && j % 32 == 0) {
          now = next;
          next = load_groups(j + 32);
        }
        const int at = __shfl_sync(0xffffffffu, now, (j + lane % BPT) & 31);
        const int st = g % nst;
        const bool again = g >= nst;
        if (again || (late && g == 0))
          ok = warp_wait(again ? &freed[st] : &b_first, again ? (g / nst - 1) & 1 : 0, a.err, failed);
        if (!ok || __any_sync(0xffffffffu, stop_requested(failed))) {
          ok = false;
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(&full[st], S::kStage);
        __syncwarp();
        if (lane < BPT)
          tma_load_4d(ring + st * S::kStage + lane * S::kBlockBytes, map, 0, 0, 0, at, &full[st],
                      policy);
      }
    }
    // every copy must land before the CTA may end
    if (lane == 0)
      for (int j = max(0, g - nst); j < g; ++j) mbar_wait(&full[j % nst], (j / nst) & 1, a.err);
    __syncwarp();
  } else if (warp == S::kWarpQ) {
    // =============================== TMA of Q ===============================
    int pieces = 0;
    while (walk.next<S>(t, &p)) {
      if (pieces > 0 && !warp_wait(&b_qfree, (pieces - 1) & 1, a.err, failed)) break;
      if (__any_sync(0xffffffffu, stop_requested(failed))) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&b_q, DC * (t.q_tokens << t.log2_g) * 128);
#pragma unroll
        for (int c = 0; c < DC; ++c)
          tma_load_3d(sQ + c * S::kQChunk, &t.tm_q, c * 64, p.kvh << t.log2_g,
                      p.q0 + p.tile * (QR >> t.log2_g), &b_q);
      }
      __syncwarp();
      ++pieces;
    }
    if (lane == 0 && pieces > 0) mbar_wait(&b_q, (pieces - 1) & 1, a.err);
    __syncwarp();
  } else if (warp == S::kWarpMma) {
    // ================================ MMA ================================
    constexpr uint32_t idesc_qk = idesc_bf16_f32(128, BN, 0, 0);
    constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, 0, 1);
    const uint32_t aQ = smem_u32(sQ), aK = smem_u32(sK), aV = smem_u32(sV);
    int g = 0, issued_pv = 0, pieces = 0;
    bool ok = true;
    auto issue_qk = [&](int i, bool last) -> bool {
      const int ks = i % S::KST;
      if (!warp_wait(&b_k[ks], (i / S::KST) & 1, a.err, failed)) return false;
      tc_fence_after();
      if (lane == 0) {
        if (i == 0) mbar_arrive(&b_first);
        const uint32_t kst = aK + ks * S::kStage;
#pragma unroll
        for (int c = 0; c < DC; ++c)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_bf16(tmem + (i & 1) * BN, smem_desc_sw128(aQ + c * S::kQChunk + kk * 32, 16, 1024),
                      smem_desc_sw128(kst + c * 1024 + kk * 32, 16, S::kGroup), idesc_qk,
                      (c | kk) != 0);
        umma_commit(&b_s[i & 1]);
        umma_commit(&b_kfree[ks]);
        if (last) umma_commit(&b_qfree);
      }
      __syncwarp();
      return true;
    };
    while (ok && walk.next<S>(t, &p)) {
      const int nt = (p.blocks + BPT - 1) / BPT;
      ok = warp_wait(&b_q, pieces & 1, a.err, failed);
      ++pieces;
      if (ok) ok = issue_qk(g, nt == 1);
      if (ok && nt > 1) ok = issue_qk(g + 1, nt == 2);
      for (int j = 0; ok && j < nt; ++j, ++g) {
        const int st = g & 1, vs = g % S::VST;
        ok = warp_wait(&b_v[vs], (g / S::VST) & 1, a.err, failed) &&
             warp_wait(&b_p[st], (g >> 1) & 1, a.err, failed);
        if (!ok || __any_sync(0xffffffffu, stop_requested(failed))) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (lane == 0) {
          const uint32_t vst = aV + vs * S::kStage;
#pragma unroll
          for (int k = 0; k < BPT; ++k)
            umma_bf16_ts(tmem + S::kTmemO, tmem + S::kTmemP + st * (BN / 2) + k * 8,
                         smem_desc_sw128(vst + k * S::kBlockBytes, 1024, S::kGroup), idesc_pv,
                         (j > 0 || k > 0) ? 1u : 0u);
          umma_commit(&b_pv[st]);
          umma_commit(&b_vfree[vs]);
        }
        __syncwarp();
        issued_pv = g + 1;
        if (j + 2 < nt) ok = issue_qk(g + 2, j + 3 == nt);
      }
    }
    // the last P V must have finished before TMEM is freed
    if (issued_pv > 0) mbar_wait(&b_pv[(issued_pv - 1) & 1], ((issued_pv - 1) >> 1) & 1, a.err);
    __syncwarp();
  } else {
    // ============================== softmax ==============================
    constexpr int SPLIT = S::kSplit, CN = S::CN;
    const int group = SPLIT == 2 ? warp & 1 : warp;  // 32 rows
    const int half = SPLIT == 2 ? warp >> 2 : 0;     // which columns of them
    const int sw = SPLIT == 2 ? group + 2 * half : warp;
    const int r = group * 32 + lane;
    const int c0 = half * CN;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(group * 32) << 16);
    // Two threads of a row give each other a value (an mbarrier per 32 rows: a
    // partner that has stopped is waited for no longer than anything else).
    int exchanges = 0;
    auto exchange = [&](float mine, float* other) -> bool {
      pair_value[exchanges & 1][half][r] = mine;
      __syncwarp();
      if (lane == 0) mbar_arrive(&b_pair[group]);
      if (!warp_wait(&b_pair[group], exchanges & 1, a.err, failed)) return false;
      *other = pair_value[exchanges & 1][half ^ 1][r];
      ++exchanges;
      return true;
    };
    const bool capped = a.softcap > 0.f;
    const float sl2 = a.scale * kLog2e;
    // scale <= 0 and caps: the logits are formed before the mask
    const bool prescale = capped || !(sl2 > 0.f);
    const float cap_in = capped ? fmaxf(fminf(a.scale / a.softcap, kFltMax), -kFltMax) : 0.f;
    const float cap_mag = fabsf(cap_in);
    const float cap_out = a.softcap * kLog2e;
    // x(s) = s (k1 + s^2 (k3 + k5 s^2)): the capped logit's short series, which
    // grows with s for cap_in > 0 (so the maximum may be taken over raw s)
    const float k1 = cap_in * cap_out;
    const float k3 = -cap_in * cap_in * k1 * (1.f / 3.f);
    const float k5 = 2.f * cap_in * cap_in * cap_in * cap_in * k1 * (1.f / 15.f);
    const bool fold_ok = capped && cap_in > 0.f && k5 > 0.f && k5 <= kFltMax;
    int g = 0, piece = 0, met = 0;
    bool ok = true;
    int4 cut = make_int4(0, 0, 0, 0);  // this chunk's segment that goes on in the next one
    while (ok && walk.next<S>(t, &p)) {
      ++piece;
      const int row = p.tile * QR + r;
      const int tok = row >> t.log2_g;
      const bool row_valid = tok < p.n;
      const bool idle = ((p.tile * QR + group * 32) >> t.log2_g) >= p.n;  // no row of this warp
      const int nt = (p.blocks + BPT - 1) / BPT;
      const int t_begin = p.j0 * kBlockSize;
      const int t_end = min(t_begin + p.blocks * kBlockSize, p.L);
      Sight see{0x40000000, p.L - p.n, 0};
      if (row_valid) {
        const uint64_t own_bits = p.n == 64 ? ~0ull : (1ull << p.n) - 1;
        const uint64_t* masks = reinterpret_cast<const uint64_t*>(a.masks) + p.q0;
        see.mask = masks[tok] & own_bits;
        const int deep = __popcll(see.mask);
        see.kmin = a.window > 0 ? max(0, see.base + max(deep, 1) - a.window) : 0;
        // Drafted keys may lie before the window: those of a tree up to 63 before the row,
        // of other masks 64 (all bits against none).
        if (a.window > 0 && a.window <= 64) {
          uint64_t left = see.mask;
          while (left != 0) {
            const int j = __ffsll(static_cast<long long>(left)) - 1;
            left &= left - 1;
            if (deep - __popcll(masks[j] & own_bits) >= a.window) see.mask &= ~(1ull << j);
          }
        }
      }
      // tiles that not every row sees whole: from the window's edge and from
      // the drafted keys on
      const int edge_lo = a.window > 0 ? max(0, p.L - a.window) : 0;
      const int edge_hi = see.base;
      float m_ref = -INFINITY, l = 0.f;
      bool seen = false;
      for (int j = 0; j < nt; ++j, ++g) {
        const int st = g & 1;
        const uint32_t ph = (g >> 1) & 1;
        const int t0 = t_begin + j * BN;
        if (__any_sync(0xffffffffu, stop_requested(failed)) ||
            !warp_wait(&b_s[st], ph, a.err, failed)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (!idle) {
          float s[CN];
          if constexpr (CN == 32) {
            tmem_ld32(lane_base + st * BN + c0, s);
          } else {
#pragma unroll
            for (int c = 0; c < CN / 64; ++c) {
              float x[64];
              tmem_ld64(lane_base + st * BN + c0 + c * 64, x);
#pragma unroll
              for (int e = 0; e < 64; ++e) s[c * 64 + e] = x[e];
            }
          }
          constexpr int kWords = (CN + 63) / 64;
          uint64_t vis[kWords];
          bool whole = true;
#pragma unroll
          for (int c = 0; c < kWords; ++c) {
            constexpr uint64_t kAll = CN < 64 ? (1ull << (CN % 64)) - 1 : ~0ull;
            const int at = c0 + c * 64;
            vis[c] = row_valid ? see.columns(t0 + at) & bit_range(0, t_end - t0 - at) & kAll : 0;
            whole = whole && vis[c] == kAll;
            seen = seen || vis[c] != 0;
          }
          // Rows of no token hold what the MMA left there: they have no say in the
          // warp's votes, and need no mask.
          const bool need_mask = __any_sync(0xffffffffu, row_valid && !whole);
          bool folded = false, have_max = false;
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          if (capped) {
            if (need_mask) {  // (what lies in a hidden column has no say either)
#pragma unroll
              for (int c = 0; c < CN; ++c)
                if (!((vis[c / 64] >> (c % 64)) & 1)) s[c] = 0.f;
            }
            float n4[4] = {INFINITY, INFINITY, INFINITY, INFINITY};
#pragma unroll
            for (int c = 0; c < CN / 2; ++c) {
              m4[c & 3] = max3f(m4[c & 3], s[2 * c], s[2 * c + 1]);
              n4[c & 3] = min3f(n4[c & 3], s[2 * c], s[2 * c + 1]);
            }
            const float amax = fmaxf(fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])),
                                     -fminf(fminf(n4[0], n4[1]), fminf(n4[2], n4[3])));
            // the form of cap * tanh(s * scale / cap): a short or a long series
            // while every argument of the warp's rows is below 1/8 or 1/2, else
            // for each of them the long series or exp2 (whose error, 7e-7 of the
            // cap, a small logit would feel)
            const float far = row_valid ? amax * cap_mag : 0.f;
            if (fold_ok && __all_sync(0xffffffffu, far < 0.125f)) {
              folded = true;
              have_max = !need_mask;
            } else if (__all_sync(0xffffffffu, far < 0.5f)) {
#pragma unroll
              for (int c = 0; c < CN; ++c) s[c] = cap_out * tanh_taylor(s[c] * cap_in);
            } else {
#pragma unroll
              for (int c = 0; c < CN; ++c) {
                const float y = s[c] * cap_in;
                s[c] = cap_out * (fabsf(y) < 0.5f ? tanh_taylor(y) : tanh_via_exp2(y));
              }
            }
          } else if (prescale) {
#pragma unroll
            for (int c = 0; c < CN; c += 2) {
              const float2 v = mul2(make_float2(s[c], s[c + 1]), make_float2(sl2, sl2));
              s[c] = v.x;
              s[c + 1] = v.y;
            }
          }
          if (need_mask) {
#pragma unroll
            for (int c = 0; c < CN; ++c)
              if (!((vis[c / 64] >> (c % 64)) & 1)) s[c] = -INFINITY;
          }
          if (!have_max) {
#pragma unroll
            for (int e = 0; e < 4; ++e) m4[e] = -INFINITY;
#pragma unroll
            for (int c = 0; c < CN / 2; ++c) m4[c & 3] = max3f(m4[c & 3], s[2 * c], s[2 * c + 1]);
          }
          float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
          if (folded)
            mx = mx * fmaf(mx * mx, fmaf(mx * mx, k5, k3), k1);
          else if (!prescale)
            mx *= sl2;
          if constexpr (SPLIT == 2) {  // the row's maximum, of both halves
            float other;
            if (!exchange(mx, &other)) {
              ok = false;
              break;
            }
            mx = fmaxf(mx, other);
          }
          const float m_new = fmaxf(m_ref, mx);
          // O moves to a new reference only when the maximum grows by more
          // than 2^8: every weight stays below 2^8, and O and the sum share
          // the reference, so the result does not depend on it
          const bool resc = j > 0 && row_valid && m_new > m_ref + 8.f;
          if (__any_sync(0xffffffffu, resc)) {
            if (!warp_wait(&b_pv[(g - 1) & 1], ((g - 1) >> 1) & 1, a.err, failed)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const float f = resc ? fast_exp2(m_ref - m_new) : 1.f;
#pragma unroll 1
            for (int c = half * (D / 32 / SPLIT); c < (half + 1) * (D / 32 / SPLIT); ++c) {
              float o[32];
              tmem_ld32(lane_base + S::kTmemO + c * 32, o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] *= f;
              tmem_st32(lane_base + S::kTmemO + c * 32, o);
            }
          }
          if (resc) l *= fast_exp2(m_ref - m_new);
          if (j == 0 || resc) m_ref = m_new;
          const float ms = m_ref == -INFINITY ? 0.f : m_ref;
          const float xs = prescale ? 1.f : sl2;
          // P_j's buffer: its last reader, P_{j-2} V_{j-2}, was issued before
          // S_j, whose completion this thread has waited for
          auto make_p = [&](auto logit) {
            float2 sum0 = make_float2(0.f, 0.f), sum1 = make_float2(0.f, 0.f);
#pragma unroll
            for (int h = 0; h < kWords; ++h) {
              constexpr int kPairs = CN < 64 ? CN / 2 : 32;
              uint32_t pk[kPairs];
#pragma unroll
              for (int e = 0; e < kPairs; ++e) {
                const float2 x = logit(make_float2(s[h * 64 + 2 * e], s[h * 64 + 2 * e + 1]));
                const float2 w = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                if (e & 1)
                  sum1 = add2(sum1, w);
                else
                  sum0 = add2(sum0, w);
                // weights go to the MMA as bf16 (off by 2^-8 of a weight at
                // most; the sum is of the unrounded ones)
                pk[e] = pack_bf16x2(w.x, w.y);
              }
              const uint32_t to = lane_base + S::kTmemP + st * (BN / 2) + c0 / 2 + h * 32;
              if constexpr (kPairs == 16)
                tmem_st16_u(to, pk);
              else
                tmem_st32_u(to, pk);
            }
            const float2 sum = add2(sum0, sum1);
            return sum.x + sum.y;
          };
          const float2 nms = make_float2(-ms, -ms);
          l += folded ? make_p([&](float2 x) {
            const float2 y = mul2(x, x);
            const float2 u =
                fma2(y, fma2(y, make_float2(k5, k5), make_float2(k3, k3)), make_float2(k1, k1));
            return fma2(x, u, nms);
          })
                      : make_p([&](float2 x) { return fma2(x, make_float2(xs, xs), nms); });
          tmem_wait_st();
        }
        if (t0 < edge_lo || t0 + BN > edge_hi) {
          // V's rows past the sequence are stale: zeros.  Infinities and NaN of
          // the keys that not every row sees become zeros here and are added to
          // the rows that see them in the end.
          const int vs = g % S::VST;
          if (!warp_wait(&b_v[vs], (g / S::VST) & 1, a.err, failed)) {
            ok = false;
            break;
          }
          uint8_t* vst = sV + vs * S::kStage;
          const int stale = min(BN, (p.L + kBlockSize - 1) / kBlockSize * kBlockSize - t0);
          bool found = tame_rows<S>(vst, 0, min(BN, edge_lo - t0), sw, lane);
          if (tame_rows<S>(vst, max(0, edge_hi - t0), min(BN, p.L - t0), sw, lane)) found = true;
          clear_rows<S>(vst, max(0, p.L - t0), stale, sw, lane);
          if (found) *const_cast<volatile int*>(&wild_piece[piece & 1]) = piece;
          fence_proxy_async_smem();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b_p[st]);
      }
      // ---------------------------------------------------------- epilogue
      if (ok) ok = warp_wait(&b_pv[(g - 1) & 1], ((g - 1) >> 1) & 1, a.err, failed);
      if (!ok) break;
      tc_fence_after();
      const bool direct = p.first && p.after == 0;
      if (p.first && p.after > 0)
        cut = make_int4(p.q0 + p.tile * (QR >> t.log2_g), p.kvh << t.log2_g,
                        min(QR, (p.n << t.log2_g) - p.tile * QR), 1 + (p.after + chunk - 1) / chunk);
      if (!idle) {
        if constexpr (SPLIT == 2) {  // the row's sum, of both halves
          float other;  // (-1: it sees keys, but they have no weight)
          if (!exchange(l == 0.f && seen ? -1.f : l, &other)) {
            ok = false;
            break;
          }
          seen = seen || other != 0.f;
          if (other != -1.f) l += other;
        }
        // A row whose visible logits are all -infinity: 0 / 0; one that sees nothing: 0.
        // A piece of such logits alone (LSE +infinity) goes on as it is, zeros, or NaN where
        // V has an infinity or a NaN: with other pieces beside it that is its share.
        const bool unweighed = l == 0.f && seen;
        const float inv = l > 0.f                  ? 1.f / l
                          : !seen                  ? 0.f
                          : direct || !unweighed   ? __int_as_float(0x7fffffff)
                                                   : 1.f;
        const float lse = unweighed  ? INFINITY
                          : l == 0.f ? -INFINITY
                                     : m_ref + log2f(l);  // (a NaN sum: NaN)
        const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + (p.first ? 1 : 0);
        float* prow = a.partial_o + (slot * (D / 4) * QR + r) * 4;
        uint16_t* orow =
            a.out + (static_cast<size_t>(p.q0 + tok) * a.Hq + (p.kvh << t.log2_g) +
                     (row & ((1 << t.log2_g) - 1))) * D;
        if (PAIR && !direct) {
          // The other CTA holds the segment's other keys: each gives the other half
          // of a thread's columns, into the place of its queries, and finishes the rest.
          constexpr int kKeep = D / SPLIT / 64;  // groups of 32 columns
          const int give = (half * 2 + (rank ^ 1)) * kKeep, keep = (half * 2 + rank) * kKeep;
          const uint32_t rows_there = shared_of(sQ, rank ^ 1) + (half * kKeep * 8 * QR + r) * 16;
          const float4* rows_here =
              reinterpret_cast<const float4*>(sQ) + half * kKeep * 8 * QR + r;
          float* lse_here = &pair_value[0][0][0] + r;
          pair_sync();  // the other CTA has done with its queries
          ++met;
#pragma unroll 1
          for (int c = 0; c < kKeep; ++c) {
            float o[32];
            tmem_ld32(lane_base + S::kTmemO + (give + c) * 32, o);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              store_far(rows_there + (c * 8 + e) * QR * 16,
                        make_float4(o[4 * e] * inv, o[4 * e + 1] * inv, o[4 * e + 2] * inv,
                                    o[4 * e + 3] * inv));
          }
          if (half == 0) store_far(shared_of(lse_here, rank ^ 1), lse);
          const volatile int* wild_here = wild_piece;
          if (wild_here[piece & 1] == piece)
            store_far(shared_of(&wild_piece[(piece & 1) ^ 1], rank ^ 1), __int_as_float(piece));
          pair_sync();
          ++met;
          const float far_lse = *lse_here;
          const bool near_weight = fabsf(lse) != INFINITY, far_weight = fabsf(far_lse) != INFINITY;
          const float top = fmaxf(near_weight ? lse : -INFINITY, far_weight ? far_lse : -INFINITY);
          const float w = near_weight ? fast_exp2(lse - top) : 0.f;
          const float far_w = far_weight ? fast_exp2(far_lse - top) : 0.f;
          // (no weight at all: NaN if one of them sees keys, else 0)
          const float den = w + far_w;
          const bool none = den == 0.f;
          const float f = !none                                       ? w * inv / den
                          : lse == INFINITY || far_lse == INFINITY ? __int_as_float(0x7fffffff)
                                                                    : 0.f;
          const float far_f = none ? 0.f : far_w / den;
#pragma unroll 1
          for (int c = 0; c < kKeep; ++c) {
            float o[32];
            tmem_ld32(lane_base + S::kTmemO + (keep + c) * 32, o);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float4 y = rows_here[(c * 8 + e) * QR];
              o[4 * e] = fmaf(f, o[4 * e], far_f * y.x);
              o[4 * e + 1] = fmaf(f, o[4 * e + 1], far_f * y.y);
              o[4 * e + 2] = fmaf(f, o[4 * e + 2], far_f * y.z);
              o[4 * e + 3] = fmaf(f, o[4 * e + 3], far_f * y.w);
            }
            if (row_valid) {
#pragma unroll
              for (int q = 0; q < 4; ++q)
                *reinterpret_cast<uint4*>(orow + (keep + c) * 32 + q * 8) =
                    make_uint4(pack_bf16x2(o[q * 8 + 0], o[q * 8 + 1]),
                               pack_bf16x2(o[q * 8 + 2], o[q * 8 + 3]),
                               pack_bf16x2(o[q * 8 + 4], o[q * 8 + 5]),
                               pack_bf16x2(o[q * 8 + 6], o[q * 8 + 7]));
            }
          }
          if (row_valid && (wild_here[0] == piece || wild_here[1] == piece)) {
            auto add = [&](int lo, int hi) {
              add_wild<kKeep * 32, false>(a, p, see, lo, hi, keep * 32, D, nullptr, 0, orow);
            };
            const int lo = first_block(a, Request{p.n, p.q0, p.L}) * kBlockSize;
            const int mid = max(lo, edge_lo);
            add(lo, mid);
            add(max(mid, edge_hi), p.L);
          }
          break;  // (a pair's CTAs take one piece)
        }
#pragma unroll 1
        for (int c = half * (D / 64 / SPLIT); c < (half + 1) * (D / 64 / SPLIT); ++c) {
          float o[64];
          tmem_ld64(lane_base + S::kTmemO + c * 64, o);
          if (direct) {
            if (row_valid) {
#pragma unroll
              for (int q = 0; q < 8; ++q)
                *reinterpret_cast<uint4*>(orow + c * 64 + q * 8) =
                    make_uint4(pack_bf16x2(o[q * 8 + 0] * inv, o[q * 8 + 1] * inv),
                               pack_bf16x2(o[q * 8 + 2] * inv, o[q * 8 + 3] * inv),
                               pack_bf16x2(o[q * 8 + 4] * inv, o[q * 8 + 5] * inv),
                               pack_bf16x2(o[q * 8 + 6] * inv, o[q * 8 + 7] * inv));
            }
          } else if (row_valid) {
            // [D / 4][QR rows] float4: each store of a warp is consecutive
#pragma unroll
            for (int e = 0; e < 16; ++e)
              *reinterpret_cast<float4*>(prow + static_cast<size_t>(c * 16 + e) * QR * 4) =
                  make_float4(o[4 * e] * inv, o[4 * e + 1] * inv, o[4 * e + 2] * inv,
                              o[4 * e + 3] * inv);
          }
        }
        if (!direct && half == 0) a.partial_lse[slot * QR + r] = lse;
        if (row_valid && *const_cast<volatile int*>(&wild_piece[piece & 1]) == piece) {
          auto add = [&](int lo, int hi) {
            if (direct)
              add_wild<D / SPLIT, false>(a, p, see, lo, hi, half * (D / SPLIT), D, nullptr, 0, orow);
            else
              add_wild<D / SPLIT, true>(a, p, see, lo, hi, half * (D / SPLIT), D, prow, QR * 4,
                                        nullptr);
          };
          const int mid = min(t_end, max(t_begin, edge_lo));
          add(t_begin, mid);
          add(max(mid, edge_hi), t_end);
        }
      }
    }
    if (threadIdx.x == 0 && a.may_cut) {
      if (!any_work || !ok) cut.w = 0;
      a.cuts[blockIdx.x] = cut;
    }
    if (PAIR)
      for (; met < 2; ++met) pair_sync();
  }
  // Every warp meets the other CTA twice: after the second time neither writes
  // into the other's memory.
  if (PAIR && (warp == S::kWarpK || warp == S::kWarpV || warp == S::kWarpMma || warp == S::kWarpQ)) {
    pair_sync();
    pair_sync();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == S::kWarpMma) tmem_dealloc(tmem, S::kTmemCols);
}

// Merge of the cut segments' pieces: M = max LSE, out = sum 2^(LSE - M) O /
// sum 2^(LSE - M).  A warp takes 32 rows x 8 columns, a row a lane; for segments
// of many pieces 2 to 8 warps share them (piece k to warp k mod their number)
// and meet in shared memory.  The order of the sums depends on the number of
// pieces alone.
constexpr int kMergeWarps = 8;

struct MergeState {
  float M, den;      // den = -1: pieces that see keys, but no weight
  float4 acc[2];
};

// Warps that share the pieces.
__device__ __forceinline__ int merge_share(int pieces) {
  return pieces <= 4 ? 1 : pieces <= 8 ? 2 : pieces <= 16 ? 4 : 8;
}

template <int D, int QR>
__global__ void __launch_bounds__(kMergeWarps * 32, 4) tree_merge_kernel(
    const __grid_constant__ TreeMergeArgs a) {
  __shared__ int first_unit[kTreeMaxCtas + 1];
  __shared__ int4 cuts[kTreeMaxCtas];
  __shared__ float sm[kMergeWarps][2][32];
  __shared__ float4 so[kMergeWarps][2][32];
  __shared__ int warp_sums[kMergeWarps];
  constexpr int kCols = D / 8;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  launch_dependents();
  wait_predecessor();
  static_assert(kTreeMaxCtas <= kMergeWarps * 32, "a thread per chunk");
  int4 c = make_int4(0, 0, 0, 0);
  if (tid < a.chunks) c = a.cuts[tid];
  const int mine = c.w > 0 ? (c.z + 31) / 32 * (kCols * merge_share(c.w) / kMergeWarps) : 0;
  int total;
  const int before = excl_scan<kMergeWarps * 32>(mine, warp_sums, &total);
  if (tid < kTreeMaxCtas) {
    first_unit[tid] = before;
    cuts[tid] = c;
  }
  __syncthreads();
  for (int u = blockIdx.x; u < total; u += gridDim.x) {
    int lo = 0, hi = kTreeMaxCtas;  // the last chunk whose units begin at or before u
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (first_unit[mid] <= u)
        lo = mid;
      else
        hi = mid;
    }
    const int4 seg = cuts[lo];
    const int share = merge_share(seg.w);
    const int rel = u - first_unit[lo], per_row = kCols * share / kMergeWarps;
    const int r = rel / per_row * 32 + lane;
    const int col = rel % per_row * (kMergeWarps / share) + warp / share;
    const int part = warp % share;
    // piece 0 lies in the second slot of its chunk, the others in the first
    // slots of the chunks that follow
    MergeState x{-INFINITY, 0.f, {}};
    bool dead = false;  // a piece that sees keys, but with no weight
    for (int k0 = part; k0 < seg.w; k0 += 4 * share) {
      float lse[4];
      float4 y[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = k0 + i * share;
        lse[i] = -INFINITY;
        y[i][0] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k < seg.w) {
          const size_t slot = 2 * static_cast<size_t>(lo + k) + (k == 0 ? 1 : 0);
          lse[i] = a.partial_lse[slot * QR + r];
          const float4* o = reinterpret_cast<const float4*>(a.partial_o) +
                            (slot * (D / 4) + col * 2) * QR + r;
          y[i][0] = o[0];
          y[i][1] = o[QR];
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // a piece that sees nothing; one of logits that are all -infinity, whose
        // row holds zeros and the infinities and NaN of V, 0 times which is NaN
        if (lse[i] == -INFINITY) continue;
        if (lse[i] == INFINITY) {
          dead = true;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            x.acc[q].x += 0.f * y[i][q].x;
            x.acc[q].y += 0.f * y[i][q].y;
            x.acc[q].z += 0.f * y[i][q].z;
            x.acc[q].w += 0.f * y[i][q].w;
          }
          continue;
        }
        const float nm = fmaxf(x.M, lse[i]);
        const float keep = x.M == -INFINITY ? 0.f : fast_exp2(x.M - nm);
        const float w = fast_exp2(lse[i] - nm);
        x.den = x.den * keep + w;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          x.acc[q].x = x.acc[q].x * keep + w * y[i][q].x;
          x.acc[q].y = x.acc[q].y * keep + w * y[i][q].y;
          x.acc[q].z = x.acc[q].z * keep + w * y[i][q].z;
          x.acc[q].w = x.acc[q].w * keep + w * y[i][q].w;
        }
        x.M = nm;
      }
    }
    if (dead && x.den == 0.f) x.den = -1.f;
    if (share > 1) {  // uniform over the CTA
      sm[warp][0][lane] = x.M;
      sm[warp][1][lane] = x.den;
      so[warp][0][lane] = x.acc[0];
      so[warp][1][lane] = x.acc[1];
      __syncthreads();
      if (part == 0) {
        float top = -INFINITY, sum = 0.f;
        bool nothing = false;
        float4 y[2] = {};
        for (int w = warp; w < warp + share; ++w) top = fmaxf(top, sm[w][0][lane]);
        for (int w = warp; w < warp + share; ++w) {
          const float m = sm[w][0][lane], d = sm[w][1][lane];
          if (d == -1.f) nothing = true;
          // (without a weight: zeros and NaN; -infinity beside one: a NaN sum)
          const bool no_weight = d == 0.f || d == -1.f;
          const float f = no_weight || m == -INFINITY ? 1.f : fast_exp2(m - top);
          if (!no_weight) sum += f * d;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const float4 v = so[w][q][lane];
            y[q].x += f * v.x;
            y[q].y += f * v.y;
            y[q].z += f * v.z;
            y[q].w += f * v.w;
          }
        }
        x.den = sum == 0.f && nothing ? -1.f : sum;
        x.acc[0] = y[0];
        x.acc[1] = y[1];
      }
      __syncthreads();
    }
    if (part == 0 && r < seg.z) {
      const float inv = x.den == 0.f    ? 0.f
                        : x.den == -1.f ? __int_as_float(0x7fffffff)
                                        : 1.f / x.den;
      const int tok = r >> a.log2_g, head = seg.y + (r & ((1 << a.log2_g) - 1));
      uint16_t* out = a.out + (static_cast<size_t>(seg.x + tok) * a.Hq + head) * D + col * 8;
      *reinterpret_cast<uint4*>(out) =
          make_uint4(pack_bf16x2(x.acc[0].x * inv, x.acc[0].y * inv),
                     pack_bf16x2(x.acc[0].z * inv, x.acc[0].w * inv),
                     pack_bf16x2(x.acc[1].x * inv, x.acc[1].y * inv),
                     pack_bf16x2(x.acc[1].z * inv, x.acc[1].w * inv));
    }
  }
}

int log2_of(int g) { return g == 1 ? 0 : g == 2 ? 1 : g == 4 ? 2 : 3; }

template <int D, int QR>
cudaError_t launch_tree_t(const TreeArgs& a, int sm_count, cudaStream_t stream) {
  using S = TreeShape<D, QR>;
  const int G = a.Hq / a.Hkv;
  TreeLaunch t{};
  t.a = a;
  t.log2_g = log2_of(G);
  t.q_tokens = a.max_query_len < QR / G ? a.max_query_len : QR / G;
  const long long rows = static_cast<long long>(a.num_blocks) * a.Hkv * kBlockSize;
  if (!tmap_query_tiles(&t.tm_q, a.q, D, a.Hq, a.total_q, G, t.q_tokens) ||
      !tmap_pool_groups(&t.tm_k, a.k, D, rows) || !tmap_pool_groups(&t.tm_v, a.v, D, rows))
    return cudaErrorInvalidValue;
  auto kern = a.pair > 0 ? tree_attn_kernel<D, QR, true> : tree_attn_kernel<D, QR, false>;
  cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kern), S::kSmemBytes);
  if (e != cudaSuccess) return e;
  const int grid = sm_count < kTreeMaxCtas ? sm_count : kTreeMaxCtas;
  if (a.pair)
    return launch_overlapped(kern, dim3(2 * a.pair), S::kThreads, S::kSmemBytes, stream, t, 2);
  e = launch_overlapped(kern, dim3(grid), S::kThreads, S::kSmemBytes, stream, t);
  if (e != cudaSuccess || !a.may_cut) return e;
  TreeMergeArgs m{};
  m.partial_o = a.partial_o;
  m.partial_lse = a.partial_lse;
  m.cuts = a.cuts;
  m.out = a.out;
  m.Hq = a.Hq;
  m.log2_g = t.log2_g;
  m.chunks = grid;
  return launch_overlapped(tree_merge_kernel<D, QR>, dim3(sm_count * 8), kMergeWarps * 32, 0,
                           stream, m);
}

}  // namespace

// A batch whose trees all fit 64 rows of a KV head takes the smaller row tile.
int tree_tile_rows(int max_query_len, int group) { return max_query_len * group <= 64 ? 64 : 128; }

cudaError_t launch_tree_attn(const TreeArgs& a, int head_dim, int sm_count, cudaStream_t stream) {
  const bool small = tree_tile_rows(a.max_query_len, a.Hq / a.Hkv) == 64;
  if (head_dim == 128)
    return small ? launch_tree_t<128, 64>(a, sm_count, stream)
                 : launch_tree_t<128, 128>(a, sm_count, stream);
  return small ? launch_tree_t<256, 64>(a, sm_count, stream)
               : launch_tree_t<256, 128>(a, sm_count, stream);
}

}  // namespace pka
