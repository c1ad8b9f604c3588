// Paged decode attention over a 4-bit cache (sm_103a).
//
// One query token per request attends over its visible keys, held as e2m1
// codes with an e4m3 scale per 16 channels (kv4.cuh).  A key and its value
// cost 9 D / 8 bytes per KV head, 3.6 times fewer than in bf16, so the
// arithmetic per byte is 3.6 times that of the bf16 decode: the design keeps
// the conversion short and every other cost off the path.
//
// Work.  A segment is one (request, KV head), a tile 16 keys of it (K and V).
// Segments stream whole or are cut into pieces of equal length (theta_piece),
// one piece per CTA; a CTA of NW warps gives each warp a run of the piece's
// tiles and merges the warps' states in shared memory.  Few segments run on CTAs
// that fill an SM (16 warps at D = 128, 8 at 256), more of them on CTAs of a
// half or a quarter of that: uniform batches of 608 segments reach 4.5 TB/s
// (1680 tokens, D = 128) to 5.5 TB/s (6720 tokens) that way.  Batches of more
// requests than the plan has room for (kMaxBatch) are not cut: 704 requests of 64
// tokens but for one of 100000 take 41 us (D = 128), 705 take 637; 712 and 713 at
// D = 256 111 and 1789.
//
// Times here and below: calls in a captured graph, three input sets in turn
// unless another condition stands beside them.
//
// Loads.  Every warp streams its own tiles: cp.async, 16 bytes a lane, into
// its own ring of STAGES tiles in shared memory, so no other warp is waited
// for inside a piece.  Streaming random 1152-byte units: 5.6 TB/s with cp.async
// against 4.9 TB/s with one bulk copy per unit.  Four tiles a warp in flight; five
// or six were slower (4 x 32..131 K keys: 43.3, 44.5, 45.1 us).
//
// What bounds it: HBM.  With long segments a tile takes an SM 56 ns (D = 128)
// or 111 ns (D = 256), 6.2 TB/s over the GPU, 92% of a plain copy, at 298 and
// 489 instructions and 2.8 and 2.3 of 4 a cycle (the difference of 2048 and 6144
// tokens, 152 segments).  Around that lie about 4 us from the launch to the first
// tiles, 1.5 us for the warps' merge and, where segments are cut, 3 us for the
// merge through global memory.  A logit cap costs the serving layer 0.7 us.
//
// Arithmetic per tile and warp: S^T = K q^T and O^T += V^T P^T with m16n8k16
// f16 MMAs (keys or channels on M, the G <= 8 query heads on N).  Codes go
// straight from 16-byte shared-memory loads to A fragments: cvt.f16x2.e2m1x2
// gives two values, one mul.f16x2 applies the e4m3 scale (code * scale has at
// most 6 significant bits and lies in [2^-10, 2688]: exact in f16).  K's pairs are
// two channels of a key; V's are one channel of two keys, for which the
// nibbles of the two keys are interleaved before the conversion.  q is f16
// after a power-of-two scaling per head that brings its largest element to
// [1, 2): exact but for elements below 2^-17 of the largest, whose error
// (2^-25 of the largest) is that of fp32 sums.  K's pool scale, the softmax
// scale and q's power of two are one fp32 factor on the logits; V's pool
// scale multiplies the finished result.
//
// Softmax in the exp2 domain with a reference m per head that all lanes
// share; it moves (and O is rescaled) only when a logit exceeds it by more
// than kGrow, so most tiles need one vote instead of a maximum over the warp.
// P = 2^(x - m + kShift) lies in (0, 2^15]: f16 (11 bits, the only rounding
// of P), of use down to 2^-32 of the largest weight.  The weights' sums are
// taken over the rounded values, in fp32 on the tensor cores.
#include <algorithm>

#include "decode_body.cuh"
#include "kv4.cuh"
#include "overlap.cuh"

namespace pka {

namespace {

// When no segment can be longer than this many tiles, none is cut: a merge
// through global memory costs about 3 us.  (16 segments of one length, us whole /
// cut: D = 128, 1024 tokens 7.6 / 8.2, 1152 8.6 / 8.3, 1600 10.4 / 8.5; D = 256,
// 640 tokens 8.6 / 8.8, 800 10.3 / 8.9.)
// The half-SM CTAs take half of it.  (200 segments of 1..n tokens: D = 128, n =
// 576 7.9 / 9.7, 768 9.1 / 10.2, 1024 10.9 / 11.1, 1536 14.5 / 12.9; D = 256, n =
// 320 8.2 / 11.3, 512 10.7 / 12.3, 768 14.0 / 14.1: the two cross at 64 and 48
// tiles only.)
constexpr int whole_tiles(int head_dim) { return head_dim == 128 ? 72 : 40; }
// The same for the small CTAs of large batches.  (608 segments of 1..n tokens:
// D = 128, n = 960 18.8 / 19.9, 1440 25.4 / 25.6, 1920 31.4 / 31.2; D = 256, n =
// 960 32.2 / 37.2, 1920 56.8 / 62.7: past 60 tiles the two are alike at D = 128,
// at 256 whole segments stay ahead.)
constexpr int kSmallWhole = 60;
// Pieces beyond one for each segment, when the segments are more than run at
// once.  (800 segments, none / 64 / 200 of them: D = 128, 16..2000 tokens 40.4 /
// 40.9 / 41.2 us; D = 256, 1..1500 tokens 65.0 / 63.2 / 62.6.)
constexpr int kMoreThan = 64;
// Else the shortest piece, in tiles.  (16 segments, 8 / 16 / 32 tiles: D = 128,
// 1280 tokens 8.6 / 8.6 / 8.8 us; D = 256, 800 tokens 9.5 / 9.0 / 9.9, 1280 11.2 /
// 9.7 / 10.7, 2560 12.0 / 12.0 / 11.6.)
constexpr int kMinPiece = 16;

constexpr float kGrow = 7.f;
constexpr float kShift = 8.f;

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same from zero.
__device__ __forceinline__ void mma_f16_16816_first(float (&d)[4], uint32_t a0, uint32_t a1,
                                                    uint32_t a2, uint32_t a3, uint32_t b0,
                                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Orders the CTA's partials (behind a barrier) before its arrival, and the
// other pieces' partials before what follows the last one.
__device__ __forceinline__ int atomic_add_acq_rel(int32_t* p, int32_t v) {
  int32_t old;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], %2;"
               : "=r"(old)
               : "l"(p), "r"(v)
               : "memory");
  return old;
}

// Transpose of an 8x8 matrix of 16-bit values held two per lane.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// 16 bytes global -> shared; `bytes` 16, or 0 for zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A CTA of NW warps with STAGES tiles in flight each, CTAS of them per SM; PW
// warps of it work the plan out; LENS: requests whose lengths it has room for.
template <int D, int NW_, int STAGES_, int CTAS_, int PW_, int LENS_>
struct Kv4Shape {
  static constexpr int NW = NW_, STAGES = STAGES_, CTAS = CTAS_, PW = PW_, LENS = LENS_;
  static constexpr int kMaxBatch = LENS - 4 * PW;   // (a warp's share of them is a multiple of 4)
  static constexpr int UNITS = D / kUnitChannels;
  static constexpr int kTile = UNITS * kUnitBytes;  // one block and head of K (or V)
  static constexpr int kFrags = UNITS * 4 * 2 * 32; // float4 of a warp's O state
  static constexpr int kItems = (kFrags + NW * 32 - 1) / (NW * 32);
  // Shared memory: the warps' rings, into which each warp's O state goes at the
  // end and then the threads' states of the pieces' merge; lengths and tiles of
  // the requests; the plan's sums; the warps' (max, sum) per head; the piece and
  // a flag; q as B fragments.
  static constexpr int kWarpRing = STAGES * 2 * kTile;
  static constexpr int kLen = NW * kWarpRing;
  static constexpr int kScr = kLen + 2 * LENS * 4;
  static constexpr int kMl = kScr + PW * 32 * 4 + (PW + 1) / 2 * 16;
  static constexpr int kPlan = kMl + NW * 8 * 8;
  static constexpr int kQ = kPlan + (sizeof(Piece) + 4 + 15) / 16 * 16;
  static constexpr int kSmem = kQ + UNITS * 8 * 32 * 8;
  static_assert(NW <= 16 && LENS % 4 == 0, "");
  static_assert(kWarpRing >= kFrags * 16 && kLen >= NW * 32 * (16 + 8), "the states fit the rings");
  static_assert(kSmem <= 232448 / CTAS - 1024, "shared memory of a CTA");
};

// The four A registers of K's k-step S (0..7) of a unit: words of row g and
// row g + 8, scaled.
template <int S, bool FIRST>
__device__ __forceinline__ void k_step(float (&acc)[4], const uint4& r0, const uint4& r1,
                                       const uint32_t (&s0)[2], const uint32_t (&s1)[2],
                                       uint32_t b0, uint32_t b1) {
  constexpr int B = (S & 1) * 2;
  const uint32_t w0 = (S / 2 == 0) ? r0.x : (S / 2 == 1) ? r0.y : (S / 2 == 2) ? r0.z : r0.w;
  const uint32_t w1 = (S / 2 == 0) ? r1.x : (S / 2 == 1) ? r1.y : (S / 2 == 2) ? r1.z : r1.w;
  const uint32_t a0 = f16x2_mul(e2m1x2_to_f16x2<B>(w0), s0[S / 4]);
  const uint32_t a1 = f16x2_mul(e2m1x2_to_f16x2<B>(w1), s1[S / 4]);
  const uint32_t a2 = f16x2_mul(e2m1x2_to_f16x2<B + 1>(w0), s0[S / 4]);
  const uint32_t a3 = f16x2_mul(e2m1x2_to_f16x2<B + 1>(w1), s1[S / 4]);
  if constexpr (FIRST)
    mma_f16_16816_first(acc, a0, a1, a2, a3, b0, b1);
  else
    mma_f16_16816(acc, a0, a1, a2, a3, b0, b1);
}

// M-tile of byte B of a V word: channels 2B and 2B + 1 of the word.
template <int B>
__device__ __forceinline__ void v_step(float (&o)[4], uint32_t lo0, uint32_t hi0, uint32_t lo1,
                                       uint32_t hi1, uint32_t sa, uint32_t sb, uint32_t p0,
                                       uint32_t p1) {
  mma_f16_16816(o, f16x2_mul(e2m1x2_to_f16x2<B>(lo0), sa), f16x2_mul(e2m1x2_to_f16x2<B>(hi0), sa),
                f16x2_mul(e2m1x2_to_f16x2<B>(lo1), sb), f16x2_mul(e2m1x2_to_f16x2<B>(hi1), sb), p0,
                p1);
}

// S^T of NT tiles for one warp.  Fragment roles (g = lane / 4, t = lane % 4):
// the rows are keys g and g + 8, the lane's channels 32 t .. 32 t + 31 of every
// unit; S^T holds those keys of heads 2t and 2t + 1.  bq: the CTA's q fragments
// in shared memory, [UNITS][8 k-steps][32 lanes].
template <int D, int NT>
__device__ __forceinline__ void kv4_scores(const uint8_t* const (&tile)[NT], const uint2* bq,
                                           float (&x)[NT][4], int lane) {
  constexpr int UNITS = D / kUnitChannels;
  float s[UNITS][NT][4];  // one chain of MMAs per unit and tile
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    uint4 r0[NT], r1[NT];
    uint32_t s0[NT][2], s1[NT][2];
#pragma unroll
    for (int k = 0; k < NT; ++k) {
      const uint8_t* base = tile[k] + u * kUnitBytes;
      r0[k] = *reinterpret_cast<const uint4*>(base + lane * 16);
      r1[k] = *reinterpret_cast<const uint4*>(base + 512 + lane * 16);
      // scales of groups 2t and 2t + 1 of key g: byte 8 g + 2 t = 2 lane
      const uint32_t c0 =
          e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(base + kUnitCodes + lane * 2));
      const uint32_t c1 =
          e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(base + kUnitCodes + 64 + lane * 2));
      s0[k][0] = prmt(c0, c0, 0x1010u);
      s0[k][1] = prmt(c0, c0, 0x3232u);
      s1[k][0] = prmt(c1, c1, 0x1010u);
      s1[k][1] = prmt(c1, c1, 0x3232u);
    }
    const uint2* q = bq + u * 8 * 32 + lane;
#define PKA_KV4_STEP(K_)                                                                \
  {                                                                                     \
    const uint2 b = q[(K_) * 32];                                                       \
    _Pragma("unroll") for (int k = 0; k < NT; ++k)                                      \
        k_step<K_, (K_) == 0>(s[u][k], r0[k], r1[k], s0[k], s1[k], b.x, b.y);           \
  }
    PKA_KV4_STEP(0)
    PKA_KV4_STEP(1)
    PKA_KV4_STEP(2)
    PKA_KV4_STEP(3)
    PKA_KV4_STEP(4)
    PKA_KV4_STEP(5)
    PKA_KV4_STEP(6)
    PKA_KV4_STEP(7)
#undef PKA_KV4_STEP
  }
#pragma unroll
  for (int k = 0; k < NT; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) x[k][i] = UNITS == 1 ? s[0][k][i] : s[0][k][i] + s[UNITS - 1][k][i];
}

// O^T += V^T P^T of one tile.  The lane holds group g of every unit for keys
// 2t, 2t + 1, 2t + 8, 2t + 9; O^T its 16 channels of heads 2t and 2t + 1.
// keep: byte masks of the scales of the four keys (0: an invisible key, whose
// stale scale may be NaN).
template <int D, bool EDGE>
__device__ __forceinline__ void kv4_values(const uint8_t* tile, float (&o)[D / 128][8][4],
                                           uint32_t pb0, uint32_t pb1, uint32_t keep0,
                                           uint32_t keep1, int lane) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int u = 0; u < D / kUnitChannels; ++u) {
    const uint8_t* base = tile + u * kUnitBytes;
    const uint8_t* row = base + g * 128;
    const int at = (t * 16) ^ ((g & 1) * 64);
    const uint4 a = *reinterpret_cast<const uint4*>(row + at);         // keys 2t (x, y), 2t + 1
    const uint4 b = *reinterpret_cast<const uint4*>(row + (at ^ 64));  // keys 2t + 8, 2t + 9
    const uint8_t* sc = base + kUnitCodes + g * 16 + t * 2;
    uint32_t ca = *reinterpret_cast<const uint16_t*>(sc);
    uint32_t cb = *reinterpret_cast<const uint16_t*>(sc + 8);
    if constexpr (EDGE) {
      ca &= keep0;
      cb &= keep1;
    }
    const uint32_t sa = e4m3x2_to_f16x2(static_cast<uint16_t>(ca));
    const uint32_t sb = e4m3x2_to_f16x2(static_cast<uint16_t>(cb));
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t a0 = j ? a.y : a.x, a1 = j ? a.w : a.z;
      const uint32_t b0 = j ? b.y : b.x, b1 = j ? b.w : b.z;
      // nibble pairs (key 2t, key 2t + 1) of the even and the odd channels
      const uint32_t alo = (a0 & 0x0f0f0f0fu) | ((a1 << 4) & 0xf0f0f0f0u);
      const uint32_t ahi = ((a0 >> 4) & 0x0f0f0f0fu) | (a1 & 0xf0f0f0f0u);
      const uint32_t blo = (b0 & 0x0f0f0f0fu) | ((b1 << 4) & 0xf0f0f0f0u);
      const uint32_t bhi = ((b0 >> 4) & 0x0f0f0f0fu) | (b1 & 0xf0f0f0f0u);
      v_step<0>(o[u][j * 4 + 0], alo, ahi, blo, bhi, sa, sb, pb0, pb1);
      v_step<1>(o[u][j * 4 + 1], alo, ahi, blo, bhi, sa, sb, pb0, pb1);
      v_step<2>(o[u][j * 4 + 2], alo, ahi, blo, bhi, sa, sb, pb0, pb1);
      v_step<3>(o[u][j * 4 + 3], alo, ahi, blo, bhi, sa, sb, pb0, pb1);
    }
  }
}

// x <- cap * tanh(x / cap) for a lane's log2-domain logits; in: ln 2 / cap,
// out: cap * log2 e.  tanh(y) = 1 - 2 / (e^{2y} + 1) has an absolute error of up
// to 7e-7, which the cap multiplies, so that it serves from |y| = 1/4 on only;
// below it the logit is x (1 - y^2/3 + 2 y^4/15 - 17 y^6/315 + 62 y^8/2835), next
// term under 2^-26.  The error is at most 2^-18 of the logit whatever the cap.
// The exp2 form is left out where no logit of the warp wants it: the serving
// layer with a cap of 50 takes 17.0 us that way, with both forms for every logit
// 17.4 (one input set); with logits that all want it 20.5 in place of 19.9 (three).
// NaN stays NaN.
template <int NT>
__device__ __forceinline__ void cap_logits(float (&x)[NT][4], float in, float out) {
  float top = 0.f, y[NT][4];
#pragma unroll
  for (int k = 0; k < NT; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[k][i] = x[k][i] * in;
      const float y2 = y[k][i] * y[k][i];
      float p = fmaf(y2, 62.f / 2835.f, -17.f / 315.f);
      p = fmaf(y2, p, 2.f / 15.f);
      p = fmaf(y2, p, -1.f / 3.f);
      x[k][i] = fmaf(x[k][i] * y2, p, x[k][i]);
      top = fmaxf(top, fabsf(y[k][i]));
    }
  if (__any_sync(0xffffffffu, top >= 0.25f)) {
#pragma unroll
    for (int k = 0; k < NT; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float e = fast_exp2(min_nan(2.f * kLog2e * y[k][i], 126.f));
        const float far = out * (1.f - __fdividef(2.f, e + 1.f));
        x[k][i] = fabsf(y[k][i]) < 0.25f ? x[k][i] : far;
      }
  }
}

// NT tiles for one warp: scores, softmax step, values.  EDGE (NT = 1): the
// tile holds keys outside [t_lo, pos].
template <int D, int NT, bool EDGE, bool CAP>
__device__ __forceinline__ void kv4_tiles(const uint8_t* const (&tile)[NT],
                                          const uint2* bq, float (&o)[D / 128][8][4],
                                          float (&m)[2], float (&l)[4],
                                          float f0, float f1, float cap_in, float cap_out,
                                          int tok0, int t_lo, int pos, int lane) {
  constexpr int UNITS = D / kUnitChannels;
  static_assert(!EDGE || NT == 1, "an edge tile goes alone");
  const int g = lane >> 2, t = lane & 3;
  float x[NT][4];
  kv4_scores<D, NT>(tile, bq, x, lane);
  uint32_t keep0 = 0xffffu, keep1 = 0xffffu;
  bool ok_lo = true, ok_hi = true;
  if constexpr (EDGE) {
    const int lo = t_lo - tok0, hi = pos - tok0;  // visible: lo <= key <= hi
    ok_lo = g >= lo && g <= hi;
    ok_hi = g + 8 >= lo && g + 8 <= hi;
    const int k0 = 2 * t;
    keep0 = (k0 >= lo && k0 <= hi ? 0xffu : 0u) | (k0 + 1 >= lo && k0 + 1 <= hi ? 0xff00u : 0u);
    keep1 = (k0 + 8 >= lo && k0 + 8 <= hi ? 0xffu : 0u) |
            (k0 + 9 >= lo && k0 + 9 <= hi ? 0xff00u : 0u);
  }
#pragma unroll
  for (int k = 0; k < NT; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) x[k][i] *= (i & 1) ? f1 : f0;
  if constexpr (CAP) cap_logits<NT>(x, cap_in, cap_out);
  float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll
  for (int k = 0; k < NT; ++k) {
    if constexpr (EDGE) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (!((i & 2) ? ok_hi : ok_lo)) x[k][i] = -INFINITY;
    }
    top0 = fmaxf(top0, fmaxf(x[k][0], x[k][2]));
    top1 = fmaxf(top1, fmaxf(x[k][1], x[k][3]));
  }
  if (__any_sync(0xffffffffu, top0 > m[0] + kGrow || top1 > m[1] + kGrow)) {
    float alpha[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float mx = j ? top1 : top0;
#pragma unroll
      for (int off = 4; off < 32; off <<= 1)
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      const float mn = fmaxf(m[j], mx);
      alpha[j] = (mn == -INFINITY) ? 1.f : fast_exp2(m[j] - mn);
      m[j] = mn;
      l[j] *= alpha[j];
      l[2 + j] *= alpha[j];
    }
#pragma unroll
    for (int u = 0; u < UNITS; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        o[u][i][0] *= alpha[0];
        o[u][i][1] *= alpha[1];
        o[u][i][2] *= alpha[0];
        o[u][i][3] *= alpha[1];
      }
  }
  // a head whose keys so far are all invisible or NaN keeps m = -inf
  const float r0 = (m[0] == -INFINITY) ? 0.f : m[0] - kShift;
  const float r1 = (m[1] == -INFINITY) ? 0.f : m[1] - kShift;
#pragma unroll
  for (int k = 0; k < NT; ++k) {
    const float p0 = fast_exp2(x[k][0] - r0), p1 = fast_exp2(x[k][1] - r1);
    const float p2 = fast_exp2(x[k][2] - r0), p3 = fast_exp2(x[k][3] - r1);
    const uint32_t pb0 = movmatrix_trans(pack_f16x2(p0, p1));  // keys 2t, 2t + 1 of head g
    const uint32_t pb1 = movmatrix_trans(pack_f16x2(p2, p3));  // keys 2t + 8, 2t + 9
    // the weights' sums, of the rounded weights as the values see them: ones
    // times P^T, every row of it the same
    mma_f16_16816(l, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u, pb0, pb1);
    kv4_values<D, EDGE>(tile[k] + UNITS * kUnitBytes, o, pb0, pb1, keep0, keep1, lane);
  }
}

// The plan: one piece per CTA, so that no CTA pays a piece's fixed cost twice.
// theta is the smallest of 32 lengths with sum over segments (request, KV head)
// of ceil(n / theta) <= CTAs; segment n gets that many pieces of equal length
// (one: its output is written without partials).  Every CTA computes the same
// plan from the lengths: each warp sums its share of the requests for all 32
// lengths, one per lane.  nbf holds the segments' tiles (an empty one counts a
// half, so that it gets a piece of its own).
__device__ __forceinline__ int theta_parts(float nb, float rtheta) {
  // 2^23 + ceil(nb * rtheta), rounded up
  return __float_as_int(__fmaf_ru(nb, rtheta, 8388608.f)) - 0x4b000000;
}

// Finds piece `cta` and writes it to *plan (fill_from: whether there is one).
// The first PW warps take part; the caller's barrier makes the result visible.
template <typename S>
__device__ __forceinline__ void theta_piece(const Kv4DecodeArgs& ka, uint8_t* smem, int cta,
                                            Piece* plan) {
  constexpr int PW = S::PW;
  const DecodeArgs& a = ka.base;
  int* slen = reinterpret_cast<int*>(smem + S::kLen);
  float* nbf = reinterpret_cast<float*>(slen + S::LENS);
  int* sums = reinterpret_cast<int*>(smem + S::kScr);    // [PW][32]
  int2* red = reinterpret_cast<int2*>(sums + PW * 32);  // [PW]
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int share = ((a.batch + PW - 1) / PW + 3) / 4 * 4;  // requests of a warp
  // 24 steps from the even share to twice of it, which fits whenever the
  // segments number at most half the CTAs, then 6 up to the longest, then one
  // piece each, which always fits
  const float near = __fdividef(24.f, 24.f + lane);
  int tiles = 0, longest = 0;
  auto sync = [&]() {
    if constexpr (PW == 1)
      __syncwarp();
    else
      named_sync(1, PW * 32);
  };
#pragma unroll 4
  for (int b = threadIdx.x; b < PW * share; b += PW * 32) {
    const int len = b < a.batch ? req_len_of(a, 0, 0, a.seq_lens[b]) : 0;
    const int nb = geo_of_len(a, len).nb;
    slen[b] = len;
    nbf[b] = b < a.batch ? fmaxf(static_cast<float>(nb), 0.5f) : 0.f;
    tiles += nb;
    longest = max(longest, nb);
  }
  tiles = __reduce_add_sync(0xffffffffu, tiles);
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (threadIdx.x == 0) plan->fill_from = 0;
  if (PW > 1 && lane == 0) red[warp] = make_int2(tiles, longest);
  sync();
  if constexpr (PW > 1) {
    const int2 r = lane < PW ? red[lane] : make_int2(0, 0);
    tiles = __reduce_add_sync(0xffffffffu, r.x);
    longest = __reduce_max_sync(0xffffffffu, r.y);
  }
  // the even share, at least split_blocks (which bounds the workspace's slots)
  // and kMinPiece tiles
  const float lo = fmaxf(static_cast<float>(max(a.split_blocks, kMinPiece)),
                         static_cast<float>(tiles) * ka.even_share);
  const float hi = fmaxf(static_cast<float>(longest), 2.f * lo);
  float rtheta = lane < 25 ? __fdividef(near, lo)
                           : __fdividef(1.f, 2.f * lo + (hi - 2.f * lo) * ((lane - 24) * (1.f / 7.f)));
  if (lane == 31) rtheta = __fdividef(0.999f, hi);
  auto parts_of = [&](float nb) { return min(theta_parts(nb, rtheta), a.num_splits); };
  int sum = 0;
#pragma unroll 4
  for (int i = 0; i < share; i += 4) {  // (padded with zeros, which give none)
    const float4 n = *reinterpret_cast<const float4*>(nbf + warp * share + i);
    sum += parts_of(n.x) + parts_of(n.y) + parts_of(n.z) + parts_of(n.w);
  }
  if constexpr (PW > 1) {
    sums[warp * 32 + lane] = sum;
    sync();
    if (warp != 0) return;
    sum = 0;
#pragma unroll
    for (int w = 0; w < PW; ++w) sum += sums[w * 32 + lane];
  }
  const int chosen = __ffs(__ballot_sync(0xffffffffu, sum <= ka.most_parts)) - 1;
  rtheta = __shfl_sync(0xffffffffu, rtheta, chosen);
  // pieces lie in (request, head, part) order: the share that has piece `cta`,
  // then in it the lane whose request has it
  int w = 0, before = 0;
  if constexpr (PW > 1) {
    const int mine = lane < PW ? sums[lane * 32 + chosen] * a.Hkv : 0;
    const int upto = warp_incl_scan(mine, lane);
    const unsigned m = __ballot_sync(0xffffffffu, cta < upto);
    if (m == 0) return;
    w = __ffs(m) - 1;
    before = __shfl_sync(0xffffffffu, upto - mine, w);
  }
  for (int i = 0; i < share; i += 32) {
    const bool in_share = i + lane < share;
    const int b = w * share + (in_share ? i + lane : 0);
    const int parts = in_share ? parts_of(nbf[b]) : 0;
    const ReqGeo geo = geo_of_len(a, slen[b]);
    const int incl = warp_incl_scan(parts * a.Hkv, lane) + before;
    const int in = cta - (incl - parts * a.Hkv);
    if (in >= 0 && cta < incl) {
      const float rparts = __fdividef(1.f, static_cast<float>(parts));
      Piece p;
      p.b = p.qrow = b;
      p.kvh = static_cast<int>((static_cast<float>(in) + 0.5f) * rparts);
      p.slot = in - p.kvh * parts;
      p.npieces = parts;
      // piece k starts at tile floor(k * n / parts), in fp32 and the same for
      // both pieces that meet there
      const float each = static_cast<float>(geo.nb) * rparts;
      const int t0 = min(static_cast<int>(each * p.slot), geo.nb);
      const int t1 =
          p.slot + 1 == parts ? geo.nb : min(static_cast<int>(each * (p.slot + 1)), geo.nb);
      p.j0 = geo.jlo + t0;
      p.ntiles = t1 - t0;
      p.t_lo = geo.t_lo;
      p.pos = geo.pos;
      p.fill_from = 1;
      *plan = p;
    }
    before = __shfl_sync(0xffffffffu, incl, 31);
  }
}

template <int D, typename S, bool CAP>
__global__ void __launch_bounds__(S::NW * 32, S::CTAS)
    kv4_decode_kernel(const __grid_constant__ Kv4DecodeArgs ka) {
  constexpr int UNITS = S::UNITS, NW = S::NW, STAGES = S::STAGES;
  extern __shared__ __align__(128) uint8_t smem[];
  const DecodeArgs& a = ka.base;
  const int G = a.Hq / a.Hkv;
  float2* ml = reinterpret_cast<float2*>(smem + S::kMl);  // [NW][8]
  Piece* plan = reinterpret_cast<Piece*>(smem + S::kPlan);
  volatile int* flag = reinterpret_cast<int*>(plan + 1);
  uint2* bq = reinterpret_cast<uint2*>(smem + S::kQ);      // [UNITS][8][32]
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * S::kWarpRing;
  const uint32_t ring_addr = smem_u32(ring);
  const int cta = static_cast<int>(blockIdx.x);

  launch_dependents();
  wait_predecessor();
  if (ka.whole) {
    // no segment is cut: piece c is segment c
    if (threadIdx.x == 0) {
      Piece p{};
      p.fill_from = cta < a.batch * a.Hkv;
      if (p.fill_from != 0) {
        p.b = cta / a.Hkv;
        p.kvh = cta - p.b * a.Hkv;
        const ReqGeo geo = geo_of_len(a, req_len_of(a, 0, 0, a.seq_lens[p.b]));
        p.j0 = geo.jlo;
        p.ntiles = geo.nb;
        p.t_lo = geo.t_lo;
        p.pos = geo.pos;
        p.qrow = p.b;
        p.npieces = 1;
      }
      *plan = p;
    }
  } else if (warp < S::PW) {
    theta_piece<S>(ka, smem, cta, plan);
  }
  __syncthreads();
  Piece pc = *plan;
  if (pc.fill_from == 0) return;
  // (log2-domain logits; a cap near 0 would give an infinite factor, and NaN
  // for a logit of 0)
  const float lscale = a.scale * ka.k_scale * kLog2e;
  const float cap_in = fminf(kLn2 / a.softcap, kFltMax), cap_out = a.softcap * kLog2e;

  // this warp's tiles of the piece: first .. first + mine - 1
  const int first = pc.ntiles * warp / NW, mine = pc.ntiles * (warp + 1) / NW - first;
  int ids = 0;  // block ids of its tiles base .. base + 31, one per lane
  auto load_ids = [&](int base) {
    const int i = base + lane;
    int id = -1;
    if (i < mine) {
      id = a.tables[static_cast<size_t>(pc.b) * a.max_blocks + pc.j0 + first + i];
      if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.num_blocks)) {
        report(a.err, PKA_DEVERR_BAD_TABLE);
        id = -1;
      }
    }
    return id;
  };
  // requests the warp's tile n (its id in lane n % 32 of ids)
  auto issue = [&](int n) {
    const int id = __shfl_sync(0xffffffffu, ids, n & 31);
    const uint32_t bytes = id >= 0 ? 16u : 0u;  // a bad id reads as zeros
    const long long off =
        (static_cast<long long>(max(id, 0)) * a.Hkv + pc.kvh) * S::kTile;
    const uint32_t dst = ring_addr + (n % STAGES) * 2 * S::kTile;
#pragma unroll
    for (int c = 0; c < S::kTile / 512; ++c) {
      cp_async16(dst + c * 512 + lane * 16, ka.k4 + off + c * 512 + lane * 16, bytes);
      cp_async16(dst + S::kTile + c * 512 + lane * 16, ka.v4 + off + c * 512 + lane * 16, bytes);
    }
    // the last S::kTile % 512 bytes of K and of V
    constexpr int kRest = S::kTile % 512 / 16;
    constexpr int kFrom = S::kTile / 512 * 512;
    if (lane < 2 * kRest) {
      const bool v = lane >= kRest;
      const int c = kFrom + (v ? lane - kRest : lane) * 16;
      cp_async16(dst + (v ? S::kTile : 0) + c, (v ? ka.v4 : ka.k4) + off + c, bytes);
    }
  };
  ids = load_ids(0);
#pragma unroll
  for (int n = 0; n < STAGES; ++n) {
    if (n < mine) issue(n);
    cp_async_commit();
  }

  // ---- q of head g as B fragments in f16, scaled by a power of two: every
  // warp finds the head's largest magnitude and writes its share for the CTA
  float fq;  // the logit factor of head g
  {
    const uint16_t* qp =
        a.q + (static_cast<size_t>(pc.qrow) * a.Hq + pc.kvh * G + (g < G ? g : 0)) * D + t * 32;
    uint4 raw[UNITS * 4];
    uint32_t top2 = 0;
#pragma unroll
    for (int i = 0; i < UNITS * 4; ++i) {
      raw[i] = (g < G) ? *reinterpret_cast<const uint4*>(
                             qp + (i >> 2) * kUnitChannels + (i & 3) * 8)
                       : make_uint4(0u, 0u, 0u, 0u);
      top2 = __vmaxu2(__vmaxu2(raw[i].x & 0x7fff7fffu, raw[i].y & 0x7fff7fffu),
                      __vmaxu2(__vmaxu2(raw[i].z & 0x7fff7fffu, raw[i].w & 0x7fff7fffu), top2));
    }
    uint32_t top = max(top2 & 0xffffu, top2 >> 16);  // as bf16 bits
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int e = min(max(254 - static_cast<int>(top >> 7), 1), 253);
    const float down = __uint_as_float(static_cast<uint32_t>(e) << 23);
    fq = lscale * __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
#pragma unroll
    for (int i = 0; i < UNITS * 4; ++i) {
      if (i % NW != warp) continue;
      float f[8];
      unpack8(raw[i], f);
#pragma unroll
      for (int k = 0; k < 2; ++k)
        bq[(i * 2 + k) * 32 + lane] =
            make_uint2(pack_f16x2(f[k * 4] * down, f[k * 4 + 1] * down),
                       pack_f16x2(f[k * 4 + 2] * down, f[k * 4 + 3] * down));
    }
    __syncthreads();
  }
  const float f0 = __shfl_sync(0xffffffffu, fq, 8 * t);
  const float f1 = __shfl_sync(0xffffffffu, fq, 8 * t + 4);

  float o[UNITS][8][4];
#pragma unroll
  for (int u = 0; u < UNITS; ++u)
#pragma unroll
    for (int i = 0; i < 8; ++i) o[u][i][0] = o[u][i][1] = o[u][i][2] = o[u][i][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[4] = {0.f, 0.f, 0.f, 0.f};

  // Invariant: tiles n .. n + STAGES - 1 are requested, one group each (empty
  // groups behind the last).
  const int count = mine, tok_first = (pc.j0 + first) * kBlockSize;
  int n = 0;
  auto is_edge = [&](int k) {
    const int tok0 = tok_first + k * kBlockSize;
    return tok0 < pc.t_lo || tok0 + kBlockSize - 1 > pc.pos;
  };
  auto refill = [&](int k) {  // the slot of tile k is free
    const int ahead = k + STAGES;
    if (ahead < count) {
      if ((ahead & 31) == 0) ids = load_ids(ahead);
      issue(ahead);
    }
    cp_async_commit();
  };
  while (n < count) {
    const uint8_t* t0 = ring + (n % STAGES) * 2 * S::kTile;
    if (n + 1 < count && !is_edge(n) && !is_edge(n + 1)) {
      cp_async_wait<STAGES - 2>();
      __syncwarp();  // every lane's part of the tiles has landed
      const uint8_t* const tiles[2] = {t0, ring + ((n + 1) % STAGES) * 2 * S::kTile};
      kv4_tiles<D, 2, false, CAP>(tiles, bq, o, m, l, f0, f1, cap_in, cap_out, 0, 0, 0,
                                  lane);
      __syncwarp();
      refill(n);
      refill(n + 1);
      n += 2;
    } else {
      cp_async_wait<STAGES - 1>();
      __syncwarp();
      const uint8_t* const tiles[1] = {t0};
      kv4_tiles<D, 1, true, CAP>(tiles, bq, o, m, l, f0, f1, cap_in, cap_out,
                                 tok_first + n * kBlockSize, pc.t_lo, pc.pos, lane);
      __syncwarp();
      refill(n);
      ++n;
    }
  }

  // ---- the warps' states merged in warp order: (max, sum) first, from which
  // every warp takes the factor of its own O, then the sum of the scaled O
  // states through shared memory (a warp without tiles holds zeros)
  if (g == 0) {
    ml[warp * 8 + 2 * t] = make_float2(m[0], l[0]);
    ml[warp * 8 + 2 * t + 1] = make_float2(m[1], l[1]);
  }
  __syncthreads();
  pc = *plan;  // not kept in registers over the loop
  const bool split = pc.npieces > 1;
  // A sum of 0 means no visible key, whose output is 0, or logits that are all
  // -infinity, whose softmax is 0 / 0 (a piece of a cut segment leaves that to
  // the merge).
  const float no_sum = split || pc.ntiles == 0 ? 0.f : NAN;
  const size_t head0 = static_cast<size_t>(pc.qrow) * a.Hq + pc.kvh * G;
  // lane (g, t) takes warps g and g + 8
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float2 none = make_float2(-INFINITY, 0.f);
    const float2 v0 = g < NW ? ml[g * 8 + 2 * t + j] : none;
    const float2 v1 = g + 8 < NW ? ml[(g + 8) * 8 + 2 * t + j] : none;
    float M = fmaxf(v0.x, v1.x);
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    if (M == -INFINITY) M = 0.f;
    float den = ((v0.x == -INFINITY) ? 1.f : fast_exp2(v0.x - M)) * v0.y +
                ((v1.x == -INFINITY) ? 1.f : fast_exp2(v1.x - M)) * v1.y;
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) den += __shfl_xor_sync(0xffffffffu, den, off);
    const float f = den == 0.f ? no_sum
                               : ((m[j] == -INFINITY) ? 1.f : fast_exp2(m[j] - M)) *
                                     __fdividef(1.f, den);
    // P carries a factor 2^kShift, the same in every piece; a NaN sum keeps
    // its weight, so that the merge of the pieces passes it on
    if (split && warp == 0 && g == 0 && 2 * t + j < G)
      __stcg(a.partial_lse + (head0 + 2 * t + j) * a.num_splits + pc.slot,
             den == 0.f ? -INFINITY : (isnan(den) ? M : M + log2f(den)) * kLn2);
#pragma unroll
    for (int u = 0; u < UNITS; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        o[u][i][j] *= f;
        o[u][i][2 + j] *= f;
      }
  }
  // four normalised output columns of a row: V's pool scale comes last, since a
  // small one divided by the weights' sum would leave fp32's range
  auto store_scaled = [&](size_t row, int d0, const float4& y) {
    const float vs = ka.v_scale;
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + row * D + d0) =
        make_uint2(pack_bf16x2(y.x * vs, y.y * vs), pack_bf16x2(y.z * vs, y.w * vs));
  };
  auto state = [&](int w, int item) {
    return reinterpret_cast<const float4*>(smem + w * S::kWarpRing) + item;
  };
  if (2 * t < G) {
    float4* row = reinterpret_cast<float4*>(ring) + lane;  // every tile of it is consumed
#pragma unroll
    for (int u = 0; u < UNITS; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          row[((u * 4 + i) * 2 + j) * 32] =
              make_float4(o[u][2 * i][j], o[u][2 * i][2 + j], o[u][2 * i + 1][j],
                          o[u][2 * i + 1][2 + j]);
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < S::kItems; ++k) {
    const int item = threadIdx.x + k * NW * 32;
    const int il = item & 31, ij = (item >> 5) & 1, ii = (item >> 6) & 3, iu = item >> 8;
    const int h = 2 * (il & 3) + ij;
    const int d0 = iu * kUnitChannels + (il >> 2) * 16 + ii * 4;
    if (item >= S::kFrags || h >= G) continue;
    float4 y = *state(0, item);
#pragma unroll
    for (int w = 1; w < NW; ++w) {
      const float4 x = *state(w, item);
      y.x += x.x;
      y.y += x.y;
      y.z += x.z;
      y.w += x.w;
    }
    if (split)
      __stcg(reinterpret_cast<float4*>(a.partial_o +
                                       ((head0 + h) * a.num_splits + pc.slot) * D + d0),
             y);
    else
      store_scaled(head0 + h, d0, y);
  }
  if (split) {
    // ---- the piece that arrives last at its segment merges the partials
    const int np = pc.npieces;
    __syncthreads();
    if (threadIdx.x == 0) {
      // the segment's counter: the pieces beyond one each of the segments
      // before it, a number that every cut segment raises
      int32_t* counter = a.seg_counters + (cta - pc.slot) - (pc.b * a.Hkv + pc.kvh);
      const bool last = atomic_add_acq_rel(counter, 1) == np - 1;
      if (last) *counter = 0;
      *flag = last;
    }
    __syncthreads();
    if (*flag != 0) {
      // The threads of an output item (four columns of a head) take every
      // parts-th piece each, up to kFlight with all loads in flight, and fold
      // them into a state (M, den, acc); the states of an item are merged
      // through shared memory.
      constexpr int kRow = D / 4;
      constexpr int kFlight = D == 256 ? 4 : 8;
      const int items = G * kRow;
      const int parts = max(1, NW * 32 / items);
      auto finish = [&](int it, const float4& acc, float den) {
        const float inv = den == 0.f ? NAN : 1.f / den;  // (a cut segment has keys)
        store_scaled(head0 + it / kRow, it % kRow * 4,
                     make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
      };
      float4* st = reinterpret_cast<float4*>(smem);           // [NW * 32]
      float2* md = reinterpret_cast<float2*>(st + NW * 32);  // [NW * 32]
      for (int item = threadIdx.x; item < items * parts; item += NW * 32) {
        const int part = item / items, it = item - part * items;
        const size_t row = (head0 + it / kRow) * a.num_splits;
        const float* po = a.partial_o + row * D + it % kRow * 4;
        float M = -INFINITY, den = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int s0 = part; s0 < np; s0 += kFlight * parts) {
          float lv[kFlight];
          float4 x[kFlight];
#pragma unroll
          for (int k = 0; k < kFlight; ++k) {
            const int sk = min(s0 + k * parts, np - 1);
            lv[k] = __ldcg(a.partial_lse + row + sk);
            x[k] = __ldcg(reinterpret_cast<const float4*>(po + static_cast<size_t>(sk) * D));
          }
          float top = M;
#pragma unroll
          for (int k = 0; k < kFlight; ++k) {
            if (s0 + k * parts >= np) lv[k] = -INFINITY;
            top = fmaxf(top, lv[k]);
          }
          if (top == -INFINITY) continue;
          const float r = fast_exp2((M - top) * kLog2e);  // 0 while M = -inf
          M = top;
          den *= r;
          acc = make_float4(acc.x * r, acc.y * r, acc.z * r, acc.w * r);
#pragma unroll
          for (int k = 0; k < kFlight; ++k) {
            if (s0 + k * parts >= np) break;
            const float w = fast_exp2((lv[k] - top) * kLog2e);
            den += w;
            acc.x = fmaf(w, x[k].x, acc.x);
            acc.y = fmaf(w, x[k].y, acc.y);
            acc.z = fmaf(w, x[k].z, acc.z);
            acc.w = fmaf(w, x[k].w, acc.w);
          }
        }
        if (parts > 1) {
          st[item] = acc;
          md[item] = make_float2(M, den);
        } else {
          finish(it, acc, den);
        }
      }
      if (parts > 1) {
        __syncthreads();
        for (int it = threadIdx.x; it < items; it += NW * 32) {
          float M = -INFINITY;
          for (int k = 0; k < parts; ++k) M = fmaxf(M, md[k * items + it].x);
          float den = 0.f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int k = 0; k < parts; ++k) {
            const float2 v = md[k * items + it];
            const float4 z = st[k * items + it];
            const float w = v.x == -INFINITY ? 0.f : fast_exp2((v.x - M) * kLog2e);
            den = fmaf(w, v.y, den);
            acc.x = fmaf(w, z.x, acc.x);
            acc.y = fmaf(w, z.y, acc.y);
            acc.z = fmaf(w, z.z, acc.z);
            acc.w = fmaf(w, z.w, acc.w);
          }
          finish(it, acc, den);
        }
      }
    }
  }
  cp_async_wait<0>();
}

template <int D, typename S>
cudaError_t launch_t(Kv4DecodeArgs a, int64_t grid, cudaStream_t stream) {
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  a.most_parts = static_cast<int>(grid / a.base.Hkv);
  a.even_share = static_cast<float>(a.base.Hkv) / grid;
  auto kern = a.base.softcap > 0.f ? kv4_decode_kernel<D, S, true> : kv4_decode_kernel<D, S, false>;
  const cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kern), S::kSmem);
  if (e != cudaSuccess) return e;
  return launch_overlapped(kern, static_cast<int>(grid), S::NW * 32, S::kSmem, stream, a);
}

// Few segments: CTAs that fill an SM.  More segments than SMs: two or four
// smaller CTAs to an SM, so that most segments stay whole and one CTA's fixed
// costs pass behind another's loads; more than run at once: the hardware hands
// the CTAs out as others end.  The pieces number at most the CTAs that run at
// once, or some more than the segments, to cut the long ones.  Batches beyond
// the plan's shared memory are not cut.
template <int D, typename S>
cudaError_t launch_s(Kv4DecodeArgs a, int64_t segments, int sms, int whole, cudaStream_t stream) {
  a.whole = a.base.batch > S::kMaxBatch || a.max_tiles <= whole;
  if (a.whole) return launch_t<D, S>(a, segments, stream);
  const int64_t at_once = S::CTAS * sms;
  const int64_t pieces = S::CTAS < 4 ? at_once : std::max(at_once, segments + kMoreThan);
  return launch_t<D, S>(a, std::min<int64_t>(pieces, segments + kKv4MaxExtra), stream);
}

template <int D, typename Big, typename Mid, typename Small>
cudaError_t launch_d(const Kv4DecodeArgs& a, int sms, cudaStream_t stream) {
  const int64_t segments = static_cast<int64_t>(a.base.batch) * a.base.Hkv;
  if (segments <= sms) return launch_s<D, Big>(a, segments, sms, whole_tiles(D), stream);
  if (segments <= 2 * sms) return launch_s<D, Mid>(a, segments, sms, whole_tiles(D) / 2, stream);
  return launch_s<D, Small>(a, segments, sms, kSmallWhole, stream);
}

}  // namespace

cudaError_t launch_kv4_decode(const Kv4DecodeArgs& a, int head_dim, int sms, cudaStream_t stream) {
  if (head_dim == 128)
    return launch_d<128, Kv4Shape<128, 16, 4, 1, 1, 224>, Kv4Shape<128, 8, 4, 2, 4, 400>,
                    Kv4Shape<128, 4, 4, 4, 4, 720>>(a, sms, stream);
  if (head_dim == 256)
    return launch_d<256, Kv4Shape<256, 8, 4, 1, 1, 224>, Kv4Shape<256, 4, 4, 2, 4, 400>,
                    Kv4Shape<256, 2, 4, 4, 2, 720>>(a, sms, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pka
