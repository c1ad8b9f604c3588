// Paged decode attention over a 4-bit cache (sm_103a).
//
// One query token per request attends over its visible keys, held as e2m1
// codes with an e4m3 scale per 16 channels (kv4.cuh).  A key and its value
// cost 9 D / 8 bytes per KV head, 3.6 times fewer than in bf16, so the
// arithmetic per byte is 3.6 times that of the bf16 decode: the design keeps
// the conversion short and every other cost off the path.
//
// Work.  The split-K line of the bf16 decode (PieceIter: segments of
// (request, KV head) cut into equal chunks, one per CTA), one persistent CTA
// of NW warps per SM.  Warp w of a CTA takes tiles w, w + NW, ... of a piece
// (a tile: 16 keys of one head, K and V).
//
// Loads.  Every warp streams its own tiles: cp.async, 16 bytes a lane, into
// its own ring of STAGES tiles in shared memory, so no other warp is waited
// for inside a piece; the next piece's first tiles are requested before the
// current piece is merged.  (Streaming random 1152-byte units: 5.6 TB/s with
// cp.async against 4.9 TB/s with one bulk copy per unit.)
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
// (2^-25 of the largest) is that of fp32 sums.  Pool scales, the softmax
// scale and q's power of two are one fp32 factor on the logits; V's pool
// scale is applied once to the result.
//
// Softmax in the exp2 domain with a reference m per head that all lanes
// share; it moves (and O is rescaled) only when a logit exceeds it by more
// than kGrow, so most tiles need one vote instead of a maximum over the warp.
// P = 2^(x - m + kShift) lies in (0, 2^15]: f16 (11 bits, the only rounding
// of P), of use down to 2^-32 of the largest weight; the sums are fp32 over
// the unrounded values.
#include "decode_body.cuh"
#include "kv4.cuh"

namespace pka {

namespace {

constexpr float kGrow = 7.f;
constexpr float kShift = 8.f;

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
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

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint16_t lds16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
}

template <int D, int NW_, int STAGES_>
struct Kv4Shape {
  static constexpr int NW = NW_, STAGES = STAGES_;
  static constexpr int UNITS = D / kUnitChannels;
  static constexpr int kTile = UNITS * kUnitBytes;  // one block and head of K (or V)
  static constexpr int kRing = NW * STAGES * 2 * kTile;
  static constexpr int kLen = kLenCache * 4;
  // the warps' (max, sum) per head, and a flag
  static constexpr int kMl = NW * 8 * 8 + 16;
  static constexpr int smem(int G) { return kRing + kLen + kMl + NW * G * D * 4; }
};

// The four A registers of K's k-step S (0..7) of a unit: words of row g and
// row g + 8, scaled.
template <int S>
__device__ __forceinline__ void k_step(float (&acc)[4], const uint4& r0, const uint4& r1,
                                       const uint32_t (&s0)[2], const uint32_t (&s1)[2],
                                       uint32_t b0, uint32_t b1) {
  constexpr int B = (S & 1) * 2;
  const uint32_t w0 = (S / 2 == 0) ? r0.x : (S / 2 == 1) ? r0.y : (S / 2 == 2) ? r0.z : r0.w;
  const uint32_t w1 = (S / 2 == 0) ? r1.x : (S / 2 == 1) ? r1.y : (S / 2 == 2) ? r1.z : r1.w;
  mma_f16_16816(acc, f16x2_mul(e2m1x2_to_f16x2<B>(w0), s0[S / 4]),
                f16x2_mul(e2m1x2_to_f16x2<B>(w1), s1[S / 4]),
                f16x2_mul(e2m1x2_to_f16x2<B + 1>(w0), s0[S / 4]),
                f16x2_mul(e2m1x2_to_f16x2<B + 1>(w1), s1[S / 4]), b0, b1);
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

// One tile (16 keys of one head) for one warp.  Fragment roles (g = lane / 4,
// t = lane % 4): K rows are keys g and g + 8, the lane's channels 32 t ..
// 32 t + 31 of every unit; S^T holds those keys of heads 2t and 2t + 1; V's
// lane holds group g of every unit for keys 2t, 2t + 1, 2t + 8, 2t + 9, and
// O^T its 16 channels of heads 2t and 2t + 1.
template <int D>
__device__ __forceinline__ void kv4_tile(uint32_t tile, const uint32_t (&bq)[D / 128][8][2],
                                         float (&o)[D / 128][8][4], float (&m)[2], float (&l)[2],
                                         float f0, float f1, float softcap, float inv_cap,
                                         bool edge, int tok0, int t_lo, int pos, int lane) {
  constexpr int UNITS = D / kUnitChannels;
  const int g = lane >> 2, t = lane & 3;
  float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    const uint32_t base = tile + u * kUnitBytes;
    const uint4 r0 = lds128(base + lane * 16);
    const uint4 r1 = lds128(base + 512 + lane * 16);
    const uint32_t c0 = e4m3x2_to_f16x2(lds16(base + kUnitCodes + g * 8 + t * 2));
    const uint32_t c1 = e4m3x2_to_f16x2(lds16(base + kUnitCodes + g * 8 + t * 2 + 64));
    const uint32_t s0[2] = {prmt(c0, c0, 0x1010u), prmt(c0, c0, 0x3232u)};
    const uint32_t s1[2] = {prmt(c1, c1, 0x1010u), prmt(c1, c1, 0x3232u)};
    k_step<0>(s[0], r0, r1, s0, s1, bq[u][0][0], bq[u][0][1]);
    k_step<1>(s[1], r0, r1, s0, s1, bq[u][1][0], bq[u][1][1]);
    k_step<2>(s[0], r0, r1, s0, s1, bq[u][2][0], bq[u][2][1]);
    k_step<3>(s[1], r0, r1, s0, s1, bq[u][3][0], bq[u][3][1]);
    k_step<4>(s[0], r0, r1, s0, s1, bq[u][4][0], bq[u][4][1]);
    k_step<5>(s[1], r0, r1, s0, s1, bq[u][5][0], bq[u][5][1]);
    k_step<6>(s[0], r0, r1, s0, s1, bq[u][6][0], bq[u][6][1]);
    k_step<7>(s[1], r0, r1, s0, s1, bq[u][7][0], bq[u][7][1]);
  }
  bool ok_lo = true, ok_hi = true;
  if (edge) {
    ok_lo = tok0 + g >= t_lo && tok0 + g <= pos;
    ok_hi = tok0 + g + 8 >= t_lo && tok0 + g + 8 <= pos;
  }
  float x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float v = (s[0][i] + s[1][i]) * ((i & 1) ? f1 : f0);
    if (softcap > 0.f) {
      // v = logit / cap; tanh(y) = 1 - 2 / (e^{2y} + 1), absolute error ~1e-7
      const float e = fast_exp2(fminf(2.f * kLog2e * v, 126.f));
      v = softcap * (1.f - __fdividef(2.f, e + 1.f)) * kLog2e;
    }
    x[i] = ((i & 2) ? ok_hi : ok_lo) ? v : -INFINITY;
  }
  const bool grow = fmaxf(x[0], x[2]) > m[0] + kGrow || fmaxf(x[1], x[3]) > m[1] + kGrow;
  if (__any_sync(0xffffffffu, grow)) {
    float alpha[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float mx = fmaxf(x[j], x[j + 2]);
#pragma unroll
      for (int off = 4; off < 32; off <<= 1)
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      const float mn = fmaxf(m[j], mx);
      alpha[j] = (mn == -INFINITY) ? 1.f : fast_exp2(m[j] - mn);
      m[j] = mn;
      l[j] *= alpha[j];
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
  const float p0 = fast_exp2(x[0] - r0), p1 = fast_exp2(x[1] - r1);
  const float p2 = fast_exp2(x[2] - r0), p3 = fast_exp2(x[3] - r1);
  l[0] += p0 + p2;
  l[1] += p1 + p3;
  const uint32_t pb0 = movmatrix_trans(pack_f16x2(p0, p1));  // keys 2t, 2t + 1 of head g
  const uint32_t pb1 = movmatrix_trans(pack_f16x2(p2, p3));  // keys 2t + 8, 2t + 9

#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    const uint32_t base = tile + (UNITS + u) * kUnitBytes;
    const uint32_t row = base + g * 128 + ((t * 16) ^ ((g & 1) * 64));
    const uint4 a = lds128(row);                       // keys 2t (x, y) and 2t + 1 (z, w)
    const uint4 b = lds128(base + g * 128 + ((t * 16 + 64) ^ ((g & 1) * 64)));
    uint32_t ca = lds16(base + kUnitCodes + g * 16 + t * 2);
    uint32_t cb = lds16(base + kUnitCodes + g * 16 + t * 2 + 8);
    if (edge) {
      // stale slots may hold the scale NaN: an invisible key's value is 0
      const int k0 = tok0 + 2 * t;
      if (k0 < t_lo || k0 > pos) ca &= 0xff00u;
      if (k0 + 1 < t_lo || k0 + 1 > pos) ca &= 0x00ffu;
      if (k0 + 8 < t_lo || k0 + 8 > pos) cb &= 0xff00u;
      if (k0 + 9 < t_lo || k0 + 9 > pos) cb &= 0x00ffu;
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

template <int D, int NW, int STAGES>
__global__ void __launch_bounds__(NW * 32, 1)
    kv4_decode_kernel(const __grid_constant__ Kv4DecodeArgs ka) {
  using S = Kv4Shape<D, NW, STAGES>;
  constexpr int UNITS = S::UNITS;
  extern __shared__ __align__(128) uint8_t smem[];
  const DecodeArgs& a = ka.base;
  const int G = a.Hq / a.Hkv;
  int* slen = reinterpret_cast<int*>(smem + S::kRing);
  float2* ml = reinterpret_cast<float2*>(smem + S::kRing + S::kLen);  // [NW][8]
  volatile int* flag = reinterpret_cast<int*>(smem + S::kRing + S::kLen + NW * 8 * 8);
  float* st = reinterpret_cast<float*>(smem + S::kRing + S::kLen + S::kMl);  // [NW][G][D]
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * STAGES * 2 * S::kTile;

  for (int b = threadIdx.x; b < min(a.batch, kLenCache); b += NW * 32)
    slen[b] = req_len_of(a, 0, 0, a.seq_lens[b]);
  __syncthreads();

  PieceIter iter;
  iter.init(a, slen, lane, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x));
  const float inv_cap = a.softcap > 0.f ? 1.f / a.softcap : 0.f;
  const float lscale = a.scale * ka.k_scale * (a.softcap > 0.f ? inv_cap : kLog2e);

  Piece pc;
  bool have = iter.next(pc, true);
  int mine = 0;        // tiles of the piece that are this warp's
  int ids = 0;         // block ids of its tiles base .. base + 31, one per lane
  auto load_ids = [&](const Piece& P, int base) {
    const int i = warp + (base + lane) * NW;
    int id = -1;
    if (i < P.ntiles) {
      id = a.tables[static_cast<size_t>(P.b) * a.max_blocks + P.j0 + i];
      if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.num_blocks)) {
        report(a.err, PKA_DEVERR_BAD_TABLE);
        id = -1;
      }
    }
    return id;
  };
  // requests the warp's tile n of piece P (its id in lane n % 32 of ids)
  auto issue = [&](const Piece& P, int n) {
    const int id = __shfl_sync(0xffffffffu, ids, n & 31);
    const uint32_t bytes = id >= 0 ? 16u : 0u;  // a bad id reads as zeros
    const long long off =
        (static_cast<long long>(max(id, 0)) * a.Hkv + P.kvh) * S::kTile;
    const uint32_t dst = ring + (n % STAGES) * 2 * S::kTile;
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
  auto prologue = [&](const Piece& P) {
    mine = P.ntiles > warp ? (P.ntiles - warp + NW - 1) / NW : 0;
    ids = load_ids(P, 0);
#pragma unroll
    for (int n = 0; n < STAGES - 1; ++n) {
      if (n < mine) issue(P, n);
      cp_async_commit();
    }
  };
  if (have) prologue(pc);

  while (have) {
    // ---- q of head g as B fragments in f16, scaled by a power of two
    uint32_t bq[UNITS][8][2];
    float fq;  // the logit factor of head g
    {
      const uint16_t* qp =
          a.q + (static_cast<size_t>(pc.qrow) * a.Hq + pc.kvh * G + (g < G ? g : 0)) * D + t * 32;
      uint4 raw[UNITS][4];
      uint32_t top = 0;  // largest magnitude, as bf16 bits
#pragma unroll
      for (int u = 0; u < UNITS; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          raw[u][i] = (g < G) ? __ldg(reinterpret_cast<const uint4*>(qp + u * kUnitChannels) + i)
                              : make_uint4(0u, 0u, 0u, 0u);
          const uint32_t w[4] = {raw[u][i].x, raw[u][i].y, raw[u][i].z, raw[u][i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            top = max(top, max(w[k] & 0x7fffu, (w[k] >> 16) & 0x7fffu));
        }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = min(max(254 - static_cast<int>(top >> 7), 1), 253);
      const float down = __uint_as_float(static_cast<uint32_t>(e) << 23);
      fq = lscale * __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
#pragma unroll
      for (int u = 0; u < UNITS; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float f[8];
          unpack8(raw[u][i], f);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            bq[u][i * 2 + k][0] = pack_f16x2(f[k * 4] * down, f[k * 4 + 1] * down);
            bq[u][i * 2 + k][1] = pack_f16x2(f[k * 4 + 2] * down, f[k * 4 + 3] * down);
          }
        }
    }
    const float f0 = __shfl_sync(0xffffffffu, fq, 8 * t);
    const float f1 = __shfl_sync(0xffffffffu, fq, 8 * t + 4);

    float o[UNITS][8][4];
#pragma unroll
    for (int u = 0; u < UNITS; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) o[u][i][0] = o[u][i][1] = o[u][i][2] = o[u][i][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    const int count = mine;
    for (int n = 0; n < count; ++n) {
      cp_async_wait<STAGES - 2>();
      __syncwarp();  // every lane's part of tile n has landed; tile n - 1 is consumed
      const int ahead = n + STAGES - 1;
      if (ahead < count) {
        if ((ahead & 31) == 0) ids = load_ids(pc, ahead);
        issue(pc, ahead);
      }
      cp_async_commit();
      const int tok0 = (pc.j0 + warp + n * NW) * kBlockSize;
      const bool edge = tok0 < pc.t_lo || tok0 + kBlockSize - 1 > pc.pos;
      kv4_tile<D>(ring + (n % STAGES) * 2 * S::kTile, bq, o, m, l, f0, f1, a.softcap, inv_cap,
                  edge, tok0, pc.t_lo, pc.pos, lane);
    }
    __syncwarp();

    Piece nx;
    const bool have_next = iter.next(nx, true);
    if (have_next) prologue(nx);

    // ---- the warps' states through shared memory, merged in warp order
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) l[j] += __shfl_xor_sync(0xffffffffu, l[j], off);
    if (g == 0) {
      ml[warp * 8 + 2 * t] = make_float2(m[0], l[0]);
      ml[warp * 8 + 2 * t + 1] = make_float2(m[1], l[1]);
    }
    if (count > 0) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int h = 2 * t + j;
        if (h < G) {
#pragma unroll
          for (int u = 0; u < UNITS; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<float4*>(st + (warp * G + h) * D + u * kUnitChannels + g * 16 +
                                         i * 4) =
                  make_float4(o[u][2 * i][j], o[u][2 * i][2 + j], o[u][2 * i + 1][j],
                              o[u][2 * i + 1][2 + j]);
        }
      }
    }
    __syncthreads();
    const bool split = !iter.direct;
    const bool has_keys = pc.ntiles > 0;
    if (!split || !has_keys || pc.slot < a.num_splits) {
      const int warps = min(NW, pc.ntiles);  // warps that had a tile
      for (int item = threadIdx.x; item < G * (D / 4); item += NW * 32) {
        const int h = item / (D / 4), d0 = item % (D / 4) * 4;
        float M = -INFINITY;
        for (int w = 0; w < warps; ++w) M = fmaxf(M, ml[w * 8 + h].x);
        const float Ms = (M == -INFINITY) ? 0.f : M;
        float den = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < warps; ++w) {
          const float2 v = ml[w * 8 + h];
          const float4 x = *reinterpret_cast<const float4*>(st + (w * G + h) * D + d0);
          const float sc = (v.x == -INFINITY) ? 1.f : fast_exp2(v.x - Ms);
          den = fmaf(sc, v.y, den);
          acc.x = fmaf(sc, x.x, acc.x);
          acc.y = fmaf(sc, x.y, acc.y);
          acc.z = fmaf(sc, x.z, acc.z);
          acc.w = fmaf(sc, x.w, acc.w);
        }
        const float inv = den == 0.f ? 0.f : ka.v_scale / den;
        acc.x *= inv;
        acc.y *= inv;
        acc.z *= inv;
        acc.w *= inv;
        const size_t head = static_cast<size_t>(pc.qrow) * a.Hq + pc.kvh * G + h;
        if (split && has_keys) {
          const size_t row = head * a.num_splits + pc.slot;
          __stcg(reinterpret_cast<float4*>(a.partial_o + row * D + d0), acc);
          // a NaN sum keeps its weight, so that the merge passes it on
          if (d0 == 0)
            __stcg(a.partial_lse + row, den == 0.f  ? -INFINITY
                                        : isnan(den) ? Ms * kLn2
                                                     : (Ms + log2f(den)) * kLn2);
        } else {
          *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + head * D + d0) =
              make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
        }
      }
    }
    if (split && has_keys) {
      // ---- the piece that arrives last at its segment merges the partials
      const int np = min(pc.npieces, a.num_splits);
      __syncthreads();
      if (threadIdx.x == 0) {
        if (pc.npieces > a.num_splits) report(a.err, PKA_DEVERR_SEQ_LEN);
        int last = 0;
        if (pc.slot < a.num_splits) {
          fence_acq_rel_gpu();
          int32_t* counter = a.seg_counters + pc.b * a.Hkv + pc.kvh;
          last = atomicAdd(counter, 1) == np - 1;
          fence_acq_rel_gpu();
          if (last) *counter = 0;
        }
        *flag = last;
      }
      __syncthreads();
      if (*flag != 0) {
        for (int item = threadIdx.x; item < G * (D / 4); item += NW * 32) {
          const int h = item / (D / 4), d0 = item % (D / 4) * 4;
          const size_t head = static_cast<size_t>(pc.qrow) * a.Hq + pc.kvh * G + h;
          float M = -INFINITY, den = 0.f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int s0 = 0; s0 < np; s0 += 4) {
            float lv[4];
            float4 x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const size_t row = head * a.num_splits + min(s0 + k, np - 1);
              lv[k] = s0 + k < np ? __ldcg(a.partial_lse + row) : -INFINITY;
              x[k] = __ldcg(reinterpret_cast<const float4*>(a.partial_o + row * D + d0));
              if (s0 + k >= np) x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
            lse_merge4(M, den, acc, lv, x);
          }
          const float inv = den == 0.f ? 0.f : 1.f / den;
          *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + head * D + d0) =
              make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv),
                         pack_bf16x2(acc.z * inv, acc.w * inv));
        }
      }
    }
    __syncthreads();  // the states' shared memory is free again
    pc = nx;
    have = have_next;
  }
  cp_async_wait<0>();
}

template <int D, int NW, int STAGES>
cudaError_t launch_t(const Kv4DecodeArgs& a, int sms, cudaStream_t stream) {
  using S = Kv4Shape<D, NW, STAGES>;
  auto kern = kv4_decode_kernel<D, NW, STAGES>;
  static_assert(S::smem(8) <= 232448, "shared memory of one CTA");
  const cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kern), S::smem(8));
  if (e != cudaSuccess) return e;
  kern<<<sms, NW * 32, S::smem(a.base.Hq / a.base.Hkv), stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_decode(const Kv4DecodeArgs& a, int head_dim, int sms, cudaStream_t stream) {
  if (head_dim == 128) return launch_t<128, 16, 4>(a, sms, stream);
  if (head_dim == 256) return launch_t<256, 8, 4>(a, sms, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pka
