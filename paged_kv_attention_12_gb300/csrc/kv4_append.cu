// Writing a 4-bit pool and expanding its blocks to bf16 (sm_103a).
//
// The format and its rounding are in kv4.cuh.  Both kernels are bound by the
// bytes they move: a value is 2 bytes in bf16 and 0.5625 in the pool.
#include <algorithm>

#include "kv4.cuh"
#include "kernels.h"
#include "overlap.cuh"

namespace pka {

namespace {

// One warp per four tokens and 128 channels of a head, of K or V or (BOTH) of
// each; a lane takes the 32 bytes of one token's group of 16 channels and writes
// 8 code bytes and a scale.  Tokens that follow one another in a block make
// whole 32-byte sectors of the stores: a K unit holds a token's groups side by
// side, a V unit a group's tokens.  Grid: y the head and 128 channels (and K or
// V), x the tokens, so that nothing is divided by sizes.  Bound by arithmetic and
// by the time a warp waits for its rows: 8192 tokens x 4 heads x 128, 21.5 MB,
// 5.0 us, 3.2 us of it HBM; its 1024 CTAs are 1.35 waves of the 760 that run at
// once (K and V on warps of their own 5.5 us, unpaired arithmetic 5.6, four CTAs
// per SM 6.0, a warp index divided by the heads 6.4, a division per value 9.8).
// 32 tokens: 1.8 us, 2.2 with BOTH.  (Calls in a captured graph, three input sets
// in turn.)
template <bool BOTH>
__global__ void __launch_bounds__(256, 5)
    kv4_append_kernel(const __grid_constant__ Kv4AppendArgs a) {
  launch_dependents();
  wait_predecessor();
  constexpr int SIDES = BOTH ? 2 : 1;
  const int lane = threadIdx.x & 31;
  const int per = a.Hkv * (a.head_dim / kUnitChannels);  // units of a block
  const int g8 = lane & 7;
  const unsigned quads = (static_cast<unsigned>(a.T) + 3) / 4;
  const unsigned stride = gridDim.x * (blockDim.x / 32);
  for (int y = blockIdx.y; y < per * (3 - SIDES); y += gridDim.y) {
    const bool second = !BOTH && y >= per;
    const int hu = second ? y - per : y;  // head * units of a head + unit
    const int chan = hu * kUnitChannels + g8 * 16;
    for (unsigned quad = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32; quad < quads;
         quad += stride) {
      const unsigned t = quad * 4 + (lane >> 3);
      if (t >= static_cast<unsigned>(a.T)) continue;
      const int s = a.slot_mapping[t];
      uint4 x[SIDES][2];
#pragma unroll
      for (int k = 0; k < SIDES; ++k) {
        const bool v = BOTH ? k == 1 : second;
        const uint4* src = reinterpret_cast<const uint4*>(
            (v ? a.v_new + t * a.v_stride : a.k_new + t * a.k_stride) + chan);
        x[k][0] = src[0];
        x[k][1] = src[1];
      }
      if (s < 0) continue;
      const int blk = s / kBlockSize, tok = s % kBlockSize;
      if (blk >= a.num_blocks) {
        if (y == 0 && g8 == 0) report(a.err, PKA_DEVERR_BAD_TABLE);
        continue;
      }
      const long long at = (static_cast<long long>(blk) * per + hu) * kUnitBytes;
#pragma unroll
      for (int k = 0; k < SIDES; ++k) {
        const bool v = BOTH ? k == 1 : second;
        uint8_t* unit = (v ? a.v_pool : a.k_pool) + at;
        uint32_t sb;
        const uint2 codes = quantise_group(x[k][0], x[k][1], v ? a.v_scale : a.k_scale,
                                           v ? a.v_scale6 : a.k_scale6, sb);
        *reinterpret_cast<uint2*>(unit + (v ? v_code_offset(tok, g8) : k_code_offset(tok, g8))) =
            codes;
        unit[v ? v_scale_offset(tok, g8) : k_scale_offset(tok, g8)] = static_cast<uint8_t>(sb);
      }
    }
  }
}

// One warp per unit (16 tokens x 128 channels of a block and head, K or V): a
// lane takes 8 channels of two tokens apart at a time, so that every store of
// the warp is two whole rows of 256 bytes; the unit's loads are in flight
// together.  Bound by HBM: 4096 blocks x 4 heads x 128, 172 MB, 30.3 us, 5.7 TB/s,
// 84% of a plain copy, three input sets in turn.  With one set, part of which
// stays in L2: 25.6 us (31 without the streaming stores; 74 with a thread per 8
// channels and an index division each).
__global__ void __launch_bounds__(256) kv4_expand_kernel(const __grid_constant__ Kv4ExpandArgs a) {
  const int lane = threadIdx.x & 31;
  const int units = a.head_dim / kUnitChannels;
  const int per_block = 2 * a.Hkv * units;
  const long long total = static_cast<long long>(a.n) * per_block;
  const long long wstride = static_cast<long long>(gridDim.x) * (blockDim.x / 32);
  const int c = lane & 15, grp = c >> 1, odd = lane >> 4;  // chunk of 8 channels, token parity
  for (long long w = static_cast<long long>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32;
       w < total; w += wstride) {
    const int item = static_cast<int>(w / per_block);
    const int in = static_cast<int>(w - static_cast<long long>(item) * per_block);
    const bool is_v = in >= a.Hkv * units;
    const int hu = is_v ? in - a.Hkv * units : in;  // head * units + unit
    const int src = __ldg(a.src_blocks + item);
    const int dst = a.dst_blocks != nullptr ? __ldg(a.dst_blocks + item) : item;
    if (src < 0 || dst < 0) continue;
    if (src >= a.src_num_blocks || dst >= a.dst_num_blocks) {
      if (lane == 0 && in == 0) report(a.err, PKA_DEVERR_BAD_TABLE);
      continue;
    }
    const uint8_t* unit = (is_v ? a.v4 : a.k4) +
                          (static_cast<long long>(src) * a.Hkv * units + hu) * kUnitBytes;
    uint32_t code[8];
    uint32_t sb[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int tok = 2 * k + odd;
      code[k] = __ldg(reinterpret_cast<const uint32_t*>(
          unit + (is_v ? v_code_offset(tok, grp) : k_code_offset(tok, grp)) + (c & 1) * 4));
      sb[k] = __ldg(unit + (is_v ? v_scale_offset(tok, grp) : k_scale_offset(tok, grp)));
    }
    const int h = hu / units, u = hu % units;
    uint16_t* out = (is_v ? a.v16 : a.k16) +
                    ((static_cast<long long>(dst) * a.Hkv + h) * kBlockSize + odd) * a.head_dim +
                    u * kUnitChannels + c * 8;
    const float scale = is_v ? a.v_scale : a.k_scale;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t s2 = e4m3x2_to_f16x2(static_cast<uint16_t>(sb[k] * 0x101u));
      const uint32_t p[4] = {e2m1x2_to_f16x2<0>(code[k]), e2m1x2_to_f16x2<1>(code[k]),
                             e2m1x2_to_f16x2<2>(code[k]), e2m1x2_to_f16x2<3>(code[k])};
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // code * e4m3 is exact in f16; the pool scale and bf16 round once each
        float lo, hi;
        f16x2_to_f32(f16x2_mul(p[j], s2), lo, hi);
        o[j] = pack_bf16x2(lo * scale, hi * scale);
      }
      __stcs(reinterpret_cast<uint4*>(out + static_cast<long long>(2 * k) * a.head_dim),
             make_uint4(o[0], o[1], o[2], o[3]));
    }
  }
}

int grid_for(long long blocks, int sm_count, int per_sm) {
  const long long cap = static_cast<long long>(sm_count > 0 ? sm_count : 1) * per_sm;
  return static_cast<int>(blocks < cap ? blocks : cap);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4AppendArgs& a, int sm_count, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  const int sms = sm_count > 0 ? sm_count : 1;
  const int per = a.Hkv * (a.head_dim / kUnitChannels);
  const long long x = (static_cast<long long>(a.T) + 31) / 32;
  // K and V on one warp once there is more to do than 40 warps an SM do at once
  const bool both = x * per * 2 > 5LL * sms;
  const int y = std::min(both ? per : 2 * per, 65535);
  const dim3 grid(static_cast<unsigned>(std::min(x, (16LL * sms + y - 1) / y)), y);
  return launch_overlapped(both ? kv4_append_kernel<true> : kv4_append_kernel<false>, grid, 256, 0,
                           stream, a);
}

cudaError_t launch_kv4_expand(const Kv4ExpandArgs& a, int sm_count, cudaStream_t stream) {
  if (a.n == 0) return cudaSuccess;
  const long long warps =
      2LL * a.n * a.Hkv * (a.head_dim / kUnitChannels);
  // a plain launch: overlapped, 128 blocks took 3.1 us instead of 2.3
  kv4_expand_kernel<<<grid_for((warps + 7) / 8, sm_count, 64), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace pka
