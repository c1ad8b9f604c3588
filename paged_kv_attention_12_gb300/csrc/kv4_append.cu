// Writing a 4-bit pool and expanding its blocks to bf16 (sm_103a).
//
// The format and its rounding are in kv4.cuh.  Both kernels are bound by the
// bytes they move: a value is 2 bytes in bf16 and 0.5625 in the pool.
#include "kv4.cuh"
#include "kernels.h"

namespace pka {

namespace {

// One thread per group of 16 channels of a (token, head) row of K or V: 32
// bytes in, 8 code bytes and a scale out.
__global__ void __launch_bounds__(256) kv4_append_kernel(const Kv4AppendArgs a) {
  const int gpr = a.head_dim / 16;  // groups per row
  const long long per_tensor = static_cast<long long>(a.T) * a.Hkv * gpr;
  const long long total = 2 * per_tensor;
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * blockDim.x) {
    const bool is_v = i >= per_tensor;
    const long long r = is_v ? i - per_tensor : i;
    const int grp = static_cast<int>(r % gpr);
    const long long th = r / gpr;
    const int h = static_cast<int>(th % a.Hkv);
    const int t = static_cast<int>(th / a.Hkv);
    const int s = a.slot_mapping[t];
    if (s < 0) continue;
    const int blk = s / kBlockSize, tok = s % kBlockSize;
    if (blk >= a.num_blocks) {
      if (grp == 0 && h == 0 && !is_v) report(a.err, PKA_DEVERR_BAD_TABLE);
      continue;
    }
    const uint16_t* src = (is_v ? a.v_new + t * a.v_stride : a.k_new + t * a.k_stride) +
                          static_cast<long long>(h) * a.head_dim + grp * 16;
    float x[16];
    {
      float lo[8], hi[8];
      unpack8(__ldg(reinterpret_cast<const uint4*>(src)), lo);
      unpack8(__ldg(reinterpret_cast<const uint4*>(src) + 1), hi);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[j] = lo[j];
        x[j + 8] = hi[j];
      }
    }
    uint32_t sb;
    const uint2 codes = quantise_group(x, is_v ? a.v_scale : a.k_scale,
                                       is_v ? a.v_scale6 : a.k_scale6, sb);
    const int units = a.head_dim / kUnitChannels;
    uint8_t* unit = (is_v ? a.v_pool : a.k_pool) +
                    ((static_cast<long long>(blk) * a.Hkv + h) * units + grp / 8) * kUnitBytes;
    const int g8 = grp % 8;
    *reinterpret_cast<uint2*>(unit + (is_v ? v_code_offset(tok, g8) : k_code_offset(tok, g8))) =
        codes;
    unit[is_v ? v_scale_offset(tok, g8) : k_scale_offset(tok, g8)] = static_cast<uint8_t>(sb);
  }
}

// One thread per 8 channels of a (block, head, token) of K or V: 4 code bytes
// in, 16 bytes out.
__global__ void __launch_bounds__(256) kv4_expand_kernel(const Kv4ExpandArgs a) {
  const int cpr = a.head_dim / 8;  // 8-channel chunks per row
  const int per_head = kBlockSize * cpr;
  const long long per_tensor = static_cast<long long>(a.n) * a.Hkv * per_head;
  const long long total = 2 * per_tensor;
  const int units = a.head_dim / kUnitChannels;
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * blockDim.x) {
    const bool is_v = i >= per_tensor;
    const long long r = is_v ? i - per_tensor : i;
    const int c = static_cast<int>(r % cpr);
    const int tok = static_cast<int>(r / cpr % kBlockSize);
    const long long bh = r / per_head;
    const int h = static_cast<int>(bh % a.Hkv);
    const int item = static_cast<int>(bh / a.Hkv);
    const int src = a.src_blocks[item];
    const int dst = a.dst_blocks != nullptr ? a.dst_blocks[item] : item;
    if (src < 0 || dst < 0) continue;
    if (src >= a.src_num_blocks || dst >= a.dst_num_blocks) {
      if (c == 0 && tok == 0 && h == 0 && !is_v) report(a.err, PKA_DEVERR_BAD_TABLE);
      continue;
    }
    const uint8_t* unit = (is_v ? a.v4 : a.k4) +
                          ((static_cast<long long>(src) * a.Hkv + h) * units + c / 16) * kUnitBytes;
    const int grp = c % 16 / 2, half = c % 2;
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(
        unit + (is_v ? v_code_offset(tok, grp) : k_code_offset(tok, grp)) + half * 4));
    const uint16_t sb = __ldg(unit + (is_v ? v_scale_offset(tok, grp) : k_scale_offset(tok, grp)));
    float s, unused;
    f16x2_to_f32(e4m3x2_to_f16x2(sb), s, unused);
    const float scale = is_v ? a.v_scale : a.k_scale;
    const uint32_t p[4] = {e2m1x2_to_f16x2<0>(w), e2m1x2_to_f16x2<1>(w), e2m1x2_to_f16x2<2>(w),
                           e2m1x2_to_f16x2<3>(w)};
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float lo, hi;
      f16x2_to_f32(p[j], lo, hi);
      // code * e4m3 is exact; the pool scale and bf16 round once each
      o[j] = pack_bf16x2(lo * s * scale, hi * s * scale);
    }
    uint16_t* out = (is_v ? a.v16 : a.k16) +
                    ((static_cast<long long>(dst) * a.Hkv + h) * kBlockSize + tok) * a.head_dim +
                    c * 8;
    *reinterpret_cast<uint4*>(out) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

int grid_for(long long threads, int sm_count, int per_sm) {
  const long long want = (threads + 255) / 256;
  const long long cap = static_cast<long long>(sm_count > 0 ? sm_count : 1) * per_sm;
  return static_cast<int>(want < cap ? want : cap);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4AppendArgs& a, int sm_count, cudaStream_t stream) {
  const long long total = 2LL * a.T * a.Hkv * (a.head_dim / 16);
  if (total == 0) return cudaSuccess;
  kv4_append_kernel<<<grid_for(total, sm_count, 8), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv4_expand(const Kv4ExpandArgs& a, int sm_count, cudaStream_t stream) {
  const long long total = 2LL * a.n * a.Hkv * kBlockSize * (a.head_dim / 8);
  if (total == 0) return cudaSuccess;
  kv4_expand_kernel<<<grid_for(total, sm_count, 8), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace pka
