// w4.cuh -- the base projection with 4-bit weights and group scales.
//
//   out[t, n] = rn( sx[t] * sum_g s[g, n] * sum_{k in group g} x[t, k] (q[n, k] - z[g, n]) )
//
// Eight weights are one 32-bit word, value i of the word in its 4-bit place
// (0, 4, 1, 5, 2, 6, 3, 7)[i]: one mask and three shifts then give the pairs
// (0, 1), (2, 3), (4, 5), (6, 7) in the halves of four registers.
#pragma once

#include "common.cuh"
#include "rmsnorm.cuh"

namespace lora {

struct W4Args {
  const void* x;        // [tok, ld_x], 16-bit elements or e4m3
  int64_t ld_x;
  const float* x_scale; // [tok] with e4m3, else null
  const uint8_t* w;     // [N, ld_w bytes]
  int64_t ld_w;
  const uint16_t* s;    // [G, ld_s]
  const uint8_t* z;     // [G, ld_s] or null (8)
  int64_t ld_s;
  uint16_t* out;        // [tok, ld_out]
  int64_t ld_out;
  int tok, K, N, group_shift;
};

// One warp computes out[t, n] of one row n for four tokens.
template <class E, bool X8>
__global__ void __launch_bounds__(256) w4_simple_kernel(const W4Args p) {
  const int lane = threadIdx.x & 31;
  const int n = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int t0 = blockIdx.y * 4;
  if (n >= p.N) return;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int k0 = lane * 8; k0 < p.K; k0 += 256) {
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(p.w + n * p.ld_w + k0 / 2));
    const int64_t at = static_cast<int64_t>(k0 >> p.group_shift) * p.ld_s + n;
    const float s = E::bits_to_f32(__ldg(p.s + at));
    const float z = p.z ? static_cast<float>(__ldg(p.z + at) & 15) : 8.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int k = k0 + i;
      if (k >= p.K) break;
      const float v = s * (static_cast<float>((w >> (16 * (i & 1) + 4 * (i >> 1))) & 15u) - z);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        if (t0 + t >= p.tok) break;
        const int64_t e = static_cast<int64_t>(t0 + t) * p.ld_x + k;
        float x;
        if (X8) {
          const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(p.x)[e], __NV_E4M3);
          x = __half2float(__half(h));
        } else {
          x = E::bits_to_f32(static_cast<const uint16_t*>(p.x)[e]);
        }
        acc[t] = fmaf(v, x, acc[t]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const float r = warp_sum(acc[t]);
    if (lane == 0 && t0 + t < p.tok)
      stg16(p.out + (t0 + t) * p.ld_out + n,
            E::f32_to_bits(X8 ? r * p.x_scale[t0 + t] : r));
  }
}

}  // namespace lora
