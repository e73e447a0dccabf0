// rmsnorm.cuh -- the RMS norm that makes the projection's input x, with the
// residual's addition before it and the rounding to 8 bits behind it.
//
//   h[t, c] = rn(x[t, c] + residual[t, c])                      (x itself without a residual)
//   v[t, c] = h[t, c] * rsqrt(sum_c h^2 / H + eps) * (w[c] + w0)
//   out = rn(v);   scale[t] = max_c |v| / 448;   q[t, c] = e4m3(v * rn(1 / scale[t]))
//
// What is normalised is h as the residual stream holds it, rounded, so that a
// later reader of the stream sees the row that was normalised.  The sum, the
// factor and v are fp32; out and q are each rounded once, from v.  (q by the
// reciprocal: a division an element took 67 instead of 60 us at 8192 x 5120, and
// on the border between two values neither is nearer to the formula in 64 bits.)
//
// One group of threads holds a row in registers between the two passes over it
// (the sum, then the outputs), so each input is read once and each output
// written once: the bound is the memory traffic, 2 bytes for each of x,
// residual, h and out and 1 for q.  8192 x 5120 with all of them: 59.8 us, 6.3
// TB/s, 96 % of the measured copy rate; one row of 4096: 1.9 us.
// Every variant may have 1024 threads a row, hence 64 registers a thread.  Rows
// of eight blocks of eight a thread spill there, 212 bytes a thread or 340 with q,
// off the 16-byte grid 1028 or 1164: those of more than 8192 elements with many
// rows (eight for each SM), of more than 16,384 with a row for each SM, of more
// than 32,768 else.  2560 x 16384 with all outputs takes 95 us, 2560 x 16383 157,
// where the traffic alone would take 58.  (Four blocks off the grid: 24, 40 bytes.)
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"
#include "sm100.cuh"

namespace lora {

struct RmsNormArgs {
  const uint16_t* x;
  int64_t ld_x;
  const uint16_t* res;  // may be null
  int64_t ld_res;
  uint16_t* res_out;    // written where res is given
  int64_t ld_res_out;
  const uint16_t* w;
  uint16_t* out;        // may be null
  int64_t ld_out;
  uint8_t* q;           // may be null
  int64_t ld_q;
  float* scale;
  int tok, H;
  float eps, w0;
  int follow;           // rows are cut where x crosses 16-byte boundaries
};

// Four fp32 values -> four e4m3 bytes, to nearest even, saturating at 448.
__device__ __forceinline__ uint32_t f4_to_e4m3(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// Eight elements e0 .. e0+7 of a row (those in [0, H)): one 16-byte load where
// they are whole and aligned, the two 16-byte blocks that cover them where
// they are whole.  Plain loads: the outputs may be written over the inputs,
// element by element.
template <bool AL>
__device__ __forceinline__ uint4 norm_load8(const uint16_t* row, int e0, int H) {
  const uint16_t* p = row + e0;
  bool whole = AL;
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15);
  if (!whole) whole = e0 >= 0 && e0 + 8 <= H && off == 0;
  if (whole) return *reinterpret_cast<const uint4*>(p);
  if (e0 >= 0 && e0 + 8 <= H) {
    const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(p) - off);
    return bytes_at(q[0], q[1], off);
  }
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = e0 + 2 * i;
    const uint32_t lo = (e >= 0 && e < H) ? p[2 * i] : 0u;
    const uint32_t hi = (e + 1 >= 0 && e + 1 < H) ? p[2 * i + 1] : 0u;
    w[i] = lo | (hi << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool AL>
__device__ __forceinline__ void norm_store8(uint16_t* row, int e0, int H, uint4 v) {
  uint16_t* p = row + e0;
  bool whole = AL;
  if (!whole) whole = e0 >= 0 && e0 + 8 <= H && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
  if (whole) {
    stg128(p, v);
    return;
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (e0 + i >= 0 && e0 + i < H) stg16(p + i, static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1))));
}

// blockDim = (threads of a row, rows of the block), the first a multiple of 32.
// VPT: blocks of eight elements that a thread holds.  AL: every row of every
// tensor is 16-byte aligned (q: 8-byte) and H is a multiple of 8.  QUANT: q is
// given.
template <class E, int VPT, bool AL, bool QUANT>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(const RmsNormArgs p) {
  __shared__ float ssum[32];
  __shared__ uint32_t smax[32];
  const int T = blockDim.x, tid = threadIdx.x;
  const int warps = T >> 5;
  const int row = blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = row < p.tok;
  const int64_t t = live ? row : 0;
  const uint16_t* x = p.x + t * p.ld_x;
  // blocks of eight start where x's row crosses 16-byte boundaries
  const int shift = AL || !p.follow ? 0 : static_cast<int>((reinterpret_cast<uintptr_t>(x) >> 1) & 7);
  // All loads before the first store, which they would have to wait for; the
  // weights too where there are registers for them, behind the sum otherwise.
  uint4 xv[VPT], rv[VPT], wv[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int e0 = 8 * (j * T + tid) - shift;
    xv[j] = rv[j] = wv[j] = make_uint4(0, 0, 0, 0);
    if (live && e0 < p.H) {
      xv[j] = norm_load8<AL>(x, e0, p.H);
      if (p.res) rv[j] = norm_load8<AL>(p.res + t * p.ld_res, e0, p.H);
      if (VPT <= 2) wv[j] = norm_load8<AL>(p.w, e0, p.H);
    }
  }
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int e0 = 8 * (j * T + tid) - shift;
    uint32_t* a = reinterpret_cast<uint32_t*>(&xv[j]);
    const uint32_t* b = reinterpret_cast<const uint32_t*>(&rv[j]);
    if (p.res) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = E::u32_to_f2(a[i]), g = E::u32_to_f2(b[i]);
        a[i] = E::f2_to_u32(f.x + g.x, f.y + g.y);
      }
      if (live && e0 < p.H) norm_store8<AL>(p.res_out + t * p.ld_res_out, e0, p.H, xv[j]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = E::u32_to_f2(a[i]);
      sum = fmaf(f.x, f.x, fmaf(f.y, f.y, sum));
    }
  }
  sum = warp_sum(sum);
  const int w0 = threadIdx.y * warps;
  if (warps > 1) {
    if ((tid & 31) == 0) ssum[w0 + (tid >> 5)] = sum;
    __syncthreads();
    sum = 0.f;
    for (int i = 0; i < warps; ++i) sum += ssum[w0 + i];
  }
  const float rstd = rsqrtf(sum / static_cast<float>(p.H) + p.eps);

  uint32_t top = 0;  // bits of max |v|; a NaN's bits are above an infinity's
  float v[QUANT ? VPT : 1][8];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int e0 = 8 * (j * T + tid) - shift;
    if (VPT > 2 && live && e0 < p.H) wv[j] = norm_load8<AL>(p.w, e0, p.H);
  }
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int e0 = 8 * (j * T + tid) - shift;
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&wv[j]);
    uint32_t* hv = reinterpret_cast<uint32_t*>(&xv[j]);
    const int jj = QUANT ? j : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = E::u32_to_f2(w[i]), g = E::u32_to_f2(hv[i]);
      const float a = g.x * rstd * (f.x + p.w0);
      const float b = g.y * rstd * (f.y + p.w0);
      v[jj][2 * i] = a;
      v[jj][2 * i + 1] = b;
      if (QUANT && live && e0 + 2 * i < p.H && e0 + 2 * i + 1 >= 0)
        top = max(top, max(__float_as_uint(fabsf(a)), __float_as_uint(fabsf(b))));
      hv[i] = E::f2_to_u32(a, b);
    }
    if (p.out && live && e0 < p.H) norm_store8<AL>(p.out + t * p.ld_out, e0, p.H, xv[j]);
  }
  if (!QUANT) return;
  top = __reduce_max_sync(0xffffffffu, top);
  if (warps > 1) {
    if ((tid & 31) == 0) smax[w0 + (tid >> 5)] = top;
    __syncthreads();
    top = 0;
    for (int i = 0; i < warps; ++i) top = max(top, smax[w0 + i]);
  }
  // a row whose scale would be subnormal (a row of zeros above all) is 0 times 0
  float scale = __uint_as_float(top) / 448.f;
  const bool none = scale < 1.17549435e-38f;
  if (none) scale = 0.f;
  const float inv = none ? 0.f : 1.f / scale;
  if (live && tid == 0) p.scale[t] = scale;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int e0 = 8 * (j * T + tid) - shift;
    if (live && e0 < p.H) {
      uint2 b;
      const float(&f)[8] = v[QUANT ? j : 0];
      b.x = f4_to_e4m3(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
      b.y = f4_to_e4m3(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv);
      uint8_t* d = p.q + t * p.ld_q + e0;
      bool whole = AL;
      if (!whole) whole = e0 >= 0 && e0 + 8 <= p.H && (reinterpret_cast<uintptr_t>(d) & 7) == 0;
      if (whole) {
        stg64(d, b);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (e0 + i >= 0 && e0 + i < p.H)
            d[i] = static_cast<uint8_t>((i < 4 ? b.x : b.y) >> (8 * (i & 3)));
      }
    }
  }
}

}  // namespace lora
