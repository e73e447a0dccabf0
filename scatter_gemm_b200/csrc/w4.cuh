// w4.cuh -- the base projection with 4-bit weights and group scales, for few
// tokens.
//
//   out[t, n] = rn( sx[t] * sum_g s[g, n] * sum_{k in group g} x[t, k] (q[n, k] - z[g, n]) )
//
// Eight weights are one 32-bit word, value i of the word at bit
// (0, 16, 4, 20, 8, 24, 12, 28)[i]: one mask after shifts by 0, 4, 8 and 12
// gives the pairs (0, 1), (2, 3), (4, 5), (6, 7) in the halves of a register,
// next to the exponent bits that make them 128 + q (bf16) or 1024 + q (fp16).
// Subtracting 128 + z or 1024 + z is exact, so the products of a group are
// exact too; a group's sum is scaled in fp32 before it joins the others.
#pragma once

#include "common.cuh"
#include "rmsnorm.cuh"
#include "sm100.cuh"

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

// The bits that turn the low four bits of each half into a number, and that number.
template <class E> struct W4Magic;
template <> struct W4Magic<Bf16> {
  static constexpr uint32_t kBits = 0x43004300u;  // 128 + q
  // the pair (128 + z, 128 + z)
  static __device__ __forceinline__ uint32_t zero(int z) {
    return kBits | (static_cast<uint32_t>(z) * 0x00010001u);
  }
  static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a),
                                     *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};
template <> struct W4Magic<Fp16> {
  static constexpr uint32_t kBits = 0x64006400u;  // 1024 + q
  static __device__ __forceinline__ uint32_t zero(int z) {
    return kBits | (static_cast<uint32_t>(z) * 0x00010001u);
  }
  static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
    const __half2 r = __hsub2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};

// The eight weights q - z of a word as four pairs; zz = zero(z).
template <class E>
__device__ __forceinline__ void w4_pairs(uint32_t w, uint32_t zz, uint32_t (&p)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    p[i] = W4Magic<E>::sub(((w >> (4 * i)) & 0x000F000Fu) | W4Magic<E>::kBits, zz);
}

// Four e4m3 bytes -> four elements of type E (exact).
template <class E>
__device__ __forceinline__ uint2 w4_from_e4m3(uint32_t b) {
  const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(b & 0xFFFFu),
                                                    __NV_E4M3);
  const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(b >> 16),
                                                    __NV_E4M3);
  const float2 f = __half22float2(__half2(lo)), g = __half22float2(__half2(hi));
  return make_uint2(E::f2_to_u32(f.x, f.y), E::f2_to_u32(g.x, g.y));
}

// C += A (16 x 16, rows of weights) * B (16 x 8, columns of tokens).
template <class E>
__device__ __forceinline__ void w4_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                       uint32_t a3, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void w4_mma<Bf16>(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void w4_mma<Fp16>(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int kMvWarps = 8;
constexpr int kMvThreads = 32 * kMvWarps;
constexpr int kMvDepth = 4;  // blocks of 128 K that a warp has in flight

// Bytes between the staged rows of x: a multiple of 128 plus 64, so that the
// two tokens that a quarter of a warp reads lie in different banks.
__host__ __device__ __forceinline__ int mv_row_bytes(int kc) { return kc * 2 + 64; }

// One block of a warp: 16 rows of 128 weights, its scales and zero points.
template <int VW>
struct MvBlock {
  uint32_t w[2][4];
  uint16_t s[2][4 / VW];
  uint8_t z[2][4 / VW];
};

// Few tokens: a block of threads keeps up to 8*NT tokens of x in shared memory
// and goes over tiles of 16 weight rows; its warps share the K range, each
// reading weights straight into registers, several blocks ahead, and multiply
// by mma.sync (16 rows x 8 tokens x 16 K): one fragment of weights serves
// eight tokens without a trip through shared memory.
//
// The pairs of a fragment may be any 16 values of k as long as both operands
// agree.  Lane t of a row takes VW neighbouring words, so that one load is
// 4*VW bytes and the 16 values of a product lie in one group of 32*VW weights:
// VW = 4, 2, 1 for groups of 128, 64, 32.
//
// grid = (row tiles in turn, token tiles).  kc: values of x staged at a time
// (all of K wherever they fit).
template <class E, bool X8, int NT, int VW>
__global__ void __launch_bounds__(kMvThreads) w4_mv_kernel(const W4Args p, const int kc) {
  extern __shared__ __align__(128) uint8_t mv_smem[];
  constexpr int kSub = 4 / VW;  // groups of a block
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const int t0 = blockIdx.y * 8 * NT;
  const int ntok = min(8 * NT, p.tok - t0);
  const int rowb = mv_row_bytes(kc);
  float* red = reinterpret_cast<float*>(mv_smem + ntok * rowb);  // [2][warps][8 NT][16]
  const int tiles = (p.N + 15) / 16;
  const int row_bytes = (p.K + 31) / 32 * 16;
  const int chunks = (p.K + kc - 1) / kc;

  for (int tile_base = blockIdx.x; tile_base < tiles;
       tile_base += chunks == 1 ? tiles : static_cast<int>(gridDim.x)) {
    // with one chunk the loop below goes over all tiles of this block
    const int my_tiles = chunks == 1 ? (tiles - tile_base + gridDim.x - 1) / gridDim.x : 1;
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
    for (int ch = 0; ch < chunks; ++ch) {
      const int k_lo = ch * kc, k_hi = min(p.K, k_lo + kc);
      const int blocks = (k_hi - k_lo + 127) / 128;
      const int per = (blocks + kMvWarps - 1) / kMvWarps;
      const int total = per * my_tiles;
      MvBlock<VW> buf[kMvDepth];

      auto fetch = [&](int it, MvBlock<VW>& b) {
        const int tile = tile_base + (it / per) * static_cast<int>(gridDim.x);
        const int blk = (it % per) * kMvWarps + warp;
        const bool live = it < total && blk < blocks;
        const int kb = k_lo / 128 + blk;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = min(tile * 16 + g + 8 * h, p.N - 1);
          const uint8_t* src = p.w + static_cast<int64_t>(row) * p.ld_w;
#pragma unroll
          for (int sub = 0; sub < kSub; ++sub) {
            const int at = kb * 64 + sub * 16 * VW + t4 * 4 * VW;
            const bool in = live && at < row_bytes;
            if constexpr (VW == 4) {
              uint4 v = make_uint4(0, 0, 0, 0);
              if (in) v = __ldcs(reinterpret_cast<const uint4*>(src + at));
              b.w[h][0] = v.x; b.w[h][1] = v.y; b.w[h][2] = v.z; b.w[h][3] = v.w;
            } else if constexpr (VW == 2) {
              uint2 v = make_uint2(0, 0);
              if (in) v = __ldg(reinterpret_cast<const uint2*>(src + at));
              b.w[h][2 * sub] = v.x; b.w[h][2 * sub + 1] = v.y;
            } else {
              b.w[h][sub] = in ? __ldg(reinterpret_cast<const uint32_t*>(src + at)) : 0u;
            }
            const int k = kb * 128 + sub * 32 * VW;
            const int64_t si = static_cast<int64_t>(k >> p.group_shift) * p.ld_s + row;
            const bool sin = live && k < p.K;
            b.s[h][sub] = sin ? __ldg(p.s + si) : static_cast<uint16_t>(0);
            b.z[h][sub] = sin && p.z ? __ldg(p.z + si) : static_cast<uint8_t>(8);
          }
        }
      };

#pragma unroll
      for (int d = 0; d < kMvDepth; ++d) fetch(d, buf[d]);

      // x: chunks of eight values, zeros behind K; within a block of 32*VW
      // values chunk c lies at (c % VW) * 4 + c / VW, so that the four lanes
      // of a token read 64 neighbouring bytes
      if (ch > 0 || tile_base != static_cast<int>(blockIdx.x)) __syncthreads();
      const int cpr = blocks * 16;
      for (int u = tid; u < ntok * cpr; u += kMvThreads) {
        const int r = u / cpr, c = u % cpr;
        const int k = k_lo + c * 8;
        const int left = min(8, p.K - k);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (left > 0) {
          const int64_t at = static_cast<int64_t>(t0 + r) * p.ld_x + k;
          uint32_t* o = reinterpret_cast<uint32_t*>(&v);
          if (X8) {
            const uint8_t* src = static_cast<const uint8_t*>(p.x) + at;
            uint32_t b[2] = {0, 0};
            if (left == 8 && (reinterpret_cast<uintptr_t>(src) & 7) == 0) {
              const uint2 d = __ldg(reinterpret_cast<const uint2*>(src));
              b[0] = d.x; b[1] = d.y;
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (i < left) b[i / 4] |= static_cast<uint32_t>(__ldg(src + i)) << (8 * (i & 3));
            }
            const uint2 lo = w4_from_e4m3<E>(b[0]), hi = w4_from_e4m3<E>(b[1]);
            v = make_uint4(lo.x, lo.y, hi.x, hi.y);
          } else {
            const uint16_t* src = static_cast<const uint16_t*>(p.x) + at;
            if (left == 8 && (reinterpret_cast<uintptr_t>(src) & 15) == 0) {
              v = __ldg(reinterpret_cast<const uint4*>(src));
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (i < left) o[i / 2] |= static_cast<uint32_t>(__ldg(src + i)) << (16 * (i & 1));
            }
          }
        }
        const int in = c & (4 * VW - 1);
        const int at = (c - in) + (in % VW) * 4 + in / VW;
        *reinterpret_cast<uint4*>(mv_smem + r * rowb + at * 16) = v;
      }
      __syncthreads();

      const uint8_t* xr[NT];
      bool xin[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        xin[n] = 8 * n + g < ntok;
        xr[n] = mv_smem + (xin[n] ? 8 * n + g : 0) * rowb + t4 * 16;
      }

      for (int it0 = 0; it0 < total; it0 += kMvDepth) {
#pragma unroll
        for (int d = 0; d < kMvDepth; ++d) {
          const int it = it0 + d;
          if (it >= total) break;
          const int blk = (it % per) * kMvWarps + warp;
          if (blk < blocks) {
            const MvBlock<VW>& b = buf[d];
#pragma unroll
            for (int sub = 0; sub < kSub; ++sub) {
              float gr[NT][4];
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) gr[n][i] = 0.f;
              const uint32_t z0 = W4Magic<E>::zero(b.z[0][sub] & 15);
              const uint32_t z1 = W4Magic<E>::zero(b.z[1][sub] & 15);
#pragma unroll
              for (int j = 0; j < VW; ++j) {
                uint32_t a[4], c[4];
                w4_pairs<E>(b.w[0][sub * VW + j], z0, a);
                w4_pairs<E>(b.w[1][sub * VW + j], z1, c);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                  uint4 xv = make_uint4(0, 0, 0, 0);
                  if (xin[n])
                    xv = *reinterpret_cast<const uint4*>(xr[n] + blk * 256 + (sub * VW + j) * 64);
                  w4_mma<E>(gr[n], a[0], c[0], a[1], c[1], xv.x, xv.y);
                  w4_mma<E>(gr[n], a[2], c[2], a[3], c[3], xv.z, xv.w);
                }
              }
              const float s0 = E::bits_to_f32(b.s[0][sub]), s1 = E::bits_to_f32(b.s[1][sub]);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                acc[n][0] = fmaf(s0, gr[n][0], acc[n][0]);
                acc[n][1] = fmaf(s0, gr[n][1], acc[n][1]);
                acc[n][2] = fmaf(s1, gr[n][2], acc[n][2]);
                acc[n][3] = fmaf(s1, gr[n][3], acc[n][3]);
              }
            }
          }
          fetch(it + kMvDepth, buf[d]);
          if (ch == chunks - 1 && it % per == per - 1) {
            // the tile is done: add the warps' parts in their order
            const int ti = it / per;
            float* rb = red + (ti & 1) * (kMvWarps * NT * 128);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              float* w = rb + (warp * NT + n) * 128 + 2 * t4 * 16 + g;
              w[0] = acc[n][0];
              w[16] = acc[n][1];
              w[8] = acc[n][2];
              w[24] = acc[n][3];
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
            }
            __syncthreads();
            const int n0 = (tile_base + ti * static_cast<int>(gridDim.x)) * 16;
            for (int e = tid; e < NT * 128; e += kMvThreads) {
              const int tk = e >> 4, row = n0 + (e & 15);
              if (tk < ntok && row < p.N) {
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < kMvWarps; ++w) v += rb[w * NT * 128 + e];
                if (X8) v *= __ldg(p.x_scale + t0 + tk);
                stg16(p.out + static_cast<int64_t>(t0 + tk) * p.ld_out + row, E::f32_to_bits(v));
              }
            }
          }
        }
      }
    }
  }
}

}  // namespace lora
