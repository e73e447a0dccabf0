// w4.cuh -- the base projection with 4-bit weights and group scales, for few
// tokens.
//
//   out[t, n] = rn( sx[t] * sum_g s[g, n] * sum_{k in group g} x[t, k] (q[n, k] - z[g, n]) )
//
// Eight weights are one 32-bit word, value i of the word at bit
// (0, 16, 4, 20, 8, 24, 12, 28)[i]: one mask after shifts by 0, 4, 8 and 12
// gives the pairs (0, 1), (2, 3), (4, 5), (6, 7) in the halves of a register.
// What is multiplied is q - z, which is exact in either element type, so the
// products of a group are exact too and a weight at its zero point adds nothing
// whatever its x; a group's sum is scaled in fp32 before it joins the others.
#pragma once

#include <type_traits>

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

// w4_tc's way from q to q - z: exponent bits next to the low four bits of each
// half make 128 + q (bf16) or 1024 + q (fp16), and 128 + z or 1024 + z is taken off.
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
  if constexpr (std::is_same<E, Fp16>::value)
    return make_uint2(lo.x | (static_cast<uint32_t>(lo.y) << 16),
                      hi.x | (static_cast<uint32_t>(hi.y) << 16));
  const float2 f = __half22float2(__half2(lo)), g = __half22float2(__half2(hi));
  return make_uint2(E::f2_to_u32(f.x, f.y), E::f2_to_u32(g.x, g.y));
}

// C = A (16 x 16, rows of weights) * B (16 x 8, columns of tokens) where
// `fresh`, else C += that.
template <class E>
__device__ __forceinline__ void w4_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                       uint32_t a3, uint32_t b0, uint32_t b1, bool fresh);
template <>
__device__ __forceinline__ void w4_mma<Bf16>(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1, bool fresh) {
  if (fresh)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void w4_mma<Fp16>(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1, bool fresh) {
  if (fresh)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Copies rows of `bytes` bytes at any address to 16-byte aligned rows of
// `pitch` bytes, zeros behind their end: a 16-byte piece a thread, from the two
// aligned pieces that cover it.
__global__ void __launch_bounds__(256) align_rows_kernel(const uint8_t* src, const int64_t ld,
                                                         uint8_t* dst, const int bytes,
                                                         const int pitch, const int64_t pieces) {
  const int per = pitch / 16;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= pieces) return;
  const int64_t t = i / per;
  const int at = static_cast<int>(i - t * per) * 16;
  const uint8_t* p = src + t * ld + at;
  uint4 v = make_uint4(0, 0, 0, 0);
  if (at + 16 <= bytes) {
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15);
    const uint4* q = reinterpret_cast<const uint4*>(p - off);
    v = __ldg(q);
    if (off) v = bytes_at(v, __ldg(q + 1), off);
  } else {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (at + e < bytes) w[e / 4] |= static_cast<uint32_t>(__ldg(p + e)) << (8 * (e & 3));
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
  stg128(dst + i * 16, v);
}

// w4_mv's way, with half the shifts: a row's zero point z, and what turns its
// packed weights into (q - z) / kOut, exactly.  The bit patterns 0 .. 255 of bf16
// and of fp16 are the numbers 0 .. 255 times their smallest subnormal, 2^-133 or
// 2^-24, so four masked bits are q times that, or 16 q where they stand four
// places up: one mask and one fused multiply-add a pair.  (By w4_pairs 24.3
// against 19.3 us for one token, 26.2 against 21.3 us for eight at 4096 x 24576.
// Products of the bare patterns, with z times the group's sum of x taken off
// behind them, took as long as this, lost x outside 2^-57 .. 2^64 in bf16 and
// gave the sums the error of x q rather than of x (q - z).)
template <class E> struct MvZero;
template <> struct MvZero<Bf16> {
  static constexpr float kOut = 0x1p6f;
  __nv_bfloat162 z;
  __device__ __forceinline__ explicit MvZero(uint32_t zero)
      : z(__float2bfloat162_rn(static_cast<float>(zero & 15) * (-1.f / kOut))) {}
  template <int SHIFT>
  __device__ __forceinline__ uint32_t pair(uint32_t w) const {
    w &= 0x000F000Fu << SHIFT;
    const __nv_bfloat162 r = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w),
                                     __float2bfloat162_rn(0x1p127f / (1 << SHIFT)), z);
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};
template <> struct MvZero<Fp16> {
  static constexpr float kOut = 0x1p9f;
  __half2 z;
  __device__ __forceinline__ explicit MvZero(uint32_t zero)
      : z(__float2half2_rn(static_cast<float>(zero & 15) * (-1.f / kOut))) {}
  template <int SHIFT>
  __device__ __forceinline__ uint32_t pair(uint32_t w) const {
    w &= 0x000F000Fu << SHIFT;
    const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&w),
                              __float2half2_rn(0x1p15f / (1 << SHIFT)), z);
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};

constexpr int kMvDepth = 4;  // blocks of 128 K that a warp has in flight
constexpr int kMvWarps = 16, kMvThreads = 32 * kMvWarps;

// Bytes between the staged rows of x: a multiple of 128 plus 64, so that the
// two tokens that a quarter of a warp reads lie in different banks.
__host__ __device__ __forceinline__ int mv_row_bytes(int kc) { return kc * 2 + 64; }

// One block of a warp: 16 rows of 128 weights, and the scale and zero point of
// each of its rows and groups, spread over the lanes of the row: lane t of a
// row holds group t % groups.  All as loaded: arithmetic on a value that is on
// its way would wait for it.
struct MvBlock {
  uint32_t w[2][4];
  uint32_t s[2], z[2];
};

// Few tokens: a block of threads keeps up to 8*NT tokens of x in shared memory
// and goes over tiles of 16 weight rows; its warps share the K range, each
// reading weights straight into registers, several blocks ahead, and multiply
// by mma.sync (16 rows x 8 tokens x 16 K): one fragment of weights serves
// eight tokens without a trip through shared memory.  Widening a word takes one
// shift, four masks and four fused multiply-adds.
//
// The pairs of a fragment may be any 16 values of k as long as both operands
// agree.  Lane t of a row takes VW neighbouring words, so that one load is
// 4*VW bytes and the 16 values of a product lie in one group of 32*VW weights:
// VW = 4, 2, 1 for groups of 128, 64, 32.
//
// A block owns a run of row tiles, and its warps take the run's blocks of
// 16 x 128 weights in turn, on across tile borders, so that together they read
// neighbouring pieces of the same rows.  At the end of a tile the warps' parts
// meet in shared memory and are added in the warps' order.
//
// One block of 16 warps an SM, as two of 8 would stage x twice: 20.6 against
// 22.6 us for 8 tokens (7.7 against 8.5 us for one token at 4096 x 6144).  At
// 4096 x 24576 one token takes 19 us, 2.7 TB/s, where the weights' 52 MB alone
// would take 8: about 5 us are start-up and end, and then the bound is what
// four warps a scheduler issue, some 210 instructions for each KB of weights, 240
// with eight tokens.
// Weights by 8, 16 or 32 rows a warp, deeper prefetch, or three and four
// smaller blocks an SM were all within 5 % of this.
//
// grid = (runs of row tiles, token tiles of `tt` tokens).
template <class E, bool X8, int NT, int VW>
__global__ void __launch_bounds__(kMvThreads, 1)
w4_mv_kernel(const W4Args p, const int tt) {
  using C = typename std::conditional<X8, Fp16, E>::type;  // the operands' type
  extern __shared__ __align__(128) uint8_t mv_smem[];
  constexpr int kSub = 4 / VW;  // groups of a block
  constexpr int WARPS = kMvWarps, kThreads = kMvThreads;
  constexpr int kPart = NT * 128;  // sums of a tile
  // two chains of products a group where there is one fragment of tokens
  constexpr bool kTwo = NT == 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const int t0 = blockIdx.y * tt;
  const int ntok = min(tt, p.tok - t0);
  const int blocks = (p.K + 127) / 128;
  const int rowb = mv_row_bytes(blocks * 128);
  float* part = reinterpret_cast<float*>(mv_smem + tt * rowb);  // [2][WARPS][8 NT][16]
  const int tiles = (p.N + 15) / 16;
  const int run0 = static_cast<int>(static_cast<int64_t>(tiles) * blockIdx.x / gridDim.x);
  const int run1 = static_cast<int>(static_cast<int64_t>(tiles) * (blockIdx.x + 1) / gridDim.x);
  const int last_col = (p.K + 31) / 32 * 16 - 4 * VW;
  const int last_g = (p.K - 1) >> p.group_shift;
  const uint32_t ld_s = static_cast<uint32_t>(p.ld_s);

  // The next block to fetch: its tile, its place in K and the lane's two rows.
  // Columns behind a row's end are read at its last words: x is 0 there, and
  // any weight will do.
  MvBlock buf[kMvDepth];
#pragma unroll
  for (int d = 0; d < kMvDepth; ++d) buf[d].z[0] = buf[d].z[1] = 8;
  int f_tile = run0, f_blk = warp;
  const uint8_t* f_w[2];
  const uint16_t* f_s[2];
  int f_row[2];
  auto rows_of = [&](int tile) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f_row[h] = min(tile * 16 + g + 8 * h, p.N - 1);
      f_w[h] = p.w + f_row[h] * p.ld_w;
      f_s[h] = p.s + f_row[h];
    }
  };
  auto skip = [&]() {  // on to the tile that holds block f_blk
    if (f_blk >= blocks) {
      do {
        f_blk -= blocks;
        ++f_tile;
      } while (f_blk >= blocks);
      rows_of(f_tile);
    }
  };
  rows_of(f_tile);
  skip();
  auto fetch = [&](MvBlock& b) {
    if (f_tile < run1) {
#pragma unroll
      for (int sub = 0; sub < kSub; ++sub) {
        const uint32_t col = min(f_blk * 64 + (sub * 16 + t4 * 4) * VW, last_col);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint8_t* src = f_w[h] + col;
          if constexpr (VW == 4) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(src));
            b.w[h][0] = v.x; b.w[h][1] = v.y; b.w[h][2] = v.z; b.w[h][3] = v.w;
          } else if constexpr (VW == 2) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(src));
            b.w[h][2 * sub] = v.x; b.w[h][2 * sub + 1] = v.y;
          } else {
            b.w[h][sub] = __ldg(reinterpret_cast<const uint32_t*>(src));
          }
        }
      }
      const uint32_t gi = min(f_blk * kSub + (t4 & (kSub - 1)), last_g);
      const uint64_t si = static_cast<uint64_t>(gi) * ld_s;
      b.s[0] = __ldg(f_s[0] + si);
      b.s[1] = __ldg(f_s[1] + si);
      if (p.z) {
        const uint8_t* z = p.z + si;
        b.z[0] = __ldg(z + f_row[0]);
        b.z[1] = __ldg(z + f_row[1]);
      }
      f_blk += WARPS;
      skip();
    }
  };

#pragma unroll
  for (int d = 0; d < kMvDepth; ++d) fetch(buf[d]);

  {
    // x: chunks of eight values, zeros behind K; within a block of 32*VW
    // values chunk c lies at (c % VW) * 4 + c / VW, so that the four lanes
    // of a token read 64 neighbouring bytes
    const int cpr = blocks * 16;
    const int units = ntok * cpr;
    const uint8_t* xb = static_cast<const uint8_t*>(p.x);
    constexpr int kEl = X8 ? 1 : 2, kPiece = 8 * kEl;  // bytes of a value, of a chunk
    // kBatch chunks a thread at a time, all of their loads first: whole chunks
    // as the one or two aligned pieces that cover them
    constexpr int kBatch = 4;
    int r = tid / cpr, c = tid - r * cpr;
    for (int u0 = 0; u0 < units; u0 += kBatch * kThreads) {
      uint4 lo[kBatch], hi[kBatch];
      int rr[kBatch], cc[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        rr[i] = r;
        cc[i] = c;
        lo[i] = hi[i] = make_uint4(0, 0, 0, 0);
        if (u0 + i * kThreads + tid < units && p.K - c * 8 >= 8) {
          const uint8_t* src = xb + ((t0 + r) * p.ld_x + c * 8) * kEl;
          const int off = static_cast<int>(reinterpret_cast<uintptr_t>(src) & (kPiece - 1));
          if constexpr (X8) {
            const uint2* q = reinterpret_cast<const uint2*>(src - off);
            const uint2 d = __ldg(q);
            lo[i].x = d.x; lo[i].y = d.y;
            if (off) {
              const uint2 e = __ldg(q + 1);
              hi[i].x = e.x; hi[i].y = e.y;
            }
          } else {
            const uint4* q = reinterpret_cast<const uint4*>(src - off);
            lo[i] = __ldg(q);
            if (off) hi[i] = __ldg(q + 1);
          }
        }
        c += kThreads;
        while (c >= cpr) {
          c -= cpr;
          ++r;
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const bool live = u0 + i * kThreads + tid < units;
        const int left = live ? p.K - cc[i] * 8 : 0;
        const uint8_t* src = xb + ((t0 + rr[i]) * p.ld_x + cc[i] * 8) * kEl;
        const int off = static_cast<int>(reinterpret_cast<uintptr_t>(src) & (kPiece - 1));
        uint4 v = lo[i];
        uint32_t* o = reinterpret_cast<uint32_t*>(&v);
        if constexpr (X8) {
          uint64_t b = (static_cast<uint64_t>(lo[i].y) << 32 | lo[i].x) >> (8 * off);
          if (off) b |= (static_cast<uint64_t>(hi[i].y) << 32 | hi[i].x) << (64 - 8 * off);
          if (left > 0 && left < 8)
            for (int e = 0; e < left; ++e) b |= static_cast<uint64_t>(__ldg(src + e)) << (8 * e);
          const uint2 x = w4_from_e4m3<C>(static_cast<uint32_t>(b));
          const uint2 y = w4_from_e4m3<C>(static_cast<uint32_t>(b >> 32));
          v = make_uint4(x.x, x.y, y.x, y.y);
        } else {
          if (off) v = bytes_at(lo[i], hi[i], off);
          if (left > 0 && left < 8) {
            v = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (e < left)
                o[e / 2] |= static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(src) + e))
                            << (16 * (e & 1));
          }
        }
        if (live) {
          const int in = cc[i] & (4 * VW - 1);
          const int at = (cc[i] - in) + (in % VW) * 4 + in / VW;
          // a product takes pairs 0 and 2 or 1 and 3 of a word: neighbours here
          *reinterpret_cast<uint4*>(mv_smem + rr[i] * rowb + at * 16) =
              make_uint4(v.x, v.z, v.y, v.w);
        }
      }
    }
  }
  __syncthreads();

  // columns of the product behind the last token repeat one and are not read
  const uint8_t* xr[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) xr[n] = mv_smem + min(8 * n + g, ntok - 1) * rowb + t4 * 16;

  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
  int done = run0, par = 0;  // tiles before `done` are written
  // every warp ends every tile, in order: the tile's parts, then its outputs
  auto end_tile = [&]() {
    float* rb = part + par * (WARPS * kPart);
    par ^= 1;
    float* o = rb + warp * kPart + 2 * t4 * 16 + g;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      o[n * 128] = acc[n][0];
      o[n * 128 + 16] = acc[n][1];
      o[n * 128 + 8] = acc[n][2];
      o[n * 128 + 24] = acc[n][3];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
    }
    __syncthreads();
    for (int e = tid; e < kPart; e += kThreads) {
      const int tk = e >> 4, row = done * 16 + (e & 15);
      if (tk < ntok && row < p.N) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) v += rb[w * kPart + e];
        v *= MvZero<C>::kOut;
        if (X8) v *= __ldg(p.x_scale + t0 + tk);
        stg16(p.out + (t0 + tk) * p.ld_out + row, E::f32_to_bits(v));
      }
    }
    ++done;
  };

  int tile = run0, blk = warp;
  while (blk >= blocks) {
    blk -= blocks;
    ++tile;
  }
  while (tile < run1) {
#pragma unroll
    for (int d = 0; d < kMvDepth; ++d) {
      if (tile >= run1) break;
      while (done < tile) end_tile();
      const MvBlock& b = buf[d];
      const uint32_t sz[2] = {b.s[0] | (b.z[0] << 16), b.s[1] | (b.z[1] << 16)};
#pragma unroll
      for (int sub = 0; sub < kSub; ++sub) {
        uint32_t sz0 = sz[0], sz1 = sz[1];
        if (kSub > 1) {
          sz0 = __shfl_sync(0xffffffffu, sz0, (lane & ~3) + sub);
          sz1 = __shfl_sync(0xffffffffu, sz1, (lane & ~3) + sub);
        }
        const MvZero<C> z0(sz0 >> 16), z1(sz1 >> 16);
        float g1[NT][4], g2[kTwo ? NT : 1][4];
#pragma unroll
        for (int j = 0; j < VW; ++j) {
          const uint32_t a = b.w[0][sub * VW + j], e = b.w[1][sub * VW + j];
          const uint32_t a8 = a >> 8, e8 = e >> 8;
          const uint32_t p0 = z0.template pair<0>(a), p1 = z0.template pair<4>(a),
                         p2 = z0.template pair<0>(a8), p3 = z0.template pair<4>(a8);
          const uint32_t q0 = z1.template pair<0>(e), q1 = z1.template pair<4>(e),
                         q2 = z1.template pair<0>(e8), q3 = z1.template pair<4>(e8);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint4 xv =
                *reinterpret_cast<const uint4*>(xr[n] + blk * 256 + (sub * VW + j) * 64);
            w4_mma<C>(g1[n], p0, q0, p2, q2, xv.x, xv.y, j == 0);
            if constexpr (kTwo)
              w4_mma<C>(g2[n], p1, q1, p3, q3, xv.z, xv.w, j == 0);
            else
              w4_mma<C>(g1[n], p1, q1, p3, q3, xv.z, xv.w, false);
          }
        }
        // a group behind K was given the last one's scale, which may be infinite;
        // its sums are 0 (to load nothing there instead took 14.7 against 11.4 us
        // for 4 tokens x 4096 x 6144 in groups of 32)
        if (kSub > 1 && blk * kSub + sub > last_g) sz0 = sz1 = 0;
        const float s0 = E::bits_to_f32(static_cast<uint16_t>(sz0));
        const float s1 = E::bits_to_f32(static_cast<uint16_t>(sz1));
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if constexpr (kTwo) {
#pragma unroll
            for (int i = 0; i < 4; ++i) g1[n][i] += g2[n][i];
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[n][i] = fmaf(i < 2 ? s0 : s1, g1[n][i], acc[n][i]);
        }
      }
      fetch(buf[d]);
      blk += WARPS;
      while (blk >= blocks) {
        blk -= blocks;
        ++tile;
      }
    }
  }
  while (done < run1) end_tile();
}

}  // namespace lora
