// w4_tc.cuh -- the base projection with 4-bit weights on the tensor cores
// (sm_100a), for more than a few tokens.
//
//   out[t, n] = rn( sx[t] * sum_g s[g, n] * sum_{k in group g} x[t, k] (q[n, k] - z[g, n]) )
//
// A tile is 128 weight rows x NT tokens; the weight rows are the rows of the
// MMA, so that a weight's row is a lane of tensor memory (TMEM) and its scale a
// scalar of the thread that owns the lane.  K goes in blocks of 128:
//  - one thread loads the block's packed weights (8 KB) and x tile by TMA;
//  - the widening warps turn each packed row into q - z in the element type of
//    x (exact: bf16, fp16, or e4m3 scaled by 2^-6) and store it to TMEM, from
//    where the MMA reads it: neither the widened weights' stores nor their
//    loads by the MMA take shared-memory bandwidth;
//  - one thread issues the MMAs of a group into one of two accumulators;
//  - the scaling warps add each group's accumulator, times its scale, to fp32
//    sums in registers, while the next group is multiplied into the other.
// So the weights are never rounded, and a scale costs one fused multiply-add
// for each group and output instead of a multiplication for each weight.
//
// With few tiles the K range is split over a thread-block cluster; the parts
// are added in rank order through distributed shared memory.
#pragma once

#include "common.cuh"
#include "sm100.cuh"
#include "w4.cuh"

namespace lora {

constexpr int kW4M = 128;   // weight rows of a tile
constexpr int kW4K = 128;   // K of a block

struct W4TcParams {
  CUtensorMap tmap_w;  // bytes: [N rows, row bytes], box {64, 128}, 64-byte swizzle
  CUtensorMap tmap_x;  // [tok rows, K], box {128 bytes, NT}, 128-byte swizzle
  W4Args a;
  int tiles_n, tiles_t;  // tiles of weight rows and of tokens
  int nkb;               // K blocks
  int cs;                // CTAs of a cluster, which share a tile's K blocks
  int stages;
  uint32_t idesc;
};

// A from tensor memory: D[tmem] (+)= A[tmem] * B[smem desc]^T.
template <bool X8>
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  if constexpr (X8)
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0; "
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p; }" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0; "
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 32 lanes x 32 bit, 16 consecutive columns: register i of lane l goes to
// column col + i of TMEM lane (warp_quarter*32 + l).
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// e4m3 codes of (q - z) * 2^-6 without their sign bit, the sign in bit 6
// instead (the codes of 1/64 .. 15/64 leave it free): byte q of the table of z.
__device__ __forceinline__ uint32_t w4_code8(int q, int z) {
  const int d = q - z, m = d < 0 ? -d : d;
  if (m == 0) return 0u;
  const int e = 31 - __clz(m);                       // m = 1.f * 2^e
  return (d < 0 ? 0x40u : 0u) | static_cast<uint32_t>((e + 1) << 3) |
         static_cast<uint32_t>(((m << 3) >> e) & 7);
}

// Four of the eight bytes of y:x by the low four 4-bit selectors of s; a
// selector's high bit asks for eight copies of the byte's sign bit.
__device__ __forceinline__ uint32_t prmt(uint32_t x, uint32_t y, uint32_t s) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(y), "r"(s));
  return r;
}

// The eight weights of a word in e4m3, four to a register; T is the table of
// the row's zero point.  A byte permutation takes four 3-bit indices; an index
// with its fourth bit set gives the sign of a table byte, and those are 0.
__device__ __forceinline__ void w4_bytes8(uint32_t w, const uint4& T, uint32_t& a, uint32_t& b) {
  const uint32_t v = w ^ 0x88888888u;
  const uint32_t even = prmt(T.x, T.y, w) | prmt(T.z, T.w, v);
  const uint32_t odd = prmt(T.x, T.y, w >> 16) | prmt(T.z, T.w, v >> 16);
  a = prmt(even, odd, 0x5140);
  b = prmt(even, odd, 0x7362);
  a += a & 0x40404040u;  // the sign from bit 6 to bit 7
  b += b & 0x40404040u;
}

// NT: tokens of a tile.  GS: log2 of the group size.  NW: widening warps and
// scaling warps each (4 or 8; with 8 the scaling warps split the tokens).
template <class E, bool X8, int NT, int GS, int NW>
struct W4Tc {
  static constexpr int kThreads = 64 * NW + 64;
  static constexpr int kGroups = 128 >> GS;                     // groups of a block
  static constexpr int kACols = X8 ? 32 : 64;                   // TMEM columns of a widened block
  static constexpr int kTmem = NT > 64 ? 512 : 256;
  static constexpr int kABufs = (kTmem - 2 * NT) / kACols >= 4 ? 4 : (kTmem - 2 * NT) / kACols;
  static constexpr int kWBytes = kW4M * 64;
  static constexpr int kXBytes = NT * (X8 ? 128 : 256);
  static constexpr int kStage = kWBytes + kXBytes;
  static constexpr int kCols = NT / (NW / 4);                   // tokens of a scaling warp
  static constexpr int kMinBlocks = NW == 4 ? 2 : 1;
  static_assert(kABufs >= 2, "two widened blocks at least");
};

template <class E, bool X8, int NT, int GS, int NW>
__global__ void __launch_bounds__((W4Tc<E, X8, NT, GS, NW>::kThreads),
                                  (W4Tc<E, X8, NT, GS, NW>::kMinBlocks))
w4_tc_kernel(const __grid_constant__ W4TcParams P) {
  using C = W4Tc<E, X8, NT, GS, NW>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const W4Args& p = P.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  // [ring of stages, later the split sums][code tables][barriers][TMEM address]
  uint4* codes = reinterpret_cast<uint4*>(smem + P.stages * C::kStage);
  uint64_t* bars = reinterpret_cast<uint64_t*>(codes + 16);
  const uint32_t full0 = smem_u32(bars);
  const uint32_t empty0 = full0 + 8 * P.stages;
  const uint32_t afull0 = empty0 + 8 * P.stages;
  const uint32_t aempty0 = afull0 + 8 * C::kABufs;
  const uint32_t dfull0 = aempty0 + 8 * C::kABufs;
  const uint32_t dempty0 = dfull0 + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * P.stages + 2 * C::kABufs + 4);

  if (tid == 0) {
    for (int s = 0; s < P.stages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, NW + 1);  // the widening warps and the MMAs
    }
    for (int s = 0; s < C::kABufs; ++s) {
      mbar_init(afull0 + 8 * s, NW);
      mbar_init(aempty0 + 8 * s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(dfull0 + 8 * s, 1);
      mbar_init(dempty0 + 8 * s, NW);
    }
    fence_mbar_init();
  }
  if (X8 && tid < 64) {
    // word tid % 4 of the table of zero point tid / 4
    uint32_t c = 0;
    for (int i = 0; i < 4; ++i) c |= w4_code8(4 * (tid & 3) + i, tid >> 2) << (8 * i);
    reinterpret_cast<uint32_t*>(codes)[tid] = c;
  }
  if (warp == 2 * NW) {
    if (lane == 0) {
      tma_prefetch_desc(&P.tmap_w);
      tma_prefetch_desc(&P.tmap_x);
    }
  } else if (warp == 2 * NW + 1) {
    tmem_alloc(smem_u32(tmem_slot), C::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t abase = tmem + 2 * NT;
  const int rank = P.cs > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int kb0 = static_cast<int>(static_cast<int64_t>(P.nkb) * rank / P.cs);
  const int kb1 = static_cast<int>(static_cast<int64_t>(P.nkb) * (rank + 1) / P.cs);
  const int tiles = P.tiles_n * P.tiles_t;
  const int first = blockIdx.x / P.cs, step = gridDim.x / P.cs;
  bool ok = true;

  if (warp < NW) {
    // =========================== widening: a lane of TMEM, and a row, a thread
    const int quad = warp & 3;
    const int row = quad * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t rsw = (row >> 1) & 3;
    constexpr int kHalves = NW == 4 ? 2 : 1;
    const int h0 = NW == 4 ? 0 : warp >> 2;
    int it = 0;
    for (int tile = first; tile < tiles && ok; tile += step) {
      const int n = (tile % P.tiles_n) * kW4M + row;
      const bool zin = p.z != nullptr && n < p.N;
      // the zero points of a block, a byte each, four blocks ahead
      auto zeros = [&](int kb) {
        uint32_t v = 0x08080808u;
        if (zin && kb < kb1) {
          v = 0;
#pragma unroll
          for (int i = 0; i < C::kGroups; ++i) {
            const int gi = kb * C::kGroups + i;
            if ((gi << GS) < p.K)
              v |= static_cast<uint32_t>(__ldg(p.z + gi * p.ld_s + n) & 15) << (8 * i);
          }
        }
        return v;
      };
      uint32_t zq[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) zq[i] = zeros(kb0 + i);
      for (int kb = kb0; kb < kb1 && ok; ++kb, ++it) {
        const uint32_t z4 = zq[0];
        zq[0] = zq[1]; zq[1] = zq[2]; zq[2] = zq[3];
        zq[3] = zeros(kb + 4);
        const int s = it % P.stages;
        ok = mbar_wait(full0 + 8 * s, (it / P.stages) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint8_t* src = smem + s * C::kStage + row * 64;
        uint4 pk[2 * kHalves];
#pragma unroll
        for (int c = 0; c < 2 * kHalves; ++c)
          pk[c] = *reinterpret_cast<const uint4*>(src + (((2 * h0 + c) ^ rsw) << 4));
        const int ab = it % C::kABufs;
        if (it >= C::kABufs) ok = mbar_wait(aempty0 + 8 * ab, (it / C::kABufs - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t dst = abase + lane_off + ab * C::kACols;
#pragma unroll
        for (int c = 0; c < 2 * kHalves; ++c) {
          // 32 weights, one group at most
          const int c4 = 2 * h0 + c;
          const int z = (z4 >> (8 * ((c4 * 32) >> GS))) & 15;
          const uint32_t w[4] = {pk[c].x, pk[c].y, pk[c].z, pk[c].w};
          if constexpr (X8) {
            if (c & 1) continue;
            const int z2 = (z4 >> (8 * (((c4 + 1) * 32) >> GS))) & 15;
            const uint32_t w2[4] = {pk[c + 1].x, pk[c + 1].y, pk[c + 1].z, pk[c + 1].w};
            const uint4 T = codes[z], T2 = codes[z2];
            uint32_t r[16];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              w4_bytes8(w[j], T, r[2 * j], r[2 * j + 1]);
              w4_bytes8(w2[j], T2, r[8 + 2 * j], r[9 + 2 * j]);
            }
            tmem_st16(dst + c4 * 8, r);
          } else {
            const uint32_t zz = W4Magic<E>::zero(z);
            uint32_t r[16];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t q[4];
              w4_pairs<E>(w[j], zz, q);
              r[4 * j] = q[0]; r[4 * j + 1] = q[1]; r[4 * j + 2] = q[2]; r[4 * j + 3] = q[3];
            }
            tmem_st16(dst + c4 * 16, r);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(afull0 + 8 * ab);
          mbar_arrive(empty0 + 8 * s);
        }
      }
    }
  } else if (warp < 2 * NW) {
    // =========================== scaling: sum += scale * accumulator, then the output
    const int w = warp - NW, quad = w & 3;
    const int row = quad * 32 + lane;
    const int col0 = (w >> 2) * C::kCols;
    const uint32_t dsrc = tmem + (static_cast<uint32_t>(quad * 32) << 16) + col0;
    int gi = 0;
    for (int tile = first; tile < tiles; tile += step) {
      const int n = (tile % P.tiles_n) * kW4M + row;
      const int tb = (tile / P.tiles_n) * NT;
      const int g0 = kb0 * C::kGroups, g1 = kb1 * C::kGroups;
      auto scale_of = [&](int g) {
        return n < p.N && g < g1 && (g << GS) < p.K
                   ? E::bits_to_f32(__ldg(p.s + g * p.ld_s + n))
                   : 0.f;
      };
      float acc[C::kCols];
#pragma unroll
      for (int c = 0; c < C::kCols; ++c) acc[c] = 0.f;
      float sq[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) sq[i] = scale_of(g0 + i);
      for (int g = g0; g < g1 && ok; ++g, ++gi) {
        const float sc = X8 ? sq[0] * 64.f : sq[0];
        sq[0] = sq[1]; sq[1] = sq[2]; sq[2] = sq[3];
        sq[3] = scale_of(g + 4);
        const int db = gi & 1;
        ok = mbar_wait(dfull0 + 8 * db, (gi >> 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < C::kCols; c += 16) {
          float v[16];
          tmem_ld16(dsrc + db * NT + c, v);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[c + i] = fmaf(sc, v[i], acc[c + i]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(dempty0 + 8 * db);
      }
      if (!ok) break;
      if (P.cs == 1) {
        if (n < p.N) {
#pragma unroll
          for (int c = 0; c < C::kCols; ++c) {
            const int t = tb + col0 + c;
            if (t < p.tok) {
              const float v = X8 ? acc[c] * __ldg(p.x_scale + t) : acc[c];
              stg16(p.out + t * p.ld_out + n, E::f32_to_bits(v));
            }
          }
        }
      } else {
        // this CTA's part: [token][row] over the ring, whose copies and MMAs
        // are all done
        float* part = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int c = 0; c < C::kCols; ++c) part[(col0 + c) * kW4M + row] = acc[c];
      }
    }
  } else if (warp == 2 * NW) {
    // =========================== TMA
    if (lane == 0) {
      int it = 0;
      for (int tile = first; tile < tiles && ok; tile += step) {
        const int n0 = (tile % P.tiles_n) * kW4M, tb = (tile / P.tiles_n) * NT;
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          const int s = it % P.stages;
          if (it >= P.stages) ok = mbar_wait(empty0 + 8 * s, (it / P.stages - 1) & 1);
          if (!ok) break;
          const uint32_t dst = sbase + s * C::kStage, bar = full0 + 8 * s;
          mbar_arrive_expect_tx(bar, C::kStage);
          tma_load_2d(dst, &P.tmap_w, bar, kb * 64, n0);
          tma_load_2d(dst + C::kWBytes, &P.tmap_x, bar, kb * kW4K, tb);
          if (!X8) tma_load_2d(dst + C::kWBytes + NT * 128, &P.tmap_x, bar, kb * kW4K + 64, tb);
        }
      }
      // after a wait that gave up: the copies still in flight
      if (!ok)
        for (int i = it < P.stages ? 0 : it - P.stages; i < it; ++i)
          mbar_wait(full0 + 8 * (i % P.stages), (i / P.stages) & 1);
    }
    __syncwarp();
  } else {
    // =========================== MMA
    if (lane == 0) {
      int it = 0, gi = 0;
      for (int tile = first; tile < tiles && ok; tile += step) {
        for (int kb = kb0; kb < kb1 && ok; ++kb, ++it) {
          const int s = it % P.stages, ab = it % C::kABufs;
          ok = mbar_wait(full0 + 8 * s, (it / P.stages) & 1) &&
               mbar_wait(afull0 + 8 * ab, (it / C::kABufs) & 1);
          const uint32_t xs = sbase + s * C::kStage + C::kWBytes;
          constexpr int kSteps = X8 ? 4 : 8;           // MMAs of a block
          constexpr int kPer = kSteps / C::kGroups;    // MMAs of a group
#pragma unroll
          for (int j = 0; j < C::kGroups && ok; ++j, ++gi) {
            const int db = gi & 1;
            if (gi >= 2) ok = mbar_wait(dempty0 + 8 * db, ((gi >> 1) - 1) & 1);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
              const int kk = j * kPer + i;
              const uint64_t bd = make_sdesc(xs + (kk / 4) * NT * 128 + (kk % 4) * 32, 128, 2);
              tc_mma_ts<X8>(tmem + db * NT, abase + ab * C::kACols + kk * 8, bd, P.idesc,
                            i > 0 ? 1u : 0u);
            }
            if (j == C::kGroups - 1) {
              tc_commit(aempty0 + 8 * ab);
              tc_commit(empty0 + 8 * s);
            }
            tc_commit(dfull0 + 8 * db);
          }
        }
      }
    }
    __syncwarp();
  }

  if (P.cs > 1) {
    // one tile: the parts of the cluster's CTAs, each CTA adding its share of
    // the tokens in rank order
    ok = __syncthreads_and(ok);
    cluster_sync();
    const int tb = (first / P.tiles_n) * NT, n0 = (first % P.tiles_n) * kW4M;
    const uint32_t mine = sbase;
    const int c0 = NT * rank / P.cs, c1 = NT * (rank + 1) / P.cs;
    for (int e = tid; e < (c1 - c0) * kW4M; e += C::kThreads) {
      const int c = c0 + e / kW4M, r = e % kW4M;
      const int t = tb + c, n = n0 + r;
      if (t < p.tok && n < p.N && ok) {
        float v = 0.f;
        for (int i = 0; i < P.cs; ++i)
          v += ld_dsmem_f32(mapa_shared(mine + static_cast<uint32_t>(c * kW4M + r) * 4, i));
        if (X8) v *= __ldg(p.x_scale + t);
        stg16(p.out + t * p.ld_out + n, E::f32_to_bits(v));
      }
    }
    cluster_sync_relaxed();
  }
  __syncthreads();
  if (warp == 2 * NW + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
}

}  // namespace lora
