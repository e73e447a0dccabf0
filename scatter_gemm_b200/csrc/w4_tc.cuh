// w4_tc.cuh -- the base projection with 4-bit weights on the tensor cores
// (sm_100a), for more than a few tokens.
//
//   out[t, n] = rn( sx[t] * sum_g s[g, n] * sum_{k in group g} x[t, k] (q[n, k] - z[g, n]) )
//
// A tile is 128 weight rows x NT tokens; the weight rows are the rows of the
// MMA, so that a weight's row is a lane of tensor memory (TMEM) and its scale a
// scalar of the thread that owns the lane.  K goes in blocks of 128:
//  - two warps load the blocks' packed weights (8 KB each) and x tiles by TMA;
//  - sets of four widening warps, a block each in turn, turn the packed rows
//    into q - z in the element type of x (exact: bf16, fp16, or e4m3 scaled by
//    2^-6) and store them to TMEM, from where the MMA reads them: neither the
//    widened weights' stores nor their loads by the MMA take shared-memory
//    bandwidth;
//  - two warps issue the MMAs, a group each in turn, into a ring of
//    accumulators;
//  - the scaling warps add each group's accumulator, times its scale, to fp32
//    sums in registers.
// So the weights are never rounded, and a scale costs one fused multiply-add
// for each group and output instead of a multiplication for each weight.  One
// block of threads an SM, most of an SM's shared memory and all of its TMEM.
//
// A role's own path through a block, its barriers above all, takes 500 to 1200
// cycles, the block's data 340 (8 KB at an SM's share of the memory
// bandwidth): hence the sets of widening warps and the two MMA warps.
//
// With few tiles the K range is split over a thread-block cluster; the parts
// are added in rank order through distributed shared memory.
//
// 2048 tokens x 5120 x 7168: 148 us, 1.01 PFLOP/s, the tensor pipe 50 % and the
// issue slots 72 % busy: a block of 128 tokens takes some 2,900 warp
// instructions where the tensor pipe's 512 cycles have 2,048 slots.  With groups
// of 64 and 32, two and four accumulators a block: 211 and 360 us; with 8-bit x
// 157, and 446 with groups of 32 (128 tokens of 8-bit x in groups of 64 or 32
// spill 32 to 34 bytes a thread, 32 tokens 8, or 20 of 16-bit x in groups of
// 128).  9 tokens x 4096 x 6144: 10.7 us; 64 tokens: 14.3 us.
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
  int tile0, tile1;      // this launch's tiles
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

// A role's place in a ring of n buffers: the buffer, and the parity of the
// phase in which it is filled (`fill`) or was last drained (`drain`; a fresh
// barrier passes a wait for parity 1).
struct RingPos {
  int i = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ uint32_t fill() const { return ph; }
  __device__ __forceinline__ uint32_t drain() const { return ph ^ 1u; }
  __device__ __forceinline__ void next(int n) {
    if (++i == n) {
      i = 0;
      ph ^= 1u;
    }
  }
};

// Two fp32 values in a 64-bit register, for the fused multiply-add of pairs:
// c = a * s + c in each half, each rounded as one fma.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ void fma2(uint64_t& c, uint64_t a, uint64_t s) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c) : "l"(a), "l"(s));
}

// Loads that stay where they are written: the compiler may move an ordinary
// load of constant data down to its use, and the prefetch is gone.
__device__ __forceinline__ uint32_t ld_early(const uint16_t* p) {
  uint16_t v;
  asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(v) : "l"(__cvta_generic_to_global(p)));
  return v;
}
__device__ __forceinline__ uint32_t ld_early(const uint8_t* p) {
  uint32_t v;
  asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(v) : "l"(__cvta_generic_to_global(p)));
  return v;
}

// mbar_wait for a role that waits much of its time: the hardware holds the
// warp back for up to 20 us a try, so that it does not take issue slots from
// the roles that it waits for.  Gives up after 1 s like every wait.
__device__ __forceinline__ bool role_wait(uint32_t bar, uint32_t parity) {
  uint64_t t0 = 0;
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000; "
        "selp.u32 %0, 1, 0, p; }"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    const uint64_t t = globaltimer();
    if (t0 == 0) t0 = t;
    if (t - t0 > kWaitLimitNs) {
      record_error(kErrWaitTimeout);
      return false;
    }
  }
}

template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(r));
  return r != 0;
}

// NT: tokens of a tile.  GS: log2 of the group size.  SETS: sets of four
// widening warps.  SW: scaling warps, four, or eight that
// split the tokens.
template <bool X8, int NT, int GS, int SETS, int SW>
struct W4Tc {
  static constexpr int kWide = 4 * SETS;                        // widening warps
  static constexpr int kTmaWarp = kWide + SW, kMmaWarp = kTmaWarp + 2;  // two of each
  static constexpr int kThreads = 32 * (kWide + SW + 4);
  static constexpr int kGroups = 128 >> GS;                     // groups of a block
  static constexpr int kACols = X8 ? 32 : 64;                   // TMEM columns of a widened block
  static constexpr int kTmem = 512;
  static constexpr int kDBufs = NT <= 64 ? 4 : 2;               // accumulators
  static constexpr int kAFit = (kTmem - kDBufs * NT) / kACols;
  // A buffer of a ring belongs to one set and one MMA warp for good: one that
  // waits on it has then seen all of its earlier phases, and cannot take the
  // parity of a phase two back for its own.  So the rings' lengths are
  // multiples of the sets' and the MMA warps' numbers.
  static constexpr int kRing = SETS % 2 ? 2 * SETS : SETS;
  static constexpr int kABufs = (kAFit < 8 ? kAFit : 8) / kRing * kRing;
  static constexpr int kWBytes = kW4M * 64;
  static constexpr int kXBytes = NT * (X8 ? 128 : 256);
  // Rings of packed weights and of x, apart: a widening set is done with the
  // weights long before the MMA is with x.
  static constexpr int kWStages = kXBytes > 16384 ? 4 : NT > 32 ? 8 : 12;
  static constexpr int kXFit = (224 * 1024 - kWStages * kWBytes) / kXBytes / 2 * 2;
  static constexpr int kXStages = kXFit < 12 ? kXFit : 12;
  static constexpr int kAllBars = 2 * (kWStages + kXStages + kABufs + kDBufs);
  static constexpr int kRings = kWStages * kWBytes + kXStages * kXBytes;
  static constexpr int kSmem = 1024 + kRings + 256 + 8 * kAllBars + 16;
  static constexpr int kCols = NT / (SW / 4);                   // tokens of a scaling warp
  static constexpr int kMmaArrive = kGroups > 1 ? 2 : 1;        // MMA warps that share a block
  // With 64 sums a thread, the scaling warps take registers over from the
  // others (setmaxnreg, by warpgroups): the three shares are at most what the
  // block is launched with, kRegs for each thread.
  static constexpr bool kSplit = kCols > 32;
  static constexpr int kRegs = 65536 / kThreads / 8 * 8;
  static constexpr int kRegsWide = 64, kRegsRest = 40, kRegsScale = 104;
  static_assert(!kSplit || kWide * kRegsWide + SW * kRegsScale + 4 * kRegsRest <=
                               (kWide + SW + 4) * kRegs,
                "more registers than the block has");
  static_assert(kWStages % kRing == 0 && kSmem <= 232448 && kRings >= NT * kW4M * 4, "rings");
  static_assert(kABufs >= kRing, "a widened block for each set");
};

// This CTA's share of a tile's outputs from the parts of its cluster's CTAs,
// [token][row] at `base` of each: four rows of a token a thread at a time, all
// ranks' loads before the first sum.
template <class E, bool X8, int NT, int THREADS>
__device__ __forceinline__ void w4_add_parts(const W4TcParams& P, int tile, int rank,
                                             uint32_t base, int tid) {
  const W4Args& p = P.a;
  const int tb = (tile / P.tiles_n) * NT, n0 = (tile % P.tiles_n) * kW4M;
  const int c0 = NT * rank / P.cs, c1 = NT * (rank + 1) / P.cs;
  for (int e = tid; e < (c1 - c0) * (kW4M / 4); e += THREADS) {
    const int c = c0 + e / (kW4M / 4), r = e % (kW4M / 4) * 4;
    const int t = tb + c;
    if (t >= p.tok) break;
    float4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < P.cs) v[i] = ld_dsmem_v4(mapa_shared(base + static_cast<uint32_t>(c * kW4M + r) * 4, i));
#pragma unroll
    for (int i = 1; i < 8; ++i)
      if (i < P.cs) {
        v[0].x += v[i].x; v[0].y += v[i].y; v[0].z += v[i].z; v[0].w += v[i].w;
      }
    const float f = X8 ? __ldg(p.x_scale + t) : 1.f;
    const float o[4] = {v[0].x * f, v[0].y * f, v[0].z * f, v[0].w * f};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n0 + r + i < p.N) stg16(p.out + t * p.ld_out + n0 + r + i, E::f32_to_bits(o[i]));
  }
}

template <class E, bool X8, int NT, int GS, int SETS, int SW>
__global__ void __launch_bounds__((W4Tc<X8, NT, GS, SETS, SW>::kThreads), 1)
w4_tc_kernel(const __grid_constant__ W4TcParams P) {
  using C = W4Tc<X8, NT, GS, SETS, SW>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const W4Args& p = P.a;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  // [weight stages][x stages], later the split sums, [code tables][barriers][TMEM address]
  constexpr uint32_t kX0 = C::kWStages * C::kWBytes;
  uint4* codes = reinterpret_cast<uint4*>(smem + C::kRings);
  uint64_t* bars = reinterpret_cast<uint64_t*>(codes + 16);
  const uint32_t wfull0 = smem_u32(bars);
  const uint32_t wempty0 = wfull0 + 8 * C::kWStages;
  const uint32_t xfull0 = wempty0 + 8 * C::kWStages;
  const uint32_t xempty0 = xfull0 + 8 * C::kXStages;
  const uint32_t afull0 = xempty0 + 8 * C::kXStages;
  const uint32_t aempty0 = afull0 + 8 * C::kABufs;
  const uint32_t dfull0 = aempty0 + 8 * C::kABufs;
  const uint32_t dempty0 = dfull0 + 8 * C::kDBufs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kAllBars);

  // the launch of the last tiles may take SMs as this one's blocks leave them
  griddep_launch_dependents();
  // a barrier a thread, in the order of their addresses
  if (tid < C::kAllBars) {
    int count = 1;  // a copy, or the MMAs of a group
    const uint32_t at = wfull0 + 8 * tid;
    if (at >= wempty0 && at < xfull0) count = 4;                    // a set of widening warps
    if (at >= xempty0 && at < afull0) count = C::kMmaArrive;
    if (at >= afull0 && at < aempty0) count = 4;
    if (at >= aempty0 && at < dfull0) count = C::kMmaArrive;
    if (at >= dempty0) count = SW;
    mbar_init(at, count);
    fence_mbar_init();
  }
  if (X8 && tid < 64) {
    // word tid % 4 of the table of zero point tid / 4
    uint32_t c = 0;
    for (int i = 0; i < 4; ++i) c |= w4_code8(4 * (tid & 3) + i, tid >> 2) << (8 * i);
    reinterpret_cast<uint32_t*>(codes)[tid] = c;
  }
  if (warp == C::kTmaWarp) {
    if (lane == 0) {
      tma_prefetch_desc(&P.tmap_w);
      tma_prefetch_desc(&P.tmap_x);
    }
  } else if (warp == C::kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), C::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const uint32_t abase = tmem + C::kDBufs * NT;
  const int rank = P.cs > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int kb0 = P.cs > 1 ? P.nkb * rank / P.cs : 0;
  const int kb1 = P.cs > 1 ? P.nkb * (rank + 1) / P.cs : P.nkb;
  const int tiles = P.tile1;
  const int first = P.tile0 + blockIdx.x / P.cs, step = gridDim.x / P.cs;
  bool ok = true;

  if (warp < C::kWide) {
    // =========================== widening: a lane of TMEM, and a row, a thread
    if constexpr (C::kSplit) regs_dec<C::kRegsWide>();
    const int quad = warp & 3, set = warp >> 2;
    const int row = quad * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t rsw = (row >> 1) & 3;
    // this set's blocks, every SETS-th of the CTA's, counted over its tiles
    RingPos st, ab;
    for (int i = 0; i < set; ++i) {
      st.next(C::kWStages);
      ab.next(C::kABufs);
    }
    int skip = set;  // blocks of the next tile before this set's first
    for (int tile = first; tile < tiles && ok; tile += step) {
      const int n = (tile % P.tiles_n) * kW4M + row;
      const uint8_t* z_row = p.z + min(n, p.N - 1);
      const int last_g = (p.K - 1) >> GS;
      // The zero points of this set's next kAhead blocks, loaded while it
      // works on the last kAhead, and used as loaded: arithmetic on a value
      // that is on its way, even moving it, would wait for it.
      constexpr int kAhead = 2;
      uint32_t zq[kAhead][C::kGroups], zn[kAhead][C::kGroups];
      auto zeros = [&](int kb, uint32_t (&v)[kAhead][C::kGroups]) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
          for (int i = 0; i < C::kGroups; ++i)
            v[u][i] = p.z ? ld_early(z_row + min((kb + u * SETS) * C::kGroups + i, last_g) * p.ld_s)
                          : 8u;
      };
      int kb = kb0 + skip;
      zeros(kb, zn);
      while (kb < kb1 && ok) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
          for (int i = 0; i < C::kGroups; ++i) zq[u][i] = zn[u][i];
        zeros(kb + kAhead * SETS, zn);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          if (kb >= kb1 || !ok) break;
          ok = role_wait(wfull0 + 8 * st.i, st.fill());
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const uint8_t* src = smem + st.i * C::kWBytes + row * 64;
          uint4 pk[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) pk[c] = *reinterpret_cast<const uint4*>(src + ((c ^ rsw) << 4));
          __syncwarp();
          if (lane == 0) mbar_arrive(wempty0 + 8 * st.i);
          ok = role_wait(aempty0 + 8 * ab.i, ab.drain());
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          const uint32_t dst = abase + lane_off + ab.i * C::kACols;
          if constexpr (X8) {
#pragma unroll
            for (int c = 0; c < 4; c += 2) {
              uint32_t r[16];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t w[4] = {pk[c + h].x, pk[c + h].y, pk[c + h].z, pk[c + h].w};
                const uint4 T = codes[zq[u][((c + h) * 32) >> GS] & 15];
#pragma unroll
                for (int j = 0; j < 4; ++j) w4_bytes8(w[j], T, r[8 * h + 2 * j], r[8 * h + 2 * j + 1]);
              }
              tmem_st16(dst + c * 8, r);
            }
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t w[4] = {pk[c].x, pk[c].y, pk[c].z, pk[c].w};
              const uint32_t zz = W4Magic<E>::zero(zq[u][(c * 32) >> GS] & 15);
              uint32_t r[16];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                uint32_t q[4];
                w4_pairs<E>(w[j], zz, q);
                r[4 * j] = q[0]; r[4 * j + 1] = q[1]; r[4 * j + 2] = q[2]; r[4 * j + 3] = q[3];
              }
              tmem_st16(dst + c * 16, r);
            }
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(afull0 + 8 * ab.i);
          }
#pragma unroll
          for (int i = 0; i < SETS; ++i) {
            st.next(C::kWStages);
            ab.next(C::kABufs);
          }
          kb += SETS;
        }
      }
      skip = kb - kb1;
    }
    // One tile: the parts of the cluster's CTAs are added in rank order, a share
    // of the tokens by each CTA, by these warps and the scaling ones (in their
    // own branch: what all roles share would have the fewest registers of all).
    // A CTA whose waits gave up has recorded it.
    if (P.cs > 1) {
      cluster_sync();
      if (ok) w4_add_parts<E, X8, NT, 32 * C::kTmaWarp>(P, first, rank, sbase, tid);
      cluster_sync_relaxed();
    }
  } else if (warp < C::kTmaWarp) {
    // =========================== scaling: sum += scale * accumulator, then the output
    if constexpr (C::kSplit) regs_inc<C::kRegsScale>();
    const int w = warp - C::kWide, quad = w & 3;
    const int row = quad * 32 + lane;
    const int col0 = (w >> 2) * C::kCols;
    const uint32_t dsrc = tmem + (static_cast<uint32_t>(quad * 32) << 16) + col0;
    RingPos db;
    for (int tile = first; tile < tiles; tile += step) {
      const int n = (tile % P.tiles_n) * kW4M + row;
      const int tb = (tile / P.tiles_n) * NT;
      const int g0 = kb0 * C::kGroups, g1 = kb1 * C::kGroups;
      // The scales of the next four groups, loaded while these four are added
      // (behind the last group, that one's: a selection would wait for the load).
      const int last_g = (p.K - 1) >> GS;
      const uint16_t* s_row = p.s + min(n, p.N - 1);
      uint32_t sq[4], sn[4];
      auto scales = [&](int g) {
#pragma unroll
        for (int u = 0; u < 4; ++u) sn[u] = ld_early(s_row + min(g + u, last_g) * p.ld_s);
      };
      scales(g0);
      uint64_t acc[C::kCols / 2];  // pairs of sums
#pragma unroll
      for (int c = 0; c < C::kCols / 2; ++c) acc[c] = 0;
      for (int g = g0; g < g1 && ok; g += 4) {
#pragma unroll
        for (int u = 0; u < 4; ++u) sq[u] = sn[u];
        scales(g + 4);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (g + u >= g1 || !ok) break;
          ok = role_wait(dfull0 + 8 * db.i, db.fill());
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          // a group behind K has sums of 0, whatever the last scale is
          const float s1 = g + u <= last_g ? E::bits_to_f32(static_cast<uint16_t>(sq[u])) : 0.f;
          const float sc = X8 ? s1 * 64.f : s1;
          tc_fence_after();
          // some columns at a time, and the accumulator is free before the
          // last ones' arithmetic
          constexpr int kLoad = C::kCols == 32 ? 32 : 16;
          const uint64_t sc2 = pack2(sc, sc);
#pragma unroll
          for (int c0 = 0; c0 < C::kCols; c0 += kLoad) {
            float v[kLoad / 16][16];
#pragma unroll
            for (int c = 0; c < kLoad; c += 16) tmem_ld16(dsrc + db.i * NT + c0 + c, v[c / 16]);
            tmem_ld_wait();
            if (c0 + kLoad == C::kCols) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(dempty0 + 8 * db.i);
            }
#pragma unroll
            for (int c = 0; c < kLoad; c += 2)
              fma2(acc[(c0 + c) / 2], pack2(v[c / 16][c % 16], v[c / 16][c % 16 + 1]), sc2);
          }
          db.next(C::kDBufs);
        }
      }
      if (!ok) break;
      if (P.cs == 1) {
        if (n < p.N) {
#pragma unroll
          for (int c = 0; c < C::kCols; ++c) {
            const int t = tb + col0 + c;
            if (t < p.tok) {
              const float2 f = unpack2(acc[c / 2]);
              const float a = c & 1 ? f.y : f.x;
              const float v = X8 ? a * __ldg(p.x_scale + t) : a;
              stg16(p.out + t * p.ld_out + n, E::f32_to_bits(v));
            }
          }
        }
      } else {
        // this CTA's part: [token][row] over the ring, whose copies and MMAs
        // are all done
        float* part = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int c = 0; c < C::kCols; c += 2) {
          const float2 f = unpack2(acc[c / 2]);
          part[(col0 + c) * kW4M + row] = f.x;
          part[(col0 + c + 1) * kW4M + row] = f.y;
        }
      }
    }
    if (P.cs > 1) {
      cluster_sync();
      if (ok) w4_add_parts<E, X8, NT, 32 * C::kTmaWarp>(P, first, rank, sbase, tid);
      cluster_sync_relaxed();
    }
  } else {
    // one instruction for the whole warpgroup, as it has to be
    if constexpr (C::kSplit) regs_dec<C::kRegsRest>();
    if (warp < C::kMmaWarp) {
      // =========================== TMA: a warp for the weights, one for x
      const bool wt = warp == C::kTmaWarp;
      const int stages = wt ? C::kWStages : C::kXStages;
      const uint32_t full0 = wt ? wfull0 : xfull0, empty0 = wt ? wempty0 : xempty0;
      RingPos st;
      int issued = 0;
      for (int tile = first; tile < tiles && ok; tile += step) {
        const int n0 = (tile % P.tiles_n) * kW4M, tb = (tile / P.tiles_n) * NT;
        for (int kb = kb0; kb < kb1; ++kb) {
          ok = role_wait(empty0 + 8 * st.i, st.drain());
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const uint32_t bar = full0 + 8 * st.i;
          if (elect_one()) {
            if (wt) {
              mbar_arrive_expect_tx(bar, C::kWBytes);
              tma_load_2d(sbase + st.i * C::kWBytes, &P.tmap_w, bar, kb * 64, n0);
            } else {
              const uint32_t dst = sbase + kX0 + st.i * C::kXBytes;
              mbar_arrive_expect_tx(bar, C::kXBytes);
              tma_load_2d(dst, &P.tmap_x, bar, kb * kW4K, tb);
              if (!X8) tma_load_2d(dst + NT * 128, &P.tmap_x, bar, kb * kW4K + 64, tb);
            }
          }
          __syncwarp();
          st.next(stages);
          ++issued;
        }
      }
      // after a wait that gave up: the copies still in flight
      if (!ok)
        for (int i = max(0, issued - stages); i < issued; ++i)
          role_wait(full0 + 8 * (i % stages), (i / stages) & 1);
    } else {
      // =========================== MMA: group i of the CTA is warp i % 2's
      const int mw = warp - C::kMmaWarp;
      constexpr int kSteps = X8 ? 4 : 8;           // MMAs of a block
      constexpr int kPer = kSteps / C::kGroups;    // MMAs of a group
      const uint64_t bd0 = make_sdesc(sbase + kX0, 128, 2);
      const uint32_t idesc = P.idesc;
      RingPos st, ab, db;
      uint32_t blk = 0;
      for (int tile = first; tile < tiles && ok; tile += step) {
        for (int kb = kb0; kb < kb1 && ok; ++kb, ++blk) {
          if (C::kGroups > 1 || (blk & 1) == static_cast<uint32_t>(mw)) {
            ok = role_wait(xfull0 + 8 * st.i, st.fill()) && role_wait(afull0 + 8 * ab.i, ab.fill());
            // addresses in a descriptor are in units of 16 bytes
            const uint64_t bd = bd0 + static_cast<uint32_t>(st.i * (C::kXBytes / 16));
            const uint32_t at = abase + ab.i * C::kACols;
#pragma unroll
            for (int j = 0; j < C::kGroups; ++j) {
              if (C::kGroups == 1 || (j & 1) == mw) {
                ok = ok && role_wait(dempty0 + 8 * db.i, db.drain());
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                  for (int i = 0; i < kPer; ++i) {
                    const int kk = j * kPer + i;
                    tc_mma_ts<X8>(tmem + db.i * NT, at + kk * 8,
                                  bd + (kk / 4) * (NT * 8) + (kk % 4) * 2, idesc, i > 0 ? 1u : 0u);
                  }
                  if (j + C::kMmaArrive >= C::kGroups) {  // this warp's last group of the block
                    tc_commit(aempty0 + 8 * ab.i);
                    tc_commit(xempty0 + 8 * st.i);
                  }
                  tc_commit(dfull0 + 8 * db.i);
                }
                __syncwarp();
              }
              db.next(C::kDBufs);
            }
          } else {
            db.next(C::kDBufs);
          }
          st.next(C::kXStages);
          ab.next(C::kABufs);
        }
      }
    }
  }
  __syncwarp();

  if (P.cs > 1 && warp >= C::kTmaWarp) {  // the others' barriers
    cluster_sync();
    cluster_sync_relaxed();
  }
  __syncthreads();
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
  // a launch that began early ends after the one before it
  griddep_wait();
}

}  // namespace lora
