// rope_append.cuh -- the rotation of the projection's q and k slices and the
// append of k and v to a paged cache, in one pass over the q/k/v row.
//
// For token t, frequency i < R/2 and p = positions[axis(i)][t], the pair (a, b)
// of a head -- elements (i, i + R/2), or (2i, 2i+1) when interleaved -- becomes
//   a' = a cos[p, i] - b sin[p, i],   b' = b cos[p, i] + a sin[p, i]
// in fp32; elements behind the first R pass through.  With head weights each
// head of q and k is first normalised: x * rsqrt(mean x^2 + eps) * (w + w0).
// q goes to q_out; k' and v, times the fp32 reciprocal of their cache's scale,
// go to slot slots[t] of the caches.  Every value is rounded once, when stored.
//
// The bound is the memory traffic: each q/k/v row read once, q and the cache
// entries written once, and the token's R table entries.  8192 tokens of 40 + 8
// + 8 heads of 128 with three axes: 46 us, 5.2 TB/s (186 us by the general
// kernel); one token: 2 us.
#pragma once

#include "common.cuh"
#include "rmsnorm.cuh"

namespace lora {

constexpr int kRopeMaxAxes = 4;
constexpr int kRopeMaxDim = 512;

struct RopeAppendArgs {
  const uint16_t* qkv;
  int64_t ld_qkv;
  int off_q, off_k, off_v;  // column offsets of the slices
  int hq, hkv, D, R;
  const void* positions;    // [axes, ld_pos], int32 or int64
  int64_t ld_pos;
  int axes;
  const float* cos_sin;     // [max_pos, R]: R/2 cosines, then R/2 sines
  int64_t max_pos;
  uint16_t* q_out;
  int64_t ld_q;
  void* kc;
  void* vc;
  int64_t k_page, k_slot, k_head, v_page, v_slot, v_head;  // strides in elements
  int64_t pages;
  int page_size;
  const void* slots;        // [tok], int32 or int64
  const uint16_t* qw;       // head weights, both null or both given
  const uint16_t* kw;
  float eps, w0, k_inv, v_inv;
  int tok, interleaved, idx64;
  uint16_t axis_of[kRopeMaxDim / 16];  // two bits for each frequency, eight frequencies a word
};

__device__ __forceinline__ int64_t rope_index(const void* p, int64_t i, int idx64) {
  return idx64 ? __ldg(static_cast<const long long*>(p) + i)
               : static_cast<int64_t>(__ldg(static_cast<const int*>(p) + i));
}

__device__ __forceinline__ int64_t rope_position(const RopeAppendArgs& p, int axis, int t) {
  const int64_t v = rope_index(p.positions, axis * p.ld_pos + t, p.idx64);
  return v < 0 ? 0 : (v >= p.max_pos ? p.max_pos - 1 : v);
}

// Any head size, stride and alignment: one warp a head, one pair a lane.  Runs
// where rope_append_kernel cannot: see its conditions.  A table entry of four
// bytes and a store of two for each element: 216 us for 8192 tokens of 40 + 8 + 8
// heads of 100, 0.9 TB/s.
template <class E, bool C8>
__global__ void __launch_bounds__(256) rope_append_general_kernel(const RopeAppendArgs p) {
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int heads = p.hq + 2 * p.hkv;
  const int64_t ti = item / heads;
  if (ti >= p.tok) return;
  const int t = static_cast<int>(ti), hd = static_cast<int>(item % heads);
  const int kind = hd < p.hq ? 0 : (hd < p.hq + p.hkv ? 1 : 2);
  const int h = kind == 0 ? hd : (kind == 1 ? hd - p.hq : hd - p.hq - p.hkv);
  const uint16_t* src = p.qkv + t * p.ld_qkv + (kind == 0 ? p.off_q : kind == 1 ? p.off_k : p.off_v) +
                        static_cast<int64_t>(h) * p.D;
  uint16_t* dst16 = nullptr;
  uint8_t* dst8 = nullptr;
  if (kind == 0) {
    dst16 = p.q_out + t * p.ld_q + static_cast<int64_t>(h) * p.D;
  } else {
    const int64_t slot = rope_index(p.slots, t, p.idx64);
    if (slot < 0 || slot >= p.pages * p.page_size) return;
    const int64_t pg = slot / p.page_size, in = slot % p.page_size;
    const int64_t at = kind == 1 ? pg * p.k_page + in * p.k_slot + h * p.k_head
                                 : pg * p.v_page + in * p.v_slot + h * p.v_head;
    void* c = kind == 1 ? p.kc : p.vc;
    if (C8) dst8 = static_cast<uint8_t*>(c) + at;
    else dst16 = static_cast<uint16_t*>(c) + at;
  }
  const float inv = kind == 1 ? p.k_inv : p.v_inv;
  auto put = [&](int e, float v) {
    if (C8 && kind) dst8[e] = static_cast<uint8_t>(f4_to_e4m3(v * inv, 0.f, 0.f, 0.f));
    else stg16(dst16 + e, E::f32_to_bits(kind ? v * inv : v));
  };
  const uint16_t* w = kind == 0 ? p.qw : kind == 1 ? p.kw : nullptr;
  float rstd = 1.f;
  if (w) {
    float s = 0.f;
    for (int e = lane; e < p.D; e += 32) {
      const float f = E::bits_to_f32(src[e]);
      s = fmaf(f, f, s);
    }
    rstd = rsqrtf(warp_sum(s) / static_cast<float>(p.D) + p.eps);
  }
  auto get = [&](int e) {
    const float f = E::bits_to_f32(src[e]);
    return w ? f * rstd * (E::bits_to_f32(__ldg(w + e)) + p.w0) : f;
  };
  const int half = kind == 2 ? 0 : p.R / 2;
  for (int i = lane; i < half; i += 32) {
    const int axis = (p.axis_of[i >> 3] >> (2 * (i & 7))) & 3;
    const float* cs = p.cos_sin + rope_position(p, axis, t) * p.R + i;
    const float c = __ldg(cs), s = __ldg(cs + half);
    const int ea = p.interleaved ? 2 * i : i, eb = p.interleaved ? 2 * i + 1 : i + half;
    const float a = get(ea), b = get(eb);
    put(ea, a * c - b * s);
    put(eb, b * c + a * s);
  }
  for (int e = 2 * half + lane; e < p.D; e += 32) put(e, get(e));
}

// Eight elements as floats, and back.
template <class E>
__device__ __forceinline__ void rope_unpack(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = E::u32_to_f2(w[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}

template <class E>
__device__ __forceinline__ uint4 rope_pack(const float (&f)[8]) {
  return make_uint4(E::f2_to_u32(f[0], f[1]), E::f2_to_u32(f[2], f[3]), E::f2_to_u32(f[4], f[5]),
                    E::f2_to_u32(f[6], f[7]));
}

// Heads of whole 16-byte pieces: 16-byte aligned rows, heads and cache entries
// (8-byte with an 8-bit cache), head_dim a multiple of 16 and, unless
// interleaved, R too.
//
// A group of LG lanes (a power of two, at least head_dim / 16) takes a head:
// each lane eight neighbouring frequencies, that is two 16-byte pieces of the
// head, R/2 apart, or next to each other when interleaved or behind the
// rotated part; so a pair never leaves its lane and a head's norm is a few
// shuffles.  A warp takes 32 / LG heads of one token at a time, `steps` times,
// DEPTH steps' loads under way: with many tokens that reads the token's
// cosines, sines and slot once for all of its heads.  Two steps ahead at 64
// registers (46 us) beat three and four at 80 (54, 57 us): the warps that fit
// hide more than the loads that a warp has under way.  At two steps ahead 48 to
// 56 bytes a thread are spilled (16 in some), with head norms 8 to 68 at their
// 80 registers: 8192 tokens of 40 + 8 + 8 heads of 128, one axis and an 8-bit
// cache take 40 us, with head norms 51.
//
// A block is eight tokens and the same heads of each, so that which slice a
// head belongs to, and where, is the same arithmetic for all of its threads.
template <class E, bool C8, bool INTER, bool NORM, int LG, int DEPTH>
__global__ void __launch_bounds__(256, DEPTH == 1 ? 1 : NORM ? 3 : 4)
rope_append_kernel(const RopeAppendArgs p, const int parts, const int steps) {
  constexpr int kPer = 32 / LG;  // heads of a step
  const int lane = threadIdx.x & 31;
  const uint32_t tb = blockIdx.x / static_cast<uint32_t>(parts);
  const int first = static_cast<int>(blockIdx.x - tb * parts) * (DEPTH > 1 ? steps : 1) * kPer;
  const int t = static_cast<int>(tb * 8u + (threadIdx.x >> 5));
  if (t >= p.tok) return;
  const int end = min(p.hq + 2 * p.hkv, first + (DEPTH > 1 ? steps : 1) * kPer);
  const int j = lane % LG, sub = lane / LG;
  const bool in = j < p.D / 16;
  const int half = p.R / 2;
  const bool rot = 8 * j < half;
  // the lane's two pieces
  const int ea = INTER || !rot ? 16 * j : 8 * j;
  const int eb = INTER || !rot ? 16 * j + 8 : 8 * j + half;

  // head hd starts at column hd * D + (its slice's start less the heads before it)
  const int base_q = p.off_q, base_k = p.off_k - p.hq * p.D,
            base_v = p.off_v - (p.hq + p.hkv) * p.D;
  const uint16_t* row = p.qkv + t * p.ld_qkv;
  uint4 a[DEPTH], b[DEPTH];
  auto load = [&](int hd, uint4& x, uint4& y) {
    if (in && hd < end) {
      const uint16_t* src =
          row + (hd * p.D + (hd < p.hq ? base_q : hd < p.hq + p.hkv ? base_k : base_v));
      x = *reinterpret_cast<const uint4*>(src + ea);
      y = *reinterpret_cast<const uint4*>(src + eb);
    }
  };
#pragma unroll
  for (int s = 0; s < DEPTH; ++s) {
    a[s] = b[s] = make_uint4(0, 0, 0, 0);
    load(first + s * kPer + sub, a[s], b[s]);
  }

  // cosines and sines of frequencies 8j .. 8j+7, unless the block has v only
  float cs[8], sn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) cs[i] = 1.f, sn[i] = 0.f;
  if (first < p.hq + p.hkv) {
    if (p.axes == 1 && half % 8 == 0 && (reinterpret_cast<uintptr_t>(p.cos_sin) & 15) == 0) {
      if (rot) {
        const float* c = p.cos_sin + rope_position(p, 0, t) * p.R + 8 * j;
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          const float4 u = __ldg(reinterpret_cast<const float4*>(c + i));
          const float4 v = __ldg(reinterpret_cast<const float4*>(c + half + i));
          cs[i] = u.x; cs[i + 1] = u.y; cs[i + 2] = u.z; cs[i + 3] = u.w;
          sn[i] = v.x; sn[i + 1] = v.y; sn[i + 2] = v.z; sn[i + 3] = v.w;
        }
      }
    } else {
      // several axes, or a table or an end off the 16-byte grid: the warp
      // gathers the token's row first, a frequency a lane, zeros behind it
      __shared__ __align__(16) float rows[8][2][kRopeMaxDim / 2 + 8];
      float(&tab)[2][kRopeMaxDim / 2 + 8] = rows[threadIdx.x >> 5];
      for (int i = lane; i < (half + 7) / 8 * 8; i += 32) {
        float u = 0.f, v = 0.f;
        if (i < half) {
          const int axis = (p.axis_of[i >> 3] >> (2 * (i & 7))) & 3;
          const float* c = p.cos_sin + rope_position(p, axis, t) * p.R + i;
          u = __ldg(c);
          v = __ldg(c + half);
        }
        tab[0][i] = u;
        tab[1][i] = v;
      }
      __syncwarp();
      if (rot) {
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          const float4 u = *reinterpret_cast<const float4*>(&tab[0][8 * j + i]);
          const float4 v = *reinterpret_cast<const float4*>(&tab[1][8 * j + i]);
          cs[i] = u.x; cs[i + 1] = u.y; cs[i + 2] = u.z; cs[i + 3] = u.w;
          sn[i] = v.x; sn[i + 1] = v.y; sn[i + 2] = v.z; sn[i + 3] = v.w;
        }
      }
    }
  }

  // the token's cache entry, less the heads before the slice
  int64_t k_at = 0, v_at = 0;
  bool entry = false;
  if (end > p.hq) {
    const int64_t slot = rope_index(p.slots, t, p.idx64);
    entry = slot >= 0 && slot < p.pages * p.page_size;
    if (entry) {
      int64_t pg, at;
      if (slot <= 0x7FFFFFFF) {
        pg = static_cast<uint32_t>(slot) / static_cast<uint32_t>(p.page_size);
        at = static_cast<uint32_t>(slot) % static_cast<uint32_t>(p.page_size);
      } else {
        pg = slot / p.page_size;
        at = slot % p.page_size;
      }
      k_at = pg * p.k_page + at * p.k_slot - p.hq * p.k_head;
      v_at = pg * p.v_page + at * p.v_slot - (p.hq + p.hkv) * p.v_head;
    }
  }

  uint16_t* q_row = p.q_out + t * p.ld_q;
  for (int s0 = 0; s0 < (DEPTH > 1 ? steps : 1); s0 += DEPTH) {
#pragma unroll
    for (int s = 0; s < DEPTH; ++s) {
      if (first + (s0 + s) * kPer >= end) break;
      const int hd = first + (s0 + s) * kPer + sub;
      const bool is_q = hd < p.hq, is_k = !is_q && hd < p.hq + p.hkv, is_v = hd >= p.hq + p.hkv;
      const float inv = is_q ? 1.f : is_k ? p.k_inv : p.v_inv;
      uint4 oa = a[s], ob = b[s];
      if (DEPTH > 1) load(hd + DEPTH * kPer, a[s], b[s]);
      // v, and pieces behind the rotated part, pass through as they are
      float fa[8], fb[8];
      rope_unpack<E>(oa, fa);
      rope_unpack<E>(ob, fb);
      if (NORM) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(fa[i], fa[i], fmaf(fb[i], fb[i], sum));
#pragma unroll
        for (int d = LG / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (!is_v && in) {
          const float rstd = rsqrtf(sum / static_cast<float>(p.D) + p.eps);
          const uint16_t* w = is_q ? p.qw : p.kw;
          float wa[8], wb[8];
          rope_unpack<E>(__ldg(reinterpret_cast<const uint4*>(w + ea)), wa);
          rope_unpack<E>(__ldg(reinterpret_cast<const uint4*>(w + eb)), wb);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            fa[i] *= rstd * (wa[i] + p.w0);
            fb[i] *= rstd * (wb[i] + p.w0);
          }
        }
      }
      if (!in || hd >= end || (!is_q && !entry)) continue;
      if (!is_v && rot) {
        if (INTER) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // the lane's frequencies may end within its pieces
            const float x = fa[2 * i], y = fa[2 * i + 1], u = fb[2 * i], v = fb[2 * i + 1];
            if (8 * j + i < half) {
              fa[2 * i] = x * cs[i] - y * sn[i];
              fa[2 * i + 1] = y * cs[i] + x * sn[i];
            }
            if (8 * j + 4 + i < half) {
              fb[2 * i] = u * cs[4 + i] - v * sn[4 + i];
              fb[2 * i + 1] = v * cs[4 + i] + u * sn[4 + i];
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float x = fa[i], y = fb[i];
            fa[i] = x * cs[i] - y * sn[i];
            fb[i] = y * cs[i] + x * sn[i];
          }
        }
      }
      if (C8 && !is_q) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          fa[i] *= inv;
          fb[i] *= inv;
        }
        uint8_t* o = static_cast<uint8_t*>(is_k ? p.kc : p.vc) +
                     (is_k ? k_at + hd * p.k_head : v_at + hd * p.v_head);
        stg64(o + ea, make_uint2(f4_to_e4m3(fa[0], fa[1], fa[2], fa[3]),
                                 f4_to_e4m3(fa[4], fa[5], fa[6], fa[7])));
        stg64(o + eb, make_uint2(f4_to_e4m3(fb[0], fb[1], fb[2], fb[3]),
                                 f4_to_e4m3(fb[4], fb[5], fb[6], fb[7])));
        continue;
      }
      if (inv != 1.f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          fa[i] *= inv;
          fb[i] *= inv;
        }
      }
      if (!is_v || inv != 1.f) {
        oa = rope_pack<E>(fa);
        ob = rope_pack<E>(fb);
      }
      uint16_t* o = is_q ? q_row + hd * p.D
                         : static_cast<uint16_t*>(is_k ? p.kc : p.vc) +
                               (is_k ? k_at + hd * p.k_head : v_at + hd * p.v_head);
      stg128(o + ea, oa);
      stg128(o + eb, ob);
    }
  }
}

}  // namespace lora
