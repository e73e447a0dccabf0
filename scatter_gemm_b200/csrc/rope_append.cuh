// rope_append.cuh -- the rotation of the projection's q and k slices and the
// append of k and v to a paged cache, in one pass over the q/k/v row.
//
// For token t, frequency i < R/2 and p = positions[axis(i)][t], the pair (a, b)
// of a head -- elements (i, i + R/2), or (2i, 2i+1) when interleaved -- becomes
//   a' = a cos[p, i] - b sin[p, i],   b' = b cos[p, i] + a sin[p, i]
// in fp32; elements behind the first R pass through.  With head weights each
// head of q and k is first normalised: x * rsqrt(mean x^2 + eps) * (w + w0).
// q goes to q_out; k' and v, divided by their cache's scale for an 8-bit cache,
// go to slot slots[t] of the caches.  Every value is rounded once, when stored.
//
// The bound is the memory traffic: each q/k/v row read once, q and the cache
// entries written once, and the token's R table entries.
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

// Any head size, stride and alignment: one warp a head, one pair a lane.
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

}  // namespace lora
