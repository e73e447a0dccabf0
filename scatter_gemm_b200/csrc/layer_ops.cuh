// layer_ops.cuh -- C ABI of the operators around the adapted projection:
// argument checks, variant selection and launches.  Included once, by
// lora_sgmv.cu, whose helpers and counters it uses.
#pragma once

#include "rmsnorm.cuh"
#include "rope_append.cuh"
#include "w4.cuh"
#include "w4_tc.cuh"

#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <type_traits>

namespace {

// Lets a kernel take up to `bytes` of dynamic shared memory, once for each
// device (`ready` holds a bit for each).
// A kernel whose warps pass registers among themselves must have been compiled
// to at least `regs` registers a thread, or a warp could wait for more than
// the block has.
bool set_smem_once(std::atomic<uint64_t>& ready, const void* kernel, int bytes, int regs = 0) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
  const uint64_t bit = uint64_t(1) << dev;
  if (ready.load(std::memory_order_acquire) & bit) return true;
  cudaFuncAttributes attr;
  if (regs && (cudaFuncGetAttributes(&attr, kernel) != cudaSuccess || attr.numRegs < regs))
    return false;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
      cudaSuccess)
    return false;
  ready.fetch_or(bit, std::memory_order_release);
  return true;
}

}  // namespace

// ------------------------------------------------------------------ RMS norm

namespace {

template <class E, int VPT, bool AL>
void launch_rmsnorm(const lora::RmsNormArgs& a, int T, cudaStream_t st) {
  const int rows = std::max(1, 256 / T);
  const unsigned grid = static_cast<unsigned>((a.tok + rows - 1) / rows);
  if (a.q)
    lora::rmsnorm_kernel<E, VPT, AL, true><<<grid, dim3(T, rows), 0, st>>>(a);
  else
    lora::rmsnorm_kernel<E, VPT, AL, false><<<grid, dim3(T, rows), 0, st>>>(a);
}

template <class E, bool AL>
lora_status rmsnorm(lora::RmsNormArgs a, int sms, cudaStream_t st) {
  // a row cut at x's 16-byte boundaries may take one block more than its
  // length; the widest rows have no thread for it and are cut at their start
  a.follow = (a.H + 14) / 8 <= 8 * 1024;
  const int blocks = AL ? a.H / 8 : (a.H + (a.follow ? 14 : 7)) / 8;
  // Blocks of eight a thread.  Where the rows fill the SMs several times over,
  // up to 256 threads a row: a row's two or three barriers then cost the least
  // (8192 x 5120: 60 us with up to 256, 65 with 512, 80 with 1024 threads a
  // row); below that more threads, for the latency of each (777 x 3583: 8.5 us
  // with 512 against 9.4 with 256).
  const int most = a.tok >= sms * 8 ? 256 : a.tok >= sms ? 512 : 1024;
  int vpt = 1;
  while (vpt < 8 && (blocks + vpt - 1) / vpt > most) vpt *= 2;
  const int T = round_up((blocks + vpt - 1) / vpt, 32);
  switch (vpt) {
    case 1: launch_rmsnorm<E, 1, AL>(a, T, st); break;
    case 2: launch_rmsnorm<E, 2, AL>(a, T, st); break;
    case 4: launch_rmsnorm<E, 4, AL>(a, T, st); break;
    default: launch_rmsnorm<E, 8, AL>(a, T, st); break;
  }
  ++g_launches;
  g_last_path = LORA_PATH_GENERAL;
  return launch_status();
}

}  // namespace

extern "C" lora_status lora_rmsnorm(const void* x, int64_t ld_x, const void* residual,
                                    int64_t ld_res, void* residual_out, int64_t ld_res_out,
                                    const void* weight, float weight_offset, float eps, void* out,
                                    int64_t ld_out, void* out_q, int64_t ld_q, float* out_scale,
                                    int tok, int H, lora_dtype dtype, void* stream) {
  if (dtype != LORA_BF16 && dtype != LORA_FP16) return LORA_ERR_UNSUPPORTED;
  if (tok < 0 || H < 1 || ld_x < H || !(eps >= 0.f)) return LORA_ERR_INVALID_ARGUMENT;
  if (!out && !out_q) return LORA_ERR_INVALID_ARGUMENT;
  if ((residual != nullptr) != (residual_out != nullptr) ||
      (out_q != nullptr) != (out_scale != nullptr))
    return LORA_ERR_INVALID_ARGUMENT;
  if ((residual && (ld_res < H || ld_res_out < H)) || (out && ld_out < H) || (out_q && ld_q < H))
    return LORA_ERR_INVALID_ARGUMENT;
  if (H > LORA_MAX_NORM_WIDTH || tok >= (1 << 30)) return LORA_ERR_UNSUPPORTED;
  if (tok == 0) return LORA_OK;
  if (!x || !weight) return LORA_ERR_INVALID_ARGUMENT;
  if (!aligned_to(x, 2) || !aligned_to(weight, 2) || !aligned_to(residual, 2) ||
      !aligned_to(residual_out, 2) || !aligned_to(out, 2) || !aligned_to(out_scale, 4))
    return LORA_ERR_INVALID_ARGUMENT;
  const lora::RmsNormArgs a{static_cast<const uint16_t*>(x), ld_x,
                            static_cast<const uint16_t*>(residual), ld_res,
                            static_cast<uint16_t*>(residual_out), ld_res_out,
                            static_cast<const uint16_t*>(weight), static_cast<uint16_t*>(out),
                            ld_out, static_cast<uint8_t*>(out_q), ld_q, out_scale, tok, H, eps,
                            weight_offset, 0};
  // (the stride of an only row says nothing)
  auto rows16 = [tok](const void* p, int64_t ld) {
    return !p || (aligned_to(p, 16) && (tok == 1 || ld % 8 == 0));
  };
  const bool al = H % 8 == 0 && rows16(x, ld_x) && rows16(residual, ld_res) &&
                  rows16(residual_out, ld_res_out) && rows16(weight, 0) && rows16(out, ld_out) &&
                  (!out_q || (aligned_to(out_q, 8) && (tok == 1 || ld_q % 8 == 0)));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const DeviceFacts* dev = device_facts();
  if (!dev) return LORA_ERR_CUDA;
  if (dtype == LORA_BF16)
    return al ? rmsnorm<lora::Bf16, true>(a, dev->sms, st) : rmsnorm<lora::Bf16, false>(a, dev->sms, st);
  return al ? rmsnorm<lora::Fp16, true>(a, dev->sms, st) : rmsnorm<lora::Fp16, false>(a, dev->sms, st);
}

// ------------------------------------------------------------------ rotate and append

namespace {

template <class E, bool C8, bool INTER, bool NORM, int DEPTH>
void launch_rope(const lora::RopeAppendArgs& a, int lg, unsigned grid, int parts,
                 int steps, cudaStream_t st) {
  if (lg == 4)
    lora::rope_append_kernel<E, C8, INTER, NORM, 4, DEPTH><<<grid, 256, 0, st>>>(a, parts, steps);
  else if (lg == 8)
    lora::rope_append_kernel<E, C8, INTER, NORM, 8, DEPTH><<<grid, 256, 0, st>>>(a, parts, steps);
  else if (lg == 16)
    lora::rope_append_kernel<E, C8, INTER, NORM, 16, DEPTH><<<grid, 256, 0, st>>>(a, parts, steps);
  else
    lora::rope_append_kernel<E, C8, INTER, NORM, 32, DEPTH><<<grid, 256, 0, st>>>(a, parts, steps);
}

template <class E, bool C8, bool INTER, bool NORM>
lora_status rope_pieces(const lora::RopeAppendArgs& a, int sms, cudaStream_t st) {
  int lg = 4;
  while (lg < a.D / 16) lg *= 2;
  const int all = ((a.hq + 2 * a.hkv) * lg + 31) / 32;  // steps of a token
  // A warp a step as long as the SMs hold most of those warps at once; then as
  // few warps to a token as still fill the SMs.
  const int64_t warps = static_cast<int64_t>(sms) * 24;
  int parts = all;
  if (static_cast<int64_t>(a.tok) * all > 2 * warps)
    parts = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(all, 2 * warps / a.tok)));
  const int steps = (all + parts - 1) / parts;
  parts = (all + steps - 1) / steps;
  const int64_t grid = (static_cast<int64_t>(a.tok) + 7) / 8 * parts;
  if (grid >= (int64_t(1) << 31)) return LORA_ERR_UNSUPPORTED;
  const unsigned g = static_cast<unsigned>(grid);
  if (steps > 1) launch_rope<E, C8, INTER, NORM, 2>(a, lg, g, parts, steps, st);
  else launch_rope<E, C8, INTER, NORM, 1>(a, lg, g, parts, steps, st);
  return LORA_OK;
}

template <class E, bool C8>
lora_status rope_append(const lora::RopeAppendArgs& a, int sms, cudaStream_t st) {
  const int heads = a.hq + 2 * a.hkv;
  auto mul = [](int64_t m, std::initializer_list<int64_t> v) {
    for (int64_t x : v)
      if (x % m) return false;
    return true;
  };
  const int cb = C8 ? 8 : 16;  // bytes of a piece of the cache
  const bool pieces =
      a.D % 16 == 0 && (a.R % 16 == 0 || a.interleaved) && aligned_to(a.qkv, 16) &&
      (a.tok == 1 || mul(8, {a.ld_qkv, a.ld_q})) &&  // an only row's stride says nothing
      mul(8, {a.off_q, a.off_k, a.off_v, a.k_page, a.k_slot, a.k_head, a.v_page, a.v_slot,
              a.v_head}) &&
      aligned_to(a.q_out, 16) && aligned_to(a.kc, cb) && aligned_to(a.vc, cb) &&
      aligned_to(a.qw, 16) && aligned_to(a.kw, 16);
  if (pieces) {
    const lora_status s = a.interleaved
                              ? (a.qw ? rope_pieces<E, C8, true, true>(a, sms, st)
                                      : rope_pieces<E, C8, true, false>(a, sms, st))
                              : (a.qw ? rope_pieces<E, C8, false, true>(a, sms, st)
                                      : rope_pieces<E, C8, false, false>(a, sms, st));
    if (s != LORA_OK) return s;
  } else {
    const int64_t grid = (static_cast<int64_t>(a.tok) * heads + 7) / 8;
    if (grid >= (int64_t(1) << 31)) return LORA_ERR_UNSUPPORTED;
    lora::rope_append_general_kernel<E, C8><<<static_cast<unsigned>(grid), 256, 0, st>>>(a);
  }
  ++g_launches;
  g_last_path = LORA_PATH_GENERAL;
  return launch_status();
}

}  // namespace

extern "C" lora_status lora_rope_append(
    const void* qkv, int64_t ld_qkv, const int32_t* qkv_offsets, int head_dim, int rotary_dim,
    const void* positions, int64_t ld_pos, int axes, const uint8_t* axis_map,
    const float* cos_sin, int64_t max_pos, int interleaved, const void* q_weight,
    const void* k_weight, float weight_offset, float eps, void* q_out, int64_t ld_q,
    void* k_cache, const int64_t* k_strides, void* v_cache, const int64_t* v_strides,
    int64_t num_pages, int page_size, lora_dtype cache_dtype, float k_scale, float v_scale,
    const void* slots, int index_bytes, int tok, lora_dtype dtype, void* stream) {
  if (dtype != LORA_BF16 && dtype != LORA_FP16) return LORA_ERR_UNSUPPORTED;
  if (cache_dtype != dtype && cache_dtype != LORA_E4M3) return LORA_ERR_UNSUPPORTED;
  if (index_bytes != 4 && index_bytes != 8) return LORA_ERR_UNSUPPORTED;
  if (!qkv_offsets || !k_strides || !v_strides) return LORA_ERR_INVALID_ARGUMENT;
  if (tok < 0 || head_dim < 1 || rotary_dim < 0 || rotary_dim > head_dim || rotary_dim % 2 ||
      axes < 1 || num_pages < 0 || page_size < 1 || !(eps >= 0.f))
    return LORA_ERR_INVALID_ARGUMENT;
  if (head_dim > lora::kRopeMaxDim || axes > lora::kRopeMaxAxes || tok >= (1 << 30))
    return LORA_ERR_UNSUPPORTED;
  const int32_t* off = qkv_offsets;
  if (off[0] < 0 || off[1] < off[0] || off[2] < off[1] || off[3] < off[2] || off[3] > ld_qkv)
    return LORA_ERR_INVALID_ARGUMENT;
  const int wq = off[1] - off[0], wk = off[2] - off[1], wv = off[3] - off[2];
  if (wq % head_dim || wk % head_dim || wk != wv || ld_q < wq) return LORA_ERR_INVALID_ARGUMENT;
  if ((q_weight != nullptr) != (k_weight != nullptr)) return LORA_ERR_INVALID_ARGUMENT;
  // positive, and with a finite reciprocal, which is what is multiplied by
  if (!(k_scale > 0.f) || !(v_scale > 0.f) || std::isinf(1.f / k_scale) || std::isinf(1.f / v_scale))
    return LORA_ERR_INVALID_ARGUMENT;
  if (rotary_dim && (max_pos < 1 || (axes > 1 && (!axis_map || ld_pos < tok))))
    return LORA_ERR_INVALID_ARGUMENT;
  for (int i = 0; i < 3; ++i)
    if (k_strides[i] < 0 || v_strides[i] < 0) return LORA_ERR_INVALID_ARGUMENT;
  lora::RopeAppendArgs a;
  std::memset(&a, 0, sizeof(a));
  if (axes > 1)
    for (int i = 0; i < rotary_dim / 2; ++i) {
      if (axis_map[i] >= axes) return LORA_ERR_INVALID_ARGUMENT;
      a.axis_of[i >> 3] |= static_cast<uint16_t>(axis_map[i] << (2 * (i & 7)));
    }
  if (tok == 0 || wq + wk == 0) return LORA_OK;
  if (!qkv || !slots || (wq && !q_out) || (wk && num_pages && (!k_cache || !v_cache)) ||
      (rotary_dim && (!positions || !cos_sin)))
    return LORA_ERR_INVALID_ARGUMENT;
  const uintptr_t ib = static_cast<uintptr_t>(index_bytes);
  const uintptr_t cb = cache_dtype == LORA_E4M3 ? 1 : 2;
  if (!aligned_to(qkv, 2) || !aligned_to(q_out, 2) || !aligned_to(k_cache, cb) ||
      !aligned_to(v_cache, cb) || !aligned_to(slots, ib) || !aligned_to(positions, ib) ||
      !aligned_to(cos_sin, 4) || !aligned_to(q_weight, 2) || !aligned_to(k_weight, 2))
    return LORA_ERR_INVALID_ARGUMENT;
  a.qkv = static_cast<const uint16_t*>(qkv);
  a.ld_qkv = ld_qkv;
  a.off_q = off[0];
  a.off_k = off[1];
  a.off_v = off[2];
  a.hq = wq / head_dim;
  a.hkv = wk / head_dim;
  a.D = head_dim;
  a.R = rotary_dim;
  a.positions = positions;
  a.ld_pos = ld_pos;
  a.axes = axes;
  a.cos_sin = cos_sin;
  a.max_pos = max_pos;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.ld_q = ld_q;
  a.kc = k_cache;
  a.vc = v_cache;
  a.k_page = k_strides[0];
  a.k_slot = k_strides[1];
  a.k_head = k_strides[2];
  a.v_page = v_strides[0];
  a.v_slot = v_strides[1];
  a.v_head = v_strides[2];
  a.pages = num_pages;
  a.page_size = page_size;
  a.slots = slots;
  a.qw = static_cast<const uint16_t*>(q_weight);
  a.kw = static_cast<const uint16_t*>(k_weight);
  a.eps = eps;
  a.w0 = weight_offset;
  a.k_inv = 1.f / k_scale;
  a.v_inv = 1.f / v_scale;
  a.tok = tok;
  a.interleaved = interleaved;
  a.idx64 = index_bytes == 8;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool c8 = cache_dtype == LORA_E4M3;
  const DeviceFacts* dev = device_facts();
  if (!dev) return LORA_ERR_CUDA;
  const int sms = dev->sms;
  if (dtype == LORA_BF16)
    return c8 ? rope_append<lora::Bf16, true>(a, sms, st) : rope_append<lora::Bf16, false>(a, sms, st);
  return c8 ? rope_append<lora::Fp16, true>(a, sms, st) : rope_append<lora::Fp16, false>(a, sms, st);
}

// ------------------------------------------------------------------ 4-bit base projection

namespace {

// 2-D map of bytes or 16-bit elements, box {box_cols, box_rows}.
bool encode_w4(CUtensorMap* m, CUtensorMapDataType type, const void* base, uint64_t cols,
               uint64_t rows, uint64_t row_bytes, uint32_t box_cols, uint32_t box_rows,
               CUtensorMapSwizzle swz) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {row_bytes};
  cuuint32_t box[2] = {box_cols, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, type, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kW4Smem = 227 * 1024;
constexpr int kMvSmem = 200 * 1024;

// Shared memory of w4_mv for tt tokens: staged x, and two tiles' parts.
template <int NT>
int64_t w4_mv_bytes(int64_t tt, int K) {
  const int64_t blocks = (K + 127) / 128;
  return tt * lora::mv_row_bytes(static_cast<int>(blocks) * 128) + 2 * lora::kMvWarps * NT * 512;
}

// Whether w4_mv holds the rows of x of up to 16 tokens at once.
inline bool w4_mv_holds(int tok, int K) {
  return (tok <= 8 ? w4_mv_bytes<1>(tok, K) : w4_mv_bytes<2>(std::min(tok, 16), K)) <= kMvSmem;
}

// Whether rows of x that TMA cannot load are copied to rows that it can (where
// there is a workspace): from 17 tokens on, and where w4_mv would read the
// weights more than once (13 x 8191 x 6144, twice: 37.9 us, copied 21.5).  Where
// it reads them once it is the faster with small groups (13 x 3583 x 6159 in
// groups of 32: 16, copied 18) and about even with large ones (13 x 3583, groups
// of 128, 6144 and 24,576 wide: 12.9 and 26.0, copied some 12.3 and 25.5).
inline bool w4_copies(int tok, int K) { return tok > 16 || !w4_mv_holds(tok, K); }

template <class E, bool X8, int NT, int VW>
lora_status w4_mv(const lora::W4Args& a, int sms, cudaStream_t st) {
  const int tiles = (a.N + 15) / 16;
  int tt = std::min(a.tok, 8 * NT);
  while (tt > 1 && w4_mv_bytes<NT>(tt, a.K) > kMvSmem) --tt;
  const int64_t bytes = w4_mv_bytes<NT>(tt, a.K);
  if (bytes > kMvSmem || a.ld_s >= (int64_t(1) << 31)) return LORA_ERR_UNSUPPORTED;
  const int smem = static_cast<int>(bytes);
  const int64_t gy = (a.tok + tt - 1) / tt;
  if (gy > 65535) return LORA_ERR_UNSUPPORTED;
  const dim3 grid(std::min(tiles, sms), static_cast<unsigned>(gy));
  auto kernel = lora::w4_mv_kernel<E, X8, NT, VW>;
  static std::atomic<uint64_t> ready{0};  // a bit for each device
  if (!set_smem_once(ready, reinterpret_cast<const void*>(kernel), kMvSmem)) return LORA_ERR_CUDA;
  kernel<<<grid, lora::kMvThreads, smem, st>>>(a, tt);
  ++g_launches;
  g_last_path = LORA_PATH_GENERAL;
  return launch_status();
}

// Clusters of 1 .. 8 blocks of a kernel, one block an SM, that a device holds at
// once (fewer than its SMs over the size, where that does not divide a GPC's).
struct ClusterFacts {
  std::atomic<int> ready{0};
  int most[9] = {0};
};

// The current device's of a kernel's facts (one for each device), which how a
// tile's K is split goes by: null where one cannot be asked for, to be asked for
// again by the next call.
template <class K>
const int* cluster_counts(ClusterFacts* facts, K kernel, int threads, size_t smem) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  ClusterFacts& f = facts[dev];
  if (f.ready.load(std::memory_order_acquire)) return f.most;
  std::lock_guard<std::mutex> lk(g_dev_mu);
  if (!f.ready.load(std::memory_order_relaxed)) {
    for (int cs = 1; cs <= 8; ++cs) {
      cudaLaunchConfig_t cfg{};
      cfg.gridDim = dim3(64 * cs);
      cfg.blockDim = dim3(threads);
      cfg.dynamicSmemBytes = smem;
      LaunchAttrs la;
      la.cluster(cs);
      la.apply(cfg);
      if (cudaOccupancyMaxActiveClusters(&f.most[cs], kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();  // a failed query must not leave a sticky launch error
        return nullptr;
      }
    }
    f.ready.store(1, std::memory_order_release);
  }
  return f.most;
}

template <class E, bool X8, int NT, int GS, int SETS, int SW>
lora_status w4_tc(const lora::W4Args& a, int sms, cudaStream_t st) {
  using C = lora::W4Tc<X8, NT, GS, SETS, SW>;
  lora::W4TcParams P;
  std::memset(&P, 0, sizeof(P));
  P.a = a;
  P.tiles_n = (a.N + lora::kW4M - 1) / lora::kW4M;
  P.tiles_t = (a.tok + NT - 1) / NT;
  P.nkb = (a.K + lora::kW4K - 1) / lora::kW4K;
  const int64_t tiles = static_cast<int64_t>(P.tiles_n) * P.tiles_t;
  if (tiles > (1 << 28)) return LORA_ERR_UNSUPPORTED;
  // all 512 TMEM columns: with this much shared memory no other block that
  // takes TMEM fits beside it (they ask for kTmemCtaMinSmem at least)
  constexpr size_t smem = std::max<size_t>(C::kSmem, 2 * kTmemCtaMinSmem);
  P.idesc = lora::make_idesc_f16(!X8 && std::is_same<E, lora::Bf16>::value ? 1 : 0, lora::kW4M, NT);
  const CUtensorMapDataType xt = X8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                 : std::is_same<E, lora::Bf16>::value
                                     ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                     : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  if (!encode_w4(&P.tmap_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w, (a.K + 31) / 32 * 16, a.N, a.ld_w,
                 64, lora::kW4M, CU_TENSOR_MAP_SWIZZLE_64B) ||
      !encode_w4(&P.tmap_x, xt, a.x, a.K, a.tok, a.ld_x * (X8 ? 1 : 2), X8 ? 128 : 64, NT,
                 CU_TENSOR_MAP_SWIZZLE_128B))
    return LORA_ERR_CUDA;
  auto kernel = lora::w4_tc_kernel<E, X8, NT, GS, SETS, SW>;
  static std::atomic<uint64_t> ready{0};  // a bit for each device
  if (!set_smem_once(ready, reinterpret_cast<const void*>(kernel), kW4Smem,
                     C::kSplit ? C::kRegs : 0))
    return LORA_ERR_CUDA;
  static ClusterFacts facts[kMaxDevices];
  const int* most = cluster_counts(facts, kernel, C::kThreads, smem);
  if (!most) return LORA_ERR_CUDA;
  // Whole waves of one tile for each SM; the tiles left over share the SMs by
  // splitting their K range over clusters, in a launch of their own that takes
  // SMs as the first one's blocks leave them.
  auto launch = [&](int64_t lo, int64_t hi, bool after) {
    P.tile0 = static_cast<int>(lo);
    P.tile1 = static_cast<int>(hi);
    // Least waves x (blocks of K each + 4): a wave's set-up and the adding up
    // of the parts cost about as much as four blocks.
    P.cs = 1;
    if (hi - lo < sms) {
      int64_t best = P.nkb + 4;
      for (int cs = 2; cs <= std::min(8, P.nkb); ++cs) {
        if (most[cs] < 1) continue;
        const int64_t cost =
            (hi - lo + most[cs] - 1) / most[cs] * ((P.nkb + cs - 1) / cs + 4);
        if (cost < best) {
          best = cost;
          P.cs = cs;
        }
      }
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(
        static_cast<unsigned>(P.cs > 1 ? (hi - lo) * P.cs : std::min<int64_t>(hi - lo, sms)));
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    LaunchAttrs la;
    if (P.cs > 1) la.cluster(static_cast<unsigned>(P.cs));
    if (after) la.programmatic();
    la.apply(cfg);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, P);
    ++g_launches;
    return e == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
  };
  const int64_t left = tiles % sms;
  // (Up to 64 tokens a second wave of whole tiles, which has the memory to
  // itself, is the shorter: 31.7 against 33.7 us at 32 tokens x 4096 x 24576.)
  const bool split = NT > 64 && tiles > sms && left > 0 && left <= sms / 2 && P.nkb > 1;
  const int64_t whole = split ? tiles - left : tiles;
  lora_status s = launch(0, whole, false);
  if (s == LORA_OK && split) s = launch(whole, tiles, true);
  g_last_path = LORA_PATH_TENSOR | (P.cs > 1 ? LORA_PATH_SPLITK : 0);
  return s;
}

// Bytes between the rows of x copied to the workspace.
inline int64_t w4_pitch(int K, bool x8) { return (static_cast<int64_t>(K) * (x8 ? 1 : 2) + 15) / 16 * 16; }

template <class E, bool X8, int GS>
lora_status w4_project_group(lora::W4Args a, void* ws, size_t ws_bytes, int sms, cudaStream_t st) {
  constexpr int VW = 1 << (GS - 5);
  const int64_t ldb = a.ld_x * (X8 ? 1 : 2);
  bool tma_x = aligned_to(a.x, 16) && ldb % 16 == 0;
  const int64_t pitch = w4_pitch(a.K, X8);
  if (!tma_x && w4_copies(a.tok, a.K) && ws && ws_bytes >= static_cast<size_t>(a.tok * pitch)) {
    const int64_t pieces = a.tok * (pitch / 16);
    lora::align_rows_kernel<<<static_cast<unsigned>((pieces + 255) / 256), 256, 0, st>>>(
        static_cast<const uint8_t*>(a.x), ldb, static_cast<uint8_t*>(ws), a.K * (X8 ? 1 : 2),
        static_cast<int>(pitch), pieces);
    ++g_launches;
    if (launch_status() != LORA_OK) return LORA_ERR_CUDA;
    a.x = ws;
    a.ld_x = pitch / (X8 ? 1 : 2);
    tma_x = true;
  }
  // w4_mv reads the weights once for eight tokens at a time (8 tokens at 4096 x
  // 24576: 21 us, against 28 with w4_tc; 9 at 4096 x 6144: 12.6 against 10.7),
  // so beyond that it only takes what TMA cannot; it needs all of K's x in
  // shared memory.
  if ((a.tok <= 8 && w4_mv_holds(a.tok, a.K)) || !tma_x)
    return a.tok <= 8 ? w4_mv<E, X8, 1, VW>(a, sms, st) : w4_mv<E, X8, 2, VW>(a, sms, st);
  if (a.tok <= 16) return w4_tc<E, X8, 16, GS, 4, 4>(a, sms, st);
  if (a.tok <= 32) return w4_tc<E, X8, 32, GS, 4, 4>(a, sms, st);
  if (a.tok <= 64) return w4_tc<E, X8, 64, GS, 4, 8>(a, sms, st);
  return w4_tc<E, X8, 128, GS, 4, 8>(a, sms, st);
}

template <class E, bool X8>
lora_status w4_project(const lora::W4Args& a, void* ws, size_t ws_bytes, int sms,
                       cudaStream_t st) {
  if (a.group_shift == 5) return w4_project_group<E, X8, 5>(a, ws, ws_bytes, sms, st);
  if (a.group_shift == 6) return w4_project_group<E, X8, 6>(a, ws, ws_bytes, sms, st);
  return w4_project_group<E, X8, 7>(a, ws, ws_bytes, sms, st);
}

}  // namespace

extern "C" size_t lora_w4_workspace_size(int tok, int K, lora_dtype x_dtype) {
  if (tok < 0 || K < 0) return 0;
  return static_cast<size_t>(tok * w4_pitch(K, x_dtype == LORA_E4M3));
}

extern "C" int lora_w4_copies_x(int tok, int K) {
  return tok > 0 && K > 0 && K <= (1 << 28) && w4_copies(tok, K);
}

extern "C" lora_status lora_w4_project(const void* x, int64_t ld_x, const float* x_scale,
                                       const void* W, int64_t ld_w, const void* w_scales,
                                       const uint8_t* w_zeros, int64_t ld_s, void* out,
                                       int64_t ld_out, int tok, int K, int N, int group,
                                       lora_dtype x_dtype, lora_dtype dtype, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  if (dtype != LORA_BF16 && dtype != LORA_FP16) return LORA_ERR_UNSUPPORTED;
  if (x_dtype != dtype && x_dtype != LORA_E4M3) return LORA_ERR_UNSUPPORTED;
  if (group != 32 && group != 64 && group != 128) return LORA_ERR_UNSUPPORTED;
  if (tok < 0 || K < 1 || N < 0 || ld_x < K || ld_out < N || ld_s < N ||
      ld_w < static_cast<int64_t>(K + 31) / 32 * 16)
    return LORA_ERR_INVALID_ARGUMENT;
  if ((x_scale != nullptr) != (x_dtype == LORA_E4M3)) return LORA_ERR_INVALID_ARGUMENT;
  if (tok >= (1 << 30) || N > (1 << 28) || K > (1 << 28)) return LORA_ERR_UNSUPPORTED;
  if (tok == 0 || N == 0) return LORA_OK;
  if (!x || !W || !w_scales || !out) return LORA_ERR_INVALID_ARGUMENT;
  if ((x_dtype != LORA_E4M3 && !aligned_to(x, 2)) || !aligned_to(x_scale, 4) ||
      !aligned_to(w_scales, 2) || !aligned_to(out, 2))
    return LORA_ERR_INVALID_ARGUMENT;
  if ((workspace_bytes && !workspace) || !aligned_to(workspace, 16)) return LORA_ERR_INVALID_ARGUMENT;
  const bool x8 = x_dtype == LORA_E4M3;
  // the stride of an only row says nothing
  if (tok == 1) ld_x = w4_pitch(K, x8) / (x8 ? 1 : 2);
  if (N == 1) ld_w = static_cast<int64_t>(K + 31) / 32 * 16;
  if (!aligned_to(W, 16) || ld_w % 16) return LORA_ERR_UNSUPPORTED;
  const lora::W4Args a{x, ld_x, x_scale, static_cast<const uint8_t*>(W), ld_w,
                       static_cast<const uint16_t*>(w_scales), w_zeros, ld_s,
                       static_cast<uint16_t*>(out), ld_out, tok, K, N,
                       group == 32 ? 5 : group == 64 ? 6 : 7};
  const DeviceFacts* dev = device_facts();
  if (!dev) return LORA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == LORA_BF16)
    return x8 ? w4_project<lora::Bf16, true>(a, workspace, workspace_bytes, dev->sms, st)
              : w4_project<lora::Bf16, false>(a, workspace, workspace_bytes, dev->sms, st);
  return x8 ? w4_project<lora::Fp16, true>(a, workspace, workspace_bytes, dev->sms, st)
            : w4_project<lora::Fp16, false>(a, workspace, workspace_bytes, dev->sms, st);
}

// ------------------------------------------------------------------ packed arguments

namespace {

// Takes the words of a packed call in their order.
class Words {
 public:
  explicit Words(const void* p) : p_(static_cast<const char*>(p)) {}
  int64_t i64() { return take<int64_t>(); }
  int i32() {
    // out of range for an int parameter: as invalid as it is there
    const int64_t v = i64();
    return v < INT32_MIN || v > INT32_MAX ? -1 : static_cast<int>(v);
  }
  float f32() { return static_cast<float>(take<double>()); }
  lora_dtype dtype() { return static_cast<lora_dtype>(i32()); }
  template <class T = void>
  T* ptr() {
    return reinterpret_cast<T*>(static_cast<uintptr_t>(i64()));
  }
  const void* rest() const { return p_; }

 private:
  template <class T>
  T take() {
    T v;
    std::memcpy(&v, p_, sizeof(v));
    p_ += 8;
    return v;
  }
  const char* p_;
};

}  // namespace

extern "C" lora_status lora_rmsnorm_packed(const void* words) {
  if (!words) return LORA_ERR_INVALID_ARGUMENT;
  Words w(words);
  const void* x = w.ptr();
  const int64_t ld_x = w.i64();
  const void* res = w.ptr();
  const int64_t ld_res = w.i64();
  void* res_out = w.ptr();
  const int64_t ld_res_out = w.i64();
  const void* weight = w.ptr();
  const float w0 = w.f32(), eps = w.f32();
  void* out = w.ptr();
  const int64_t ld_out = w.i64();
  void* q = w.ptr();
  const int64_t ld_q = w.i64();
  float* scale = w.ptr<float>();
  const int tok = w.i32(), H = w.i32();
  const lora_dtype dt = w.dtype();
  return lora_rmsnorm(x, ld_x, res, ld_res, res_out, ld_res_out, weight, w0, eps, out, ld_out, q,
                      ld_q, scale, tok, H, dt, w.ptr());
}

extern "C" lora_status lora_w4_project_packed(const void* words) {
  if (!words) return LORA_ERR_INVALID_ARGUMENT;
  Words w(words);
  const void* x = w.ptr();
  const int64_t ld_x = w.i64();
  const float* x_scale = w.ptr<float>();
  const void* W = w.ptr();
  const int64_t ld_w = w.i64();
  const void* s = w.ptr();
  const uint8_t* z = w.ptr<uint8_t>();
  const int64_t ld_s = w.i64();
  void* out = w.ptr();
  const int64_t ld_out = w.i64();
  const int tok = w.i32(), K = w.i32(), N = w.i32(), group = w.i32();
  const lora_dtype x_dt = w.dtype(), dt = w.dtype();
  void* ws = w.ptr();
  const size_t ws_bytes = static_cast<size_t>(w.i64());
  return lora_w4_project(x, ld_x, x_scale, W, ld_w, s, z, ld_s, out, ld_out, tok, K, N, group,
                         x_dt, dt, ws, ws_bytes, w.ptr());
}

extern "C" lora_status lora_rope_append_packed(const void* words) {
  if (!words) return LORA_ERR_INVALID_ARGUMENT;
  Words w(words);
  const void* qkv = w.ptr();
  const int64_t ld_qkv = w.i64();
  int32_t off[4];
  for (int32_t& o : off) o = w.i32();
  const int D = w.i32(), R = w.i32();
  const void* pos = w.ptr();
  const int64_t ld_pos = w.i64();
  const int axes = w.i32();
  const bool map = w.i64() != 0;
  const float* cs = w.ptr<float>();
  const int64_t max_pos = w.i64();
  const int inter = w.i32();
  const void* qw = w.ptr();
  const void* kw = w.ptr();
  const float w0 = w.f32(), eps = w.f32();
  void* q_out = w.ptr();
  const int64_t ld_q = w.i64();
  void* kc = w.ptr();
  int64_t ks[3], vs[3];
  for (int64_t& v : ks) v = w.i64();
  void* vc = w.ptr();
  for (int64_t& v : vs) v = w.i64();
  const int64_t pages = w.i64();
  const int page = w.i32();
  const lora_dtype cdt = w.dtype();
  const float k_scale = w.f32(), v_scale = w.f32();
  const void* slots = w.ptr();
  const int ib = w.i32(), tok = w.i32();
  const lora_dtype dt = w.dtype();
  void* stream = w.ptr();
  return lora_rope_append(qkv, ld_qkv, off, D, R, pos, ld_pos, axes,
                          map ? static_cast<const uint8_t*>(w.rest()) : nullptr, cs, max_pos,
                          inter, qw, kw, w0, eps, q_out, ld_q, kc, ks, vc, vs, pages, page, cdt,
                          k_scale, v_scale, slots, ib, tok, dt, stream);
}
