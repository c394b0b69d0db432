// Muon's element passes: the momentum of the flat grads and the update to
// orthogonalise, and the orthogonalised update's step on the fp32 master with
// the cast back to 16 bits; and the matrix plan they share with
// zds_newton_schulz.
//
// Both passes are streams with no reuse, bound by HBM: momentum reads the grad
// and m and writes m and the update (12 B per element with 16-bit grads and a
// BF16 update), apply reads the update and the master and writes the master
// and the 16-bit params (12 B). Every lane moves one quad of consecutive
// elements and its block ends: short blocks with one access of each array in
// flight for a wave run best here. Measured at 202,375,168 elements (a 7B
// decoder layer): momentum 373 us (6.5 TB/s) with blocks of 256, 391 and 396
// with 512 and 1024; apply 376 us (6.46 TB/s) with blocks of 512 and a quad a
// lane, 377 with 256, 381 with 1024, and 420 with 256 and four quads one
// after another. Arrays not aligned to four elements go one element a lane: 560
// and 536 us.
#include <algorithm>
#include <new>

#include "zds_device.h"
#include "zds_matrix.h"

namespace zds {

constexpr int kMuonBlock = 256;
constexpr int kApplyBlock = kApplyChunk / 4;

struct MomentumArgs {
  const zds_step_scalars *sc;
  const void *g;
  float *m;
  void *u;
  int64_t n;
  float mu, omu;
  int32_t nesterov;
};

// One element, one rounding per operation, in this order.
__device__ __forceinline__ float momentum_elem(float x, float gs, const MomentumArgs &a, float &m) {
  const float g = x * gs;
  const float t = a.omu * g;
  m = a.mu * m + t;
  return a.nesterov ? a.mu * m + t : m;
}

template <int D>
__device__ __forceinline__ void store_update(void *u, int64_t q, const float (&x)[4]) {
  if constexpr (D == ZDS_FP32) store_quad(static_cast<float *>(u), q, x);
  else store_quad16<D>(u, q, x);
}
template <int D>
__device__ __forceinline__ void store_update1(void *u, int64_t e, float x) {
  if constexpr (D == ZDS_FP32) static_cast<float *>(u)[e] = x;
  else static_cast<uint16_t *>(u)[e] = narrow1<D>(x);
}

template <int GD, int UD, bool VEC>
__global__ void __launch_bounds__(kMuonBlock) muon_momentum_kernel(const MomentumArgs a) {
  if (a.sc->overflow) return;
  const float gs = a.sc->grad_scale;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kMuonBlock;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kMuonBlock + threadIdx.x;
  int64_t done = 0;
  if constexpr (VEC) {
    const int64_t quads = a.n >> 2;
    for (int64_t q = first; q < quads; q += stride) {
      float x[4], m[4], u[4];
      load_quad<GD>(a.g, q, x);
      load_quad<ZDS_FP32>(a.m, q, m);
#pragma unroll
      for (int j = 0; j < 4; ++j) u[j] = momentum_elem(x[j], gs, a, m[j]);
      store_quad(a.m, q, m);
      store_update<UD>(a.u, q, u);
    }
    done = quads << 2;
  }
  for (int64_t e = done + first; e < a.n; e += stride) {
    float m = a.m[e];
    const float u = momentum_elem(widen1<GD>(a.g, e), gs, a, m);
    a.m[e] = m;
    store_update1<UD>(a.u, e, u);
  }
}

struct ApplyArgs {
  const zds_step_scalars *sc;
  const ApplyChunk *chunks;
  const void *u;
  float *p;
  void *out;
  double lr;
  float decay;
  int32_t scale;
  int64_t nchunks;
};

__device__ __forceinline__ float apply_elem(float u, float p, float decay, float f) {
  p = p * decay;
  return p - f * u;
}

// One chunk of one matrix per block.
template <int UD, int PD, bool WRITE_OUT>
__global__ void __launch_bounds__(kApplyBlock) muon_apply_kernel(const ApplyArgs a) {
  if (a.sc->overflow) return;
  for (int64_t k = blockIdx.x; k < a.nchunks; k += gridDim.x) {
    const ApplyChunk c = a.chunks[k];
    const float sf = a.scale == ZDS_MUON_SCALE_RMS ? c.rms : (a.scale == ZDS_MUON_SCALE_ASPECT ? c.aspect : 1.0f);
    const float f = static_cast<float>(a.lr * static_cast<double>(sf));
    float *p = a.p + c.first;
    const void *u = static_cast<const char *>(a.u) + c.first * (UD == ZDS_FP32 ? 4 : 2);
    uint16_t *out = WRITE_OUT ? static_cast<uint16_t *>(a.out) + c.first : nullptr;
    int done = 0;
    if (aligned(p, 16) && aligned(u, UD == ZDS_FP32 ? 16 : 8) && (!WRITE_OUT || aligned(out, 8))) {  // uniform per block
      const int quads = c.len >> 2;
      for (int q = threadIdx.x; q < quads; q += kApplyBlock) {
        float x[4], v[4];
        load_quad<UD>(u, q, x);
        load_quad<ZDS_FP32>(p, q, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = apply_elem(x[j], v[j], a.decay, f);
        store_quad(p, q, v);
        if (WRITE_OUT) store_quad16<PD>(out, q, v);
      }
      done = quads << 2;
    }
    for (int e = done + threadIdx.x; e < c.len; e += kApplyBlock) {
      const float v = apply_elem(widen1<UD>(u, e), p[e], a.decay, f);
      p[e] = v;
      if (WRITE_OUT) out[e] = narrow1<PD>(v);
    }
  }
}

template <int GD, int UD>
static void launch_momentum(bool vec, hipStream_t s, const MomentumArgs &a) {
  const int64_t items = vec ? (a.n + 3) / 4 : a.n;
  int64_t g = (items + kMuonBlock - 1) / kMuonBlock;
  if (g > max_blocks(kMuonBlock)) g = max_blocks(kMuonBlock);
  if (vec)
    hipLaunchKernelGGL((muon_momentum_kernel<GD, UD, true>), dim3(static_cast<uint32_t>(g)), dim3(kMuonBlock), 0, s, a);
  else
    hipLaunchKernelGGL((muon_momentum_kernel<GD, UD, false>), dim3(static_cast<uint32_t>(g)), dim3(kMuonBlock), 0, s, a);
}

template <int UD, int PD, bool WO>
static void launch_apply(hipStream_t s, const ApplyArgs &a) {
  const int64_t g = a.nchunks < max_blocks(kApplyBlock) ? a.nchunks : max_blocks(kApplyBlock);
  hipLaunchKernelGGL((muon_apply_kernel<UD, PD, WO>), dim3(static_cast<uint32_t>(g)), dim3(kApplyBlock), 0, s, a);
}

static zds_status check_hparams(const char *fn, const zds_muon_hparams *hp) {
  if (!hp) return fail(ZDS_EINVAL, "%s: null hparams", fn);
  if (!(hp->lr >= 0.0f) || !(hp->weight_decay >= 0.0f) || !(hp->lr <= FLT_MAX) || !(hp->weight_decay <= FLT_MAX))
    return fail(ZDS_EINVAL, "%s: need finite lr >= 0 and weight_decay >= 0", fn);
  if (!(hp->momentum >= 0.0f && hp->momentum < 1.0f)) return fail(ZDS_EINVAL, "%s: momentum must lie in [0, 1)", fn);
  if (hp->nesterov != 0 && hp->nesterov != 1) return fail(ZDS_EINVAL, "%s: nesterov must be 0 or 1", fn);
  if (hp->scale < ZDS_MUON_SCALE_NONE || hp->scale > ZDS_MUON_SCALE_RMS) return fail(ZDS_EINVAL, "%s: bad scale %d", fn, hp->scale);
  return ZDS_OK;
}

static void matrix_plan_free(zds_matrix_plan *p) {
  if (!p) return;
  for (NsMatrix *m : p->d_mats)
    if (m) (void)hipFree(m);
  if (p->d_tiles) (void)hipFree(p->d_tiles);
  if (p->d_chunks) (void)hipFree(p->d_chunks);
  delete p;
}

static zds_status check_overlap(const int64_t *offset, const int32_t *rows, const int32_t *cols, int32_t num) {
  std::vector<std::pair<int64_t, int64_t>> spans;
  for (int32_t i = 0; i < num; ++i) {
    const int64_t len = static_cast<int64_t>(rows[i]) * cols[i];
    if (len > 0) spans.emplace_back(offset[i], offset[i] + len);
  }
  std::sort(spans.begin(), spans.end());
  for (size_t i = 1; i < spans.size(); ++i)
    if (spans[i].first < spans[i - 1].second)
      return fail(ZDS_EINVAL, "zds_matrix_plan_create: matrices overlap at flat offset %lld", static_cast<long long>(spans[i].first));
  return ZDS_OK;
}

static zds_status build_matrix_plan(zds_matrix_plan *p, const int64_t *offset, const int32_t *rows, const int32_t *cols,
                                    int32_t num) {
  std::vector<ApplyChunk> chunks;
  for (int32_t i = 0; i < num; ++i) {
    const int64_t len = static_cast<int64_t>(rows[i]) * cols[i];
    if (offset[i] + len > p->span) p->span = offset[i] + len;
    if (len == 0) continue;
    if (chunks.empty() || offset[i] < p->first) p->first = offset[i];
    const double r = rows[i], c = cols[i];
    const float aspect = static_cast<float>(sqrt(r > c ? r / c : 1.0));
    const float rms = static_cast<float>(0.2 * sqrt(r > c ? r : c));
    for (int64_t e = 0; e < len; e += kApplyChunk)
      chunks.push_back(ApplyChunk{offset[i] + e, static_cast<int32_t>(std::min<int64_t>(kApplyChunk, len - e)), aspect, rms, 0});
  }
  p->num_chunks = static_cast<int64_t>(chunks.size());
  if (!chunks.empty()) {
    const size_t bytes = chunks.size() * sizeof(ApplyChunk);
    hipError_t e = hipMalloc(reinterpret_cast<void **>(&p->d_chunks), bytes);
    if (e != hipSuccess) return fail(ZDS_ENOMEM, "zds_matrix_plan_create: hipMalloc tables: %s", hipGetErrorString(e));
    e = hipMemcpy(p->d_chunks, chunks.data(), bytes, hipMemcpyHostToDevice);
    if (e != hipSuccess) return hip_fail(e, "zds_matrix_plan_create: table upload");
  }
  return build_newton_schulz(p, offset, rows, cols, num);
}

}  // namespace zds

using namespace zds;

extern "C" zds_status zds_matrix_plan_create(zds_matrix_plan **out, const int64_t *offset, const int32_t *rows,
                                             const int32_t *cols, int32_t num_matrices) {
  clear_error();
  const char *fn = "zds_matrix_plan_create";
  if (!out) return fail(ZDS_EINVAL, "%s: null out", fn);
  *out = nullptr;
  if (num_matrices < 0 || (num_matrices > 0 && (!offset || !rows || !cols)))
    return fail(ZDS_EINVAL, "%s: null pointer or negative matrix count", fn);
  for (int32_t i = 0; i < num_matrices; ++i) {
    if (rows[i] < 0 || cols[i] < 0 || rows[i] >= (1 << 17) || cols[i] >= (1 << 17))
      return fail(ZDS_EINVAL, "%s: matrix %d: sizes must lie in [0, 2^17)", fn, i);
    if (static_cast<int64_t>(rows[i]) * cols[i] >= (int64_t(1) << 31))
      return fail(ZDS_EINVAL, "%s: matrix %d holds 2^31 elements or more", fn, i);
    if (offset[i] < 0 || offset[i] >= (int64_t(1) << 40)) return fail(ZDS_EINVAL, "%s: matrix %d: offset must lie in [0, 2^40)", fn, i);
  }
  zds_matrix_plan *p = new (std::nothrow) zds_matrix_plan;
  if (!p) return fail(ZDS_ENOMEM, "%s: host allocation failed", fn);
  p->num = num_matrices;
  zds_status st = ZDS_OK;
  try {
    st = check_overlap(offset, rows, cols, num_matrices);
    if (st == ZDS_OK) {
      const hipError_t he = hipGetDevice(&p->device);
      st = he != hipSuccess ? hip_fail(he, "zds_matrix_plan_create: hipGetDevice")
                            : build_matrix_plan(p, offset, rows, cols, num_matrices);
    }
  } catch (const std::bad_alloc &) {
    st = fail(ZDS_ENOMEM, "%s: host allocation failed", fn);
  }
  if (st != ZDS_OK) {
    matrix_plan_free(p);
    return st;
  }
  *out = p;
  return ZDS_OK;
}

extern "C" void zds_matrix_plan_destroy(zds_matrix_plan *plan) { matrix_plan_free(plan); }

extern "C" int32_t zds_matrix_plan_num_matrices(const zds_matrix_plan *plan) { return plan ? plan->num : -1; }

extern "C" int64_t zds_matrix_plan_span(const zds_matrix_plan *plan) { return plan ? plan->span : -1; }

extern "C" zds_status zds_muon_momentum(const zds_muon_hparams *hp, const void *grads, zds_dtype grad_dtype,
                                        float *momentum, void *update, zds_dtype update_dtype, int64_t n,
                                        const zds_step_scalars *scalars_dev, void *stream) {
  clear_error();
  const char *fn = "zds_muon_momentum";
  zds_status st = check_hparams(fn, hp);
  if (st != ZDS_OK) return st;
  if (!valid_dtype(grad_dtype)) return fail(ZDS_EINVAL, "%s: bad grad dtype", fn);
  if (update_dtype != ZDS_BF16 && update_dtype != ZDS_FP32) return fail(ZDS_EINVAL, "%s: update dtype must be bf16 or fp32", fn);
  if (n < 0 || n >= (int64_t(1) << 40)) return fail(ZDS_EINVAL, "%s: n must lie in [0, 2^40)", fn);
  if (n == 0) return ZDS_OK;
  if (!grads || !momentum || !update || !scalars_dev) return fail(ZDS_EINVAL, "%s: null pointer", fn);
  if (!aligned(grads, static_cast<uintptr_t>(dtype_size(grad_dtype))) || !aligned(momentum, 4) ||
      !aligned(update, static_cast<uintptr_t>(dtype_size(update_dtype))) || !aligned(scalars_dev, 8))
    return fail(ZDS_EALIGN, "%s: pointer not aligned to its element size", fn);
  const int64_t gb = n * dtype_size(grad_dtype), ub = n * dtype_size(update_dtype);
  if (ranges_meet(momentum, n * 4, grads, gb) || ranges_meet(momentum, n * 4, update, ub) ||
      (ranges_meet(grads, gb, update, ub) && !(grads == update && gb == ub)))
    return fail(ZDS_EINVAL, "%s: grads, momentum and update overlap", fn);
  const MomentumArgs a{scalars_dev, grads, momentum, update, n, hp->momentum, 1.0f - hp->momentum, hp->nesterov};
  const bool vec = aligned(grads, grad_dtype == ZDS_FP32 ? 16 : 8) && aligned(momentum, 16) &&
                   aligned(update, update_dtype == ZDS_FP32 ? 16 : 8);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool f = update_dtype == ZDS_FP32;
  switch (grad_dtype) {
    case ZDS_FP16: f ? launch_momentum<ZDS_FP16, ZDS_FP32>(vec, s, a) : launch_momentum<ZDS_FP16, ZDS_BF16>(vec, s, a); break;
    case ZDS_BF16: f ? launch_momentum<ZDS_BF16, ZDS_FP32>(vec, s, a) : launch_momentum<ZDS_BF16, ZDS_BF16>(vec, s, a); break;
    default: f ? launch_momentum<ZDS_FP32, ZDS_FP32>(vec, s, a) : launch_momentum<ZDS_FP32, ZDS_BF16>(vec, s, a); break;
  }
  return check_launch("muon_momentum kernel");
}

extern "C" zds_status zds_muon_apply(const zds_muon_hparams *hp, const zds_matrix_plan *plan, const void *update,
                                     zds_dtype update_dtype, float *master, void *params_out, zds_dtype param_dtype,
                                     const zds_step_scalars *scalars_dev, void *stream) {
  clear_error();
  const char *fn = "zds_muon_apply";
  zds_status st = check_hparams(fn, hp);
  if (st != ZDS_OK) return st;
  if (!plan) return fail(ZDS_EINVAL, "%s: null plan", fn);
  if (update_dtype != ZDS_BF16 && update_dtype != ZDS_FP32) return fail(ZDS_EINVAL, "%s: update dtype must be bf16 or fp32", fn);
  if (params_out && param_dtype != ZDS_FP16 && param_dtype != ZDS_BF16)
    return fail(ZDS_EINVAL, "%s: param dtype must be fp16 or bf16", fn);
  if (plan->num_chunks == 0) return ZDS_OK;
  if (!update || !master || !scalars_dev) return fail(ZDS_EINVAL, "%s: null pointer", fn);
  if (!aligned(update, static_cast<uintptr_t>(dtype_size(update_dtype))) || !aligned(master, 4) ||
      (params_out && !aligned(params_out, 2)) || !aligned(scalars_dev, 8))
    return fail(ZDS_EALIGN, "%s: pointer not aligned to its element size", fn);
  int dev = 0;
  const hipError_t he = hipGetDevice(&dev);
  if (he != hipSuccess) return hip_fail(he, "hipGetDevice");
  if (dev != plan->device) return fail(ZDS_EINVAL, "%s: plan belongs to device %d, current is %d", fn, plan->device, dev);
  // what the plan covers of each array
  const auto from = [&](const void *p, int64_t es) { return static_cast<const char *>(p) + plan->first * es; };
  const int64_t len = plan->span - plan->first, ue = dtype_size(update_dtype);
  if (ranges_meet(from(master, 4), len * 4, from(update, ue), len * ue) ||
      (params_out && ranges_meet(from(master, 4), len * 4, from(params_out, 2), len * 2)) ||
      (params_out && ranges_meet(from(update, ue), len * ue, from(params_out, 2), len * 2) &&
       !(params_out == update && ue == 2)))
    return fail(ZDS_EINVAL, "%s: update, master and params_out overlap", fn);
  const double lr = hp->lr;
  const ApplyArgs a{scalars_dev, plan->d_chunks, update, master, params_out, lr,
                    static_cast<float>(1.0 - lr * static_cast<double>(hp->weight_decay)), hp->scale, plan->num_chunks};
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool f = update_dtype == ZDS_FP32;
  if (!params_out) {
    f ? launch_apply<ZDS_FP32, ZDS_BF16, false>(s, a) : launch_apply<ZDS_BF16, ZDS_BF16, false>(s, a);
  } else if (param_dtype == ZDS_BF16) {
    f ? launch_apply<ZDS_FP32, ZDS_BF16, true>(s, a) : launch_apply<ZDS_BF16, ZDS_BF16, true>(s, a);
  } else {
    f ? launch_apply<ZDS_FP32, ZDS_FP16, true>(s, a) : launch_apply<ZDS_BF16, ZDS_FP16, true>(s, a);
  }
  return check_launch("muon_apply kernel");
}
