// AdamW on moments in fewer bits: zds_adam_step's update on a first moment in
// E4M3 and a second one in UE5M3 or BF16, read back and quantised again at
// random (include/zds.h; zds_quantised.h has the formats' arithmetic,
// zds_adam.h the update).
#include "zds_adam.h"
#include "zds_quantised.h"

namespace zds {

struct AdamQ8Args {
  const zds_step_scalars *sc;
  const zds_step_state *state;
  const void *g;
  float *p;
  void *m;
  uint8_t *me;
  void *v;
  uint8_t *ve;
  void *out;
  int64_t n;
  uint64_t seed;
  int64_t first;
};

// One unit of 512 elements by a wave: each lane a quad of either half. FULL:
// the unit lies inside the arrays, and they are aligned.
template <int GD, int PD, int VF, bool FULL>
__device__ __forceinline__ void q8_unit(const AdamQ8Args &a, const ElemConsts &c, int64_t u, uint32_t steps, int lane) {
  const QuadBits rb = unit_random_bits(a.seed, static_cast<uint64_t>((a.first + u * kStateUnit) >> 3), steps, lane);
  uint8_t *mc = static_cast<uint8_t *>(a.m);
  uint8_t *vc = static_cast<uint8_t *>(a.v);
  uint16_t *v16 = static_cast<uint16_t *>(a.v);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t e = u * kStateUnit + 256 * h + 4 * lane;
    const bool any = FULL || e < a.n;
    float g[4], p[4], m[4], v[4];
    uint32_t mw = 0, vw = 0;
    const uint32_t ms = any ? a.me[e >> 5] : 0u;
    const uint32_t vs = VF != ZDS_STATE_BF16 && any ? a.ve[e >> 5] : 0u;
    if (FULL) {
      load_quad<GD>(a.g, e >> 2, g);
      load_quad<ZDS_FP32>(a.p, e >> 2, p);
      mw = ld_stream(reinterpret_cast<const uint32_t *>(mc + e));
      if constexpr (VF == ZDS_STATE_BF16) load_quad<ZDS_BF16>(a.v, e >> 2, v);
      else vw = ld_stream(reinterpret_cast<const uint32_t *>(vc + e));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool in = e + i < a.n;
        g[i] = in ? widen1<GD>(a.g, e + i) : 0.0f;
        p[i] = in ? a.p[e + i] : 0.0f;
        mw |= (in ? static_cast<uint32_t>(mc[e + i]) : 0u) << (8 * i);
        if constexpr (VF == ZDS_STATE_BF16) v[i] = in ? widen1<ZDS_BF16>(a.v, e + i) : 0.0f;
        else vw |= (in ? static_cast<uint32_t>(vc[e + i]) : 0u) << (8 * i);
      }
    }
    decode_quad<ZDS_STATE_E4M3>(mw, ms, m);
    if constexpr (VF != ZDS_STATE_BF16) decode_quad<VF>(vw, vs, v);
    uint32_t mm = 0, vm = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      adam_elem(g[i], c, p[i], m[i], v[i]);
      if (!FULL && e + i >= a.n) m[i] = v[i] = 0.0f;
      mm = magnitude(m[i]) > mm ? magnitude(m[i]) : mm;
      vm = magnitude(v[i]) > vm ? magnitude(v[i]) : vm;
    }
    const uint32_t (&w)[2] = h ? rb.r1 : rb.r0;
    mm = block_max(mm);
    const uint32_t ms1 = exponent_byte<ZDS_STATE_E4M3>(mm);
    mw = encode_quad<ZDS_STATE_E4M3, true>(m, ms1, mm, w);
    u32x2 v2{};
    uint32_t vs1 = 0;
    if constexpr (VF == ZDS_STATE_BF16) {
      v2 = encode_quad_bf16<true>(v, w);
    } else {
      vm = block_max(vm);
      vs1 = exponent_byte<VF>(vm);
      vw = encode_quad<VF, true, true>(v, vs1, vm, w);
    }
    if (FULL) {
      store_quad(a.p, e >> 2, p);
      if constexpr (PD >= 0) store_quad16<PD>(a.out, e >> 2, p);
      st_stream(reinterpret_cast<uint32_t *>(mc + e), mw);
      if constexpr (VF == ZDS_STATE_BF16) st_stream(reinterpret_cast<u32x2 *>(v16 + e), v2);
      else st_stream(reinterpret_cast<uint32_t *>(vc + e), vw);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (e + i >= a.n) break;
        a.p[e + i] = p[i];
        if constexpr (PD >= 0) static_cast<uint16_t *>(a.out)[e + i] = narrow1<PD>(p[i]);
        mc[e + i] = static_cast<uint8_t>(mw >> (8 * i));
        if constexpr (VF == ZDS_STATE_BF16) v16[e + i] = static_cast<uint16_t>((i < 2 ? v2.x : v2.y) >> (16 * (i & 1)));
        else vc[e + i] = static_cast<uint8_t>(vw >> (8 * i));
      }
    }
    if ((lane & 7) == 0 && any) {
      a.me[e >> 5] = static_cast<uint8_t>(ms1);
      if constexpr (VF != ZDS_STATE_BF16) a.ve[e >> 5] = static_cast<uint8_t>(vs1);
    }
  }
}

// PD: the params' type, -1 for none.
template <int GD, int PD, int VF, bool VEC>
__global__ void __launch_bounds__(256) adam_q8_kernel(AdamQ8Args a) {
  if (a.sc->overflow) return;  // the step is skipped: uniform, nothing is touched
  const ElemConsts c = load_consts(a.sc);
  const uint32_t steps = a.state->steps_seen;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t units = (a.n + kStateUnit - 1) / kStateUnit;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * 4 + wave; u < units; u += static_cast<int64_t>(gridDim.x) * 4) {
    if (VEC && (u + 1) * kStateUnit <= a.n) q8_unit<GD, PD, VF, VEC>(a, c, u, steps, lane);
    else q8_unit<GD, PD, VF, false>(a, c, u, steps, lane);
  }
}

template <int GD, int PD, int VF>
static void q8_go(bool vec, const AdamQ8Args &a, hipStream_t s) {
  int64_t g = (a.n + 4 * kStateUnit - 1) / (4 * kStateUnit);
  if (g > max_blocks(256)) g = max_blocks(256);
  if (vec) hipLaunchKernelGGL((adam_q8_kernel<GD, PD, VF, true>), dim3(static_cast<uint32_t>(g)), dim3(256), 0, s, a);
  else hipLaunchKernelGGL((adam_q8_kernel<GD, PD, VF, false>), dim3(static_cast<uint32_t>(g)), dim3(256), 0, s, a);
}
template <int GD, int PD>
static void q8_vf(zds_state_format f, bool vec, const AdamQ8Args &a, hipStream_t s) {
  if (f == ZDS_STATE_BF16) q8_go<GD, PD, ZDS_STATE_BF16>(vec, a, s);
  else q8_go<GD, PD, ZDS_STATE_UE5M3>(vec, a, s);
}
template <int GD>
static void q8_pd(zds_dtype pdt, zds_state_format f, bool vec, const AdamQ8Args &a, hipStream_t s) {
  if (!a.out) q8_vf<GD, -1>(f, vec, a, s);
  else if (pdt == ZDS_BF16) q8_vf<GD, ZDS_BF16>(f, vec, a, s);
  else q8_vf<GD, ZDS_FP16>(f, vec, a, s);
}

}  // namespace zds

using namespace zds;

extern "C" zds_status zds_adam_step_q8(const zds_adamw_hparams *hp, const void *grads, zds_dtype grad_dtype,
                                       float *master, void *exp_avg, uint8_t *exp_avg_exps, void *exp_avg_sq,
                                       zds_state_format sq_format, uint8_t *exp_avg_sq_exps, void *params_out,
                                       zds_dtype param_dtype, int64_t n, uint64_t seed, int64_t first,
                                       zds_step_scalars *scalars_dev, const zds_step_state *state_dev, void *stream) {
  clear_error();
  const char *fn = "zds_adam_step_q8";
  zds_status st = check_adamw(fn, hp);
  if (st != ZDS_OK) return st;
  if (!valid_dtype(grad_dtype)) return fail(ZDS_EINVAL, "%s: bad grad dtype", fn);
  if (params_out && param_dtype != ZDS_FP16 && param_dtype != ZDS_BF16)
    return fail(ZDS_EINVAL, "%s: param dtype must be fp16 or bf16", fn);
  if (sq_format != ZDS_STATE_UE5M3 && sq_format != ZDS_STATE_BF16)
    return fail(ZDS_EINVAL, "%s: the second moment's format must be UE5M3 or BF16", fn);
  if (n < 0 || n >= kStateMost) return fail(ZDS_EINVAL, "%s: n must lie in [0, 2^40)", fn);
  if (first < 0 || first % 32 != 0) return fail(ZDS_EINVAL, "%s: first must be a multiple of 32, >= 0", fn);
  if (n == 0) return ZDS_OK;
  const bool wide = sq_format == ZDS_STATE_BF16;
  if (!grads || !master || !exp_avg || !exp_avg_exps || !exp_avg_sq || (!wide && !exp_avg_sq_exps) || !scalars_dev ||
      !state_dev)
    return fail(ZDS_EINVAL, "%s: null pointer", fn);
  if (wide && exp_avg_sq_exps) return fail(ZDS_EINVAL, "%s: a BF16 second moment takes no exps", fn);
  if (!aligned(grads, static_cast<uintptr_t>(dtype_size(grad_dtype))) || !aligned(master, 4) ||
      (wide && !aligned(exp_avg_sq, 2)) || (params_out && !aligned(params_out, 2)) || !aligned(scalars_dev, 8) ||
      !aligned(state_dev, 8))
    return fail(ZDS_EALIGN, "%s: pointer not aligned to its element size", fn);
  const int64_t blocks = (n + 31) / 32;
  const struct {
    const void *p;
    int64_t bytes;
  } arrays[] = {{grads, n * dtype_size(grad_dtype)}, {params_out, params_out ? n * 2 : 0}, {master, n * 4},
                {exp_avg, n},                        {exp_avg_exps, blocks},              {exp_avg_sq, wide ? 2 * n : n},
                {exp_avg_sq_exps, wide ? 0 : blocks}};
  for (int i = 0; i < 7; ++i) {
    for (int j = 0; j < i; ++j) {
      if (i == 1 && params_out == grads && grad_dtype != ZDS_FP32) continue;
      if (ranges_meet(arrays[i].p, arrays[i].bytes, arrays[j].p, arrays[j].bytes))
        return fail(ZDS_EINVAL, "%s: two of the arrays overlap", fn);
    }
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  st = launch_adam_constants(*hp, state_dev, scalars_dev, s);
  if (st != ZDS_OK) return st;
  const AdamQ8Args a{scalars_dev, state_dev,       grads,      master, exp_avg, exp_avg_exps,
                     exp_avg_sq,  exp_avg_sq_exps, params_out, n,      seed,    first};
  const bool vec = aligned(grads, grad_dtype == ZDS_FP32 ? 16 : 8) && aligned(master, 16) && aligned(exp_avg, 4) &&
                   aligned(exp_avg_sq, wide ? 8 : 4) && (!params_out || aligned(params_out, 8));
  switch (grad_dtype) {
    case ZDS_FP16: q8_pd<ZDS_FP16>(param_dtype, sq_format, vec, a, s); break;
    case ZDS_BF16: q8_pd<ZDS_BF16>(param_dtype, sq_format, vec, a, s); break;
    default: q8_pd<ZDS_FP32>(param_dtype, sq_format, vec, a, s); break;
  }
  return check_launch("adam_step_q8 kernel");
}
