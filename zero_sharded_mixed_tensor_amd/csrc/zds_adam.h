// What AdamW's update kernels share: their scalars, the update of an element and
// the scheduling of their waves.
#pragma once

#include "zds_device.h"
#include "zds_internal.h"

namespace zds {

struct ElemConsts {
  float b1, b2, omb1, omb2, eps, step_size, decay, gs;
  double inv_bc2;
};

// 1 - beta is formed here in fp32, as the step's definition does (one fp32
// subtraction; exact for beta in [0.5, 1]).
__device__ __forceinline__ ElemConsts load_consts(const zds_step_scalars *sc) {
  ElemConsts c;
  c.b1 = sc->beta1;
  c.b2 = sc->beta2;
  c.eps = sc->eps;
  c.omb1 = 1.0f - c.b1;
  c.omb2 = 1.0f - c.b2;
  c.step_size = sc->step_size;
  c.inv_bc2 = sc->inv_bc2_sqrt;
  c.decay = sc->decay;
  c.gs = sc->grad_scale;
  return c;
}

// The step's constants into the scalars struct.
__device__ __forceinline__ void store_consts(const AdamConsts &c, zds_step_scalars *sc) {
  sc->inv_bc2_sqrt = c.inv_bc2_sqrt;
  sc->step_size = c.step_size;
  sc->bc2_sqrt = c.bc2_sqrt;
  sc->decay = c.decay;
  sc->beta1 = c.b1;
  sc->beta2 = c.b2;
  sc->eps = c.eps;
}

// One element, fp32, one rounding per operation, in this order: the moments, the
// denominator, the parameter (adam_elem does all three).
__device__ __forceinline__ void adam_moments(float x, const ElemConsts &c, float &m, float &v) {
  const float g = x * c.gs;
  m = c.b1 * m + c.omb1 * g;
  v = c.b2 * v + c.omb2 * (g * g);
}
// sqrt(v) / bc2 (bc2 = sqrt(1 - beta2^t) in fp32) is formed as
// fp32(float64(sqrt(v)) * r) with r = 1 / float64(bc2) correctly rounded.
// That is the correctly rounded fp32 quotient: r carries a relative error of
// at most 2^-53 and the float64 product another 2^-53, so the product is
// within 2^-52 (relatively) of the exact quotient; the exact quotient a/b of
// two fp32 numbers is never a point halfway between two fp32 numbers (a
// halfway point times b would need more than 24 significant bits), and lies at
// least 2^-49 (relatively) away from every such point, because
// |a - b*M| is a non-zero multiple of the coarser of a's and b*M's
// granularities. So no rounding boundary separates the product from the
// exact quotient. Here a = sqrt(v) is 0, NaN, inf or at least 2^-74.5, and
// the quotient stays in the normal range; bc2 = 0 (beta2 = 1) gives
// r = inf and the same inf / NaN as the division.
__device__ __forceinline__ float adam_denom(float v, const ElemConsts &c) {
  const float q = static_cast<float>(static_cast<double>(sqrtf(v)) * c.inv_bc2);
  return q + c.eps;
}
__device__ __forceinline__ void adam_param(float m, float denom, const ElemConsts &c, float &p) {
  p = p * c.decay;
  p = p - c.step_size * (m / denom);
}
__device__ __forceinline__ void adam_elem(float x, const ElemConsts &c, float &p, float &m, float &v) {
  adam_moments(x, c, m, v);
  adam_param(m, adam_denom(v, c), c, p);
}

// Scheduling priority of a wave: raised while it issues its loads and stores,
// lowered for the update.
__device__ __forceinline__ void memory_phase() { __builtin_amdgcn_s_setprio(3); }
__device__ __forceinline__ void update_phase() { __builtin_amdgcn_s_setprio(0); }

}  // namespace zds
