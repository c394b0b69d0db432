// The scalars of AdamW's update kernels and the scheduling of their waves.
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

// Scheduling priority of a wave: raised while it issues its loads and stores,
// lowered for the update.
__device__ __forceinline__ void memory_phase() { __builtin_amdgcn_s_setprio(3); }
__device__ __forceinline__ void update_phase() { __builtin_amdgcn_s_setprio(0); }

}  // namespace zds
