// AdamW on moments in fewer bits: zds_adam_step's update on a first moment in
// E4M3 and a second one in UE5M3 or BF16, read back and quantised again at
// random (include/zds.h; zds_quantised.h has the formats' arithmetic).
//
// A stream of 16.1 B an element (16-bit grads; 18.1 with a BF16 second moment)
// and about 65 VALU instructions an element, 6 of them the generator's and 20 the
// correctly rounded root and quotient: on 842M elements 2.06 ms of memory at the
// rate of a copy and 1.8 of all SIMDs, so what counts is that the one hides the
// other. A block of 8 waves takes a tile of 2048 elements; the waves fetch it 16
// bytes a lane, one access in flight each, the master's quads straight into the
// registers of the thread that updates them, grads and codes through LDS; four of
// the waves make the generator's calls meanwhile; the results go out the same way.
// 842M elements, bf16: 2.19 ms (6.2 TB/s). The hardware's root and reciprocal, 16
// instructions fewer, take 2.15, but then master is no longer zds_adam_step's.
// Layouts, timed with those (2.13 then): each lane moving its own quad of every
// array (4-byte accesses to the codes) 2.36, of which the arithmetic was not the
// cause (2.48 without it); a wave's own 1024 elements through its own LDS, no
// barriers 2.24; tiles of 4096 in two pipelined halves, as the fp32 step's, 2.28 to
// 2.39; tiles of 1024 with one access a wave 2.73.
#include "zds_adam.h"
#include "zds_quantised.h"

namespace zds {

struct AdamQ8Args {
  zds_step_scalars *sc;
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
  int64_t tile0;  // the launch's first tile
  zds_adamw_hparams hp;
};

// The step's constants, formed here from the hyperparameters and the step state,
// and by one thread written where a launch in front would have left them. (No
// block of this kernel reads those fields.)
__device__ __forceinline__ ElemConsts derive_consts(const AdamQ8Args &a, bool store) {
  const AdamConsts k = adam_constants(a.hp, a.state->beta1_pow, a.state->beta2_pow);
  if (store) store_consts(k, a.sc);
  return ElemConsts{k.b1, k.b2, k.omb1, k.omb2, k.eps, k.step_size, k.decay, a.sc->grad_scale, k.inv_bc2_sqrt};
}

// sqrt(v) / bc2 + eps as adam_denom has it, for v of 0 or from 2^-149 to 2^63, with
// a shorter root: v enters times 2^64, so that no step of it underflows, and the
// root's 2^32 leaves in the product with 1 / bc2, in fp64. One Newton step from the
// hardware's reciprocal root, the residual in one rounding, is correctly rounded
// for each of the 1.78e9 fp32 numbers from 2^-85 to 2^127 (compared with sqrtf one
// by one); 0 stays 0, as the reciprocal root is that of 2^-90 then. 6 instructions
// and the reciprocal root, where sqrtf, which has to serve every number, takes 15
// and the root: 842M elements 2.19 ms, with sqrtf 2.27.
constexpr uint32_t kRootMost = 0x5f000000u;  // the bits of 2^63
__device__ __forceinline__ float adam_denom_in_range(float v, const ElemConsts &c) {
  const float x = v * 0x1p64f;
  const float y = __builtin_amdgcn_rsqf(__builtin_fmaxf(x, 0x1p-90f));
  const float s = x * y;
  const float root = __builtin_fmaf(__builtin_fmaf(-s, s, x), 0.5f * y, s);
  const float q = static_cast<float>(static_cast<double>(root) * (c.inv_bc2 * 0x1p-32));
  return q + c.eps;
}

// One element on each lane, the block of 32 that shares an exponent in half a
// wave: what is not a whole tile, and arrays without the tiles' alignment. All
// lanes of a wave call it; e is past the end on some.
template <int GD, int PD, int VF>
__device__ __forceinline__ void q8_element(const AdamQ8Args &a, const ElemConsts &c, int64_t e, uint32_t steps) {
  const bool in = e < a.n;
  uint8_t *mc = static_cast<uint8_t *>(a.m);
  uint8_t *vc = static_cast<uint8_t *>(a.v);
  uint16_t *v16 = static_cast<uint16_t *>(a.v);
  float p = 0.0f, m = 0.0f, v = 0.0f;
  if (in) {
    p = a.p[e];
    m = decode1<ZDS_STATE_E4M3>(mc[e], a.me[e >> 5]);
    if constexpr (VF == ZDS_STATE_BF16) v = __uint_as_float(static_cast<uint32_t>(v16[e]) << 16);
    else v = decode1<VF>(vc[e], a.ve[e >> 5]);
    adam_elem(widen1<GD>(a.g, e), c, p, m, v);
  }
  const uint32_t r = element_random_bits(a.seed, static_cast<uint64_t>(a.first + e), steps);
  const uint32_t rs = swap_bytes(r);
  const uint32_t ms = exponent_byte<ZDS_STATE_E4M3>(block_max_lanes(magnitude(m)));
  const uint32_t mcode = encode1<ZDS_STATE_E4M3, true>(m, ms, r);
  uint32_t vs = 0, vcode;
  if constexpr (VF == ZDS_STATE_BF16) {
    vcode = encode_bf16<true>(v, rs);
  } else {
    vs = exponent_byte<VF>(block_max_lanes(magnitude(v)));
    vcode = encode1<VF, true>(v, vs, rs);
  }
  if (!in) return;
  a.p[e] = p;
  if constexpr (PD >= 0) static_cast<uint16_t *>(a.out)[e] = narrow1<PD>(p);
  mc[e] = static_cast<uint8_t>(mcode);
  if constexpr (VF == ZDS_STATE_BF16) v16[e] = static_cast<uint16_t>(vcode);
  else vc[e] = static_cast<uint8_t>(vcode);
  if ((threadIdx.x & 31) == 0) {
    a.me[e >> 5] = static_cast<uint8_t>(ms);
    if constexpr (VF != ZDS_STATE_BF16) a.ve[e >> 5] = static_cast<uint8_t>(vs);
  }
}

// Elements of a tile: one quad for each thread of a block.
constexpr int kQ8Block = 512;
constexpr int kQ8Tile = 4 * kQ8Block;

// What the waves of a block hand each other: what they move 16 bytes a lane
// and use a quad a lane, and the generator's calls (one for 8 elements).
template <int VF>
struct Q8Tile {
  u32x4 io[256];  // 16-bit grads in, 16-bit params out
  u32x4 m[128];   // codes, in and out
  u32x4 v[VF == ZDS_STATE_BF16 ? 256 : 128];
  u32x4 random[256];
  uint8_t me[64], ve[64];
  ElemConsts consts;
};

// Up to this many elements the blocks form the step's constants themselves, by
// one wave while the loads are in flight, instead of a launch in front of them:
// a call of 1M elements takes 6.8 us in a graph instead of 7.5 (and 10 us on the
// host instead of 13), of 2M 9.0 and 9.2; of 4M 16.7 and 15.3, of 8M 28.9 and
// 25.5, as every block pays for the divisions.
constexpr int64_t kQ8OwnConsts = int64_t(1) << 21;

// One tile a block, and a last block for the elements behind the last whole
// tile. PD: the params' type, -1 for none. OWN: the constants are formed here.
template <int GD, int PD, int VF, bool OWN>
__global__ void __launch_bounds__(kQ8Block, 8) adam_q8_tile_kernel(AdamQ8Args a) {
  __shared__ Q8Tile<VF> sh;
  constexpr bool WIDE = VF == ZDS_STATE_BF16;
  if (a.sc->overflow) {  // the step is skipped: uniform, nothing else is touched
    if (OWN && blockIdx.x == 0 && threadIdx.x == 0) derive_consts(a, true);
    return;
  }
  ElemConsts c;
  if (!OWN) c = load_consts(a.sc);
  const uint32_t steps = a.state->steps_seen;
  const int t = threadIdx.x, lane = t & 63;
  const int64_t first = (a.tile0 + blockIdx.x) * kQ8Tile;
  if (first + kQ8Tile > a.n) {
    if (OWN) c = derive_consts(a, blockIdx.x == 0 && t == 0);
    for (int64_t e = first + t; e < ((a.n + 63) & ~int64_t(63)); e += kQ8Block) q8_element<GD, PD, VF>(a, c, e, steps);
    return;
  }
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);
  uint16_t *gp = static_cast<uint16_t *>(const_cast<void *>(a.g)) + first;
  uint8_t *mp = static_cast<uint8_t *>(a.m) + first;
  uint8_t *vp = static_cast<uint8_t *>(a.v) + (WIDE ? 2 * first : first);
  float *pp = a.p + first;
  // The pieces that this wave moves: 16-bit grads (and params) by waves 0-3;
  // 8-bit codes of m by waves 4-5 and of v by waves 6-7; a 16-bit v by waves
  // 4-7, and then m by waves 2-3.
  const bool has_g = GD != ZDS_FP32 && w < 4, has_o = PD >= 0 && w < 4;
  const bool has_m = WIDE ? w == 2 || w == 3 : w == 4 || w == 5;
  const bool has_v = WIDE ? w >= 4 : w >= 6;
  const uint32_t at_m = 16 * (t - (WIDE ? 128 : 256)), at_v = 16 * (t - (WIDE ? 256 : 384));
  memory_phase();
  u32x4 x0{}, x1{};
  uint32_t eb = 0;
  if (has_g) x0 = ld_stream_global(reinterpret_cast<const u32x4 *>(gp) + t);
  if (has_m) x1 = ld_stream_global(reinterpret_cast<const u32x4 *>(mp + at_m));
  if (has_v) x0 = ld_stream_global(reinterpret_cast<const u32x4 *>(vp + at_v));
  if (w == 4) eb = a.me[(first >> 5) + lane];
  if (!WIDE && w == 6) eb = a.ve[(first >> 5) + lane];
  wait_vmem();
  const f32x4 p4 = ld_stream_global(reinterpret_cast<const f32x4 *>(pp) + t);
  f32x4 g4{};
  if (GD == ZDS_FP32) g4 = ld_stream_global(reinterpret_cast<const f32x4 *>(static_cast<const float *>(a.g) + first) + t);
  update_phase();
  if (w < 4) {
    const RandomWords q = random_words(a.seed, static_cast<uint64_t>((a.first + first) >> 3) + t, steps, kStreamRounding);
    sh.random[t] = u32x4{q.w[0], q.w[1], q.w[2], q.w[3]};
  }
  if (OWN && w == 7) {
    const ElemConsts d = derive_consts(a, blockIdx.x == 0 && lane == 0);
    if (lane == 0) sh.consts = d;
  }
  uint8_t *sm = reinterpret_cast<uint8_t *>(sh.m), *sv = reinterpret_cast<uint8_t *>(sh.v);
  if (has_g) sh.io[t] = x0;
  if (has_m) *reinterpret_cast<u32x4 *>(sm + at_m) = x1;
  if (has_v) *reinterpret_cast<u32x4 *>(sv + at_v) = x0;
  if (w == 4) sh.me[lane] = static_cast<uint8_t>(eb);
  if (!WIDE && w == 6) sh.ve[lane] = static_cast<uint8_t>(eb);
  __syncthreads();
  if (OWN) {
    const auto uniform = [](float x) { return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(x))); };
    const ElemConsts d = sh.consts;
    const int lo = __builtin_amdgcn_readfirstlane(__double2loint(d.inv_bc2)),
              hi = __builtin_amdgcn_readfirstlane(__double2hiint(d.inv_bc2));
    c = ElemConsts{uniform(d.b1),  uniform(d.b2),        uniform(d.omb1),  uniform(d.omb2),
                   uniform(d.eps), uniform(d.step_size), uniform(d.decay), a.sc->grad_scale,
                   __hiloint2double(hi, lo)};
  }
  float g[4], p[4] = {p4.x, p4.y, p4.z, p4.w}, m[4], v[4];
  u32x2 *io2 = reinterpret_cast<u32x2 *>(sh.io);
  if constexpr (GD == ZDS_FP32) {
    g[0] = g4.x; g[1] = g4.y; g[2] = g4.z; g[3] = g4.w;
  } else {
    const u32x2 q = io2[t];
    g[0] = lo_of<GD>(q.x); g[1] = hi_of<GD>(q.x); g[2] = lo_of<GD>(q.y); g[3] = hi_of<GD>(q.y);
  }
  uint32_t *sm1 = reinterpret_cast<uint32_t *>(sh.m), *sv1 = reinterpret_cast<uint32_t *>(sh.v);
  u32x2 *sv2 = reinterpret_cast<u32x2 *>(sh.v);
  decode_quad<ZDS_STATE_E4M3>(sm1[t], sh.me[t >> 3], m);
  if constexpr (WIDE) {
    const u32x2 q = sv2[t];
    v[0] = bf16_lo(q.x); v[1] = bf16_hi(q.x); v[2] = bf16_lo(q.y); v[3] = bf16_hi(q.y);
  } else {
    decode_quad<VF>(sv1[t], sh.ve[t >> 3], v);
  }
  uint32_t mm = 0, vm = 0, vb = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    adam_moments(g[i], c, m[i], v[i]);
    mm = magnitude(m[i]) > mm ? magnitude(m[i]) : mm;
    vm = magnitude(v[i]) > vm ? magnitude(v[i]) : vm;
    vb = __float_as_uint(v[i]) > vb ? __float_as_uint(v[i]) : vb;
  }
  // (a BF16 state may hold negative numbers, whose bits are the larger ones)
  const bool in_range = (WIDE ? vb : vm) < kRootMost;
  float denom[4];
  if (in_range) {
#pragma unroll
    for (int i = 0; i < 4; ++i) denom[i] = adam_denom_in_range(v[i], c);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) denom[i] = adam_denom(v[i], c);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) adam_param(m[i], denom[i], c, p[i]);
  st_stream_at(pp, 16 * t, f32x4{p[0], p[1], p[2], p[3]});
  const u32x2 rr = reinterpret_cast<const u32x2 *>(sh.random)[t];
  const uint32_t rw[2] = {rr.x, rr.y};
  mm = block_max(mm);
  const uint32_t ms = exponent_byte<ZDS_STATE_E4M3>(mm);
  sm1[t] = encode_quad<ZDS_STATE_E4M3, true>(m, ms, mm, rw);
  if ((lane & 7) == 0) sh.me[t >> 3] = static_cast<uint8_t>(ms);
  if constexpr (WIDE) {
    sv2[t] = encode_quad_bf16<true>(v, rw);
  } else {
    vm = block_max(vm);
    const uint32_t vs = exponent_byte<VF>(vm);
    sv1[t] = encode_quad<VF, true, true>(v, vs, vm, rw);
    if ((lane & 7) == 0) sh.ve[t >> 3] = static_cast<uint8_t>(vs);
  }
  if constexpr (PD >= 0) io2[t] = u32x2{pack2<PD>(p[0], p[1]), pack2<PD>(p[2], p[3])};
  __syncthreads();
  memory_phase();
  wait_vmem();
  if (has_o) st_stream_at(static_cast<uint16_t *>(a.out) + first, 16 * t, sh.io[t]);
  if (has_m) st_stream_at(mp, at_m, *reinterpret_cast<u32x4 *>(sm + at_m));
  if (has_v) st_stream_at(vp, at_v, *reinterpret_cast<u32x4 *>(sv + at_v));
  if (w == 4) a.me[(first >> 5) + lane] = sh.me[lane];
  if (!WIDE && w == 6) a.ve[(first >> 5) + lane] = sh.ve[lane];
}

// Element by element.
template <int GD, int PD, int VF>
__global__ void __launch_bounds__(256) adam_q8_element_kernel(AdamQ8Args a) {
  if (a.sc->overflow) return;
  const ElemConsts c = load_consts(a.sc);
  const uint32_t steps = a.state->steps_seen;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; e < ((a.n + 63) & ~int64_t(63));
       e += static_cast<int64_t>(gridDim.x) * 256)
    q8_element<GD, PD, VF>(a, c, e, steps);
}

template <int GD, int PD, int VF>
static void q8_go(bool vec, const AdamQ8Args &a, hipStream_t s) {
  if (!vec) {
    int64_t g = (a.n + 255) / 256;
    if (g > max_blocks(256)) g = max_blocks(256);
    hipLaunchKernelGGL((adam_q8_element_kernel<GD, PD, VF>), dim3(static_cast<uint32_t>(g)), dim3(256), 0, s, a);
    return;
  }
  if (a.n <= kQ8OwnConsts) {
    hipLaunchKernelGGL((adam_q8_tile_kernel<GD, PD, VF, true>), dim3(static_cast<uint32_t>((a.n + kQ8Tile - 1) / kQ8Tile)),
                       dim3(kQ8Block), 0, s, a);
    return;
  }
  AdamQ8Args b = a;
  const int64_t tiles = (a.n + kQ8Tile - 1) / kQ8Tile;
  for (b.tile0 = 0; b.tile0 < tiles; b.tile0 += max_blocks(kQ8Block)) {  // one launch below 2^34 elements
    const int64_t left = tiles - b.tile0;
    hipLaunchKernelGGL((adam_q8_tile_kernel<GD, PD, VF, false>),
                       dim3(static_cast<uint32_t>(left < max_blocks(kQ8Block) ? left : max_blocks(kQ8Block))),
                       dim3(kQ8Block), 0, s, b);
  }
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
  if (hp->eps < 0x1p-100f) return fail(ZDS_EINVAL, "%s: eps must be 2^-100 or more", fn);
  if (!valid_dtype(grad_dtype)) return fail(ZDS_EINVAL, "%s: bad grad dtype", fn);
  if (params_out && param_dtype != ZDS_FP16 && param_dtype != ZDS_BF16)
    return fail(ZDS_EINVAL, "%s: param dtype must be fp16 or bf16", fn);
  if (sq_format != ZDS_STATE_UE5M3 && sq_format != ZDS_STATE_BF16)
    return fail(ZDS_EINVAL, "%s: the second moment's format must be UE5M3 or BF16", fn);
  if (n < 0 || n >= kStateMost) return fail(ZDS_EINVAL, "%s: n must lie in [0, 2^40)", fn);
  if (first < 0 || first % 32 != 0 || first > INT64_MAX - n)
    return fail(ZDS_EINVAL, "%s: first must be a multiple of 32 in [0, 2^63 - n)", fn);
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
  const AdamQ8Args a{scalars_dev, state_dev,       grads,      master, exp_avg, exp_avg_exps,
                     exp_avg_sq,  exp_avg_sq_exps, params_out, n,      seed,    first,        0, *hp};
  const bool vec = aligned(grads, 16) && aligned(master, 16) && aligned(exp_avg, 16) && aligned(exp_avg_sq, 16) &&
                   (!params_out || aligned(params_out, 16));
  if (!vec || n > kQ8OwnConsts) {
    st = launch_adam_constants(*hp, state_dev, scalars_dev, s);
    if (st != ZDS_OK) return st;
  }
  switch (grad_dtype) {
    case ZDS_FP16: q8_pd<ZDS_FP16>(param_dtype, sq_format, vec, a, s); break;
    case ZDS_BF16: q8_pd<ZDS_BF16>(param_dtype, sq_format, vec, a, s); break;
    default: q8_pd<ZDS_FP32>(param_dtype, sq_format, vec, a, s); break;
  }
  return check_launch("adam_step_q8 kernel");
}
