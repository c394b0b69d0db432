// Moments in fewer bits: quantising fp32 arrays and reading them back
// (include/zds.h describes the formats; zds_quantised.h has the arithmetic).
//
// Both are HBM-bound streams: 4 B read and a code (1 + 1/32 or 2 B) written
// per element, and the other way round. Quantising, a wave takes units of 512
// elements, each lane a quad of each half, so that a block of 32 lies in 8
// neighbouring lanes and its largest magnitude takes three cross-lane moves:
// 202M elements to 8 bits 155 us to nearest, 157 at random (6.5 TB/s, the rate of
// a copy), to BF16 183 (6.6).
#include "zds_internal.h"
#include "zds_quantised.h"

namespace zds {

struct ConvertArgs {
  const void *src;
  void *dst;
  uint8_t *exps;
  const uint8_t *exps_in;
  int64_t n;
  uint64_t seed;
  int64_t first;
  const zds_step_state *state;
};

// Unaligned or cut quads: element by element.
template <typename T>
__device__ __forceinline__ void load_elements(const T *p, int64_t e, int64_t n, T (&x)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = e + i < n ? p[e + i] : T(0);
}

template <int F, bool RANDOM, bool VEC>
__global__ void __launch_bounds__(256) quantise_kernel(ConvertArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t units = (a.n + kStateUnit - 1) / kStateUnit;
  const float *src = static_cast<const float *>(a.src);
  const uint32_t steps = RANDOM ? a.state->steps_seen : 0u;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6); u < units;
       u += static_cast<int64_t>(gridDim.x) * 4) {
    QuadBits rb{};
    if (RANDOM) rb = unit_random_bits(a.seed, static_cast<uint64_t>((a.first + u * kStateUnit) >> 3), steps, lane);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t e = u * kStateUnit + 256 * h + 4 * lane;
      const bool whole = e + 4 <= a.n;
      float x[4];
      if (VEC && whole) load_quad<ZDS_FP32>(src, e >> 2, x);
      else load_elements(src, e, a.n, x);
      const uint32_t (&w)[2] = h ? rb.r1 : rb.r0;
      if constexpr (F == ZDS_STATE_BF16) {
        const u32x2 c = encode_quad_bf16<RANDOM>(x, w);
        if (VEC && whole) {
          st_stream(static_cast<u32x2 *>(a.dst) + (e >> 2), c);
        } else {
          uint16_t *d = static_cast<uint16_t *>(a.dst);
          for (int i = 0; i < 4; ++i)
            if (e + i < a.n) d[e + i] = static_cast<uint16_t>((i < 2 ? c.x : c.y) >> (16 * (i & 1)));
        }
      } else {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = magnitude(x[i]) > m ? magnitude(x[i]) : m;
        m = block_max(m);
        const uint32_t s = exponent_byte<F>(m);
        const uint32_t c = encode_quad<F, RANDOM>(x, s, m, w);
        uint8_t *d = static_cast<uint8_t *>(a.dst);
        if (VEC && whole) {
          st_stream(reinterpret_cast<uint32_t *>(d + e), c);
        } else {
          for (int i = 0; i < 4; ++i)
            if (e + i < a.n) d[e + i] = static_cast<uint8_t>(c >> (8 * i));
        }
        if ((lane & 7) == 0 && e < a.n) a.exps[e >> 5] = static_cast<uint8_t>(s);
      }
    }
  }
}

// The value of element e.
template <int F>
__device__ __forceinline__ float read_element(const ConvertArgs &a, int64_t e) {
  if constexpr (F == ZDS_STATE_BF16) return widen1<ZDS_BF16>(a.src, e);
  else return decode1<F>(static_cast<const uint8_t *>(a.src)[e], a.exps_in[e >> 5]);
}
template <int D>
__device__ __forceinline__ void write_element(void *dst, int64_t e, float x) {
  if constexpr (D == ZDS_FP32) static_cast<float *>(dst)[e] = x;
  else static_cast<uint16_t *>(dst)[e] = narrow1<ZDS_BF16>(x);
}

// Reading back, a unit of 1024 elements a wave: the codes come in 16 bytes a
// lane and are used as what a lane stores 16 bytes of, through the wave's own
// LDS, and a wave has one store in flight. 842M elements of 8 bits to fp32 /
// bf16: 0.68 / 0.39 ms (6.25 / 6.5 TB/s); its stores back to back 0.73 / 0.39;
// with 4-byte loads of a quad's codes a lane 0.76 / 0.61. The wave that holds
// the last elements, if they are no whole unit, reads them one by one.
constexpr int kReadUnit = 1024;
template <int F, int D>
__global__ void __launch_bounds__(256) read_back_kernel(ConvertArgs a) {
  constexpr bool WIDE = F == ZDS_STATE_BF16;
  __shared__ u32x4 codes[4][WIDE ? 128 : 64];
  __shared__ uint8_t exps[4][32];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * 4 + w) * kReadUnit;
  if (first + kReadUnit > a.n) {
    for (int64_t e = first + lane; e < a.n; e += 64) write_element<D>(a.dst, e, read_element<F>(a, e));
    return;
  }
  const u32x4 *src = reinterpret_cast<const u32x4 *>(static_cast<const uint8_t *>(a.src) + (WIDE ? 2 * first : first));
  u32x4 *sc = codes[w];
  uint8_t *se = exps[w];
  uint32_t eb = 0;
  if (!WIDE && lane < 32) eb = a.exps_in[(first >> 5) + lane];
  const u32x4 c0 = ld_stream_global(src + lane);
  u32x4 c1{};
  if (WIDE) c1 = ld_stream_global(src + 64 + lane);
  sc[lane] = c0;
  if (WIDE) sc[64 + lane] = c1;
  else if (lane < 32) se[lane] = static_cast<uint8_t>(eb);
  __builtin_amdgcn_wave_barrier();
  if constexpr (D == ZDS_FP32) {
    float *dst = static_cast<float *>(a.dst) + first;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const int k = 64 * h + lane;
      float x[4];
      if constexpr (WIDE) {
        const u32x2 q = reinterpret_cast<const u32x2 *>(sc)[k];
        x[0] = bf16_lo(q.x); x[1] = bf16_hi(q.x); x[2] = bf16_lo(q.y); x[3] = bf16_hi(q.y);
      } else {
        decode_quad<F>(reinterpret_cast<const uint32_t *>(sc)[k], se[k >> 3], x);
      }
      if (h > 0) wait_vmem();
      st_stream_at(dst, 16 * k, f32x4{x[0], x[1], x[2], x[3]});
    }
  } else {
    uint16_t *dst = static_cast<uint16_t *>(a.dst) + first;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = 64 * h + lane;
      if (h > 0) wait_vmem();
      if constexpr (WIDE) {
        st_stream_at(dst, 16 * k, sc[k]);
      } else {
        const u32x2 q = reinterpret_cast<const u32x2 *>(sc)[k];
        const uint32_t s = se[k >> 2];
        float x[4], y[4];
        decode_quad<F>(q.x, s, x);
        decode_quad<F>(q.y, s, y);
        st_stream_at(dst, 16 * k, u32x4{pack2<ZDS_BF16>(x[0], x[1]), pack2<ZDS_BF16>(x[2], x[3]),
                                        pack2<ZDS_BF16>(y[0], y[1]), pack2<ZDS_BF16>(y[2], y[3])});
      }
    }
  }
}

// Arrays without the units' alignment.
template <int F, int D>
__global__ void __launch_bounds__(256) read_back_element_kernel(ConvertArgs a) {
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; e < a.n;
       e += static_cast<int64_t>(gridDim.x) * 256)
    write_element<D>(a.dst, e, read_element<F>(a, e));
}

template <int F, bool RANDOM>
static void quantise_go(bool vec, const ConvertArgs &a, hipStream_t s) {
  int64_t g = (a.n + 4 * kStateUnit - 1) / (4 * kStateUnit);
  if (g > max_blocks(256)) g = max_blocks(256);
  if (vec) hipLaunchKernelGGL((quantise_kernel<F, RANDOM, true>), dim3(static_cast<uint32_t>(g)), dim3(256), 0, s, a);
  else hipLaunchKernelGGL((quantise_kernel<F, RANDOM, false>), dim3(static_cast<uint32_t>(g)), dim3(256), 0, s, a);
}

template <int F, int D>
static void dequantise_go(bool vec, const ConvertArgs &a, hipStream_t s) {
  if (!vec) {
    int64_t g = (a.n + 255) / 256;
    if (g > max_blocks(256)) g = max_blocks(256);
    hipLaunchKernelGGL((read_back_element_kernel<F, D>), dim3(static_cast<uint32_t>(g)), dim3(256), 0, s, a);
    return;
  }
  // units of one launch: a dispatch holds fewer than 2^32 work-items
  constexpr int64_t most = max_blocks(256) * 4 * kReadUnit;
  for (int64_t at = 0; at < a.n; at += most) {
    ConvertArgs b = a;
    b.src = static_cast<const uint8_t *>(a.src) + (F == ZDS_STATE_BF16 ? 2 * at : at);
    if (F != ZDS_STATE_BF16) b.exps_in = a.exps_in + (at >> 5);
    b.dst = static_cast<uint8_t *>(a.dst) + (D == ZDS_FP32 ? 4 : 2) * at;
    b.n = a.n - at < most ? a.n - at : most;
    hipLaunchKernelGGL((read_back_kernel<F, D>), dim3(static_cast<uint32_t>((b.n + 4 * kReadUnit - 1) / (4 * kReadUnit))),
                       dim3(256), 0, s, b);
  }
}

static bool valid_format(int f) { return f == ZDS_STATE_E4M3 || f == ZDS_STATE_UE5M3 || f == ZDS_STATE_BF16; }
static int64_t code_size(zds_state_format f) { return f == ZDS_STATE_BF16 ? 2 : 1; }

// What both conversions check; plain_size: bytes per element of the array that is no code.
static zds_status check_convert(const char *fn, const void *codes, const void *exps, int64_t n, zds_state_format f,
                                const void *plain, int64_t plain_size) {
  if (!codes || !plain) return fail(ZDS_EINVAL, "%s: null pointer", fn);
  if ((f == ZDS_STATE_BF16) != (exps == nullptr))
    return fail(ZDS_EINVAL, f == ZDS_STATE_BF16 ? "%s: BF16 takes no exps" : "%s: null exps", fn);
  if (!aligned(plain, static_cast<uintptr_t>(plain_size)) || !aligned(codes, static_cast<uintptr_t>(code_size(f))))
    return fail(ZDS_EALIGN, "%s: pointer not aligned to its element size", fn);
  const int64_t nb = (n + 31) / 32, cb = n * code_size(f), pb = n * plain_size;
  if (ranges_meet(codes, cb, plain, pb) ||
      (exps && (ranges_meet(exps, nb, codes, cb) || ranges_meet(exps, nb, plain, pb))))
    return fail(ZDS_EINVAL, "%s: the arrays overlap", fn);
  return ZDS_OK;
}

}  // namespace zds

using namespace zds;

extern "C" zds_status zds_random_words_host(uint64_t seed, uint64_t call, uint32_t steps_seen, uint32_t stream,
                                            uint32_t *out4) {
  clear_error();
  if (!out4) return fail(ZDS_EINVAL, "zds_random_words_host: null output");
  const RandomWords q = random_words(seed, call, steps_seen, stream);
  for (int i = 0; i < 4; ++i) out4[i] = q.w[i];
  return ZDS_OK;
}

extern "C" zds_status zds_state_quantise(const float *src, int64_t n, zds_state_format format, zds_rounding rounding,
                                         uint64_t seed, int64_t first, const zds_step_state *state_dev, void *codes,
                                         uint8_t *exps, void *stream) {
  clear_error();
  const char *fn = "zds_state_quantise";
  if (!valid_format(format)) return fail(ZDS_EINVAL, "%s: bad format", fn);
  if (rounding != ZDS_ROUND_NEAREST && rounding != ZDS_ROUND_RANDOM) return fail(ZDS_EINVAL, "%s: bad rounding", fn);
  if (n < 0 || n >= kStateMost) return fail(ZDS_EINVAL, "%s: n must lie in [0, 2^40)", fn);
  const bool random = rounding == ZDS_ROUND_RANDOM;
  if (random && (first < 0 || first % 32 != 0 || first > INT64_MAX - n))
    return fail(ZDS_EINVAL, "%s: first must be a multiple of 32 in [0, 2^63 - n)", fn);
  if (n == 0) return ZDS_OK;
  if (random && !state_dev) return fail(ZDS_EINVAL, "%s: null state", fn);
  if (random && !aligned(state_dev, 8)) return fail(ZDS_EALIGN, "%s: state not 8-byte aligned", fn);
  const zds_status st = check_convert(fn, codes, exps, n, format, src, 4);
  if (st != ZDS_OK) return st;
  const ConvertArgs a{src, codes, exps, nullptr, n, seed, random ? first : 0, state_dev};
  const bool vec = aligned(src, 16) && aligned(codes, format == ZDS_STATE_BF16 ? 8 : 4);
  hipStream_t s = static_cast<hipStream_t>(stream);
  switch (format) {
    case ZDS_STATE_E4M3: random ? quantise_go<ZDS_STATE_E4M3, true>(vec, a, s) : quantise_go<ZDS_STATE_E4M3, false>(vec, a, s); break;
    case ZDS_STATE_UE5M3: random ? quantise_go<ZDS_STATE_UE5M3, true>(vec, a, s) : quantise_go<ZDS_STATE_UE5M3, false>(vec, a, s); break;
    default: random ? quantise_go<ZDS_STATE_BF16, true>(vec, a, s) : quantise_go<ZDS_STATE_BF16, false>(vec, a, s); break;
  }
  return check_launch("state_quantise kernel");
}

extern "C" zds_status zds_state_dequantise(const void *codes, const uint8_t *exps, int64_t n, zds_state_format format,
                                           void *dst, zds_dtype dst_dtype, void *stream) {
  clear_error();
  const char *fn = "zds_state_dequantise";
  if (!valid_format(format)) return fail(ZDS_EINVAL, "%s: bad format", fn);
  if (dst_dtype != ZDS_FP32 && dst_dtype != ZDS_BF16) return fail(ZDS_EINVAL, "%s: dst dtype must be bf16 or fp32", fn);
  if (n < 0 || n >= kStateMost) return fail(ZDS_EINVAL, "%s: n must lie in [0, 2^40)", fn);
  if (n == 0) return ZDS_OK;
  const zds_status st = check_convert(fn, codes, exps, n, format, dst, dtype_size(dst_dtype));
  if (st != ZDS_OK) return st;
  const ConvertArgs a{codes, dst, nullptr, exps, n, 0, 0, nullptr};
  const bool f = dst_dtype == ZDS_FP32;
  const bool vec = aligned(dst, 16) && aligned(codes, 16);
  hipStream_t s = static_cast<hipStream_t>(stream);
  switch (format) {
    case ZDS_STATE_E4M3: f ? dequantise_go<ZDS_STATE_E4M3, ZDS_FP32>(vec, a, s) : dequantise_go<ZDS_STATE_E4M3, ZDS_BF16>(vec, a, s); break;
    case ZDS_STATE_UE5M3: f ? dequantise_go<ZDS_STATE_UE5M3, ZDS_FP32>(vec, a, s) : dequantise_go<ZDS_STATE_UE5M3, ZDS_BF16>(vec, a, s); break;
    default: f ? dequantise_go<ZDS_STATE_BF16, ZDS_FP32>(vec, a, s) : dequantise_go<ZDS_STATE_BF16, ZDS_BF16>(vec, a, s); break;
  }
  return check_launch("state_dequantise kernel");
}
