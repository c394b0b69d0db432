// Gradient dropout: the two ends of an exchange in which every group of
// `ratio` consecutive elements sends one, chosen by the counter-based
// generator (include/zds.h has the definition, zds_random.h the generator).
//
// Every kernel works on tiles: a block first makes the kept places of the
// tile's groups in LDS (one generator call covers 16 groups), then streams.
#include "zds_internal.h"
#include "zds_quantised.h"

namespace zds {

// Elements of a tile of the kernels that walk a gradient, and groups of a tile
// of those that walk a message.
constexpr int kDropTile = 4096;
constexpr int kDropGroups = 4096;

struct DropArgs {
  const void *x;
  float *err;
  void *values;
  const void *peers[kMaxPeers];
  void *dst;
  int64_t n, groups;
  int64_t j0;        // generator index of local group 0
  uint64_t seed;
  int32_t shift;     // log2(ratio)
  int32_t npeers;
  const zds_step_scalars *sc;
  const zds_step_state *state;
};

// The kept places of local groups g .. g + count - 1, as the generator's bytes:
// group g + k has its byte at kept[k + (returned offset)]. kept holds count +
// 31 bytes, 16-byte aligned. All threads of the block call it; it ends with a
// barrier.
__device__ __forceinline__ int make_kept(const DropArgs &a, int64_t g, int count, uint8_t *kept) {
  const int64_t j = a.j0 + g;
  const int off = static_cast<int>(j & 15);
  const int calls = (off + count + 15) >> 4;
  const uint32_t steps = a.state->steps_seen;
  for (int k = threadIdx.x; k < calls; k += blockDim.x) {
    const RandomWords q = random_words(a.seed, static_cast<uint64_t>((j >> 4) + k), steps, kStreamDropout);
    *reinterpret_cast<u32x4 *>(kept + 16 * k) = u32x4{q.w[0], q.w[1], q.w[2], q.w[3]};
  }
  __syncthreads();
  return off;
}

// fp32 -> a value of type D at index i; returns what was stored, widened.
template <int D>
__device__ __forceinline__ float put(void *base, int64_t i, float x) {
  if constexpr (D == ZDS_FP32) {
    static_cast<float *>(base)[i] = x;
    return x;
  } else {
    const uint16_t h = narrow1<D>(x);
    static_cast<uint16_t *>(base)[i] = h;
    return D == ZDS_BF16 ? __uint_as_float(static_cast<uint32_t>(h) << 16) : __half2float(__ushort_as_half(h));
  }
}

template <int XD, bool VEC>
__device__ __forceinline__ void load_x(const void *p, int64_t e, int64_t n, bool whole, float (&x)[4]) {
  if (VEC && whole) {
    load_quad<XD>(p, e >> 2, x);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = e + i < n ? widen1<XD>(p, e + i) : 0.0f;
  }
}

// With error feedback: reads x and the error, writes the error and the values.
template <int XD, int D, bool VEC>
__global__ void __launch_bounds__(256) dropout_encode_kernel(DropArgs a) {
  __shared__ __align__(16) uint8_t kept[kDropTile / 2 + 32];
  const int64_t tiles = (a.n + kDropTile - 1) / kDropTile;
  const int ratio = 1 << a.shift;
  const bool skip = a.sc && a.sc->overflow;
  const float scale = a.state->scale, inv = 1.0f / scale;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t g0 = (t * kDropTile) >> a.shift;
    const int off = make_kept(a, g0, kDropTile >> a.shift, kept);
    for (int q = threadIdx.x; q < kDropTile / 4; q += 256) {
      const int64_t e = t * kDropTile + 4 * q;
      if (e >= a.n) break;
      const bool whole = e + 4 <= a.n;
      if (skip) {
        for (int i = 0; i < 4; ++i)
          if (e + i < a.n && ((4 * q + i) & (ratio - 1)) == 0) put<D>(a.values, (e + i) >> a.shift, __uint_as_float(0x7fc00000u));
        continue;
      }
      float x[4], er[4];
      load_x<XD, VEC>(a.x, e, a.n, whole, x);
      load_x<ZDS_FP32, VEC>(a.err, e, a.n, whole, er);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int in = (4 * q + i) & (ratio - 1), k = (4 * q + i) >> a.shift;
        const int place = kept[off + k] >> (8 - a.shift);
        float c = x[i] + scale * er[i];
        if (e + i < a.n) {
          if (in == place) {
            const float sent = put<D>(a.values, g0 + k, c);
            if (magnitude(sent) < 0x7f800000u) c = c - sent;
          } else if (in == 0 && e + i + place >= a.n) {
            put<D>(a.values, g0 + k, 0.0f);  // the place of a cut last group lies past the end
          }
        }
        er[i] = c * inv;
      }
      if (VEC && whole) {
        store_quad(a.err, e >> 2, er);
      } else {
        for (int i = 0; i < 4; ++i)
          if (e + i < a.n) a.err[e + i] = er[i];
      }
    }
    __syncthreads();  // the next tile's places
  }
}

// Without feedback: only the kept elements are read.
template <int XD, int D>
__global__ void __launch_bounds__(256) dropout_gather_kernel(DropArgs a) {
  __shared__ __align__(16) uint8_t kept[kDropGroups + 32];
  const int64_t tiles = (a.groups + kDropGroups - 1) / kDropGroups;
  const float ratio = static_cast<float>(1 << a.shift);
  const bool skip = a.sc && a.sc->overflow;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t g0 = t * kDropGroups;
    const int off = make_kept(a, g0, kDropGroups, kept);
    for (int k = threadIdx.x; k < kDropGroups && g0 + k < a.groups; k += 256) {
      const int64_t e = ((g0 + k) << a.shift) + (kept[off + k] >> (8 - a.shift));
      float v = e < a.n ? ratio * widen1<XD>(a.x, e) : 0.0f;
      if (skip) v = __uint_as_float(0x7fc00000u);
      put<D>(a.values, g0 + k, v);
    }
    __syncthreads();
  }
}

// The sum of the peers' values of group g, in peer order.
template <int D>
__device__ __forceinline__ float peer_sum(const DropArgs &a, int64_t g) {
  float t = widen1<D>(a.peers[0], g);
  for (int k = 1; k < a.npeers; ++k) t = t + widen1<D>(a.peers[k], g);
  return t;
}

// Every element of the gradient is written.
template <int D, int OD, bool VEC>
__global__ void __launch_bounds__(256) dropout_spread_kernel(DropArgs a) {
  __shared__ __align__(16) uint8_t kept[kDropTile / 2 + 32];
  __shared__ float sum[kDropTile / 2];
  const int64_t tiles = (a.n + kDropTile - 1) / kDropTile;
  const int ratio = 1 << a.shift;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t g0 = (t * kDropTile) >> a.shift;
    const int count = kDropTile >> a.shift;
    for (int k = threadIdx.x; k < count && g0 + k < a.groups; k += 256) sum[k] = peer_sum<D>(a, g0 + k);
    const int off = make_kept(a, g0, count, kept);
    for (int q = threadIdx.x; q < kDropTile / 4; q += 256) {
      const int64_t e = t * kDropTile + 4 * q;
      if (e >= a.n) break;
      float o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int in = (4 * q + i) & (ratio - 1), k = (4 * q + i) >> a.shift;
        o[i] = in == (kept[off + k] >> (8 - a.shift)) ? sum[k] : 0.0f;
      }
      if (VEC && e + 4 <= a.n) {
        if constexpr (OD == ZDS_FP32) store_quad(static_cast<float *>(a.dst), e >> 2, o);
        else store_quad16<OD>(a.dst, e >> 2, o);
      } else {
        for (int i = 0; i < 4; ++i)
          if (e + i < a.n) put<OD>(a.dst, e + i, o[i]);
      }
    }
    __syncthreads();
  }
}

// Only the kept elements are read and written.
template <int D, int OD>
__global__ void __launch_bounds__(256) dropout_add_kernel(DropArgs a) {
  __shared__ __align__(16) uint8_t kept[kDropGroups + 32];
  const int64_t tiles = (a.groups + kDropGroups - 1) / kDropGroups;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t g0 = t * kDropGroups;
    const int off = make_kept(a, g0, kDropGroups, kept);
    for (int k = threadIdx.x; k < kDropGroups && g0 + k < a.groups; k += 256) {
      const int64_t e = ((g0 + k) << a.shift) + (kept[off + k] >> (8 - a.shift));
      if (e < a.n) put<OD>(a.dst, e, widen1<OD>(a.dst, e) + peer_sum<D>(a, g0 + k));
    }
    __syncthreads();
  }
}

static uint32_t blocks_for(int64_t items, int per_block) {
  const int64_t g = (items + per_block - 1) / per_block;
  return static_cast<uint32_t>(g < max_blocks(256) ? g : max_blocks(256));
}

template <int XD, int D>
static void compress_go(const DropArgs &a, bool vec, hipStream_t s) {
  if (!a.err)
    hipLaunchKernelGGL((dropout_gather_kernel<XD, D>), dim3(blocks_for(a.groups, kDropGroups)), dim3(256), 0, s, a);
  else if (vec)
    hipLaunchKernelGGL((dropout_encode_kernel<XD, D, true>), dim3(blocks_for(a.n, kDropTile)), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((dropout_encode_kernel<XD, D, false>), dim3(blocks_for(a.n, kDropTile)), dim3(256), 0, s, a);
}
template <int XD>
static void compress_values(zds_dtype d, const DropArgs &a, bool vec, hipStream_t s) {
  if (d == ZDS_FP16) compress_go<XD, ZDS_FP16>(a, vec, s);
  else if (d == ZDS_BF16) compress_go<XD, ZDS_BF16>(a, vec, s);
  else compress_go<XD, ZDS_FP32>(a, vec, s);
}

template <int D, int OD>
static void decompress_go(const DropArgs &a, bool add, bool vec, hipStream_t s) {
  if (add)
    hipLaunchKernelGGL((dropout_add_kernel<D, OD>), dim3(blocks_for(a.groups, kDropGroups)), dim3(256), 0, s, a);
  else if (vec)
    hipLaunchKernelGGL((dropout_spread_kernel<D, OD, true>), dim3(blocks_for(a.n, kDropTile)), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((dropout_spread_kernel<D, OD, false>), dim3(blocks_for(a.n, kDropTile)), dim3(256), 0, s, a);
}
template <int D>
static void decompress_to(zds_dtype od, const DropArgs &a, bool add, bool vec, hipStream_t s) {
  if (od == ZDS_FP32) decompress_go<D, ZDS_FP32>(a, add, vec, s);
  else decompress_go<D, D>(a, add, vec, s);
}

// What both ends check, and log2(ratio).
static zds_status check_dropout(const char *fn, int64_t n, int32_t ratio, int64_t first, zds_dtype values,
                                int32_t *shift) {
  if (ratio < 2 || ratio > 256 || (ratio & (ratio - 1)) != 0)
    return fail(ZDS_EINVAL, "%s: ratio must be a power of two in [2, 256]", fn);
  if (!valid_dtype(values)) return fail(ZDS_EINVAL, "%s: bad value dtype", fn);
  if (n < 0 || n >= kStateMost) return fail(ZDS_EINVAL, "%s: n must lie in [0, 2^40)", fn);
  if (first < 0 || first % ratio != 0) return fail(ZDS_EINVAL, "%s: first must be a multiple of ratio, >= 0", fn);
  *shift = 0;
  while ((1 << *shift) < ratio) ++*shift;
  return ZDS_OK;
}

}  // namespace zds

using namespace zds;

extern "C" zds_status zds_dropout_compress(const void *x, zds_dtype x_dtype, float *error, int64_t n, int32_t ratio,
                                           uint64_t seed, int64_t first, const zds_step_scalars *scalars_dev,
                                           const zds_step_state *state_dev, void *values, zds_dtype value_dtype,
                                           void *stream) {
  clear_error();
  const char *fn = "zds_dropout_compress";
  int32_t shift = 0;
  const zds_status st = check_dropout(fn, n, ratio, first, value_dtype, &shift);
  if (st != ZDS_OK) return st;
  if (!valid_dtype(x_dtype)) return fail(ZDS_EINVAL, "%s: bad x dtype", fn);
  if (n == 0) return ZDS_OK;
  if (!x || !values || !state_dev) return fail(ZDS_EINVAL, "%s: null pointer", fn);
  if (!aligned(x, static_cast<uintptr_t>(dtype_size(x_dtype))) || (error && !aligned(error, 4)) ||
      !aligned(values, static_cast<uintptr_t>(dtype_size(value_dtype))) || !aligned(state_dev, 8) ||
      (scalars_dev && !aligned(scalars_dev, 8)))
    return fail(ZDS_EALIGN, "%s: pointer not aligned to its element size", fn);
  const int64_t groups = (n + ratio - 1) / ratio;
  const int64_t xb = n * dtype_size(x_dtype), eb = error ? n * 4 : 0, vb = groups * dtype_size(value_dtype);
  if (ranges_meet(x, xb, error, eb) || ranges_meet(x, xb, values, vb) || ranges_meet(error, eb, values, vb))
    return fail(ZDS_EINVAL, "%s: x, error and values overlap", fn);
  DropArgs a{};
  a.x = x;
  a.err = error;
  a.values = values;
  a.n = n;
  a.groups = groups;
  a.j0 = first >> shift;
  a.seed = seed;
  a.shift = shift;
  a.sc = scalars_dev;
  a.state = state_dev;
  const bool vec = aligned(x, x_dtype == ZDS_FP32 ? 16 : 8) && aligned(error, 16);
  hipStream_t s = static_cast<hipStream_t>(stream);
  switch (x_dtype) {
    case ZDS_FP16: compress_values<ZDS_FP16>(value_dtype, a, vec, s); break;
    case ZDS_BF16: compress_values<ZDS_BF16>(value_dtype, a, vec, s); break;
    default: compress_values<ZDS_FP32>(value_dtype, a, vec, s); break;
  }
  return check_launch("dropout_compress kernel");
}

extern "C" zds_status zds_dropout_decompress(const void *const *peer_values, int32_t num_peers, zds_dtype value_dtype,
                                             int64_t n, int32_t ratio, uint64_t seed, int64_t first,
                                             const zds_step_state *state_dev, void *dst, zds_dtype dst_dtype,
                                             zds_accum_mode mode, void *stream) {
  clear_error();
  const char *fn = "zds_dropout_decompress";
  if (num_peers < 1 || num_peers > kMaxPeers) return fail(ZDS_EINVAL, "%s: num_peers must be in [1, %d]", fn, kMaxPeers);
  if (mode != ZDS_OVERWRITE && mode != ZDS_ACCUMULATE) return fail(ZDS_EINVAL, "%s: mode must be overwrite or accumulate", fn);
  int32_t shift = 0;
  const zds_status st = check_dropout(fn, n, ratio, first, value_dtype, &shift);
  if (st != ZDS_OK) return st;
  if (dst_dtype != ZDS_FP32 && dst_dtype != value_dtype)
    return fail(ZDS_EINVAL, "%s: dst must be fp32 or of the values' type", fn);
  if (n == 0) return ZDS_OK;
  if (!peer_values || !dst || !state_dev) return fail(ZDS_EINVAL, "%s: null pointer", fn);
  const int64_t groups = (n + ratio - 1) / ratio;
  DropArgs a{};
  for (int k = 0; k < num_peers; ++k) {
    if (!peer_values[k]) return fail(ZDS_EINVAL, "%s: peer %d is null", fn, k);
    if (!aligned(peer_values[k], static_cast<uintptr_t>(dtype_size(value_dtype))))
      return fail(ZDS_EALIGN, "%s: peer %d misaligned", fn, k);
    if (ranges_meet(peer_values[k], groups * dtype_size(value_dtype), dst, n * dtype_size(dst_dtype)))
      return fail(ZDS_EINVAL, "%s: dst overlaps peer %d", fn, k);
    a.peers[k] = peer_values[k];
  }
  if (!aligned(dst, static_cast<uintptr_t>(dtype_size(dst_dtype))) || !aligned(state_dev, 8))
    return fail(ZDS_EALIGN, "%s: pointer not aligned to its element size", fn);
  a.dst = dst;
  a.n = n;
  a.groups = groups;
  a.j0 = first >> shift;
  a.seed = seed;
  a.shift = shift;
  a.npeers = num_peers;
  a.state = state_dev;
  const bool vec = aligned(dst, dst_dtype == ZDS_FP32 ? 16 : 8);
  hipStream_t s = static_cast<hipStream_t>(stream);
  switch (value_dtype) {
    case ZDS_FP16: decompress_to<ZDS_FP16>(dst_dtype, a, mode == ZDS_ACCUMULATE, vec, s); break;
    case ZDS_BF16: decompress_to<ZDS_BF16>(dst_dtype, a, mode == ZDS_ACCUMULATE, vec, s); break;
    default: decompress_to<ZDS_FP32>(dst_dtype, a, mode == ZDS_ACCUMULATE, vec, s); break;
  }
  return check_launch("dropout_decompress kernel");
}
