// Gradient dropout: the two ends of an exchange in which every group of
// `ratio` consecutive elements sends one, chosen by the counter-based
// generator (include/zds.h has the definition, zds_random.h the generator).
//
// Streams, all bound by HBM. With feedback, encoding reads x and the error and
// writes the error (2 or 4 + 8 B an element) and the values. Decoding writes the
// whole gradient (4 or 2 B an element). Encoding without feedback and adding need
// one element of each group, and memory gives whole lines of 128 bytes: in groups
// of up to a line (32 fp32 or 64 16-bit elements) every line is touched, so all
// of x is streamed, or all of dst read and written back; in longer groups only the
// kept elements are read, or read and written.
// A block first makes the kept places of its groups in LDS: one call of the
// generator covers 16 groups, so its arithmetic does not show.
#include "zds_internal.h"
#include "zds_quantised.h"

namespace zds {

// Elements of a block's tile where a gradient is encoded with feedback.
constexpr int kEncodeBlock = 512;
constexpr int kEncodeTile = 4 * kEncodeBlock;
// Elements of a block's tile where a whole gradient is written.
constexpr int kSpreadBlock = 256;
constexpr int kSpreadTile = 16 * kSpreadBlock;
// Consecutive tiles that one XCD gets where tiles share lines of a message.
constexpr int kXcdRun = 16;
// Groups of a block where only the kept elements are read or added to.
constexpr int kDropGroups = 1024;

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
  int64_t tile0;     // the launch's first tile
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

// What becomes of an element with c = x + scale * error: sent if it is kept;
// returns the new error. in: its place in its group, place: the kept one;
// missing: that one lies past the end. value(v) stores a value and returns it as
// stored.
template <typename Put>
__device__ __forceinline__ float encode_element(float c, float inv, int in, int place, bool missing, const Put &value) {
  if (in == place) {
    const float sent = value(c);
    if (magnitude(sent) < 0x7f800000u) c = c - sent;
  } else if (missing && in == 0) {
    value(0.0f);
  }
  return c * inv;
}

// A tile, or what there is of it, by a block, one element by one.
template <int XD, int D>
__device__ __forceinline__ void encode_elements(const DropArgs &a, int64_t first, float scale, float inv, uint8_t *kept) {
  const int64_t g0 = first >> a.shift;
  const int mask = (1 << a.shift) - 1;
  const int off = make_kept(a, g0, kEncodeTile >> a.shift, kept);
  for (int k = threadIdx.x; k < kEncodeTile && first + k < a.n; k += kEncodeBlock) {
    const int64_t e = first + k;
    const int in = k & mask, g = k >> a.shift, place = kept[off + g] >> (8 - a.shift);
    const float c = widen1<XD>(a.x, e) + scale * a.err[e];
    a.err[e] = encode_element(c, inv, in, place, e - in + place >= a.n, [&](float v) { return put<D>(a.values, g0 + g, v); });
  }
}

// With feedback. A block takes a tile of 2048 elements, each thread a quad;
// 16-bit x comes in 16 bytes a lane by waves 0-3, and the values go out so,
// through LDS; a wave has one load in flight. VEC: whole tiles are aligned.
// bf16, ratio 16, 842M elements: 1.32 ms (6.5 TB/s); four quads a thread loaded
// where they are used: 1.43.
template <int XD, int D, bool VEC>
__global__ void __launch_bounds__(kEncodeBlock) dropout_encode_kernel(DropArgs a) {
  __shared__ __align__(16) uint8_t kept[kEncodeTile / 2 + 32];
  __shared__ u32x4 xs[XD == ZDS_FP32 ? 1 : kEncodeTile / 8];
  __shared__ u32x4 out[kEncodeTile / (D == ZDS_FP32 ? 8 : 16)];
  const int t = threadIdx.x;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int64_t first = (a.tile0 + blockIdx.x) * kEncodeTile;
  const int64_t g0 = first >> a.shift;
  const int groups = kEncodeTile >> a.shift, mask = (1 << a.shift) - 1;
  if (a.sc && a.sc->overflow) {  // uniform
    for (int k = t; k < groups && g0 + k < a.groups; k += kEncodeBlock) put<D>(a.values, g0 + k, __uint_as_float(0x7fc00000u));
    return;
  }
  const float scale = a.state->scale, inv = 1.0f / scale;
  if (!VEC || first + kEncodeTile > a.n) {
    encode_elements<XD, D>(a, first, scale, inv, kept);
    return;
  }
  float *err = a.err + first;
  f32x4 xf{};
  if (XD == ZDS_FP32) {
    xf = ld_stream_global(reinterpret_cast<const f32x4 *>(static_cast<const float *>(a.x) + first) + t);
    wait_vmem();
  } else if (w < 4) {
    xs[t] = ld_stream_global(reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(a.x) + first) + t);
  }
  const f32x4 e4 = ld_stream_global(reinterpret_cast<const f32x4 *>(err) + t);
  const int off = make_kept(a, g0, groups, kept);
  float x[4], er[4] = {e4.x, e4.y, e4.z, e4.w};
  if constexpr (XD == ZDS_FP32) {
    x[0] = xf.x; x[1] = xf.y; x[2] = xf.z; x[3] = xf.w;
  } else {
    const u32x2 q = reinterpret_cast<const u32x2 *>(xs)[t];
    x[0] = lo_of<XD>(q.x); x[1] = hi_of<XD>(q.x); x[2] = lo_of<XD>(q.y); x[3] = hi_of<XD>(q.y);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = 4 * t + i, g = k >> a.shift, place = kept[off + g] >> (8 - a.shift);
    er[i] = encode_element(x[i] + scale * er[i], inv, k & mask, place, false, [&](float v) { return put<D>(out, g, v); });
  }
  st_stream_at(err, 16 * t, f32x4{er[0], er[1], er[2], er[3]});
  __syncthreads();
  constexpr int size = D == ZDS_FP32 ? 4 : 2;
  if (16 * t < groups * size) st_stream_at(static_cast<uint8_t *>(a.values) + g0 * size, 16 * t, out[t]);
}

// Without feedback and with short groups, aligned: x is streamed, four 16-byte
// pieces a thread (4096 fp32 or 8192 16-bit elements a block), and the values go
// out 16 bytes a lane.
template <int XD>
constexpr int kPickTile = 256 * 4 * (XD == ZDS_FP32 ? 4 : 8);
template <int XD, int D>
__global__ void __launch_bounds__(256) dropout_pick_kernel(DropArgs a) {
  constexpr int E = XD == ZDS_FP32 ? 4 : 8, tile = kPickTile<XD>, size = D == ZDS_FP32 ? 4 : 2;
  __shared__ __align__(16) uint8_t kept[tile / 2 + 32];
  __shared__ u32x4 out[tile / 2 * size / 16];
  const int t = threadIdx.x;
  const int64_t first = (a.tile0 + blockIdx.x) * tile;
  const int64_t g0 = first >> a.shift;
  const int groups = tile >> a.shift, mask = (1 << a.shift) - 1;
  const float ratio = static_cast<float>(1 << a.shift);
  const bool skip = a.sc && a.sc->overflow;
  if (skip || first + tile > a.n) {
    const int off = make_kept(a, g0, groups, kept);
    for (int k = t; k < groups && g0 + k < a.groups; k += 256) {
      const int64_t e = ((g0 + k) << a.shift) + (kept[off + k] >> (8 - a.shift));
      put<D>(a.values, g0 + k, skip ? __uint_as_float(0x7fc00000u) : e < a.n ? ratio * widen1<XD>(a.x, e) : 0.0f);
    }
    return;
  }
  const u32x4 *src = reinterpret_cast<const u32x4 *>(static_cast<const uint8_t *>(a.x) + first * (XD == ZDS_FP32 ? 4 : 2));
  u32x4 q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = ld_stream_global(src + 256 * i + t);
  const int off = make_kept(a, g0, groups, kept);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
    for (int l = 0; l < E; l += 4) {
      const int k = E * (256 * i + t) + l, g = k >> a.shift;
      float x[4];
      if constexpr (XD == ZDS_FP32) {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = __uint_as_float(w[j]);
      } else {
        x[0] = lo_of<XD>(w[l / 2]); x[1] = hi_of<XD>(w[l / 2]); x[2] = lo_of<XD>(w[l / 2 + 1]); x[3] = hi_of<XD>(w[l / 2 + 1]);
      }
      if (a.shift > 1) {  // a quad lies in one group
        const int at = (kept[off + g] >> (8 - a.shift)) - (k & mask);
        if (at >= 0 && at < 4) put<D>(out, g, ratio * (at < 2 ? (at == 0 ? x[0] : x[1]) : (at == 2 ? x[2] : x[3])));
      } else {
        put<D>(out, g, ratio * (kept[off + g] >> 7 ? x[1] : x[0]));
        put<D>(out, g + 1, ratio * (kept[off + g + 1] >> 7 ? x[3] : x[2]));
      }
    }
  }
  __syncthreads();
  for (int k = t; 16 * k < groups * size; k += 256) st_stream_at(static_cast<uint8_t *>(a.values) + g0 * size, 16 * k, out[k]);
}

// Without feedback: only the kept elements are loaded.
template <int XD, int D>
__global__ void __launch_bounds__(256) dropout_gather_kernel(DropArgs a) {
  __shared__ __align__(16) uint8_t kept[kDropGroups + 32];
  const float ratio = static_cast<float>(1 << a.shift);
  const bool skip = a.sc && a.sc->overflow;
  const int64_t g0 = (a.tile0 + blockIdx.x) * kDropGroups;
  const int off = make_kept(a, g0, kDropGroups, kept);
  float v[kDropGroups / 256];
#pragma unroll
  for (int i = 0; i < kDropGroups / 256; ++i) {
    const int k = threadIdx.x + 256 * i;
    const int64_t e = ((g0 + k) << a.shift) + (kept[off + k] >> (8 - a.shift));
    v[i] = skip ? __uint_as_float(0x7fc00000u) : e < a.n ? ratio * widen1<XD>(a.x, e) : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < kDropGroups / 256; ++i) {
    const int k = threadIdx.x + 256 * i;
    if (g0 + k < a.groups) put<D>(a.values, g0 + k, v[i]);
  }
}

// The sum of the peers' values of group g, in peer order.
template <int D>
__device__ __forceinline__ float peer_sum(const DropArgs &a, int64_t g) {
  float t = widen1<D>(a.peers[0], g);
  for (int k = 1; k < a.npeers; ++k) t = t + widen1<D>(a.peers[k], g);
  return t;
}

// Every element of the gradient is written (ADD: read, and all but the kept ones
// written back as they are), a tile of 4096 a block. The
// messages come in 16 bytes a lane, dealt out over all waves, into LDS (as many
// messages at a time as 16 KiB hold), where each thread sums its groups in peer
// order; then the tile is written 16 bytes a lane. VEC: whole tiles are aligned.
// 8 bf16 messages, ratio 8, 842M fp32 elements: 0.823 ms (6.14 TB/s); blocks
// of 512 threads 0.835; a lane reading all messages of its 8 groups, one after
// another or together, left most waves without a load: 0.93 to 0.96 (tiles of
// 16384). Tiles of 8192 and 16384 are slower wherever messages are read to any
// amount (202M elements, ratio 2, 8 messages: 411 us, 488), a little faster
// for many messages of a high ratio, of which a tile reads a few bytes each.
// Blocks go to the 8 XCDs in turn. Where a tile reads less than a 128-byte line
// of a message, an XCD gets runs of 16 tiles, or the line is fetched by several
// L2s: 202M elements, ratio 256, bf16 messages into bf16, 8 of them 125 -> 73 us,
// 16 123 -> 77; into fp32 167 -> 130, 173 -> 130 (runs of 4: 74, 88; 152, 152). Of
// lower ratios it gains 3 to 8 % at 2 and loses 8 to 13 % at 8.
template <int D, int OD, bool VEC, bool ADD>
__global__ void __launch_bounds__(kSpreadBlock) dropout_spread_kernel(DropArgs a) {
  constexpr int kGroups = kSpreadTile / 2, kRaw = 16384;
  __shared__ __align__(16) uint8_t kept[kGroups + 32];
  __shared__ u32x4 raw[kRaw / 16];
  const int t = threadIdx.x;
  uint32_t tile = blockIdx.x;
  constexpr uint32_t R = kXcdRun, X = 8 * R;
  if (!ADD && (kSpreadTile >> a.shift) * (D == ZDS_FP32 ? 4 : 2) < 128 && tile / X < gridDim.x / X)
    tile = tile / X * X + tile % 8 * R + tile / 8 % R;
  const int64_t first = (a.tile0 + tile) * kSpreadTile;
  const int64_t g0 = first >> a.shift;
  const int groups = kSpreadTile >> a.shift, mask = (1 << a.shift) - 1;
  float *sum = reinterpret_cast<float *>(raw);
  if (!VEC || first + kSpreadTile > a.n) {
    for (int k = t; k < groups && g0 + k < a.groups; k += kSpreadBlock) sum[k] = peer_sum<D>(a, g0 + k);
    const int off = make_kept(a, g0, groups, kept);
    for (int k = t; k < kSpreadTile && first + k < a.n; k += kSpreadBlock) {
      const int g = k >> a.shift;
      if (ADD) {
        if ((k & mask) == (kept[off + g] >> (8 - a.shift))) put<OD>(a.dst, first + k, widen1<OD>(a.dst, first + k) + sum[g]);
        continue;
      }
      put<OD>(a.dst, first + k, (k & mask) == (kept[off + g] >> (8 - a.shift)) ? sum[g] : 0.0f);
    }
    return;
  }
  constexpr int size = D == ZDS_FP32 ? 4 : 2;
  const int bytes = groups * size;                          // of one message's part of the tile
  const int pieces_shift = 31 - __builtin_clz(bytes >> 4);  // (32 bytes at least: 16 groups at a ratio of 256)
  const int most = kRaw / bytes;
  constexpr int E = OD == ZDS_FP32 ? 4 : 8, W = kSpreadTile / E / kSpreadBlock;
  u32x4 old[W];
  if (ADD) {
#pragma unroll
    for (int i = 0; i < W; ++i)
      old[i] = ld_stream_global(reinterpret_cast<const u32x4 *>(static_cast<const uint8_t *>(a.dst) + first * (16 / E)) +
                                t + kSpreadBlock * i);
  }
  const int off = make_kept(a, g0, groups, kept);
  float s[kGroups / kSpreadBlock];
  for (int j0 = 0; j0 < a.npeers; j0 += most) {
    const int peers = a.npeers - j0 < most ? a.npeers - j0 : most;
    if (j0 > 0) __syncthreads();
    const auto fetch = [&](const void *from, int k) {
      raw[k] = ld_stream_global(reinterpret_cast<const u32x4 *>(static_cast<const uint8_t *>(from) + g0 * size) +
                                (k & ((1 << pieces_shift) - 1)));
    };
    if (pieces_shift >= 6) {  // a wave's pieces are of one message: its address comes from the scalar arguments
      for (int k = t; k < peers << pieces_shift; k += kSpreadBlock)
        fetch(a.peers[j0 + __builtin_amdgcn_readfirstlane(k >> pieces_shift)], k);
    } else {
      for (int k = t; k < peers << pieces_shift; k += kSpreadBlock) fetch(a.peers[j0 + (k >> pieces_shift)], k);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kGroups / kSpreadBlock; ++i) {
      const int g = t + kSpreadBlock * i;
      if (g >= groups) break;
#pragma unroll 4
      for (int j = 0; j < peers; ++j) {
        const float x = widen1<D>(raw, j * groups + g);
        s[i] = j0 + j == 0 ? x : s[i] + x;
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kGroups / kSpreadBlock; ++i)
    if (t + kSpreadBlock * i < groups) sum[t + kSpreadBlock * i] = s[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const int q = t + kSpreadBlock * i;
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if (ADD) {
      w[0] = old[i].x; w[1] = old[i].y; w[2] = old[i].z; w[3] = old[i].w;
    }
#pragma unroll
    for (int l = 0; l < E; l += 4) {
      const int k = E * q + l, g = k >> a.shift;
      const bool one = a.shift > 1;  // a quad lies in one group, or is two
      const int at = one ? (kept[off + g] >> (8 - a.shift)) - (k & mask) : kept[off + g] >> 7;
      const int at2 = one ? at : 2 + (kept[off + g + 1] >> 7);
      const float x = sum[g], x2 = one ? x : sum[g + 1];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool is = at == j || at2 == j;
        const float y = j < 2 ? x : x2;
        if constexpr (OD == ZDS_FP32) {
          w[j] = is ? __float_as_uint(ADD ? __uint_as_float(w[j]) + y : y) : w[j];
        } else {
          const int u = (l + j) / 2;
          const float before = (j & 1) ? hi_of<OD>(w[u]) : lo_of<OD>(w[u]);
          const uint32_t h = narrow1<OD>(ADD ? before + y : y);
          w[u] = !is ? w[u] : (j & 1) ? (w[u] & 0xffffu) | (h << 16) : (w[u] & 0xffff0000u) | h;
        }
      }
    }
    st_stream_at(static_cast<uint8_t *>(a.dst) + first * (16 / E), 16 * q, u32x4{w[0], w[1], w[2], w[3]});
  }
}

// Adding to the kept elements of long groups, or to a dst that is not aligned;
// only they are read and written: of a gradient of 45M fp32
// elements at ratio 64, 705K lines of 128 bytes are read for 4 bytes each and
// written back in part (counters: 96 MB read, 22.5 MB written), 30 us. Fewer
// groups a block (29 us), the messages' loads before or after the gradient's (31)
// make little difference, and accesses that bypass the caches are slower (43).
template <int D, int OD>
__global__ void __launch_bounds__(256) dropout_add_kernel(DropArgs a) {
  __shared__ __align__(16) uint8_t kept[kDropGroups + 32];
  constexpr int N = kDropGroups / 256;
  const int64_t g0 = (a.tile0 + blockIdx.x) * kDropGroups;
  const int off = make_kept(a, g0, kDropGroups, kept);
  int64_t e[N];
  float o[N], s[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int k = threadIdx.x + 256 * i;
    e[i] = ((g0 + k) << a.shift) + (kept[off + k] >> (8 - a.shift));
    o[i] = e[i] < a.n ? widen1<OD>(a.dst, e[i]) : 0.0f;
    s[i] = 0.0f;
  }
  for (int j = 0; j < a.npeers; ++j) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t g = g0 + threadIdx.x + 256 * i;
      const float x = g < a.groups ? widen1<D>(a.peers[j], g) : 0.0f;
      s[i] = j == 0 ? x : s[i] + x;
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (e[i] < a.n) put<OD>(a.dst, e[i], o[i] + s[i]);
}

// One block for each of `count` tiles, in launches below 2^32 work-items.
template <typename Launch>
static void each_tile(DropArgs a, int64_t count, int threads, const Launch &launch) {
  const int64_t most = max_blocks(threads);
  for (a.tile0 = 0; a.tile0 < count; a.tile0 += most)
    launch(a, dim3(static_cast<uint32_t>(count - a.tile0 < most ? count - a.tile0 : most)));
}
static int64_t pieces(int64_t items, int64_t of) { return (items + of - 1) / of; }

// Without feedback groups of up to a 128-byte line are streamed, since every line
// of x is read either way; of longer ones only the kept elements are loaded. 45M
// elements, us gathered / streamed: fp32 at ratio 2 49 / 43, 16 36 / 31, 32 (128
// bytes) 33 / 29; bf16 at 2 41 / 23, 16 20 / 17, 64 (128 bytes) 19 / 15. At twice
// the line a gather reads half of them: fp32 at 64 17.
template <int XD, int D>
static void compress_go(const DropArgs &a, bool vec, hipStream_t s) {
  if (a.err) {
    each_tile(a, pieces(a.n, kEncodeTile), kEncodeBlock, [&](const DropArgs &b, dim3 g) {
      if (vec) hipLaunchKernelGGL((dropout_encode_kernel<XD, D, true>), g, dim3(kEncodeBlock), 0, s, b);
      else hipLaunchKernelGGL((dropout_encode_kernel<XD, D, false>), g, dim3(kEncodeBlock), 0, s, b);
    });
  } else if (vec && ((XD == ZDS_FP32 ? 4 : 2) << a.shift) <= 128) {
    each_tile(a, pieces(a.n, kPickTile<XD>), 256, [&](const DropArgs &b, dim3 g) {
      hipLaunchKernelGGL((dropout_pick_kernel<XD, D>), g, dim3(256), 0, s, b);
    });
  } else {
    each_tile(a, pieces(a.groups, kDropGroups), 256, [&](const DropArgs &b, dim3 g) {
      hipLaunchKernelGGL((dropout_gather_kernel<XD, D>), g, dim3(256), 0, s, b);
    });
  }
}
template <int XD>
static void compress_values(zds_dtype d, const DropArgs &a, bool vec, hipStream_t s) {
  if (d == ZDS_FP16) compress_go<XD, ZDS_FP16>(a, vec, s);
  else if (d == ZDS_BF16) compress_go<XD, ZDS_BF16>(a, vec, s);
  else compress_go<XD, ZDS_FP32>(a, vec, s);
}

// Adding: a group of up to a 128-byte line is streamed like an overwrite, since
// every line of dst is read and written either way; of longer ones only the kept
// elements are. 202M elements, bf16 messages, us by element / streamed: fp32 dst,
// one message, ratio 2 357 / 294, 8 336 / 270, 32 (128 bytes) 356 / 267, 64 146 /
// 266; bf16 dst, 2 311 / 157, 8 169 / 135, 64 (128 bytes) 138 / 126, 128 54 / 126;
// 16 messages at ratio 2 1,771 / 830 and 1,728 / 704.
template <int D, int OD>
static void decompress_go(const DropArgs &a, bool add, bool vec, hipStream_t s) {
  if (add && !(vec && ((OD == ZDS_FP32 ? 4 : 2) << a.shift) <= 128)) {
    each_tile(a, pieces(a.groups, kDropGroups), 256, [&](const DropArgs &b, dim3 g) {
      hipLaunchKernelGGL((dropout_add_kernel<D, OD>), g, dim3(256), 0, s, b);
    });
    return;
  }
  each_tile(a, pieces(a.n, kSpreadTile), kSpreadBlock, [&](const DropArgs &b, dim3 g) {
    if (add) hipLaunchKernelGGL((dropout_spread_kernel<D, OD, true, true>), g, dim3(kSpreadBlock), 0, s, b);
    else if (vec) hipLaunchKernelGGL((dropout_spread_kernel<D, OD, true, false>), g, dim3(kSpreadBlock), 0, s, b);
    else hipLaunchKernelGGL((dropout_spread_kernel<D, OD, false, false>), g, dim3(kSpreadBlock), 0, s, b);
  });
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
  if (first < 0 || first % ratio != 0 || first > INT64_MAX - n)
    return fail(ZDS_EINVAL, "%s: first must be a multiple of ratio in [0, 2^63 - n)", fn);
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
  const bool vec = aligned(x, 16) && aligned(error, 16) && aligned(values, 16);
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
  bool vec = aligned(dst, 16);
  for (int k = 0; k < num_peers; ++k) vec = vec && aligned(peer_values[k], 16);
  hipStream_t s = static_cast<hipStream_t>(stream);
  switch (value_dtype) {
    case ZDS_FP16: decompress_to<ZDS_FP16>(dst_dtype, a, mode == ZDS_ACCUMULATE, vec, s); break;
    case ZDS_BF16: decompress_to<ZDS_BF16>(dst_dtype, a, mode == ZDS_ACCUMULATE, vec, s); break;
    default: decompress_to<ZDS_FP32>(dst_dtype, a, mode == ZDS_ACCUMULATE, vec, s); break;
  }
  return check_launch("dropout_decompress kernel");
}
