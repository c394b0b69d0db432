// Newton-Schulz orthogonalisation of the matrices of a flat buffer:
//   X_0 = G / (||G||_F + eps);  A = X X^T;  B = b A + c A^2;  X <- a X + B X
// on the smaller side of each matrix (a tall G is worked on as its transpose).
//
// Every product is a sum over the rows' elements of two operands. A = X X^T and
// A^2 = A A^T (A is symmetric) take both operands as they lie; in B X the
// summed axis runs down X's rows, and its pieces are turned on the way from
// LDS to the registers (transposing LDS reads), so X is kept in one
// orientation. A and B are symmetric: only tiles on and below the diagonal
// are computed, and each is stored twice, which takes a step from
// 4 m^2 n + 2 m^3 operations to 3 m^2 n + m^3.
//
// Numbers. The matrix instructions take fp16 operands and sum in fp32. X, A and
// B have bounded spectra, so powers of two bring them into fp16's range,
// where they keep 11 bits (bf16 would keep 8 at the same speed). For BF16
// results X is carried with what its fp16 value leaves (a second fp16 array,
// read and written by the epilogue only, but for pairs). For FP32 every operand is a pair of
// fp16 numbers (high and low) and a product runs its sum over three pieces,
// low*high + high*low + high*high, into the same fp32 accumulators. So do A A
// and B X of a BF16 result with up to 64 rows, where little averages out
// (NsMatrix::pair; the error over that of the last rounding alone: 16 x 32
// 1.47 -> 1.09, 32 x 1000 1.66 -> 1.03; next to larger matrices, 1 x 513 among
// 1000 x 4096 and others, 474 -> 483 us).
#include <algorithm>
#include <cmath>
#include <new>
#include <type_traits>

#include "zds_device.h"
#include "zds_matrix.h"

namespace zds {

typedef _Float16 half_t;
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) const void global_cvoid;

constexpr int kMaxSteps = 16;
constexpr double kNormEps = 1e-7;
// A partial sum of squares covers this many elements or more; a matrix has at
// most kMaxParts of them.
constexpr int64_t kNormChunk = 32768;
constexpr int kMaxParts = 1024;
constexpr int kUnits = 256;  // compute units
constexpr int kConvTile = 64;
constexpr int kPairRows = 64;  // rows up to which A and B of a BF16 result are pairs

// A matrix's first X as stored and true: X_true = alpha * X_stored.
struct NsScale {
  float alpha;
};

// An fp32 number as two fp16 ones, high + low. The empty statement holds the
// number at its fp32 value: without it the compiler rounds a product once more
// straight to fp16 for one use of the high half and by way of fp32 for the
// other, and next to a tie the low half then belongs to another high half (one
// in about 16000 numbers off by 2^-11: fp32 lands on a tie of fp16 once in 8192,
// half of the time from the other side. FP32 results of 312 matrices of 8 x 8:
// 7.1 times the error of plain fp32, and 1.4 with one rounding).
struct HalfPair {
  half_t high, low;
};
__device__ __forceinline__ HalfPair split(float v) {
  asm("" : "+v"(v));
  const half_t h = static_cast<half_t>(v);
  return {h, static_cast<half_t>(v - static_cast<float>(h))};
}

// ---------------------------------------------------------------------------
// Norm and conversion
// ---------------------------------------------------------------------------

// 16-byte accesses at an element's address: a matrix may begin at any element
// and have rows of any length.
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));

// Eight consecutive elements.
template <int D>
__device__ __forceinline__ void load_eight(const char *p, float (&v)[8]) {
  if constexpr (D == ZDS_FP32) {
    const f32x4 a = reinterpret_cast<const f32x4_any *>(p)[0], b = reinterpret_cast<const f32x4_any *>(p)[1];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = a[j];
      v[4 + j] = b[j];
    }
  } else {
    const u32x4 w = *reinterpret_cast<const u32x4_any *>(p);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = lo_of<D>(w[j]);
      v[2 * j + 1] = hi_of<D>(w[j]);
    }
  }
}

// Sum of squares of one chunk (mt.chunk elements) of a matrix, in a fixed order.
template <int D>
__global__ void __launch_bounds__(256) ns_norm_kernel(const NsMatrix *mats, const NsTile *chunks, const void *src,
                                                      double *partials, const zds_step_scalars *sc) {
  if (sc && sc->overflow) return;
  const NsTile t = chunks[blockIdx.x];
  const NsMatrix mt = mats[t.mat];
  const int64_t all = static_cast<int64_t>(mt.rows) * mt.cols;
  const int64_t lo = static_cast<int64_t>(t.ti) * mt.chunk;
  const int64_t hi = lo + mt.chunk < all ? lo + mt.chunk : all;
  constexpr int ES = D == ZDS_FP32 ? 4 : 2;
  const char *base = static_cast<const char *>(src) + (mt.offset + lo) * ES;
  double acc[2] = {0.0, 0.0};
  const int64_t groups = (hi - lo) / 8;
  auto add = [&](const float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j & 1] = sq_add(v[j], acc[j & 1]);
  };
  int64_t g = threadIdx.x;
  for (; g + 3 * 256 < groups; g += 4 * 256) {
    float v[4][8];
#pragma unroll
    for (int r = 0; r < 4; ++r) load_eight<D>(base + (g + r * 256) * 8 * ES, v[r]);
#pragma unroll
    for (int r = 0; r < 4; ++r) add(v[r]);
  }
  for (; g < groups; g += 256) {
    float v[8];
    load_eight<D>(base + g * 8 * ES, v);
    add(v);
  }
  for (int64_t i = groups * 8 + threadIdx.x; i < hi - lo; i += 256) acc[0] = sq_add(widen1<D>(base, i), acc[0]);
  const double b = block_sum<256>(acc[0] + acc[1]);
  if (threadIdx.x == 0) partials[mt.part0 + t.ti] = b;
}

// Writes the first step's X (padded with zeros; the transpose of a tall
// matrix), scaled by the power of two that brings the norm into [2^13, 2^14):
// exact for bf16 but for elements below 2^-28 of the norm. A block turns one
// 64 x 64 tile. Each block adds its matrix's partial sums again (at most
// kMaxParts of them), in a fixed order, so every block has the same norm; the
// matrix's first block stores alpha.
template <int D, int SEG>
__global__ void __launch_bounds__(256) ns_convert_kernel(const NsMatrix *mats, const NsTile *tiles, const void *src,
                                                         const double *partials, NsScale *scales,
                                                         half_t *ws, const zds_step_scalars *sc) {
  if (sc && sc->overflow) return;
  __shared__ float sh[kConvTile][kConvTile + 1];
  __shared__ double ssum;
  const NsTile t = tiles[blockIdx.x];
  const NsMatrix mt = mats[t.mat];
  constexpr int ES = D == ZDS_FP32 ? 4 : 2;
  const char *base = static_cast<const char *>(src) + mt.offset * ES;
  // tile (ti, tj) of the rows x cols matrix as it lies in src: two eights of a
  // row for each thread, their loads under way while the norm is added up
  const int r0 = t.ti * kConvTile, c0 = t.tj * kConvTile;
  const int tr = threadIdx.x >> 3, tc = (threadIdx.x & 7) * 8;
  float v[2][8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = r0 + tr + 32 * h, c = c0 + tc;
    const int64_t e = static_cast<int64_t>(r) * mt.cols + c;
    if (r < mt.rows && c + 8 <= mt.cols) {
      load_eight<D>(base + e * ES, v[h]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[h][j] = r < mt.rows && c + j < mt.cols ? widen1<D>(base, e + j) : 0.0f;
    }
  }
  double acc = 0.0;
  for (int i = threadIdx.x; i < mt.nparts; i += 256) acc += partials[mt.part0 + i];
  const double tot = block_sum<256>(acc);
  if (threadIdx.x == 0) ssum = tot;
  __syncthreads();
  const double norm = sqrt(ssum);
  int ex = 0;
  (void)frexp(norm, &ex);
  int p2 = norm > 0.0 && norm <= DBL_MAX ? 14 - ex : 0;
  p2 = p2 > 126 ? 126 : (p2 < -126 ? -126 : p2);
  const float up = ldexpf(1.0f, p2);
  if (t.ti == 0 && t.tj == 0 && threadIdx.x == 0)
    scales[t.mat].alpha = static_cast<float>(ldexp(1.0 / (norm + kNormEps), -p2));
  const int64_t plane = static_cast<int64_t>(mt.mp) * mt.np;
  half_t *x = ws + mt.x[0];
  auto put = [&](int64_t e, const float (&f)[8]) {
    f16x8 h, l;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const HalfPair y = split(f[j] * up);
      h[j] = y.high;
      l[j] = y.low;
    }
    *reinterpret_cast<f16x8 *>(x + e) = h;
    if (SEG == 3) *reinterpret_cast<f16x8 *>(x + plane + e) = l;
  };
  if (!mt.tall) {
#pragma unroll
    for (int h = 0; h < 2; ++h) put(static_cast<int64_t>(r0 + tr + 32 * h) * mt.np + c0 + tc, v[h]);
    return;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 8; ++j) sh[tr + 32 * h][tc + j] = v[h][j];
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = sh[tc + j][tr + 32 * h];
    put(static_cast<int64_t>(c0 + tr + 32 * h) * mt.np + r0 + tc, u);
  }
}

// ---------------------------------------------------------------------------
// The products
// ---------------------------------------------------------------------------
//
// One kernel for the three: C = P Q^T in tiles of T x T, a block of four waves
// a tile, the operands' tiles of 64 deep through LDS. What bounds it is the
// card's power: with the matrix units 68 to 80 % busy the clock falls to 1.6 -
// 1.75 GHz of 2.4 (B X at 8192 x 22016: 2.31 ms, 1.28 PFLOP/s; a library
// product of two large fp16 matrices reaches 1.4 - 1.5 on the same card). So
// the shape is the one that moves the fewest bytes per product:
// - T = 256, a wave 128 x 128 of it in 256 accumulator registers: an operand
//   element read from LDS serves 128 products. 16 x 16 x 32 instructions
//   (32 x 32 x 16 ones: 23.2 ms instead of 22.2 for the MLP of a 65B layer).
// - Loads go from global memory straight to LDS, each placed right behind a
//   product, P's and Q's in turn, so that two barriers a step are enough and
//   neither waits for a load that was just issued.
// - X lies in one orientation only (transposing LDS reads for B X).
// - The epilogue reads and writes whole 16-byte rows through strips in LDS,
//   the inputs of four strips under way at once.
// Smaller tiles where there are too few of 256 to fill the units; which, the
// cost of the launches decides (kCosts). Small matrices are bound by the
// launches' latency (about 5 us each, 17 in a call of five steps).

// kGramPiece, kPolyPiece: pieces of cut tiles.
enum NsKind { kGram = 0, kPoly = 1, kUpdate = 2, kLast = 3, kGramPiece = 4, kPolyPiece = 5 };

struct NsArgs {
  const NsMatrix *mats;
  const NsTile *tiles;
  const NsScale *scales;
  half_t *ws;
  void *dst;
  const zds_step_scalars *sc;
  float *pieces;       // of cut tiles: accumulators as the threads hold them
  float a, b, c;       // the step's coefficients (a: with B's shift)
  float al, alb;       // X's remainder in row i counts al + alb B_ii (as stored) times, where B X leaves it out
  float shift;         // subtracted from B's diagonal, as stored
  float sa, sb, sx;    // powers of two: A, B and X (but the first) as stored
  int32_t first;       // the first step: X is scaled by its own alpha
  int32_t odd;         // which X is read
};

// A block of four waves computes a T x T tile, each wave a quarter. STAGES
// depth steps lie in LDS at once: as many as fit for T = 192 (three against
// two: 1307 and 1330 us for a 4096 x 4096 matrix).
template <int T, int STAGES_ = T == 192 ? 3 : 2>
struct NsShape {
  static constexpr int WAVES = 4;
  static constexpr int TW = T / 2;                 // a wave's part of the tile, TW x TW
  static constexpr int MT = 16;                    // the matrix instruction's tile, 16 x 16 x 32
  static constexpr int MI = TW / MT;
  static constexpr int LOADS = T / 8 / WAVES;      // 1 KiB loads of a wave per operand and depth step
  static constexpr int STAGE = T * 128;            // bytes of an operand's tile in LDS
  static constexpr int STAGES = STAGES_;
  // tiles of 192 may hang over the padded sizes
  static constexpr bool OVER = T == 192;
  // the epilogue's strip: MT rows of the wave's part, 16 bits an element, in
  // LDS rows of a power of two
  static constexpr int CHUNKS = T == 192 ? 16 : TW / 8, ROW = CHUNKS * 16;
  static constexpr int STRIP = MT * ROW;
  static constexpr int MOVES = STRIP / 1024;       // 1 KiB accesses of a wave per strip
  static constexpr int AHEAD = OVER ? 3 : MI < 4 ? MI : 4;  // strips in LDS, two planes each
};

// Positions of the 16-byte chunks in LDS, so that one access of a wave falls on
// all banks alike. An operand read as it lies: tile rows of 128 bytes, 16 (or
// 32) rows read at one chunk.
__device__ __forceinline__ int ns_swizzle(int row, int chunk) { return chunk ^ ((row >> 1) & 7); }
// X in B X: 64 rows of 2 T bytes; half a wave's transposing read takes 32 bytes
// of each of 8 rows (r..r+3, r+8..r+11), here from all 64 banks (with the rows
// 64 bytes apart instead, conflicts held the LDS for 10 % of the time).
template <int T>
__device__ __forceinline__ int ns_swizzle_x(int row, int chunk) {
  if (T > 64) return chunk ^ (((row & 3) | ((row >> 1) & 4)) << 1);
  return chunk ^ ((((row >> 1) & 1) | ((row >> 2) & 2)) << 1);
}
// A strip of the epilogue, written by columns and read by rows.
template <int T>
__device__ __forceinline__ int ns_swizzle_strip(int row, int chunk) { return chunk ^ (row & (NsShape<T>::CHUNKS - 1)); }

// Four rows of 16-bit columns turned: within 16 lanes, lane i addresses 8 bytes
// of row i / 4 and receives column i of the four rows.
__device__ __forceinline__ f16x4 read_turned(const char *p) {
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  return __builtin_bit_cast(f16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p)));
}

// 16 bytes a lane from global memory to LDS, 1 KiB from LDS address `lds` on in
// lane order. Written out, because the compiler takes every transposing read
// for a reader of what its own form of this load brings and waits for all
// loads in front of each. It has no output register; the waits are this
// file's own, and so is the wait state between the write of m0 and its use.
__device__ __forceinline__ void to_lds(const void *global, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(global), "{m0}"(lds) : "memory");
}
// 4 bytes a lane, 256 from `lds` on.
__device__ __forceinline__ void diag_to_lds(const void *global, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(global), "{m0}"(lds) : "memory");
}
// The same as to_lds in the form that costs the wave no address arithmetic: a buffer
// descriptor (base, size in bytes: an access behind it loads nothing), a
// lane's offset and the load's.
__device__ __forceinline__ u32x4 buffer_at(const void *p, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  return u32x4{static_cast<uint32_t>(a), static_cast<uint32_t>(a >> 32) & 0xffffu, bytes, 0x00027000u};
}
__device__ __forceinline__ void buffer_to_lds(u32x4 desc, uint32_t lane_off, uint32_t off, uint32_t lds) {
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds" ::"v"(lane_off), "s"(desc), "s"(off), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ uint32_t lds_address(const void *p) {
  return __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_void *)p)));
}
// Waits until at most n of the wave's memory accesses are under way (n is a
// constant once the caller's loop is unrolled).
__device__ __forceinline__ void wait_loads(int n) {
  asm volatile("" ::: "memory");
  // vmcnt in bits 3:0 and 15:14, the other counters at their maxima
  switch (n < 63 ? n : 63) {
#define ZDS_WAIT(k) case k: __builtin_amdgcn_s_waitcnt(0x0f70 | ((k) & 15) | ((k) >> 4) << 14); break;
#define ZDS_WAIT4(k) ZDS_WAIT(k) ZDS_WAIT(k + 1) ZDS_WAIT(k + 2) ZDS_WAIT(k + 3)
#define ZDS_WAIT16(k) ZDS_WAIT4(k) ZDS_WAIT4(k + 4) ZDS_WAIT4(k + 8) ZDS_WAIT4(k + 12)
    ZDS_WAIT16(0) ZDS_WAIT16(16) ZDS_WAIT16(32) ZDS_WAIT16(48)
#undef ZDS_WAIT16
#undef ZDS_WAIT4
#undef ZDS_WAIT
  }
  asm volatile("" ::: "memory");
}
__device__ __forceinline__ void block_barrier() {
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// PAIR: matrices whose A and B are pairs may be among a BF16 launch's
// (NsMatrix::pair).
template <int T, int SEG, int WHAT, int STAGES, bool PAIR>
__global__ void __launch_bounds__(256, T >= 192 || STAGES > 2 ? 1 : 2) ns_product_kernel(const NsArgs q) {
  typedef NsShape<T, STAGES> S;
  constexpr bool CUT = WHAT == kGramPiece || WHAT == kPolyPiece;
  constexpr int KIND = WHAT == kGramPiece ? kGram : WHAT == kPolyPiece ? kPoly : WHAT;
  constexpr bool TURN = KIND == kUpdate || KIND == kLast;  // P is X, read down its rows
  constexpr bool REST = SEG == 1 && TURN;  // X's remainder stands beside the product
  __shared__ __align__(1024) char smem[S::STAGES][2][S::STAGE];
  __shared__ __align__(256) uint32_t diag[REST ? T : 64];  // B's diagonal in the tile's rows, in one half each
  if (q.sc && q.sc->overflow) return;
  const NsTile t = q.tiles[blockIdx.x];
  const NsMatrix mt = q.mats[t.mat];  // all of it now: the waits below count every access
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wi = w >> 1, wj = w & 1;
  const float alpha = q.first ? q.scales[t.mat].alpha : 1.0f / q.sx;
  const int64_t mp = mt.mp, np = mt.np;
  const int64_t xplane = mp * np, aplane = mp * mp;
  // C = P Q^T, tile (ti, tj): rows of P are columns of what is stored
  half_t *const xin = q.ws + (q.odd ? mt.x[1] : mt.x[0]);
  half_t *const xout = q.ws + (q.odd ? mt.x[0] : mt.x[1]);
  const half_t *const P = KIND == kPoly ? q.ws + mt.a : xin;
  const half_t *const Q = KIND == kGram ? xin : q.ws + (KIND == kPoly ? mt.a : mt.b);
  const int64_t pld = KIND == kPoly ? mp : np, qld = KIND == kGram ? np : mp;
  const int64_t pplane = KIND == kPoly ? aplane : xplane, qplane = KIND == kGram ? xplane : aplane;
  const int steps = (KIND == kGram ? mt.np : mt.mp) / kNsDepth;
  const bool pair = PAIR && mt.pair;
  // X's remainder; as an operand's low half it is read while others write theirs
  half_t *const lo_in = q.ws + mt.lo + (pair && q.odd ? xplane : 0);
  half_t *const lo_out = q.ws + mt.lo + (pair && !q.odd ? xplane : 0);
  const int all = steps * (!pair || KIND == kGram ? SEG : TURN && q.first ? 2 : 3);
  const int from = CUT ? t.part * all / t.parts : 0;  // depth steps of this piece
  const int total = CUT ? (t.part + 1) * all / t.parts : all;

  f32x4 acc[S::MI][S::MI];
#pragma unroll
  for (int i = 0; i < S::MI; ++i)
#pragma unroll
    for (int j = 0; j < S::MI; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // Loads of a depth step: global to LDS without passing through registers.
  // The LDS side of a load is linear (1 KiB), so the lane takes the chunk that
  // belongs at its position. Load r of wave w is piece w + 4 r of the tile; the
  // swizzle of its rows is the same for every r, but for X at T = 256, where
  // it alternates.
  const int lrow = w * 8 + (lane >> 3);
  const uint32_t q_off = static_cast<uint32_t>(lrow * qld * 2 + ns_swizzle(lrow, lane & 7) * 16);
  const uint32_t q_step = static_cast<uint32_t>(32 * qld * 2);
  constexpr int XC = T / 8;  // chunks of a row of X's tile
  const int xrow = w * (64 / XC) + lane / XC;
  uint32_t p_off[2];
#pragma unroll
  for (int v = 0; v < 2; ++v)
    p_off[v] = TURN ? static_cast<uint32_t>(xrow * pld * 2 + ns_swizzle_x<T>(xrow + v * 8 * (T == 256), lane % XC) * 16)
                    : static_cast<uint32_t>(lrow * pld * 2 + ns_swizzle(lrow, lane & 7) * 16);
  const uint32_t p_step = static_cast<uint32_t>((TURN ? 256 / XC : 32) * pld * 2);
  // a tile that hangs over: load r's offsets, with the last row in place of rows
  // that are not there
  uint32_t p_over[S::LOADS], q_over[S::LOADS];
#pragma unroll
  for (int r = 0; S::OVER && r < S::LOADS; ++r) {
    const int row = lrow + 32 * r, pl = mt.mp - t.ti * T - 1, ql = mt.mp - t.tj * T - 1;
    p_over[r] = static_cast<uint32_t>((row < pl ? row : pl) * pld * 2 + ns_swizzle(lrow, lane & 7) * 16);
    q_over[r] = static_cast<uint32_t>((row < ql ? row : ql) * qld * 2 + ns_swizzle(lrow, lane & 7) * 16);
  }
  const auto lane_p = [&](int r) { return S::OVER ? p_over[r] : p_off[r & 1]; };
  const auto lane_q = [&](int r) { return S::OVER ? q_over[r] : q_off; };
  const auto load_at = [&](int r, uint32_t step) { return S::OVER ? 0u : static_cast<uint32_t>(r * step); };
  const half_t *const p0 = P + (TURN ? static_cast<int64_t>(t.ti) * T : static_cast<int64_t>(t.ti) * T * pld);
  const half_t *const q0 = Q + static_cast<int64_t>(t.tj) * T * qld;
  const int64_t plow = pair && TURN ? lo_in - P : pplane;  // P's low half
  // the operands of depth step k; behind the last step nothing is loaded
  u32x4 pk, qk;
  auto aim = [&](int k) {
    int seg = 2, kk = k < total ? k : total - 1;
    if (SEG == 3 || (pair && KIND != kGram)) {  // P's low*high, high*Q's low, high*high: the small sums first
      seg = (kk >= steps) + (kk >= 2 * steps);
      kk -= seg * steps;
      if (pair && TURN && q.first) ++seg;  // the first X has no low half
    }
    const uint32_t bytes = k < total ? 0x80000000u : 0u;
    pk = buffer_at(p0 + (seg == 0 ? plow : 0) + static_cast<int64_t>(kk) * kNsDepth * (TURN ? pld : 1), bytes);
    qk = buffer_at(q0 + (seg == 1 ? qplane : 0) + static_cast<int64_t>(kk) * kNsDepth, bytes);
  };
  const uint32_t lds0 = lds_address(smem) + w * 1024;
  // Operand pieces in registers: P's of this half of a depth step and the next,
  // half of Q's of a half step and the next half of them.
  constexpr int NQ = S::MI / 2;
  const int fr = lane & 15, fc = lane >> 4;
  f16x8 fp[2][S::MI], fq[2][NQ];
  int off_p[2], off_q[2], off_x[S::MI];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int rp = wi * S::TW + fr, rq = wj * S::TW + fr;
    off_p[h] = rp * 128 + ns_swizzle(rp, h * 4 + fc) * 16;
    off_q[h] = rq * 128 + ns_swizzle(rq, h * 4 + fc) * 16;
  }
#pragma unroll
  for (int r = 0; r < S::MI; ++r) {
    const int row = 8 * fc + (fr >> 2), col = wi * S::TW + r * S::MT + (lane & 3) * 4;
    off_x[r] = row * 2 * T + ns_swizzle_x<T>(row, col >> 3) * 16 + (col & 4) * 2;
  }
  // piece r of half h of P
  auto read_p = [&](int buf, int h, int r) {
    if constexpr (TURN) {
      const char *x = smem[buf][0] + off_x[r] + h * 32 * 2 * T;
      const f16x4 a = read_turned(x), b = read_turned(x + 4 * 2 * T);
      fp[h][r] = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
      fp[h][r] = *reinterpret_cast<const f16x8 *>(smem[buf][0] + off_p[h] + r * 128 * S::MT);
    }
  };
  // piece r of quarter u of Q: the quarter's half u / 2, its pieces (u % 2) NQ on
  auto read_q = [&](int buf, int u, int r) {
    fq[u & 1][r] = *reinterpret_cast<const f16x8 *>(smem[buf][1] + off_q[u >> 1] + ((u & 1) * NQ + r) * 128 * S::MT);
  };
  constexpr int PER = S::MI * NQ, HALF = 2 * PER;  // products of a quarter, of a half step
  auto load_p = [&](int buf, int r) {
    buffer_to_lds(pk, lane_p(r), load_at(r, p_step), lds0 + buf * 2 * S::STAGE + r * 4096);
  };
  auto load_q = [&](int buf, int r) {
    buffer_to_lds(qk, lane_q(r), load_at(r, q_step), lds0 + (buf * 2 + 1) * S::STAGE + r * 4096);
  };
  // A product, and right behind it a load, for which the product stands in as
  // the wait state behind the write of m0. The accumulators are updated in
  // place by an instruction written out: left to itself the compiler copies
  // all 256 of them in every step. (It knows the registers but not the
  // instruction's latency: nothing reads them before the wait behind the
  // loop.)
  auto product = [&](int u, int e) {
    const int i = e / NQ, j = e % NQ;
    asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0"
                 : "+a"(acc[i][(u & 1) * NQ + j])
                 : "v"(fp[u >> 1][i]), "v"(fq[u & 1][j]));
  };
  auto product_load = [&](int u, int e, bool is_p, int buf, int r) {
    const int i = e / NQ, j = e % NQ;
    const uint32_t at = lds0 + (buf * 2 + !is_p) * S::STAGE + r * 4096;
    asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0\n\tbuffer_load_dwordx4 %3, %4, %5 offen lds"
                 : "+a"(acc[i][(u & 1) * NQ + j])
                 : "v"(fp[u >> 1][i]), "v"(fq[u & 1][j]), "v"(is_p ? lane_p(r) : lane_q(r)), "s"(is_p ? pk : qk),
                   "s"(load_at(r, is_p ? p_step : q_step)), "{m0}"(at)
                 : "memory");
  };
  // A depth step is four quarters u: two halves in depth, and in each the two
  // halves of Q's pieces. Between the products stand
  // - the reads of P's next half and of Q's next quarter, done an eighth before
  //   the end of what they stand in;
  // - the loads of step k + 2: P's behind the barrier in the middle of step k
  //   (both halves of P have been read then), Q's behind the next, a quarter
  //   later, into the next step's first half.
  // A barrier waits for the loads that the reads behind it need: P's of step
  // k + 1 in the middle (Q's are younger), Q's of step k + 1 a quarter later
  // (but for the first of P's of step k + 2 they are the youngest). Behind the
  // last steps the reads find tiles that are there and not used.
  constexpr int WINDOW = HALF * 3 / 4;  // products that an operand's loads are spread over
  constexpr auto at_p = [](int i) { return i * WINDOW / S::LOADS; };
  constexpr auto at_q = [](int i) { return WINDOW + i * WINDOW / S::LOADS; };
  constexpr auto before = [](auto at, int x) {
    int n = 0;
    for (int i = 0; i < S::LOADS; ++i) n += at(i) < x;
    return n;
  };
  constexpr int YOUNGER = before(at_p, PER);  // P's loads in front of the second barrier
  constexpr int EARLY = before(at_q, HALF);   // Q's loads in front of a step's first half
  // the place in LDS of step k + d
  int turn = from % S::STAGES;
  auto stage = [&](int k, int d) {
    if ((S::STAGES & (S::STAGES - 1)) == 0) return (k + d) & (S::STAGES - 1);
    return turn + d < S::STAGES ? turn + d : turn + d - S::STAGES;
  };
  auto quarter = [&](int k, auto which) {
    constexpr int u = decltype(which)::value, h = u >> 1;
    const int buf = stage(k, 0), next = stage(k, 1), last = stage(k, S::STAGES - 1);
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const int x = (u & 1) * PER + e;  // place in the half
      int is_p = -1, is_q = -1;
#pragma unroll
      for (int i = 0; i < S::LOADS; ++i) {
        if (h == 1 && at_p(i) == x) is_p = i;
        if (at_q(i) == x + (h == 1 ? 0 : HALF)) is_q = i;
      }
      if (is_p >= 0) product_load(u, e, true, buf, is_p);
      else if (is_q >= 0) product_load(u, e, false, h == 1 ? buf : last, is_q);
      else product(u, e);
#pragma unroll
      for (int r = 0; r < NQ; ++r)
        if (r * (PER - PER / 8) / NQ == e) read_q(u == 3 ? next : buf, (u + 1) & 3, r);
#pragma unroll
      for (int r = 0; r < S::MI; ++r)
        if (r * (HALF - HALF / 8) / S::MI == x) read_p(h ? next : buf, h ^ 1, r);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  if (REST && w * 64 < T) {  // (older than all that the waits below count)
    const int64_t row = static_cast<int64_t>(t.tj) * T + w * 64 + lane;
    diag_to_lds(Q + row * mp + (row & ~1), lds_address(diag) + w * 256);
  }
#pragma unroll
  for (int d = 0; d < S::STAGES; ++d) {
    aim(from + d);
#pragma unroll
    for (int g = 0; g < S::LOADS; ++g) load_p(stage(from, d), g);
#pragma unroll
    for (int g = 0; g < (d + 1 < S::STAGES ? S::LOADS : EARLY); ++g) load_q(stage(from, d), g);
  }
  constexpr int BEHIND = 2 * S::LOADS * (S::STAGES - 2);  // loads of whole steps behind the next
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(BEHIND + S::LOADS + EARLY) : "memory");
  block_barrier();
#pragma unroll
  for (int g = 0; g < S::MI; ++g) read_p(stage(from, 0), 0, g);
#pragma unroll
  for (int g = 0; g < NQ; ++g) read_q(stage(from, 0), 0, g);
  auto depth_step = [&](int k) {
    quarter(k, std::integral_constant<int, 0>{});
    quarter(k, std::integral_constant<int, 1>{});
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(BEHIND + S::LOADS) : "memory");
    block_barrier();
    aim(k + S::STAGES);
    quarter(k, std::integral_constant<int, 2>{});
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(BEHIND + YOUNGER) : "memory");
    block_barrier();
    quarter(k, std::integral_constant<int, 3>{});
    turn = stage(k, 1);
  };
  if constexpr (CUT) {
    int k = from;  // every piece has a step
    do depth_step(k);
    while (++k < total);
  } else {
    for (int k = 0; k < total; ++k) depth_step(k);
  }
  asm volatile("s_nop 15\n\ts_nop 15\n\ts_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  block_barrier();

  // A piece of a cut tile leaves its sums in memory, for ns_join_kernel.
  if constexpr (CUT) {
    f32x4 *mine = reinterpret_cast<f32x4 *>(q.pieces) + (static_cast<int64_t>(t.slot) * t.parts + t.part) * (T * T / 4) + threadIdx.x;
#pragma unroll
    for (int i = 0; i < S::MI; ++i)
#pragma unroll
      for (int j = 0; j < S::MI; ++j) mine[(i * S::MI + j) * 256] = acc[i][j];
  } else {

  // Epilogue, in strips of MT rows of what is stored, each wave on its own in
  // its part of the LDS (room for AHEAD strips). A lane holds row fr of a strip,
  // of each instruction tile i four elements from column 16 i + 4 fc on. The
  // strip's inputs come in rows (high and low plane) and are overwritten by its
  // outputs, which leave in rows, and for a symmetric result also turned.
  char *const room = smem[0][0] + w * S::AHEAD * 2 * S::STRIP;
  const uint32_t room_lds = lds_address(room);
  static_assert(4 * S::AHEAD * 2 * S::STRIP <= 4 * S::STAGE, "each wave's strips fit");
  const int64_t prow = static_cast<int64_t>(t.ti) * T + wi * S::TW;  // first column of the wave's part
  const int64_t qrow = static_cast<int64_t>(t.tj) * T + wj * S::TW;  // first row
  const int64_t old = TURN ? np : mp;
  const int64_t here = qrow * old + prow;
  const half_t *in_h = TURN ? xin : q.ws + mt.a;
  const half_t *in_l = SEG == 3 || (pair && !TURN) ? in_h + (TURN ? xplane : aplane) : lo_in;
  const bool low_in = SEG == 3 || (TURN ? !q.first : pair);
  constexpr int RPI = 64 / S::CHUNKS;  // rows of a 1 KiB access
  constexpr int GR = S::MT / 8;        // groups of 8 rows in a strip
  constexpr int PC = 64 / GR;          // columns that a wave's turned access covers
  int sl, mrow, mchunk, tgrp, tcol;
  // The lane's places, taken anew for every strip: kept for all of them the
  // addresses cost registers that the accumulators need.
  auto places = [&] {
    sl = lane;
    asm volatile("" : "+v"(sl));
    mrow = sl / S::CHUNKS;
    mchunk = sl % S::CHUNKS;
    tgrp = (sl >> 4) % GR * 8;
    tcol = (sl >> 4) / GR * 16 + (sl & 15);
  };
  // what the lane loads of strip s in access g; where nothing is, from a place
  // that is there
  auto source = [&](int s, int g) {
    const int r = g * RPI + mrow, c = ns_swizzle_strip<T>(r, mchunk);
    if (!S::OVER) return r * old + c * 8;
    const int64_t last = mp - 1 - (qrow + s * S::MT);
    return (r < last ? r : last) * old + (c < S::TW / 8 && prow + c * 8 < mp ? c * 8 : 0);
  };
  auto fetch = [&](int s) {
    if (KIND == kGram) return;
    const uint32_t at = room_lds + s % S::AHEAD * 2 * S::STRIP;
    const half_t *h = in_h + here + s * S::MT * old, *l = in_l + here + s * S::MT * old;
#pragma unroll
    for (int g = 0; g < S::MOVES; ++g) to_lds(h + source(s, g), at + g * 1024);
    if (low_in) {
#pragma unroll
      for (int g = 0; g < S::MOVES; ++g) to_lds(l + source(s, g), at + S::STRIP + g * 1024);
    }
  };
  // rows of plane `at` to global memory
  auto put_rows = [&](const char *at, half_t *out, int s) {
    half_t *o = out + here + s * S::MT * old;
#pragma unroll
    for (int g = 0; g < S::MOVES; ++g) {
      const int r = g * RPI + mrow;
      const f16x8 v = *reinterpret_cast<const f16x8 *>(at + r * S::ROW + ns_swizzle_strip<T>(r, mchunk) * 16);
      if (!S::OVER || (mchunk < S::TW / 8 && prow + mchunk * 8 < mp && qrow + s * S::MT < mp))
        *reinterpret_cast<f16x8 *>(o + r * old + mchunk * 8) = v;
    }
  };
  // eight rows of plane `at` from row r on, turned: column col of them
  auto turned8 = [&](const char *at, int r, int col) {
    // within the lane's group of 16: row (lane & 15) / 4, columns 4 (lane & 3) on
    const int cc = (col & ~15) + (sl & 3) * 4, ra = r + ((sl & 15) >> 2), rb = ra + 4;
    const f16x4 a = read_turned(at + ra * S::ROW + ns_swizzle_strip<T>(ra, cc >> 3) * 16 + (cc & 4) * 2);
    const f16x4 b = read_turned(at + rb * S::ROW + ns_swizzle_strip<T>(rb, cc >> 3) * 16 + (cc & 4) * 2);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  auto put_turned = [&](const char *at, half_t *out, int s) {
    half_t *o = out + prow * old + qrow + s * S::MT;
#pragma unroll
    for (int c = 0; c < S::TW; c += PC) {
      const f16x8 v = turned8(at, tgrp, c + tcol);
      if (!S::OVER || (prow + c + tcol < mp && qrow + s * S::MT < mp))
        *reinterpret_cast<f16x8 *>(o + (c + tcol) * old + tgrp) = v;
    }
  };
  places();
#pragma unroll
  for (int s = 0; s < S::AHEAD; ++s) fetch(s);
#pragma unroll
  for (int s = 0; s < S::MI; ++s) {
    char *at = room + s % S::AHEAD * 2 * S::STRIP;
    places();
    const int fr = sl & 15, fc = sl >> 4;
    if (KIND != kGram) {
      // wait for the strip's loads only: behind them stand the loads of the
      // AHEAD - 1 next strips and the stores of as many (at least STORES each)
      // (a wave whose tile hangs over may skip its stores)
      constexpr int STORES = S::OVER ? 0 : KIND == kUpdate ? 2 * S::MOVES : KIND == kPoly ? SEG * S::MOVES : 0;
      const int left = S::MI - 1 - s < S::AHEAD - 1 ? S::MI - 1 - s : S::AHEAD - 1;
      const int gone = s < S::AHEAD - 1 ? s : S::AHEAD - 1;
      if (low_in) wait_loads(left * 2 * S::MOVES + gone * STORES);
      else wait_loads(left * S::MOVES + gone * STORES);
    }
    const char *line = at + fr * S::ROW;
    float f0 = 0.0f, f1, f2 = 0.0f;  // v = f0 high + f2 low + f1 acc
    if (KIND == kGram) {
      f1 = alpha * alpha * q.sa;
    } else if (KIND == kPoly) {
      f0 = f2 = q.b * (q.sb / q.sa);
      f1 = q.c * (q.sb / (q.sa * q.sa));
    } else {
      const float os = KIND == kLast ? 1.0f : q.sx;
      f0 = q.a * alpha * os;
      f2 = f0;
      if (REST && !pair) {
        const uint32_t both = diag[wj * S::TW + s * S::MT + fr];
        f2 = (q.al + q.alb * __builtin_bit_cast(f16x2, both)[fr & 1]) * alpha * os;
      }
      f1 = alpha / q.sb * os;
    }
#pragma unroll
    for (int i = 0; i < S::MI; ++i) {
        const int col = i * S::MT + fc * 4;
        char *p = const_cast<char *>(line) + ns_swizzle_strip<T>(fr, col >> 3) * 16 + (col & 4) * 2;
        f16x4 h = {}, l = {};
        if (KIND != kGram) h = *reinterpret_cast<const f16x4 *>(p);
        if (KIND != kGram && low_in) l = *reinterpret_cast<const f16x4 *>(p + S::STRIP);
        float v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          v[r] = f1 * acc[i][s][r];
          if (KIND != kGram) v[r] += f0 * static_cast<float>(h[r]) + f2 * static_cast<float>(l[r]);
          if (KIND == kPoly && qrow + s * S::MT + fr == prow + col + r) v[r] -= q.shift;
        }
        if constexpr (KIND == kLast) {
          if constexpr (SEG == 1) {
            const u32x2 o = {pack2<ZDS_BF16>(v[0], v[1]), pack2<ZDS_BF16>(v[2], v[3])};
            *reinterpret_cast<u32x2 *>(p) = o;
          } else {
            // fp32: straight from the registers
            const int64_t i0 = qrow + s * S::MT + fr, j0 = prow + col;
            if (i0 < mt.m) {
#pragma unroll
              for (int r = 0; r < 4; ++r)
                if (j0 + r < mt.n)
                  static_cast<float *>(q.dst)[mt.offset + (mt.tall ? (j0 + r) * mt.cols + i0 : i0 * mt.cols + j0 + r)] = v[r];
            }
          }
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const HalfPair y = split(v[r]);
            h[r] = y.high;
            l[r] = y.low;
          }
          *reinterpret_cast<f16x4 *>(p) = h;
          if (SEG == 3 || KIND == kUpdate || pair) *reinterpret_cast<f16x4 *>(p + S::STRIP) = l;
        }
      }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if constexpr (KIND == kGram || KIND == kPoly) {
      half_t *out = q.ws + (KIND == kGram ? mt.a : mt.b);
      put_rows(at, out, s);
      if (SEG == 3 || pair) put_rows(at + S::STRIP, out + aplane, s);
      if (t.ti != t.tj) {
        put_turned(at, out, s);
        if (SEG == 3 || pair) put_turned(at + S::STRIP, out + aplane, s);
      }
    } else if constexpr (KIND == kUpdate) {
      put_rows(at, xout, s);
      put_rows(at + S::STRIP, SEG == 3 ? xout + xplane : lo_out, s);
    } else if constexpr (SEG == 1) {
      // the result, in its own orientation and inside its bounds
      uint16_t *dst = static_cast<uint16_t *>(q.dst) + mt.offset;
      const int64_t i0 = qrow + s * S::MT, j0 = prow;
      auto put = [&](int64_t row, int64_t col, u32x4 v) {
        if (row >= mt.rows || col >= mt.cols) return;
        uint16_t *o = dst + row * mt.cols + col;
        if (col + 8 <= mt.cols) {
          *reinterpret_cast<u32x4_any *>(o) = v;
        } else {
#pragma unroll
          for (int j = 0; j < 7; ++j)
            if (col + j < mt.cols) o[j] = static_cast<uint16_t>(v[j / 2] >> (j & 1) * 16);
        }
      };
      if (!mt.tall) {
#pragma unroll
        for (int g = 0; g < S::MOVES; ++g) {
          const int r = g * RPI + mrow;
          put(i0 + r, j0 + mchunk * 8,
              *reinterpret_cast<const u32x4 *>(at + r * S::ROW + ns_swizzle_strip<T>(r, mchunk) * 16));
        }
      } else {
#pragma unroll
        for (int c = 0; c < S::TW; c += PC)
          put(j0 + c + tcol, i0 + tgrp, __builtin_bit_cast(u32x4, turned8(at, tgrp, c + tcol)));
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (s + S::AHEAD < S::MI) fetch(s + S::AHEAD);
  }
  }
}

// The sums of cut tiles: block (k, j) adds, in the pieces' order, column j of
// the instruction tiles of each wave's part of tile k, and stores it and its
// mirror image. POLY: b A + c A^2, else A.
template <int T, int SEG, bool POLY>
__global__ void __launch_bounds__(256) ns_join_kernel(const NsArgs q, int parts) {
  typedef NsShape<T> S;
  if (q.sc && q.sc->overflow) return;
  const NsTile t = q.tiles[blockIdx.x];
  const NsMatrix mt = q.mats[t.mat];
  const int j = blockIdx.y, lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t mp = mt.mp, aplane = mp * mp;
  const f32x4 *o = reinterpret_cast<const f32x4 *>(q.pieces) + static_cast<int64_t>(t.slot) * parts * (T * T / 4) + threadIdx.x;
  f32x4 v[S::MI];
#pragma unroll
  for (int i = 0; i < S::MI; ++i) v[i] = o[(i * S::MI + j) * 256];
  for (int p = 1; p < parts; ++p) {
    o += T * T / 4;
#pragma unroll
    for (int i = 0; i < S::MI; ++i) v[i] += o[(i * S::MI + j) * 256];
  }
  const bool low = SEG == 3 || mt.pair;
  const float alpha = q.first ? q.scales[t.mat].alpha : 1.0f / q.sx;
  const float f1 = POLY ? q.c * (q.sb / (q.sa * q.sa)) : alpha * alpha * q.sa;
  half_t *const out = q.ws + (POLY ? mt.b : mt.a);
  const int64_t row = static_cast<int64_t>(t.tj) * T + (w & 1) * S::TW + j * S::MT + (lane & 15);
#pragma unroll
  for (int i = 0; i < S::MI; ++i) {
    const int64_t col = static_cast<int64_t>(t.ti) * T + (w >> 1) * S::TW + i * S::MT + (lane >> 4) * 4;
    const half_t *a = q.ws + mt.a + row * mp + col;
    f16x4 ah = {}, al = {}, h, l;
    if (POLY) ah = *reinterpret_cast<const f16x4 *>(a);
    if (POLY && low) al = *reinterpret_cast<const f16x4 *>(a + aplane);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float x = f1 * v[i][r];
      if (POLY) x += q.b * (q.sb / q.sa) * (static_cast<float>(ah[r]) + static_cast<float>(al[r]));
      if (POLY && row == col + r) x -= q.shift;
      const HalfPair y = split(x);
      h[r] = y.high;
      l[r] = y.low;
    }
    *reinterpret_cast<f16x4 *>(out + row * mp + col) = h;
    if (low) *reinterpret_cast<f16x4 *>(out + aplane + row * mp + col) = l;
    if (t.ti != t.tj) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        out[(col + r) * mp + row] = h[r];
        if (low) out[aplane + (col + r) * mp + row] = l[r];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// Largest |a s + b s^3 + c s^5| and |b s^2 + c s^4| over [0, top]: at the ends
// or where a slope is zero, a root of a quadratic in l = s^2. (Once for every
// step of every call: on 4097 samples a call of five steps took 60 us longer.)
static void poly_bound(const float *k, double top, double *x, double *bx) {
  const double a = k[0], b = k[1], c = k[2], end = top * top;
  *x = *bx = HUGE_VAL;
  if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return;
  const auto low = [&](double l) { return b * l + c * l * l; };
  *x = fabs(top * (a + low(end)));
  *bx = fabs(low(end));
  // 5 c l^2 + 3 b l + a = 0; the roots' products and sums in the order that cancels nothing
  const double d = 9.0 * b * b - 20.0 * a * c;
  if (d >= 0.0) {
    const double q = -0.5 * (3.0 * b + (b < 0.0 ? -sqrt(d) : sqrt(d)));
    for (double l : {q / (5.0 * c), a / q})
      if (l > 0.0 && l < end) *x = std::max(*x, fabs(sqrt(l) * (a + low(l))));
  }
  const double l = -b / (2.0 * c);
  if (l > 0.0 && l < end) *bx = std::max(*bx, fabs(low(l)));
}

// What is subtracted from B's diagonal as it is stored, and given back to X as
// (a + shift) X, which takes no rounding. In the last steps most singular
// values are near 1 and B near (b + c) I, so the rounding of its diagonal to
// fp16 would be the largest of all. The error of a BF16 result over that of
// rounding the exact one: 96 x 160 1.43 -> 1.26, 512 x 1024 1.29 -> 1.18; of an
// FP32 one: 0.9e-6 -> 0.7e-6 and 1.5e-6 -> 1.4e-6.
//
// The remainder of X that B X leaves out would count a + B times: a where
// singular values are small, and in the mean of a row's directions a + B_ii.
// It counts halfway between the two, whatever the coefficients.
static float shift_of(const float *coef, int step, int steps) {
  if (step + 3 < steps) return 0.0f;
  const float d = coef[3 * step + 1] + coef[3 * step + 2];
  return step + 1 < steps ? d : 0.5f * d;
}

static float pow2_under(double limit, double value) {  // largest power of two with p * value <= limit
  int e = 0;
  (void)frexp(limit / value, &e);
  return ldexpf(1.0f, e - 1);
}

// Tiles of 128 that have a unit each to themselves: four depth steps in LDS
// (2048 x 2048: X X^T 22.4 -> 19.4 us). Where two blocks share a unit two steps
// leave room for both (16 of 1100 x 1100: 42 us against 45).
constexpr int kAlone = 4;

template <int T, int SEG, int STAGES, bool PAIR>
static void launch_tiles(dim3 grid, const NsArgs &q, int kind, hipStream_t s) {
  const dim3 block(NsShape<T>::WAVES * 64);
  if (kind == kGram) {
    hipLaunchKernelGGL((ns_product_kernel<T, SEG, kGram, STAGES, PAIR>), grid, block, 0, s, q);
  } else if (kind == kPoly) {
    hipLaunchKernelGGL((ns_product_kernel<T, SEG, kPoly, STAGES, PAIR>), grid, block, 0, s, q);
  } else if constexpr (T != 192) {
    if (kind == kUpdate) hipLaunchKernelGGL((ns_product_kernel<T, SEG, kUpdate, STAGES, PAIR>), grid, block, 0, s, q);
    else hipLaunchKernelGGL((ns_product_kernel<T, SEG, kLast, STAGES, PAIR>), grid, block, 0, s, q);
  }
}

template <int T, int SEG, bool PAIR>
static void launch_list(const NsList &l, const NsTile *tiles, NsArgs q, int kind, hipStream_t s) {
  constexpr int STAGES = NsShape<T>::STAGES;
  if constexpr (T == 256 || T == 128) {
    if (l.cut) {
      const dim3 block(NsShape<T>::WAVES * 64);
      const dim3 pgrid(static_cast<uint32_t>(l.cut * l.parts)), jgrid(static_cast<uint32_t>(l.cut), NsShape<T>::MI);
      q.tiles = tiles + l.pieces;
      // (X X^T takes X's high halves only and leaves its sums to the join)
      if (kind == kGram) hipLaunchKernelGGL((ns_product_kernel<T, SEG, kGramPiece, STAGES, false>), pgrid, block, 0, s, q);
      else hipLaunchKernelGGL((ns_product_kernel<T, SEG, kPolyPiece, STAGES, PAIR>), pgrid, block, 0, s, q);
      q.tiles = tiles + l.join;
      if (kind == kGram) hipLaunchKernelGGL((ns_join_kernel<T, SEG, false>), jgrid, dim3(256), 0, s, q, l.parts);
      else hipLaunchKernelGGL((ns_join_kernel<T, SEG, true>), jgrid, dim3(256), 0, s, q, l.parts);
      if (!l.count) return;
    }
  }
  q.tiles = tiles + l.first;
  const dim3 grid(static_cast<uint32_t>(l.count));
  if constexpr (T == 128) {
    if (l.count <= kUnits) return launch_tiles<T, SEG, kAlone, PAIR>(grid, q, kind, s);
  }
  launch_tiles<T, SEG, STAGES, PAIR>(grid, q, kind, s);
}

template <int SEG>
static void launch_products(const NsGroup &g, const NsTile *tiles, const NsArgs &q, int kind, hipStream_t s) {
  const NsList &l = kind == kGram ? g.gram : kind == kPoly ? g.poly : g.full;
  constexpr bool P = SEG == 1;
  // (the larger tiles' kernels without pairs are a little shorter)
  if (l.tile == 64) launch_list<64, SEG, P>(l, tiles, q, kind, s);
  else if (l.tile == 256) P && g.pair ? launch_list<256, SEG, P>(l, tiles, q, kind, s) : launch_list<256, SEG, false>(l, tiles, q, kind, s);
  else if (l.tile == 192) P && g.pair ? launch_list<192, SEG, P>(l, tiles, q, kind, s) : launch_list<192, SEG, false>(l, tiles, q, kind, s);
  else P && g.pair ? launch_list<128, SEG, P>(l, tiles, q, kind, s) : launch_list<128, SEG, false>(l, tiles, q, kind, s);
}

// Rounds `n` tiles (already in an order whose neighbours share operands) so
// that the blocks of one die, those with the same index modulo 8, take
// neighbouring tiles: each round of 256 is cut into 8 runs.
static void spread_over_dies(std::vector<NsTile> &v, size_t from) {
  const std::vector<NsTile> in(v.begin() + static_cast<int64_t>(from), v.end());
  v.resize(from);
  for (size_t r = 0; r < in.size(); r += 256) {
    const size_t cnt = in.size() - r < 256 ? in.size() - r : 256;
    for (size_t k = 0; k < (cnt + 7) / 8; ++k)
      for (size_t x = 0; x < 8; ++x) {
        const size_t lo = x * cnt / 8, hi = (x + 1) * cnt / 8;
        if (lo + k < hi) v.push_back(in[r + lo + k]);
      }
  }
}

// Tiles in patches of 8 x 4, so that a run of 32 reads 8 + 4 operand tiles.
static void add_tiles(std::vector<NsTile> &v, int mat, int ni, int nj, bool triangle) {
  for (int pj = 0; pj < nj; pj += 4)
    for (int pi = 0; pi < ni; pi += 8)
      for (int j = pj; j < pj + 4 && j < nj; ++j)
        for (int i = pi; i < pi + 8 && i < ni; ++i)
          if (!triangle || i >= j) v.push_back(NsTile{mat, i, j, 0, 1, 0});
}

static int64_t round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

// Sizes are padded to a multiple of 256, 128 or 64: the largest that costs at
// most 15 % more of the full product than 64 does, since a larger tile reads
// its operands less often.
static int padding_of(int64_t m, int64_t n) {
  const auto work = [&](int64_t t) { return static_cast<double>(round_up(m, t)) * round_up(m, t) * round_up(n, t); };
  for (int t : {256, 128})
    if (work(t) <= 1.15 * work(64)) return t;
  return 64;
}

// What launches of T x T tiles take, in us, fitted to measured ones (1 to 2048
// tiles of 16 to 172 depth steps): a block's fixed part (a full product's
// epilogue also reads and writes X's low halves), and a step's time by how
// many blocks share a unit. X X^T at 1024 x 4096 (64 steps; 10 tiles of 256, 36
// of 128, 136 of 64) takes 71, 35 and 27 us, B X at 4096 x 4096 (64 steps; 256,
// 1024, 4096 tiles) 119, 131 and 244 us. Tiles of 192 are for X X^T and A A
// only: at 4096 x 4096 there are 253, one a unit (78 us), against 136 of 256 or
// 528 of 128 (94 us, the last 16 in pieces).
struct LaunchCost {
  int tile, blocks;  // blocks of a unit at once
  double fixed[4], full[4], step[4];
};
static const LaunchCost kCosts[4] = {
    {256, 1, {12.0}, {22.0}, {1.25}},
    {192, 1, {10.0}, {}, {0.95}},
    {128, 2, {5.0, 8.0}, {7.0, 11.0}, {0.45, 0.95}},
    {64, 4, {4.0, 5.0, 6.0, 7.5}, {5.5, 6.5, 8.0, 9.5}, {0.37, 0.5, 0.67, 0.85}},
};
static double round_cost(const LaunchCost &k, bool full, int64_t tiles, double steps) {
  const int64_t share = (tiles + kUnits - 1) / kUnits - 1;
  return (full ? k.full : k.fixed)[share] + steps * k.step[share];
}
// Storing and joining the pieces of cut tiles (4 MB of them take 7 us, 63 MB 20).
static double join_cost(int tile, int64_t pieces) {
  return 6.0 + 0.25e-6 * 4.0 * static_cast<double>(pieces) * tile * tile;
}
constexpr int kMaxPieces = 8;

// The tiles of a product over a group's matrices (which come in falling depth).
// Where the last round of blocks would leave units idle, its tiles' sums may be
// cut into pieces that fill it (of A and B; at 8192 x 22016, X X^T has 528
// tiles of 256: two rounds and 16 tiles). Returns the cost, and with `tiles`
// adds the list to it.
static double make_list(int kind, const std::vector<NsMatrix> &mats, int padding, int seg, NsList *l, std::vector<NsTile> *tiles) {
  const bool full = kind == kUpdate;
  double least = -1.0;
  for (const LaunchCost &k : kCosts) {
    if (k.tile > padding || (full && k.tile == 192)) continue;
    std::vector<std::pair<int64_t, double>> runs;  // tiles, steps
    int64_t n = 0;
    for (const NsMatrix &m : mats) {
      const int64_t a = (m.mp + k.tile - 1) / k.tile, b = m.np / k.tile;
      const int pieces = m.pair && kind != kGram ? 3 : seg;
      const double steps = static_cast<double>(pieces) * (kind == kGram ? m.np : m.mp) / kNsDepth;
      runs.emplace_back(full ? a * b : a * (a + 1) / 2, steps);
      n += runs.back().first;
    }
    // average depth of the last `tail` tiles, and of the ones in front
    const int64_t slots = static_cast<int64_t>(kUnits) * k.blocks, tail = n % slots, front = n - tail;
    double all = 0.0, behind = 0.0, least_steps = HUGE_VAL;
    int64_t left = tail;
    for (size_t i = runs.size(); i-- > 0;) {
      const int64_t c = std::min(left, runs[i].first);
      behind += static_cast<double>(c) * runs[i].second;
      if (c) least_steps = std::min(least_steps, runs[i].second);
      left -= c;
      all += static_cast<double>(runs[i].first) * runs[i].second;
    }
    const double whole = front ? static_cast<double>(front / slots) * round_cost(k, full, slots, (all - behind) / static_cast<double>(front)) : 0.0;
    const double deep = tail ? behind / static_cast<double>(tail) : 0.0;
    const int most = full || k.tile == 192 || k.tile == 64 ? 1 : kMaxPieces;
    for (int parts = 1; parts <= most; ++parts) {
      // every piece has a step of its own
      if (parts > 1 && (tail == 0 || tail * parts > slots || least_steps < parts)) break;
      const double c = whole + (tail ? round_cost(k, full, tail * parts, deep / parts) : 0.0) + (parts > 1 ? join_cost(k.tile, tail * parts) : 0.0);
      if (least < 0.0 || c < least) {
        least = c;
        *l = NsList{};
        l->tile = k.tile;
        l->parts = parts;
        l->cut = parts > 1 ? static_cast<int32_t>(tail) : 0;
      }
    }
  }
  if (!tiles) return least;
  std::vector<NsTile> v;
  for (size_t i = 0; i < mats.size(); ++i)
    add_tiles(v, static_cast<int>(i), ((full ? mats[i].np : mats[i].mp) + l->tile - 1) / l->tile,
              (mats[i].mp + l->tile - 1) / l->tile, !full);
  l->join = static_cast<int32_t>(tiles->size());
  for (int32_t k = 0; k < l->cut; ++k) {
    NsTile t = v[v.size() - static_cast<size_t>(l->cut - k)];
    t.slot = static_cast<uint16_t>(k);
    tiles->push_back(t);
  }
  l->pieces = static_cast<int32_t>(tiles->size());
  for (int part = 0; part < l->parts && l->cut; ++part)
    for (int32_t k = 0; k < l->cut; ++k) {
      NsTile t = (*tiles)[static_cast<size_t>(l->join + k)];
      t.part = static_cast<uint8_t>(part);
      t.parts = static_cast<uint8_t>(l->parts);
      tiles->push_back(t);
    }
  spread_over_dies(*tiles, static_cast<size_t>(l->pieces));
  v.resize(v.size() - static_cast<size_t>(l->cut));
  l->first = static_cast<int32_t>(tiles->size());
  tiles->insert(tiles->end(), v.begin(), v.end());
  spread_over_dies(*tiles, static_cast<size_t>(l->first));
  l->count = static_cast<int32_t>(tiles->size()) - l->first;
  return least;
}

// A group's matrices share a padding; it is closed when its elements reach
// this many (the workspace is about 9 bytes an element): enough to fill the
// chip many times over.
constexpr int64_t kGroupElements = int64_t(1) << 28;

// The workspace: partial sums of squares, scales, the pieces of cut tiles,
// and the fp16 arrays; the front is the same for every group.
struct NsWorkspace {
  double *partials;
  NsScale *scales;
  float *pieces;
  half_t *arrays;
  size_t front;
  NsWorkspace(const zds_matrix_plan &p, bool f, void *ws) {
    size_t at = 0;
    auto take = [&](size_t bytes) {
      char *here = static_cast<char *>(ws) + at;
      at += (bytes + 255) / 256 * 256;
      return static_cast<void *>(here);
    };
    partials = static_cast<double *>(take(sizeof(double) * static_cast<size_t>(p.max_parts)));
    scales = static_cast<NsScale *>(take(sizeof(NsScale) * static_cast<size_t>(p.max_mats)));
    pieces = static_cast<float *>(take(sizeof(float) * static_cast<size_t>(p.piece_elems[f])));
    arrays = static_cast<half_t *>(take(0));
    front = at;
  }
  size_t bytes(int64_t halves) const { return front + static_cast<size_t>(halves) * 2; }
};

zds_status build_newton_schulz(zds_matrix_plan *p, const int64_t *offset, const int32_t *rows, const int32_t *cols,
                               int32_t num) {
  // the longest sums first
  std::vector<int32_t> order;
  for (int32_t i = 0; i < num; ++i)
    if (rows[i] > 0 && cols[i] > 0) order.push_back(i);
  std::stable_sort(order.begin(), order.end(), [&](int32_t a, int32_t b) {
    const auto key = [&](int32_t i) { return std::make_pair(std::max(rows[i], cols[i]), std::min(rows[i], cols[i])); };
    return key(a) > key(b);
  });
  std::vector<NsTile> tiles;
  std::vector<NsMatrix> mats[2];
  for (int f = 0; f < 2; ++f) {
    const int seg = f ? 3 : 1;
    // Groups, each of one padding: every matrix with the padding that suits it,
    // or, where that makes several short sequences of launches, all with one.
    struct Draft {
      int padding;
      std::vector<NsMatrix> mats;
    };
    std::vector<Draft> drafts;
    double least = -1.0;
    // (a larger padding of matrices of up to 64 rows alone is work for nothing)
    const bool small = std::all_of(order.begin(), order.end(), [&](int32_t i) { return std::min(rows[i], cols[i]) <= 64; });
    for (int only : {64, 0, 256, 128}) {
      if (small && only != 64) break;
      std::vector<Draft> d;
      for (int padding : {256, 128, 64}) {
        int64_t elems = kGroupElements;
        for (int32_t i : order) {
          NsMatrix m{};
          m.offset = offset[i];
          m.rows = rows[i];
          m.cols = cols[i];
          m.tall = rows[i] > cols[i];
          m.m = m.tall ? cols[i] : rows[i];
          m.n = m.tall ? rows[i] : cols[i];
          if ((only ? only : padding_of(m.m, m.n)) != padding) continue;
          m.mp = static_cast<int32_t>(round_up(m.m, padding));
          m.np = static_cast<int32_t>(round_up(m.n, padding));
          m.pair = f == 0 && m.m <= kPairRows;  // whatever the padding, and so whatever else the plan holds
          if (elems >= kGroupElements) {
            d.push_back(Draft{padding, {}});
            elems = 0;
          }
          elems += static_cast<int64_t>(m.mp) * m.np;
          d.back().mats.push_back(m);
        }
      }
      double cost = 0.0;
      NsList l;
      for (const Draft &k : d)
        for (int kind : {kGram, kPoly, kUpdate}) cost += make_list(kind, k.mats, k.padding, seg, &l, nullptr);
      if (least < 0.0 || cost < least) {
        least = cost;
        drafts = std::move(d);
      }
    }
    int64_t most = 0;
    for (Draft &draft : drafts) {
      NsGroup g{};
      g.mat0 = static_cast<int32_t>(mats[f].size());
      g.nmat = static_cast<int32_t>(draft.mats.size());
      int64_t pos = 0;
      int32_t parts = 0;
      const int64_t planes = f ? 2 : 1;
      for (NsMatrix &m : draft.mats) {
        const int64_t len = static_cast<int64_t>(m.rows) * m.cols;
        m.part0 = parts;
        m.chunk = static_cast<int32_t>(std::max(kNormChunk, round_up((len + kMaxParts - 1) / kMaxParts, 2048)));
        m.nparts = static_cast<int32_t>((len + m.chunk - 1) / m.chunk);
        parts += m.nparts;
        const int64_t xe = static_cast<int64_t>(m.mp) * m.np, ae = static_cast<int64_t>(m.mp) * m.mp;
        const auto take = [&](int64_t e) {
          const int64_t at = pos;
          pos += e;
          return at;
        };
        m.x[0] = take(xe * planes);
        m.x[1] = take(xe * planes);
        m.lo = f ? 0 : take(m.pair ? xe * 2 : xe);
        g.pair |= m.pair;
        m.a = take(m.pair ? ae * 2 : ae * planes);
        m.b = take(m.pair ? ae * 2 : ae * planes);
        mats[f].push_back(m);
      }
      most = std::max(most, pos);
      p->max_parts = std::max(p->max_parts, parts);
      p->max_mats = std::max(p->max_mats, g.nmat);
      g.chunk0 = static_cast<int32_t>(tiles.size());
      for (int32_t k = 0; k < g.nmat; ++k)
        for (int c = 0; c < draft.mats[static_cast<size_t>(k)].nparts; ++c) tiles.push_back(NsTile{k, c, 0, 0, 1, 0});
      g.nchunk = static_cast<int32_t>(tiles.size()) - g.chunk0;
      g.conv0 = static_cast<int32_t>(tiles.size());
      for (int32_t k = 0; k < g.nmat; ++k) {
        const NsMatrix &m = draft.mats[static_cast<size_t>(k)];
        const int rp = (m.tall ? m.np : m.mp) / kConvTile, cp = (m.tall ? m.mp : m.np) / kConvTile;
        for (int a = 0; a < rp; ++a)
          for (int b = 0; b < cp; ++b) tiles.push_back(NsTile{k, a, b, 0, 1, 0});
      }
      g.nconv = static_cast<int32_t>(tiles.size()) - g.conv0;
      (void)make_list(kGram, draft.mats, draft.padding, seg, &g.gram, &tiles);
      (void)make_list(kPoly, draft.mats, draft.padding, seg, &g.poly, &tiles);
      (void)make_list(kUpdate, draft.mats, draft.padding, seg, &g.full, &tiles);
      for (const NsList &l : {g.gram, g.poly})
        p->piece_elems[f] = std::max(p->piece_elems[f], static_cast<int64_t>(l.cut) * l.parts * l.tile * l.tile);
      p->groups[f].push_back(g);
    }
    p->arrays[f] = most;
  }
  if (order.empty()) return ZDS_OK;
  for (int f = 0; f < 2; ++f) p->ws_bytes[f] = NsWorkspace(*p, f, nullptr).bytes(p->arrays[f]);
  const char *what = "zds_matrix_plan_create";
  auto upload = [&](void **d, const void *h, size_t bytes) -> zds_status {
    hipError_t e = hipMalloc(d, bytes);
    if (e != hipSuccess) return fail(ZDS_ENOMEM, "%s: hipMalloc tables: %s", what, hipGetErrorString(e));
    e = hipMemcpy(*d, h, bytes, hipMemcpyHostToDevice);
    if (e != hipSuccess) return hip_fail(e, "zds_matrix_plan_create: table upload");
    return ZDS_OK;
  };
  for (int f = 0; f < 2; ++f) {
    const zds_status st = upload(reinterpret_cast<void **>(&p->d_mats[f]), mats[f].data(), mats[f].size() * sizeof(NsMatrix));
    if (st != ZDS_OK) return st;
  }
  return upload(reinterpret_cast<void **>(&p->d_tiles), tiles.data(), tiles.size() * sizeof(NsTile));
}

template <int D, int SEG>
static zds_status run_newton_schulz(const zds_matrix_plan &p, const void *src, void *dst, const float *coef, const float *shift,
                                    int32_t steps, double xb, double bb, const zds_step_scalars *sc, void *ws, hipStream_t s) {
  const NsWorkspace w(p, SEG == 3, ws);
  NsArgs q{};
  q.scales = w.scales;
  q.ws = w.arrays;
  q.pieces = w.pieces;
  q.dst = dst;
  q.sc = sc;
  // fp16 holds up to 65504: X up to xb, A up to xb^2, B up to bb stay below half of that
  q.sx = pow2_under(32768.0, xb);
  q.sa = pow2_under(32768.0, xb * xb);
  // (a B below 2^-24 changes nothing that a result shows; its power would pass fp32's range)
  q.sb = pow2_under(32768.0, std::max(bb, 0x1p-24));
  for (const NsGroup &g : p.groups[SEG == 3]) {
    q.mats = p.d_mats[SEG == 3] + g.mat0;
    hipLaunchKernelGGL((ns_norm_kernel<D>), dim3(g.nchunk), dim3(256), 0, s, q.mats, p.d_tiles + g.chunk0, src, w.partials, sc);
    hipLaunchKernelGGL((ns_convert_kernel<D, SEG>), dim3(g.nconv), dim3(256), 0, s, q.mats, p.d_tiles + g.conv0, src,
                       w.partials, w.scales, w.arrays, sc);
    zds_status st = check_launch("newton_schulz conversion");
    if (st != ZDS_OK) return st;
    for (int k = 0; k < steps; ++k) {
      q.a = coef[3 * k];
      q.b = coef[3 * k + 1];
      q.c = coef[3 * k + 2];
      q.first = k == 0;
      q.odd = k & 1;
      q.a += shift[k];
      q.al = coef[3 * k] + 0.5f * shift[k];
      q.alb = 0.5f / q.sb;
      q.shift = shift[k] * q.sb;
      launch_products<SEG>(g, p.d_tiles, q, kGram, s);
      launch_products<SEG>(g, p.d_tiles, q, kPoly, s);
      launch_products<SEG>(g, p.d_tiles, q, k + 1 == steps ? kLast : kUpdate, s);
      st = check_launch("newton_schulz products");
      if (st != ZDS_OK) return st;
    }
  }
  return ZDS_OK;
}

}  // namespace zds

using namespace zds;

extern "C" size_t zds_newton_schulz_workspace_bytes(const zds_matrix_plan *plan, zds_dtype dtype) {
  if (!plan || (dtype != ZDS_BF16 && dtype != ZDS_FP32)) return 0;
  return plan->ws_bytes[dtype == ZDS_FP32];
}

extern "C" zds_status zds_newton_schulz(const zds_matrix_plan *plan, const void *src, void *dst, zds_dtype dtype,
                                        const float *coef, int32_t steps, const zds_step_scalars *scalars_dev, void *ws,
                                        size_t ws_bytes, void *stream) {
  clear_error();
  const char *fn = "zds_newton_schulz";
  if (dtype != ZDS_BF16 && dtype != ZDS_FP32) return fail(ZDS_EINVAL, "%s: dtype must be bf16 or fp32", fn);
  if (steps < 1 || steps > kMaxSteps) return fail(ZDS_EINVAL, "%s: steps must be in [1, %d]", fn, kMaxSteps);
  float k[3 * kMaxSteps];
  for (int i = 0; i < steps; ++i) {
    static const float quintic[3] = {3.4445f, -4.7750f, 2.0315f};
    for (int j = 0; j < 3; ++j) k[3 * i + j] = coef ? coef[3 * i + j] : quintic[j];
  }
  // The largest singular value any step can leave. Rounding X, A and B to 11 bits
  // moves one by at most about 2^-10 of itself in a step even where all roundings
  // point one way (a matrix of equal elements); 2^-8 over.
  double x = 1.0, xb = 1.0, bb = 0.0;
  float shift[kMaxSteps];
  for (int i = 0; i < steps; ++i) {
    double nx = 0.0, nb = 0.0;
    poly_bound(k + 3 * i, x * (1.0 + 0x1p-8), &nx, &nb);
    if (!(nx <= 8.0) || !(nb <= 1e4))
      return fail(ZDS_EINVAL, "%s: step %d's coefficients can take a singular value past 8", fn, i);
    // (a value at s = 1 that B does not reach is no use)
    shift[i] = fabs(shift_of(k, i, steps)) <= nb ? shift_of(k, i, steps) : 0.0f;
    nb += fabs(static_cast<double>(shift[i]));
    x = nx;
    xb = x > xb ? x : xb;
    bb = nb > bb ? nb : bb;
  }
  if (!plan) return fail(ZDS_EINVAL, "%s: null plan", fn);
  if (plan->groups[0].empty()) return ZDS_OK;
  if (!src || !dst) return fail(ZDS_EINVAL, "%s: null src or dst", fn);
  const uintptr_t es = static_cast<uintptr_t>(dtype_size(dtype));
  if (!aligned(src, es) || !aligned(dst, es) || (scalars_dev && !aligned(scalars_dev, 8)))
    return fail(ZDS_EALIGN, "%s: pointer not aligned to its element size", fn);
  const size_t need = zds_newton_schulz_workspace_bytes(plan, dtype);
  if (!ws || ws_bytes < need || !aligned(ws, 256))
    return fail(ZDS_EINVAL, "%s: workspace of %zu bytes needed (256-byte aligned)", fn, need);
  const int64_t len = (plan->span - plan->first) * static_cast<int64_t>(es);
  const char *from = static_cast<const char *>(src) + plan->first * static_cast<int64_t>(es);
  const char *to = static_cast<const char *>(dst) + plan->first * static_cast<int64_t>(es);
  if (src != dst && ranges_meet(from, len, to, len)) return fail(ZDS_EINVAL, "%s: dst overlaps src and is not src", fn);
  if (ranges_meet(ws, static_cast<int64_t>(need), from, len) || ranges_meet(ws, static_cast<int64_t>(need), to, len))
    return fail(ZDS_EINVAL, "%s: the workspace overlaps src or dst", fn);
  int dev = 0;
  const hipError_t he = hipGetDevice(&dev);
  if (he != hipSuccess) return hip_fail(he, "hipGetDevice");
  if (dev != plan->device) return fail(ZDS_EINVAL, "%s: plan belongs to device %d, current is %d", fn, plan->device, dev);
  hipStream_t s = static_cast<hipStream_t>(stream);
  return dtype == ZDS_BF16 ? run_newton_schulz<ZDS_BF16, 1>(*plan, src, dst, k, shift, steps, xb, bb, scalars_dev, ws, s)
                           : run_newton_schulz<ZDS_FP32, 3>(*plan, src, dst, k, shift, steps, xb, bb, scalars_dev, ws, s);
}
