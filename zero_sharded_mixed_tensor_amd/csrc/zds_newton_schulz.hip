// Newton-Schulz orthogonalisation of the matrices of a flat buffer:
//   X_0 = G / (||G||_F + eps);  A = X X^T;  B = b A + c A^2;  X <- a X + B X
// on the smaller side of each matrix (a tall G is worked on as its transpose).
//
// Every product is of the form C = P Q^T with both operands contiguous along
// the summed axis: A = X X^T, A^2 = A A^T (A is symmetric) and B X = B (X^T)^T,
// so one kernel serves all three and X is kept in both orientations. A and B
// are symmetric: only tiles on and below the diagonal are computed, and each
// is stored twice, which takes a step from 4 m^2 n + 2 m^3 operations to
// 3 m^2 n + m^3.
//
// Numbers. The matrix instructions take fp16 operands and sum in fp32. X, A and
// B have bounded spectra, so powers of two bring them into fp16's range,
// where they keep 11 bits (bf16 would keep 8 at the same speed). For BF16
// results X is carried with what its fp16 value leaves (a second fp16 array,
// read and written by the epilogue only). For FP32 every operand is a pair of
// fp16 numbers (high and low) and a product runs its sum over three pieces,
// high*high + high*low + low*high, into the same fp32 accumulators.
#include <new>
#include <type_traits>

#include "zds_device.h"
#include "zds_matrix.h"

namespace zds {

typedef _Float16 half_t;
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) const void global_cvoid;

constexpr int kMaxSteps = 16;
constexpr double kNormEps = 1e-7;
// A partial sum of squares covers this many elements.
constexpr int kNormChunk = 32768;
constexpr int kConvTile = 64;

// A matrix's first X as stored and true: X_true = alpha * X_stored.
struct NsScale {
  float alpha;
};

// ---------------------------------------------------------------------------
// Norm and conversion
// ---------------------------------------------------------------------------

template <int D>
__global__ void __launch_bounds__(256) ns_norm_kernel(const NsMatrix *mats, const NsTile *chunks, const void *src,
                                                      double *partials, const zds_step_scalars *sc) {
  if (sc && sc->overflow) return;
  const NsTile t = chunks[blockIdx.x];
  const NsMatrix &mt = mats[t.mat];
  const int64_t total = static_cast<int64_t>(mt.rows) * mt.cols;
  const int64_t lo = static_cast<int64_t>(t.ti) * kNormChunk;
  const int64_t hi = lo + kNormChunk < total ? lo + kNormChunk : total;
  constexpr int ES = D == ZDS_FP32 ? 4 : 2;
  constexpr int PER = 16 / ES;
  const char *base = static_cast<const char *>(src) + mt.offset * ES;
  double acc = 0.0;
  int64_t e = lo;
  if (aligned(base, 16)) {  // lo is a multiple of PER
    const int64_t groups = (hi - lo) / PER;
    for (int64_t g = threadIdx.x; g < groups; g += 256) {
      float v[PER];
      if constexpr (D == ZDS_FP32) {
        const f32x4 w = reinterpret_cast<const f32x4 *>(base)[lo / PER + g];
        v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
      } else {
        const u32x4 w = reinterpret_cast<const u32x4 *>(base)[lo / PER + g];
        v[0] = lo_of<D>(w.x); v[1] = hi_of<D>(w.x); v[2] = lo_of<D>(w.y); v[3] = hi_of<D>(w.y);
        v[4] = lo_of<D>(w.z); v[5] = hi_of<D>(w.z); v[6] = lo_of<D>(w.w); v[7] = hi_of<D>(w.w);
      }
#pragma unroll
      for (int j = 0; j < PER; ++j) acc = sq_add(v[j], acc);
    }
    e = lo + groups * PER;
  }
  for (int64_t i = e + threadIdx.x; i < hi; i += 256) acc = sq_add(widen1<D>(base, i), acc);
  const double b = block_sum<256>(acc);
  if (threadIdx.x == 0) partials[mt.part0 + t.ti] = b;
}

// Writes X and X^T (both padded with zeros) of the first step, scaled by the
// power of two that brings the norm into [2^13, 2^14): exact for bf16 but for
// elements below 2^-28 of the norm. Each block adds its matrix's partial sums
// again, in index order (every block the same value); the matrix's first
// block stores alpha.
template <int D, int SEG>
__global__ void __launch_bounds__(256) ns_convert_kernel(const NsMatrix *mats, const NsTile *tiles, const void *src,
                                                         const double *partials, NsScale *scales, half_t *ws,
                                                         const zds_step_scalars *sc) {
  if (sc && sc->overflow) return;
  __shared__ float sh[kConvTile][kConvTile + 1];
  __shared__ double ssum;
  const NsTile t = tiles[blockIdx.x];
  const NsMatrix &mt = mats[t.mat];
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
  constexpr int ES = D == ZDS_FP32 ? 4 : 2;
  const char *base = static_cast<const char *>(src) + mt.offset * ES;
  // tile (ti, tj) of the rows x cols matrix as it lies in src
  const int r0 = t.ti * kConvTile, c0 = t.tj * kConvTile;
  for (int k = threadIdx.x; k < kConvTile * kConvTile; k += 256) {
    const int r = k >> 6, c = k & 63;
    float v = 0.0f;
    if (r0 + r < mt.rows && c0 + c < mt.cols) v = widen1<D>(base, static_cast<int64_t>(r0 + r) * mt.cols + c0 + c);
    sh[r][c] = v * up;
  }
  __syncthreads();
  const int64_t plane = static_cast<int64_t>(mt.mp) * mt.np;
  half_t *straight = ws + (mt.tall ? mt.xt[0] : mt.x);   // rows x cols order
  half_t *turned = ws + (mt.tall ? mt.x : mt.xt[0]);
  const int64_t sld = mt.tall ? mt.mp : mt.np, tld = mt.tall ? mt.np : mt.mp;
  for (int k = threadIdx.x; k < kConvTile * 8; k += 256) {
    const int r = k >> 3, c = (k & 7) * 8;
    f16x8 h, l, th, tl;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float v = sh[r][c + j], w = sh[c + j][r];
      h[j] = static_cast<half_t>(v);
      th[j] = static_cast<half_t>(w);
      l[j] = static_cast<half_t>(v - static_cast<float>(h[j]));
      tl[j] = static_cast<half_t>(w - static_cast<float>(th[j]));
    }
    const int64_t s = (r0 + r) * sld + c0 + c, u = (c0 + r) * tld + r0 + c;
    *reinterpret_cast<f16x8 *>(straight + s) = h;
    *reinterpret_cast<f16x8 *>(turned + u) = th;
    if (SEG == 3) {
      *reinterpret_cast<f16x8 *>(straight + plane + s) = l;
      *reinterpret_cast<f16x8 *>(turned + plane + u) = tl;
    }
  }
}

// ---------------------------------------------------------------------------
// The product C = P Q^T
// ---------------------------------------------------------------------------

enum NsKind { kGram = 0, kPoly = 1, kUpdate = 2, kLast = 3 };

struct NsArgs {
  const NsMatrix *mats;
  const NsTile *tiles;
  const NsScale *scales;
  half_t *ws;
  void *dst;
  const zds_step_scalars *sc;
  float a, b, c;       // the step's coefficients
  float sa, sb, sx;    // powers of two: A, B and X (but the first) as stored
  float carry;         // factor of X's remainder in a X
  int32_t first;       // the first step: X is scaled by its own alpha
  int32_t odd;         // which X^T is read
};

template <int T>
struct NsShape {
  static constexpr int WN = 2, WAVES = 4;
  static constexpr int TM = T / 2, TN = T / 2;     // a wave's part of the tile
  static constexpr int MT = T == 64 ? 16 : 32;     // the matrix instruction's tile, MT x MT x (512 / MT)
  static constexpr int MI = TM / MT, NI = TN / MT;
  static constexpr int KI = MT / 16;               // instructions deep in half a depth step
  static constexpr int GROUPS = MT * MT / 256;     // a lane's runs of 4 rows in an instruction's tile
  static constexpr int LOADS = T / 8 / WAVES;      // 1 KiB loads of a wave per operand and depth step
};

// Position of 16-byte chunk c of row r in an operand's LDS tile (128-byte
// rows): the 16 rows that a matrix instruction's operand read covers at once
// fall on all banks.
__device__ __forceinline__ int ns_swizzle(int r, int c) { return c ^ ((r >> 1) & 7); }

template <int T, int SEG, int KIND>
__global__ void __launch_bounds__(NsShape<T>::WAVES * 64, T == 256 ? 1 : 2) ns_product_kernel(const NsArgs q) {
  typedef NsShape<T> S;
  constexpr int STAGE = T * 128;  // bytes of one operand's tile
  __shared__ __align__(1024) char smem[2][2][STAGE];
  if (q.sc && q.sc->overflow) return;
  const NsTile t = q.tiles[blockIdx.x];
  const NsMatrix &mt = q.mats[t.mat];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wi = w / S::WN, wj = w % S::WN;
  const int64_t mp = mt.mp, np = mt.np;
  const int64_t xplane = mp * np, aplane = mp * mp;
  const half_t *P, *Q;
  int64_t pplane, qplane;
  int depth;       // summed elements
  int64_t ld;
  if constexpr (KIND == kGram) {
    P = Q = q.ws + mt.x;
    pplane = qplane = xplane;
    depth = mt.np;
    ld = np;
  } else if constexpr (KIND == kPoly) {
    P = Q = q.ws + mt.a;
    pplane = qplane = aplane;
    depth = mt.mp;
    ld = mp;
  } else {
    P = q.ws + mt.b;
    Q = q.ws + mt.xt[q.odd];
    pplane = aplane;
    qplane = xplane;
    depth = mt.mp;
    ld = mp;
  }
  const int steps = depth / kNsDepth;
  const int total = steps * SEG;
  // the lane's place in a load: row lane / 8 of the wave's 8 rows, chunk by
  // the swizzle (the same for all of the wave's loads: their first rows are
  // 8 WAVES apart, a multiple of 16)
  const int lrow = w * 8 + (lane >> 3);
  const uint32_t lane_off = static_cast<uint32_t>(lrow * ld * 2 + ns_swizzle(lrow, lane & 7) * 16);
  const uint32_t row_step = static_cast<uint32_t>(8 * S::WAVES * ld * 2);
  const half_t *p0 = P + static_cast<int64_t>(t.ti) * T * ld;
  const half_t *q0 = Q + static_cast<int64_t>(t.tj) * T * ld;
  typedef float AccT __attribute__((ext_vector_type(4 * S::GROUPS)));
  AccT acc[S::MI][S::NI];
#pragma unroll
  for (int i = 0; i < S::MI; ++i)
#pragma unroll
    for (int j = 0; j < S::NI; ++j)
#pragma unroll
      for (int r = 0; r < 4 * S::GROUPS; ++r) acc[i][j][r] = 0.0f;

  // Load g of depth step k (T / 16 of them, P's before Q's): global to LDS
  // without passing through registers; the LDS side is linear, so the lane
  // takes the chunk that belongs at its position.
  const half_t *pk = p0, *qk = q0;
  auto aim = [&](int k) {
    int seg = 0, kk = k;
    if (SEG == 3) {
      seg = k / steps;
      kk = k - seg * steps;
    }
    // pieces: high*high, high*low, low*high
    pk = p0 + (seg == 2 ? pplane : 0) + static_cast<int64_t>(kk) * kNsDepth;
    qk = q0 + (seg == 1 ? qplane : 0) + static_cast<int64_t>(kk) * kNsDepth;
  };
  auto load = [&](int buf, int g) {
    const int o = g / S::LOADS, r = g % S::LOADS;
    const char *p = reinterpret_cast<const char *>(o ? qk : pk) + static_cast<uint64_t>(r) * row_step;
    __builtin_amdgcn_global_load_lds((global_cvoid *)(p + lane_off),
                                     (lds_void *)(smem[buf][o] + (w + r * S::WAVES) * 1024), 16, 0, 0);
  };
  const int fr = lane % S::MT, fc = lane / S::MT;
  // operand pieces of half h of a depth step: buffer h in registers
  f16x8 fp[2][S::KI][S::MI], fq[2][S::KI][S::NI];
  int off_p[2][S::KI], off_q[2][S::KI];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int c = 0; c < S::KI; ++c) {
      const int rp = wi * S::TM + fr, rq = wj * S::TN + fr, chunk = h * 4 + c * (64 / S::MT) + fc;
      off_p[h][c] = rp * 128 + ns_swizzle(rp, chunk) * 16;
      off_q[h][c] = rq * 128 + ns_swizzle(rq, chunk) * 16;
    }
  // read g of half h: for each instruction depth the MI pieces of P, then the
  // NI of Q; MT rows on are 128 MT bytes on
  auto read = [&](int buf, int h, int g) {
    const int c = g / (S::MI + S::NI), r = g % (S::MI + S::NI);
    if (r < S::MI) fp[h][c][r] = *reinterpret_cast<const f16x8 *>(smem[buf][0] + off_p[h][c] + r * 128 * S::MT);
    else fq[h][c][r - S::MI] = *reinterpret_cast<const f16x8 *>(smem[buf][1] + off_q[h][c] + (r - S::MI) * 128 * S::MT);
  };
  constexpr int MFMAS = S::MI * S::NI * S::KI, READS = (S::MI + S::NI) * S::KI, ALL_LOADS = 2 * S::LOADS;
  auto product = [&](int h, int e) {
    const int c = e / (S::MI * S::NI), i = e / S::NI % S::MI, j = e % S::NI;
    if constexpr (S::MT == 32)
      asm volatile("v_mfma_f32_32x32x16_f16 %0, %1, %2, %0" : "+a"(acc[i][j]) : "v"(fp[h][c][i]), "v"(fq[h][c][j]));
    else
      acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fp[h][c][i], fq[h][c][j], acc[i][j], 0, 0, 0);
  };
  // The products of half h. Between them the reads of half h ^ 1 (of tiles
  // `buf`), as early as they can go but behind the first product, and for
  // `reload` the loads into tiles `to`.
  auto half_step = [&](int buf, int h, bool reload, int to) {
#pragma unroll
    for (int e = 0; e < MFMAS; ++e) {
      product(h, e);
      constexpr int RATE = READS > MFMAS ? READS / MFMAS : 1;  // reads behind a product
#pragma unroll
      for (int r = 0; r < RATE; ++r)
        if (e * RATE + r < READS) read(buf, h ^ 1, e * RATE + r);
      if (h == 1) {
#pragma unroll
        for (int g = e * ALL_LOADS / MFMAS; g < (e + 1) * ALL_LOADS / MFMAS; ++g)
          if (reload) load(to, g);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  aim(0);
#pragma unroll
  for (int g = 0; g < ALL_LOADS; ++g) load(0, g);
  if (total > 1) {
    aim(1);
#pragma unroll
    for (int g = 0; g < ALL_LOADS; ++g) load(1, g);
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(ALL_LOADS) : "memory");
  } else {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  }
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
#pragma unroll
  for (int g = 0; g < READS; ++g) read(0, 0, g);
  // One depth step. While the products of its first half run, the second
  // half's operands are read; then one barrier (every wave has read the
  // step's tiles, and the next step's have arrived), and while the second
  // half's products run, the tiles just read are refilled with the step after
  // next and the next step's first operands are read (after the last step:
  // tiles that are there and not used).
  for (int k = 0; k < total; ++k) {
    const int buf = k & 1;
    half_step(buf, 0, false, 0);
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    const bool reload = k + 2 < total;
    if (reload) aim(k + 2);
    half_step(buf ^ 1, 1, reload, buf);
  }
  asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");

  // Epilogue. A lane holds column fr of an instruction's tile and, in run g, its
  // rows 4 (64 / MT) g + 4 fc + 0..3: four consecutive values of a row of C^T.
  const float alpha = q.first ? q.scales[t.mat].alpha : 1.0f / q.sx;
  auto split = [](float v, half_t &h, half_t &l) {
    h = static_cast<half_t>(v);
    l = static_cast<half_t>(v - static_cast<float>(h));
  };
#pragma unroll
  for (int i = 0; i < S::MI; ++i)
#pragma unroll
    for (int jg = 0; jg < S::NI * S::GROUPS; ++jg) {
      const int j = jg / S::GROUPS, gr = jg % S::GROUPS;
      const int64_t row = static_cast<int64_t>(t.ti) * T + wi * S::TM + i * S::MT + gr * 8 + fc * 4;
      const int64_t col = static_cast<int64_t>(t.tj) * T + wj * S::TN + j * S::MT + fr;
      f32x4 cv;
#pragma unroll
      for (int r = 0; r < 4; ++r) cv[r] = acc[i][j][gr * 4 + r];
      f16x4 h, l;
      if constexpr (KIND == kGram || KIND == kPoly) {
        half_t *out = q.ws + (KIND == kGram ? mt.a : mt.b);
        float v[4];
        if constexpr (KIND == kGram) {
          const float f = alpha * alpha * q.sa;
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] = cv[r] * f;
        } else {
          // A is stored whole, so its value at (row, col) is that at (col, row)
          const f16x4 ah = *reinterpret_cast<const f16x4 *>(q.ws + mt.a + col * mp + row);
          f16x4 al = {};
          if (SEG == 3) al = *reinterpret_cast<const f16x4 *>(q.ws + mt.a + aplane + col * mp + row);
          const float fb = q.b * (q.sb / q.sa), fc2 = q.c * (q.sb / (q.sa * q.sa));
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float av = static_cast<float>(ah[r]);
            if (SEG == 3) av += static_cast<float>(al[r]);
            v[r] = fb * av + fc2 * cv[r];
          }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) { half_t hh, ll; split(v[r], hh, ll); h[r] = hh; l[r] = ll; }
        *reinterpret_cast<f16x4 *>(out + col * mp + row) = h;
        if (SEG == 3) *reinterpret_cast<f16x4 *>(out + aplane + col * mp + row) = l;
        if (t.ti != t.tj) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            out[(row + r) * mp + col] = h[r];
            if (SEG == 3) out[aplane + (row + r) * mp + col] = l[r];
          }
        }
      } else {
        const half_t *xin = q.ws + mt.xt[q.odd];
        const f16x4 xh = *reinterpret_cast<const f16x4 *>(xin + col * mp + row);
        f16x4 xl = {};
        if (SEG == 3) xl = *reinterpret_cast<const f16x4 *>(xin + xplane + col * mp + row);
        else if (!q.first) xl = *reinterpret_cast<const f16x4 *>(q.ws + mt.lo + col * mp + row);
        const float out_scale = KIND == kLast ? 1.0f : q.sx;
        const float fa = q.a * alpha * out_scale, fb = alpha / q.sb * out_scale;
        float v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
          v[r] = fa * (static_cast<float>(xh[r]) + q.carry * static_cast<float>(xl[r])) + fb * cv[r];
        if constexpr (KIND == kUpdate) {
#pragma unroll
          for (int r = 0; r < 4; ++r) { half_t hh, ll; split(v[r], hh, ll); h[r] = hh; l[r] = ll; }
          half_t *xout = q.ws + mt.xt[q.odd ^ 1];
          *reinterpret_cast<f16x4 *>(xout + col * mp + row) = h;
          *reinterpret_cast<f16x4 *>((SEG == 3 ? xout + xplane : q.ws + mt.lo) + col * mp + row) = l;
          half_t *x = q.ws + mt.x;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            x[(row + r) * np + col] = h[r];
            if (SEG == 3) x[xplane + (row + r) * np + col] = l[r];
          }
        } else {
          if (col < mt.n) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              if (row + r < mt.m) {
                const int64_t e = mt.offset + (mt.tall ? col * mt.cols + row + r : (row + r) * mt.cols + col);
                if (SEG == 3) static_cast<float *>(q.dst)[e] = v[r];
                else static_cast<uint16_t *>(q.dst)[e] = narrow1<ZDS_BF16>(v[r]);
              }
            }
          }
        }
      }
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// Largest |a s + b s^3 + c s^5| over [0, top], and largest |b s^2 + c s^4|.
static void poly_bound(const float *k, double top, double *x, double *bx) {
  double mx = 0.0, mb = 0.0;
  for (int i = 0; i <= 4096; ++i) {
    const double s = top * i / 4096, l = s * s;
    const double b = l * (static_cast<double>(k[1]) + static_cast<double>(k[2]) * l);
    const double v = fabs(s * (static_cast<double>(k[0]) + b));
    if (!(v <= mx)) mx = v;
    if (!(fabs(b) <= mb)) mb = fabs(b);
  }
  *x = mx;
  *bx = mb;
}

static float pow2_under(double limit, double value) {  // largest power of two with p * value <= limit
  int e = 0;
  (void)frexp(limit / value, &e);
  return ldexpf(1.0f, e - 1);
}

template <int T, int SEG>
static void launch_products(const NsGroup &g, const NsTile *tiles, NsArgs q, int kind, hipStream_t s) {
  const dim3 block(NsShape<T>::WAVES * 64);
  if (kind == kGram || kind == kPoly) {
    q.tiles = tiles + g.tri0;
    if (kind == kGram) hipLaunchKernelGGL((ns_product_kernel<T, SEG, kGram>), dim3(g.ntri), block, 0, s, q);
    else hipLaunchKernelGGL((ns_product_kernel<T, SEG, kPoly>), dim3(g.ntri), block, 0, s, q);
  } else {
    q.tiles = tiles + g.full0;
    if (kind == kUpdate) hipLaunchKernelGGL((ns_product_kernel<T, SEG, kUpdate>), dim3(g.nfull), block, 0, s, q);
    else hipLaunchKernelGGL((ns_product_kernel<T, SEG, kLast>), dim3(g.nfull), block, 0, s, q);
  }
}

template <int SEG>
static void launch_products(const NsGroup &g, const NsTile *tiles, const NsArgs &q, int kind, hipStream_t s) {
  if (g.tile == 256) launch_products<256, SEG>(g, tiles, q, kind, s);
  else if (g.tile == 128) launch_products<128, SEG>(g, tiles, q, kind, s);
  else launch_products<64, SEG>(g, tiles, q, kind, s);
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
          if (!triangle || i >= j) v.push_back(NsTile{mat, i, j, 0});
}

static int64_t round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

// The product tile of a matrix by its smaller size.
static int tile_of(int m, int n) {
  if (m >= 1024) return 256;
  if (m > 128) return 128;
  return 64;
}

// A group's matrices share a tile size; it is closed when its elements reach
// this many (the workspace is about 9 bytes an element): enough to fill the
// chip many times over.
constexpr int64_t kGroupElements = int64_t(1) << 28;

zds_status build_newton_schulz(zds_matrix_plan *p, const int64_t *offset, const int32_t *rows, const int32_t *cols,
                               int32_t num) {
  std::vector<NsMatrix> mats[2];
  std::vector<NsTile> tiles;
  size_t head = 0;  // bytes in front of the fp16 arrays, the same for every group
  int64_t most[2] = {0, 0};
  for (int tile : {256, 128, 64}) {
    int32_t i = 0;
    while (i < num) {
      NsGroup g{};
      g.tile = tile;
      g.mat0 = static_cast<int32_t>(mats[0].size());
      int64_t elems = 0, pos[2] = {0, 0};
      int32_t parts = 0;
      for (; i < num && elems < kGroupElements; ++i) {
        if (rows[i] == 0 || cols[i] == 0) continue;
        NsMatrix m{};
        m.offset = offset[i];
        m.rows = rows[i];
        m.cols = cols[i];
        m.tall = rows[i] > cols[i];
        m.m = m.tall ? cols[i] : rows[i];
        m.n = m.tall ? rows[i] : cols[i];
        if (tile_of(m.m, m.n) != tile) continue;
        m.mp = static_cast<int32_t>(round_up(m.m, tile));
        m.np = static_cast<int32_t>(round_up(m.n, tile));
        m.part0 = parts;
        m.nparts = static_cast<int32_t>((static_cast<int64_t>(m.rows) * m.cols + kNormChunk - 1) / kNormChunk);
        parts += m.nparts;
        const int64_t xe = static_cast<int64_t>(m.mp) * m.np, ae = static_cast<int64_t>(m.mp) * m.mp;
        for (int f = 0; f < 2; ++f) {
          const int64_t planes = f ? 2 : 1;
          NsMatrix d = m;
          auto take = [&](int64_t e) { const int64_t at = pos[f]; pos[f] += e; return at; };
          d.x = take(xe * planes);
          d.xt[0] = take(xe * planes);
          d.xt[1] = take(xe * planes);
          d.lo = f ? 0 : take(xe);
          d.a = take(ae * planes);
          d.b = take(ae * planes);
          mats[f].push_back(d);
        }
        elems += xe;
      }
      g.nmat = static_cast<int32_t>(mats[0].size()) - g.mat0;
      if (g.nmat == 0) continue;
      for (int f = 0; f < 2; ++f) most[f] = pos[f] > most[f] ? pos[f] : most[f];
      if (parts > p->max_parts) p->max_parts = parts;
      if (g.nmat > p->max_mats) p->max_mats = g.nmat;
      auto each = [&](auto &&fn) { for (int32_t k = 0; k < g.nmat; ++k) fn(k, mats[0][static_cast<size_t>(g.mat0 + k)]); };
      g.chunk0 = static_cast<int32_t>(tiles.size());
      each([&](int32_t k, const NsMatrix &m) { for (int c = 0; c < m.nparts; ++c) tiles.push_back(NsTile{k, c, 0, 0}); });
      g.nchunk = static_cast<int32_t>(tiles.size()) - g.chunk0;
      g.conv0 = static_cast<int32_t>(tiles.size());
      each([&](int32_t k, const NsMatrix &m) {
        const int rp = (m.tall ? m.np : m.mp) / kConvTile, cp = (m.tall ? m.mp : m.np) / kConvTile;
        for (int a = 0; a < rp; ++a)
          for (int b = 0; b < cp; ++b) tiles.push_back(NsTile{k, a, b, 0});
      });
      g.nconv = static_cast<int32_t>(tiles.size()) - g.conv0;
      g.tri0 = static_cast<int32_t>(tiles.size());
      each([&](int32_t k, const NsMatrix &m) { add_tiles(tiles, k, m.mp / tile, m.mp / tile, true); });
      spread_over_dies(tiles, static_cast<size_t>(g.tri0));
      g.ntri = static_cast<int32_t>(tiles.size()) - g.tri0;
      g.full0 = static_cast<int32_t>(tiles.size());
      each([&](int32_t k, const NsMatrix &m) { add_tiles(tiles, k, m.mp / tile, m.np / tile, false); });
      spread_over_dies(tiles, static_cast<size_t>(g.full0));
      g.nfull = static_cast<int32_t>(tiles.size()) - g.full0;
      p->groups.push_back(g);
    }
  }
  head = static_cast<size_t>(round_up(p->max_parts * 8 + p->max_mats * static_cast<int64_t>(sizeof(NsScale)), 256));
  for (int f = 0; f < 2; ++f) p->ws_bytes[f] = p->groups.empty() ? 0 : head + static_cast<size_t>(most[f]) * 2;
  if (p->groups.empty()) return ZDS_OK;
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
static zds_status run_newton_schulz(const zds_matrix_plan &p, const void *src, void *dst, const float *coef, int32_t steps,
                                    double xb, double bb, const zds_step_scalars *sc, void *ws, hipStream_t s) {
  double *partials = static_cast<double *>(ws);
  NsScale *scales = reinterpret_cast<NsScale *>(partials + p.max_parts);
  const size_t head = static_cast<size_t>(
      round_up(p.max_parts * 8 + p.max_mats * static_cast<int64_t>(sizeof(NsScale)), 256));
  half_t *arrays = reinterpret_cast<half_t *>(static_cast<char *>(ws) + head);
  NsArgs q{};
  q.scales = scales;
  q.ws = arrays;
  q.dst = dst;
  q.sc = sc;
  // fp16 holds up to 65504: X up to xb, A up to xb^2, B up to bb stay below half of that
  q.sx = pow2_under(32768.0, xb);
  q.sa = pow2_under(32768.0, xb * xb);
  q.sb = pow2_under(32768.0, bb > 0.0 ? bb : 1.0);
  for (const NsGroup &g : p.groups) {
    q.mats = p.d_mats[SEG == 3] + g.mat0;
    hipLaunchKernelGGL((ns_norm_kernel<D>), dim3(g.nchunk), dim3(256), 0, s, q.mats, p.d_tiles + g.chunk0, src, partials, sc);
    hipLaunchKernelGGL((ns_convert_kernel<D, SEG>), dim3(g.nconv), dim3(256), 0, s, q.mats, p.d_tiles + g.conv0, src,
                       partials, scales, arrays, sc);
    zds_status st = check_launch("newton_schulz conversion");
    if (st != ZDS_OK) return st;
    for (int k = 0; k < steps; ++k) {
      q.a = coef[3 * k];
      q.b = coef[3 * k + 1];
      q.c = coef[3 * k + 2];
      q.first = k == 0;
      q.odd = k & 1;
      q.carry = SEG == 3 || k + 2 < steps ? 1.0f : (k + 1 < steps ? 0.5f : 0.25f);
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
  // the largest singular value any step can leave (2 % over for rounding)
  double x = 1.0, xb = 1.0, bb = 0.0;
  for (int i = 0; i < steps; ++i) {
    double nx = 0.0, nb = 0.0;
    poly_bound(k + 3 * i, x * 1.02, &nx, &nb);
    if (!(nx <= 8.0) || !(nb <= 1e4))
      return fail(ZDS_EINVAL, "%s: step %d's coefficients can take a singular value past 8", fn, i);
    x = nx;
    xb = x > xb ? x : xb;
    bb = nb > bb ? nb : bb;
  }
  if (!plan) return fail(ZDS_EINVAL, "%s: null plan", fn);
  if (plan->groups.empty()) return ZDS_OK;
  if (!src || !dst) return fail(ZDS_EINVAL, "%s: null src or dst", fn);
  const uintptr_t es = static_cast<uintptr_t>(dtype_size(dtype));
  if (!aligned(src, es) || !aligned(dst, es) || (scalars_dev && !aligned(scalars_dev, 8)))
    return fail(ZDS_EALIGN, "%s: pointer not aligned to its element size", fn);
  const size_t need = zds_newton_schulz_workspace_bytes(plan, dtype);
  if (!ws || ws_bytes < need || !aligned(ws, 256))
    return fail(ZDS_EINVAL, "%s: workspace of %zu bytes needed (256-byte aligned)", fn, need);
  int dev = 0;
  const hipError_t he = hipGetDevice(&dev);
  if (he != hipSuccess) return hip_fail(he, "hipGetDevice");
  if (dev != plan->device) return fail(ZDS_EINVAL, "%s: plan belongs to device %d, current is %d", fn, plan->device, dev);
  hipStream_t s = static_cast<hipStream_t>(stream);
  return dtype == ZDS_BF16 ? run_newton_schulz<ZDS_BF16, 1>(*plan, src, dst, k, steps, xb, bb, scalars_dev, ws, s)
                           : run_newton_schulz<ZDS_FP32, 3>(*plan, src, dst, k, steps, xb, bb, scalars_dev, ws, s);
}
