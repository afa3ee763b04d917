// Newton-Schulz orthogonalisation of matrices whose smaller side is at most 128.
//
// Every iterate is a polynomial of H = X X^T times X0 (the normalised input),
// so for m <= 128 the steps run on m x m matrices alone, all of them in one
// workgroup's LDS, and X is read twice whatever the number of steps:
//   ortho_small_gram   sums over column ranges of X0 X0^T
//   ortho_small_steps  a workgroup per matrix: with P = a + b H + c H^2,
//                      Q <- P Q and H <- P H P, every step
//   ortho_small_apply  the result Q X0, to U or the weights
// Bound by its launches and, past m = 64, by the LDS reads of the m x m products.
// In us, against three launches per step of the tiled path: 16 x 16 alone 21 :
// 72, 16 of 64 x 64 31 : 79, 64 of 128 x 128 69 : 85, 2 of 128 x 4096 72 : 115,
// 64 of 96 x 4000 116 : 353, 1000 of 128 x 256 450 : 651.
//
// Numbers. Q X0 cancels: Q is a^steps (485) on the directions of small singular
// values and near 1 / sigma on the others, and they only separate through Q's
// own rounding. So all m x m matrices are pairs of fp16 values (22 bits, three
// products of fp16 MFMAs), scaled so that the lower one stays normal; X0 is a
// pair too, unless it is a bf16 gradient, which fp16 holds exactly. Off by
// 1e-3 at rank 1, 1e-4 at most others, before the bf16 output rounding. Q is near
// a^steps where singular values are small: past 1000 the bits do not reach, and
// below 2^-8 a pair of fp16 no longer holds 22 of them (Q is resolved to 2^-30:
// with a = 0.3 and 16 steps, 4e-9, it came out 13 % off). The tiled path runs then.
#include <cmath>

#include "ortho_device.h"

namespace moe {
namespace ortho {

namespace {

constexpr float kHScale = 1024.f;  // of H, T and P (at most 32)
constexpr float kQScale = 32.f;    // of Q (at most 1024)
constexpr int kSub = 64;           // columns of X in LDS at a time

// A block of fp16 pairs: the upper values' blocks, then the lower values'.
template <int NB>
struct Pairs {
  static constexpr int kBlocks = 2 * NB * NB;  // an m x m matrix: 2 NB column blocks of NB row blocks
  _Float16 hi[kBlocks * kBlock];
  _Float16 lo[kBlocks * kBlock];
};

__device__ __forceinline__ f16x8 fragment(const _Float16* blocks, int nb, int rb, int kk) {
  return *reinterpret_cast<const f16x8*>(blocks + (kk * nb + rb) * kBlock + in_block(lane_id() & 31, lane_id() >> 5));
}

// A wave for each 32 x 32 sub-tile (i, j) of an m x m matrix, four at least (8
// waves with two sub-tiles each of 128 x 128: 54 us, 16 waves 45).
template <int NB>
constexpr int kWaves = NB * NB < 4 ? 4 : NB * NB;
template <int NB>
__device__ __forceinline__ bool has_tile() { return wave_id() < NB * NB; }

// acc = M N^T for symmetric (or row-major) M, N, times f: upper x upper, then
// the two mixed products.
template <int NB>
__device__ __forceinline__ void multiply(const Pairs<NB>& M, const Pairs<NB>& N, float f, f32x16& acc) {
  if (!has_tile<NB>()) return;
  const int i = wave_id() / NB, j = wave_id() % NB;
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[r] = 0.f;
#pragma unroll
  for (int kk = 0; kk < 2 * NB; ++kk) {
    const f16x8 mh = fragment(M.hi, NB, i, kk), ml = fragment(M.lo, NB, i, kk);
    const f16x8 nh = fragment(N.hi, NB, j, kk), nl = fragment(N.lo, NB, j, kk);
    acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(nl, mh, acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(nh, ml, acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(nh, mh, acc, 0, 0, 0);
  }
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[r] *= f;
}

// acc times f as fp16 pairs.
template <int NB>
__device__ __forceinline__ void store_pairs(const f32x16& acc, float f, _Float16* hi, _Float16* lo) {
  if (!has_tile<NB>()) return;
  u32x2 wh[4], wl[4];
#pragma unroll
  for (int g = 0; g < 4; ++g)
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      const float x = acc[4 * g + 2 * d] * f, y = acc[4 * g + 2 * d + 1] * f;
      wh[g][d] = pack_f16(x, y);
      wl[g][d] = pack_f16(x - half_of(wh[g][d], 0), y - half_of(wh[g][d], 1));
    }
  const int i = wave_id() / NB, j = wave_id() % NB;
  put_subtile(wh, hi, 32 * NB, 32 * i, 32 * j);
  put_subtile(wl, lo, 32 * NB, 32 * i, 32 * j);
}

// Columns c0 .. c0 + 63 of X0 as fp16 pairs in blocks. ALONG: entities are rows
// of X and k its columns (the sums of X X^T); otherwise entities are columns
// and k rows (Q X). Elements past the matrix are zeros.
template <int NB, bool ALONG, bool LO, int THREADS>
__device__ __forceinline__ void load_columns(const OrthoIn& in, const OrthoDims& d, int64_t e, int c0, int p,
                                             bool finite, _Float16* hi, _Float16* lo) {
  constexpr int kRows = 32 * NB;
  // an item: 8 neighbours in memory, along X's columns or (tall) along its rows
  const int items = kRows * kSub / 8;
  for (int it = threadIdx.x; it < items; it += THREADS) {
    const int r = d.tall ? 8 * (it % (kRows / 8)) : it / (kSub / 8);
    const int c = d.tall ? it / (kRows / 8) : 8 * (it % (kSub / 8));
    float x[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) x[t] = 0.f;
    const int gr = d.tall ? c0 + c : r, gc = d.tall ? r : c0 + c;
    if (gr < d.R && gc < d.C) {
      const int64_t at = (e * d.R + gr) * d.C + gc;
      input_row(in, at, d.C - gc, x);
#pragma unroll
      for (int t = 0; t < 8; ++t) x[t] = finite ? ldexpf(x[t], p) : NAN;
    }
    u32x4 h, l;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      h[t] = pack_f16(x[2 * t], x[2 * t + 1]);
      l[t] = pack_f16(x[2 * t] - half_of(h[t], 0), x[2 * t + 1] - half_of(h[t], 1));
    }
    // entity and k of the first element; the eight run along k or along the entities
    const int ent = ALONG ? r : c, k = ALONG ? c : r;
    constexpr int kEntBlocks = ALONG ? NB : kSub / 32;
    if (ALONG != d.tall) {
      const int o = ((k >> 4) * kEntBlocks + (ent >> 5)) * kBlock + in_block(ent & 31, (k >> 3) & 1);
      *reinterpret_cast<u32x4*>(hi + o) = h;
      if (LO) *reinterpret_cast<u32x4*>(lo + o) = l;
    } else {
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const int en = ent + t;
        const int o = ((k >> 4) * kEntBlocks + (en >> 5)) * kBlock + in_block(en & 31, (k >> 3) & 1) + (k & 7);
        hi[o] = __builtin_bit_cast(_Float16, uint16_t(h[t >> 1] >> (16 * (t & 1))));
        if (LO) lo[o] = __builtin_bit_cast(_Float16, uint16_t(l[t >> 1] >> (16 * (t & 1))));
      }
    }
  }
}

// Sums over a range of columns of X0 X0^T, as the accumulators hold them:
// [part][tile][4][lane][4].
template <int NB, bool LO>
__global__ __launch_bounds__(64 * kWaves<NB>) void ortho_small_gram_kernel(OrthoIn in, OrthoDims d,
                                                                    const NormPart* __restrict__ part, float eps,
                                                                    int part_cols, float* __restrict__ gram) {
  __shared__ __attribute__((aligned(16))) _Float16 hi[4 * NB * kBlock];
  __shared__ __attribute__((aligned(16))) _Float16 lo[LO ? 4 * NB * kBlock : 8];
  const int64_t e = blockIdx.y;
  int p;
  float s;
  matrix_scale(part + e * d.parts, d.parts, eps, &p, &s);
  const bool finite = s == s;
  f32x16 acc;
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[r] = 0.f;
  const int i = wave_id() / NB, j = wave_id() % NB;
  const int c1 = min(d.n, int(blockIdx.x + 1) * part_cols);
  for (int c0 = blockIdx.x * part_cols; c0 < c1; c0 += kSub) {
    __syncthreads();
    load_columns<NB, true, LO, 64 * kWaves<NB>>(in, d, e, c0, p, finite, hi, lo);
    __syncthreads();
    if (!has_tile<NB>()) continue;
#pragma unroll
    for (int kk = 0; kk < kSub / 16; ++kk) {
      const f16x8 a = fragment(hi, NB, i, kk), b = fragment(hi, NB, j, kk);
      if (LO) {
        acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(fragment(lo, NB, j, kk), a, acc, 0, 0, 0);
        acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(b, fragment(lo, NB, i, kk), acc, 0, 0, 0);
      }
      acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(b, a, acc, 0, 0, 0);
    }
  }
  if (!has_tile<NB>()) return;
  float* out = gram + (e * gridDim.x + blockIdx.x) * (NB * NB * 1024) + wave_id() * 1024;
#pragma unroll
  for (int g = 0; g < 4; ++g)
    *reinterpret_cast<f32x4*>(out + (g * 64 + lane_id()) * 4) =
        f32x4{acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]};
}

// P = a + b H + c H^2, of which P holds H^2.
template <int NB>
__device__ __forceinline__ void polynomial(const f32x16& H, float ca, float cb, float cc, f32x16& P) {
  const bool diag = wave_id() / NB == wave_id() % NB;
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    const bool one = diag && (lane_id() & 31) == 8 * (q >> 2) + 4 * (lane_id() >> 5) + (q & 3);
    P[q] = (one ? ca : 0.f) + cb * H[q] + cc * P[q];
  }
}

// The steps on H and Q. Up to 96 x 96 every matrix has its place in LDS, and T = P H
// and P Q run side by side: three barriers a step. At 128 x 128 two fit: M1 holds
// H, then T, Q and the next H in turn, M2 holds P.
template <int NB>
__global__ __launch_bounds__(64 * kWaves<NB>) void ortho_small_steps_kernel(const float* __restrict__ gram, int parts,
                                                                     const NormPart* __restrict__ norm, int norms,
                                                                     float eps, int steps, float ca, float cb, float cc,
                                                                     _Float16* __restrict__ Qout) {
  __shared__ __attribute__((aligned(16))) Pairs<NB> M1, M2;
  const int64_t e = blockIdx.x;
  int p;
  float s;
  matrix_scale(norm + e * norms, norms, eps, &p, &s);
  f32x16 H, Q, P;
#pragma unroll
  for (int r = 0; r < 16; ++r) H[r] = Q[r] = P[r] = 0.f;
  const bool mine = has_tile<NB>();
#pragma unroll 4
  for (int c = 0; c < (mine ? parts : 0); ++c) {
    const float* src = gram + (e * parts + c) * (NB * NB * 1024) + wave_id() * 1024;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(src + (g * 64 + lane_id()) * 4);
#pragma unroll
      for (int t = 0; t < 4; ++t) H[4 * g + t] += v[t];
    }
  }
#pragma unroll
  for (int r = 0; r < 16; ++r) H[r] *= s * s;
  store_pairs<NB>(H, kHScale, M1.hi, M1.lo);
  __syncthreads();
  constexpr float kHH = 1.f / (kHScale * kHScale), kHQ = 1.f / (kHScale * kQScale);
  if constexpr (NB <= 3) {
    __shared__ __attribute__((aligned(16))) Pairs<NB> MT, MQ;
    for (int k = 0; k < steps; ++k) {
      const bool last = k + 1 == steps;
      multiply<NB>(M1, M1, kHH, P);
      polynomial<NB>(H, ca, cb, cc, P);
      store_pairs<NB>(P, kHScale, M2.hi, M2.lo);
      __syncthreads();
      if (!last) multiply<NB>(M2, M1, kHH, H);  // T = P H
      if (k == 0) Q = P; else multiply<NB>(M2, MQ, kHQ, Q);
      if (last) break;
      store_pairs<NB>(H, kHScale, MT.hi, MT.lo);
      __syncthreads();
      multiply<NB>(M2, MT, kHH, H);  // P T^T
      store_pairs<NB>(H, kHScale, M1.hi, M1.lo);
      store_pairs<NB>(Q, kQScale, MQ.hi, MQ.lo);
      __syncthreads();
    }
  } else {
    for (int k = 0; k < steps; ++k) {
      const bool last = k + 1 == steps;
      multiply<NB>(M1, M1, kHH, P);  // H^2
      polynomial<NB>(H, ca, cb, cc, P);
      store_pairs<NB>(P, kHScale, M2.hi, M2.lo);
      __syncthreads();
      if (!last) {
        multiply<NB>(M2, M1, kHH, H);  // T = P H
        __syncthreads();
        store_pairs<NB>(H, kHScale, M1.hi, M1.lo);
        __syncthreads();
        multiply<NB>(M2, M1, kHH, H);  // P T^T
      }
      __syncthreads();
      if (k == 0) {
        Q = P;
      } else {
        store_pairs<NB>(Q, kQScale, M1.hi, M1.lo);
        __syncthreads();
        multiply<NB>(M2, M1, kHQ, Q);  // P Q
        __syncthreads();
      }
      if (!last) {
        store_pairs<NB>(H, kHScale, M1.hi, M1.lo);
        __syncthreads();
      }
    }
  }
  constexpr int kHalves = Pairs<NB>::kBlocks * kBlock;
  _Float16* out = Qout + e * 2 * kHalves;
  store_pairs<NB>(Q, kQScale, out, out + kHalves);
}

// Q X0 for 64 columns of X: a wave for 64 rows.
template <int NB, bool LO>
__global__ __launch_bounds__((NB + 1) / 2 * 64) void ortho_small_apply_kernel(OrthoIn in, OrthoDims d,
                                                                              const NormPart* __restrict__ part,
                                                                              float eps,
                                                                              const _Float16* __restrict__ Qm,
                                                                              OrthoOut out) {
  constexpr int kApply = (NB + 1) / 2;  // waves
  constexpr int kCols = 4 * NB * kBlock;
  __shared__ __attribute__((aligned(16))) _Float16 cols[(LO ? 2 : 1) * kCols];
  __shared__ __attribute__((aligned(16))) uint16_t images[kApply][4096];
  static_assert(2 * kCols >= kApply * 4096, "the second images take the columns' place");
  _Float16 *const hi = cols, *const lo = cols + (LO ? kCols : 0);
  const int64_t e = blockIdx.y;
  const int c0 = blockIdx.x * kSub;
  int p;
  float s;
  matrix_scale(part + e * d.parts, d.parts, eps, &p, &s);
  // Q's rows of the wave on their way while the columns are laid out
  constexpr int kHalves = Pairs<NB>::kBlocks * kBlock;
  const _Float16* Qh = Qm + e * 2 * kHalves;
  f16x8 qh[2][2 * NB], ql[2][2 * NB];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int rb = min(2 * wave_id() + i, NB - 1);  // an odd last row block is done twice, stored once
#pragma unroll
    for (int kk = 0; kk < 2 * NB; ++kk) {
      qh[i][kk] = fragment(Qh, NB, rb, kk);
      ql[i][kk] = fragment(Qh + kHalves, NB, rb, kk);
    }
  }
  load_columns<NB, false, LO, kApply * 64>(in, d, e, c0, p, s == s, hi, lo);
  __syncthreads();
  f32x16 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
#pragma unroll
  for (int kk = 0; kk < 2 * NB; ++kk) {
    f16x8 xh[2], xl[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      xh[j] = fragment(hi, kSub / 32, j, kk);
      if (LO) xl[j] = fragment(lo, kSub / 32, j, kk);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (LO) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(xl[j], qh[i][kk], acc[i][j], 0, 0, 0);
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(xh[j], ql[i][kk], acc[i][j], 0, 0, 0);
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(xh[j], qh[i][kk], acc[i][j], 0, 0, 0);
      }
    }
  }
  const float f = s * (1.f / kQScale);
  uint16_t* im = images[wave_id()];
  uint16_t* im2 = im;
  const int lane = lane_id();
  if constexpr (LO) {  // a step of weights is never without its momentum
    if (!out.U) {
      im2 = reinterpret_cast<uint16_t*>(cols) + wave_id() * 4096;
      __syncthreads();  // the columns are read
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x16& c = acc[i][j];
        const float y0 = c[4 * g] * f, y1 = c[4 * g + 1] * f, y2 = c[4 * g + 2] * f, y3 = c[4 * g + 3] * f;
        // the step of the weights as pairs of bf16, as in the tiled path
        const u32x2 a = pair_bf16x2(y0, y1), b = pair_bf16x2(y2, y3);
        const int row = 32 * i + (lane & 31), piece = 8 * j + 2 * g + (lane >> 5);
        image_put(im, row, piece, a[0], b[0]);
        if (LO && !out.U) image_put(im2, row, piece, a[1], b[1]);
      }
  image_sync();
  put_image(out, im, im2, d, e, 64 * wave_id(), c0);
}

template <int NB>
hipError_t run(const OrthoArgs& a, const OrthoIn& in, const OrthoDims& d, const NormPart* part, const OrthoOut& out,
               char* ws, hipStream_t st, KernelTimer* timer) {
  const SmallPlan p = small_plan(a, d.E);
  float* gram = reinterpret_cast<float*>(ws + p.gram);
  _Float16* q = reinterpret_cast<_Float16*>(ws + p.q);
  const bool lo = a.grad_f32 || in.mom;
  const unsigned E = unsigned(d.E);
  {
    TimedLaunch tl(timer, "ortho_small_gram", st);
    hipLaunchKernelGGL((lo ? ortho_small_gram_kernel<NB, true> : ortho_small_gram_kernel<NB, false>),
                       dim3(unsigned(p.parts), E), dim3(64 * kWaves<NB>), 0, st, in, d, part, a.eps, p.part_cols, gram);
  }
  {
    TimedLaunch tl(timer, "ortho_small_steps", st);
    hipLaunchKernelGGL(ortho_small_steps_kernel<NB>, dim3(E), dim3(64 * kWaves<NB>), 0, st, gram, p.parts, part, d.parts, a.eps, a.steps,
                       a.a, a.b, a.c, q);
  }
  TimedLaunch tl(timer, "ortho_small_apply", st);
  hipLaunchKernelGGL((lo ? ortho_small_apply_kernel<NB, true> : ortho_small_apply_kernel<NB, false>),
                     dim3(unsigned((d.n + kSub - 1) / kSub), E), dim3((NB + 1) / 2 * 64), 0, st, in, d, part, a.eps, q,
                     out);
  return hipGetLastError();
}

int row_blocks(const OrthoArgs& a) { return ((a.R < a.C ? a.R : a.C) + 31) / 32; }

}  // namespace

namespace {

// The largest |s (a + b s^2 + c s^4)| for s in [0, r], or r if that is larger.
double grown(const OrthoArgs& a, double r) {
  double most = r;
  auto at = [&](double x) { most = std::fmax(most, std::fabs(std::sqrt(x) * (a.a + x * (a.b + x * a.c)))); };
  at(r * r);
  const double p = 3.0 * a.b, q = 5.0 * a.c, disc = p * p - 4.0 * q * a.a;  // a + 3 b x + 5 c x^2 = 0
  if (q == 0.0) {
    if (p != 0.0 && -a.a / p > 0.0 && -a.a / p < r * r) at(-a.a / p);
  } else if (disc >= 0.0) {
    for (double x : {(-p - std::sqrt(disc)) / (2.0 * q), (-p + std::sqrt(disc)) / (2.0 * q)})
      if (x > 0.0 && x < r * r) at(x);
  }
  return most;
}

}  // namespace

// The squared singular values of the iterates must stay in [0, 2] (they start in
// [0, 1]), P = a + b x + c x^2 in [-a, a] there, and a^steps must leave Q the bits it
// needs, from above and from below.
bool small_fits(const OrthoArgs& a) {
  if ((a.R < a.C ? a.R : a.C) > kSmallSide) return false;
  if (!(a.a > 0.f && a.a <= 30.f && a.b <= 0.f && a.c >= 0.f)) return false;
  const double small_values = std::pow(double(a.a), a.steps);
  if (small_values > 1000.0 || small_values < 0x1p-8) return false;
  if (2.f * a.c > -a.b) return false;                                  // P(2) <= a, so P <= a on [0, 2]
  double r = 1.0;
  for (int i = 1; i < a.steps && r * r <= 2.0; ++i) r = grown(a, r);
  if (!(r * r <= 2.0)) return false;
  const float low = a.c > 0.f && -a.b < 4.f * a.c ? a.a - a.b * a.b / (4.f * a.c)  // the vertex lies in [0, 2]
                                                  : a.a + 2.f * a.b + 4.f * a.c;
  return low >= -a.a;
}

SmallPlan small_plan(const OrthoArgs& a, int64_t matrices) {
  SmallPlan p;
  const int n = a.R < a.C ? a.C : a.R;
  const int64_t mm = int64_t(row_blocks(a)) * row_blocks(a) * 1024;
  // at most 16 column ranges, of 64 columns at least
  p.part_cols = ((n + 15) / 16 + kSub - 1) / kSub * kSub;
  p.parts = (n + p.part_cols - 1) / p.part_cols;
  p.gram = 0;
  p.q = (size_t(matrices) * p.parts * mm * 4 + 255) / 256 * 256;
  p.total = p.q + size_t(matrices) * mm * 4;
  return p;
}

hipError_t launch_small(const OrthoArgs& a, const OrthoIn& in, const OrthoDims& d, const NormPart* part,
                        const OrthoOut& out, void* ws, hipStream_t st, KernelTimer* timer) {
  char* base = static_cast<char*>(ws);
  switch (row_blocks(a)) {
    case 1: return run<1>(a, in, d, part, out, base, st, timer);
    case 2: return run<2>(a, in, d, part, out, base, st, timer);
    case 3: return run<3>(a, in, d, part, out, base, st, timer);
    default: return run<4>(a, in, d, part, out, base, st, timer);
  }
}

}  // namespace ortho
}  // namespace moe
