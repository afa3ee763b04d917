// Newton-Schulz orthogonalisation of stacks of matrices (formulas and number
// formats in include/moe.h).
//
// A matrix is worked on as X [m][n] with m <= n (a tall G is transposed on the
// way in and out), padded with zeros to multiples of 128: the padding stays
// zero through every product. Per group of matrices:
//   ortho_norm    (momentum step and) the sum of squares, in 64 bits
//   ortho_load    X0 = G times a power of two, as fp16 value + E4M3 remainder
//   then per step
//   ortho_gram    A = X X^T
//   ortho_square  B = b A + c A A (A is symmetric, so A A = A A^T)
//   ortho_update  X' = a X + B X
// The last update writes U, or updates the weights, instead of X'.
//
// Numbers. Singular values far below the norm are multiplied by a (3.44) at
// every step, 480-fold in five, and so is whatever a step rounds away in
// their directions. X is therefore kept to about 15 bits (fp16 plus an E4M3
// remainder) in the linear term a X, whereas the products, whose factor B is
// small exactly in those directions, take the fp16 part. B's diagonal is near
// b + c for converged rows and would carry the largest rounding: what its
// rounding lost is kept in fp32 and added with the linear term. Measured
// against 64 bits after the bf16 output rounding (1.7e-3 by itself): 1.8e-3
// to 2.3e-3 on inputs of every rank; fp16 alone is 2.6e-2 off on low ranks,
// bf16 products 1.3e-2 on full ones.
#include <cmath>

#include "device_common.h"
#include "kernels.h"

namespace moe {

namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

constexpr int kNormThreads = 256;
constexpr int kNormParts = 64;      // partial sums per matrix
constexpr int kLoadTile = 64;
// iterates after the first step are stored times 2^10 (so that rows far below
// the norm keep their bits in fp16); their remainder times another 2^10
constexpr float kXScale = 1024.f;
constexpr float kLoScale = 1024.f;
// X0 has a norm in [2^14, 2^15): a remainder is below 2^4
constexpr int kX0Exp = 14;
constexpr float kLoScale0 = 16.f;

struct OrthoDims {
  int64_t E;   // matrices of the group
  int R, C;    // as given
  int m, n;    // smaller, larger side
  int mp, np;  // padded
  bool tall;   // R > C: X = G^T
};

// ------------------------------------------------------------------ input

__device__ __forceinline__ float grad_at(const void* g, bool f32, int64_t i) {
  return f32 ? static_cast<const float*>(g)[i]
             : __uint_as_float(uint32_t(static_cast<const uint16_t*>(g)[i]) << 16);
}

// Partial sums of squares, after the momentum step if there is one.
__global__ __launch_bounds__(kNormThreads) void ortho_norm_kernel(const void* __restrict__ grad, bool f32,
                                                                  float* __restrict__ mom, float mu, bool nesterov,
                                                                  int64_t count, double* __restrict__ part) {
  __shared__ double sm[kNormThreads];
  const int64_t base = int64_t(blockIdx.y) * count;
  double s = 0.0;
  for (int64_t i = int64_t(blockIdx.x) * kNormThreads + threadIdx.x; i < count; i += int64_t(kNormParts) * kNormThreads) {
    float x = grad_at(grad, f32, base + i);
    if (mom) {
      const float m = mu * mom[base + i] + x;
      mom[base + i] = m;
      x = nesterov ? x + mu * m : m;
    }
    s += double(x) * double(x);
  }
  sm[threadIdx.x] = s;
  __syncthreads();
  for (int o = kNormThreads / 2; o > 0; o >>= 1) {
    if (int(threadIdx.x) < o) sm[threadIdx.x] += sm[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) part[int64_t(blockIdx.y) * kNormParts + blockIdx.x] = sm[0];
}

// The exponent p of X0 = G 2^p, and s = 1 / ((|G| + eps) 2^p).
__device__ __forceinline__ void matrix_scale(const double* __restrict__ part, float eps, int* p, float* s) {
  double q = 0.0;
  for (int i = 0; i < kNormParts; ++i) q += part[i];
  const double norm = sqrt(q);
  const bool plain = norm > 0.0 && norm < 1e300;
  *p = plain ? kX0Exp - ilogb(norm) : 0;
  *s = norm == 0.0 ? 0.f : float(ldexp(1.0 / (norm + double(eps)), -*p));
  if (!(norm < 1e300)) *s = NAN;
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const _Float16 x = static_cast<_Float16>(a), y = static_cast<_Float16>(b);
  return uint32_t(__builtin_bit_cast(uint16_t, x)) | (uint32_t(__builtin_bit_cast(uint16_t, y)) << 16);
}

__device__ __forceinline__ uint8_t e4m3_of(float v) {
  const float c = fminf(fmaxf(v, -448.f), 448.f);
  return uint8_t(__builtin_amdgcn_cvt_pk_fp8_f32(c, 0.f, 0, false) & 0xff);
}
__device__ __forceinline__ float e4m3_to(uint8_t v) {
  return __builtin_amdgcn_cvt_f32_fp8(int(v), 0);
}

// X0 and its remainder, 64 x 64 elements a workgroup, through LDS when G is
// transposed.
__global__ __launch_bounds__(256) void ortho_load_kernel(const void* __restrict__ grad, bool f32,
                                                         const float* __restrict__ mom, float mu, bool nesterov,
                                                         OrthoDims d, const double* __restrict__ part, float eps,
                                                         _Float16* __restrict__ X, uint8_t* __restrict__ Xl,
                                                         float* __restrict__ scale) {
  __shared__ float tile[kLoadTile][kLoadTile + 1];
  const int e = blockIdx.z, r0 = blockIdx.y * kLoadTile, c0 = blockIdx.x * kLoadTile;
  int p;
  float s;
  matrix_scale(part + int64_t(e) * kNormParts, eps, &p, &s);
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) scale[e] = s;
  // r, c: position in X
  for (int i = threadIdx.x; i < kLoadTile * kLoadTile; i += 256) {
    const int a = i / kLoadTile, b = i % kLoadTile;
    const int gr = d.tall ? c0 + a : r0 + a, gc = d.tall ? r0 + b : c0 + b;
    float x = 0.f;
    if (gr < d.R && gc < d.C) {
      const int64_t at = (int64_t(e) * d.R + gr) * d.C + gc;
      x = grad_at(grad, f32, at);
      if (mom) x = nesterov ? x + mu * mom[at] : mom[at];
      x = s == s ? ldexpf(x, p) : NAN;
    }
    tile[d.tall ? b : a][d.tall ? a : b] = x;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kLoadTile * kLoadTile; i += 256) {
    const int a = i / kLoadTile, b = i % kLoadTile;
    const float x = tile[a][b];
    const _Float16 h = static_cast<_Float16>(x);
    const int64_t at = (int64_t(e) * d.mp + r0 + a) * d.np + c0 + b;
    X[at] = h;
    if (Xl) Xl[at] = e4m3_of((x - float(h)) * kLoScale0);
  }
}

// ------------------------------------------------------------------ products

// One 128 x 128 tile of P Q^T-like products on v_mfma_f32_32x32x16_f16: 4
// waves of 64 x 64, k-slabs of 32 through registers into LDS.
constexpr int kT = 128;
constexpr int kK = 32;
constexpr int kLd = kK + 8;

struct TileAcc {
  f32x16 c[2][2];
};

// rows [e0, e0 + 128) of a k-contiguous operand
__device__ __forceinline__ void stage_k(const _Float16* __restrict__ src, int64_t ld, int e0, int k0, _Float16* lds) {
  for (int i = threadIdx.x; i < kT * kK / 8; i += 256) {
    const int r = i / (kK / 8), c = i % (kK / 8);
    *reinterpret_cast<f16x8*>(lds + r * kLd + 8 * c) =
        *reinterpret_cast<const f16x8*>(src + int64_t(e0 + r) * ld + k0 + 8 * c);
  }
}
// columns [e0, e0 + 128) of an operand whose rows are k
__device__ __forceinline__ void stage_mn(const _Float16* __restrict__ src, int64_t ld, int e0, int k0, _Float16* lds) {
  for (int i = threadIdx.x; i < kT * kK / 8; i += 256) {
    const int k = i / (kT / 8), c = i % (kT / 8);
    const f16x8 v = *reinterpret_cast<const f16x8*>(src + int64_t(k0 + k) * ld + e0 + 8 * c);
#pragma unroll
    for (int j = 0; j < 8; ++j) lds[(8 * c + j) * kLd + k] = v[j];
  }
}

template <bool Q_MN>
__device__ __forceinline__ void tile_product(const _Float16* __restrict__ P, int64_t ldp, int p0,
                                             const _Float16* __restrict__ Q, int64_t ldq, int q0, int K,
                                             _Float16* lp, _Float16* lq, TileAcc& acc) {
  const int wave = threadIdx.x >> 6, lane = lane_id();
  const int pm = (wave >> 1) * 64, qn = (wave & 1) * 64;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc.c[i][j][r] = 0.f;
  for (int k0 = 0; k0 < K; k0 += kK) {
    __syncthreads();
    stage_k(P, ldp, p0, k0, lp);
    if (Q_MN) stage_mn(Q, ldq, q0, k0, lq); else stage_k(Q, ldq, q0, k0, lq);
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < kK; kk += 16) {
      f16x8 pf[2], qf[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        pf[i] = *reinterpret_cast<const f16x8*>(lp + (pm + 32 * i + (lane & 31)) * kLd + kk + 8 * (lane >> 5));
        qf[i] = *reinterpret_cast<const f16x8*>(lq + (qn + 32 * i + (lane & 31)) * kLd + kk + 8 * (lane >> 5));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc.c[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(qf[j], pf[i], acc.c[i][j], 0, 0, 0);
    }
  }
}

// Row and first of 4 columns, inside the tile, of registers 4g .. 4g+3 of sub-tile (i, j).
__device__ __forceinline__ int tile_row(int i) { return ((threadIdx.x >> 7) * 64) + 32 * i + (lane_id() & 31); }
__device__ __forceinline__ int tile_col(int j, int g) {
  return ((threadIdx.x >> 6) & 1) * 64 + 32 * j + 8 * g + 4 * (lane_id() >> 5);
}

// A = X X^T times the square of the iterate's scale. Symmetric: tiles (bi, bj)
// with bj <= bi only, each also written transposed.
__global__ __launch_bounds__(256) void ortho_gram_kernel(const _Float16* __restrict__ X, OrthoDims d,
                                                         const float* __restrict__ scale, _Float16* __restrict__ A) {
  __shared__ __attribute__((aligned(16))) _Float16 lp[kT * kLd], lq[kT * kLd];
  const int bi = blockIdx.y, bj = blockIdx.x, e = blockIdx.z;
  if (bj > bi) return;
  const _Float16* Xe = X + int64_t(e) * d.mp * d.np;
  _Float16* Ae = A + int64_t(e) * d.mp * d.mp;
  TileAcc acc;
  tile_product<false>(Xe, d.np, bi * kT, Xe, d.np, bj * kT, d.np, lp, lq, acc);
  const float s = scale ? scale[e] : 1.f / kXScale;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int r = bi * kT + tile_row(i), c = bj * kT + tile_col(j, g) + t;
          const _Float16 v = static_cast<_Float16>(acc.c[i][j][4 * g + t] * s * s);
          Ae[int64_t(r) * d.mp + c] = v;
          if (bi != bj) Ae[int64_t(c) * d.mp + r] = v;
        }
}

// B = b A + c A A in fp16, and what the rounding of its diagonal lost.
__global__ __launch_bounds__(256) void ortho_square_kernel(const _Float16* __restrict__ A, OrthoDims d, float cb,
                                                           float cc, _Float16* __restrict__ B,
                                                           float* __restrict__ diag) {
  __shared__ __attribute__((aligned(16))) _Float16 lp[kT * kLd], lq[kT * kLd];
  const int bi = blockIdx.y, bj = blockIdx.x, e = blockIdx.z;
  if (bj > bi) return;
  const _Float16* Ae = A + int64_t(e) * d.mp * d.mp;
  _Float16* Be = B + int64_t(e) * d.mp * d.mp;
  TileAcc acc;
  tile_product<false>(Ae, d.mp, bi * kT, Ae, d.mp, bj * kT, d.mp, lp, lq, acc);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int r = bi * kT + tile_row(i), c = bj * kT + tile_col(j, g) + t;
          const float x = cb * float(Ae[int64_t(r) * d.mp + c]) + cc * acc.c[i][j][4 * g + t];
          const _Float16 v = static_cast<_Float16>(x);
          Be[int64_t(r) * d.mp + c] = v;
          if (bi != bj) Be[int64_t(c) * d.mp + r] = v;
          if (r == c) diag[int64_t(e) * d.mp + r] = x - float(v);
        }
}

struct OrthoOut {
  _Float16* X;      // next iterate (NULL in the last step)
  uint8_t* Xl;      // its remainder
  uint16_t* U;      // last step: the result, or
  uint16_t* W;      // the weights it updates (with master: their fp32 form)
  float* master;
  float keep, step;  // W keep - step U
};

__global__ __launch_bounds__(256) void ortho_update_kernel(const _Float16* __restrict__ X,
                                                           const uint8_t* __restrict__ Xl, float lo_inv,
                                                           const _Float16* __restrict__ B,
                                                           const float* __restrict__ diag, OrthoDims d, float ca,
                                                           const float* __restrict__ scale, OrthoOut out) {
  __shared__ __attribute__((aligned(16))) _Float16 lp[kT * kLd], lq[kT * kLd];
  const int bi = blockIdx.y, bj = blockIdx.x, e = blockIdx.z;
  const int64_t xo = int64_t(e) * d.mp * d.np;
  TileAcc acc;
  tile_product<true>(B + int64_t(e) * d.mp * d.mp, d.mp, bi * kT, X + xo, d.np, bj * kT, d.mp, lp, lq, acc);
  const float s = scale ? scale[e] : 1.f / kXScale;  // takes a stored iterate to its value
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = bi * kT + tile_row(i);
    const float lin = ca + diag[int64_t(e) * d.mp + r];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int c = bj * kT + tile_col(j, g) + t;
          const int64_t at = xo + int64_t(r) * d.np + c;
          float x = float(X[at]);
          if (Xl) x += e4m3_to(Xl[at]) * lo_inv;
          const float y = (lin * x + acc.c[i][j][4 * g + t]) * s;
          if (out.X) {
            const float z = y * kXScale;
            const _Float16 h = static_cast<_Float16>(z);
            out.X[at] = h;
            if (out.Xl) out.Xl[at] = e4m3_of((z - float(h)) * kLoScale);
          } else if (r < d.m && c < d.n) {
            const int64_t o = int64_t(e) * d.R * d.C + (d.tall ? int64_t(c) * d.C + r : int64_t(r) * d.C + c);
            if (out.U) {
              out.U[o] = uint16_t(pack_bf16x2(y, 0.f));
            } else {
              const float w = out.master ? out.master[o] : __uint_as_float(uint32_t(out.W[o]) << 16);
              const float v = out.keep * w - out.step * y;
              if (out.master) out.master[o] = v;
              out.W[o] = uint16_t(pack_bf16x2(v, 0.f));
            }
          }
        }
  }
}

// ------------------------------------------------------------------ plan

struct OrthoPlan {
  OrthoDims d;
  int64_t group;                            // matrices at a time
  size_t part, scale, X[2], Xl[2], A, B, diag, total;  // workspace offsets
};

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

OrthoPlan ortho_plan(const OrthoArgs& a) {
  OrthoPlan p;
  OrthoDims& d = p.d;
  d.R = a.R;
  d.C = a.C;
  d.tall = a.R > a.C;
  d.m = d.tall ? a.C : a.R;
  d.n = d.tall ? a.R : a.C;
  d.mp = (d.m + kT - 1) / kT * kT;
  d.np = (d.n + kT - 1) / kT * kT;
  const int64_t x = int64_t(d.mp) * d.np, q = int64_t(d.mp) * d.mp;
  // at most about 4 GiB of state
  const int64_t bytes = 6 * x + 4 * q;
  int64_t g = (int64_t(4) << 30) / bytes;
  g = g < 1 ? 1 : (g > 4096 ? 4096 : g);
  p.group = a.E < g ? (a.E > 0 ? a.E : 1) : g;
  size_t o = 0;
  p.part = o;  o = up256(o + size_t(p.group) * kNormParts * 8);
  p.scale = o; o = up256(o + size_t(p.group) * 4);
  p.diag = o;  o = up256(o + size_t(p.group) * d.mp * 4);
  for (int i = 0; i < 2; ++i) {
    p.X[i] = o;  o = up256(o + size_t(p.group) * x * 2);
    p.Xl[i] = o; o = up256(o + size_t(p.group) * x);
  }
  p.A = o; o = up256(o + size_t(p.group) * q * 2);
  p.B = o; o = up256(o + size_t(p.group) * q * 2);
  p.total = o;
  return p;
}

}  // namespace

size_t ortho_workspace_bytes(const OrthoArgs& a) { return ortho_plan(a).total; }

hipError_t launch_ortho(const OrthoArgs& a, const OrthoTarget& t, void* ws, hipStream_t st, KernelTimer* timer) {
  if (a.E <= 0) return hipSuccess;
  const OrthoPlan p = ortho_plan(a);
  char* base = static_cast<char*>(ws);
  auto f16 = [&](size_t o) { return reinterpret_cast<_Float16*>(base + o); };
  auto u8 = [&](size_t o) { return reinterpret_cast<uint8_t*>(base + o); };
  auto f32 = [&](size_t o) { return reinterpret_cast<float*>(base + o); };
  double* part = reinterpret_cast<double*>(base + p.part);
  const int64_t count = int64_t(a.R) * a.C;
  const size_t gsize = a.grad_f32 ? 4 : 2;
  for (int64_t e0 = 0; e0 < a.E; e0 += p.group) {
    OrthoDims d = p.d;
    d.E = a.E - e0 < p.group ? a.E - e0 : p.group;
    const unsigned ge = unsigned(d.E);
    const void* grad = static_cast<const char*>(t.grad) + size_t(e0) * count * gsize;
    float* mom = t.momentum ? t.momentum + e0 * count : nullptr;
    {
      TimedLaunch tl(timer, "ortho_norm", st);
      hipLaunchKernelGGL(ortho_norm_kernel, dim3(kNormParts, ge), dim3(kNormThreads), 0, st, grad, a.grad_f32, mom, t.mu,
                         t.nesterov, count, part);
    }
    const bool lo0 = a.grad_f32 || mom;  // a bf16 G is exact in fp16
    {
      TimedLaunch tl(timer, "ortho_load", st);
      hipLaunchKernelGGL(ortho_load_kernel, dim3(d.np / kLoadTile, d.mp / kLoadTile, ge), dim3(256), 0, st, grad,
                         a.grad_f32, mom, t.mu, t.nesterov, d, part, a.eps, f16(p.X[0]), lo0 ? u8(p.Xl[0]) : nullptr,
                         f32(p.scale));
    }
    for (int k = 0; k < a.steps; ++k) {
      const int in = k & 1;
      const float* scale = k == 0 ? f32(p.scale) : nullptr;
      const dim3 sym(d.mp / kT, d.mp / kT, ge);
      {
        TimedLaunch tl(timer, "ortho_gram", st);
        hipLaunchKernelGGL(ortho_gram_kernel, sym, dim3(256), 0, st, f16(p.X[in]), d, scale, f16(p.A));
      }
      {
        TimedLaunch tl(timer, "ortho_square", st);
        hipLaunchKernelGGL(ortho_square_kernel, sym, dim3(256), 0, st, f16(p.A), d, a.b, a.c, f16(p.B), f32(p.diag));
      }
      OrthoOut out{};
      if (k + 1 < a.steps) {
        out.X = f16(p.X[1 - in]);
        out.Xl = u8(p.Xl[1 - in]);
      } else {
        out.U = t.U ? t.U + e0 * count : nullptr;
        out.W = t.W ? t.W + e0 * count : nullptr;
        out.master = t.master ? t.master + e0 * count : nullptr;
        out.keep = t.keep;
        out.step = t.step;
      }
      const bool lo = k > 0 || lo0;
      TimedLaunch tl(timer, "ortho_update", st);
      hipLaunchKernelGGL(ortho_update_kernel, dim3(d.np / kT, d.mp / kT, ge), dim3(256), 0, st, f16(p.X[in]),
                         lo ? u8(p.Xl[in]) : nullptr, 1.f / (k == 0 ? kLoScale0 : kLoScale), f16(p.B), f32(p.diag), d,
                         a.a, scale, out);
    }
  }
  return hipGetLastError();
}

}  // namespace moe
