// What the kernels of the Newton-Schulz orthogonalisation share (ortho.hip: matrices
// of any size in tiles; ortho_small.hip: small ones): input, scales, the block
// layout of fragments, and the way out to the caller's matrices.
#pragma once

#include "device_common.h"
#include "kernels.h"

namespace moe {
namespace ortho {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

constexpr int kNormThreads = 256;
// Vectors at any address of their elements: the caller's rows begin anywhere.
typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));

constexpr int kLoadTile = 64;
// An iterate is stored times 2^15 (its elements stay below 2, fp16 ends at
// 65504), X0 times the power of two that takes its largest element to [2^14,
// 2^15): what the rounding to fp16 leaves is 16 at most, and lies well inside
// E4M3's range for elements down to 2^-20 of the largest.
constexpr float kXScale = 32768.f;
constexpr int kX0Exp = 14;

struct OrthoDims {
  int64_t E;   // matrices of the group
  int R, C;    // as given
  int m, n;    // smaller, larger side
  int mp, np;  // padded
  bool tall;   // R > C: X = G^T
  int parts;   // partial sums of the norm: 64 or 256
};

// X, A and B live in the workspace in blocks of 32 rows x 16 columns (1 KiB), the
// row blocks of a column block one after the other. A block is an MFMA fragment
// in the order of its lanes: 16-byte chunk h (columns 8 h .. 8 h + 7) of row r
// at slot 32 h + (r ^ 4 h). So a load of a wave moves a block into LDS as it
// lies, a fragment with k along the rows is one linear LDS read, a store of a
// 32 x 16 result is one linear 1 KiB, and in the transpose read (two chunks of four
// rows) the 16 lanes of a group find their rows of both chunks in different banks
// (the xor). The two groups of a half wave read column blocks 1 KiB apart, which are
// the same banks: 29 to 32 % of the update's LDS cycles are conflicts.
// Row-major matrices (64-byte pieces of 16 rows a load) cost 13 to 25 % of the
// products' time.
constexpr int kBlock = 512;  // halves
__device__ __forceinline__ int64_t block_at(int rows, int rb, int cb) { return (int64_t(cb) * (rows / 32) + rb) * kBlock; }
// element (r, 8 h ..) inside a block
__device__ __forceinline__ int in_block(int r, int h) { return (32 * h + (r ^ (4 * h))) * 8; }

// ------------------------------------------------------------------ input

__device__ __forceinline__ float grad_at(const void* g, bool f32, int64_t i) {
  return f32 ? static_cast<const float*>(g)[i]
             : __uint_as_float(uint32_t(static_cast<const uint16_t*>(g)[i]) << 16);
}

// What is orthogonalised.
struct OrthoIn {
  const void* grad;
  bool f32;
  float* mom;  // NULL: the gradient itself
  float mu;
  bool nesterov;
};

// Eight neighbouring gradient values.
__device__ __forceinline__ void grad8(const OrthoIn& in, int64_t i, float (&x)[8]) {
  if (in.f32) {
    const f32x4u* p = reinterpret_cast<const f32x4u*>(static_cast<const float*>(in.grad) + i);
    const f32x4 a = p[0], b = p[1];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      x[t] = a[t];
      x[4 + t] = b[t];
    }
  } else {
    const u32x4 a = *reinterpret_cast<const u32x4u*>(static_cast<const uint16_t*>(in.grad) + i);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      x[2 * t] = bf16_lo(a[t]);
      x[2 * t + 1] = bf16_hi(a[t]);
    }
  }
}

// One element of what is orthogonalised, the momentum being up to date.
__device__ __forceinline__ float input_at(const OrthoIn& in, int64_t i) {
  if (!in.mom) return grad_at(in.grad, in.f32, i);
  return in.nesterov ? grad_at(in.grad, in.f32, i) + in.mu * in.mom[i] : in.mom[i];
}
__device__ __forceinline__ void input8(const OrthoIn& in, int64_t i, float (&x)[8]) {
  if (!in.mom || in.nesterov) grad8(in, i, x);
  if (in.mom) {
    const f32x4u* p = reinterpret_cast<const f32x4u*>(in.mom + i);
    const f32x4 a = p[0], b = p[1];
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const float m = t < 4 ? a[t & 3] : b[t & 3];
      x[t] = in.nesterov ? x[t] + in.mu * m : m;
    }
  }
}

// The same of a row's end: `left` of them exist, the others are not touched.
__device__ __forceinline__ void input_row(const OrthoIn& in, int64_t i, int left, float (&x)[8]) {
  if (left >= 8) {
    input8(in, i, x);
  } else {
#pragma unroll
    for (int t = 0; t < 8; ++t)
      if (t < left) x[t] = input_at(in, i + t);
  }
}

// What the norm pass leaves of a part of a matrix.
struct NormPart {
  double sum;  // of squares
  float amax;  // largest magnitude
  float pad;
};

// The exponent p of X0 = G 2^p, and s = 1 / ((|G| + eps) 2^p), in every lane.
__device__ __forceinline__ void matrix_scale(const NormPart* __restrict__ part, int parts, float eps, int* p, float* s) {
  double q = part[lane_id()].sum;
  float m = part[lane_id()].amax;
  if (parts > 64) {
    NormPart n[3];  // 256 parts, read at once
#pragma unroll
    for (int i = 0; i < 3; ++i) n[i] = part[64 * (i + 1) + lane_id()];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      q += n[i].sum;
      m = fmaxf(m, n[i].amax);
    }
  }
  for (int o = 32; o > 0; o >>= 1) {
    q += __shfl_xor(q, o);
    m = fmaxf(m, __shfl_xor(m, o));
  }
  const double norm = sqrt(q);
  const bool finite = norm < 1e300;
  *p = finite && m > 0.f ? kX0Exp - ilogbf(m) : 0;
  *s = !finite ? NAN : norm == 0.0 ? 0.f : float(ldexp(1.0 / (norm + double(eps)), -*p));
}

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {  // v_cvt_pk_f16_f32, nearest even
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
}

// ------------------------------------------------------------------ fragments and images

typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef short v8i16 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) v4i16 lds_v4i16;

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6)); }
__device__ __forceinline__ float half_of(uint32_t w, int t) {
  return float(__builtin_bit_cast(_Float16, uint16_t(t ? w >> 16 : w)));
}

// A 32 x 32 sub-tile of a matrix of blocks as the accumulators hold it: w[g]
// the lane's four values of run g (row lane % 32, columns 8 g + 4 (lane / 32) ..
// + 3). The swap of the upper half of one register with the lower half of
// another turns whole 16-byte chunks into runs, and back in put_subtile.
__device__ __forceinline__ void get_subtile(const _Float16* __restrict__ src, int rows, int row0, int col0,
                                            u32x2 (&w)[4]) {
  const int at = in_block(lane_id() & 31, lane_id() >> 5);
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(src + block_at(rows, row0 / 32, col0 / 16 + p) + at);
    const auto a = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
    w[2 * p] = u32x2{a[0], b[0]};
    w[2 * p + 1] = u32x2{a[1], b[1]};
  }
}
__device__ __forceinline__ void put_subtile(const u32x2 (&w)[4], _Float16* __restrict__ out, int rows, int row0,
                                            int col0) {
  const int at = in_block(lane_id() & 31, lane_id() >> 5);
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const auto a = __builtin_amdgcn_permlane32_swap(w[2 * p][0], w[2 * p + 1][0], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(w[2 * p][1], w[2 * p + 1][1], false, false);
    *reinterpret_cast<u32x4*>(out + block_at(rows, row0 / 32, col0 / 16 + p) + at) = u32x4{a[0], b[0], a[1], b[1]};
  }
}

// ------------------------------------------------------------------ images
//
// What has to leave in another order than the registers' (the mirrored half of
// a symmetric product, the caller's row-major result) goes through LDS, 64
// rows x 64 columns of 16-bit values of a wave at a time (8 KiB of its own: no
// barrier): 16-byte chunk c of row r at c ^ ((r / 2) % 8). Rows come out as
// 16-byte pieces, columns through the transpose read.

// four values of row r (0 .. 63), columns 4 q .. 4 q + 3
__device__ __forceinline__ void image_put(uint16_t* im, int r, int q, uint32_t lo, uint32_t hi) {
  u32x2 v = {lo, hi};
  *reinterpret_cast<u32x2*>(im + r * 64 + (((q >> 1) ^ ((r >> 1) & 7)) << 3) + (q & 1) * 4) = v;
}
// eight values of row r, columns 8 c .. 8 c + 7
__device__ __forceinline__ u32x4 image_row(const uint16_t* im, int r, int c) {
  return *reinterpret_cast<const u32x4*>(im + r * 64 + ((c ^ ((r >> 1) & 7)) << 3));
}
// Every lane: eight values of one column, rows r0 .. r0 + 7, for the 16
// columns from n0 on (column n0 + lane % 16; r0 and n0 may differ from one
// 16-lane group to another).
__device__ __forceinline__ u32x4 image_col(const uint16_t* im, int r0, int n0) {
  const int p = lane_id() & 15;
  const int r = r0 + (p >> 2), n = n0 + 4 * (p & 3);
  // rows r and r + 4 differ in the chunk's position
  const uint16_t* a = im + r * 64 + (((n >> 3) ^ ((r >> 1) & 7)) << 3) + (n & 7);
  const uint16_t* b = im + (r + 4) * 64 + (((n >> 3) ^ (((r + 4) >> 1) & 7)) << 3) + (n & 7);
  const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(a));
  const v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(b));
  return __builtin_bit_cast(u32x4, v8i16(__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7)));
}
// LDS writes of the wave are visible to its own reads
__device__ __forceinline__ void image_sync() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  asm volatile("" ::: "memory");
}

struct OrthoOut {
  _Float16* X;      // next iterate (NULL in the last step)
  uint8_t* Xl;      // its remainder
  uint16_t* U;      // last step: the result, or
  uint16_t* W;      // the weights it updates (with master: their fp32 form)
  float* master;
  float keep, step;  // W keep - step U
};

__device__ __forceinline__ float bf16_at(const uint16_t* p) { return __uint_as_float(uint32_t(*p) << 16); }

// Two values as pairs of bf16 (16 bits and fp32's range): upper and lower halves.
__device__ __forceinline__ u32x2 pair_bf16x2(float a, float b) {
  const uint32_t hi = pack_bf16x2(a, b);
  return u32x2{hi, pack_bf16x2(a - bf16_lo(hi), b - bf16_hi(hi))};
}

// Eight consecutive elements of the result at element `at` of matrix storage:
// v holds bf16 values of U; for the step of W, v and l hold its pairs. Only `count`
// of them exist; eight go at once.
__device__ __forceinline__ void put_result(const OrthoOut& out, int64_t at, const u32x4& v, const u32x4& l, int count) {
  const bool vec = count >= 8;
  if (out.U) {
    if (vec) {
      *reinterpret_cast<u32x4u*>(out.U + at) = v;
    } else {
#pragma unroll
      for (int t = 0; t < 8; ++t)
        if (t < count) out.U[at + t] = uint16_t(v[t >> 1] >> (16 * (t & 1)));
    }
    return;
  }
  float w[8];
  if (vec) {
    if (out.master) {
      const f32x4 a = *reinterpret_cast<const f32x4u*>(out.master + at);
      const f32x4 b = *reinterpret_cast<const f32x4u*>(out.master + at + 4);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        w[t] = a[t];
        w[4 + t] = b[t];
      }
    } else {
      const u32x4 a = *reinterpret_cast<const u32x4u*>(out.W + at);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        w[2 * t] = bf16_lo(a[t]);
        w[2 * t + 1] = bf16_hi(a[t]);
      }
    }
  } else {
#pragma unroll
    for (int t = 0; t < 8; ++t) w[t] = t < count ? (out.master ? out.master[at + t] : bf16_at(out.W + at + t)) : 0.f;
  }
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    const float u = t & 1 ? bf16_hi(v[t >> 1]) + bf16_hi(l[t >> 1]) : bf16_lo(v[t >> 1]) + bf16_lo(l[t >> 1]);
    w[t] = out.keep * w[t] - out.step * u;
  }
  if (vec) {
    if (out.master) {
      *reinterpret_cast<f32x4u*>(out.master + at) = f32x4{w[0], w[1], w[2], w[3]};
      *reinterpret_cast<f32x4u*>(out.master + at + 4) = f32x4{w[4], w[5], w[6], w[7]};
    }
    *reinterpret_cast<u32x4u*>(out.W + at) = u32x4{pack_bf16x2(w[0], w[1]), pack_bf16x2(w[2], w[3]),
                                                  pack_bf16x2(w[4], w[5]), pack_bf16x2(w[6], w[7])};
  } else {
#pragma unroll
    for (int t = 0; t < 8; ++t)
      if (t < count) {
        if (out.master) out.master[at + t] = w[t];
        out.W[at + t] = uint16_t(pack_bf16x2(w[t], 0.f));
      }
  }
}

// The 64 x 64 values of a wave's image (rows row0 .., columns col0 .. of X) to the
// caller's matrix e. iml: the image of the pairs' lower halves, for the step of W.
__device__ __forceinline__ void put_image(const OrthoOut& out, const uint16_t* im, const uint16_t* iml,
                                          const OrthoDims& d, int64_t e, int row0, int col0) {
  const int lane = lane_id();
  for (int q = 0; q < 8; ++q) {
    if (!d.tall) {
      const int r = row0 + 8 * q + (lane >> 3), c = col0 + 8 * (lane & 7);
      const u32x4 v = image_row(im, 8 * q + (lane >> 3), lane & 7);
      u32x4 l = {0u, 0u, 0u, 0u};
      if (!out.U) l = image_row(iml, 8 * q + (lane >> 3), lane & 7);
      if (r < d.m && c < d.n) put_result(out, (e * d.R + r) * int64_t(d.C) + c, v, l, d.n - c);
    } else {
      // 16 columns of X (rows of the result) x four pieces of 8 rows: 64 bytes a row
      const int r0 = 32 * (q & 1) + 8 * (lane >> 4), n0 = 16 * (q >> 1);
      const int r = row0 + r0, c = col0 + n0 + (lane & 15);
      const u32x4 v = image_col(im, r0, n0);
      u32x4 l = {0u, 0u, 0u, 0u};
      if (!out.U) l = image_col(iml, r0, n0);
      if (r < d.m && c < d.n) put_result(out, (e * d.R + c) * int64_t(d.C) + r, v, l, d.m - r);
    }
  }
}

// ------------------------------------------------------------------ small matrices (ortho_small.hip)

// Sides up to this run there, where small_fits says so.
constexpr int kSmallSide = 128;
bool small_fits(const OrthoArgs& a);
// Workspace of a group: the sums over parts of X X^T, then the factors Q.
struct SmallPlan {
  int parts;        // column ranges of X
  int part_cols;    // their width, a multiple of 64
  size_t gram, q, total;
};
SmallPlan small_plan(const OrthoArgs& a, int64_t matrices);
hipError_t launch_small(const OrthoArgs& a, const OrthoIn& in, const OrthoDims& d, const NormPart* part,
                        const OrthoOut& out, void* ws, hipStream_t st, KernelTimer* timer);

}  // namespace ortho
}  // namespace moe
