// Newton-Schulz orthogonalisation of stacks of matrices (formulas and number
// formats in include/moe.h).
//
// A matrix is worked on as X [m][n] with m <= n (a tall G is transposed on the
// way in and out), padded with zeros to multiples of 128: the padding stays
// zero through every product. Per group of matrices:
//   ortho_norm    (momentum step and) the sum of squares, in 64 bits
//   ortho_load    X0 = G times a power of two, as fp16 value + E4M3 remainder
//   then per step
//   ortho_gram    A = X X^T (few tiles over a long axis: in parts, ortho_gram_part
//                 and ortho_gram_join)
//   ortho_square  B = b A + c A A (A is symmetric, so A A = A A^T)
//   ortho_update  X' = a X + B X
// The last update writes U, or updates the weights, instead of X'. Wide matrices
// take the first two steps as one (ortho_pairs): with P = a + B, the second step's
// X X^T is P A P, and X'' = P2 P X = (a^2 + D) X, all but the last product m x m.
// Matrices of at most 128 rows have a path of their own (ortho_small.hip).
//
// Numbers. Singular values far below the norm are multiplied by a (3.44) at
// every step, 480-fold in five, and so is whatever a step rounds away in
// their directions. X is therefore kept to about 15 bits (fp16 plus an E4M3
// remainder) in the linear term a X, whereas the products, whose factor B is
// small exactly in those directions, take the fp16 part. B's diagonal is near
// b + c for converged rows and would carry the largest rounding: what its
// rounding lost is kept in fp32 and added with the linear term. Measured
// against 64 bits after the bf16 output rounding (1.7e-3 by itself): 1.6e-3
// to 2.4e-3 on bf16 inputs of every rank (fp32 inputs, which X0 rounds: 3.9e-3 on
// rank one, 2.1e-3 on full rank); fp16 alone is 2.6e-2 off on low ranks,
// bf16 products 1.3e-2 on full ones.
#include <cmath>

#include "ortho_device.h"

namespace moe {

using namespace ortho;

namespace {

// Partial sums of squares and maxima, after the momentum step if there is one.
// HBM-bound (128 of 768 x 2048 in bf16: 403 MB in 87 us, 4.6 TB/s).
__global__ __launch_bounds__(kNormThreads) void ortho_norm_kernel(OrthoIn in, int64_t count,
                                                                  NormPart* __restrict__ part) {
  __shared__ double sm[kNormThreads / 64];
  __shared__ float mx[kNormThreads / 64];
  const int64_t base = int64_t(blockIdx.y) * count;
  const int64_t first = int64_t(blockIdx.x) * kNormThreads + threadIdx.x;
  const int64_t step = int64_t(gridDim.x) * kNormThreads;
  double s = 0.0;
  float m = 0.f;  // fmaxf drops a NaN; the sum keeps it
#pragma unroll 2
  for (int64_t i = first * 8; i + 8 <= count; i += step * 8) {
    float x[8];
    grad8(in, base + i, x);
    if (in.mom) {
      f32x4u* p = reinterpret_cast<f32x4u*>(in.mom + base + i);
      f32x4 a = p[0], b = p[1];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        a[t] = in.mu * a[t] + x[t];
        b[t] = in.mu * b[t] + x[4 + t];
        x[t] = in.nesterov ? x[t] + in.mu * a[t] : a[t];
        x[4 + t] = in.nesterov ? x[4 + t] + in.mu * b[t] : b[t];
      }
      p[0] = a;
      p[1] = b;
    }
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      s += double(x[t]) * double(x[t]);
      m = fmaxf(m, fabsf(x[t]));
    }
  }
  if (first < (count & 7)) {  // what is left of a matrix past its last eight
    const int64_t i = (count & ~int64_t(7)) + first;
    float x = grad_at(in.grad, in.f32, base + i);
    if (in.mom) {
      const float v = in.mu * in.mom[base + i] + x;
      in.mom[base + i] = v;
      x = in.nesterov ? x + in.mu * v : v;
    }
    s += double(x) * double(x);
    m = fmaxf(m, fabsf(x));
  }
  for (int o = 32; o > 0; o >>= 1) {
    s += __shfl_xor(s, o);
    m = fmaxf(m, __shfl_xor(m, o));
  }
  if ((threadIdx.x & 63) == 0) {
    sm[threadIdx.x >> 6] = s;
    mx[threadIdx.x >> 6] = m;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0.0;
    for (int i = 0; i < kNormThreads / 64; ++i) {
      s += sm[i];
      m = fmaxf(m, mx[i]);
    }
    part[int64_t(blockIdx.y) * gridDim.x + blockIdx.x] = NormPart{s, m, 0.f};
  }
}

// The remainders are kept in the order in which the update's lanes hold 64 x 64
// elements: [64 columns][64 rows][2 x 2 sub-tiles][lane][16 bytes], so they are
// read and written 16 bytes a lane. r0, c0: multiples of 64.
__device__ __forceinline__ int64_t lo_offset(int rows, int r0, int c0, int sub, int lane) {
  return (((int64_t(c0 / 64) * (rows / 64) + r0 / 64) * 4 + sub) * 64 + lane) * 16;
}

// Four remainders in E4M3, times 16 (the conversions scale as they go): at most
// 256, of an element near 65504, and off by 2^-4 of themselves, or by 2^-14 where
// they are below 2^-10. Unscaled, the large elements' remainders would be as
// good, and those below 2^-9 lost: 3.0e-3 instead of 1.8e-3 on a matrix of rank one.
constexpr float kLoStep = 0.0625f;
__device__ __forceinline__ uint32_t pack_lo(const float (&r)[4]) {
  typedef short v2i16 __attribute__((ext_vector_type(2)));
  v2i16 v = {0, 0};
  v = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(v, r[0], r[1], kLoStep, false);
  v = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(v, r[2], r[3], kLoStep, true);
  return __builtin_bit_cast(uint32_t, v);
}

// X0 and its remainder, 64 x 64 elements a workgroup, through LDS (transposed
// when G is tall). HBM-bound (the same stack: 136 us for 805 MB, some of what it
// reads still in the last-level cache from ortho_norm).
__global__ __launch_bounds__(256) void ortho_load_kernel(OrthoIn in, OrthoDims d, const NormPart* __restrict__ part,
                                                         float eps, _Float16* __restrict__ X,
                                                         uint8_t* __restrict__ Xl, float* __restrict__ scale) {
  __shared__ float tile[kLoadTile][kLoadTile + 1];
  const int e = blockIdx.z, r0 = blockIdx.y * kLoadTile, c0 = blockIdx.x * kLoadTile;
  int p;
  float s;
  matrix_scale(part + int64_t(e) * d.parts, d.parts, eps, &p, &s);
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) scale[e] = s;
  // a, b: row and column of G inside the tile
  const int g0 = d.tall ? c0 : r0, h0 = d.tall ? r0 : c0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int a = 32 * i + int(threadIdx.x >> 3), b = int(threadIdx.x & 7) * 8;
    float x[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) x[t] = 0.f;
    const int left = g0 + a < d.R ? d.C - (h0 + b) : 0;
    if (left > 0) {
      input_row(in, (int64_t(e) * d.R + g0 + a) * d.C + h0 + b, left, x);
#pragma unroll
      for (int t = 0; t < 8; ++t) x[t] = s == s ? ldexpf(x[t], p) : NAN;
    }
#pragma unroll
    for (int t = 0; t < 8; ++t) tile[d.tall ? b + t : a][d.tall ? a : b + t] = x[t];
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int blk = 4 * q + int(threadIdx.x >> 6), lane = lane_id();  // 2 x 4 blocks
    const int h = lane >> 5, r = (lane & 31) ^ (4 * h);
    const float* src = &tile[32 * (blk & 1) + r][16 * (blk >> 1) + 8 * h];
    u32x4 v;
#pragma unroll
    for (int t = 0; t < 4; ++t) v[t] = pack_f16(src[2 * t], src[2 * t + 1]);
    *reinterpret_cast<u32x4*>(X + int64_t(e) * d.mp * d.np +
                              block_at(d.mp, r0 / 32 + (blk & 1), c0 / 16 + (blk >> 1)) + 8 * lane) = v;
  }
  if (Xl) {
    // the 64 x 64 elements are half of a wave's part of an update tile: 2 x 2
    // sub-tiles of 64 lanes of 16 bytes
    const int lane = threadIdx.x & 63, sub = threadIdx.x >> 6;
    const int r = 32 * (sub >> 1) + (lane & 31);
    u32x4 v;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      float q[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float x = tile[r][32 * (sub & 1) + 8 * g + 4 * (lane >> 5) + t];
        q[t] = x - float(static_cast<_Float16>(x));
      }
      v[g] = pack_lo(q);
    }
    *reinterpret_cast<u32x4*>(Xl + int64_t(e) * d.mp * d.np + lo_offset(d.mp, r0, c0, sub, lane)) = v;
  }
}

// ------------------------------------------------------------------ products
//
// Every product is C = P Q^T (or P Q), v_mfma_f32_32x32x16_f16 with fp32
// accumulators, in tiles of one of two shapes:
//   Big    256 x 256, 8 waves of 128 x 64 in a 2 x 4 grid (two a SIMD), one
//          workgroup a CU. What bounds its loop is moving the slabs into LDS
//          (20 TB/s from L2 over the chip with no products at all), so the
//          tile is as large as the registers allow: 256 x 128 tiles, two
//          workgroups a CU, move half as much again per product, and their
//          epilogues did not run under the other workgroup's products.
//   Small  128 x 128, 4 waves of 64 x 64, two workgroups a CU, for stacks with
//          too few big tiles to go round.
// The k-slabs of 32 go straight into LDS (buffer_load ... lds), four stages:
// while a slab is multiplied, the next two are on their way and the loads of a
// third are issued.
//   * k-major slab (P, and Q of the symmetric products): for each 16 k the
//     blocks of the tile's rows, fragments with one ds_read_b128.
//   * mn-major slab (Q of the update): blocks of 32 k-rows x 16 columns, read
//     with the LDS transpose read ds_read_b64_tr_b16 (four consecutive k of
//     one entity a lane).
// The MFMA's A operand is the Q fragment, so a lane holds one row m and four
// runs of four consecutive columns n of each 32 x 32 sub-tile.
// The stages are separate LDS objects, named at compile time, so that the
// compiler can tell a slab's reads from the loads in flight.

constexpr int kBK = 32;

// TI: 32-row sub-tiles of a wave (2 sub-tiles wide); WN: waves side by side.
template <int TI_, int WN_>
struct TileShape {
  static constexpr int TI = TI_, WN = WN_;
  static constexpr int kWaves = 2 * WN;
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int kRows = 64 * TI, kCols = 64 * WN;
  static constexpr int kSlabP = kRows * kBK;             // halves of the P part of a stage
  static constexpr int kStage = (kRows + kCols) * kBK;   // halves of a stage
  // each operand's slab is 2 kWaves blocks: two loads a wave
  static_assert(2 * TI == kWaves && 2 * WN == kWaves, "a wave per row block of either operand");

  static __device__ __forceinline__ int wave_m();
  static __device__ __forceinline__ int wave_n();
  template <int S>
  static __device__ __forceinline__ _Float16* stage() {
    __shared__ __attribute__((aligned(1024))) _Float16 buf[kStage];
    return buf;
  }
  // a wave's 8 KiB for an image of its results, and for a second one, in the stages
  // once they are free
  static __device__ __forceinline__ uint16_t* image();
  static __device__ __forceinline__ uint16_t* image2();
};
using Big = TileShape<4, 4>;
using Small = TileShape<2, 2>;

template <int TI_, int WN_>
__device__ __forceinline__ int TileShape<TI_, WN_>::wave_m() { return wave_id() / WN; }
template <int TI_, int WN_>
__device__ __forceinline__ int TileShape<TI_, WN_>::wave_n() { return wave_id() % WN; }
template <int TI_, int WN_>
__device__ __forceinline__ uint16_t* TileShape<TI_, WN_>::image() {
  constexpr int kPerStage = kStage / 4096;
  static_assert(kPerStage * 2 == kWaves, "two stages hold the images");
  const int w = wave_id();
  return reinterpret_cast<uint16_t*>(w < kPerStage ? stage<0>() : stage<1>()) + (w % kPerStage) * 4096;
}
template <int TI_, int WN_>
__device__ __forceinline__ uint16_t* TileShape<TI_, WN_>::image2() {
  constexpr int kPerStage = kStage / 4096;
  const int w = wave_id();
  return reinterpret_cast<uint16_t*>(w < kPerStage ? stage<2>() : stage<3>()) + (w % kPerStage) * 4096;
}

template <class T>
struct Acc {
  f32x16 c[T::TI][2];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < T::TI; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) c[i][j][r] = 0.f;
  }
};

// One operand of a product: load i (0, 1) of wave w moves block kWaves i + w of
// a slab. What lies past the matrix's rows or columns goes to waves without results.
struct Operand {
  __amdgpu_buffer_rsrc_t rsrc;
  uint32_t blk;    // byte offset of block w of slab 0
  uint32_t next;   // bytes from block w to block kWaves + w
  uint32_t slab;   // bytes from one slab to the next
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const _Float16* base, int64_t halves) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<_Float16*>(base), 0, int(uint32_t(halves * 2)), 0x00020000);
}

// Rows from e0 on, k along the columns: block j is row block j % kWaves of
// column block j / kWaves.
__device__ __forceinline__ Operand operand_k(const _Float16* base, int rows, int cols, int e0) {
  Operand o;
  o.rsrc = rsrc_of(base, int64_t(rows) * cols);
  o.blk = uint32_t(block_at(rows, e0 / 32 + wave_id(), 0)) * 2u;
  o.next = uint32_t(rows / 32) * kBlock * 2u;
  o.slab = uint32_t(rows / 32) * 2u * kBlock * 2u;
  return o;
}
// Columns from e0 on, k along the rows: block j is column block j.
template <class T>
__device__ __forceinline__ Operand operand_mn(const _Float16* base, int rows, int cols, int e0) {
  Operand o;
  o.rsrc = rsrc_of(base, int64_t(rows) * cols);
  o.blk = uint32_t(block_at(rows, 0, e0 / 16 + wave_id())) * 2u;
  o.next = uint32_t(rows / 32) * T::kWaves * kBlock * 2u;
  o.slab = kBlock * 2;
  return o;
}

template <class T>
__device__ __forceinline__ void load_slab(const Operand& o, int kt, _Float16* lds) {
  const int w = wave_id();
  const uint32_t off = uint32_t(lane_id()) * 16u;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        o.rsrc, (__attribute__((address_space(3))) void*)(lds + (T::kWaves * i + w) * kBlock), 16, off,
        int(o.blk + kt * o.slab + i * o.next), 0, 0);
}
// Slab kt of both operands; past the last one, the last one again.
template <class T>
__device__ __forceinline__ void load_stage(const Operand& P, const Operand& Q, int kt, int nk, _Float16* lds) {
  kt = kt < nk ? kt : nk - 1;
  load_slab<T>(P, kt, lds);
  load_slab<T>(Q, kt, lds + T::kSlabP);
}

// 32 entities x 16 k of a k-major slab, from entity ent0 and k = 16 kk on.
template <class T>
__device__ __forceinline__ f16x8 frag_k(const _Float16* lds, int ent0, int kk) {
  return *reinterpret_cast<const f16x8*>(lds + (kk * T::kWaves + (ent0 >> 5)) * kBlock +
                                         in_block(lane_id() & 31, lane_id() >> 5));
}
// The same of an mn-major slab: in each 16-lane group the transpose read gives
// lane p element p % 4 of the 8-byte pieces that lanes 4 j + p / 4 address. The
// lane offset passes through an empty asm operand, or the compiler loses
// which LDS object the read touches and waits for every load in flight.
__device__ __forceinline__ f16x8 frag_mn(const _Float16* lds, int ent0, int kk) {
  const int g = lane_id() >> 4, p = lane_id() & 15;
  const int k = 8 * (g >> 1) + (p >> 2);
  const int at = (g & 1) * kBlock + 4 * (p & 1);  // 16 columns on, 4 columns on
  int lo = at + in_block(k, (p & 3) >> 1), hi = at + in_block(k + 4, (p & 3) >> 1);
  asm("" : "+v"(lo), "+v"(hi));
  const _Float16* a = lds + (ent0 >> 4) * kBlock + kk * 16 * 8;
  const v4i16 l = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(a + lo));
  const v4i16 h = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(a + hi));
  return __builtin_bit_cast(f16x8, v8i16(__builtin_shufflevector(l, h, 0, 1, 2, 3, 4, 5, 6, 7)));
}

template <class T, bool Q_MN>
__device__ __forceinline__ void mma_slab(const _Float16* lds, Acc<T>& acc) {
  __builtin_amdgcn_iglp_opt(0);
  const int pm = T::wave_m() * 32 * T::TI, qn = T::wave_n() * 64;
#pragma unroll
  for (int kk = 0; kk < kBK / 16; ++kk) {
    f16x8 pf[T::TI], qf[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if constexpr (Q_MN) qf[j] = frag_mn(lds + T::kSlabP, qn + 32 * j, kk);
      else qf[j] = frag_k<T>(lds + T::kSlabP, qn + 32 * j, kk);
    }
#pragma unroll
    for (int i = 0; i < T::TI; ++i) pf[i] = frag_k<T>(lds, pm + 32 * i, kk);
#pragma unroll
    for (int i = 0; i < T::TI; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        acc.c[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(qf[j], pf[i], acc.c[i][j], 0, 0, 0);
  }
}

// s_waitcnt immediates: vmcnt(n), lgkmcnt(0) (a wave's LDS reads are done
// before it lets the others overwrite the stage).
constexpr int wait_imm(int vm) { return 0x0070 | (vm & 15) | ((vm >> 4) << 14); }

// Slab kt out of stage S, while slabs kt + 1 and kt + 2 are on their way and the
// loads of slab kt + 3 go to the stage that slab kt - 1 has left. ACTIVE
// false: the wave only moves data.
template <class T, int S, bool Q_MN, bool ACTIVE>
__device__ __forceinline__ void slab_step(const Operand& P, const Operand& Q, int kt, int nk, Acc<T>& acc) {
  __builtin_amdgcn_s_waitcnt(wait_imm(8));  // four loads a slab
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  load_stage<T>(P, Q, kt + 3, nk, T::template stage<(S + 3) % 4>());
  if constexpr (ACTIVE) mma_slab<T, Q_MN>(T::template stage<S>(), acc);
}

// The loads of the first three slabs.
template <class T>
__device__ __forceinline__ void first_slabs(const Operand& P, const Operand& Q, int nk) {
  load_stage<T>(P, Q, 0, nk, T::template stage<0>());
  load_stage<T>(P, Q, 1, nk, T::template stage<1>());
  load_stage<T>(P, Q, 2, nk, T::template stage<2>());
}

// The k loop, four slabs a turn (nk is a multiple of four: matrices are padded
// to 128): one body and no branch in it (more exits, or work on the
// accumulators under a condition, made the compiler copy them), so that it
// also counts the loads and waits for a slab's own only.
template <class T, bool Q_MN, bool ACTIVE>
__device__ __forceinline__ void turns(const Operand& P, const Operand& Q, int from, int to, int nk, Acc<T>& acc) {
  for (int kt = from; kt < to; kt += 4) {
    slab_step<T, 0, Q_MN, ACTIVE>(P, Q, kt, nk, acc);
    slab_step<T, 1, Q_MN, ACTIVE>(P, Q, kt + 1, nk, acc);
    slab_step<T, 2, Q_MN, ACTIVE>(P, Q, kt + 2, nk, acc);
    slab_step<T, 3, Q_MN, ACTIVE>(P, Q, kt + 3, nk, acc);
  }
}
__device__ __forceinline__ void slabs_end() {
  __builtin_amdgcn_s_waitcnt(wait_imm(0));
  __syncthreads();  // the stages are free for the epilogue's images
}
template <class T, bool Q_MN, bool ACTIVE>
__device__ __forceinline__ void slabs(const Operand& P, const Operand& Q, int nk, Acc<T>& acc) {
  turns<T, Q_MN, ACTIVE>(P, Q, 0, nk, nk, acc);
  slabs_end();
}

// The image's 64 x 64 values transposed into a matrix of blocks: image column n
// is row col0 + n, image row r column row0 + r. Lane n takes column n, 8 image
// rows (a chunk) at a time.
__device__ __forceinline__ void put_blocks_mirrored(const uint16_t* im, _Float16* __restrict__ out, int rows, int row0,
                                                    int col0) {
  const int n = lane_id();
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const u32x4 v = image_col(im, 8 * q, 16 * (n >> 4));
    *reinterpret_cast<u32x4*>(out + block_at(rows, col0 / 32 + (n >> 5), row0 / 16 + (q >> 1)) +
                              in_block(n & 31, q & 1)) = v;
  }
}
// ------------------------------------------------------------------ tiles
//
// Workgroups of one launch are dealt to the eight XCDs in turn (blockIdx % 8);
// each XCD takes a contiguous range of (matrix, tile), so that the tiles of a
// matrix share its operands in that XCD's L2.

__device__ __forceinline__ bool take_tile(int64_t total, int tiles, int64_t* e, int* t) {
  const int64_t per = (total + 7) / 8;
  const int64_t id = int64_t(blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if ((blockIdx.x >> 3) >= per || id >= total) return false;
  *e = id / tiles;
  *t = int(id % tiles);
  return true;
}
unsigned grid_of(int64_t total) { return unsigned((total + 7) / 8 * 8); }

// The tiles of a symmetric product: those on and below the diagonal; of a
// tile, the 128 x 128 blocks on and below it.
int sym_tiles(int mp, int rows) {
  const int h = (mp + rows - 1) / rows;
  return h * (h + 1) / 2;
}
__device__ __forceinline__ void sym_tile(int t, int* bi, int* bj) {
  int b = int((sqrtf(8.f * float(t) + 1.f) - 1.f) * 0.5f);
  while (b * (b + 1) / 2 > t) --b;
  while ((b + 1) * (b + 2) / 2 <= t) ++b;
  *bi = b;
  *bj = t - b * (b + 1) / 2;
}

// A wave's part of tile (bi, bj).
template <class T>
struct WavePart {
  int row0, col0;
  __device__ __forceinline__ WavePart(int bi, int bj)
      : row0(bi * T::kRows + T::wave_m() * 32 * T::TI), col0(bj * T::kCols + T::wave_n() * 64) {}
};

// The blocks of a symmetric result, fp16, times f, and their mirror images.
// diag (or NULL): what the rounding of the diagonal lost.
template <class T>
__device__ __forceinline__ void store_symmetric(const Acc<T>& acc, float f, _Float16* __restrict__ out, int rows,
                                                WavePart<T> at, float* __restrict__ diag) {
  uint16_t* im = T::image();
  const bool mirror = at.row0 / 128 != at.col0 / 128;
  const int lane = lane_id();
#pragma unroll
  for (int h = 0; h < T::TI / 2; ++h) {
#pragma unroll
    for (int ii = 0; ii < 2; ++ii) {
      const int i = 2 * h + ii;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const f32x16& c = acc.c[i][j];
        u32x2 w[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          w[g] = u32x2{pack_f16(c[4 * g] * f, c[4 * g + 1] * f), pack_f16(c[4 * g + 2] * f, c[4 * g + 3] * f)};
          if (mirror) image_put(im, 32 * ii + (lane & 31), 8 * j + 2 * g + (lane >> 5), w[g][0], w[g][1]);
        }
        put_subtile(w, out, rows, at.row0 + 32 * i, at.col0 + 32 * j);
        if (diag && at.row0 + 32 * i == at.col0 + 32 * j) {
          // register q of the lane is row lane % 32, column 8 (q / 4) + 4 (lane / 32) + q % 4
          const int n = lane & 31;
#pragma unroll
          for (int q = 0; q < 16; ++q)
            if (n == 8 * (q >> 2) + 4 * (lane >> 5) + (q & 3)) {
              const float x = c[q] * f;
              diag[at.row0 + 32 * i + n] = x - float(static_cast<_Float16>(x));
            }
        }
      }
    }
    if (mirror) {
      image_sync();
      put_blocks_mirrored(im, out, rows, at.row0 + 64 * h, at.col0);
      image_sync();
    }
  }
}

// A = X X^T times the square of the iterate's scale. MFMA-bound: 128 of 768 x 2048
// in 180 us, 1.15 PFLOP/s of the six tiles of nine that it computes (a square
// library product of 8192 reaches 1.21).
template <class T>
__global__ __launch_bounds__(T::kThreads, 2) void ortho_gram_kernel(const _Float16* __restrict__ X, OrthoDims d,
                                                                    int tiles, const float* __restrict__ scale,
                                                                    _Float16* __restrict__ A) {
  int64_t e;
  int t, bi, bj;
  if (!take_tile(d.E * tiles, tiles, &e, &t)) return;
  sym_tile(t, &bi, &bj);
  const _Float16* Xe = X + e * d.mp * d.np;
  const WavePart<T> at(bi, bj);
  const Operand P = operand_k(Xe, d.mp, d.np, bi * T::kRows), Q = operand_k(Xe, d.mp, d.np, bj * T::kCols);
  const int nk = d.np / kBK;
  Acc<T> acc;
  first_slabs<T>(P, Q, nk);
  if (at.row0 >= d.mp || at.col0 / 128 > at.row0 / 128) {
    slabs<T, false, false>(P, Q, nk, acc);
    return;
  }
  acc.zero();
  slabs<T, false, true>(P, Q, nk, acc);
  const float s = scale ? scale[e] : 1.f / kXScale;
  store_symmetric<T>(acc, s * s, A + e * d.mp * d.mp, d.mp, at, nullptr);
}

// The same of few tiles over a long axis: each part of the k loop is a workgroup of
// its own, [matrix][tile][part][wave][2 x 2 sub-tiles][4][lane][4] in fp32.
__global__ __launch_bounds__(Small::kThreads, 2) void ortho_gram_part_kernel(const _Float16* __restrict__ X, OrthoDims d,
                                                                             int tiles, int parts, int part_slabs,
                                                                             float* __restrict__ sums) {
  using T = Small;
  int64_t e;
  int t, bi, bj;
  if (!take_tile(d.E * tiles * parts, tiles * parts, &e, &t)) return;
  const int part = t / tiles;  // the tiles of a part follow each other: they share its columns
  t %= tiles;
  sym_tile(t, &bi, &bj);
  const _Float16* Xe = X + e * d.mp * d.np;
  Operand P = operand_k(Xe, d.mp, d.np, bi * T::kRows), Q = operand_k(Xe, d.mp, d.np, bj * T::kCols);
  P.blk += uint32_t(part * part_slabs) * P.slab;
  Q.blk += uint32_t(part * part_slabs) * Q.slab;
  const int nk = min(part_slabs, d.np / kBK - part * part_slabs);
  Acc<T> acc;
  first_slabs<T>(P, Q, nk);
  acc.zero();
  slabs<T, false, true>(P, Q, nk, acc);
  float* out = sums + (((e * tiles + t) * parts + part) * T::kWaves + wave_id()) * 4096;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<f32x4*>(out + (((2 * i + j) * 4 + g) * 64 + lane_id()) * 4) =
            f32x4{acc.c[i][j][4 * g], acc.c[i][j][4 * g + 1], acc.c[i][j][4 * g + 2], acc.c[i][j][4 * g + 3]};
}

// Adds the parts, in their order: a wave for each 32 x 32 sub-tile.
constexpr int kJoinWaves = 4;
__global__ __launch_bounds__(64 * kJoinWaves) void ortho_gram_join_kernel(const float* __restrict__ sums, OrthoDims d,
                                                                          int tiles, int parts,
                                                                          const float* __restrict__ scale,
                                                                          _Float16* __restrict__ A) {
  using T = Small;
  constexpr int kRow = 40;  // halves: 16-byte chunks of the mirror image's rows
  __shared__ __attribute__((aligned(16))) _Float16 mirror[kJoinWaves][32 * kRow];
  const int64_t id = int64_t(blockIdx.x) * kJoinWaves + wave_id();
  const int sub = int(id & 15), lane = lane_id();
  const int64_t tile = id >> 4, e = tile / tiles;  // 16 sub-tiles a tile: the grid is exact
  int bi, bj;
  sym_tile(int(tile % tiles), &bi, &bj);
  const int wave = sub >> 2, i = (sub >> 1) & 1, j = sub & 1;
  const float* src = sums + (tile * parts * T::kWaves + wave) * 4096 + (sub & 3) * 1024 + lane * 4;
  f32x4 c[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) c[g] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int p = 0; p < parts; ++p)
#pragma unroll
    for (int g = 0; g < 4; ++g) c[g] += *reinterpret_cast<const f32x4*>(src + int64_t(p) * T::kWaves * 4096 + g * 256);
  const float s = scale ? scale[e] : 1.f / kXScale;
  const float f = s * s;
  const int row0 = bi * T::kRows + (wave / T::WN) * 64 + 32 * i, col0 = bj * T::kCols + (wave % T::WN) * 64 + 32 * j;
  _Float16* out = A + e * d.mp * d.mp;
  _Float16* im = mirror[wave_id()];
  u32x2 w[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    w[g] = u32x2{pack_f16(c[g][0] * f, c[g][1] * f), pack_f16(c[g][2] * f, c[g][3] * f)};
    // row lane % 32, columns 8 g + 4 (lane / 32) + 0 .. 3
#pragma unroll
    for (int q = 0; q < 4; ++q)
      im[(8 * g + 4 * (lane >> 5) + q) * kRow + (lane & 31)] =
          __builtin_bit_cast(_Float16, uint16_t(w[g][q >> 1] >> (16 * (q & 1))));
  }
  put_subtile(w, out, d.mp, row0, col0);
  if (bi == bj) return;
  image_sync();
  // the mirrored sub-tile: rows col0 + n, 16-byte chunks of eight columns
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int n = lane & 31, chunk = 2 * q + (lane >> 5);
    *reinterpret_cast<u32x4*>(out + block_at(d.mp, col0 / 32, row0 / 16 + (chunk >> 1)) + in_block(n, chunk & 1)) =
        *reinterpret_cast<const u32x4*>(im + n * kRow + 8 * chunk);
  }
}

// A product of m x m matrices that are polynomials of X X^T, so symmetric and
// commuting: out = f (P Q^T + (r1 + d1) M1 + r2 M2) in fp16, d1 a diagonal (or
// NULL), M2 NULL if there is none; on the diagonal also re (e1 + e2) (or NULL).
// The accumulators start from the terms besides the product. 128 of 768 x 768 in
// 111 us: 0.70 PFLOP/s of the six tiles of nine, 300 to 450 MB to and from HBM,
// and an epilogue (the mirrored store) for every 24 slabs.
struct SymProduct {
  const _Float16 *P, *Q, *M1, *M2;
  float r1, r2, f, re;
  const float *d1, *e1, *e2;
  bool product;    // false: without P Q^T
  _Float16* out;
  float* diag;     // what the rounding of out's diagonal lost (or NULL)
};

template <class T>
__global__ __launch_bounds__(T::kThreads, 2) void ortho_product_kernel(SymProduct a, OrthoDims d, int tiles) {
  int64_t e;
  int t, bi, bj;
  if (!take_tile(d.E * tiles, tiles, &e, &t)) return;
  sym_tile(t, &bi, &bj);
  const int64_t mo = e * d.mp * d.mp, vo = e * d.mp;
  const WavePart<T> at(bi, bj);
  const Operand P = operand_k(a.P + mo, d.mp, d.mp, bi * T::kRows), Q = operand_k(a.Q + mo, d.mp, d.mp, bj * T::kCols);
  const int nk = a.product ? d.mp / kBK : 0;
  Acc<T> acc;
  if (a.product) first_slabs<T>(P, Q, nk);
  if (at.row0 >= d.mp || at.col0 / 128 > at.row0 / 128) {
    slabs<T, false, false>(P, Q, nk, acc);
    return;
  }
  const int lane = lane_id();
#pragma unroll
  for (int i = 0; i < T::TI; ++i) {
    const int row = at.row0 + 32 * i + (lane & 31);
    const float r1 = a.r1 + (a.d1 ? a.d1[vo + row] : 0.f);
    const float on = a.e1 ? a.re * (a.e1[vo + row] + a.e2[vo + row]) : 0.f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      u32x2 w[4];
      get_subtile(a.M1 + mo, d.mp, at.row0 + 32 * i, at.col0 + 32 * j, w);
#pragma unroll
      for (int q = 0; q < 16; ++q) acc.c[i][j][q] = r1 * half_of(w[q >> 2][(q >> 1) & 1], q & 1);
      if (a.M2) {
        get_subtile(a.M2 + mo, d.mp, at.row0 + 32 * i, at.col0 + 32 * j, w);
#pragma unroll
        for (int q = 0; q < 16; ++q)
          acc.c[i][j][q] = fmaf(a.r2, half_of(w[q >> 2][(q >> 1) & 1], q & 1), acc.c[i][j][q]);
      }
      if (a.e1 && at.row0 + 32 * i == at.col0 + 32 * j) {
#pragma unroll
        for (int q = 0; q < 16; ++q)
          if ((lane & 31) == 8 * (q >> 2) + 4 * (lane >> 5) + (q & 3)) acc.c[i][j][q] += on;
      }
    }
  }
  slabs<T, false, true>(P, Q, nk, acc);
  store_symmetric<T>(acc, a.f, a.out + mo, d.mp, at, a.diag ? a.diag + vo : nullptr);
}

// The slab whose k are the rows of sub-tile row i holds, as Q, the sub-tiles of X
// itself: acc += lin X.
template <class T>
__device__ __forceinline__ void add_linear(const _Float16* lds, int i, float lin, Acc<T>& acc) {
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const f16x4 v =
          *reinterpret_cast<const f16x4*>(lds + T::kSlabP + (T::wave_n() * 4 + 2 * j + (g >> 1)) * kBlock +
                                         in_block(lane_id() & 31, g & 1) + 4 * (lane_id() >> 5));
#pragma unroll
      for (int t = 0; t < 4; ++t) acc.c[i][j][4 * g + t] = fmaf(float(v[t]), lin, acc.c[i][j][4 * g + t]);
    }
}
// The turn of the tile's own rows (a big tile's wave has a turn of its own; the
// two waves of a small tile share one).
template <class T, int S>
__device__ __forceinline__ void own_step(const Operand& P, const Operand& Q, int own, int nk, const float (&lin)[T::TI],
                                         Acc<T>& acc) {
  slab_step<T, S, true, true>(P, Q, own + S, nk, acc);
  if (T::TI == 4 || T::wave_m() == S / 2) add_linear<T>(T::template stage<S>(), S % T::TI, lin[S % T::TI], acc);
}

// X' = (a + diag) X + B X. In the turn whose k are the tile's rows, X's fp16
// part is taken for the linear term as it passes (read again from memory, it
// took the update 13 % longer). FIRST: X is X0, whose value is scale[e] times
// what is stored (and whose remainder may be zero: Xl NULL). LAST: the result
// is written instead of X'. U leaves as bf16; the step of the weights goes
// through LDS as pairs of bf16, to 2^-17 of each element at any magnitude (fp16's
// range ends where |G| is small against eps, or the polynomial is steep; 256 of
// 768 x 2048 in 8.25 ms, with fp16 8.19). 128 of 768 x 2048 in 403 us: 0.77 PFLOP/s
// and 1.2 GB, 3.0 TB/s. The MFMAs alone would take 255, the bytes 246; a tile's first
// loads and last stores do not run under its products (the wait counter holds loads
// and stores in one order, so a next tile's loads would wait for the stores too).
template <class T, bool FIRST, bool LAST>
__global__ __launch_bounds__(T::kThreads, 2) void ortho_update_kernel(const _Float16* __restrict__ X,
                                                                      const uint8_t* __restrict__ Xl,
                                                                      const _Float16* __restrict__ B,
                                                                      const float* __restrict__ diag, OrthoDims d,
                                                                      int tiles, float ca,
                                                                      const float* __restrict__ scale, OrthoOut out) {
  int64_t e;
  int t;
  if (!take_tile(d.E * tiles, tiles, &e, &t)) return;
  const int nrow = (d.mp + T::kRows - 1) / T::kRows;
  const int bi = t % nrow, bj = t / nrow;  // the row tiles of a column panel follow each other
  const WavePart<T> at(bi, bj);
  const bool active = at.row0 < d.mp && at.col0 < d.np;
  const int64_t xo = e * d.mp * d.np;
  const int lane = lane_id();
  const Operand P = operand_k(B + e * d.mp * d.mp, d.mp, d.mp, bi * T::kRows);
  const Operand Q = operand_mn<T>(X + xo, d.mp, d.np, bj * T::kCols);
  const int nk = d.mp / kBK;
  float lin[T::TI];
#pragma unroll
  for (int i = 0; i < T::TI; ++i) lin[i] = active ? ca + diag[e * d.mp + at.row0 + 32 * i + (lane & 31)] : 0.f;
  u32x4 lo[2 * T::TI];
#pragma unroll
  for (int q = 0; q < 2 * T::TI; ++q) {
    lo[q] = u32x4{0u, 0u, 0u, 0u};
    if (active && (!FIRST || Xl))
      lo[q] = *reinterpret_cast<const u32x4*>(Xl + xo + lo_offset(d.mp, at.row0 + 64 * (q >> 2), at.col0, q & 3, lane));
  }
  Acc<T> acc;
  first_slabs<T>(P, Q, nk);
  if (!active) {
    slabs<T, true, false>(P, Q, nk, acc);
    return;
  }
  acc.zero();
  const int own = (T::TI == 4 ? at.row0 : bi * T::kRows) / kBK;
  turns<T, true, true>(P, Q, 0, own, nk, acc);
  own_step<T, 0>(P, Q, own, nk, lin, acc);
  own_step<T, 1>(P, Q, own, nk, lin, acc);
  own_step<T, 2>(P, Q, own, nk, lin, acc);
  own_step<T, 3>(P, Q, own, nk, lin, acc);
  turns<T, true, true>(P, Q, own + 4, nk, nk, acc);
  slabs_end();
  const float s = FIRST ? scale[e] : 1.f / kXScale;  // takes a stored iterate to its value
#pragma unroll
  for (int h = 0; h < T::TI / 2; ++h) {
#pragma unroll
    for (int ii = 0; ii < 2; ++ii) {
      const int i = 2 * h + ii;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        u32x4 nlo;
        u32x2 w[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(lo[2 * i + j][g], kLoStep, false);
          const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(lo[2 * i + j][g], kLoStep, true);
          float y[4] = {a[0], a[1], b[0], b[1]};
#pragma unroll
          for (int q = 0; q < 4; ++q) y[q] = fmaf(y[q], lin[i], acc.c[i][j][4 * g + q]);
          if constexpr (!LAST) {
            if constexpr (FIRST) {
#pragma unroll
              for (int q = 0; q < 4; ++q) y[q] *= s * kXScale;
            }
            w[g] = u32x2{pack_f16(y[0], y[1]), pack_f16(y[2], y[3])};
#pragma unroll
            for (int q = 0; q < 4; ++q) y[q] -= half_of(w[g][q >> 1], q & 1);
            nlo[g] = pack_lo(y);
          } else if (out.U) {
            w[g] = u32x2{pack_bf16x2(y[0] * s, y[1] * s), pack_bf16x2(y[2] * s, y[3] * s)};
          } else {
            const u32x2 a = pair_bf16x2(y[0] * s, y[1] * s), b = pair_bf16x2(y[2] * s, y[3] * s);
            w[g] = u32x2{a[0], b[0]};
            image_put(T::image2(), 32 * ii + (lane & 31), 8 * j + 2 * g + (lane >> 5), a[1], b[1]);
          }
        }
        if constexpr (!LAST) {
          put_subtile(w, out.X + xo, d.mp, at.row0 + 32 * i, at.col0 + 32 * j);
          *reinterpret_cast<u32x4*>(out.Xl + xo + lo_offset(d.mp, at.row0 + 64 * h, at.col0, 2 * ii + j, lane)) = nlo;
        } else {
#pragma unroll
          for (int g = 0; g < 4; ++g)
            image_put(T::image(), 32 * ii + (lane & 31), 8 * j + 2 * g + (lane >> 5), w[g][0], w[g][1]);
        }
      }
    }
    if constexpr (LAST) {
      image_sync();
      put_image(out, T::image(), T::image2(), d, e, at.row0 + 64 * h, at.col0);
      image_sync();
    }
  }
}

// ------------------------------------------------------------------ plan

// Big tiles of a product from which they are used: two rounds of the 256 CUs.
// Gram / square / update in us, big against small tiles: 128 matrices 768 x 2048
// (6, 6 and 24 big tiles each) 180 : 215, 111 : 116, 403 : 458; 16 of 1536 x 2048
// (21, 21, 48) 105 : 108, 91 : 81, 179 : 197; 6 of 777 x 1000 (10, 10, 16)
// 26 : 15, 28 : 15, 29 : 21. Eight stages instead of four for small
// tiles of one workgroup a CU changed nothing: the turns of a lone workgroup are
// as long as its LDS reads and MFMAs one after the other.
constexpr int64_t kBigTiles = 512;

struct OrthoPlan {
  OrthoDims d;
  int64_t group;                            // matrices at a time
  size_t part, scale, X[2], Xl[2], M[3], diag, sums, total;  // workspace offsets
  int gram_parts, gram_part_slabs;          // of the k loop of X X^T
  size_t small;                             // of the small matrices' path
};

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

constexpr int64_t kSmallGroup = 1024;

// Elements of a matrix from which its norm is 256 partial sums instead of 64: one of
// 1024 x 4096 in 7.5 us instead of 16.4; for 128 of 768 x 2048 ortho_norm would gain 5
// us of 87 and ortho_load, which adds them, lose as much.
constexpr int64_t kManyElements = 1 << 21;

// Parts of the k loop of X X^T: enough for two workgroups a CU, of 512 columns at
// least, where the tiles leave most CUs without work. In us a call, whole and in
// parts: 1 of 256 x 16384 533 : 176, 3 of 300 x 4000 238 : 170, 1 of 1024 x 4096 (36
// tiles) 302 : 248, 10 of 256 x 2048 (30) 174 : 153, 20 of 200 x 1500 (60) 181 : 176;
// 2 of 1024 x 2048 (72) 241 : 245, 30 of 256 x 2048 (90) 234 : 263; 512 x 1024 152 : 150.
// (A matrix of a stack whose products are split may differ in its last bits
// from itself in a larger stack.)
constexpr int64_t kSplitTiles = 64;
constexpr int kSplitSlabs = 16, kSplitFrom = 48;
void gram_split(const OrthoArgs& a, OrthoPlan* p) {
  const int nk = p->d.np / kBK;
  const int64_t tiles = a.E * sym_tiles(p->d.mp, Small::kRows);
  p->gram_parts = 1;
  p->gram_part_slabs = nk;
  if (a.E > p->group || a.E < 1 || tiles > kSplitTiles || nk < kSplitFrom) return;
  const int most = int(512 / tiles) < nk / kSplitSlabs ? int(512 / tiles) : nk / kSplitSlabs;
  p->gram_part_slabs = ((nk + most - 1) / most + 3) / 4 * 4;  // turns of four slabs
  p->gram_parts = (nk + p->gram_part_slabs - 1) / p->gram_part_slabs;
}

OrthoPlan ortho_plan(const OrthoArgs& a) {
  OrthoPlan p{};
  OrthoDims& d = p.d;
  d.R = a.R;
  d.C = a.C;
  d.tall = a.R > a.C;
  d.m = d.tall ? a.C : a.R;
  d.n = d.tall ? a.R : a.C;
  d.mp = (d.m + 127) / 128 * 128;
  d.np = (d.n + 127) / 128 * 128;
  d.parts = int64_t(d.R) * d.C >= kManyElements ? 256 : 64;
  if (small_fits(a)) {
    p.group = a.E < 1 ? 1 : a.E > kSmallGroup ? kSmallGroup : a.E;
    p.part = 0;
    p.small = up256(size_t(p.group) * d.parts * sizeof(NormPart));
    p.total = p.small + small_plan(a, p.group).total;
    return p;
  }
  const int64_t x = int64_t(d.mp) * d.np, q = int64_t(d.mp) * d.mp;
  // At most about 4 GiB of state (256 matrices 1536 x 4096: 1 GiB 44.6 ms, 2 GiB
  // 42.9, 4 GiB 40.3, 8 GiB 40.0, 16 GiB 39.7: the last round of tiles of each
  // launch). As many matrices as fit, the rest last; groups of equal size 41.0.
  const int64_t bytes = 6 * x + 6 * q;
  int64_t g = (int64_t(4) << 30) / bytes;
  g = g < 1 ? 1 : (g > 4096 ? 4096 : g);
  p.group = a.E < g ? (a.E > 0 ? a.E : 1) : g;
  size_t o = 0;
  // A big tile's operands reach up to 128 rows or columns past a matrix: row blocks
  // past mp are those of the next column block, and past the last block lies what
  // follows in the workspace (each m x m matrix is followed by X, each X by its
  // remainders) or, where the buffer resource ends, zeros. None of it reaches a
  // result: the waves whose rows and columns those are only move data.
  p.part = o;  o = up256(o + size_t(p.group) * d.parts * sizeof(NormPart));
  p.scale = o; o = up256(o + size_t(p.group) * 4);
  p.diag = o;  o = up256(o + size_t(p.group) * d.mp * 4 * 3);
  for (int i = 0; i < 3; ++i) {
    p.M[i] = o; o = up256(o + size_t(p.group) * q * 2);
  }
  for (int i = 0; i < 2; ++i) {
    p.X[i] = o;  o = up256(o + size_t(p.group) * x * 2);
    p.Xl[i] = o; o = up256(o + size_t(p.group) * x);
  }
  gram_split(a, &p);
  p.sums = o;
  if (p.gram_parts > 1) o = up256(o + size_t(p.group) * sym_tiles(d.mp, Small::kRows) * p.gram_parts * Small::kRows * Small::kCols * 4);
  p.total = o;
  return p;
}

// Whether the first two steps run as one update: it saves a pass over X (X X^T and
// the update, 1.5 m^2 n multiply-adds) for three more m x m products (1.5 m^3).
// Measured, apart and as one: n / m = 2.67 (128 of 768 x 2048) 3.70 and 3.47 ms, n / m
// = 2.67 (256 of 1536 x 4096) 44.3 and 40.4 ms, n / m = 1.33 1.99 and 1.99
// ms, n / m = 1.29 283 and 303 us. fp16's range limits a^2.
bool ortho_pairs(const OrthoArgs& a, const OrthoDims& d) {
  return a.steps >= 2 && std::fabs(a.a) <= 16.f && 2 * int64_t(d.n) >= 3 * int64_t(d.m);
}

// The caller's result from element `first` on.
OrthoOut target_of(const OrthoTarget& t, int64_t first) {
  OrthoOut out{};
  out.U = t.U ? t.U + first : nullptr;
  out.W = t.W ? t.W + first : nullptr;
  out.master = t.master ? t.master + first : nullptr;
  out.keep = t.keep;
  out.step = t.step;
  return out;
}

// The steps of one group.
struct OrthoSteps {
  const OrthoArgs& a;
  const OrthoTarget& t;
  const OrthoPlan& p;
  OrthoDims d;
  char* base;
  int64_t count, e0;
  bool lo0;
  hipStream_t st;
  KernelTimer* timer;

  void go() const {
    if (d.E * sym_tiles(d.mp, Big::kRows) >= kBigTiles) steps<Big>(); else steps<Small>();
  }

 private:
  template <class U>
  U* at(size_t o) const {
    return reinterpret_cast<U*>(base + o);
  }
  _Float16* M(int i) const { return at<_Float16>(p.M[i]); }
  float* diag(int i) const { return at<float>(p.diag) + int64_t(i) * p.group * d.mp; }
  template <class T>
  int64_t update_tiles() const {
    return int64_t((d.mp + T::kRows - 1) / T::kRows) * ((d.np + T::kCols - 1) / T::kCols);
  }

  // T: tile shape of the symmetric products
  template <class T>
  void steps() const {
    int done = 0, updates = 0;
    if (ortho_pairs(a, d)) {
      // the first two steps as one update: with P = a + B, B = b A + c A A,
      // A2 = P A P is the second step's X X^T and X2 = P2 P X = (a^2 + D) X
      gram<T>(0, M(0));
      square<T>(M(0), M(1), diag(0));
      product<T>("ortho_square", SymProduct{M(1), M(0), M(0), nullptr, a.a, 0.f, 1.f, 0.f, diag(0), nullptr, nullptr, true,
                                            M(2), nullptr});   // P A
      product<T>("ortho_square", SymProduct{M(1), M(2), M(2), nullptr, a.a, 0.f, 1.f, 0.f, diag(0), nullptr, nullptr, true,
                                            M(0), nullptr});   // A2
      square<T>(M(0), M(2), diag(1));
      product<T>("ortho_square", SymProduct{M(2), M(1), M(1), M(2), a.a, a.a, 1.f, a.a, nullptr, diag(0), diag(1), true,
                                            M(0), diag(2)});   // D
      done = 2;
      update(updates++, M(0), a.a * a.a, diag(2), done == a.steps);
    }
    for (; done < a.steps; ++updates) {
      gram<T>(updates, M(0));
      square<T>(M(0), M(1), diag(0));
      ++done;
      update(updates, M(1), a.a, diag(0), done == a.steps);
    }
  }

  template <class T>
  void gram(int updates, _Float16* out) const {
    const int tiles = sym_tiles(d.mp, T::kRows);
    if constexpr (T::kRows == Small::kRows) {
      if (p.gram_parts > 1) {
        {
          TimedLaunch tl(timer, "ortho_gram_part", st);
          hipLaunchKernelGGL(ortho_gram_part_kernel, dim3(grid_of(d.E * tiles * p.gram_parts)), dim3(T::kThreads), 0, st,
                             at<_Float16>(p.X[updates & 1]), d, tiles, p.gram_parts, p.gram_part_slabs, at<float>(p.sums));
        }
        TimedLaunch tl(timer, "ortho_gram_join", st);
        hipLaunchKernelGGL(ortho_gram_join_kernel, dim3(unsigned(d.E * tiles * 16 / kJoinWaves)), dim3(64 * kJoinWaves), 0,
                           st, at<float>(p.sums), d, tiles, p.gram_parts, updates == 0 ? at<float>(p.scale) : nullptr, out);
        return;
      }
    }
    TimedLaunch tl(timer, "ortho_gram", st);
    hipLaunchKernelGGL(ortho_gram_kernel<T>, dim3(grid_of(d.E * tiles)), dim3(T::kThreads), 0, st,
                       at<_Float16>(p.X[updates & 1]), d, tiles, updates == 0 ? at<float>(p.scale) : nullptr, out);
  }
  template <class T>
  void product(const char* name, const SymProduct& q) const {
    const int tiles = sym_tiles(d.mp, T::kRows);
    TimedLaunch tl(timer, name, st);
    hipLaunchKernelGGL(ortho_product_kernel<T>, dim3(grid_of(d.E * tiles)), dim3(T::kThreads), 0, st, q, d, tiles);
  }
  // B = b A + c A A as c (A A + b / c A); a c below 2^-20 of b adds nothing that fp16 holds
  template <class T>
  void square(const _Float16* A, _Float16* B, float* dg) const {
    const bool whole = std::fabs(a.c) > 1e-6f * std::fabs(a.b);
    product<T>("ortho_square", SymProduct{A, A, A, nullptr, whole ? a.b / a.c : a.b, 0.f, whole ? a.c : 1.f, 0.f, nullptr,
                                          nullptr, nullptr, whole, B, dg});
  }

  // X <- (lin + dg) X + B X
  void update(int updates, const _Float16* B, float lin, const float* dg, bool last) const {
    if (d.E * update_tiles<Big>() >= kBigTiles) update_in<Big>(updates, B, lin, dg, last);
    else update_in<Small>(updates, B, lin, dg, last);
  }
  template <class T>
  void update_in(int updates, const _Float16* B, float lin, const float* dg, bool last) const {
    const int tiles = int(update_tiles<T>()), cur = updates & 1;
    const bool first = updates == 0;
    const uint8_t* xl = !first || lo0 ? at<uint8_t>(p.Xl[cur]) : nullptr;
    OrthoOut out{};
    if (!last) {
      out.X = at<_Float16>(p.X[1 - cur]);
      out.Xl = at<uint8_t>(p.Xl[1 - cur]);
    } else {
      out = target_of(t, e0 * count);
    }
    TimedLaunch tl(timer, last ? "ortho_update_last" : "ortho_update", st);
    const auto kernel = first ? (last ? ortho_update_kernel<T, true, true> : ortho_update_kernel<T, true, false>)
                              : (last ? ortho_update_kernel<T, false, true> : ortho_update_kernel<T, false, false>);
    hipLaunchKernelGGL(kernel, dim3(grid_of(d.E * tiles)), dim3(T::kThreads), 0, st, at<_Float16>(p.X[cur]), xl, B, dg,
                       d, tiles, lin, first ? at<float>(p.scale) : nullptr, out);
  }
};

}  // namespace

// What any stack of up to a.E such matrices needs: the parts' sums of a smaller one
// may be more than a larger one, without parts, has besides.
size_t ortho_workspace_bytes(const OrthoArgs& a) {
  const OrthoPlan p = ortho_plan(a);
  size_t most = p.total;
  if (small_fits(a) || p.d.np / kBK < kSplitFrom) return most;
  OrthoArgs fewer = a;
  for (fewer.E = 1; fewer.E < a.E && fewer.E * sym_tiles(p.d.mp, Small::kRows) <= kSplitTiles; ++fewer.E) {
    const size_t n = ortho_plan(fewer).total;
    if (n > most) most = n;
  }
  return most;
}

hipError_t launch_ortho(const OrthoArgs& a, const OrthoTarget& t, void* ws, hipStream_t st, KernelTimer* timer) {
  if (a.E <= 0) return hipSuccess;
  const OrthoPlan p = ortho_plan(a);
  char* base = static_cast<char*>(ws);
  auto f16 = [&](size_t o) { return reinterpret_cast<_Float16*>(base + o); };
  auto u8 = [&](size_t o) { return reinterpret_cast<uint8_t*>(base + o); };
  auto f32 = [&](size_t o) { return reinterpret_cast<float*>(base + o); };
  NormPart* part = reinterpret_cast<NormPart*>(base + p.part);
  const int64_t count = int64_t(a.R) * a.C;
  const size_t gsize = a.grad_f32 ? 4 : 2;
  for (int64_t e0 = 0; e0 < a.E; e0 += p.group) {
    OrthoDims d = p.d;
    d.E = a.E - e0 < p.group ? a.E - e0 : p.group;
    const unsigned ge = unsigned(d.E);
    const OrthoIn in{static_cast<const char*>(t.grad) + size_t(e0) * count * gsize, a.grad_f32,
                     t.momentum ? t.momentum + e0 * count : nullptr, t.mu, t.nesterov};
    {
      TimedLaunch tl(timer, "ortho_norm", st);
      hipLaunchKernelGGL(ortho_norm_kernel, dim3(unsigned(d.parts), ge), dim3(kNormThreads), 0, st, in, count, part);
    }
    if (small_fits(a)) {
      const hipError_t e = launch_small(a, in, d, part, target_of(t, e0 * count), base + p.small, st, timer);
      if (e != hipSuccess) return e;
      continue;
    }
    const bool lo0 = a.grad_f32 || in.mom;  // a bf16 G is exact in fp16
    {
      TimedLaunch tl(timer, "ortho_load", st);
      hipLaunchKernelGGL(ortho_load_kernel, dim3(d.np / kLoadTile, d.mp / kLoadTile, ge), dim3(256), 0, st, in, d, part,
                         a.eps, f16(p.X[0]), lo0 ? u8(p.Xl[0]) : nullptr, f32(p.scale));
    }
    OrthoSteps{a, t, p, d, base, count, e0, lo0, st, timer}.go();
  }
  return hipGetLastError();
}

}  // namespace moe
