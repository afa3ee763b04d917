// Dense products with bias, activation and residual, and their gradients
// (include/moe.h: moe_linear, moe_linear_bwd): the router's logits and a shared
// expert beside the routed ones (the pages' layer is the routed experts alone).
//
// Every product is C[m][n] = sum_k P[m][k] Q[n][k]:
//   forward  P = X, Q = W                    both with k along their rows (k-major)
//   dX       P = dP, Q = W^T                 W has one memory row per k (mn-major)
//   dW       P = dP^T, Q = X^T               both mn-major, k the token
// Tiles of BM x BN, slabs of 64 k staged in LDS by loads that go there directly
// (buffer_load ... lds), sent for as many slabs ahead as there are stages: 256 x 256 by
// eight waves with two stages (128 KiB, one workgroup a CU), 128 x 128 by four with two, 64 x
// 128 by four with four. Waves take 32 x 32 sub-tiles with v_mfma_f32_32x32x16_bf16, Q's
// fragment as the A operand, so that a lane holds one row m and runs of four columns n.
//   k-major operand in LDS: rows of 64 k, 16-byte chunk c of row r at slot c ^ (r / 2) % 8:
//     fragment reads (16 rows, one chunk) then touch 16 different bank groups.
//   mn-major operand: k-rows of the tile's entities, chunk c of k-row k at slot
//     c ^ 4 (k % 4) (64 entities: c ^ 4 ((k / 2) % 2)); a fragment comes from two
//     transpose reads (ds_read_b64_tr_b16), whose 16 (row, chunk) pairs lie in
//     different bank groups.
// Measured: 16384 x 4096 x 1536 186 us (1.11 PFLOP/s; a library product of that size takes
// 153 to 164), with a residual 193, with operands and results that come from HBM and not from the
// last-level cache 215 to 230. A slab of a 256 x 256 tile takes 1.5 us, the MFMAs alone would
// 0.86 (they are busy 46 % of the cycles): the fragments' reads and the slabs' arrival
// take the LDS as long as the products take the MFMAs, and the next slab is all that fits
// beside the one at work. Lines fetched into L2 a slab earlier made it slower (206 us), as
// did tiles whose results wait for memory one after the other. Waves of 128 x 128, which
// would read a third less from LDS, need all 512 registers, and the compiler spilled.
// Rows and columns past the matrix are read from a valid row or as zeros and not
// stored; k past the end is zero in both operands. Rows that are no multiple of 16 bytes
// are first copied to rows that are.
#include <algorithm>

#include "device_common.h"
#include "kernels.h"

namespace moe {
namespace lin {

constexpr int BK = 64;
constexpr uint32_t kPast = 0x80000000u;  // an offset beyond any extent: reads as zero

typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef short v8i16 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) v4i16 lds_v4i16;
typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, int(uint32_t(bytes)), 0x00020000);
}

// 16 bytes a lane from the resource's offset off + at (zeros past its end) into 1 KiB of LDS
__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t r, uint16_t* lds, uint32_t off, int at) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)(lds), 16, off, at, 0, 0);
}
__device__ __forceinline__ void load_lds(const void* base, int64_t bytes, uint16_t* lds, uint32_t off) {
  load_lds(rsrc(base, bytes), lds, off, 0);
}

// ------------------------------------------------------------------ what a result goes through

// P's columns c .. c+7 of row r on their way out. For SwiGLU u holds the up part.
struct Out {
  const float* bias;
  const void* residual;
  void* Y;
  uint16_t* pre;
  int64_t M;
  int N;      // columns of Y
  int act;    // kAct*
  bool f32;   // type of Y and residual
};

__device__ __forceinline__ float sigmoid(float x) { return sigmoidf_fast(x); }
// sigmoid(2 sqrt(2 / pi) (x + 0.044715 x^3)): GELU's factor in its tanh form
__device__ __forceinline__ float gelu_gate(float x) { return sigmoid(1.5957691216057308f * (x + 0.044715f * x * x * x)); }

__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8], int cols) {
  if (cols >= 8) {
    *reinterpret_cast<u32x4u*>(p) =
        u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < cols) p[i] = uint16_t(pack_bf16x2(v[i], 0.f));
  }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8], int cols) {
  if (cols >= 8) {
    f32x4u* q = reinterpret_cast<f32x4u*>(p);
    q[0] = f32x4{v[0], v[1], v[2], v[3]};
    q[1] = f32x4{v[4], v[5], v[6], v[7]};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < cols) p[i] = v[i];
  }
}
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8], int cols) {
  if (cols >= 8) {
    const u32x4 a = *reinterpret_cast<const u32x4u*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(a[i]);
      v[2 * i + 1] = bf16_hi(a[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < cols ? __uint_as_float(uint32_t(p[i]) << 16) : 0.f;
  }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8], int cols) {
  if (cols >= 8) {
    const f32x4u* q = reinterpret_cast<const f32x4u*>(p);
    const f32x4 a = q[0], b = q[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < cols ? p[i] : 0.f;
  }
}

__device__ __forceinline__ void activate8(int act, float (&v)[8]) {
  if (act == kActRelu) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] > 0.f || v[i] != v[i] ? v[i] : 0.f;
  } else if (act == kActSilu) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= sigmoid(v[i]);
  } else if (act == kActGelu) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= gelu_gate(v[i]);
  }
}

template <bool PAIR>
__device__ __forceinline__ void finish8(const Out& o, int64_t r, int c, float (&v)[8], float (&u)[8]) {
  const int cols = o.N - c;
  float b[8];
  if (o.bias) {
    load8(o.bias + c, b, cols);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += b[i];
  }
  if constexpr (PAIR) {
    if (o.bias) {
      load8(o.bias + o.N + c, b, cols);
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] += b[i];
    }
    if (o.pre) {
      store8(o.pre + r * (2 * int64_t(o.N)) + c, v, cols);
      store8(o.pre + r * (2 * int64_t(o.N)) + o.N + c, u, cols);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * sigmoid(v[i]) * u[i];
  } else {
    if (o.pre) store8(o.pre + r * int64_t(o.N) + c, v, cols);
    activate8(o.act, v);
  }
  const int64_t at = r * int64_t(o.N) + c;
  if (o.residual) {
    if (o.f32) load8(static_cast<const float*>(o.residual) + at, b, cols);
    else load8(static_cast<const uint16_t*>(o.residual) + at, b, cols);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += b[i];
  }
  if (o.f32) store8(static_cast<float*>(o.Y) + at, v, cols);
  else store8(static_cast<uint16_t*>(o.Y) + at, v, cols);
}

// ------------------------------------------------------------------ operands

struct Operand {
  const uint16_t* data;
  int64_t ld;    // elements from row to row, a multiple of 8
  int64_t ents;  // entities (rows m of P, n of Q)
  bool pair;     // SwiGLU's W: entities are read as 32 gate rows, 32 up rows, ...
};

// Matrix row (k-major) of tile entity q of a paired operand with ents = 2 N rows:
// 32 gate rows and their 32 up rows take turns.
__device__ __forceinline__ int64_t paired_row(int64_t q0, int q, int64_t N) {
  const int64_t o = (q0 >> 1) + (q >> 6) * 32 + (q & 31);
  return (q >> 5 & 1) * N + (o < N ? o : N - 1);
}

// k-major: thread t's load i fills LDS slot t + THREADS i (row = slot / 8).
template <int ROWS, int THREADS>
struct KMajor {
  static constexpr int kPer = ROWS * 8 / THREADS;
  __amdgpu_buffer_rsrc_t data;
  uint32_t off[kPer];
  int chunk;  // of every row this thread loads
  int K;      // a multiple of 8
  __device__ __forceinline__ void init(const Operand& op, int64_t e0, int64_t, int Kp) {
    const int r0 = threadIdx.x >> 3;
    chunk = int(threadIdx.x & 7) ^ (r0 >> 1 & 7);
    K = Kp;
    const int64_t left = op.ents - e0;
    const int64_t first = op.pair ? 0 : e0;
    data = rsrc(op.data + first * op.ld, op.pair ? op.ents * op.ld * 2 : (left < ROWS ? left : ROWS) * op.ld * 2);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int q = r0 + THREADS / 8 * i;
      const int64_t row = op.pair ? paired_row(e0, q, op.ents >> 1) : (q < left ? q : left - 1);
      off[i] = uint32_t(row * op.ld * 2) + 16u * chunk;
    }
  }
  // slab kt into `lds`, zeros if there is none (kt is 0 then). Past the end of a row a lane's own
  // offset is past every extent; the slab's is within every row.
  __device__ __forceinline__ void load(int kt, bool some, uint16_t* lds) const {
    const int w = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const uint32_t past = some && kt * BK + 8 * chunk < K ? 0u : kPast;
#pragma unroll
    for (int i = 0; i < kPer; ++i) load_lds(data, lds + (64 * w + THREADS * i) * 8, off[i] | past, kt * 2 * BK);
  }
};

// mn-major: slab kt is memory rows 64 kt ..; its buffer resource ends with the last k.
template <int COLS, int THREADS>
struct MNMajor {
  static constexpr int kPer = COLS * 8 / THREADS;
  static constexpr int kRow = COLS / 8;  // chunks of a k-row
  const uint16_t* base;
  int64_t ld, kend, e0;
  uint32_t off[kPer];
  __device__ __forceinline__ void init(const Operand& op, int64_t e, int64_t kred, int) {
    base = op.data;
    ld = op.ld;
    kend = kred;
    e0 = e;
    const int64_t left = op.ents - e;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int q = int(threadIdx.x) + THREADS * i;
      const int k = q / kRow, c = (q % kRow) ^ (COLS >= 128 ? 4 * (k & 3) : 4 * (k >> 1 & 1));
      off[i] = uint32_t((k * ld + 8 * c) * 2) | (8 * c < left ? 0u : kPast);
    }
  }
  __device__ __forceinline__ void load(int kt, bool some, uint16_t* lds) const {
    const int w = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int64_t k0 = some ? int64_t(kt) * BK : 0;
    const int64_t rows = kend - k0 < BK ? kend - k0 : BK;
    const int64_t bytes = some ? (rows * ld - e0) * 2 : 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      load_lds(base + k0 * ld + e0, bytes, lds + (64 * w + THREADS * i) * 8, off[i]);
  }
};

template <bool MN, int ENTS, int THREADS>
struct LoaderOf { using type = KMajor<ENTS, THREADS>; };
template <int ENTS, int THREADS>
struct LoaderOf<true, ENTS, THREADS> { using type = MNMajor<ENTS, THREADS>; };

// slot of chunk c of k-row k of an mn-major slab `ents` wide
__device__ __forceinline__ int mn_swz(int ents, int k) { return ents >= 128 ? 4 * (k & 3) : 4 * (k >> 1 & 1); }

// 32 entities x 16 k: lane holds entity lane % 32, k = 16 kk + 8 (lane / 32) + 0..7.
__device__ __forceinline__ bf16x8 frag_k(const uint16_t* lds, int ent0, int kk) {
  const int lane = lane_id();
  const int e = ent0 + (lane & 31), c = 2 * kk + (lane >> 5);
  return *reinterpret_cast<const bf16x8*>(lds + e * BK + ((c ^ (e >> 1 & 7)) << 3));
}
// The same of an mn-major slab. In each 16-lane group lane p addresses k-row k0 + p / 4
// at entities n0 + 4 (p % 4) and receives four consecutive k of entity n0 + p; rows k and
// k + 4 have the same swizzle.
__device__ __forceinline__ bf16x8 frag_mn(const uint16_t* lds, int ents, int ent0, int kk) {
  const int lane = lane_id();
  const int g = lane >> 4, p = lane & 15;
  const int n = ent0 + 16 * (g & 1) + 4 * (p & 3);
  const int k0 = 8 * (g >> 1) + (p >> 2);
  int off = k0 * ents + (((n >> 3) ^ mn_swz(ents, k0)) << 3) + (n & 7);
  asm("" : "+v"(off));  // one offset for all of a sub-tile's reads
  const uint16_t* a = lds + off + kk * 16 * ents;
  const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(a));
  const v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(a + 4 * ents));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}
template <bool MN, int ENTS>
__device__ __forceinline__ bf16x8 frag(const uint16_t* lds, int ent0, int kk) {
  if constexpr (MN) return frag_mn(lds, ENTS, ent0, kk);
  return frag_k(lds, ent0, kk);
}

// ------------------------------------------------------------------ the tile kernel

struct Problem {
  Operand P, Q;
  int64_t kred;     // k that exist
  int Kp;           // kred rounded up to 8 (k-major operands)
  int mt, nt;       // tiles
  int splits;       // parts of the k axis; more than one: sums go to `partial`
  int slabs;        // slabs of a part
  float* partial;   // fp32 [splits][M][ldp]
  int64_t ldp;
  Out out;
};

// A barrier that waits for nothing by itself (__syncthreads waits for every load into
// LDS); memory accesses stay on their side of it.
__device__ __forceinline__ void meet_all() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The operand of s_waitcnt for lgkmcnt(0) and vmcnt(n)
constexpr int wait_code(int n) { return (n & 15) | (n >> 4) << 14 | 0x0070; }

// The b-th tile: the eight XCDs (b % 8) take contiguous ranges of tiles, and a range
// walks groups of eight row tiles column by column, so that tiles that run at once in
// an XCD share rows of both operands in its L2.
__device__ __forceinline__ void tile_of(const Problem& p, uint32_t b, uint32_t total, int* m, int* n, int* s) {
  const uint32_t q = total / 8, r = total % 8, x = b % 8;
  uint32_t t = x * q + (x < r ? x : r) + b / 8;
  const uint32_t per = uint32_t(p.mt) * uint32_t(p.nt);
  *s = int(t / per);
  t %= per;
  const uint32_t group = t / (8u * uint32_t(p.nt));
  const uint32_t rows = min(8u, uint32_t(p.mt) - 8u * group);
  t -= group * 8u * uint32_t(p.nt);
  *m = int(8u * group + t % rows);
  *n = int(t / rows);
}

// Four columns of each half of the wave become eight of each lane: a holds columns 0..3
// (lanes below 32) and 4..7, b columns 8..11 and 12..15; after it a lane below 32 has 0..7
// in (a, b), one above 8..15.
__device__ __forceinline__ void join_halves(float& a, float& b) {
  typedef uint32_t u2 __attribute__((ext_vector_type(2)));
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  a = __uint_as_float(r[0]);
  b = __uint_as_float(r[1]);
}

// What a tile's sums go through: as they are (with bias, residual), an activation, SwiGLU,
// or as a part of a split product into `partial`.
enum { kPlain, kActs, kPair, kSplit };

// The lane, as a value that the compiler does not know: what is computed from it is not
// kept in registers through the products (it spilled).
__device__ __forceinline__ int fresh_lane() {
  int x = lane_id();
  asm volatile("" : "+v"(x));
  return x;
}

// A wave's chunk of 16 bytes of the 32 staged rows.
__device__ __forceinline__ uint16_t* staged(uint16_t* buf, int chunks, int row, int c) {
  return buf + (row * chunks + (c ^ (row & (chunks - 1)))) * 8;
}

// Staged rows [32][CH chunks] of T out to a matrix of row length ld: `out` is the element
// of the first row and chunk, of which `rows` rows and `cols` columns exist. A row's chunks
// leave from neighbouring lanes.
template <class T, int CH>
__device__ __forceinline__ void copy_out(uint16_t* buf, T* out, int ld, int rows, int cols) {
  constexpr int EC = 16 / sizeof(T), RP = 64 / CH;
  const int lane = fresh_lane(), c = lane % CH;
  const int n = min(EC, cols - EC * c);
  if (n <= 0) return;
  int r = lane / CH, off = r * ld + EC * c;
#pragma unroll 1
  for (int q = 0; q < 32 / RP; q += 2, r += 2 * RP, off += 2 * RP * ld) {
    u32x4 v[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) v[w] = *reinterpret_cast<const u32x4*>(staged(buf, CH, r + w * RP, c));
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      T* dst = out + off + w * RP * ld;
      if (r + w * RP >= rows) {
      } else if (n == EC) {
        __builtin_nontemporal_store(v[w], reinterpret_cast<u32x4u*>(dst));
      } else {
#pragma unroll 1
        for (int i = 0; i < n; ++i) dst[i] = T(sizeof(T) == 2 ? v[w][i / 2] >> (16 * (i & 1)) : v[w][i & 3]);
      }
    }
  }
}
// The same inwards, in two halves, so that the loads can be on their way early; what is not
// there is zero.
template <class T, int CH>
__device__ __forceinline__ void copy_in_load(u32x4 (&v)[CH / 2], const T* in, int ld, int rows, int cols) {
  constexpr int EC = 16 / sizeof(T), RP = 64 / CH;
  const int lane = fresh_lane(), c = lane % CH, r0 = lane / CH;
  const int n = min(EC, cols - EC * c);
#pragma unroll
  for (int q = 0; q < CH / 2; ++q) {
    v[q] = u32x4{0u, 0u, 0u, 0u};
    if (n == EC && r0 + q * RP < rows) v[q] = *reinterpret_cast<const u32x4u*>(in + (r0 + q * RP) * ld + EC * c);
  }
}
template <class T, int CH>
__device__ __forceinline__ void copy_in_put(uint16_t* buf, const u32x4 (&v)[CH / 2], const T* in, int ld, int rows,
                                            int cols) {
  constexpr int EC = 16 / sizeof(T), RP = 64 / CH;
  const int lane = fresh_lane(), c = lane % CH, r0 = lane / CH;
  const int n = min(EC, cols - EC * c);
#pragma unroll
  for (int q = 0; q < CH / 2; ++q) *reinterpret_cast<u32x4*>(staged(buf, CH, r0 + q * RP, c)) = v[q];
  if (n > 0 && n < EC) {
#pragma unroll 1
    for (int r = r0; r < min(32, rows); r += RP)
#pragma unroll 1
      for (int i = 0; i < n; ++i) reinterpret_cast<T*>(staged(buf, CH, r, c))[i] = in[r * ld + EC * c + i];
  }
}

// A wave's WTM x WTN sums at (m0, n0) of the product on their way out, 32 rows at a time:
// bias, activation and residual in fp32 with eight columns of a row in a lane, then through
// the wave's LDS, so that memory sees whole lines. A sub-tile at a time, and offsets of 32
// bits from addresses that are the same in every lane: more of them at once would spill.
template <int WTM, int WTN, int MODE>
__device__ __forceinline__ void results(const Problem& p, f32x16 (&acc)[WTM / 32][WTN / 32], uint16_t* buf, int64_t m0,
                                        int64_t n0, int part) {
  constexpr int TM = WTM / 32, TN = WTN / 32;
  constexpr bool kIsPair = MODE == kPair;
  constexpr int kCols = kIsPair ? WTN / 2 : WTN;  // result columns of a wave
  constexpr int CH16 = kCols / 8;                 // chunks of a staged row of bf16
  constexpr int kHalves = kIsPair ? 1 : 2;        // fp32 rows are staged in this many parts
  constexpr int CH32 = kCols / kHalves / 4;
  constexpr int JS = kIsPair ? 2 : 1;             // sub-tiles that make 32 result columns
  const Out& o = p.out;
  const int64_t N = MODE == kSplit ? p.ldp : o.N;
  const int64_t c0 = kIsPair ? n0 / 2 : n0;  // first result column
  const int ld = int(N), cols = int(max(int64_t(0), min(int64_t(kCols), N - c0)));
  const bool f32 = MODE == kSplit || o.f32;
  u32x4 ahead[CH16 / 2];
  if (MODE != kSplit && !f32 && o.residual)
    copy_in_load<uint16_t, CH16>(ahead, static_cast<const uint16_t*>(o.residual) + m0 * N + c0, ld,
                                 int(max(int64_t(0), min(int64_t(32), p.P.ents - m0))), cols);
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int lane = fresh_lane(), row = lane & 31, up = lane >> 5;
    const int64_t r0 = m0 + 32 * i;
    const int rows = int(max(int64_t(0), min(int64_t(32), p.P.ents - r0)));
    const int64_t at = r0 * N + c0;
    __builtin_amdgcn_sched_barrier(0);
    auto take = [&](const f32x16& x, int h, float (&y)[8]) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        y[r] = x[8 * h + r];
        y[4 + r] = x[8 * h + 4 + r];
        join_halves(y[r], y[4 + r]);
      }
    };
    auto add = [&](float (&y)[8], int64_t c) {  // bias of eight columns from c of W's rows
      float x[8];
      load8(o.bias + c, x, int(min(int64_t(8), N - (c >= N && kIsPair ? c - N : c))));
#pragma unroll
      for (int q = 0; q < 8; ++q) y[q] += x[q];
    };
    auto put16 = [&](int n, const float (&y)[8]) {
      *reinterpret_cast<u32x4*>(staged(buf, CH16, row, 2 * n + up)) =
          u32x4{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7])};
    };
    // P itself first where it is kept: the gate part, then the up part of a pair
    if (MODE != kSplit && o.pre) {
#pragma unroll
      for (int q = 0; q < JS; ++q) {
#pragma unroll
        for (int n = 0; n < kCols / 16; ++n) {
          float v[8];
          take(acc[i][n / 2 * JS + q], n % 2, v);
          const int64_t c = c0 + 16 * n + 8 * up;
          if (o.bias && c < N) add(v, c + q * N);
          put16(n, v);
        }
        copy_out<uint16_t, CH16>(buf, o.pre + r0 * (JS * N) + q * N + c0, JS * ld, rows, cols);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    // chunk n of this lane: its value before the residual
    auto value = [&](int n, float (&v)[8]) {
      take(acc[i][n / 2 * JS], n % 2, v);
      if constexpr (MODE != kSplit) {
        const int64_t c = c0 + 16 * n + 8 * up;
        if (o.bias && c < N) add(v, c);
        if constexpr (kIsPair) {
          float u[8];
          take(acc[i][n / 2 * JS + 1], n % 2, u);
          if (o.bias && c < N) add(u, N + c);
#pragma unroll
          for (int q = 0; q < 8; ++q) v[q] = v[q] * sigmoid(v[q]) * u[q];
        }
        if constexpr (MODE == kActs) activate8(o.act, v);
      }
    };
    if (f32) {
      float* out = MODE == kSplit ? p.partial + int64_t(part) * p.P.ents * N : static_cast<float*>(o.Y);
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        constexpr int kPart = kCols / kHalves;
        const bool res = MODE != kSplit && o.residual;
        if (res) {
          const uint32_t* in = static_cast<const uint32_t*>(o.residual) + at + h * kPart;
          u32x4 x[CH32 / 2];
          copy_in_load<uint32_t, CH32>(x, in, ld, rows, cols - h * kPart);
          copy_in_put<uint32_t, CH32>(buf, x, in, ld, rows, cols - h * kPart);
        }
#pragma unroll
        for (int n = 0; n < kPart / 16; ++n) {
          float v[8];
          value(n + h * (kPart / 16), v);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            f32x4* s = reinterpret_cast<f32x4*>(staged(buf, CH32, row, 4 * n + 2 * up + q));
            f32x4 x = {v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
            if (res) x += *s;
            *s = x;
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        copy_out<uint32_t, CH32>(buf, reinterpret_cast<uint32_t*>(out) + at + h * kPart, ld, rows, cols - h * kPart);
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
      if (o.residual) {
        const uint16_t* in = static_cast<const uint16_t*>(o.residual) + at;
        copy_in_put<uint16_t, CH16>(buf, ahead, in, ld, rows, cols);
        __builtin_amdgcn_sched_barrier(0);
        // the next rows' part, while these are worked on
        if (i + 1 < TM)
          copy_in_load<uint16_t, CH16>(ahead, in + 32 * N, ld, int(max(int64_t(0), min(int64_t(32), p.P.ents - r0 - 32))),
                                       cols);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int n = 0; n < kCols / 16; ++n) {
        float v[8];
        value(n, v);
        if (o.residual) {
          const u32x4 x = *reinterpret_cast<const u32x4*>(staged(buf, CH16, row, 2 * n + up));
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            v[2 * q] += bf16_lo(x[q]);
            v[2 * q + 1] += bf16_hi(x[q]);
          }
        }
        put16(n, v);
        __builtin_amdgcn_sched_barrier(0);
      }
      copy_out<uint16_t, CH16>(buf, static_cast<uint16_t*>(o.Y) + at, ld, rows, cols);
    }
  }
}

// A persistent walk: workgroup b takes the tiles b, b + grid, ... The slabs of all of
// them are one stream, sent for NS slabs ahead, across the tiles' ends too: results leave
// through LDS of each wave's own, so the next tile's slabs are on their way meanwhile. The
// number of a tile's slabs is made a multiple of NS (the last may be zeros), so that a stage
// is known at compile time.
// NS: stages, that is how many slabs ahead are sent for. s0 .. s3: the stages' LDS; out: 32
// rows of each wave's results, WTN / 8 chunks of 16 bytes a row, chunk c at slot c ^ row.
template <int BM, int BN, int WM, int WN, int NS, bool P_MN, bool Q_MN, int MODE>
__device__ __forceinline__ void walk(const Problem& p, uint32_t first, uint32_t grid, uint16_t* s0, uint16_t* s1,
                                     uint16_t* s2, uint16_t* s3, uint16_t* out) {
  constexpr int kThreads = 64 * WM * WN;
  constexpr int WTM = BM / WM, WTN = BN / WN, TM = WTM / 32, TN = WTN / 32;
  static_assert(TN % 2 == 0, "a wave has gate and up columns of a pair");
  static_assert(NS == 2 || NS == 4, "stages");
  const int wave = threadIdx.x >> 6, wm = wave / WN, wn = wave % WN;
  const uint32_t total = uint32_t(p.mt) * uint32_t(p.nt) * uint32_t(p.splits);
  const int all = int((p.kred + BK - 1) / BK);
  typename LoaderOf<P_MN, BM, kThreads>::type lp;
  typename LoaderOf<Q_MN, BN, kThreads>::type lq;
  int mi, ni, si;
  auto open = [&](uint32_t t) {
    tile_of(p, t, total, &mi, &ni, &si);
    mi = __builtin_amdgcn_readfirstlane(mi);
    ni = __builtin_amdgcn_readfirstlane(ni);
    si = __builtin_amdgcn_readfirstlane(si);
    lp.init(p.P, int64_t(mi) * BM, p.kred, p.Kp);
    lq.init(p.Q, int64_t(ni) * BN, p.kred, p.Kp);
  };
  f32x16 acc[TM][TN];
  struct Frags {
    bf16x8 p[TM], q[TN];
  };
  auto read = [&](const uint16_t* s, int kk, Frags& f) {
#pragma unroll
    for (int j = 0; j < TN; ++j) f.q[j] = frag<Q_MN, BN>(s + BM * BK, wn * WTN + 32 * j, kk);
#pragma unroll
    for (int i = 0; i < TM; ++i) f.p[i] = frag<P_MN, BM>(s, wm * WTM + 32 * i, kk);
  };
  auto multiply = [&](const Frags& f) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = mfma_32x32x16(f.q[j], f.p[i], acc[i][j]);
  };
  // Which slab is sent for next: number f of the tile's nf (a multiple of NS), which end at fend. Past
  // the last tile's end slabs of zeros are sent for.
  uint32_t t = first;
  int f = 0, nf, f0, fend;
  bool more = true;
  auto begin = [&]() {
    f = 0;
    f0 = si * p.slabs;
    fend = min(f0 + p.slabs, all);
    nf = (fend - f0 + NS - 1) & ~(NS - 1);
  };
  auto advance = [&]() {
    if (more && f == nf) {
      t += grid;
      more = t < total;
      if (more) {
        open(t);
        begin();
      }
    }
  };
  auto send = [&](uint16_t* s) {
    const bool some = more && f0 + f < fend;
    const int kt = some ? f0 + f : 0;
    lp.load(kt, some, s);
    lq.load(kt, some, s + BM * BK);
    ++f;
  };
  // The slab whose first fragments are in `a` and the next's are read: every step's
  // products run while the next step's fragments come, in this order of issue: reads
  // (and sends) spread over the products. Left to itself the compiler puts them behind the
  // products, right before those that wait for them.
  Frags a, b;
  constexpr int kReads = (P_MN ? 2 : 1) * TM + (Q_MN ? 2 : 1) * TN, kMfmas = TM * TN;
  constexpr int kBurst = (kReads + kMfmas - 2) / (kMfmas - 1);
  constexpr int kSends = (BM + BN) * 8 / kThreads;
  constexpr int kSendBurst = (kSends + kMfmas - 1) / kMfmas;
  auto order = [&](bool sends) {
#pragma unroll
    for (int i = 0; i < kMfmas; ++i) {
      if (i * kBurst < kReads) __builtin_amdgcn_sched_group_barrier(0x100, kBurst, 0);
      if (sends && i * kSendBurst < kSends) __builtin_amdgcn_sched_group_barrier(0x10, kSendBurst, 0);
      __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto step = [&](const uint16_t* s, int kk, Frags& next, const Frags& now) {
    read(s, kk, next);
    multiply(now);
    order(false);
  };
  // the rest of a slab, then everybody has read it and the next one is there
  auto steps = [&](const uint16_t* s) {
    step(s, 1, b, a);
    step(s, 2, a, b);
    step(s, 3, b, a);
    // lgkmcnt(0), and all loads but those of the NS - 2 slabs after the next
    __builtin_amdgcn_s_waitcnt(wait_code((NS - 2) * kSends));
    meet_all();
    __builtin_amdgcn_sched_barrier(0);
  };
  // its last products, while another slab is sent for into its place
  auto turn = [&](uint16_t* done, const uint16_t* nxt) {
    advance();
    __builtin_amdgcn_sched_barrier(0);
    send(done);
    read(nxt, 0, a);
    multiply(b);
    order(true);
  };
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  };
  open(t);
  begin();
  int64_t m0 = int64_t(mi) * BM, n0 = int64_t(ni) * BN;  // of the tile that is multiplied
  int part = si, left = nf;
  send(s0);
  advance();
  send(s1);
  if constexpr (NS > 2) {
    advance();
    send(s2);
    advance();
    send(s3);
  }
  __builtin_amdgcn_s_waitcnt(wait_code((NS - 1) * kSends));
  meet_all();
  clear();
  read(s0, 0, a);
  steps(s0);
  // At the top a slab in s0 lacks its last products.
  while (true) {
    turn(s0, s1);
    steps(s1);
    if constexpr (NS > 2) {
      turn(s1, s2);
      steps(s2);
      turn(s2, s3);
      steps(s3);
      turn(s3, s0);
    } else {
      turn(s1, s0);
    }
    left -= NS;
    if (left == 0) {
      results<WTM, WTN, MODE>(p, acc, out + wave * 32 * WTN, m0 + wm * WTM, n0 + wn * WTN, part);
      // slabs of the next tile are there or under way, if there is one
      if (!more) break;
      m0 = int64_t(mi) * BM;
      n0 = int64_t(ni) * BN;
      part = si;
      left = nf;
      clear();
      read(s0, 0, a);  // again, so that it takes no registers in between
    }
    steps(s0);
  }
}

// An LDS object for each stage, so that the compiler can tell reads of one from loads in
// flight into another.
#define MOE_LINEAR_LDS                                                                  \
  constexpr int kStage = (BM + BN) * BK, kMore = NS > 2 ? kStage : 8;                   \
  __shared__ __attribute__((aligned(16))) uint16_t s0[kStage];                          \
  __shared__ __attribute__((aligned(16))) uint16_t s1[kStage];                          \
  __shared__ __attribute__((aligned(16))) uint16_t s2[kMore];                           \
  __shared__ __attribute__((aligned(16))) uint16_t s3[kMore];                           \
  __shared__ __attribute__((aligned(16))) uint16_t s_out[WM * 32 * BN];

template <int BM, int BN, int WM, int WN, int NS, bool P_MN, bool Q_MN, int MODE>
__global__ __launch_bounds__(64 * WM * WN, NS == 2 ? 2 : 1) void tile_kernel(const Problem p) {
  MOE_LINEAR_LDS
  walk<BM, BN, WM, WN, NS, P_MN, Q_MN, MODE>(p, blockIdx.x, gridDim.x, s0, s1, s2, s3, s_out);
}

// out[c] = sum over the blocks of sums[block][c], of 64 columns; no blocks: zeros
__device__ void bias_sums(const float* __restrict__ sums, int blocks, int cols, float* __restrict__ out, int block,
                          float (&red)[4][64]) {
  const int lane = lane_id(), w = threadIdx.x >> 6;
  const int c = block * 64 + lane;
  float s = 0.f;
  if (c < cols) {
    int b = w;
    for (; b + 28 < blocks; b += 32) {  // eight loads under way
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = sums[int64_t(b + 4 * i) * cols + c];
#pragma unroll
      for (int i = 0; i < 8; ++i) s += x[i];
    }
    for (; b < blocks; b += 4) s += sums[int64_t(b) * cols + c];
  }
  red[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < cols) out[c] = (red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane]);
}

// What both_kernel's last workgroups add up: dbias, or nothing.
struct BiasArgs {
  const float* sums;
  int blocks, cols;
  float* out;
};

// dX and dW at once where neither fills the CUs, and dbias: the first `nx` workgroups have
// dX's tiles, one each, the next `nw` dW's, the last dbias (1003 x 777 x 1001: 12 us for
// the products instead of 11 and 12, and dbias's 4 us within them).
template <int BM, int BN, int WM, int WN, int NS>
__global__ __launch_bounds__(64 * WM * WN, NS == 2 ? 2 : 1) void both_kernel(const Problem x, const Problem w, uint32_t nx,
                                                                             uint32_t nw, const BiasArgs bias) {
  MOE_LINEAR_LDS
  __shared__ float red[4][64];
  if (blockIdx.x < nx)
    walk<BM, BN, WM, WN, NS, false, true, kPlain>(x, blockIdx.x, nx, s0, s1, s2, s3, s_out);
  else if (blockIdx.x < nx + nw)
    walk<BM, BN, WM, WN, NS, true, true, kPlain>(w, blockIdx.x - nx, nw, s0, s1, s2, s3, s_out);
  else
    bias_sums(bias.sums, bias.blocks, bias.cols, bias.out, int(blockIdx.x - nx - nw), red);
}

// Few rows (M <= 32): W is read once, straight into the fragments of
// v_mfma_f32_16x16x32_bf16, and nothing waits for anything but its own loads. A workgroup
// has 16 rows of W (a pair's: 8 gate rows and their 8 up rows); its waves take turns at
// units of 64 k (a 128-byte line of each row), the sums meet in LDS. X comes from the
// caches. MT: fragments of 16 rows of X. One token, 1536 rows of 2048 (SwiGLU): 7.4 us,
// where a launch takes 2.7 and the 6.3 MB of W 1.3 at the memory's rate: its 96 workgroups
// leave 160 CUs without loads, and the rest is latency.
constexpr int kFewWaves = 8;
constexpr int kFewUnits = 4;  // of a wave in flight

// Eight k of a row, zeros past its end; rows begin anywhere.
__device__ __forceinline__ u32x4 row8(const uint16_t* p, int k, int K) {
  if (k + 8 <= K) return *reinterpret_cast<const u32x4u*>(p + k);
  u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (k + i < K) v[i / 2] |= uint32_t(p[k + i]) << (16 * (i & 1));
  return v;
}

template <int MT>
__global__ __launch_bounds__(64 * kFewWaves) void few_rows_kernel(const uint16_t* __restrict__ X,
                                                                  const uint16_t* __restrict__ W, int M, int K,
                                                                  bool pair, Out o) {
  __shared__ float sums[kFewWaves][16 * MT][17];
  const int lane = lane_id(), wave = threadIdx.x >> 6;
  const int e = lane & 15, kq = 8 * (lane >> 4);
  const int n0 = int(blockIdx.x) * (pair ? 8 : 16);
  const int n = pair ? n0 + (e & 7) : n0 + e;
  const uint16_t* w = W + (int64_t(n < o.N ? n : o.N - 1) + (pair && e >= 8 ? o.N : 0)) * K;
  const uint16_t* x[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) x[i] = X + int64_t(min(16 * i + e, M - 1)) * K;
  f32x4 acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int k0 = 64 * wave; k0 < K; k0 += 64 * kFewWaves * kFewUnits) {
    u32x4 wf[2 * kFewUnits], xf[2 * kFewUnits][MT];
#pragma unroll
    for (int q = 0; q < 2 * kFewUnits; ++q) {
      const int k = k0 + (q / 2) * 64 * kFewWaves + 32 * (q & 1) + kq;
      wf[q] = row8(w, k, K);
#pragma unroll
      for (int i = 0; i < MT; ++i) xf[q][i] = row8(x[i], k, K);
    }
#pragma unroll
    for (int q = 0; q < 2 * kFewUnits; ++q)
#pragma unroll
      for (int i = 0; i < MT; ++i)
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, wf[q]),
                                                         __builtin_bit_cast(bf16x8, xf[q][i]), acc[i], 0, 0, 0);
  }
  // lane: row 16 i + lane % 16 of X, rows 4 (lane / 16) + r of the 16 of W
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) sums[wave][16 * i + e][4 * (lane >> 4) + r] = acc[i][r];
  __syncthreads();
  const int chunks = pair ? 1 : 2;
  for (int q = threadIdx.x; q < M * chunks; q += 64 * kFewWaves) {
    const int m = q / chunks, c = 8 * (q % chunks);
    if (n0 + c >= o.N) continue;
    float v[8], u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = u[i] = 0.f;
    for (int g = 0; g < kFewWaves; ++g)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] += sums[g][m][c + i];
        if (pair) u[i] += sums[g][m][8 + i];
      }
    if (pair) finish8<true>(o, m, n0 + c, v, u);
    else finish8<false>(o, m, n0 + c, v, u);
  }
}

// The parts of a split product added in their order, and on through the epilogue. A
// paired product's columns stand in the order its tiles have them. Five parts of 1536 x 2048:
// 13 us (69 MB, mostly from the last-level cache).
__global__ __launch_bounds__(256) void join_kernel(const float* __restrict__ partial, int splits, int64_t ldp, bool pair,
                                                   Out o) {
  const int per = (o.N + 7) / 8;
  const int64_t total = o.M * per;
  for (int64_t q = int64_t(blockIdx.x) * 256 + threadIdx.x; q < total; q += int64_t(gridDim.x) * 256) {
    const int64_t m = q / per;
    const int c = int(q % per) * 8;
    const int col = pair ? (c >> 5) * 64 + (c & 31) : c;
    float v[8], u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = u[i] = 0.f;
    const float* src = partial + m * ldp + col;
    for (int s = 0; s < splits; ++s, src += o.M * ldp) {
      float a[8];
      load8(src, a, 8);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += a[i];
      if (pair) {
        load8(src + 32, a, 8);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] += a[i];
      }
    }
    if (pair) finish8<true>(o, m, c, v, u);
    else finish8<false>(o, m, c, v, u);
  }
}

// ------------------------------------------------------------------ passes around the products

// rows [R, C] -> [R, ld], the columns past C zero
struct PadJob {
  const uint16_t* in;
  uint16_t* out;
  int64_t R;
  int C;
  int64_t ld;
  int blocks;
};
__device__ void pad_rows(const PadJob& a, int block) {
  const int per = int(a.ld / 8);
  for (int64_t q = int64_t(block) * 256 + threadIdx.x; q < a.R * per; q += int64_t(a.blocks) * 256) {
    const int64_t r = q / per;
    const int c = int(q % per) * 8;
    const uint16_t* src = a.in + r * a.C + c;
    u32x4 v = {0u, 0u, 0u, 0u};
    if (c + 8 <= a.C) {
      v = *reinterpret_cast<const u32x4u*>(src);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < a.C) v[i / 2] |= uint32_t(src[i]) << (16 * (i & 1));
    }
    *reinterpret_cast<u32x4*>(a.out + r * a.ld + c) = v;
  }
}

struct DpArgs {
  const void* dY;
  const uint16_t* pre;
  int64_t M;
  int N;       // columns of dY
  int act;
  bool f32;    // type of dY
  uint16_t* dP;  // [M, ld], columns past N' zero, or NULL
  int64_t ld;
  float* sums;  // [blocks][cols] column sums of dP, or NULL
  int cols;     // N'
  int rows;     // rows of a block
  int blocks;   // along the rows; as many for every 256 columns of dY
};

// dP = dY act'(P), and its column sums. dP is held in bf16, also where dY is fp32: the
// matrix instructions take 16 bits, and the bits beyond would be a second product of the same size.
// It costs dX and dW 0.0023 of their norm against 0.0017 with dP in fp32 (their own rounding);
// the column sums are of dP before it. A workgroup takes `rows` rows of 8 x 32 = 256
// columns; thread t the columns 8 (t % 32) of rows t / 32, + 8, ...
__device__ void slope_rows(const DpArgs& a, int block, float (&red)[8][256]) {
  const int tr = threadIdx.x >> 5, tc = threadIdx.x & 31;
  const int by = block / a.blocks, bx = block % a.blocks;
  const int c = by * 256 + 8 * tc;
  const int64_t r0 = int64_t(bx) * a.rows;
  const bool pair = a.act == kActSwiglu;
  const int cols = a.N - c;
  float sv[8], su[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sv[i] = su[i] = 0.f;
  if (cols > 0) {
    for (int64_t r = r0 + tr; r < min(a.M, r0 + a.rows); r += 8) {
      float d[8], g[8], u[8], o[8], up[8];
      if (a.f32) load8(static_cast<const float*>(a.dY) + r * a.N + c, d, cols);
      else load8(static_cast<const uint16_t*>(a.dY) + r * a.N + c, d, cols);
      if (a.act != kActNone) load8(a.pre + r * a.cols + c, g, cols);
      if (pair) load8(a.pre + r * a.cols + a.N + c, u, cols);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        up[i] = 0.f;
        o[i] = d[i];
        if (a.act == kActRelu) {
          o[i] = g[i] > 0.f ? d[i] : (g[i] != g[i] ? g[i] : 0.f);
        } else if (a.act == kActGelu) {
          // far from 0 the gate is 0 or 1 and constant, and g^2 may be past fp32's range
          const float s = gelu_gate(g[i]), q = s * (1.f - s);
          const float bend = q == 0.f ? 0.f : g[i] * q * 1.5957691216057308f * (1.f + 0.134145f * g[i] * g[i]);
          o[i] = d[i] * (s + bend);
        } else if (a.act == kActSilu || pair) {
          const float s = sigmoid(g[i]);
          const float slope = s * (1.f + g[i] * (1.f - s));
          // what may be 0 first: d u and d g may be past fp32's range where dP is not. (The
          // slope is up to 1.1, so half of it: u slope stays in the range)
          o[i] = pair ? u[i] * (0.5f * slope) * d[i] * 2.f : d[i] * slope;
          if (pair) up[i] = g[i] * s * d[i];
        }
        sv[i] += o[i];
        su[i] += up[i];
      }
      if (a.dP) {
        // a row's last chunk takes the zeros behind it along (up's, for a pair)
        uint16_t* dst = a.dP + r * a.ld + c;
        if (!pair) {
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = i < cols ? o[i] : 0.f;
          store8(dst, o, 8);
        } else {
          store8(dst, o, cols);
          store8(dst + a.N, up, cols);
          if (cols <= 8)
            for (int64_t z = 2 * int64_t(a.N); z < a.ld; ++z) a.dP[r * a.ld + z] = 0;
        }
      }
    }
  }
  if (!a.sums) return;
  for (int part = 0; part < (pair ? 2 : 1); ++part) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) red[tr][8 * tc + i] = part ? su[i] : sv[i];
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += red[i][threadIdx.x];
    const int col = by * 256 + int(threadIdx.x);
    if (col < a.N) a.sums[int64_t(bx) * a.cols + part * a.N + col] = s;
  }
}

// What has to be done before the products, in one launch: dP, and rows made a multiple of
// 16 bytes. 16384 x 768 SwiGLU: 29 us for 126 MB (4.3 TB/s); 1003 x 777 with X and W of
// 1001 columns: 6.7 us, latency and launch (9.5 with 16 rows a block).
__global__ __launch_bounds__(256) void before_kernel(const DpArgs d, int slopes, const PadJob a, const PadJob b) {
  __shared__ float red[8][256];
  int block = int(blockIdx.x);
  if (block < slopes) return slope_rows(d, block, red);
  block -= slopes;
  if (block < a.blocks) return pad_rows(a, block);
  pad_rows(b, block - a.blocks);
}

// dbias from the blocks' sums; no blocks: zeros
__global__ __launch_bounds__(256) void bias_kernel(const float* __restrict__ sums, int blocks, int cols,
                                                   float* __restrict__ out) {
  __shared__ float red[4][64];
  bias_sums(sums, blocks, cols, out, int(blockIdx.x), red);
}

__global__ __launch_bounds__(256) void zero_kernel(uint16_t* __restrict__ p, int64_t n) {
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) p[i] = 0;
}

// ------------------------------------------------------------------ plans

// How a product M x N over kred is cut.
struct Plan {
  int tile;    // rows of a tile: 256 (x 256), 128 (x 128) or 64 (x 128)
  int splits;  // parts of the k axis
};

constexpr int kMaxSplits = 16;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int tile_cols(int tile) { return tile == 256 ? 256 : 128; }
int slots_of(int tile) { return tile == 128 ? 512 : 256; }  // workgroups that run at once

// The least of an estimate in microseconds, from products of 25 shapes in each of the three
// forms with every tile and splits of 1, 2, 4, 8 and 16 (the choice was the fastest, or
// within 10 % of it): a slab takes 1.6 us in a 256 x 256 tile (one a CU), 0.74 in a 128 x 128
// one alone on its CU and 1.0 with a second beside it, 0.37 in a 64 x 128 one (one a CU:
// four stages take its LDS); a tile's start and results 8, 3 and 2; joining parts a launch
// and their sums written and read.
Plan plan_of(int64_t M, int64_t N, int64_t kred) {
  const int64_t slabs = ceil_div(kred, BK);
  Plan best{64, 1};
  double least = 1e300;
  for (int tile : {256, 128, 64}) {
    const int64_t tiles = ceil_div(M, tile) * ceil_div(N, tile_cols(tile));
    // Very many short products wait for their results to be written, of which the estimate
    // knows nothing: 2^24 x 2048 x 16 takes 15.8 ms in 256 x 256 tiles and 18.2 in 128 x 128, 2^22 x 8192 x 16
    // 15.3 and 18.2. (Tiles are counted in 32 bits; M N < 2^36 makes them less than 2^24.)
    if (tile < 256 && tiles > (1 << 20)) continue;
    const int64_t slots = slots_of(tile);
    for (int64_t s = 1; s <= kMaxSplits && s <= slabs; ++s) {
      if (s > 1 && tiles * s > slots) break;
      const int64_t n = tiles * s, part = ceil_div(slabs, s), rest = n % slots;
      const double results = tile == 256 ? 8.0 : tile == 128 ? 3.0 : 2.0;
      const double slab = tile == 256 ? 1.6 : tile == 128 ? 1.0 : 0.37;
      const double last = tile == 128 && rest <= 256 ? 0.74 : slab;
      double t = double(n / slots) * (double(part) * slab + results);
      if (rest) t += double(part) * last + results;
      if (s > 1) t += 5.0 + 0.3 * double(s) + double(s) * double(M) * double(N) * 8.0 / 12e6;
      if (t < least) {
        least = t;
        best = Plan{tile, int(s)};
      }
    }
  }
  return best;
}

int64_t pad8(int64_t n) { return (n + 7) & ~int64_t(7); }

template <int BM, int BN, int WM, int WN, int NS>
hipError_t launch_tiles(const Problem& p, bool pmn, bool qmn, int64_t slots, hipStream_t st) {
  const int64_t tiles = int64_t(p.mt) * p.nt * p.splits;
  const dim3 grid(unsigned(std::min(tiles, slots))), block(64 * WM * WN);
  const bool split = p.splits > 1;
  // gradients have no activation, bias or residual
  auto kernel = pmn   ? (split ? tile_kernel<BM, BN, WM, WN, NS, true, true, kSplit> : tile_kernel<BM, BN, WM, WN, NS, true, true, kPlain>)
                : qmn ? (split ? tile_kernel<BM, BN, WM, WN, NS, false, true, kSplit>
                               : tile_kernel<BM, BN, WM, WN, NS, false, true, kPlain>)
                : split                     ? tile_kernel<BM, BN, WM, WN, NS, false, false, kSplit>
                : p.Q.pair                  ? tile_kernel<BM, BN, WM, WN, NS, false, false, kPair>
                : p.out.act != kActNone     ? tile_kernel<BM, BN, WM, WN, NS, false, false, kActs>
                                            : tile_kernel<BM, BN, WM, WN, NS, false, false, kPlain>;
  hipLaunchKernelGGL(kernel, grid, block, 0, st, p);
  return hipGetLastError();
}

// What the parts of a split product M x N may take at most: kMaxSplits of them, and as
// many tiles as run at once. Grows with M, so a scratch serves smaller M.
size_t partial_bytes(int64_t M, int64_t N) {
  const size_t all = size_t(kMaxSplits) * size_t(M) * size_t(ceil_div(N, 64) * 64) * 4;
  return std::min(all, size_t(256) * 256 * 256 * 4);
}

Problem problem(const Plan& pl, const Operand& P, const Operand& Q, int64_t kred, const Out& out, float* partial) {
  Problem p;
  p.P = P;
  p.Q = Q;
  p.kred = kred;
  p.Kp = int(pad8(kred));
  p.mt = int(ceil_div(P.ents, pl.tile));
  // a pair's columns come in groups of 64 with 32 of each part
  const int64_t ncols = Q.pair ? ceil_div(Q.ents / 2, 32) * 64 : Q.ents;
  p.nt = int(ceil_div(ncols, tile_cols(pl.tile)));
  const int64_t slabs = ceil_div(kred, BK);
  p.slabs = int(ceil_div(slabs, pl.splits));
  p.splits = int(ceil_div(slabs, p.slabs));
  p.partial = partial;
  p.ldp = ceil_div(ncols, 64) * 64;
  p.out = out;
  return p;
}

hipError_t product(const Operand& P, bool pmn, const Operand& Q, bool qmn, int64_t kred, const Out& out, float* partial,
                   hipStream_t st, KernelTimer* timer, const char* name) {
  const Plan pl = plan_of(P.ents, Q.ents, kred);
  const Problem p = problem(pl, P, Q, kred, out, partial);
  hipError_t e;
  {
    TimedLaunch tl(timer, name, st);
    e = pl.tile == 256 ? launch_tiles<256, 256, 2, 4, 2>(p, pmn, qmn, slots_of(256), st)
        : pl.tile == 128 ? launch_tiles<128, 128, 2, 2, 2>(p, pmn, qmn, slots_of(128), st)
                         : launch_tiles<64, 128, 2, 2, 4>(p, pmn, qmn, slots_of(64), st);
  }
  if (e != hipSuccess || p.splits == 1) return e;
  TimedLaunch tl(timer, "linear_join", st);
  const int64_t blocks = ceil_div(out.M * ceil_div(out.N, 8), 256);
  hipLaunchKernelGGL(join_kernel, dim3(unsigned(std::min<int64_t>(blocks, 4096))), dim3(256), 0, st, partial, p.splits,
                     p.ldp, Q.pair, out);
  return hipGetLastError();
}

PadJob pad_job(const uint16_t* in, int64_t R, int64_t C, uint16_t* out) {
  return PadJob{in, out, R, int(C), pad8(C), int(std::min<int64_t>(ceil_div(R * (pad8(C) / 8), 256), 8192))};
}

hipError_t before(const DpArgs& d, bool slopes, const PadJob& a, const PadJob& b, hipStream_t st, KernelTimer* timer) {
  const int64_t n = slopes ? int64_t(d.blocks) * ceil_div(d.N, 256) : 0;
  const int64_t grid = n + a.blocks + b.blocks;
  if (grid == 0) return hipSuccess;
  TimedLaunch tl(timer, "linear_before", st);
  hipLaunchKernelGGL(before_kernel, dim3(unsigned(grid)), dim3(256), 0, st, d, int(n), a, b);
  return hipGetLastError();
}

constexpr size_t kAlign = 256;
size_t up(size_t n) { return (n + kAlign - 1) / kAlign * kAlign; }

constexpr int64_t kDpRows = 8, kDpBlocks = 256;
// rows of a block of slope_rows: no more than kDpBlocks blocks
int64_t dp_rows(int64_t M) { return std::max<int64_t>(kDpRows, ceil_div(M, kDpBlocks)); }

// Rows that few_rows_kernel takes: whole calls of 1, 32 and 48 rows take 7.6, 10.7 and 12.8 us in
// it for N' = 1536, K = 2048 (SwiGLU) and 12.7, 13.8, 14.1 in tiles; for 4096 x 4096 9.3, 15.5, 20.2
// and 15.5, 15.9, 16.3; for 1001 x 777 8.1, 12.1, 16.4 and 14.3, 14.8, 14.9. One border for all
// sizes: at 48 rows the first would gain a tenth, the others lose a tenth and a quarter.
constexpr int64_t kFewRows = 32;

struct Layout {
  size_t x, w, dp, sums, partial, total;
};

Layout layout(const LinearArgs& a, bool bwd) {
  const int64_t R = a.act == kActSwiglu ? 2 * a.N : a.N;
  Layout L{};
  size_t o = 0;
  const bool odd = a.K % 8 != 0;
  L.x = o; o += odd ? up(size_t(a.M) * pad8(a.K) * 2) : 0;
  L.w = o; o += odd ? up(size_t(R) * pad8(a.K) * 2) : 0;
  if (!bwd) {
    L.partial = o;
    o += up(partial_bytes(a.M, R));
  } else {
    L.dp = o; o += up(size_t(a.M) * pad8(R) * 2);
    L.sums = o; o += up(size_t(std::min<int64_t>(ceil_div(a.M, kDpRows), kDpBlocks)) * R * 4);
    L.partial = o;
    o += up(std::max(partial_bytes(a.M, a.K), partial_bytes(R, a.K)));
  }
  L.total = o;
  return L;
}

}  // namespace lin

size_t linear_workspace_bytes(const LinearArgs& a, bool bwd) { return lin::layout(a, bwd).total; }

hipError_t launch_linear(const LinearArgs& a, const uint16_t* X, const uint16_t* W, const float* bias,
                         const void* residual, void* Y, uint16_t* pre, void* ws, hipStream_t st, KernelTimer* timer) {
  using namespace lin;
  if (a.M <= 0) return hipSuccess;
  const Layout L = layout(a, false);
  char* base = static_cast<char*>(ws);
  const int64_t R = a.act == kActSwiglu ? 2 * a.N : a.N;
  const Out out{bias, residual, Y, pre, a.M, int(a.N), a.act, a.out_f32};
  if (a.M <= kFewRows) {
    TimedLaunch tl(timer, "linear_few", st);
    const bool pair = a.act == kActSwiglu;
    const dim3 grid(unsigned(ceil_div(a.N, pair ? 8 : 16))), block(64 * kFewWaves);
    auto kernel = a.M <= 16 ? few_rows_kernel<1> : few_rows_kernel<2>;
    hipLaunchKernelGGL(kernel, grid, block, 0, st, X, W, int(a.M), int(a.K), pair, out);
    return hipGetLastError();
  }
  if (a.K % 8 != 0) {
    uint16_t* xp = reinterpret_cast<uint16_t*>(base + L.x);
    uint16_t* wp = reinterpret_cast<uint16_t*>(base + L.w);
    const hipError_t e = before(DpArgs{}, false, pad_job(X, a.M, a.K, xp), pad_job(W, R, a.K, wp), st, timer);
    if (e != hipSuccess) return e;
    X = xp;
    W = wp;
  }
  return product(Operand{X, pad8(a.K), a.M, false}, false, Operand{W, pad8(a.K), R, a.act == kActSwiglu}, false, a.K, out,
                 reinterpret_cast<float*>(base + L.partial), st, timer, "linear");
}

hipError_t launch_linear_bwd(const LinearArgs& a, const void* dY, const uint16_t* X, const uint16_t* W,
                             const uint16_t* pre, uint16_t* dX, uint16_t* dW, float* dbias, void* ws, hipStream_t st,
                             KernelTimer* timer) {
  using namespace lin;
  const int64_t R = a.act == kActSwiglu ? 2 * a.N : a.N;
  hipError_t e = hipSuccess;
  if (a.M <= 0) {
    if (dW) {
      TimedLaunch tl(timer, "linear_zero", st);
      hipLaunchKernelGGL(zero_kernel, dim3(unsigned(std::min<int64_t>(ceil_div(R * a.K, 256), 8192))), dim3(256), 0, st,
                         dW, R * a.K);
      e = hipGetLastError();
    }
    if (e == hipSuccess && dbias) {
      TimedLaunch tl(timer, "linear_dbias", st);
      hipLaunchKernelGGL(bias_kernel, dim3(unsigned(ceil_div(R, 64))), dim3(256), 0, st, nullptr, 0, int(R), dbias);
      e = hipGetLastError();
    }
    return e;
  }
  const Layout L = layout(a, true);
  char* base = static_cast<char*>(ws);
  const bool as_is = a.act == kActNone && !a.out_f32 && R % 8 == 0;  // dY is dP already
  const uint16_t* dP = static_cast<const uint16_t*>(dY);
  const bool products = dX || dW, slopes = dbias || (products && !as_is), odd = a.K % 8 != 0;
  DpArgs d{};
  if (slopes) {
    d.dY = dY;
    d.pre = pre;
    d.M = a.M;
    d.N = int(a.N);
    d.act = a.act;
    d.f32 = a.out_f32;
    d.dP = products && !as_is ? reinterpret_cast<uint16_t*>(base + L.dp) : nullptr;
    d.ld = pad8(R);
    d.sums = dbias ? reinterpret_cast<float*>(base + L.sums) : nullptr;
    d.cols = int(R);
    // (a grid has less than 2^32 threads)
    d.rows = int(dbias ? dp_rows(a.M) : std::max(kDpRows, ceil_div(a.M * ceil_div(a.N, 256), int64_t(1) << 20)));
    d.blocks = int(ceil_div(a.M, d.rows));
    if (d.dP) dP = d.dP;
  }
  uint16_t* wp = reinterpret_cast<uint16_t*>(base + L.w);
  uint16_t* xp = reinterpret_cast<uint16_t*>(base + L.x);
  e = before(d, slopes, dX && odd ? pad_job(W, R, a.K, wp) : PadJob{}, dW && odd ? pad_job(X, a.M, a.K, xp) : PadJob{},
             st, timer);
  if (e != hipSuccess) return e;
  if (odd) {
    W = wp;
    X = xp;
  }
  const int64_t ldr = pad8(R), ldk = pad8(a.K);
  float* partial = reinterpret_cast<float*>(base + L.partial);
  const Out ox{nullptr, nullptr, dX, nullptr, a.M, int(a.K), kActNone, false};
  const Out ow{nullptr, nullptr, dW, nullptr, R, int(a.K), kActNone, false};
  const Operand px{dP, ldr, a.M, false}, qx{W, ldk, a.K, false}, pw{dP, ldr, R, false}, qw{X, ldk, a.K, false};
  const int64_t nb = dbias ? ceil_div(R, 64) : 0;
  if (dX && dW) {
    const Plan plx = plan_of(a.M, a.K, R), plw = plan_of(R, a.K, a.M);
    if (plx.tile == 64 && plw.tile == 64 && plx.splits == 1 && plw.splits == 1) {
      const Problem x = problem(plx, px, qx, R, ox, partial), w = problem(plw, pw, qw, a.M, ow, partial);
      const int64_t nx = int64_t(x.mt) * x.nt, nw = int64_t(w.mt) * w.nt;
      if (nx + nw + nb <= slots_of(64)) {
        TimedLaunch tl(timer, "linear_dx_dw", st);
        hipLaunchKernelGGL((both_kernel<64, 128, 2, 2, 4>), dim3(unsigned(nx + nw + nb)), dim3(256), 0, st, x, w,
                           uint32_t(nx), uint32_t(nw), BiasArgs{d.sums, d.blocks, int(R), dbias});
        return hipGetLastError();
      }
    }
  }
  if (dbias) {
    TimedLaunch tl(timer, "linear_dbias", st);
    hipLaunchKernelGGL(bias_kernel, dim3(unsigned(nb)), dim3(256), 0, st, d.sums, d.blocks, int(R), dbias);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (dX && (e = product(px, false, qx, true, R, ox, partial, st, timer, "linear_dx")) != hipSuccess) return e;
  if (dW) e = product(pw, true, qw, true, a.M, ow, partial, st, timer, "linear_dw");
  return e;
}

}  // namespace moe
