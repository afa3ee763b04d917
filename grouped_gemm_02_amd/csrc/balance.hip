// Balance of the routing: load-balance loss, router z-loss, per-expert counts
// and their gradient to the logits (formulas in include/moe.h).
//
// A token's row of E logits is held by LPT = 4 .. 64 neighbouring lanes, four
// consecutive experts a lane and V such chunks (E <= 4 LPT V), so a wave
// works on 64 / LPT tokens at once and reads 16 bytes a lane. Row maxima and
// sums are butterflies over the LPT lanes in DPP and permlane swaps, and every
// group of lanes has the rows of several tokens in flight.
//
// Forward, in a fixed order without float atomics:
//   balance_partial  a workgroup per chunk of tokens (131,072 x 256 in 37 us,
//                    3.8 TB/s). The part of sequence q
//                    that lies in chunk b is piece b + q: b and q only grow
//                    from one piece to the next, so the numbers are distinct
//                    and at most chunks + S of them exist, without a scan.
//                    Each piece gets its sums of p and lse^2, its counts
//                    (integer atomics in LDS) and its live tokens.
//   balance_seq      a workgroup per sequence and 32 experts adds its pieces.
//   balance_finish   adds the sequences. (The last workgroup of balance_seq doing
//                    it, behind device-wide fences: 3 us more on 16,384 x 128, 9
//                    on 131,072 x 256.)
#include "device_common.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kBalThreads = 256;
constexpr int kBalRows = 4;  // 16-byte loads of logits a lane has in flight

typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));

// Tokens times row_cost up to which one workgroup does the whole forward of one
// sequence. In us (replayed), against the three launches: 2048 x 8 8.0 : 11.7, 4096 x 1
// 12.1 : 11.6, 4096 x 16 11.5 : 11.5, 1024 x 40 13.3 : 12.2, 256 x 130 15.4 : 14.0, 128 x 300
// 11.0 : 12.8, 64 x 1024 8.9 : 12.1, 80 x 805 10.4 : 12.6, 100 x 600 13.0 : 12.7; past it 8192 x 8
// 21.4 : 12.8, 32768 x 2 71.7 : 19.2, 1500 x 40 18.4 : 12.2, 400 x 160 23.1 : 14.2. (A workgroup
// that takes several sequences in turn: 4 to 7 us each.)
constexpr int64_t kSmallWork = 65536;

// Chunks of four experts a lane has of a row.
constexpr int lane_chunks(int E) { return E <= 256 ? 1 : E <= 512 ? 2 : 4; }
// Experts that a row costs the lanes of its layout: 4 LPT of with_layout, and those
// it has in the layout of four chunks, whose last ones are mostly past the row.
constexpr int row_cost(int E) {
  if (E > 512) return E;
  int w = 16;
  while (w < E) w *= 2;
  return w;
}

// Two rounds of loads a workgroup until kBalChunks workgroups are reached, then more (32
// tokens for any E: 3000 x 805 20.1 us instead of 16.8, 30 x 805 20.5 instead of 15.0).
constexpr int64_t kBalChunks = 1024;
int least_chunk(int E) { return 32 / lane_chunks(E); }
int balance_chunk_tokens(int64_t T, int E) {
  const int base = least_chunk(E);
  const int64_t c = ((T + kBalChunks - 1) / kBalChunks + base - 1) / base * base;
  return int(c < base ? base : c);
}

// Four logits of a row from expert e0 on; experts past E are -inf.
__device__ __forceinline__ f32x4 load4(const float* __restrict__ row, int e0, int E) {
  if (e0 + 4 <= E) return *reinterpret_cast<const f32x4u*>(row + e0);
  f32x4 v;
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = e0 + j < E ? row[e0 + j] : -INFINITY;
  return v;
}

// One step of a butterfly over 2, 4, 8, 16, 32, 64 lanes: the value that meets
// this lane's. The mirrors do for lanes that already agree in 4s and 8s what
// xor 4 and 8 would; the swaps give both halves at once.
template <int W, class Op>
__device__ __forceinline__ float butterfly(float v, Op op) {
  if constexpr (W == 2) return op(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 15, 15, true)));
  if constexpr (W == 4) return op(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 15, 15, true)));
  if constexpr (W == 8) return op(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 15, 15, true)));
  if constexpr (W == 16)
    return op(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 15, 15, true)));
  if constexpr (W == 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return op(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  if constexpr (W == 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return op(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  return v;
}
template <int LPT, class Op>
__device__ __forceinline__ float group_reduce(float v, Op op) {
  if constexpr (LPT >= 2) v = butterfly<2>(v, op);
  if constexpr (LPT >= 4) v = butterfly<4>(v, op);
  if constexpr (LPT >= 8) v = butterfly<8>(v, op);
  if constexpr (LPT >= 16) v = butterfly<16>(v, op);
  if constexpr (LPT >= 32) v = butterfly<32>(v, op);
  if constexpr (LPT >= 64) v = butterfly<64>(v, op);
  return v;
}
template <int LPT>
__device__ __forceinline__ float group_max(float v) {
  return group_reduce<LPT>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int LPT>
__device__ __forceinline__ float group_sum(float v) {
  return group_reduce<LPT>(v, [](float a, float b) { return a + b; });
}

// The sums over the groups of LPT lanes of a wave, lane by lane (rotations in
// rows of 16 lanes, then the swaps), in every group.
template <int LPT>
__device__ __forceinline__ float wave_groups_sum(float v) {
  if constexpr (LPT <= 8)
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x128, 15, 15, true));
  if constexpr (LPT <= 4)
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x124, 15, 15, true));
  if constexpr (LPT <= 16) v = butterfly<32>(v, [](float a, float b) { return a + b; });
  if constexpr (LPT <= 32) v = butterfly<64>(v, [](float a, float b) { return a + b; });
  return v;
}

// The softmax of one row, in powers of two on the transcendental unit: v
// becomes 2^((v - max) log2(e)), sum its sum, lse the log-sum-exp. The maximum is
// taken off first: finite logits of any magnitude leave differences in [-inf, 0]
// and a sum of 1 at least (scaled first, the maximum's own rounding grows with it
// and is past the exponent's range from 2^31 on). fmaxf drops a NaN, so a NaN
// reaches the sum through the power. A row of -inf alone gives v = 0 and sum = 0
// (and lse = -inf).
template <int LPT, int V>
__device__ __forceinline__ void row_softmax(f32x4 (&v)[V], float& sum, float& lse) {
  constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) m = fmaxf(m, v[i][j]);
  m = group_max<LPT>(m);
  if (m == -INFINITY) m = 0.f;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[i][j] = __builtin_amdgcn_exp2f((v[i][j] - m) * kLog2e);
      s += v[i][j];
    }
  sum = group_sum<LPT>(s);
  lse = fmaf(__builtin_amdgcn_logf(sum), kLn2, m);
}
// 1 / sum; 0 for a row of -inf alone, NaN stays
__device__ __forceinline__ float inverse_of(float sum) { return sum == 0.f ? 0.f : __builtin_amdgcn_rcpf(sum); }

// The last sequence that starts at or before t, in [0, S).
__device__ __forceinline__ int seq_of(const int32_t* __restrict__ off, int S, int64_t t) {
  int lo = 0, hi = S;  // off[lo] <= t (or lo == 0), hi: first known to start behind t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

struct BalancePieces {
  float* p;        // [pieces][E]
  int32_t* c;      // [pieces][E]
  double* z;       // [pieces]
  int32_t* n;      // [pieces]
};

// Sums over the tokens [lo, hi), by a workgroup of kGroups groups of LPT lanes:
// on return (after a barrier by the caller) sp[wave][e] holds the sums of p,
// sc[e] the counts, sz and sn each wave's sum of lse^2 and live tokens. The squares
// are 64-bit: a finite lse's may leave fp32 where their mean does not.
template <int LPT, int V, int kGroups>
__device__ __forceinline__ void sum_tokens(const float* __restrict__ logits, const int32_t* __restrict__ idx,
                                           int64_t lo, int64_t hi, int E, int k, const uint8_t* __restrict__ mask,
                                           float* sp, int32_t* sc, double* sz, int32_t* sn) {
  constexpr int U = kBalRows / V;
  const int grp = threadIdx.x / LPT, l = threadIdx.x % LPT;
  f32x4 acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  double z = 0.0;
  int32_t n = 0;
  // the trip count is the same for a whole wave: the butterflies stay converged
  for (int64_t b = lo; b < hi; b += kGroups * U) {
    // no load waits for another: rows and ids are read whatever the mask says
    f32x4 v[U][V];
    bool live[U];
    int e[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t tt = b + u * kGroups + grp;
      const int64_t tr = tt < hi ? tt : lo;
      live[u] = tt < hi && (!mask || mask[tr] != 0);
      e[u] = l < k ? idx[tr * k + l] : -1;
#pragma unroll
      for (int i = 0; i < V; ++i) v[u][i] = load4(logits + tr * E, 4 * (l + LPT * i), E);
    }
    for (int j0 = 0; j0 < k; j0 += LPT) {
      if (j0 > 0) {
#pragma unroll
        for (int u = 0; u < U; ++u)
          e[u] = live[u] && j0 + l < k ? idx[(b + u * kGroups + grp) * k + j0 + l] : -1;
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (live[u] && e[u] >= 0 && e[u] < E) atomicAdd(&sc[e[u]], 1);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float sum, lse;
      row_softmax<LPT, V>(v[u], sum, lse);
      if (live[u]) {
        const float inv = inverse_of(sum);
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] += v[u][i][j] * inv;
        z += sum == 0.f ? 0.0 : double(lse) * double(lse);
        ++n;
      }
    }
  }
#pragma unroll
  for (int o = LPT; o < 64; o *= 2) z += __shfl_xor(z, o);
  const float nf = wave_groups_sum<LPT>(float(n));  // exact: below 2^24 tokens a workgroup
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = wave_groups_sum<LPT>(acc[i][j]);
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) < LPT) {
#pragma unroll
    for (int i = 0; i < V; ++i) *reinterpret_cast<f32x4*>(sp + wave * 4 * LPT * V + 4 * (l + LPT * i)) = acc[i];
  }
  if ((threadIdx.x & 63) == 0) {
    sz[wave] = z;
    sn[wave] = int32_t(nf);
  }
}

template <int LPT, int V>
__global__ __launch_bounds__(kBalThreads) void balance_partial_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ idx, int64_t T, int E, int k,
    const int32_t* __restrict__ off, int S, const uint8_t* __restrict__ mask, int chunk, BalancePieces out) {
  constexpr int kGroups = kBalThreads / LPT, kWaves = kBalThreads / 64;
  __shared__ __attribute__((aligned(16))) float sp[kWaves * 4 * LPT * V];
  __shared__ int32_t sc[4 * LPT * V];
  __shared__ double sz[kWaves];
  __shared__ int32_t sn[kWaves];
  const int tid = threadIdx.x;
  const int64_t t0 = int64_t(blockIdx.x) * chunk, t1 = min(T, t0 + chunk);
  int q = off ? seq_of(off, S, t0) : 0;
  for (int64_t t = t0; t < t1 && q < S; ++q) {
    const int64_t qb = off ? int64_t(off[q]) : 0, qe = off ? int64_t(off[q + 1]) : T;
    const int64_t lo = max(t, qb), hi = min(t1, qe);
    if (qb >= t1) break;
    if (hi <= lo) continue;
    t = hi;
    for (int i = tid; i < E; i += kBalThreads) sc[i] = 0;
    __syncthreads();
    sum_tokens<LPT, V, kGroups>(logits, idx, lo, hi, E, k, mask, sp, sc, sz, sn);
    __syncthreads();
    const int64_t piece = int64_t(blockIdx.x) + q;
    for (int e = tid; e < E; e += kBalThreads) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) s += sp[w * 4 * LPT * V + e];
      out.p[piece * E + e] = s;
      out.c[piece * E + e] = sc[e];
    }
    if (tid == 0) {
      double s = 0.0;
      int32_t m = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        s += sz[w];
        m += sn[w];
      }
      out.z[piece] = s;
      out.n[piece] = m;
    }
    __syncthreads();
  }
}

// What balance_finish needs of each sequence.
struct BalanceSeq {
  double* term;  // [S][blocks of 32 experts] sum_e c P
  double* z;     // [S] sum of lse^2
  int32_t* n;    // [S] live tokens
};

// Sums over the workgroup's W waves, in every thread.
template <int N, int W>
__device__ __forceinline__ void block_sum(double (&v)[N], double (&sm)[N][W]) {
  const int tid = threadIdx.x;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor(v[i], o);
  if ((tid & 63) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) sm[i][tid >> 6] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = 0.0;
#pragma unroll
    for (int w = 0; w < W; ++w) v[i] += sm[i][w];
  }
}

constexpr int kSeqExperts = 32;

// 32 experts x 16 pieces at a time, kSeqBatch of them in flight. (1024 threads: 48
// sequences of 85 pieces and 256 experts 10.5 us instead of 7.4, a single one of
// 512 pieces and 128 experts 8.6 instead of 8.9.)
constexpr int kSeqBatch = 8, kSeqRows = 16, kSeqThreads = 32 * kSeqRows;
__global__ __launch_bounds__(kSeqThreads) void balance_seq_kernel(int64_t T, int E, const int32_t* __restrict__ off,
                                                           int chunk, BalancePieces in,
                                                           int32_t* __restrict__ seq_counts,
                                                           float* __restrict__ seq_probs, BalanceSeq out) {
  __shared__ double sm[2][kSeqThreads / 64];
  __shared__ double sP[kSeqRows][kSeqExperts + 1];
  __shared__ int32_t sC[kSeqRows][kSeqExperts + 1];
  const int q = blockIdx.x, tid = threadIdx.x;
  const int64_t lo = off ? max(int64_t(0), int64_t(off[q])) : 0;
  const int64_t hi = off ? min(T, int64_t(off[q + 1])) : T;
  const int64_t p0 = lo / chunk + q, p1 = hi > lo ? (hi - 1) / chunk + q + 1 : p0;
  const int e = blockIdx.y * kSeqExperts + (tid & 31);
  const int pl = tid >> 5;
  double zn[2] = {0.0, 0.0};
  for (int64_t p = p0 + tid; p < p1; p += kSeqThreads) {
    zn[0] += in.z[p];
    zn[1] += in.n[p];
  }
  double P = 0.0;
  int32_t c = 0;
  for (int64_t p = p0 + pl; p < p1; p += kSeqRows * kSeqBatch) {
    float x[kSeqBatch];
    int32_t y[kSeqBatch];
#pragma unroll
    for (int u = 0; u < kSeqBatch; ++u) {
      const int64_t at = (p + kSeqRows * u < p1 ? p + kSeqRows * u : p) * E + (e < E ? e : 0);
      x[u] = in.p[at];
      y[u] = in.c[at];
    }
#pragma unroll
    for (int u = 0; u < kSeqBatch; ++u)
      if (e < E && p + kSeqRows * u < p1) {
        P += x[u];
        c += y[u];
      }
  }
  sP[pl][tid & 31] = P;
  sC[pl][tid & 31] = c;
  block_sum(zn, sm);
  const double z = zn[0], n = zn[1];
  double term = 0.0;
  if (tid < kSeqExperts) {
    P = 0.0;
    c = 0;
#pragma unroll 8
    for (int i = 0; i < kSeqRows; ++i) {
      P += sP[i][tid];
      c += sC[i][tid];
    }
    if (e < E) {
      seq_counts[int64_t(q) * E + e] = c;
      seq_probs[int64_t(q) * E + e] = n > 0.0 ? float(P / n) : 0.f;
    }
    term = double(c) * P;
    for (int o = 16; o > 0; o >>= 1) term += __shfl_xor(term, o, 32);
    if (tid == 0) {
      out.term[int64_t(q) * gridDim.y + blockIdx.y] = term;
      if (blockIdx.y == 0) {
        out.z[q] = z;
        out.n[q] = int32_t(n);
      }
    }
  }
}

// Workgroup 0: the losses and the factors; the others 64 experts' counts each.
__global__ __launch_bounds__(1024) void balance_finish_kernel(int E, int k, int S, int blocks, BalanceSeq in,
                                                              const int32_t* __restrict__ seq_counts,
                                                              float* __restrict__ loss, int32_t* __restrict__ counts,
                                                              float* __restrict__ seq_scale) {
  __shared__ double sm[4][16];
  __shared__ int32_t sC[16][64];
  const int tid = threadIdx.x;
  if (blockIdx.x > 0) {
    const int e = (blockIdx.x - 1) * 64 + (tid & 63);
    int32_t c = 0;
    if (e < E) {
#pragma unroll 4
      for (int q = tid >> 6; q < S; q += 16) c += seq_counts[int64_t(q) * E + e];
    }
    sC[tid >> 6][tid & 63] = c;
    __syncthreads();
    if (tid < 64 && e < E) {
      c = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) c += sC[i][tid];
      counts[e] = c;
    }
    return;
  }
  double v[4] = {0.0, 0.0, 0.0, 0.0};  // the balance terms, lse^2, live tokens, sequences with any
  for (int q = tid; q < S; q += 1024) {
    const double nq = in.n[q];
    double t = 0.0;
#pragma unroll 8
    for (int b = 0; b < blocks; ++b) t += in.term[int64_t(q) * blocks + b];
    v[1] += in.z[q];
    v[2] += nq;
    if (nq > 0.0) {
      v[0] += t * double(E) / (double(k) * nq * nq);
      v[3] += 1.0;
    }
  }
  block_sum(v, sm);
  const double term = v[0], z = v[1], n = v[2], used = v[3];
  for (int q = tid; q < S; q += 1024) {
    const double nq = in.n[q];
    seq_scale[q] = nq > 0.0 ? float(double(E) / (used * double(k) * nq * nq)) : 0.f;
  }
  if (tid == 0) {
    loss[0] = used > 0.0 ? float(term / used) : 0.f;
    loss[1] = n > 0.0 ? float(z / n) : 0.f;
    seq_scale[S] = n > 0.0 ? float(1.0 / n) : 0.f;
  }
}

// The whole forward of one sequence in one workgroup.
template <int LPT, int V>
__global__ __launch_bounds__(1024) void balance_small_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ idx, int64_t T, int E, int k,
    const int32_t* __restrict__ off, const uint8_t* __restrict__ mask, float* __restrict__ loss,
    int32_t* __restrict__ counts, int32_t* __restrict__ seq_counts, float* __restrict__ seq_probs,
    float* __restrict__ seq_scale) {
  constexpr int kGroups = 1024 / LPT;
  __shared__ __attribute__((aligned(16))) float sp[16 * 4 * LPT * V];
  __shared__ int32_t sc[4 * LPT * V];
  __shared__ double sz[16];
  __shared__ int32_t sn[16];
  __shared__ double sm[1][16];
  const int tid = threadIdx.x;
  const int64_t lo = off ? max(int64_t(0), int64_t(off[0])) : 0;
  const int64_t hi = off ? min(T, int64_t(off[1])) : T;
  if (tid < E) sc[tid] = 0;  // E <= 1024
  __syncthreads();
  sum_tokens<LPT, V, kGroups>(logits, idx, lo, hi, E, k, mask, sp, sc, sz, sn);
  __syncthreads();
  double z = 0.0, n = 0.0, P = 0.0;
#pragma unroll
  for (int w = 0; w < 16; ++w) {
    z += sz[w];
    n += double(sn[w]);
  }
  int32_t c = 0;
  if (tid < E) {
#pragma unroll
    for (int w = 0; w < 16; ++w) P += sp[w * 4 * LPT * V + tid];
    c = sc[tid];
    counts[tid] = c;
    seq_counts[tid] = c;
    seq_probs[tid] = n > 0.0 ? float(P / n) : 0.f;
  }
  double t[1] = {double(c) * P};
  block_sum(t, sm);
  if (tid == 0) {
    const bool any = n > 0.0;
    loss[0] = any ? float(t[0] * double(E) / (double(k) * n * n)) : 0.f;
    loss[1] = any ? float(z / n) : 0.f;
    seq_scale[0] = any ? float(double(E) / (double(k) * n * n)) : 0.f;
    seq_scale[1] = any ? float(1.0 / n) : 0.f;
  }
}

// Rows a group of the backward has in flight, and the tokens of a workgroup.
// 131,072 x 256: two rows and 32 tokens 71 us, four rows 83, two rows and 64
// tokens 85, four rows and 128 tokens 113 (fewer registers and more
// workgroups: more loads in flight); 16,384 x 128: 16 tokens 9.6 us, 32 10.6; below
// 4096 tokens as many workgroups as CUs: 30 x 805 8.4 us, with 16 tokens 12.9, 3000 x
// 805 10.7 and 12.1.
constexpr int bwd_rows(int V) { return V == 1 ? 2 : 1; }
int bwd_chunk(int64_t T, int groups, int V) {
  const int base = T >= 65536 ? 32 : T >= 16 * 256 ? 16 : int((T + 255) / 256), batch = groups * bwd_rows(V);
  return base > batch ? (base + batch - 1) / batch * batch : batch;
}

// One pass over the logits. HBM-bound for long batches (reads and writes a
// row of E floats a token: 131,072 x 256 in 72 us, 3.9 TB/s; 75 without the
// streaming stores), latency-bound for short ones.
template <int LPT, int V>
__global__ __launch_bounds__(kBalThreads) void balance_bwd_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ idx, const float* __restrict__ w,
    const float* __restrict__ dw, int64_t T, int E, int k, int renorm, const int32_t* __restrict__ off, int S,
    const uint8_t* __restrict__ mask, const int32_t* __restrict__ seq_counts, const float* __restrict__ seq_scale,
    const float* __restrict__ d_loss, int chunk, float* __restrict__ dz) {
  constexpr int kGroups = kBalThreads / LPT;
  constexpr int U = bwd_rows(V);
  __shared__ __attribute__((aligned(16))) float sel[U * kGroups * 4 * LPT * V];
  const int tid = threadIdx.x, grp = tid / LPT, l = tid % LPT;
  const int64_t t0 = int64_t(blockIdx.x) * chunk, t1 = min(T, t0 + chunk);
  const float gb = d_loss[0], gz = 2.f * d_loss[1] * seq_scale[S];
  int q = -1;              // the sequence whose B is in bal
  int64_t qb = 0, qe = 0;  // its bounds
  f32x4 bal[V];
#pragma unroll
  for (int i = 0; i < V; ++i) bal[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  float* const row = sel + grp * 4 * LPT * V;  // the group's selected experts' values, kRow apart
  constexpr int kRow = kGroups * 4 * LPT * V;
  for (int64_t b = t0; b < t1; b += kGroups * U) {
    f32x4 v[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = b + u * kGroups + grp;
      const int64_t tr = t < t1 ? t : t0;
#pragma unroll
      for (int i = 0; i < V; ++i) v[u][i] = load4(logits + tr * E, 4 * (l + LPT * i), E);
    }
    // the first LPT slots of each row; more are read below
    int ej[U];
    float dj[U], wj[U];
    bool on[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = b + u * kGroups + grp;
      const bool has = dw && t < t1 && l < k;
      ej[u] = has ? idx[t * k + l] : -1;
      dj[u] = has ? dw[t * k + l] : 0.f;
      wj[u] = has && renorm ? w[t * k + l] : 0.f;
      on[u] = t < t1 && (!mask || mask[t] != 0);
    }
    if (dw) {
      // the slots' values to their experts through LDS; the lanes of a group
      // are in one wave, whose LDS operations are in order
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < V; ++i)
          *reinterpret_cast<f32x4*>(row + u * kRow + 4 * (l + LPT * i)) = f32x4{0.f, 0.f, 0.f, 0.f};
      asm volatile("" ::: "memory");
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t t = b + u * kGroups + grp;
        const int kt = t < t1 ? k : 0;
        float c = 0.f;
        if (renorm) {
          c = wj[u] * dj[u];
          for (int j = l + LPT; j < kt; j += LPT) c += w[t * k + j] * dw[t * k + j];
          c = group_sum<LPT>(c);
        }
        if (ej[u] >= 0 && ej[u] < E) atomicAdd(row + u * kRow + ej[u], renorm ? wj[u] * (dj[u] - c) : dj[u]);
        for (int j = l + LPT; j < kt; j += LPT) {
          const int e = idx[t * k + j];
          const float d = dw[t * k + j];
          if (e >= 0 && e < E) atomicAdd(row + u * kRow + e, renorm ? w[t * k + j] * (d - c) : d);
        }
      }
      asm volatile("" ::: "memory");
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = b + u * kGroups + grp;
      const bool in = t < t1;
      if (in && (q < 0 || t >= qe || t < qb)) {
        q = off ? seq_of(off, S, t) : 0;
        qb = off ? int64_t(off[q]) : 0;
        qe = off ? int64_t(off[q + 1]) : T;
        const float sc = gb * seq_scale[q];
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int e = 4 * (l + LPT * i) + j;
            bal[i][j] = e < E ? sc * float(seq_counts[int64_t(q) * E + e]) : 0.f;
          }
      }
      const bool live = on[u] && t >= qb && t < qe;
      float sum, lse;
      row_softmax<LPT, V>(v[u], sum, lse);
      const float inv = inverse_of(sum);
      // G: what is weighted by p; H: the renormalised weights' gradient, added as it
      // is. A row outside the losses may hold anything: without G there, p is 0.
      const bool need = live || (dw && !renorm);
      f32x4 G[V], H[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        H[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        v[u][i] = need ? v[u][i] * inv : H[i];
        G[i] = live ? bal[i] : H[i];
        if (dw) {
          const f32x4 x = *reinterpret_cast<const f32x4*>(row + u * kRow + 4 * (l + LPT * i));
          if (renorm) H[i] = x; else G[i] += x;
        }
      }
      float pg = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) pg += v[u][i][j] * G[i][j];
      pg = group_sum<LPT>(pg);
      const float zt = live && sum != 0.f ? gz * lse : 0.f;
      if (in) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int e0 = 4 * (l + LPT * i);
          f32x4 o;
#pragma unroll
          for (int j = 0; j < 4; ++j) o[j] = v[u][i][j] * (G[i][j] - pg + zt) + H[i][j];
          float* dst = dz + t * E + e0;
          if (e0 + 4 <= E) {
            __builtin_nontemporal_store(o, reinterpret_cast<f32x4u*>(dst));
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (e0 + j < E) dst[j] = o[j];
          }
        }
      }
    }
    asm volatile("" ::: "memory");
  }
}

// Runs f with the lane layout of E experts: f.template operator()<LPT, V>().
template <class F>
void with_layout(int E, F f) {
  if (E <= 16) f.template operator()<4, 1>();
  else if (E <= 32) f.template operator()<8, 1>();
  else if (E <= 64) f.template operator()<16, 1>();
  else if (E <= 128) f.template operator()<32, 1>();
  else if (E <= 256) f.template operator()<64, 1>();
  else if (E <= 512) f.template operator()<64, 2>();
  else f.template operator()<64, 4>();
}

struct BalanceWs {
  size_t p, c, z, n, term, qz, qn, total;
};
int seq_blocks(int E) { return (E + kSeqExperts - 1) / kSeqExperts; }
size_t up256(size_t v) { return (v + 255) / 256 * 256; }
BalanceWs balance_ws(int64_t T, int E, int64_t S) {
  // chunks: the most of any batch of up to T tokens, so that its scratch serves them all
  const int64_t most = (T + least_chunk(E) - 1) / least_chunk(E);
  const size_t pieces = size_t((most < kBalChunks ? most : kBalChunks) + S);
  BalanceWs L;
  size_t o = 0;
  L.p = o;    o = up256(o + pieces * size_t(E) * 4);
  L.c = o;    o = up256(o + pieces * size_t(E) * 4);
  L.z = o;    o = up256(o + pieces * 8);
  L.n = o;    o = up256(o + pieces * 4);
  L.term = o; o = up256(o + size_t(S) * seq_blocks(E) * 8);
  L.qz = o;   o = up256(o + size_t(S) * 8);
  L.qn = o;   o = up256(o + size_t(S) * 4);
  L.total = o;
  return L;
}

struct PartialLaunch {
  const BalanceArgs& a;
  BalancePieces pc;
  int chunk;
  dim3 grid;
  hipStream_t st;
  template <int LPT, int V>
  void operator()() const {
    hipLaunchKernelGGL((balance_partial_kernel<LPT, V>), grid, dim3(kBalThreads), 0, st, a.logits, a.idx, a.T, a.E, a.k,
                       a.off, int(a.S), a.mask, chunk, pc);
  }
};

struct SmallLaunch {
  const BalanceArgs& a;
  float* loss;
  int32_t *counts, *seq_counts;
  float *seq_probs, *seq_scale;
  hipStream_t st;
  template <int LPT, int V>
  void operator()() const {
    hipLaunchKernelGGL((balance_small_kernel<LPT, V>), dim3(1), dim3(1024), 0, st, a.logits, a.idx, a.T, a.E, a.k, a.off,
                       a.mask, loss, counts, seq_counts, seq_probs, seq_scale);
  }
};

struct BwdLaunch {
  const BalanceArgs& a;
  const float *w, *dw;
  int renorm;
  const int32_t* seq_counts;
  const float *seq_scale, *d_loss;
  float* dz;
  hipStream_t st;
  template <int LPT, int V>
  void operator()() const {
    const int chunk = bwd_chunk(a.T, kBalThreads / LPT, V);
    const dim3 grid(unsigned((a.T + chunk - 1) / chunk));
    hipLaunchKernelGGL((balance_bwd_kernel<LPT, V>), grid, dim3(kBalThreads), 0, st, a.logits, a.idx, w, dw, a.T, a.E,
                       a.k, renorm, a.off, int(a.S), a.mask, seq_counts, seq_scale, d_loss, chunk, dz);
  }
};

}  // namespace

size_t balance_scratch_bytes(int64_t T, int E, int64_t S) { return balance_ws(T, E, S).total; }

hipError_t launch_balance(const BalanceArgs& a, float* loss, int32_t* counts, int32_t* seq_counts, float* seq_probs,
                          float* seq_scale, void* ws, hipStream_t st, KernelTimer* timer) {
  if (a.S == 1 && a.T * row_cost(a.E) <= kSmallWork) {
    TimedLaunch tl(timer, "balance_small", st);
    with_layout(a.E, SmallLaunch{a, loss, counts, seq_counts, seq_probs, seq_scale, st});
    return hipGetLastError();
  }
  const BalanceWs L = balance_ws(a.T, a.E, a.S);
  char* base = static_cast<char*>(ws);
  const BalancePieces pc{reinterpret_cast<float*>(base + L.p), reinterpret_cast<int32_t*>(base + L.c),
                         reinterpret_cast<double*>(base + L.z), reinterpret_cast<int32_t*>(base + L.n)};
  const BalanceSeq sq{reinterpret_cast<double*>(base + L.term), reinterpret_cast<double*>(base + L.qz),
                      reinterpret_cast<int32_t*>(base + L.qn)};
  const int chunk = balance_chunk_tokens(a.T, a.E);
  if (a.T > 0) {
    TimedLaunch tl(timer, "balance_partial", st);
    with_layout(a.E, PartialLaunch{a, pc, chunk, dim3(unsigned((a.T + chunk - 1) / chunk)), st});
  }
  const int blocks = seq_blocks(a.E);
  {
    TimedLaunch tl(timer, "balance_seq", st);
    hipLaunchKernelGGL(balance_seq_kernel, dim3(unsigned(a.S), unsigned(blocks)), dim3(kSeqThreads), 0, st, a.T, a.E, a.off,
                       chunk, pc, seq_counts, seq_probs, sq);
  }
  {
    TimedLaunch tl(timer, "balance_finish", st);
    hipLaunchKernelGGL(balance_finish_kernel, dim3(unsigned(1 + (a.E + 63) / 64)), dim3(1024), 0, st, a.E, a.k, int(a.S),
                       blocks, sq, seq_counts, loss, counts, seq_scale);
  }
  return hipGetLastError();
}

hipError_t launch_balance_bwd(const BalanceArgs& a, const float* w, const float* dw, int renorm,
                              const int32_t* seq_counts, const float* seq_scale, const float* d_loss, float* dz,
                              hipStream_t st, KernelTimer* timer) {
  if (a.T <= 0) return hipSuccess;
  TimedLaunch tl(timer, "balance_bwd", st);
  with_layout(a.E, BwdLaunch{a, w, dw, renorm, seq_counts, seq_scale, d_loss, dz, st});
  return hipGetLastError();
}

}  // namespace moe
