// Balance of the routing: load-balance loss, router z-loss, per-expert counts
// and their gradient to the logits (formulas in include/moe.h).
//
// A token's row of E logits is held by LPT = 4 .. 64 neighbouring lanes, four
// consecutive experts a lane and V such chunks (E <= 4 LPT V), so a wave
// works on 64 / LPT tokens at once and reads 16 bytes a lane. Row maxima and
// sums are butterflies over the LPT lanes.
//
// Forward, in a fixed order without float atomics:
//   balance_partial  a workgroup per chunk of tokens. The part of sequence q
//                    that lies in chunk b is piece b + q: b and q only grow
//                    from one piece to the next, so the numbers are distinct
//                    and at most chunks + S of them exist, without a scan.
//                    Each piece gets its sums of p and lse^2, its counts
//                    (integer atomics in LDS) and its live tokens.
//   balance_seq      a workgroup per sequence adds its pieces.
//   balance_finish   one workgroup adds the sequences.
#include "device_common.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kBalThreads = 256;

typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));

int balance_chunk_tokens(int64_t T) {
  // 32 tokens a workgroup until 1024 workgroups are reached, then more
  int64_t c = (T + 1023) / 1024;
  c = (c + 31) / 32 * 32;
  return int(c < 32 ? 32 : c);
}

// Four logits of a row from expert e0 on; experts past E are -inf.
__device__ __forceinline__ f32x4 load4(const float* __restrict__ row, int e0, int E) {
  if (e0 + 4 <= E) return *reinterpret_cast<const f32x4u*>(row + e0);
  f32x4 v;
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = e0 + j < E ? row[e0 + j] : -INFINITY;
  return v;
}

template <int LPT>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int off = LPT / 2; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off));
  return v;
}
template <int LPT>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int off = LPT / 2; off > 0; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

// The softmax of one row: v becomes exp(v - max), sum its sum, lse the
// log-sum-exp. fmaxf drops a NaN, so a NaN reaches the sum through exp. A row
// of -inf alone gives v = 0 and sum = 0 (and lse = -inf).
template <int LPT, int V>
__device__ __forceinline__ void row_softmax(f32x4 (&v)[V], float& sum, float& lse) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) m = fmaxf(m, v[i][j]);
  m = group_max<LPT>(m);
  const float ref = m == -INFINITY ? 0.f : m;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[i][j] = expf(v[i][j] - ref);
      s += v[i][j];
    }
  sum = group_sum<LPT>(s);
  lse = m + logf(sum);
}

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
  float* z;        // [pieces]
  int32_t* n;      // [pieces]
};

template <int LPT, int V>
__global__ __launch_bounds__(kBalThreads) void balance_partial_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ idx, int64_t T, int E, int k,
    const int32_t* __restrict__ off, int S, const uint8_t* __restrict__ mask, int chunk, BalancePieces out) {
  constexpr int kGroups = kBalThreads / LPT;
  __shared__ float sp[kGroups * 4 * LPT * V];
  __shared__ int32_t sc[4 * LPT * V];
  __shared__ float sz[kGroups];
  __shared__ int32_t sn[kGroups];
  const int tid = threadIdx.x, grp = tid / LPT, l = tid % LPT;
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
    f32x4 acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    float z = 0.f;
    int32_t n = 0;
    // the trip count is the same for a whole wave: shuffles stay converged
    for (int64_t b = lo; b < hi; b += kGroups) {
      const int64_t tt = b + grp;
      const bool in = tt < hi;
      const bool live = in && (!mask || mask[tt] != 0);
      if (!__any(live)) continue;
      const int64_t tr = live ? tt : lo;
      f32x4 v[V];
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = load4(logits + tr * E, 4 * (l + LPT * i), E);
      float sum, lse;
      row_softmax<LPT, V>(v, sum, lse);
      if (live) {
        const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] += v[i][j] * inv;
        z += sum == 0.f ? 0.f : lse * lse;
        ++n;
        for (int j = l; j < k; j += LPT) {
          const int e = idx[tt * k + j];
          if (e >= 0 && e < E) atomicAdd(&sc[e], 1);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) sp[grp * 4 * LPT * V + 4 * (l + LPT * i) + j] = acc[i][j];
    if (l == 0) {
      sz[grp] = z;
      sn[grp] = n;
    }
    __syncthreads();
    const int64_t piece = int64_t(blockIdx.x) + q;
    for (int e = tid; e < E; e += kBalThreads) {
      float s = 0.f;
#pragma unroll 8
      for (int g = 0; g < kGroups; ++g) s += sp[g * 4 * LPT * V + e];
      out.p[piece * E + e] = s;
      out.c[piece * E + e] = sc[e];
    }
    if (tid == 0) {
      float s = 0.f;
      int32_t m = 0;
      for (int g = 0; g < kGroups; ++g) {
        s += sz[g];
        m += sn[g];
      }
      out.z[piece] = s;
      out.n[piece] = m;
    }
    __syncthreads();
  }
}

// What balance_finish needs of each sequence.
struct BalanceSeq {
  double* term;  // [S] sum_e c P
  double* z;     // [S] sum of lse^2
  int32_t* n;    // [S] live tokens
};

__device__ __forceinline__ double block_sum(double v, double* sm) {
  const int tid = threadIdx.x;
  sm[tid] = v;
  __syncthreads();
  for (int o = blockDim.x / 2; o > 0; o >>= 1) {
    if (tid < o) sm[tid] += sm[tid + o];
    __syncthreads();
  }
  const double r = sm[0];
  __syncthreads();
  return r;
}

__global__ __launch_bounds__(kBalThreads) void balance_seq_kernel(int64_t T, int E, const int32_t* __restrict__ off,
                                                                  int chunk, BalancePieces in,
                                                                  int32_t* __restrict__ seq_counts,
                                                                  float* __restrict__ seq_probs, BalanceSeq out) {
  __shared__ double sm[kBalThreads];
  const int q = blockIdx.x, tid = threadIdx.x;
  const int64_t lo = off ? max(int64_t(0), int64_t(off[q])) : 0;
  const int64_t hi = off ? min(T, int64_t(off[q + 1])) : T;
  const int64_t p0 = lo / chunk + q, p1 = hi > lo ? (hi - 1) / chunk + q + 1 : p0;
  double z = 0.0, n = 0.0;
  for (int64_t p = p0 + tid; p < p1; p += kBalThreads) {
    z += in.z[p];
    n += in.n[p];
  }
  z = block_sum(z, sm);
  n = block_sum(n, sm);
  double term = 0.0;
  for (int e = tid; e < E; e += kBalThreads) {
    double P = 0.0;
    int32_t c = 0;
    for (int64_t p = p0; p < p1; ++p) {
      P += in.p[p * E + e];
      c += in.c[p * E + e];
    }
    seq_counts[int64_t(q) * E + e] = c;
    seq_probs[int64_t(q) * E + e] = n > 0.0 ? float(P / n) : 0.f;
    term += double(c) * P;
  }
  term = block_sum(term, sm);
  if (tid == 0) {
    out.term[q] = term;
    out.z[q] = z;
    out.n[q] = int32_t(n);
  }
}

__global__ __launch_bounds__(kBalThreads) void balance_finish_kernel(int E, int k, int S, BalanceSeq in,
                                                                     const int32_t* __restrict__ seq_counts,
                                                                     float* __restrict__ loss,
                                                                     int32_t* __restrict__ counts,
                                                                     float* __restrict__ seq_scale) {
  __shared__ double sm[kBalThreads];
  const int tid = threadIdx.x;
  double term = 0.0, z = 0.0, n = 0.0, used = 0.0;
  for (int q = tid; q < S; q += kBalThreads) {
    const double nq = in.n[q];
    z += in.z[q];
    n += nq;
    if (nq > 0.0) {
      term += in.term[q] * double(E) / (double(k) * nq * nq);
      used += 1.0;
    }
  }
  term = block_sum(term, sm);
  z = block_sum(z, sm);
  n = block_sum(n, sm);
  used = block_sum(used, sm);
  for (int q = tid; q < S; q += kBalThreads) {
    const double nq = in.n[q];
    seq_scale[q] = nq > 0.0 ? float(double(E) / (used * double(k) * nq * nq)) : 0.f;
  }
  for (int e = tid; e < E; e += kBalThreads) {
    int32_t c = 0;
    for (int q = 0; q < S; ++q) c += seq_counts[int64_t(q) * E + e];
    counts[e] = c;
  }
  if (tid == 0) {
    loss[0] = used > 0.0 ? float(term / used) : 0.f;
    loss[1] = n > 0.0 ? float(z / n) : 0.f;
    seq_scale[S] = n > 0.0 ? float(1.0 / n) : 0.f;
  }
}

// One pass over the logits. HBM-bound for long batches (reads and writes a
// row of E floats a token), latency-bound for short ones.
template <int LPT, int V>
__global__ __launch_bounds__(kBalThreads) void balance_bwd_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ idx, const float* __restrict__ w,
    const float* __restrict__ dw, int64_t T, int E, int k, int renorm, const int32_t* __restrict__ off, int S,
    const uint8_t* __restrict__ mask, const int32_t* __restrict__ seq_counts, const float* __restrict__ seq_scale,
    const float* __restrict__ d_loss, int chunk, float* __restrict__ dz) {
  constexpr int kGroups = kBalThreads / LPT;
  const int tid = threadIdx.x, grp = tid / LPT, l = tid % LPT;
  const int64_t t0 = int64_t(blockIdx.x) * chunk, t1 = min(T, t0 + chunk);
  const float gb = d_loss[0], gz = 2.f * d_loss[1] * seq_scale[S];
  int q = -1;              // the sequence whose B is in bal
  int64_t qb = 0, qe = 0;  // its bounds
  f32x4 bal[V];
#pragma unroll
  for (int i = 0; i < V; ++i) bal[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int64_t b = t0; b < t1; b += kGroups) {
    const int64_t t = b + grp;
    const bool in = t < t1;
    const int64_t tr = in ? t : t0;
    f32x4 v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = load4(logits + tr * E, 4 * (l + LPT * i), E);
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
    const bool live = in && t >= qb && t < qe && (!mask || mask[t] != 0);
    float sum, lse;
    row_softmax<LPT, V>(v, sum, lse);
    const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
    // G: what is weighted by p; H: the renormalised weights' gradient, added as it is
    f32x4 G[V], H[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      v[i] *= inv;
      H[i] = f32x4{0.f, 0.f, 0.f, 0.f};
      G[i] = live ? bal[i] : H[i];
    }
    if (dw) {
      float c = 0.f;
      if (renorm) {
        for (int j = l; j < k; j += LPT) c += w[tr * k + j] * dw[tr * k + j];
        c = group_sum<LPT>(c);
      }
      for (int j0 = 0; j0 < k; j0 += LPT) {
        const int j = j0 + l;
        const int ej = j < k ? idx[tr * k + j] : -1;
        const float dj = j < k ? dw[tr * k + j] : 0.f;
        const float xj = renorm && j < k ? w[tr * k + j] * (dj - c) : dj;
        const int nj = min(LPT, k - j0);
        for (int s = 0; s < nj; ++s) {
          const int e = __shfl(ej, s, LPT);
          const float x = __shfl(xj, s, LPT);
#pragma unroll
          for (int i = 0; i < V; ++i)
#pragma unroll
            for (int jj = 0; jj < 4; ++jj)
              if (e == 4 * (l + LPT * i) + jj) {
                if (renorm) H[i][jj] += x; else G[i][jj] += x;
              }
        }
      }
    }
    float pg = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) pg += v[i][j] * G[i][j];
    pg = group_sum<LPT>(pg);
    const float zt = live && sum != 0.f ? gz * lse : 0.f;
    if (in) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e0 = 4 * (l + LPT * i);
        f32x4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = v[i][j] * (G[i][j] - pg + zt) + H[i][j];
        float* dst = dz + t * E + e0;
        if (e0 + 4 <= E) {
          *reinterpret_cast<f32x4u*>(dst) = o;
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (e0 + j < E) dst[j] = o[j];
        }
      }
    }
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
size_t up256(size_t v) { return (v + 255) / 256 * 256; }
BalanceWs balance_ws(int64_t T, int E, int64_t S) {
  const int chunk = balance_chunk_tokens(T);
  const size_t pieces = size_t((T + chunk - 1) / chunk + S);
  BalanceWs L;
  size_t o = 0;
  L.p = o;    o = up256(o + pieces * size_t(E) * 4);
  L.c = o;    o = up256(o + pieces * size_t(E) * 4);
  L.z = o;    o = up256(o + pieces * 4);
  L.n = o;    o = up256(o + pieces * 4);
  L.term = o; o = up256(o + size_t(S) * 8);
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

struct BwdLaunch {
  const BalanceArgs& a;
  const float *w, *dw;
  int renorm;
  const int32_t* seq_counts;
  const float *seq_scale, *d_loss;
  float* dz;
  int chunk;
  dim3 grid;
  hipStream_t st;
  template <int LPT, int V>
  void operator()() const {
    hipLaunchKernelGGL((balance_bwd_kernel<LPT, V>), grid, dim3(kBalThreads), 0, st, a.logits, a.idx, w, dw, a.T, a.E,
                       a.k, renorm, a.off, int(a.S), a.mask, seq_counts, seq_scale, d_loss, chunk, dz);
  }
};

}  // namespace

size_t balance_scratch_bytes(int64_t T, int E, int64_t S) { return balance_ws(T, E, S).total; }

hipError_t launch_balance(const BalanceArgs& a, float* loss, int32_t* counts, int32_t* seq_counts, float* seq_probs,
                          float* seq_scale, void* ws, hipStream_t st, KernelTimer* timer) {
  const BalanceWs L = balance_ws(a.T, a.E, a.S);
  char* base = static_cast<char*>(ws);
  const BalancePieces pc{reinterpret_cast<float*>(base + L.p), reinterpret_cast<int32_t*>(base + L.c),
                         reinterpret_cast<float*>(base + L.z), reinterpret_cast<int32_t*>(base + L.n)};
  const BalanceSeq sq{reinterpret_cast<double*>(base + L.term), reinterpret_cast<double*>(base + L.qz),
                      reinterpret_cast<int32_t*>(base + L.qn)};
  const int chunk = balance_chunk_tokens(a.T);
  if (a.T > 0) {
    TimedLaunch tl(timer, "balance_partial", st);
    with_layout(a.E, PartialLaunch{a, pc, chunk, dim3(unsigned((a.T + chunk - 1) / chunk)), st});
  }
  {
    TimedLaunch tl(timer, "balance_seq", st);
    hipLaunchKernelGGL(balance_seq_kernel, dim3(unsigned(a.S)), dim3(kBalThreads), 0, st, a.T, a.E, a.off, chunk, pc,
                       seq_counts, seq_probs, sq);
  }
  {
    TimedLaunch tl(timer, "balance_finish", st);
    hipLaunchKernelGGL(balance_finish_kernel, dim3(1), dim3(kBalThreads), 0, st, a.E, a.k, int(a.S), sq, seq_counts,
                       loss, counts, seq_scale);
  }
  return hipGetLastError();
}

hipError_t launch_balance_bwd(const BalanceArgs& a, const float* w, const float* dw, int renorm,
                              const int32_t* seq_counts, const float* seq_scale, const float* d_loss, float* dz,
                              hipStream_t st, KernelTimer* timer) {
  if (a.T <= 0) return hipSuccess;
  TimedLaunch tl(timer, "balance_bwd", st);
  const int chunk = balance_chunk_tokens(a.T);
  with_layout(a.E, BwdLaunch{a, w, dw, renorm, seq_counts, seq_scale, d_loss, dz, chunk,
                             dim3(unsigned((a.T + chunk - 1) / chunk)), st});
  return hipGetLastError();
}

}  // namespace moe
