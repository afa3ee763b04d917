// Choice of experts by softmax or sigmoid scores with a bias for balance, groups
// and a token mask, and its gradient (include/moe.h: moe_gate, moe_gate_bwd; the
// router is outside the pages' layer, ic.work analysis, section on idealised
// assumptions).
//
// What the choice goes by is a value of 64 bits, so that ids do not depend on how an exp
// rounds. Two ways lead there:
//   k <= 16 (and groups that end where lanes do): several tokens a wave, fp32 scores as
//   integer keys, and 64 bits only where keys are too close ("the quick way" below).
//   16,384 tokens of 128 experts, k = 8, sigmoid and bias: 7.4 us, of which 2.7 are a
//   launch; 131,072 of 256 in 8 groups: 54 to 65 us (134 MB; the memory's time is 29). Its
//   vector instructions take 46 of them, 835 for four tokens of 256 experts: two
//   transcendentals an expert, the keys, the lanes' sorts (108), nine rounds of 17; the rest
//   is waiting that 2.3 waves a SIMD do not cover.
//   Rows of equal keys (logits all alike) are all taken again: 48 and 819 us.
//   Otherwise: one wave per token, lane l at the experts l + 64 i (E <= 1024: at most 16 a
//   lane; instantiated for 2, 4 and 16), everything in 64 bits, experts taken one at a time
//   by a wave-wide arg-max. The same sizes in this way: 41 and 601 us; 131,072 tokens of 160
//   experts in 8 groups of 20, k = 6: 413.
// Weights come from the chosen logits in fp32 in the quick way (1e-7 of a row's largest) and
// in 64 bits in the other: both within 1e-5, and ids are the same in both.
// The gradient for k <= 16 puts rows together in LDS and is bound by memory: 100,007
// tokens of 60 experts through a whole softmax 11.9 us (51 MB at 4.3 TB/s; 39.9 with a wave
// a token), 16,384 of 128 5.2 us (14.6).
#include "device_common.h"
#include "kernels.h"

namespace moe {
namespace gate {

constexpr int kWaves = 4;

__device__ __forceinline__ float wave_maxf(float v) {
  for (int off = 32; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off));
  return v;
}
__device__ __forceinline__ float wave_sumf(float v) {
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
  return v;
}
__device__ __forceinline__ double wave_sumd(double v) {
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
  return v;
}
__device__ __forceinline__ double wave_maxd(double v) {
  for (int off = 32; off > 0; off >>= 1) v = fmax(v, __shfl_xor(v, off));
  return v;
}
// (v, id) of the largest v, ties to the smaller id, in every lane
__device__ __forceinline__ void wave_argmaxd(double& v, int& id) {
  for (int off = 32; off > 0; off >>= 1) {
    const double ov = __shfl_xor(v, off);
    const int oi = __shfl_xor(id, off);
    if (ov > v || (ov == v && oi < id)) {
      v = ov;
      id = oi;
    }
  }
}

// 1 / (1 + e^-x), 0 of -inf
__device__ __forceinline__ double sigmoid64(float x) {
  const double q = exp(-fabs(double(x)));
  return x == -INFINITY ? 0.0 : (x >= 0.f ? 1.0 : q) / (1.0 + q);
}

// The wave's token in 64 bits throughout: writes its k ids and weights. SLOTS: k / 64,
// rounded up (as PER is for E).
template <int PER, int SLOTS>
__device__ __forceinline__ void choose_token(const GateArgs& a, int64_t t, int32_t* __restrict__ idx,
                                             float* __restrict__ w) {
  const int lane = lane_id(), E = a.E, k = a.k;
  const float* __restrict__ z = a.logits + t * E;
  int32_t* __restrict__ oi = idx + t * k;
  float* __restrict__ ow = w + t * k;
  if (a.mask && a.mask[t] == 0) {
    for (int j = lane; j < k; j += 64) {
      oi[j] = -1;
      ow[j] = 0.f;
    }
    return;
  }
  const double kOff = -__builtin_inf();
  double c[PER];
  float zv[PER];
  bool bad = false;
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 64 * i;
    zv[i] = e < E ? z[e] : -INFINITY;
    const float b = e < E && a.bias ? a.bias[e] : 0.f;
    // also true of NaN
    bad |= !(zv[i] < INFINITY) || !(b < INFINITY);
    m = fmaxf(m, zv[i]);
    c[i] = b;
  }
  if (__any(bad)) {
    for (int j = lane; j < k; j += 64) {
      oi[j] = j;
      ow[j] = __builtin_nanf("");
    }
    return;
  }
  m = wave_maxf(m);
  double sum = 1.0;
  // s of a logit (0 of -inf); computed where it is needed, which takes fewer registers
  auto score = [&](float x) {
    if (x == -INFINITY) return 0.0;
    return a.sigmoid ? sigmoid64(x) : exp(double(x) - double(m)) / sum;
  };
  if (!a.sigmoid) {
    double part = 0.0;
#pragma unroll
    for (int i = 0; i < PER; ++i) part += score(zv[i]);
    sum = wave_sumd(part);
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const double b = c[i];
    const bool live = zv[i] > -INFINITY && b > kOff;
    c[i] = !live ? kOff : (a.bias ? score(zv[i]) + b : double(zv[i]));
  }
  // what groups are compared by
  auto by = [&](int i) { return a.bias || a.group_top == 1 || !(c[i] > kOff) ? c[i] : score(zv[i]); };
  if (a.groups > 1) {
    const int gs = E / a.groups;
    double mine = kOff;  // lane g: the score of group g
    for (int g = 0; g < a.groups; ++g) {
      double v = kOff;
      int id = 0x7fffffff;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int e = lane + 64 * i;
        if (e >= g * gs && e < (g + 1) * gs) {
          const double x = by(i);
          if (x > v || (x == v && e < id)) {
            v = x;
            id = e;
          }
        }
      }
      wave_argmaxd(v, id);
      double score = v;
      if (a.group_top == 2) {
        double u = kOff;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int e = lane + 64 * i;
          if (e >= g * gs && e < (g + 1) * gs && e != id) u = fmax(u, by(i));
        }
        u = wave_maxd(u);
        if (u > kOff) score += u;
      }
      if (lane == g) mine = score;
    }
    int ahead = 0;  // groups before this lane's
    for (int g = 0; g < a.groups; ++g) {
      const double o = __shfl(mine, g);
      ahead += (o > mine || (o == mine && g < lane)) ? 1 : 0;
    }
    const uint64_t kept = __ballot(lane < a.groups && ahead < a.groups_kept);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane + 64 * i;
      if (e < E && !((kept >> (e / gs)) & 1)) c[i] = kOff;
    }
  }
  // slot j is kept by lane j % 64 in its register j / 64
  int sel[SLOTS];
  double ss[SLOTS];
  float sz[SLOTS];
  int found = 0;
  float top = -INFINITY;  // the largest logit chosen
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) {
    sel[i] = -1;
    ss[i] = 0.0;
    sz[i] = -INFINITY;
  }
  for (int j = 0; j < k; ++j) {
    double v = kOff;
    int id = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane + 64 * i;
      if (c[i] > v) {
        v = c[i];
        id = e;
      }
    }
    wave_argmaxd(v, id);
    if (!(v > kOff)) break;  // the same in every lane
    float ez = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (id == lane + 64 * i) {
        c[i] = kOff;
        ez = zv[i];
      }
    ez = __shfl(ez, id & 63);
#pragma unroll
    for (int i = 0; i < SLOTS; ++i)
      if (j == lane + 64 * i) {
        sel[i] = id;
        sz[i] = ez;
      }
    top = fmaxf(top, ez);
    found = j + 1;
  }
  if (a.renorm) {
    // the chosen scores over the largest of them, which every factor common to
    // them leaves: exp(z - top), or for sigmoids (1 / (1 + e^-z)) / e^min(top, 0)
    const double ref = a.sigmoid ? fmin(double(top), 0.0) : double(top);
    double d = 0.0;
#pragma unroll
    for (int i = 0; i < SLOTS; ++i)
      if (lane + 64 * i < found) {
        const double x = sz[i];
        ss[i] = !a.sigmoid ? exp(x - ref) : (x >= 0 ? 1.0 / (1.0 + exp(-x)) : exp(x - ref) / (1.0 + exp(x)));
        d += ss[i];
      }
    d = wave_sumd(d);
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) ss[i] = lane + 64 * i < found ? ss[i] / d : 0.0;
  } else {
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) ss[i] = score(sz[i]);
  }
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) {
    const int j = lane + 64 * i;
    if (j < k) {
      oi[j] = sel[i];
      ow[j] = float(double(a.scale) * ss[i]);
    }
  }
}

template <int PER>
__global__ __launch_bounds__(64 * kWaves) void choose_kernel(GateArgs a, int32_t* __restrict__ idx,
                                                             float* __restrict__ w) {
  const int64_t t = int64_t(blockIdx.x) * kWaves + (threadIdx.x >> 6);
  if (t >= a.T) return;  // the whole wave
  choose_token<PER, PER>(a, t, idx, w);
}

// ------------------------------------------------------------------ the quick way
// k <= 16: LPT lanes a token (64 / LPT tokens a wave), V neighbouring experts a lane. What
// the choice goes by is computed in fp32 with a known bound on its error and turned into
// integers: a fixed-point number of its distance from the row's largest (up to 24 bits
// over the row's range) above the expert's id, so that keys are different, their order
// needs no second comparison, and a lane sorts its own with min and max. A round of the
// choice takes the largest of the lanes' first keys (DPP) and moves its lane's list up.
// Where two keys of the choice are closer than twice the error, what they stand for is
// computed in 64 bits and put in order (softmax scores with a bias need the whole row for
// that); where that does not settle it, where groups are too close, where something is
// not finite and where a group has too few experts, the wave takes the token again in 64
// bits. The ids are those of 64 bits always. Logits themselves (no bias) map to keys in
// their order, so there only equal keys are too close. (About one token in 1,500 of 128
// experts has close keys; the whole token in 64 bits holds its wave up for 5 us.)

typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t umin(uint32_t a, uint32_t b) { return a < b ? a : b; }

// the value of the lane that a butterfly over groups of W lanes meets
template <int W>
__device__ __forceinline__ uint32_t meet(uint32_t v) {
  if constexpr (W == 2) return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0xB1, 15, 15, true));
  if constexpr (W == 4) return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x4E, 15, 15, true));
  if constexpr (W == 8) return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x141, 15, 15, true));
  if constexpr (W == 16) return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x140, 15, 15, true));
  return 0;
}
// op over the LPT lanes of a token (16, 32 or 64), in every one of them
template <int LPT, class Op>
__device__ __forceinline__ uint32_t over(uint32_t v, Op op) {
  v = op(v, meet<2>(v));
  v = op(v, meet<4>(v));
  v = op(v, meet<8>(v));
  v = op(v, meet<16>(v));
  if constexpr (LPT >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = op(r[0], r[1]);
  }
  if constexpr (LPT >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = op(r[0], r[1]);
  }
  return v;
}
template <int LPT>
__device__ __forceinline__ float over_max(float v) {
  return __uint_as_float(over<LPT>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
template <int LPT>
__device__ __forceinline__ float over_sum(float v) {
  return __uint_as_float(over<LPT>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
template <int LPT>
__device__ __forceinline__ uint32_t over_umax(uint32_t v) {
  return over<LPT>(v, [](uint32_t a, uint32_t b) { return umax(a, b); });
}

// Descending, by Batcher's odd-even merging (63 comparisons of 16). Every index is a
// template's: as loops the compiler left some of them, and indexed registers by selects.
template <int A, int B, int V>
__device__ __forceinline__ void in_order(uint32_t (&s)[V]) {
  const uint32_t a = s[A], b = s[B];
  s[A] = umax(a, b);
  s[B] = umin(a, b);
}
template <int LO, int N, int R, int I, int V>  // comparisons of I, I + 2 R, ... with their R-th next
__device__ __forceinline__ void merge_pairs(uint32_t (&s)[V]) {
  if constexpr (I + R < LO + N) {
    in_order<I, I + R>(s);
    merge_pairs<LO, N, R, I + 2 * R>(s);
  }
}
template <int LO, int N, int R, int V>  // every R-th of N from LO on: two sorted halves into one
__device__ __forceinline__ void merge_halves(uint32_t (&s)[V]) {
  if constexpr (2 * R < N) {
    merge_halves<LO, N, 2 * R>(s);
    merge_halves<LO + R, N, 2 * R>(s);
    merge_pairs<LO, N, R, LO + R>(s);
  } else {
    in_order<LO, LO + R>(s);
  }
}
template <int LO, int N, int V>
__device__ __forceinline__ void sort_down(uint32_t (&s)[V]) {
  if constexpr (N > 1) {
    sort_down<LO, N / 2>(s);
    sort_down<LO + N / 2, N / 2>(s);
    merge_halves<LO, N, 1>(s);
  }
}

template <int LO, int H, int I, int V>
__device__ __forceinline__ void halve(uint32_t (&s)[V]) {
  if constexpr (I < H) {
    in_order<LO + I, LO + I + H>(s);
    halve<LO, H, I + 1>(s);
  }
}
template <int LO, int N, int V>
__device__ __forceinline__ void bitonic_down(uint32_t (&s)[V]) {
  if constexpr (N > 1) {
    halve<LO, N / 2, 0>(s);
    bitonic_down<LO, N / 2>(s);
    bitonic_down<LO + N / 2, N / 2>(s);
  }
}

// The D largest of V in front, descending: both halves sorted, the larger of each pair
// (the i-th largest of one, the i-th smallest of the other's D) and those in order again.
template <int D, int V>
__device__ __forceinline__ void largest_down(uint32_t (&s)[V]) {
  if constexpr (D == V) {
    sort_down<0, V>(s);
  } else {
    static_assert(2 * D == V, "halves");
    sort_down<0, D>(s);
    sort_down<D, D>(s);
#pragma unroll
    for (int i = 0; i < D; ++i) s[i] = umax(s[i], s[V - 1 - i]);
    if constexpr (D > 4) bitonic_down<0, D>(s);
    else sort_down<0, D>(s);
  }
}

template <int V>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int e0, int E, bool there, float (&z)[V]) {
  if (there && e0 + V <= E && V >= 4) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const f32x4 x = *reinterpret_cast<const f32x4u*>(row + e0 + i);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < V) z[i + j] = x[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) z[i] = there && e0 + i < E ? row[e0 + i] : -INFINITY;
  }
}

constexpr float kLog2e = 1.4426950408889634f;

// e^x to two units, x <= 0 (0 below the normal range): 2^t on the transcendental unit, and
// what t = x log2(e) lost in its rounding made good.
__device__ __forceinline__ float power(float x) {
  const float t = fmaxf(x, -200.f) * kLog2e;
  const float r = fmaf(fmaxf(x, -200.f), kLog2e, -t) + x * 1.925963033500912e-8f;
  const float p = __builtin_amdgcn_exp2f(t);
  return x >= -200.f ? fmaf(p, r * 0.6931471805599453f, p) : 0.f;
}
constexpr float kWindow = 16.f;  // of a row's range that keys resolve at most

// SLOW: PER of the path in 64 bits. D: keys of a lane that are kept in order (k <= D, or
// all of them). batches: of 64 / LPT tokens a wave takes. lanes_group: lanes of a group.
template <int LPT, int V, int D, int SLOW>
__global__ __launch_bounds__(64 * kWaves, SLOW <= 2 ? 5 : SLOW <= 4 ? 4 : 2) void choose_quick_kernel(GateArgs a, int batches, int lanes_group,
                                                                   int32_t* __restrict__ idx, float* __restrict__ w) {
  constexpr int TPW = 64 / LPT;
  constexpr int IB = LPT * V == 1024 ? 10 : LPT * V == 512 ? 9 : LPT * V == 256 ? 8 : LPT * V == 128 ? 7
                   : LPT * V == 64 ? 6 : LPT * V == 32 ? 5 : 4;
  static_assert((1 << IB) == LPT * V, "ids fill their bits");
  constexpr int KB = 32 - IB < 24 ? 32 - IB : 24;
  constexpr float kTop = float((1 << KB) - 1);
  const int lane = lane_id(), l = lane % LPT, E = a.E, k = a.k, e0 = l * V;
  const int64_t wave = int64_t(blockIdx.x) * kWaves + (threadIdx.x >> 6);
  const int64_t first = wave * batches * TPW;
  if (first >= a.T) return;  // the whole wave
  float bias[V];
  bool bad_bias = false;
  load_row<V>(a.bias, e0, E, a.bias != nullptr, bias);
#pragma unroll
  for (int i = 0; i < V; ++i) bad_bias |= !(bias[i] < INFINITY);
  const bool spoilt = __any(bad_bias);
  const bool few = (a.sigmoid || !a.bias) && k < 16;  // close keys are told apart by themselves
  float c[V], zn[V];  // a batch's logits, then what the choice goes by; the next one's logits
  bool live_token, next_live;  // there, and not masked
  auto fetch = [&](int64_t t0, float (&x)[V], bool& live) {
    const int64_t t = t0 + lane / LPT;
    live = t < a.T && (!a.mask || a.mask[t] != 0);
    // a masked row is read and not used: no load waits for the mask
    load_row<V>(a.logits + t * E, e0, E, t < a.T, x);
  };
  uint64_t todo = 0;  // lane n: the lanes of batch n whose tokens are taken again
  fetch(first, zn, next_live);
  for (int n = 0; n < batches; ++n) {
    const int64_t t0 = first + int64_t(n) * TPW, t = t0 + lane / LPT;
    if (t0 >= a.T) break;
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = zn[i];
    live_token = next_live;
    if (n + 1 < batches && t0 + TPW < a.T) fetch(t0 + TPW, zn, next_live);

    // an infinity or a NaN anywhere shows in the sum
    bool odd = spoilt;
    float total = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) total += c[i];
    uint32_t off = 0u;  // experts that are off
    const bool uneven = __any(!(fabsf(total) < INFINITY));
    if (uneven) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        odd |= !(c[i] < INFINITY);
        off |= c[i] == -INFINITY ? 1u << i : 0u;
      }
    }
    float zt = -INFINITY, sum = 0.f;  // the row's maximum, sum of exp(z - zt)
    float error = 0.f;                // of what the choice goes by
    if (!a.sigmoid && (a.bias || !a.renorm)) {
#pragma unroll
      for (int i = 0; i < V; ++i) zt = fmaxf(zt, c[i]);
      zt = over_max<LPT>(zt);
      float q[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        q[i] = __builtin_amdgcn_exp2f((c[i] - zt) * kLog2e);
        if (uneven && c[i] == -INFINITY) q[i] = 0.f;
        sum += q[i];
      }
      sum = over_sum<LPT>(sum);
      if (a.bias) {
        const float inv = __builtin_amdgcn_rcpf(sum);
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] = q[i] * inv + bias[i];
        // each power's argument and value, 22 sums, their weighted share of the arguments'
        // errors: below 64 units of 2^-24 of the largest probability
        error = 0x1p-18f * inv;
      }
    } else if (a.bias) {
      // s (1 - s) (|z| 1.5 + 2) of the power, s of the sum, 2 s of the reciprocal: below
      // 4 units of 2^-24
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * c[i])) + bias[i];
      error = 0x1p-22f;
    }
    if (uneven) {
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = off >> i & 1u ? -INFINITY : c[i];
    }
    // Keys resolve twice the distance from the row's largest to the least of the lanes'
    // largest, so LPT experts at least; what is below has the key 0.
    float top = c[0];
#pragma unroll
    for (int i = 1; i < V; ++i) top = fmaxf(top, c[i]);
    const float least = -over_max<LPT>(top > -INFINITY ? -top : -INFINITY);  // of live lanes
    top = over_max<LPT>(top);
    const float window = fminf(2.f * (top - least), kWindow);
    float scale = (kTop - 2.f) * __builtin_amdgcn_rcpf(window);
    if (!(window > 0.f && scale < 1e30f)) scale = 1.f;  // equal ones have equal keys, and are taken again
    if (a.bias) error += 0x1p-23f * (fabsf(top) + window);
    const float close = a.bias ? 2.f * error * scale + 1.f : 0.f;
    odd |= !(close < 0x1p+22f);
    const uint32_t near = uint32_t(fminf(close, 0x1p+22f));
    // (the shift is rounded alike for all; where it is off by much the first keys meet at the
    // top and are taken again)
    const float shift = fmaf(-top, scale, kTop);
    uint32_t s[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float h = __builtin_amdgcn_fmed3f(fmaf(c[i], scale, shift), 0.f, kTop);
      s[i] = (uint32_t(h) << IB) | uint32_t(V - 1 - i);
    }
    largest_down<D>(s);
    // the id's other bits, which the lane's experts share
#pragma unroll
    for (int i = 0; i < D; ++i) s[i] |= uint32_t((LPT - 1 - l) * V);

    if (a.groups > 1) {
      // the group's two largest keys in each of its lanes
      uint32_t g0 = s[0], g1 = V > 1 ? s[V > 1 ? 1 : 0] : 0u;
      auto join = [&](uint32_t b0, uint32_t b1) {
        g1 = umax(umin(g0, b0), umax(g1, b1));
        g0 = umax(g0, b0);
      };
      if (lanes_group >= 2) join(meet<2>(g0), meet<2>(g1));
      if (lanes_group >= 4) join(meet<4>(g0), meet<4>(g1));
      if (lanes_group >= 8) join(meet<8>(g0), meet<8>(g1));
      if (lanes_group >= 16) join(meet<16>(g0), meet<16>(g1));
      const uint32_t group = uint32_t(l / lanes_group);
      uint32_t score = g0 >> IB;
      uint32_t far = near;
      if (a.group_top == 2) {
        // a sum needs both of its keys: none below the window or off
        odd |= e0 < E && (g1 >> IB) == 0u;
        score += g1 >> IB;
        far = 2u * near + 4u;
      }
      score = score ? (score << 6) | (63u - group) : 0u;
      uint32_t last = 0u;
      uint32_t kept = 0u;
      for (int r = 0; r <= a.groups_kept; ++r) {
        const uint32_t m = over_umax<LPT>(score);
        if (r == a.groups_kept) {  // the best group that is left out
          odd |= r < a.groups && (last >> 6) - (m >> 6) <= far;
        } else {
          odd |= m == 0u;  // a group with nothing above the window
          const uint32_t hit = score == m ? ~0u : 0u;
          kept |= hit;
          score &= ~hit;
        }
        last = m;
      }
#pragma unroll
      for (int i = 0; i < D; ++i) s[i] &= kept;
    }

    // the k largest keys, key j in lane j; and the next one
    uint32_t mine = 0u, next = 0u, won = 0u;
    for (int j = 0; j <= k; ++j) {
      const uint32_t m = over_umax<LPT>(s[0]);
      mine = l == j ? m : mine;
      next = m;
      // by masks: a choice between two elements becomes an index the compiler cannot resolve
      const uint32_t win = s[0] == m ? ~0u : 0u;
#pragma unroll
      for (int i = 0; i + 1 < D; ++i) s[i] = (s[i + 1] & win) | (s[i] & ~win);
      s[D - 1] &= ~win;
      won -= win;
    }
    if (D < V) odd |= won >= uint32_t(D);  // the lane had more than its list held
    // lane j's follower: key j + 1
    uint32_t follow = uint32_t(__builtin_amdgcn_update_dpp(0, int(mine), 0x101, 15, 15, true));  // row_shl:1
    if (l == k - 1) follow = next;
    // (a key of 0 where one is wanted: all that is left is off, or below the window)
    const uint32_t hm = mine >> IB, hf = follow >> IB;
    bool tight = l < k && hm - hf <= near;
    odd |= tight && (!few || hf == 0u);
    tight &= few && live_token;
    if (__any(tight)) {
      // Whatever else there is is below these k keys, or below the next one too where that is
      // as close: their order in 64 bits is all that is missing.
      const uint32_t after = over_umax<LPT>(s[0]);
      odd |= tight && l == k - 1 && (next >> IB) - (after >> IB) <= near;
      const int base = lane & ~(LPT - 1);
      const uint32_t key = l == k ? next : mine;
      const int id = LPT * V - 1 - int(key & uint32_t(LPT * V - 1));
      double value = -__builtin_inf();
      if (l <= k && (key >> IB) != 0u) {
        const float x = a.logits[t * E + id];
        value = a.bias ? sigmoid64(x) + double(a.bias[id]) : double(x);
      }
      int rank = 0;
      for (int j = 0; j <= k; ++j) {
        const double o = __shfl(value, base + j);
        const int oi = __shfl(id, base + j);
        rank += o > value || (o == value && oi < id) ? 1 : 0;
      }
      int from = l;
      for (int j = 0; j <= k; ++j)
        if (__shfl(l <= k ? rank : -1, base + j) == l) from = j;
      const uint32_t sorted = __shfl(key, base + from);
      const uint64_t mark = __ballot(tight) >> base;
      if (l < k && (LPT == 64 ? mark : mark & ((uint64_t(1) << (LPT & 63)) - 1)) != 0) mine = sorted;
    }

    const int e = LPT * V - 1 - int(mine & uint32_t(LPT * V - 1));
    const bool some = l < k && (mine >> IB) != 0u;
    const float x = some ? a.logits[t * E + e] : -INFINITY;
    float v = 0.f;
    if (!a.sigmoid) {
      if (a.renorm) zt = over_max<LPT>(x);
      if (some) v = power(x - zt);
      if (a.renorm) sum = over_sum<LPT>(v);
    } else {
      const float q = power(-fabsf(x));
      v = (x >= 0.f ? 1.f : q) * __builtin_amdgcn_rcpf(1.f + q);
      if (a.renorm) {
        // scores below e^ref, all of them, in units of it
        const float ref = over_max<LPT>(x);
        if (__any(ref < 0.f)) v = ref < 0.f ? power(x - ref) * __builtin_amdgcn_rcpf(1.f + q) : v;
        v = some ? v : 0.f;
        sum = over_sum<LPT>(v);
      }
    }
    if (a.renorm || !a.sigmoid) v *= __builtin_amdgcn_rcpf(sum);
    const uint64_t again = __ballot(odd && live_token);
    const uint64_t own = LPT == 64 ? ~uint64_t(0) : ((uint64_t(1) << (LPT & 63)) - 1) << (lane / LPT * (LPT & 63));
    if (t < a.T && l < k && !(again & own)) {
      idx[t * k + l] = live_token ? e : -1;
      w[t * k + l] = live_token ? a.scale * v : 0.f;
    }
    if (lane == n) todo = again;
  }
  // after the batches, so that their registers are free
  if (!__any(todo != 0)) return;
#pragma unroll 1
  for (int n = 0; n < batches; ++n) {
    const uint64_t again = __shfl(todo, n);
#pragma unroll 1
    for (int q = 0; q < TPW; ++q)
      if ((again >> (q * (LPT & 63))) & (LPT == 64 ? ~uint64_t(0) : (uint64_t(1) << (LPT & 63)) - 1))
        choose_token<SLOW, 1>(a, first + int64_t(n) * TPW + q, idx, w);
  }
}

// Lanes of a group in the quick way, or 0 where it does not serve: the groups' ends are
// lanes' ends, two, four, ... of them; without a bias groups compared by sums of scores
// and experts by logits would take two kinds of keys.
int quick_group_lanes(const GateArgs& a, int V) {
  if (a.k > 16) return 0;
  if (a.groups == 1) return 1;
  if (!a.bias && a.group_top == 2) return 0;
  const int gs = a.E / a.groups;
  if (gs % V != 0) return 0;
  const int n = gs / V;
  return n <= 16 && (n & (n - 1)) == 0 ? n : 0;
}

template <int LPT, int V, int D, int SLOW>
bool launch_quick(const GateArgs& a, int32_t* idx, float* w, hipStream_t st) {
  const int lanes = quick_group_lanes(a, V);
  if (lanes == 0) return false;
  constexpr int TPW = 64 / LPT;
  // several batches a wave where there are many: the next one's logits come meanwhile
  // (262,144 x 64 35.8 us with two, 40.8 with one, 37.7 with eight; 65,536 x 128 17.2, 17.3, 23.3)
  const int64_t waves = (a.T + TPW - 1) / TPW;
  const int batches = int(waves >= 16384 ? 2 : 1);
  const int64_t blocks = (waves + int64_t(batches) * kWaves - 1) / (int64_t(batches) * kWaves);
  hipLaunchKernelGGL((choose_quick_kernel<LPT, V, D, SLOW>), dim3(unsigned(blocks)), dim3(64 * kWaves), 0, st, a,
                     batches, lanes, idx, w);
  return true;
}

bool launch_quick(const GateArgs& a, int32_t* idx, float* w, hipStream_t st) {
  if (a.E <= 16) return launch_quick<16, 1, 1, 1>(a, idx, w, st);
  if (a.E <= 32) return launch_quick<16, 2, 2, 1>(a, idx, w, st);
  if (a.E <= 64) return launch_quick<16, 4, 4, 1>(a, idx, w, st);
  if (a.E <= 128) return launch_quick<16, 8, 8, 2>(a, idx, w, st);
  if (a.k <= 8) {
    if (a.E <= 256) return launch_quick<16, 16, 8, 4>(a, idx, w, st);
    if (a.E <= 512) return launch_quick<32, 16, 8, 8>(a, idx, w, st);
    return launch_quick<64, 16, 8, 16>(a, idx, w, st);
  }
  if (a.E <= 256) return launch_quick<16, 16, 16, 4>(a, idx, w, st);
  if (a.E <= 512) return launch_quick<32, 16, 16, 8>(a, idx, w, st);
  return launch_quick<64, 16, 16, 16>(a, idx, w, st);
}

// The gradient of one token (one wave): slot j's value goes to the lane of its
// expert, slots in their order, so an expert named twice takes both.
template <int PER>
__global__ __launch_bounds__(64 * kWaves) void bwd_kernel(GateArgs a, const int32_t* __restrict__ idx,
                                                          const float* __restrict__ dw, int accumulate,
                                                          float* __restrict__ dz) {
  const int64_t t = int64_t(blockIdx.x) * kWaves + (threadIdx.x >> 6);
  if (t >= a.T) return;
  const int lane = lane_id(), E = a.E, k = a.k;
  const float* __restrict__ z = a.logits + t * E;
  const bool dense = !a.sigmoid && !a.renorm;
  float g[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) g[i] = 0.f;
  float top = -INFINITY, total = 0.f, pd = 0.f;
  auto expert = [&](int j) {
    const int e = j < k ? idx[t * k + j] : -1;
    return e < E ? e : -1;
  };
  // a chosen expert's score over what the renormalisation divides out
  auto score = [&](float x, float ref) {
    if (!a.sigmoid) return expf(x - ref);
    return x >= 0.f ? 1.f / (1.f + expf(-x)) : expf(x - ref) / (1.f + expf(x));
  };
  float ref = 0.f;
  if (a.renorm) {
    for (int j0 = 0; j0 < k; j0 += 64) {
      const int e = expert(j0 + lane);
      if (e >= 0) top = fmaxf(top, z[e]);
    }
    top = wave_maxf(top);
    ref = a.sigmoid ? fminf(top, 0.f) : top;
    for (int j0 = 0; j0 < k; j0 += 64) {
      const int j = j0 + lane, e = expert(j);
      if (e >= 0 && z[e] != -INFINITY) {
        const float v = score(z[e], ref);
        total += v;
        pd += v * dw[t * k + j];
      }
    }
    total = wave_sumf(total);
    pd = wave_sumf(pd) / total;
  }
  bool some = false;
  for (int j0 = 0; j0 < k; j0 += 64) {
    const int j = j0 + lane, ej = expert(j);
    some |= ej >= 0;
    float val = 0.f;
    if (ej >= 0 && (dense || z[ej] != -INFINITY)) {
      const float d = dw[t * k + j], x = z[ej];
      if (dense) {
        val = d;
      } else {
        const float p = a.renorm ? score(x, ref) / total : score(x, 0.f);
        const float slope = a.sigmoid ? (x >= 0.f ? expf(-x) / (1.f + expf(-x)) : 1.f / (1.f + expf(x))) : 1.f;
        val = p * slope * (d - pd);
      }
    }
    const int n = min(64, k - j0);
    for (int q = 0; q < n; ++q) {
      const int e = __shfl(ej, q);
      const float v = __shfl(val, q);
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (e == lane + 64 * i) g[i] += v;
    }
  }
  if (dense) {
    float v[PER];
    float m = -INFINITY, sum = 0.f, pg = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      v[i] = lane + 64 * i < E ? z[lane + 64 * i] : -INFINITY;
      m = fmaxf(m, v[i]);
    }
    m = wave_maxf(m);
    const bool none = !__any(some);  // no choice, no gradient, whatever the logits are
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      // a row of -inf alone has no probabilities; a NaN stays one
      v[i] = none || v[i] == -INFINITY ? 0.f : expf(v[i] - m);
      sum += v[i];
      pg += v[i] * g[i];
    }
    sum = wave_sumf(sum);
    pg = wave_sumf(pg) / sum;
#pragma unroll
    for (int i = 0; i < PER; ++i) g[i] = v[i] == 0.f ? 0.f : v[i] / sum * (g[i] - pg);
  }
  float* out = dz + t * E;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 64 * i;
    if (e < E) out[e] = accumulate ? out[e] + a.scale * g[i] : a.scale * g[i];
  }
}

// ------------------------------------------------------------------ the quick way back
// k <= 16, LPT lanes a token as above, slot j in lane j. The row is put together in LDS:
// zeros, the slots' values at their experts (one after the other only where an expert is
// named twice), and for the dense form p (G - <p, G>) with lane l at the experts l + LPT i;
// then a wave's rows, which lie one after the other in memory, leave as one run.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

template <int LPT, int V, bool DENSE>
__global__ __launch_bounds__(64 * kWaves) void bwd_quick_kernel(GateArgs a, const int32_t* __restrict__ idx,
                                                                const float* __restrict__ dw, int accumulate,
                                                                float* __restrict__ dz) {
  constexpr int TPW = 64 / LPT;
  __shared__ __attribute__((aligned(16))) float s_rows[kWaves][LPT * V * TPW + 4];
  const int lane = lane_id(), l = lane % LPT, E = a.E, k = a.k;
  const int64_t t0 = (int64_t(blockIdx.x) * kWaves + (threadIdx.x >> 6)) * TPW, t = t0 + lane / LPT;
  if (t0 >= a.T) return;  // the whole wave
  float* rows = s_rows[threadIdx.x >> 6];
  float* row = rows + lane / LPT * E;
  const int n = int(min(int64_t(TPW), a.T - t0)) * E;  // elements of the wave's rows
  const bool slot = l < k && t < a.T;
  int e = slot ? idx[t * k + l] : -1;
  if (e >= E) e = -1;
  const float d = e >= 0 ? dw[t * k + l] : 0.f;
  float p[V];
  float x = 0.f, sum = 0.f;
  if constexpr (DENSE) {
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int o = l + LPT * i;
      p[i] = t < a.T && o < E ? a.logits[t * E + o] : -INFINITY;
      top = fmaxf(top, p[i]);
    }
    top = over_max<LPT>(top);
    // a token without a choice has no gradient, whatever its logits are
    const uint64_t chosen = __ballot(e >= 0) >> (lane & ~(LPT - 1));
    const bool none = (LPT == 64 ? chosen : chosen & ((uint64_t(1) << (LPT & 63)) - 1)) == 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      // a row of -inf alone has no probabilities; a NaN stays one
      p[i] = none || p[i] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((p[i] - top) * kLog2e);
      sum += p[i];
    }
    sum = over_sum<LPT>(sum);
  } else if (e >= 0) {
    x = a.logits[t * E + e];
  }
  for (int i = 4 * lane; i < n; i += 256) *reinterpret_cast<f32x4*>(rows + i) = f32x4{0.f, 0.f, 0.f, 0.f};
  float val = d;
  if constexpr (!DENSE) {
    const bool some = e >= 0 && x != -INFINITY;
    float v = 0.f, slope = 1.f;
    if (a.sigmoid) {
      const float q = power(-fabsf(x)), r = __builtin_amdgcn_rcpf(1.f + q);
      v = (x >= 0.f ? 1.f : q) * r;
      slope = (x >= 0.f ? q : 1.f) * r;
      if (a.renorm) {
        const float ref = over_max<LPT>(some ? x : -INFINITY);
        if (__any(ref < 0.f)) v = ref < 0.f ? power(x - ref) * r : v;
      }
    } else {
      const float top = over_max<LPT>(some ? x : -INFINITY);
      v = power(x - top);
    }
    if (x != x) v = x;
    v = some ? v : 0.f;
    float g = d;
    if (a.renorm) {
      v *= __builtin_amdgcn_rcpf(over_sum<LPT>(v));
      g = d - over_sum<LPT>(some ? v * d : 0.f);
    }
    val = some ? v * slope * g : 0.f;
  }
  // is an expert named twice? Every slot against those behind it, in the token's row of lanes
  bool twice = false;
  for (int j = 1; j < k; ++j) {
    const int o = __shfl(e, (lane & ~(LPT - 1)) + ((l + j) & (LPT - 1)));
    twice |= l + j < k && e >= 0 && o == e;
  }
  wave_sync();
  if (!__any(twice)) {
    if (e >= 0) row[e] = val;
  } else {
    for (int j = 0; j < k; ++j) {
      if (l == j && e >= 0) row[e] += val;
      wave_sync();
    }
  }
  wave_sync();
  if constexpr (DENSE) {
    float g[V];
    float pg = 0.f;
    const float inv = __builtin_amdgcn_rcpf(sum);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int o = l + LPT * i;
      g[i] = o < E ? row[o] : 0.f;
      pg += p[i] * g[i];
    }
    pg = over_sum<LPT>(pg) * inv;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int o = l + LPT * i;
      if (o < E) row[o] = p[i] == 0.f ? 0.f : p[i] * inv * (g[i] - pg);
    }
    wave_sync();
  }
  float* out = dz + t0 * E;
  for (int i = 4 * lane; i < n; i += 256) {
    f32x4 v = *reinterpret_cast<const f32x4*>(rows + i);
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] *= a.scale;
    if (i + 4 <= n) {
      if (accumulate) v += *reinterpret_cast<const f32x4u*>(out + i);
      *reinterpret_cast<f32x4u*>(out + i) = v;
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (i + q < n) out[i + q] = accumulate ? out[i + q] + v[q] : v[q];
    }
  }
}

template <int LPT, int V>
void launch_bwd_quick(const GateArgs& a, const int32_t* idx, const float* dw, int accumulate, float* dz, hipStream_t st) {
  const int64_t per = int64_t(kWaves) * (64 / LPT);
  const dim3 grid(unsigned((a.T + per - 1) / per)), block(64 * kWaves);
  if (!a.sigmoid && !a.renorm)
    hipLaunchKernelGGL((bwd_quick_kernel<LPT, V, true>), grid, block, 0, st, a, idx, dw, accumulate, dz);
  else
    hipLaunchKernelGGL((bwd_quick_kernel<LPT, V, false>), grid, block, 0, st, a, idx, dw, accumulate, dz);
}

}  // namespace gate

hipError_t launch_gate(const GateArgs& a, int32_t* idx, float* w, hipStream_t st, KernelTimer* timer) {
  if (a.T <= 0) return hipSuccess;
  TimedLaunch tl(timer, "gate", st);
  if (gate::launch_quick(a, idx, w, st)) return hipGetLastError();
  const dim3 grid(unsigned((a.T + gate::kWaves - 1) / gate::kWaves)), block(64 * gate::kWaves);
  if (a.E <= 128)
    hipLaunchKernelGGL(gate::choose_kernel<2>, grid, block, 0, st, a, idx, w);
  else if (a.E <= 256)
    hipLaunchKernelGGL(gate::choose_kernel<4>, grid, block, 0, st, a, idx, w);
  else
    hipLaunchKernelGGL(gate::choose_kernel<16>, grid, block, 0, st, a, idx, w);
  return hipGetLastError();
}

hipError_t launch_gate_bwd(const GateArgs& a, const int32_t* idx, const float* dw, int accumulate, float* dz,
                           hipStream_t st, KernelTimer* timer) {
  if (a.T <= 0) return hipSuccess;
  TimedLaunch tl(timer, "gate_bwd", st);
  if (a.k <= 16) {
    if (a.E <= 16) gate::launch_bwd_quick<16, 1>(a, idx, dw, accumulate, dz, st);
    else if (a.E <= 32) gate::launch_bwd_quick<16, 2>(a, idx, dw, accumulate, dz, st);
    else if (a.E <= 64) gate::launch_bwd_quick<16, 4>(a, idx, dw, accumulate, dz, st);
    else if (a.E <= 128) gate::launch_bwd_quick<16, 8>(a, idx, dw, accumulate, dz, st);
    else if (a.E <= 256) gate::launch_bwd_quick<16, 16>(a, idx, dw, accumulate, dz, st);
    else if (a.E <= 512) gate::launch_bwd_quick<32, 16>(a, idx, dw, accumulate, dz, st);
    else gate::launch_bwd_quick<64, 16>(a, idx, dw, accumulate, dz, st);
    return hipGetLastError();
  }
  const dim3 grid(unsigned((a.T + gate::kWaves - 1) / gate::kWaves)), block(64 * gate::kWaves);
  if (a.E <= 128)
    hipLaunchKernelGGL(gate::bwd_kernel<2>, grid, block, 0, st, a, idx, dw, accumulate, dz);
  else if (a.E <= 256)
    hipLaunchKernelGGL(gate::bwd_kernel<4>, grid, block, 0, st, a, idx, dw, accumulate, dz);
  else
    hipLaunchKernelGGL(gate::bwd_kernel<16>, grid, block, 0, st, a, idx, dw, accumulate, dz);
  return hipGetLastError();
}

}  // namespace moe
