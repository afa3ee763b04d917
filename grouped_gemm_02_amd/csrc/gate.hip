// Choice of experts by softmax or sigmoid scores with a bias for balance, groups
// and a token mask, and its gradient (include/moe.h: moe_gate, moe_gate_bwd; the
// router is outside the pages' layer, ic.work analysis, section on idealised
// assumptions).
//
// One wave per token; lane l holds the experts l + 64 i (E <= 1024: at most 16 a
// lane; instantiated for 2, 4 and 16). What the choice goes by is computed and
// compared in 64 bits, so that ids do not depend on how an exp rounds; experts are
// taken one at a time by a wave-wide arg-max.
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

// The wave's token in 64 bits throughout: writes its k ids and weights.
template <int PER>
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
  double c[PER], s[PER];
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
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    s[i] = 0.0;
    if (zv[i] > -INFINITY) {
      const double x = zv[i];
      if (a.sigmoid) {
        const double q = exp(-fabs(x));
        s[i] = (x >= 0 ? 1.0 : q) / (1.0 + q);
      } else {
        s[i] = exp(x - double(m));
      }
    }
    sum += s[i];
  }
  if (!a.sigmoid) {
    sum = wave_sumd(sum);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (zv[i] > -INFINITY) s[i] /= sum;
  }
  double by[PER];  // what groups are compared by
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const double b = c[i];
    const bool live = zv[i] > -INFINITY && b > kOff;
    c[i] = !live ? kOff : (a.bias ? s[i] + b : double(zv[i]));
    by[i] = !live ? kOff : (a.bias ? c[i] : (a.group_top == 2 ? s[i] : double(zv[i])));
  }
  if (a.groups > 1) {
    const int gs = E / a.groups;
    double mine = kOff;  // lane g: the score of group g
    for (int g = 0; g < a.groups; ++g) {
      double v = kOff;
      int id = 0x7fffffff;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int e = lane + 64 * i;
        if (e >= g * gs && e < (g + 1) * gs && (by[i] > v || (by[i] == v && e < id))) {
          v = by[i];
          id = e;
        }
      }
      wave_argmaxd(v, id);
      double score = v;
      if (a.group_top == 2) {
        double u = kOff;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int e = lane + 64 * i;
          if (e >= g * gs && e < (g + 1) * gs && e != id) u = fmax(u, by[i]);
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
  int sel[PER];
  double ss[PER];
  float sz[PER];
  int found = 0;
  float top = -INFINITY;  // the largest logit chosen
#pragma unroll
  for (int i = 0; i < PER; ++i) {
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
    double es = 0.0;
    float ez = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (id == lane + 64 * i) {
        c[i] = kOff;
        es = s[i];
        ez = zv[i];
      }
    es = __shfl(es, id & 63);
    ez = __shfl(ez, id & 63);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (j == lane + 64 * i) {
        sel[i] = id;
        ss[i] = es;
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
    for (int i = 0; i < PER; ++i)
      if (lane + 64 * i < found) {
        const double x = sz[i];
        ss[i] = !a.sigmoid ? exp(x - ref) : (x >= 0 ? 1.0 / (1.0 + exp(-x)) : exp(x - ref) / (1.0 + exp(x)));
        d += ss[i];
      }
    d = wave_sumd(d);
#pragma unroll
    for (int i = 0; i < PER; ++i) ss[i] = lane + 64 * i < found ? ss[i] / d : 0.0;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
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
  choose_token<PER>(a, t, idx, w);
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
  for (int j0 = 0; j0 < k; j0 += 64) {
    const int j = j0 + lane, ej = expert(j);
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
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      // a row of -inf alone has no probabilities; a NaN stays one
      v[i] = v[i] == -INFINITY ? 0.f : expf(v[i] - m);
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

}  // namespace gate

hipError_t launch_gate(const GateArgs& a, int32_t* idx, float* w, hipStream_t st, KernelTimer* timer) {
  if (a.T <= 0) return hipSuccess;
  TimedLaunch tl(timer, "gate", st);
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
