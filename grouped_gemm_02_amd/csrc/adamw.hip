// One AdamW step over many tensors (include/moe.h: moe_adamw_step; the pages end at
// the weight gradients).
//
// Memory alone bounds it: each element's weight, gradient and moments are read and
// written once, with streaming accesses. A launch takes up to kMaxTensors tensors, whose
// addresses are kernel arguments (nothing is copied to the device, and a captured launch
// replays them); a workgroup takes kChunk elements of one tensor, found by bisecting the
// tensors' first chunks. A thread takes eight neighbouring elements and is done: with two
// or four such pieces one after the other the 8-bit step of 604 M bf16 weights took 1.15
// and 1.20 ms instead of 1.06 (now 1.02: 6.05 GB at 5.9 TB/s), 12.6 M fp32 ones 84 and 97 us
// instead of 78. Sixteen threads hold the 128 elements that share a scale where moments are
// held in 8 bits; what is rare there (numbers that are not finite, roots that would round
// to 0) is looked for in all eight at once, as the arithmetic of a piece comes near the
// memory's time (0.84 of 1.2 ms before).
#include <algorithm>

#include "device_common.h"
#include "kernels.h"

namespace moe {
namespace adamw {

constexpr int kThreads = 256;
constexpr int kChunk = 8 * kThreads;  // elements of a workgroup
constexpr int kMaxTensors = 48;
constexpr uint32_t kMaxChunks = uint32_t(1) << 22;  // of a launch, which has less than 2^32 threads

// Vectors at any address of their elements: a tensor begins anywhere.
typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2u __attribute__((ext_vector_type(2), aligned(1)));

struct Batch {
  AdamwHyper h;
  const float* grad_scale;
  const float* hyper;
  int count;
  uint32_t first[kMaxTensors + 1];  // a tensor's first chunk
  AdamwTensor e[kMaxTensors];
};
static_assert(sizeof(Batch) <= 4096, "kernel arguments");

__device__ __forceinline__ void load8(const float* p, int64_t i, float (&x)[8]) {
  const f32x4u* q = reinterpret_cast<const f32x4u*>(p + i);
  const f32x4 a = __builtin_nontemporal_load(q), b = __builtin_nontemporal_load(q + 1);
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    x[t] = a[t];
    x[4 + t] = b[t];
  }
}
__device__ __forceinline__ void load8(const uint16_t* p, int64_t i, float (&x)[8]) {
  const u32x4 a = __builtin_nontemporal_load(reinterpret_cast<const u32x4u*>(p + i));
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    x[2 * t] = bf16_lo(a[t]);
    x[2 * t + 1] = bf16_hi(a[t]);
  }
}
__device__ __forceinline__ void store8(float* p, int64_t i, const float (&x)[8]) {
  f32x4u* q = reinterpret_cast<f32x4u*>(p + i);
  __builtin_nontemporal_store(f32x4{x[0], x[1], x[2], x[3]}, q);
  __builtin_nontemporal_store(f32x4{x[4], x[5], x[6], x[7]}, q + 1);
}
__device__ __forceinline__ void store8(uint16_t* p, int64_t i, const float (&x)[8]) {
  __builtin_nontemporal_store(
      u32x4{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])},
      reinterpret_cast<u32x4u*>(p + i));
}
__device__ __forceinline__ float load1(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float load1(const uint16_t* p, int64_t i) { return __uint_as_float(uint32_t(p[i]) << 16); }
__device__ __forceinline__ void store1(float* p, int64_t i, float x) { p[i] = x; }
__device__ __forceinline__ void store1(uint16_t* p, int64_t i, float x) { p[i] = uint16_t(pack_bf16x2(x, 0.f)); }

// Eight elements from i of n (as many as there are; the others read as zero).
template <class T>
__device__ __forceinline__ void get(const T* p, int64_t i, int64_t n, float (&x)[8]) {
  if (i + 8 <= n) {
    load8(p, i, x);
  } else {
#pragma unroll
    for (int t = 0; t < 8; ++t) x[t] = i + t < n ? load1(p, i + t) : 0.f;
  }
}
template <class T>
__device__ __forceinline__ void put(T* p, int64_t i, int64_t n, const float (&x)[8]) {
  if (i + 8 <= n) {
    store8(p, i, x);
  } else {
#pragma unroll
    for (int t = 0; t < 8; ++t)
      if (i + t < n) store1(p, i + t, x[t]);
  }
}

// Moments in 8 bits: E4M3 codes, scale byte e + 127 per 128 elements (a byte of 0,
// as a cleared buffer has, makes every code 0).
__device__ __forceinline__ void get_codes(const uint8_t* p, const uint8_t* scale, int64_t i, int64_t n, float (&x)[8]) {
  uint32_t lo = 0, hi = 0;
  if (i + 8 <= n) {
    const u32x2 a = __builtin_nontemporal_load(reinterpret_cast<const u32x2u*>(p + i));
    lo = a[0];
    hi = a[1];
  } else {
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const uint32_t b = i + t < n ? p[i + t] : 0;
      if (t < 4) lo |= b << (8 * t); else hi |= b << (8 * t - 32);
    }
  }
  const float s = i < n ? __uint_as_float(uint32_t(scale[i >> 7]) << 23) : 0.f;
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(int(lo), false), b = __builtin_amdgcn_cvt_pk_f32_fp8(int(lo), true);
  const f32x2 c = __builtin_amdgcn_cvt_pk_f32_fp8(int(hi), false), d = __builtin_amdgcn_cvt_pk_f32_fp8(int(hi), true);
  x[0] = a[0] * s; x[1] = a[1] * s; x[2] = b[0] * s; x[3] = b[1] * s;
  x[4] = c[0] * s; x[5] = c[1] * s; x[6] = d[0] * s; x[7] = d[1] * s;
}

__device__ __forceinline__ uint32_t row_umax16(uint32_t v) {
  v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0xB1, 15, 15, true)));
  v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x4E, 15, 15, true)));
  v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x141, 15, 15, true)));
  return max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x140, 15, 15, true)));
}

__device__ __forceinline__ void pack_codes(const float (&y)[8], uint32_t (&c)[2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int a = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * h], y[4 * h + 1], 0, false);
    c[h] = uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(y[4 * h + 2], y[4 * h + 3], a, true));
  }
}

// Every lane of the block's sixteen comes here, those behind the tensor's end with zeros.
// KEEP: x is not negative, and what is above 0 is not held as 0.
template <bool KEEP>
__device__ __forceinline__ void put_codes(uint8_t* p, uint8_t* scale, int64_t i, int64_t n, const float (&x)[8]) {
  // magnitudes in the order of their bits: a NaN is above infinity, infinity above the rest
  uint32_t top = 0;
#pragma unroll
  for (int t = 0; t < 8; ++t) top = max(top, __float_as_uint(x[t]) & 0x7fffffffu);
  uint32_t odd = 0;  // which are not finite: they do not bear on the scale
  if (__any(top >= 0x7f800000u)) {
    top = 0;
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const uint32_t u = __float_as_uint(x[t]) & 0x7fffffffu;
      if (u >= 0x7f800000u) odd |= 1u << t;
      else top = max(top, u);
    }
  }
  top = row_umax16(top);
  // 448 = 1.75 * 2^8
  int e = int(top >> 23) - 135 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = top ? min(max(e, -126), 126) : 0;
  const float inv = __uint_as_float(uint32_t(127 - e) << 23);
  float y[8];
#pragma unroll
  for (int t = 0; t < 8; ++t) y[t] = x[t] * inv;
  if (odd) {
#pragma unroll
    for (int t = 0; t < 8; ++t) y[t] = odd >> t & 1 ? 0.f : y[t];
  }
  uint32_t c[2];
  pack_codes(y, c);
  if constexpr (KEEP) {
    // bytes of 0 (the lowest of them is found whatever is above it)
    const uint32_t zero = (((c[0] - 0x01010101u) & ~c[0]) | ((c[1] - 0x01010101u) & ~c[1])) & 0x80808080u;
    if (__any(zero != 0)) {
#pragma unroll
      for (int t = 0; t < 8; ++t) y[t] = x[t] > 0.f && y[t] < 0x1p-9f ? 0x1p-9f : y[t];
      pack_codes(y, c);
    }
  }
  if (odd) {
#pragma unroll
    for (int t = 0; t < 8; ++t)
      if (odd >> t & 1) c[t / 4] |= 0x7fu << (8 * (t & 3));
  }
  if (i + 8 <= n) {
    __builtin_nontemporal_store(u32x2{c[0], c[1]}, reinterpret_cast<u32x2u*>(p + i));
  } else {
#pragma unroll
    for (int t = 0; t < 8; ++t)
      if (i + t < n) p[i + t] = uint8_t(c[t / 4] >> (8 * (t & 3)));
  }
  if ((i & 127) == 0 && i < n) scale[i >> 7] = uint8_t(e + 127);
}

// Square roots to one unit in the last place, of numbers below the normal range too (which
// the instruction takes for zero).
__device__ __forceinline__ void roots(const float (&v)[8], float (&r)[8]) {
  uint32_t least = ~0u;  // 0 wraps to the top and is no reason
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    r[t] = __builtin_amdgcn_sqrtf(v[t]);
    least = min(least, __float_as_uint(v[t]) - 1u);
  }
  if (__any(least < 0x0f800000u)) {  // 2^-96
#pragma unroll
    for (int t = 0; t < 8; ++t)
      if (v[t] < 0x1p-96f) r[t] = __builtin_amdgcn_sqrtf(v[t] * 0x1p+64f) * 0x1p-32f;
  }
}

template <class PT, class GT, bool EIGHT, bool MASTER>
__global__ __launch_bounds__(kThreads) void step_kernel(const Batch b) {
#pragma clang fp contract(off)
  int lo = 0, hi = b.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (b.first[mid] <= blockIdx.x) lo = mid; else hi = mid;
  }
  const AdamwTensor& en = b.e[lo];
  const int64_t n = en.n;
  float lr = b.h.lr, bias1 = b.h.bias1, root2 = b.h.root2, gs = 1.f;
  if (b.hyper) {
    lr = b.hyper[0];
    bias1 = b.hyper[1];
    root2 = 1.f / sqrtf(b.hyper[2]);
    gs = b.hyper[3];
  } else if (b.grad_scale) {
    gs = b.grad_scale[0];
  }
  if (!(fabsf(gs) < INFINITY)) return;  // nothing changes
  lr *= en.lr_mul;
  const float size = lr / bias1, keep = 1.f - lr * (b.h.weight_decay * en.decay_mul);
  const float b1 = b.h.beta1, b2 = b.h.beta2, a1 = b.h.alpha1, a2 = b.h.alpha2, eps = b.h.eps;
  PT* param = static_cast<PT*>(en.param);
  const GT* grad = static_cast<const GT*>(en.grad);
  const int64_t i = int64_t(blockIdx.x - b.first[lo]) * kChunk + 8 * int64_t(threadIdx.x);
  float w[8], g[8], m[8], v[8], r[8];
  get(grad, i, n, g);
  if constexpr (MASTER) get(static_cast<const float*>(en.master), i, n, w); else get(param, i, n, w);
  if constexpr (EIGHT) {
    get_codes(static_cast<const uint8_t*>(en.m), en.m_scale, i, n, m);
    get_codes(static_cast<const uint8_t*>(en.v), en.v_scale, i, n, v);
  } else {
    get(static_cast<const float*>(en.m), i, n, m);
    get(static_cast<const float*>(en.v), i, n, v);
  }
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    const float x = g[t] * gs;
    if constexpr (EIGHT) v[t] = v[t] * v[t];
    m[t] = m[t] * b1 + x * a1;
    v[t] = v[t] * b2 + x * a2 * x;
  }
  roots(v, r);
  // the reciprocal's last unit is far below the update's share in w
#pragma unroll
  for (int t = 0; t < 8; ++t)
    w[t] = fmaf(m[t] * -size, __builtin_amdgcn_rcpf(fmaf(r[t], root2, eps)), w[t] * keep);
  if constexpr (EIGHT) {
    put_codes<false>(static_cast<uint8_t*>(en.m), en.m_scale, i, n, m);
    put_codes<true>(static_cast<uint8_t*>(en.v), en.v_scale, i, n, r);
  } else {
    put(static_cast<float*>(en.m), i, n, m);
    put(static_cast<float*>(en.v), i, n, v);
  }
  if constexpr (MASTER) put(en.master, i, n, w);
  put(param, i, n, w);
}

template <class PT, class GT, bool EIGHT, bool MASTER>
void launch(const Batch& b, hipStream_t st) {
  hipLaunchKernelGGL((step_kernel<PT, GT, EIGHT, MASTER>), dim3(b.first[b.count]), dim3(kThreads), 0, st, b);
}

template <class PT, class GT, bool MASTER>
void launch_state(const Batch& b, bool eight, hipStream_t st) {
  eight ? launch<PT, GT, true, MASTER>(b, st) : launch<PT, GT, false, MASTER>(b, st);
}

}  // namespace adamw

hipError_t launch_adamw(const AdamwArgs& a, const AdamwTensor* tensors, int64_t count, hipStream_t st,
                        KernelTimer* timer) {
  using namespace adamw;
  Batch b;
  b.h = a.h;
  b.grad_scale = a.grad_scale;
  b.hyper = a.hyper;
  // tensors with and without a master copy in launches of their own
  for (int master = 0; master < 2; ++master) {
    b.count = 0;
    b.first[0] = 0;
    int64_t i = 0, at = 0;  // tensor, its element
    while (i < count || b.count > 0) {
      if (i < count) {
        const AdamwTensor& t = tensors[i];
        if (t.n <= at || (t.master != nullptr) != (master == 1)) {
          ++i;
          at = 0;
          if (i < count) continue;
        } else {
          // a longer tensor goes on in the next launch
          const int64_t room = int64_t(kMaxChunks) - b.first[b.count];
          const int64_t n = std::min(t.n - at, room * kChunk);
          const int64_t psz = a.param_bf16 ? 2 : 4, gsz = a.grad_bf16 ? 2 : 4, ssz = a.eight ? 1 : 4;
          AdamwTensor& e = b.e[b.count];
          e = t;
          e.param = static_cast<char*>(t.param) + at * psz;
          e.grad = static_cast<const char*>(t.grad) + at * gsz;
          if (t.master) e.master = t.master + at;
          e.m = static_cast<char*>(t.m) + at * ssz;
          e.v = static_cast<char*>(t.v) + at * ssz;
          if (t.m_scale) e.m_scale = t.m_scale + at / 128;
          if (t.v_scale) e.v_scale = t.v_scale + at / 128;
          e.n = n;
          b.first[b.count + 1] = b.first[b.count] + uint32_t((n + kChunk - 1) / kChunk);
          ++b.count;
          at += n;
          if (at >= t.n) {
            ++i;
            at = 0;
          }
          if (b.count < kMaxTensors && b.first[b.count] < kMaxChunks && i < count) continue;
        }
      }
      if (b.count > 0) {
        TimedLaunch tl(timer, "adamw", st);
        if (master)
          a.grad_bf16 ? launch_state<uint16_t, uint16_t, true>(b, a.eight, st)
                      : launch_state<uint16_t, float, true>(b, a.eight, st);
        else if (a.param_bf16)
          a.grad_bf16 ? launch_state<uint16_t, uint16_t, false>(b, a.eight, st)
                      : launch_state<uint16_t, float, false>(b, a.eight, st);
        else
          a.grad_bf16 ? launch_state<float, uint16_t, false>(b, a.eight, st)
                      : launch_state<float, float, false>(b, a.eight, st);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        b.count = 0;
        b.first[0] = 0;
      }
    }
  }
  return hipSuccess;
}

}  // namespace moe
