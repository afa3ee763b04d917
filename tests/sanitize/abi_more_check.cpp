// Host-side checks of the gate, the dense products and AdamW under AddressSanitizer
// and UndefinedBehaviorSanitizer (built by tests/test_host_sanitizers_more.py). Every
// call is refused, or answered, before any device work.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "../../include/moe.h"

static int g_fail = 0;
#define EXPECT(cond)                                               \
  do {                                                             \
    if (!(cond)) {                                                 \
      std::fprintf(stderr, "FAILED %s:%d %s\n", __FILE__, __LINE__, #cond); \
      ++g_fail;                                                    \
    }                                                              \
  } while (0)

int main() {
  void* const P = reinterpret_cast<void*>(uintptr_t(1) << 20);  // aligned stand-in, never dereferenced
  void* const Q = reinterpret_cast<void*>((uintptr_t(1) << 20) + 2);
  float* const F = static_cast<float*>(P);
  int32_t* const N = static_cast<int32_t*>(P);
  uint8_t* const U = static_cast<uint8_t*>(P);

  // dense products: every size that is served has a scratch, larger ones serve smaller M
  const int64_t sides[] = {1, 2, 7, 8, 31, 64, 65, 127, 256, 777, 1001, 2048, 16384, 65537, 1 << 20, (1 << 20) + 1};
  const int64_t rows[] = {0, 1, 15, 64, 65, 1003, 4097, 16384, 131072, 1 << 24, (1 << 24) + 1};
  int served = 0, refused = 0;
  for (int act = MOE_ACT_NONE; act <= MOE_ACT_SWIGLU; ++act)
    for (int out = MOE_DT_BF16; out <= MOE_DT_F32; ++out)
      for (int64_t n : sides)
        for (int64_t k : sides) {
          size_t before_f = 0, before_b = 0;
          for (int64_t m : rows) {
            const moe_linear_shape s = {m, n, k, act, out, 0};
            const int64_t r = act == MOE_ACT_SWIGLU ? 2 * n : n, side = 1 << 20;
            const bool ok = m <= (1 << 24) && n <= side && k <= side && r <= side && m * k < int64_t(1) << 36 &&
                            m * r < int64_t(1) << 36 && r * ((k + 7) / 8 * 8) <= int64_t(1) << 30;
            size_t f = 0, b = 0;
            const moe_status st = moe_linear_workspace_size(&s, &f, &b);
            EXPECT(st == (ok ? MOE_OK : MOE_ERR_SHAPE));
            if (!ok) {
              ++refused;
              continue;
            }
            ++served;
            EXPECT(f >= before_f && b >= before_b);
            before_f = f;
            before_b = b;
            const moe_status none = m == 0 ? MOE_OK : MOE_ERR_NULL;
            EXPECT(moe_linear(&s, nullptr, P, nullptr, nullptr, P, nullptr, P, f, nullptr) == none);
            if (m == 0) continue;
            EXPECT(moe_linear(&s, P, P, nullptr, nullptr, P, nullptr, P, f - 1, nullptr) == MOE_ERR_WORKSPACE);
            EXPECT(moe_linear(&s, P, Q, nullptr, nullptr, P, nullptr, P, f, nullptr) == MOE_ERR_ALIGN);
            EXPECT(moe_linear_bwd(&s, P, P, P, P, nullptr, nullptr, nullptr, P, b, nullptr) == MOE_OK);  // nothing asked
            EXPECT(moe_linear_bwd(&s, P, P, P, P, P, P, F, P, b - 1, nullptr) == MOE_ERR_WORKSPACE);
            EXPECT(moe_linear_bwd(&s, P, nullptr, P, P, P, P, F, P, b, nullptr) == MOE_ERR_NULL);
            EXPECT(moe_linear_bwd(&s, P, P, P, P, P, Q, F, P, b, nullptr) == MOE_ERR_ALIGN);
          }
        }
  EXPECT(served > 1000 && refused > 1000);
  moe_linear_shape bad = {4, 4, 4, MOE_ACT_NONE, MOE_DT_BF16, 0};
  size_t f = 0, b = 0;
  EXPECT(moe_linear_workspace_size(&bad, nullptr, nullptr) == MOE_OK);
  EXPECT(moe_linear_workspace_size(nullptr, &f, &b) == MOE_ERR_NULL);
  for (int64_t v : {INT64_MIN, int64_t(-1), INT64_MAX}) {
    for (int at = 0; at < 3; ++at) {
      moe_linear_shape s = bad;
      (at == 0 ? s.M : at == 1 ? s.N : s.K) = v;
      EXPECT(moe_linear_workspace_size(&s, &f, &b) == MOE_ERR_SHAPE);
    }
    moe_linear_shape s = bad;
    s.reserved = v;
    EXPECT(moe_linear_workspace_size(&s, &f, &b) == MOE_ERR_SHAPE);
  }
  bad.act = 5;
  EXPECT(moe_linear_workspace_size(&bad, &f, &b) == MOE_ERR_PRECISION);
  bad.act = 0;
  bad.out_dtype = 2;
  EXPECT(moe_linear_workspace_size(&bad, &f, &b) == MOE_ERR_PRECISION);

  // the gate
  moe_shape m;
  std::memset(&m, 0, sizeof(m));
  m.H = 256; m.I = 128;
  for (int64_t E : {int64_t(1), int64_t(60), int64_t(128), int64_t(1024)})
    for (int64_t k : {int64_t(1), int64_t(2), int64_t(16), int64_t(1024)})
      for (int32_t G : {INT32_MIN, -1, 0, 1, 4, 60, 64, 65, INT32_MAX})
        for (int32_t L : {INT32_MIN, 0, 1, 2, 64, INT32_MAX})
          for (int32_t top : {0, 1, 2, 3}) {
            m.T = 5; m.E = E; m.k = k;
            const moe_gate_params p = {MOE_SCORE_SIGMOID, 1, G, L, top, 1.f, 0};
            const bool ok = k <= E && G >= 1 && G <= 64 && E % G == 0 && L >= 1 && L <= G && (top == 1 || top == 2) &&
                            k <= L * (E / G);
            const moe_status st = moe_gate(&m, &p, nullptr, F, U, N, F, nullptr);
            EXPECT(st == (ok ? MOE_ERR_NULL : MOE_ERR_SHAPE));
            EXPECT(moe_gate_bwd(&m, &p, F, N, F, 0, static_cast<float*>(Q), nullptr) == (ok ? MOE_ERR_ALIGN : MOE_ERR_SHAPE));
            m.T = 0;
            EXPECT(moe_gate(&m, &p, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr) == (ok ? MOE_OK : MOE_ERR_SHAPE));
          }
  m.T = 5; m.E = 8; m.k = 2;
  moe_gate_params g = {MOE_SCORE_SOFTMAX, 1, 1, 1, 1, 1.f, 0};
  EXPECT(moe_gate(&m, nullptr, F, F, U, N, F, nullptr) == MOE_ERR_NULL);
  for (float v : {INFINITY, -INFINITY, NAN}) {
    g.scale = v;
    EXPECT(moe_gate(&m, &g, F, F, U, N, F, nullptr) == MOE_ERR_SHAPE);
  }
  g.scale = 1.f;
  g.score = 2;
  EXPECT(moe_gate(&m, &g, F, F, U, N, F, nullptr) == MOE_ERR_PRECISION);

  // AdamW
  moe_adamw_tensor t[3];
  std::memset(t, 0, sizeof(t));
  moe_adamw_params p;
  std::memset(&p, 0, sizeof(p));
  p.lr = 1e-3; p.beta1 = 0.9; p.beta2 = 0.999; p.eps = 1e-8; p.weight_decay = 0.1;
  p.param_dtype = MOE_DT_BF16; p.grad_dtype = MOE_DT_F32; p.step = 1;
  EXPECT(moe_adamw_step(nullptr, t, 3, nullptr, nullptr, nullptr) == MOE_ERR_NULL);
  EXPECT(moe_adamw_step(&p, nullptr, 0, nullptr, nullptr, nullptr) == MOE_OK);
  EXPECT(moe_adamw_step(&p, nullptr, 3, nullptr, nullptr, nullptr) == MOE_ERR_NULL);
  EXPECT(moe_adamw_step(&p, t, -1, nullptr, nullptr, nullptr) == MOE_ERR_SHAPE);
  EXPECT(moe_adamw_step(&p, t, 3, F, F, nullptr) == MOE_ERR_SHAPE);
  const double wild[] = {INFINITY, -INFINITY, NAN, 1e300, -1e300, 1.0, -0.5};
  for (double v : wild)
    for (int at = 0; at < 5; ++at) {
      moe_adamw_params q = p;
      (at == 0 ? q.lr : at == 1 ? q.beta1 : at == 2 ? q.beta2 : at == 3 ? q.eps : q.weight_decay) = v;
      const bool fine = std::fabs(v) <= 1.0 && !(at == 1 || at == 2) && !(at == 3 && v < 0);
      t[0].n = fine ? -1 : 0;  // what is fine gets as far as the tensors
      EXPECT(moe_adamw_step(&q, t, 3, nullptr, nullptr, nullptr) == MOE_ERR_SHAPE);
    }
  for (int64_t n : {INT64_MIN, int64_t(-1), int64_t(1) << 40, INT64_MAX}) {
    t[0].n = n;
    EXPECT(moe_adamw_step(&p, t, 3, nullptr, nullptr, nullptr) == MOE_ERR_SHAPE);
  }
  for (int64_t step : {INT64_MIN, int64_t(0)}) {
    moe_adamw_params q = p;
    q.step = step;
    EXPECT(moe_adamw_step(&q, t, 3, nullptr, nullptr, nullptr) == MOE_ERR_SHAPE);
  }
  t[0].n = 5;
  t[0].param = P; t[0].grad = P; t[0].m = P;
  EXPECT(moe_adamw_step(&p, t, 3, nullptr, nullptr, nullptr) == MOE_ERR_NULL);  // v
  t[0].v = P; t[0].m_scale = U;
  EXPECT(moe_adamw_step(&p, t, 3, nullptr, nullptr, nullptr) == MOE_ERR_NULL);  // scales with fp32 moments
  t[0].m_scale = nullptr;
  t[0].grad = Q;
  EXPECT(moe_adamw_step(&p, t, 3, nullptr, nullptr, nullptr) == MOE_ERR_ALIGN);
  p.param_dtype = MOE_DT_F32;
  t[0].master = F;
  EXPECT(moe_adamw_step(&p, t, 3, nullptr, nullptr, nullptr) == MOE_ERR_SHAPE);
  if (g_fail) return 1;
  std::puts("abi more checks passed");
  return 0;
}
