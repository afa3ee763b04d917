// Host-side checks of the balance and orthogonalisation entry points under
// AddressSanitizer and UndefinedBehaviorSanitizer (built by
// tests/test_host_sanitizers_train.py). Every call is refused, or answered,
// before any device work.
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

static moe_ortho_shape ortho(int64_t E, int64_t R, int64_t C, int dtype = MOE_DT_BF16) {
  moe_ortho_shape s;
  std::memset(&s, 0, sizeof(s));
  s.E = E; s.R = R; s.C = C;
  s.steps = 5;
  s.grad_dtype = dtype;
  s.a = 3.4445f; s.b = -4.7750f; s.c = 2.0315f;
  s.eps = 1e-7f;
  return s;
}

int main() {
  void* const P = reinterpret_cast<void*>(uintptr_t(1) << 20);  // aligned stand-in, never dereferenced
  void* const Q = reinterpret_cast<void*>((uintptr_t(1) << 20) + 8);
  float* const F = static_cast<float*>(P);
  int32_t* const N = static_cast<int32_t*>(P);
  const int64_t sides[] = {1, 2, 31, 32, 33, 64, 96, 127, 128, 129, 255, 256, 257, 768, 1000, 2048, 4096, 16384};
  const int64_t stacks[] = {0, 1, 2, 1023, 1024, 1025, 100000};
  for (int dtype = MOE_DT_BF16; dtype <= MOE_DT_F32; ++dtype)
    for (int64_t R : sides)
      for (int64_t C : sides)
        for (int64_t E : stacks) {
          const moe_ortho_shape s = ortho(E, R, C, dtype);
          size_t n = 0, more = 0;
          const moe_status st = moe_ortho_workspace_size(&s, &n);
          if (E * R * C >= int64_t(1) << 40) {
            EXPECT(st == MOE_ERR_SHAPE);
            continue;
          }
          EXPECT(st == MOE_OK && n > 0);
          if (E == 0) {
            EXPECT(moe_orthogonalize(&s, nullptr, nullptr, nullptr, 0, nullptr) == MOE_OK);
            continue;
          }
          EXPECT(moe_orthogonalize(&s, P, P, P, n - 1, nullptr) == MOE_ERR_WORKSPACE);
          EXPECT(moe_orthogonalize(&s, P, Q, P, n, nullptr) == MOE_ERR_ALIGN);
          // a stack twice as high needs at least as much
          moe_ortho_shape t = s;
          t.E = 2 * E;
          if (moe_ortho_workspace_size(&t, &more) == MOE_OK && R * C < 1000000) EXPECT(more + 4096 >= n);
        }
  const float odd[] = {0.f, 1.f, -1.f, 1e-30f, 1e30f, 65504.f, -3e38f};
  for (float a : odd)
    for (float b : odd)
      for (float c : odd)
        for (int steps : {1, 2, 32}) {
          moe_ortho_shape s = ortho(3, 100, 200);
          s.a = a; s.b = b; s.c = c; s.steps = steps;
          size_t n = 0;
          EXPECT(moe_ortho_workspace_size(&s, &n) == MOE_OK && n > 0);
        }
  moe_ortho_shape s = ortho(2, 64, 64);
  moe_muon_params p;
  std::memset(&p, 0, sizeof(p));
  p.lr = 0.1f; p.mu = 0.9f; p.scale = 1.f;
  size_t n = 0;
  EXPECT(moe_ortho_workspace_size(&s, nullptr) == MOE_ERR_NULL && moe_ortho_workspace_size(nullptr, &n) == MOE_ERR_NULL);
  EXPECT(moe_ortho_workspace_size(&s, &n) == MOE_OK);
  EXPECT(moe_muon_step(&s, &p, P, F, P, nullptr, P, n - 1, nullptr) == MOE_ERR_WORKSPACE);
  EXPECT(moe_muon_step(&s, nullptr, P, F, P, nullptr, P, n, nullptr) == MOE_ERR_NULL);
  EXPECT(moe_muon_step(&s, &p, P, nullptr, P, nullptr, P, n, nullptr) == MOE_ERR_NULL);
  EXPECT(moe_muon_step(&s, &p, P, F, P, static_cast<float*>(Q), P, n, nullptr) == MOE_ERR_ALIGN);
  p.mu = NAN;
  EXPECT(moe_muon_step(&s, &p, P, F, P, nullptr, P, n, nullptr) == MOE_ERR_SHAPE);

  moe_shape m;
  std::memset(&m, 0, sizeof(m));
  m.H = 2048; m.I = 768; m.k = 2;
  for (int64_t T : {int64_t(0), int64_t(1), int64_t(1000), int64_t(131072), int64_t(690000)})
    for (int64_t E : {int64_t(2), int64_t(33), int64_t(1024)})
      for (int64_t S : {int64_t(1), int64_t(2), int64_t(5000), int64_t(1) << 20, (int64_t(1) << 20) + 1}) {
        m.T = T; m.E = E;
        const size_t need = moe_balance_scratch_bytes(&m, S);
        if (S > (int64_t(1) << 20) || S * E >= int64_t(1) << 28) {
          EXPECT(need == 0);
          continue;
        }
        EXPECT(need > 0);
        EXPECT(moe_balance(&m, F, N, N, S, nullptr, F, N, N, F, F, P, need - 1, nullptr) == MOE_ERR_WORKSPACE);
        EXPECT(moe_balance(&m, F, N, N, S, nullptr, F, N, N, F, F, nullptr, need, nullptr) == MOE_ERR_NULL);
        const moe_status st = moe_balance_bwd(&m, F, N, F, F, 1, N, S, nullptr, N, F, nullptr, F, nullptr);
        EXPECT(st == (T == 0 ? MOE_OK : MOE_ERR_NULL));
      }
  if (g_fail) return 1;
  std::puts("abi train checks passed");
  return 0;
}
