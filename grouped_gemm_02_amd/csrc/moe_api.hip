// C ABI of the MoE expert layer: validation, buffer layout, launch order.
// Declarations and the contract of every entry point are in include/moe.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <string>
#include <vector>

#include "../../include/moe.h"
#include "kernels.h"

namespace {

using namespace moe;

constexpr size_t kAlign = 256;
size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

// ------------------------------------------------------------ shape checks

moe_status check_shape(const moe_shape* s) {
  if (!s) return MOE_ERR_NULL;
  if (s->precision < MOE_BF16 || s->precision > MOE_FP8_BWD_F32) return MOE_ERR_PRECISION;
  if (s->T < 0 || s->E < 1 || s->E > 1024 || s->k < 1 || s->k > s->E) return MOE_ERR_SHAPE;
  if (s->H < 256 || s->H > 16384 || s->H % 256 != 0) return MOE_ERR_SHAPE;
  if (s->I < 128 || s->I > 8192 || s->I % 128 != 0) return MOE_ERR_SHAPE;
  if (s->T * s->k >= (int64_t(1) << 31)) return MOE_ERR_SHAPE;
  if (s->T * s->H >= (int64_t(1) << 31)) return MOE_ERR_SHAPE;  // 32-bit row offsets into x, dY
  if (s->T * s->k * s->I >= (int64_t(1) << 30)) return MOE_ERR_SHAPE;  // 32-bit byte offsets into [g | u] rows
  if (s->num_cus < 0 || s->reserved != 0) return MOE_ERR_SHAPE;
  if ((s->flags & ~MOE_FLAG_FP8_WGRAD) != 0) return MOE_ERR_PRECISION;
  if ((s->flags & MOE_FLAG_FP8_WGRAD) != 0) {
    if (s->precision == MOE_BF16 || s->precision == MOE_FP8_FP4) return MOE_ERR_PRECISION;  // no FP8 backward
    // the row-axis quantizer has the power-of-two and MX rules only
    if (s->precision == MOE_FP8_BLOCK_F32 || s->precision == MOE_FP8_BWD_F32) return MOE_ERR_UNSUPPORTED;
    // 32-bit offsets inside a weight-gradient tile's 256 rows of Kp codes
    if (s->T * s->k >= (int64_t(1) << 23)) return MOE_ERR_SHAPE;
  }
  return MOE_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool fp8_forward(const moe_shape& s) {
  return s.precision == MOE_FP8_BLOCK || s.precision == MOE_MXFP8 || s.precision == MOE_FP8_FP4 ||
         s.precision == MOE_FP8_BLOCK_F32;
}
bool fp8_backward(const moe_shape& s) {
  return s.precision == MOE_FP8_BLOCK || s.precision == MOE_MXFP8 || s.precision == MOE_FP8_BWD ||
         s.precision == MOE_FP8_BLOCK_F32 || s.precision == MOE_FP8_BWD_F32;
}
bool fp4_weights(const moe_shape& s) { return s.precision == MOE_FP8_FP4; }
// blockwise with fp32 block scales
bool f32_scales(const moe_shape& s) { return s.precision == MOE_FP8_BLOCK_F32 || s.precision == MOE_FP8_BWD_F32; }
// activation block (32 or 128 values along the reduction axis) and scale rule
bool mx_acts(const moe_shape& s) { return s.precision == MOE_MXFP8 || s.precision == MOE_FP8_FP4; }
int act_block(const moe_shape& s) { return mx_acts(s) ? 32 : 128; }
int scale_rule(const moe_shape& s) { return mx_acts(s) ? kRuleMx : (f32_scales(s) ? kRuleF32 : kRulePow2); }
bool fp8_wgrad(const moe_shape& s) { return (s.flags & MOE_FLAG_FP8_WGRAD) != 0; }
// an upper bound of the sum over experts of rows rounded up to 128
int64_t wgrad_rows_cap(const moe_shape& s) { return 128 * ((s.T * s.k) / 128 + s.E); }

// bytes of E4M3 codes [rows, K] and of their scale bytes [rows, K/32]
size_t codes_bytes(int64_t rows, int64_t K) { return align_up(size_t(rows) * size_t(K)); }
size_t scale_bytes(int64_t rows, int64_t K) { return align_up(size_t(rows) * size_t(K / 32)); }

// ------------------------------------------------------------ buffer layouts

struct FwdLayout {
  size_t perm;     // permutation scratch (status word first)
  size_t rows;     // bf16 [Tk, H] weighted expert outputs
  size_t inf;      // saved-like area used when no saved buffer is given
  size_t xq, xs;   // FP8 forward: x codes [T, H], scales [T, H/32]
  size_t aq, as;   // FP8 forward: w*silu(g)*u codes [Tk, I], scales [Tk, I/32]
  size_t total;
};

moe_wq_layout wq_layout(const moe_shape& s) {
  moe_wq_layout L;
  L.w13 = L.w13_scale = L.w2 = L.w2_scale = SIZE_MAX;
  L.w2t = L.w2t_scale = L.w13t = L.w13t_scale = SIZE_MAX;
  size_t o = 0;
  const int64_t E = s.E, H = s.H, I = s.I;
  if (fp8_forward(s)) {
    const int64_t div = fp4_weights(s) ? 2 : 1;  // FP4: two codes per byte
    L.w13 = o;       o += codes_bytes(E * 2 * I, H / div);
    L.w13_scale = o; o += scale_bytes(E * 2 * I, H);
    L.w2 = o;        o += codes_bytes(E * H, I / div);
    L.w2_scale = o;  o += scale_bytes(E * H, I);
  }
  if (fp8_backward(s)) {
    L.w2t = o;        o += codes_bytes(E * I, H);
    L.w2t_scale = o;  o += scale_bytes(E * I, H);
    L.w13t = o;       o += codes_bytes(E * H, 2 * I);
    L.w13t_scale = o; o += scale_bytes(E * H, 2 * I);
  }
  L.total = o;
  return L;
}

moe_saved_layout saved_layout(const moe_shape& s) {
  const int64_t Tk = s.T * s.k;
  moe_saved_layout L;
  size_t o = 0;
  L.counts = o;  o = align_up(o + size_t(s.E) * 4);
  L.offsets = o; o = align_up(o + size_t(s.E + 1) * 4);
  L.row_of = o;  o = align_up(o + size_t(Tk) * 4);
  L.src_of = o;  o = align_up(o + size_t(Tk) * 4);
  L.wrow = o;    o = align_up(o + size_t(Tk) * 4);
  L.h13 = o;     o = align_up(o + size_t(Tk) * size_t(2 * s.I) * 2);
  L.act = o;     o = align_up(o + size_t(Tk) * size_t(s.I) * 2);
  L.total = o;
  return L;
}

FwdLayout fwd_layout(const moe_shape& s) {
  const int64_t Tk = s.T * s.k;
  FwdLayout L;
  size_t o = 0;
  L.perm = o; o = align_up(o + permute_scratch_bytes(Tk, int(s.E)));
  L.rows = o; o = align_up(o + size_t(Tk) * size_t(s.H) * 2);
  L.inf = o;  o = align_up(o + saved_layout(s).total);
  L.xq = L.xs = L.aq = L.as = 0;
  if (fp8_forward(s)) {
    L.xq = o; o += codes_bytes(s.T, s.H);
    L.xs = o; o += scale_bytes(s.T, s.H);
    L.aq = o; o += codes_bytes(Tk, s.I);
    L.as = o; o += scale_bytes(Tk, s.I);
  }
  L.total = o;
  return L;
}

struct BwdLayout {
  size_t queues;   // int32: tile queues, then the split plans, of the weight-gradient GEMMs
  size_t partial;  // fp32 partial tiles of split weight-gradient items
  size_t dh13, dwpart, dxrows;
  size_t dyq, dys;  // FP8 backward: dY codes [T, H], scales [T, H/32]
  size_t dhq, dhs;  // FP8 backward: [dg | du] codes [Tk, 2I], scales [Tk, 2I/32]
  // FP8 weight gradients: operands quantized along tokens (codes, scales) of
  // [dg | du], x, dY and w*silu(g)*u
  size_t wgd, wgds, wgx, wgxs, wgy, wgys, wga, wgas;
  size_t total;
};

BwdLayout bwd_layout(const moe_shape& s) {
  const int64_t Tk = s.T * s.k;
  BwdLayout L;
  size_t o = 0;
  L.queues = o; o = align_up(o + size_t(kQueueWords) * 4);
  L.partial = o; o = align_up(o + size_t(kSplitFloats) * 4);
  L.dh13 = o;   o = align_up(o + size_t(Tk) * size_t(2 * s.I) * 2);
  L.dwpart = o; o = align_up(o + size_t(Tk) * size_t(dh_num_parts(s.I)) * 4);
  L.dxrows = o; o = align_up(o + size_t(Tk) * size_t(s.H) * 2);
  L.dyq = L.dys = L.dhq = L.dhs = 0;
  if (fp8_backward(s)) {
    L.dyq = o; o += codes_bytes(s.T, s.H);
    L.dys = o; o += scale_bytes(s.T, s.H);
    L.dhq = o; o += codes_bytes(Tk, 2 * s.I);
    L.dhs = o; o += scale_bytes(Tk, 2 * s.I);
  }
  L.wgd = L.wgds = L.wgx = L.wgxs = L.wgy = L.wgys = L.wga = L.wgas = 0;
  if (fp8_wgrad(s)) {
    const int64_t K = wgrad_rows_cap(s);
    L.wgd = o; o += codes_bytes(2 * s.I, K);
    L.wgds = o; o += scale_bytes(2 * s.I, K);
    L.wgx = o; o += codes_bytes(s.H, K);
    L.wgxs = o; o += scale_bytes(s.H, K);
    L.wgy = o; o += codes_bytes(s.H, K);
    L.wgys = o; o += scale_bytes(s.H, K);
    L.wga = o; o += codes_bytes(s.I, K);
    L.wgas = o; o += scale_bytes(s.I, K);
  }
  L.total = o;
  return L;
}

// ------------------------------------------------------------ device info

struct DevInfo {
  bool checked = false;
  bool gfx950 = false;
  int cus = 0;
};
std::mutex g_dev_mu;
DevInfo g_dev[64];

moe_status device_info(int* cus_out) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return MOE_ERR_LAUNCH;
  std::lock_guard<std::mutex> lk(g_dev_mu);
  DevInfo& d = g_dev[dev];
  if (!d.checked) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return MOE_ERR_LAUNCH;
    d.gfx950 = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
    d.cus = prop.multiProcessorCount;
    d.checked = true;
  }
  if (!d.gfx950) return MOE_ERR_ARCH;
  *cus_out = d.cus;
  return MOE_OK;
}

// ------------------------------------------------------------ kernel timing

struct EventTimer : KernelTimer {
  struct Rec {
    std::string name;
    hipEvent_t a, b;
  };
  std::vector<Rec> recs;
  std::vector<hipEvent_t> pool;
  hipEvent_t get() {
    if (!pool.empty()) {
      hipEvent_t e = pool.back();
      pool.pop_back();
      return e;
    }
    hipEvent_t e = nullptr;
    if (hipEventCreate(&e) != hipSuccess) return nullptr;
    return e;
  }
  void begin(const char* name, hipStream_t st) override {
    Rec r{name, get(), get()};
    if (r.a) (void)hipEventRecord(r.a, st);
    recs.push_back(r);
  }
  void end(hipStream_t st) override {
    if (!recs.empty() && recs.back().b) (void)hipEventRecord(recs.back().b, st);
  }
};

std::mutex g_timer_mu;
bool g_timing = false;
EventTimer g_timer;

KernelTimer* timer() { return g_timing ? &g_timer : nullptr; }

moe_status launch_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH; }

template <class T>
T* at(void* base, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(base) + off);
}
template <class T>
const T* at(const void* base, size_t off) {
  return reinterpret_cast<const T*>(static_cast<const char*>(base) + off);
}

// ------------------------------------------------------------ balance, orthogonalisation

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool sequences_fit(const moe_shape& s, int64_t S) {
  return S >= 1 && S <= (int64_t(1) << 20) && S * s.E < (int64_t(1) << 28);
}

moe_status check_sequences(const moe_shape& s, const int32_t* seq_offsets, int64_t S) {
  if (!sequences_fit(s, S)) return MOE_ERR_SHAPE;
  if (!seq_offsets && S != 1) return MOE_ERR_NULL;
  return MOE_OK;
}

moe_status check_ortho(const moe_ortho_shape* s) {
  if (!s) return MOE_ERR_NULL;
  if (s->grad_dtype != MOE_DT_BF16 && s->grad_dtype != MOE_DT_F32) return MOE_ERR_PRECISION;
  if (s->E < 0 || s->R < 1 || s->C < 1 || s->R > 16384 || s->C > 16384) return MOE_ERR_SHAPE;
  if (s->E > ((int64_t(1) << 40) - 1) / (s->R * s->C)) return MOE_ERR_SHAPE;  // E R C < 2^40
  if (s->steps < 1 || s->steps > 32 || s->reserved != 0) return MOE_ERR_SHAPE;
  if (!std::isfinite(s->a) || !std::isfinite(s->b) || !std::isfinite(s->c)) return MOE_ERR_SHAPE;
  if (!std::isfinite(s->eps) || s->eps < 0.f) return MOE_ERR_SHAPE;
  return MOE_OK;
}

OrthoArgs ortho_args(const moe_ortho_shape& s) {
  return OrthoArgs{s.E, int(s.R), int(s.C), s.steps, s.grad_dtype == MOE_DT_F32, s.a, s.b, s.c, s.eps};
}

// ------------------------------------------------------------ gate, dense products, AdamW

moe_status check_gate(const moe_shape& s, const moe_gate_params* p) {
  if (!p) return MOE_ERR_NULL;
  if (p->score != MOE_SCORE_SOFTMAX && p->score != MOE_SCORE_SIGMOID) return MOE_ERR_PRECISION;
  if (p->groups < 1 || p->groups > 64 || s.E % p->groups != 0) return MOE_ERR_SHAPE;
  if (p->groups_kept < 1 || p->groups_kept > p->groups || p->group_top < 1 || p->group_top > 2) return MOE_ERR_SHAPE;
  if (s.k > p->groups_kept * (s.E / p->groups)) return MOE_ERR_SHAPE;
  if (!std::isfinite(p->scale) || p->reserved != 0) return MOE_ERR_SHAPE;
  return MOE_OK;
}

GateArgs gate_args(const moe_shape& s, const moe_gate_params& p, const float* logits, const float* bias,
                   const uint8_t* mask) {
  return GateArgs{logits, bias, mask, s.T, int(s.E), int(s.k), p.score == MOE_SCORE_SIGMOID, p.renorm != 0,
                  p.groups, p.groups_kept, p.group_top, p.scale};
}

int64_t linear_rows(const moe_linear_shape& s) { return s.act == MOE_ACT_SWIGLU ? 2 * s.N : s.N; }

moe_status check_linear(const moe_linear_shape* s) {
  if (!s) return MOE_ERR_NULL;
  if (s->act < MOE_ACT_NONE || s->act > MOE_ACT_SWIGLU) return MOE_ERR_PRECISION;
  if (s->out_dtype != MOE_DT_BF16 && s->out_dtype != MOE_DT_F32) return MOE_ERR_PRECISION;
  const int64_t side = int64_t(1) << 20, area = int64_t(1) << 36;
  if (s->M < 0 || s->M > (int64_t(1) << 24) || s->N < 1 || s->K < 1 || s->N > side || s->K > side) return MOE_ERR_SHAPE;
  const int64_t R = linear_rows(*s);
  if (R > side || s->M * s->K >= area || s->M * R >= area) return MOE_ERR_SHAPE;
  // 32-bit byte offsets into W
  if (R * ((s->K + 7) / 8 * 8) > (int64_t(1) << 30) || s->reserved != 0) return MOE_ERR_SHAPE;
  return MOE_OK;
}

LinearArgs linear_args(const moe_linear_shape& s) {
  static_assert(MOE_ACT_NONE == kActNone && MOE_ACT_RELU == kActRelu && MOE_ACT_SILU == kActSilu &&
                    MOE_ACT_GELU == kActGelu && MOE_ACT_SWIGLU == kActSwiglu,
                "the kernels know the activations by the same numbers");
  return LinearArgs{s.M, s.N, s.K, s.act, s.out_dtype == MOE_DT_F32};
}

bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

int effective_cus(const moe_shape& s, int dev_cus) {
  return (s.num_cus > 0 && s.num_cus < dev_cus) ? s.num_cus : dev_cus;
}

}  // namespace

extern "C" {

const char* moe_status_string(moe_status st) {
  switch (st) {
    case MOE_OK: return "MOE_OK";
    case MOE_ERR_NULL: return "MOE_ERR_NULL: a required pointer is NULL";
    case MOE_ERR_SHAPE: return "MOE_ERR_SHAPE: shape violates H%256, I%128, 1<=k<=E or size limits";
    case MOE_ERR_ALIGN: return "MOE_ERR_ALIGN: a tensor pointer is not 16-byte aligned";
    case MOE_ERR_PRECISION: return "MOE_ERR_PRECISION: unknown precision";
    case MOE_ERR_ARCH: return "MOE_ERR_ARCH: current device is not gfx950";
    case MOE_ERR_WORKSPACE: return "MOE_ERR_WORKSPACE: workspace smaller than required";
    case MOE_ERR_LAUNCH: return "MOE_ERR_LAUNCH: HIP launch or runtime call failed";
    case MOE_ERR_ROUTING: return "MOE_ERR_ROUTING: an expert id was outside [0, E)";
    case MOE_ERR_UNSUPPORTED: return "MOE_ERR_UNSUPPORTED: not implemented by this library";
  }
  return "unknown moe_status";
}

moe_status moe_workspace_size(const moe_shape* s, size_t* fwd_ws, size_t* saved_bytes,
                              size_t* bwd_ws) {
  const moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  if (fwd_ws) *fwd_ws = fwd_layout(*s).total;
  if (saved_bytes) *saved_bytes = saved_layout(*s).total;
  if (bwd_ws) *bwd_ws = bwd_layout(*s).total;
  return MOE_OK;
}

moe_status moe_get_saved_layout(const moe_shape* s, moe_saved_layout* out) {
  const moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  if (!out) return MOE_ERR_NULL;
  *out = saved_layout(*s);
  return MOE_OK;
}

size_t moe_permute_scratch_bytes(const moe_shape* s) {
  if (check_shape(s) != MOE_OK) return 0;
  return permute_scratch_bytes(s->T * s->k, int(s->E));
}

moe_status moe_permute(const moe_shape* s, const int32_t* topk_idx, int32_t* counts,
                       int32_t* offsets, int32_t* row_of, int32_t* src_of, void* scratch,
                       void* stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  const int64_t Tk = s->T * s->k;
  if (!counts || !offsets || !scratch || (Tk > 0 && (!topk_idx || !row_of || !src_of)))
    return MOE_ERR_NULL;
  if (!aligned16(scratch)) return MOE_ERR_ALIGN;
  int cus = 0;
  if ((st = device_info(&cus)) != MOE_OK) return st;
  std::lock_guard<std::mutex> lk(g_timer_mu);
  return launch_status(launch_permute(topk_idx, Tk, int(s->E), counts, offsets, row_of, src_of,
                                      scratch, static_cast<hipStream_t>(stream), timer()));
}

moe_status moe_permute_noalloc(const moe_shape* s, const int32_t* topk_idx, int32_t* counts, int32_t* offsets,
                               int32_t* row_of, int32_t* src_of, int32_t* status, void* stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  const int64_t Tk = s->T * s->k;
  if (!counts || !offsets || !status || (Tk > 0 && (!topk_idx || !row_of || !src_of))) return MOE_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(status) & 3u) != 0) return MOE_ERR_ALIGN;
  // the chunk table must fit the library's fixed array
  if (int64_t(permute_num_chunks(Tk)) * (s->E + 1) > kStaticPermuteWords) return MOE_ERR_WORKSPACE;
  int cus = 0;
  if ((st = device_info(&cus)) != MOE_OK) return st;
  int32_t* table = nullptr;
  if (permute_static_scratch(&table) != hipSuccess) return MOE_ERR_LAUNCH;
  std::lock_guard<std::mutex> lk(g_timer_mu);
  return launch_status(launch_permute_split(topk_idx, Tk, int(s->E), counts, offsets, row_of, src_of, status,
                                            table, static_cast<hipStream_t>(stream), timer()));
}

moe_status moe_get_wq_layout(const moe_shape* s, moe_wq_layout* out) {
  const moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  if (!out) return MOE_ERR_NULL;
  *out = wq_layout(*s);
  return MOE_OK;
}

moe_status moe_quantize_weights(const moe_shape* s, const void* W13, const void* W2, void* wq,
                                void* stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  if (s->precision == MOE_BF16) return MOE_OK;
  if (!W13 || !W2 || !wq) return MOE_ERR_NULL;
  if (!aligned16(W13) || !aligned16(W2) || !aligned16(wq)) return MOE_ERR_ALIGN;
  int cus = 0;
  if ((st = device_info(&cus)) != MOE_OK) return st;
  const moe_wq_layout L = wq_layout(*s);
  const uint16_t* w13 = static_cast<const uint16_t*>(W13);
  const uint16_t* w2 = static_cast<const uint16_t*>(W2);
  const int H = int(s->H), I = int(s->I), rule = scale_rule(*s);
  hipStream_t hs = static_cast<hipStream_t>(stream);
  std::lock_guard<std::mutex> lk(g_timer_mu);
  KernelTimer* tm = timer();
  if (fp4_weights(*s)) {  // forward only: W13 along H, W2 along I
    hipError_t e = launch_quant_fp4_rows(w13, s->E * 2 * I, H, at<uint8_t>(wq, L.w13), at<uint8_t>(wq, L.w13_scale),
                                         hs, tm);
    if (e != hipSuccess) return MOE_ERR_LAUNCH;
    return launch_status(launch_quant_fp4_rows(w2, s->E * H, I, at<uint8_t>(wq, L.w2), at<uint8_t>(wq, L.w2_scale),
                                               hs, tm));
  }
  const bool fwd = fp8_forward(*s);
  hipError_t e = launch_quant_weights(w13, s->E, 2 * I, H, fwd ? at<uint8_t>(wq, L.w13) : nullptr,
                                      fwd ? at<uint8_t>(wq, L.w13_scale) : nullptr, at<uint8_t>(wq, L.w13t),
                                      at<uint8_t>(wq, L.w13t_scale), rule, hs, tm);
  if (e != hipSuccess) return MOE_ERR_LAUNCH;
  e = launch_quant_weights(w2, s->E, H, I, fwd ? at<uint8_t>(wq, L.w2) : nullptr,
                           fwd ? at<uint8_t>(wq, L.w2_scale) : nullptr, at<uint8_t>(wq, L.w2t),
                           at<uint8_t>(wq, L.w2t_scale), rule, hs, tm);
  return launch_status(e);
}

moe_status moe_quantize_rows(const moe_shape* s, const void* in, int64_t rows, int64_t K, void* codes,
                             void* scales, void* stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  if (s->precision == MOE_BF16) return MOE_ERR_PRECISION;
  if (rows < 0 || K < 128 || K > 65536 || K % 128 != 0 || rows * K >= (int64_t(1) << 31)) return MOE_ERR_SHAPE;
  if (rows == 0) return MOE_OK;
  if (!in || !codes || !scales) return MOE_ERR_NULL;
  if (!aligned16(in) || !aligned16(codes)) return MOE_ERR_ALIGN;
  if (f32_scales(*s) && (reinterpret_cast<uintptr_t>(scales) & 3u) != 0) return MOE_ERR_ALIGN;
  int cus = 0;
  if ((st = device_info(&cus)) != MOE_OK) return st;
  std::lock_guard<std::mutex> lk(g_timer_mu);
  return launch_status(launch_quant_rows(static_cast<const uint16_t*>(in), rows, int(K), static_cast<uint8_t*>(codes),
                                         static_cast<uint8_t*>(scales), act_block(*s), scale_rule(*s),
                                         static_cast<hipStream_t>(stream), timer(), "quant_rows"));
}

moe_status moe_quantize_tokens(const moe_shape* s, const void* in, int64_t ld, int64_t C, const int32_t* counts,
                               const int32_t* offsets, const int32_t* src_of, void* codes, void* scales,
                               void* stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  if (s->precision == MOE_BF16) return MOE_ERR_PRECISION;
  if (f32_scales(*s)) return MOE_ERR_UNSUPPORTED;  // the row-axis reading has pow2 and MX scales only
  if (C < 128 || C > 65536 || C % 128 != 0 || ld < C || ld % 8 != 0) return MOE_ERR_SHAPE;
  if (s->T * s->k >= (int64_t(1) << 23)) return MOE_ERR_SHAPE;
  if (s->T == 0) return MOE_OK;
  if (!in || !counts || !offsets || !codes || !scales) return MOE_ERR_NULL;
  if (!aligned16(in) || !aligned16(codes)) return MOE_ERR_ALIGN;
  int cus = 0;
  if ((st = device_info(&cus)) != MOE_OK) return st;
  std::lock_guard<std::mutex> lk(g_timer_mu);
  return launch_status(launch_quant_tokens(static_cast<const uint16_t*>(in), ld, int(C), counts, offsets,
                                           int(s->E), s->T * s->k, src_of, src_of ? int(s->k) : 1,
                                           static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales),
                                           scale_rule(*s), static_cast<hipStream_t>(stream), timer(),
                                           "quant_tokens"));
}

}  // extern "C"

namespace {

// The forward; with logits != nullptr the router runs first, fused with the
// permutation's histogram pass, and writes topk_idx and topk_w.
moe_status fwd_impl(const moe_shape* s, const void* x, const float* logits, int32_t renorm, int32_t* topk_idx,
                    float* topk_w, const void* W13, const void* W2, const void* wq, void* y, void* saved, void* ws,
                    size_t ws_bytes, void* stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  if (s->precision == MOE_BF16 && wq) return MOE_ERR_PRECISION;
  const bool f8 = fp8_forward(*s);
  const int64_t Tk = s->T * s->k;
  // the FP8 forwards read only the quantized weights
  if ((!f8 && (!W13 || !W2)) || !ws || (f8 && !wq) ||
      (s->T > 0 && (!x || !topk_idx || !topk_w || !y)))
    return MOE_ERR_NULL;
  const void* ptrs[] = {x, topk_idx, topk_w, W13, W2, y, saved, ws, wq, logits};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return MOE_ERR_ALIGN;
  const FwdLayout FL = fwd_layout(*s);
  if (ws_bytes < FL.total) return MOE_ERR_WORKSPACE;
  int cus = 0;
  if ((st = device_info(&cus)) != MOE_OK) return st;

  const moe_saved_layout SL = saved_layout(*s);
  void* sv = saved ? saved : at<char>(ws, FL.inf);
  int32_t* counts = at<int32_t>(sv, SL.counts);
  int32_t* offsets = at<int32_t>(sv, SL.offsets);
  int32_t* row_of = at<int32_t>(sv, SL.row_of);
  int32_t* src_of = at<int32_t>(sv, SL.src_of);
  float* wrow = at<float>(sv, SL.wrow);
  uint16_t* h13 = saved ? at<uint16_t>(sv, SL.h13) : nullptr;
  uint16_t* act = at<uint16_t>(sv, SL.act);
  uint16_t* rows = at<uint16_t>(ws, FL.rows);
  hipStream_t hs = static_cast<hipStream_t>(stream);

  std::lock_guard<std::mutex> lk(g_timer_mu);
  KernelTimer* tm = timer();
  int32_t* perm_status = at<int32_t>(ws, FL.perm);
  int32_t* chunk_tab = at<int32_t>(ws, FL.perm + 256);
  hipError_t e = hipSuccess;
  if (logits) {
    e = launch_route_hist(logits, s->T, int(s->E), int(s->k), renorm, topk_idx, topk_w, chunk_tab, hs, tm);
    if (e != hipSuccess) return MOE_ERR_LAUNCH;
  }
  e = launch_permute_split(topk_idx, Tk, int(s->E), counts, offsets, row_of, src_of, perm_status, chunk_tab, hs, tm,
                           topk_w, wrow, logits != nullptr);
  if (e != hipSuccess || s->T == 0) return launch_status(e);
  GemmProblem gp{s->T, s->H, s->I, s->E, s->k, effective_cus(*s, cus), counts, offsets, src_of, topk_w, wrow};
  GemmOperand gx{x, nullptr}, gw13{W13, nullptr}, ga{act, nullptr}, gw2{W2, nullptr};
  if (f8) {
    const moe_wq_layout WL = wq_layout(*s);
    const int blk = act_block(*s), rule = scale_rule(*s);
    uint8_t* xq = at<uint8_t>(ws, FL.xq);
    uint8_t* xs = at<uint8_t>(ws, FL.xs);
    if ((e = launch_quant_rows(static_cast<const uint16_t*>(x), s->T, int(s->H), xq, xs, blk, rule, hs, tm,
                               "quant_x")) != hipSuccess)
      return MOE_ERR_LAUNCH;
    const bool w4 = fp4_weights(*s), f32 = f32_scales(*s);
    gx = GemmOperand{xq, xs, false, f32};
    gw13 = GemmOperand{at<uint8_t>(wq, WL.w13), at<uint8_t>(wq, WL.w13_scale), w4, f32};
    gw2 = GemmOperand{at<uint8_t>(wq, WL.w2), at<uint8_t>(wq, WL.w2_scale), w4, f32};
  }
  if ((e = launch_gemm1_swiglu(gp, gx, gw13, h13, act, hs, tm)) != hipSuccess) return MOE_ERR_LAUNCH;
  if (f8) {
    uint8_t* aq = at<uint8_t>(ws, FL.aq);
    uint8_t* as = at<uint8_t>(ws, FL.as);
    if ((e = launch_quant_rows(act, Tk, int(s->I), aq, as, act_block(*s), scale_rule(*s), hs, tm,
                               "quant_act")) != hipSuccess)
      return MOE_ERR_LAUNCH;
    ga = GemmOperand{aq, as, false, f32_scales(*s)};
  }
  // top-1: the down GEMM writes y's rows directly; the combine only zeroes
  // the rows of dropped tokens
  const bool direct = s->k == 1;
  if ((e = launch_gemm2(gp, ga, gw2, direct ? static_cast<uint16_t*>(y) : rows, hs, tm)) != hipSuccess)
    return MOE_ERR_LAUNCH;
  e = launch_combine(direct ? nullptr : rows, row_of, s->T, int(s->k), s->H, static_cast<uint16_t*>(y), nullptr, 0,
                     nullptr, hs, tm, "combine_y");
  return launch_status(e);
}

}  // namespace

extern "C" {

moe_status moe_fwd(const moe_shape* s, const void* x, const int32_t* topk_idx,
                   const float* topk_w, const void* W13, const void* W2, const void* wq,
                   void* y, void* saved, void* ws, size_t ws_bytes, void* stream) {
  // read only: without logits fwd_impl writes neither routing buffer
  return fwd_impl(s, x, nullptr, 0, const_cast<int32_t*>(topk_idx), const_cast<float*>(topk_w), W13, W2, wq, y,
                  saved, ws, ws_bytes, stream);
}

moe_status moe_fwd_logits(const moe_shape* s, const void* x, const float* logits, int32_t renorm,
                          int32_t* topk_idx, float* topk_w, const void* W13, const void* W2, const void* wq,
                          void* y, void* saved, void* ws, size_t ws_bytes, void* stream) {
  if (s && s->T > 0 && !logits) return MOE_ERR_NULL;
  return fwd_impl(s, x, s && s->T > 0 ? logits : nullptr, renorm, topk_idx, topk_w, W13, W2, wq, y, saved, ws,
                  ws_bytes, stream);
}

moe_status moe_bwd(const moe_shape* s, const void* dy, const void* x, const int32_t* topk_idx,
                   const float* topk_w, const void* W13, const void* W2, const void* wq,
                   const void* saved, void* dx, float* d_topk_w, void* dW13, void* dW2, void* ws,
                   size_t ws_bytes, void* stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  if (s->precision == MOE_BF16 && wq) return MOE_ERR_PRECISION;
  if (s->precision == MOE_FP8_FP4) return MOE_ERR_PRECISION;  // an inference forward: no backward
  const bool f8 = fp8_backward(*s);
  (void)topk_idx;  // the permutation comes from `saved`
  // the FP8 backwards read only the quantized weights
  if ((!f8 && (!W13 || !W2)) || !saved || !dW13 || !dW2 || !ws || (f8 && !wq) ||
      (s->T > 0 && (!dy || !x || !topk_w || !dx || !d_topk_w)))
    return MOE_ERR_NULL;
  const void* ptrs[] = {dy, x, topk_idx, topk_w, W13, W2, saved, dx, d_topk_w, dW13, dW2, ws, wq};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return MOE_ERR_ALIGN;
  const BwdLayout BL = bwd_layout(*s);
  if (ws_bytes < BL.total) return MOE_ERR_WORKSPACE;
  int cus = 0;
  if ((st = device_info(&cus)) != MOE_OK) return st;

  const moe_saved_layout SL = saved_layout(*s);
  const int32_t* counts = at<int32_t>(saved, SL.counts);
  const int32_t* offsets = at<int32_t>(saved, SL.offsets);
  const int32_t* row_of = at<int32_t>(saved, SL.row_of);
  const int32_t* src_of = at<int32_t>(saved, SL.src_of);
  const float* wrow = at<float>(saved, SL.wrow);
  const uint16_t* h13 = at<uint16_t>(saved, SL.h13);
  const uint16_t* act = at<uint16_t>(saved, SL.act);
  uint16_t* dh13 = at<uint16_t>(ws, BL.dh13);
  float* dwpart = at<float>(ws, BL.dwpart);
  uint16_t* dxrows = at<uint16_t>(ws, BL.dxrows);
  hipStream_t hs = static_cast<hipStream_t>(stream);
  const uint16_t* dy16 = static_cast<const uint16_t*>(dy);
  const uint16_t* x16 = static_cast<const uint16_t*>(x);

  std::lock_guard<std::mutex> lk(g_timer_mu);
  KernelTimer* tm = timer();
  GemmProblem gp{s->T, s->H, s->I, s->E, s->k, effective_cus(*s, cus), counts, offsets, src_of, topk_w, wrow};
  int32_t* queues = at<int32_t>(ws, BL.queues);
  int32_t* plan13 = queues + kNumQueues;  // split plans of the two weight-gradient GEMMs
  int32_t* plan2 = plan13 + kSplitWords;
  float* partial = at<float>(ws, BL.partial);
  hipError_t e = launch_zero_queues(queues, hs, tm);
  if (e != hipSuccess) return MOE_ERR_LAUNCH;
  const bool wg8 = fp8_wgrad(*s);
  const int64_t Tk = s->T * s->k;
  const int I = int(s->I), H = int(s->H), E = int(s->E), kk = int(s->k), rule = scale_rule(*s);
  if (s->T > 0) {
    GemmOperand gdy{dy, nullptr}, gw2{W2, nullptr}, gdh{dh13, nullptr}, gw13{W13, nullptr};
    if (f8) {
      const moe_wq_layout WL = wq_layout(*s);
      uint8_t* dyq = at<uint8_t>(ws, BL.dyq);
      uint8_t* dys = at<uint8_t>(ws, BL.dys);
      if (wg8 && kk == 1) {
        // each token row occurs once among the expert rows: one pass gives
        // dY's codes along H (for dH) and along the expert rows (for dW2)
        e = launch_quant_tokens(dy16, H, H, counts, offsets, E, Tk, src_of, kk, at<uint8_t>(ws, BL.wgy),
                                at<uint8_t>(ws, BL.wgys), rule, hs, tm, "quant_wg_dy", dyq, dys);
      } else {
        e = launch_quant_rows(dy16, s->T, H, dyq, dys, act_block(*s), rule, hs, tm, "quant_dy");
      }
      if (e != hipSuccess) return MOE_ERR_LAUNCH;
      const bool f32 = f32_scales(*s);
      gdy = GemmOperand{dyq, dys, false, f32};
      gw2 = GemmOperand{at<uint8_t>(wq, WL.w2t), at<uint8_t>(wq, WL.w2t_scale), false, f32};
      gw13 = GemmOperand{at<uint8_t>(wq, WL.w13t), at<uint8_t>(wq, WL.w13t_scale), false, f32};
    }
    if ((e = launch_gemm_dh(gp, gdy, gw2, h13, dh13, dwpart, hs, tm)) != hipSuccess) return MOE_ERR_LAUNCH;
    if (f8) {
      uint8_t* dhq = at<uint8_t>(ws, BL.dhq);
      uint8_t* dhs = at<uint8_t>(ws, BL.dhs);
      if (wg8)  // [dg | du] along 2I (for dX) and along the expert rows (for dW13) in one pass
        e = launch_quant_tokens(dh13, 2 * I, 2 * I, counts, offsets, E, Tk, nullptr, 1, at<uint8_t>(ws, BL.wgd),
                                at<uint8_t>(ws, BL.wgds), rule, hs, tm, "quant_wg_dh13", dhq, dhs);
      else
        e = launch_quant_rows(dh13, Tk, 2 * I, dhq, dhs, act_block(*s), rule, hs, tm, "quant_dh13");
      if (e != hipSuccess) return MOE_ERR_LAUNCH;
      gdh = GemmOperand{dhq, dhs, false, f32_scales(*s)};
    }
    const bool direct = s->k == 1;  // top-1: dX rows go straight to dx
    if ((e = launch_gemm_dx(gp, gdh, gw13, direct ? static_cast<uint16_t*>(dx) : dxrows, hs, tm)) != hipSuccess)
      return MOE_ERR_LAUNCH;
    if ((e = launch_combine(direct ? nullptr : dxrows, row_of, s->T, int(s->k), s->H, static_cast<uint16_t*>(dx), dwpart,
                            dh_num_parts(s->I), d_topk_w, hs, tm, "combine_dx_dw")) != hipSuccess)
      return MOE_ERR_LAUNCH;
  }
  if (wg8) {
    // [dg | du] (and, for top-1, dY) were quantized along the expert rows
    // above; with no tokens every expert is empty and no operand is read
    uint8_t* wgd = at<uint8_t>(ws, BL.wgd);
    uint8_t* wgds = at<uint8_t>(ws, BL.wgds);
    uint8_t* wgx = at<uint8_t>(ws, BL.wgx);
    uint8_t* wgxs = at<uint8_t>(ws, BL.wgxs);
    uint8_t* wgy = at<uint8_t>(ws, BL.wgy);
    uint8_t* wgys = at<uint8_t>(ws, BL.wgys);
    uint8_t* wga = at<uint8_t>(ws, BL.wga);
    uint8_t* wgas = at<uint8_t>(ws, BL.wgas);
    if ((e = launch_quant_tokens(x16, H, H, counts, offsets, E, Tk, src_of, kk, wgx, wgxs, rule, hs, tm,
                                 "quant_wg_x")) != hipSuccess ||
        (e = launch_gemm_dw_fp8(gp, wgd, wgds, 2 * I, wgx, wgxs, H, static_cast<uint16_t*>(dW13), queues, partial,
                                plan13, hs, tm, "gemm_dw13_fp8", "dw13_split_sum")) != hipSuccess)
      return MOE_ERR_LAUNCH;
    if (kk != 1 && (e = launch_quant_tokens(dy16, H, H, counts, offsets, E, Tk, src_of, kk, wgy, wgys, rule, hs,
                                            tm, "quant_wg_dy")) != hipSuccess)
      return MOE_ERR_LAUNCH;
    if ((e = launch_quant_tokens(act, I, I, counts, offsets, E, Tk, nullptr, 1, wga, wgas, rule, hs, tm,
                                 "quant_wg_act")) != hipSuccess)
      return MOE_ERR_LAUNCH;
    e = launch_gemm_dw_fp8(gp, wgy, wgys, H, wga, wgas, I, static_cast<uint16_t*>(dW2), queues + kQueuesPerGemm, partial,
                           plan2, hs, tm, "gemm_dw2_fp8", "dw2_split_sum");
    return launch_status(e);
  }
  if ((e = launch_gemm_dw13(gp, dh13, x16, static_cast<uint16_t*>(dW13), queues, partial, plan13, hs, tm)) !=
      hipSuccess)
    return MOE_ERR_LAUNCH;
  e = launch_gemm_dw2(gp, dy16, act, static_cast<uint16_t*>(dW2), queues + kQueuesPerGemm, partial, plan2, hs, tm);
  return launch_status(e);
}

moe_status moe_route(const moe_shape* s, const float* logits, int32_t renorm, int32_t* topk_idx, float* topk_w,
                     void* stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  if (s->T == 0) return MOE_OK;
  if (!logits || !topk_idx || !topk_w) return MOE_ERR_NULL;
  int cus = 0;
  if ((st = device_info(&cus)) != MOE_OK) return st;
  std::lock_guard<std::mutex> lk(g_timer_mu);
  return launch_status(launch_route(logits, s->T, int(s->E), int(s->k), renorm != 0, topk_idx, topk_w,
                                    static_cast<hipStream_t>(stream), timer()));
}

moe_status moe_route_bwd(const moe_shape* s, const float* logits, const int32_t* topk_idx, const float* topk_w,
                         const float* d_topk_w, int32_t renorm, float* d_logits, void* stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  if (s->T == 0) return MOE_OK;
  if (!logits || !topk_idx || !topk_w || !d_topk_w || !d_logits) return MOE_ERR_NULL;
  int cus = 0;
  if ((st = device_info(&cus)) != MOE_OK) return st;
  std::lock_guard<std::mutex> lk(g_timer_mu);
  return launch_status(launch_route_bwd(logits, s->T, int(s->E), int(s->k), renorm != 0, topk_idx, topk_w, d_topk_w,
                                        d_logits, static_cast<hipStream_t>(stream), timer()));
}

size_t moe_balance_scratch_bytes(const moe_shape* s, int64_t S) {
  if (check_shape(s) != MOE_OK || !sequences_fit(*s, S)) return 0;
  return balance_scratch_bytes(s->T, int(s->E), S);
}

moe_status moe_balance(const moe_shape* s, const float* logits, const int32_t* topk_idx, const int32_t* seq_offsets,
                       int64_t S, const uint8_t* mask, float* loss, int32_t* counts, int32_t* seq_counts,
                       float* seq_probs, float* seq_scale, void* ws, size_t ws_bytes, void* stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  if ((st = check_sequences(*s, seq_offsets, S)) != MOE_OK) return st;
  if (!loss || !counts || !seq_counts || !seq_probs || !seq_scale || !ws) return MOE_ERR_NULL;
  if (s->T > 0 && (!logits || !topk_idx)) return MOE_ERR_NULL;
  for (const void* p : {static_cast<const void*>(logits), static_cast<const void*>(topk_idx),
                        static_cast<const void*>(seq_offsets), static_cast<const void*>(loss),
                        static_cast<const void*>(counts), static_cast<const void*>(seq_counts),
                        static_cast<const void*>(seq_probs), static_cast<const void*>(seq_scale)})
    if (!aligned4(p)) return MOE_ERR_ALIGN;
  if (!aligned16(ws)) return MOE_ERR_ALIGN;
  if (ws_bytes < balance_scratch_bytes(s->T, int(s->E), S)) return MOE_ERR_WORKSPACE;
  int cus = 0;
  if ((st = device_info(&cus)) != MOE_OK) return st;
  std::lock_guard<std::mutex> lk(g_timer_mu);
  return launch_status(launch_balance(BalanceArgs{logits, topk_idx, s->T, int(s->E), int(s->k), seq_offsets, S, mask},
                                      loss, counts, seq_counts, seq_probs, seq_scale, ws,
                                      static_cast<hipStream_t>(stream), timer()));
}

moe_status moe_balance_bwd(const moe_shape* s, const float* logits, const int32_t* topk_idx, const float* topk_w,
                           const float* d_topk_w, int32_t renorm, const int32_t* seq_offsets, int64_t S,
                           const uint8_t* mask, const int32_t* seq_counts, const float* seq_scale,
                           const float* d_loss, float* d_logits, void* stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  if ((st = check_sequences(*s, seq_offsets, S)) != MOE_OK) return st;
  if (s->T == 0) return MOE_OK;
  if (!logits || !seq_counts || !seq_scale || !d_loss || !d_logits) return MOE_ERR_NULL;
  if (d_topk_w && (!topk_idx || !topk_w)) return MOE_ERR_NULL;
  for (const void* p : {static_cast<const void*>(logits), static_cast<const void*>(topk_idx),
                        static_cast<const void*>(topk_w), static_cast<const void*>(d_topk_w),
                        static_cast<const void*>(seq_offsets), static_cast<const void*>(seq_counts),
                        static_cast<const void*>(seq_scale), static_cast<const void*>(d_loss),
                        static_cast<const void*>(d_logits)})
    if (!aligned4(p)) return MOE_ERR_ALIGN;
  int cus = 0;
  if ((st = device_info(&cus)) != MOE_OK) return st;
  std::lock_guard<std::mutex> lk(g_timer_mu);
  return launch_status(launch_balance_bwd(
      BalanceArgs{logits, topk_idx, s->T, int(s->E), int(s->k), seq_offsets, S, mask}, topk_w, d_topk_w, renorm != 0,
      seq_counts, seq_scale, d_loss, d_logits, static_cast<hipStream_t>(stream), timer()));
}

moe_status moe_ortho_workspace_size(const moe_ortho_shape* s, size_t* ws_bytes) {
  const moe_status st = check_ortho(s);
  if (st != MOE_OK) return st;
  if (!ws_bytes) return MOE_ERR_NULL;
  *ws_bytes = ortho_workspace_bytes(ortho_args(*s));
  return MOE_OK;
}

moe_status moe_orthogonalize(const moe_ortho_shape* s, const void* G, void* U, void* ws, size_t ws_bytes,
                             void* stream) {
  moe_status st = check_ortho(s);
  if (st != MOE_OK) return st;
  if (s->E == 0) return MOE_OK;
  if (!G || !U || !ws) return MOE_ERR_NULL;
  if (!aligned16(G) || !aligned16(U) || !aligned16(ws)) return MOE_ERR_ALIGN;
  const OrthoArgs a = ortho_args(*s);
  if (ws_bytes < ortho_workspace_bytes(a)) return MOE_ERR_WORKSPACE;
  int cus = 0;
  if ((st = device_info(&cus)) != MOE_OK) return st;
  OrthoTarget t{};
  t.grad = G;
  t.U = static_cast<uint16_t*>(U);
  std::lock_guard<std::mutex> lk(g_timer_mu);
  return launch_status(launch_ortho(a, t, ws, static_cast<hipStream_t>(stream), timer()));
}

moe_status moe_muon_step(const moe_ortho_shape* s, const moe_muon_params* p, const void* grad, float* momentum,
                         void* W, float* master, void* ws, size_t ws_bytes, void* stream) {
  moe_status st = check_ortho(s);
  if (st != MOE_OK) return st;
  if (!p) return MOE_ERR_NULL;
  if (!std::isfinite(p->lr) || !std::isfinite(p->mu) || p->mu < 0.f || p->mu >= 1.f || !std::isfinite(p->weight_decay) ||
      !std::isfinite(p->scale) || p->reserved != 0)
    return MOE_ERR_SHAPE;
  if (!std::isfinite(p->lr * p->scale) || !std::isfinite(p->lr * p->weight_decay)) return MOE_ERR_SHAPE;
  if (s->E == 0) return MOE_OK;
  if (!grad || !momentum || !W || !ws) return MOE_ERR_NULL;
  if (!aligned16(grad) || !aligned16(momentum) || !aligned16(W) || !aligned16(master) || !aligned16(ws))
    return MOE_ERR_ALIGN;
  const OrthoArgs a = ortho_args(*s);
  if (ws_bytes < ortho_workspace_bytes(a)) return MOE_ERR_WORKSPACE;
  int cus = 0;
  if ((st = device_info(&cus)) != MOE_OK) return st;
  OrthoTarget t{};
  t.grad = grad;
  t.momentum = momentum;
  t.mu = p->mu;
  t.nesterov = p->nesterov != 0;
  t.W = static_cast<uint16_t*>(W);
  t.master = master;
  t.keep = 1.f - p->lr * p->weight_decay;
  t.step = p->lr * p->scale;
  std::lock_guard<std::mutex> lk(g_timer_mu);
  return launch_status(launch_ortho(a, t, ws, static_cast<hipStream_t>(stream), timer()));
}

moe_status moe_gate(const moe_shape* s, const moe_gate_params* p, const float* logits, const float* bias,
                    const uint8_t* mask, int32_t* topk_idx, float* topk_w, void* stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  if ((st = check_gate(*s, p)) != MOE_OK) return st;
  if (s->T == 0) return MOE_OK;
  if (!logits || !topk_idx || !topk_w) return MOE_ERR_NULL;
  if (!aligned4(logits) || !aligned4(bias) || !aligned4(topk_idx) || !aligned4(topk_w)) return MOE_ERR_ALIGN;
  int cus = 0;
  if ((st = device_info(&cus)) != MOE_OK) return st;
  std::lock_guard<std::mutex> lk(g_timer_mu);
  return launch_status(launch_gate(gate_args(*s, *p, logits, bias, mask), topk_idx, topk_w,
                                   static_cast<hipStream_t>(stream), timer()));
}

moe_status moe_gate_bwd(const moe_shape* s, const moe_gate_params* p, const float* logits, const int32_t* topk_idx,
                        const float* d_topk_w, int32_t accumulate, float* d_logits, void* stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  if ((st = check_gate(*s, p)) != MOE_OK) return st;
  if (s->T == 0) return MOE_OK;
  if (!logits || !topk_idx || !d_topk_w || !d_logits) return MOE_ERR_NULL;
  if (!aligned4(logits) || !aligned4(topk_idx) || !aligned4(d_topk_w) || !aligned4(d_logits)) return MOE_ERR_ALIGN;
  int cus = 0;
  if ((st = device_info(&cus)) != MOE_OK) return st;
  std::lock_guard<std::mutex> lk(g_timer_mu);
  return launch_status(launch_gate_bwd(gate_args(*s, *p, logits, nullptr, nullptr), topk_idx, d_topk_w, accumulate != 0,
                                       d_logits, static_cast<hipStream_t>(stream), timer()));
}

moe_status moe_linear_workspace_size(const moe_linear_shape* s, size_t* fwd_ws, size_t* bwd_ws) {
  const moe_status st = check_linear(s);
  if (st != MOE_OK) return st;
  if (fwd_ws) *fwd_ws = linear_workspace_bytes(linear_args(*s), false);
  if (bwd_ws) *bwd_ws = linear_workspace_bytes(linear_args(*s), true);
  return MOE_OK;
}

moe_status moe_linear(const moe_linear_shape* s, const void* X, const void* W, const float* bias, const void* residual,
                      void* Y, void* pre, void* ws, size_t ws_bytes, void* stream) {
  moe_status st = check_linear(s);
  if (st != MOE_OK) return st;
  if (s->M == 0) return MOE_OK;
  const LinearArgs a = linear_args(*s);
  const size_t need = linear_workspace_bytes(a, false);
  if (!X || !W || !Y || (need > 0 && !ws)) return MOE_ERR_NULL;
  for (const void* p : {X, W, static_cast<const void*>(bias), residual, static_cast<const void*>(Y),
                        static_cast<const void*>(pre), static_cast<const void*>(ws)})
    if (!aligned16(p)) return MOE_ERR_ALIGN;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE;
  int cus = 0;
  if ((st = device_info(&cus)) != MOE_OK) return st;
  std::lock_guard<std::mutex> lk(g_timer_mu);
  return launch_status(launch_linear(a, static_cast<const uint16_t*>(X), static_cast<const uint16_t*>(W), bias, residual,
                                     Y, static_cast<uint16_t*>(pre), ws, static_cast<hipStream_t>(stream), timer()));
}

moe_status moe_linear_bwd(const moe_linear_shape* s, const void* dY, const void* X, const void* W, const void* pre,
                          void* dX, void* dW, float* dbias, void* ws, size_t ws_bytes, void* stream) {
  moe_status st = check_linear(s);
  if (st != MOE_OK) return st;
  if (!dX && !dW && !dbias) return MOE_OK;
  const LinearArgs a = linear_args(*s);
  const size_t need = linear_workspace_bytes(a, true);
  if (s->M > 0) {
    if (!dY || (dW && !X) || (dX && !W) || (s->act != MOE_ACT_NONE && !pre) || (need > 0 && !ws)) return MOE_ERR_NULL;
    if (ws_bytes < need) return MOE_ERR_WORKSPACE;
  }
  for (const void* p : {dY, X, W, pre, static_cast<const void*>(dX), static_cast<const void*>(dW),
                        static_cast<const void*>(dbias), static_cast<const void*>(ws)})
    if (!aligned16(p)) return MOE_ERR_ALIGN;
  int cus = 0;
  if ((st = device_info(&cus)) != MOE_OK) return st;
  std::lock_guard<std::mutex> lk(g_timer_mu);
  return launch_status(launch_linear_bwd(a, dY, static_cast<const uint16_t*>(X), static_cast<const uint16_t*>(W),
                                         static_cast<const uint16_t*>(pre), static_cast<uint16_t*>(dX),
                                         static_cast<uint16_t*>(dW), dbias, ws, static_cast<hipStream_t>(stream),
                                         timer()));
}

moe_status moe_adamw_step(const moe_adamw_params* p, const moe_adamw_tensor* tensors, int64_t count,
                          const float* grad_scale, const float* hyper, void* stream) {
  if (!p) return MOE_ERR_NULL;
  if ((p->param_dtype != MOE_DT_BF16 && p->param_dtype != MOE_DT_F32) ||
      (p->grad_dtype != MOE_DT_BF16 && p->grad_dtype != MOE_DT_F32) ||
      (p->state != MOE_STATE_F32 && p->state != MOE_STATE_8BIT))
    return MOE_ERR_PRECISION;
  const double most = 3.4028234e38;  // of fp32, and false for NaN
  // the kernel takes a reciprocal, which knows no numbers below the normal range: a smaller eps would
  // make 0 / eps a NaN, a larger one every update 0
  const float eps = float(p->eps);
  const bool eps_ok = p->eps == 0.0 || (eps >= 0x1p-126f && eps <= 0x1p+100f);
  if (!(std::fabs(p->lr) <= most) || !eps_ok || !(std::fabs(p->weight_decay) <= most) ||
      !(std::fabs(p->lr * p->weight_decay) <= most))
    return MOE_ERR_SHAPE;
  const double below = 1.0 - 0x1p-24;  // what rounds to 1 in fp32 is no average
  if (!(p->beta1 >= 0.0 && p->beta1 < below && p->beta2 >= 0.0 && p->beta2 < below)) return MOE_ERR_SHAPE;
  if (p->step < 1 || p->reserved != 0 || count < 0) return MOE_ERR_SHAPE;
  if (count == 0) return MOE_OK;
  if (!tensors) return MOE_ERR_NULL;
  if (!aligned4(grad_scale) || !aligned4(hyper)) return MOE_ERR_ALIGN;
  if (hyper && grad_scale) return MOE_ERR_SHAPE;
  AdamwArgs a;
  a.param_bf16 = p->param_dtype == MOE_DT_BF16;
  a.grad_bf16 = p->grad_dtype == MOE_DT_BF16;
  a.eight = p->state == MOE_STATE_8BIT;
  for (int64_t i = 0; i < count; ++i) {
    const moe_adamw_tensor& t = tensors[i];
    if (t.n < 0 || t.n >= (int64_t(1) << 40) || !std::isfinite(t.lr_mul) || !std::isfinite(t.decay_mul)) return MOE_ERR_SHAPE;
    if (t.master && !a.param_bf16) return MOE_ERR_SHAPE;
    if (t.n == 0) continue;
    if (!t.param || !t.grad || !t.m || !t.v || a.eight != (t.m_scale != nullptr) || a.eight != (t.v_scale != nullptr))
      return MOE_ERR_NULL;
    if (!aligned_to(t.param, a.param_bf16 ? 2 : 4) || !aligned_to(t.grad, a.grad_bf16 ? 2 : 4) || !aligned4(t.master) ||
        !aligned_to(t.m, a.eight ? 1 : 4) || !aligned_to(t.v, a.eight ? 1 : 4))
      return MOE_ERR_ALIGN;
  }
  const double t = double(p->step);
  a.h.lr = float(p->lr);
  a.h.beta1 = float(p->beta1);
  a.h.beta2 = float(p->beta2);
  a.h.alpha1 = float(1.0 - p->beta1);
  a.h.alpha2 = float(1.0 - p->beta2);
  a.h.eps = eps;
  a.h.weight_decay = float(p->weight_decay);
  a.h.bias1 = float(1.0 - std::pow(p->beta1, t));
  a.h.root2 = float(1.0 / std::sqrt(1.0 - std::pow(p->beta2, t)));
  a.grad_scale = grad_scale;
  a.hyper = hyper;
  int cus = 0;
  moe_status st;
  if ((st = device_info(&cus)) != MOE_OK) return st;
  static_assert(sizeof(AdamwTensor) == sizeof(moe_adamw_tensor), "the launcher takes the tensors as they are");
  std::lock_guard<std::mutex> lk(g_timer_mu);
  return launch_status(launch_adamw(a, reinterpret_cast<const AdamwTensor*>(tensors), count,
                                    static_cast<hipStream_t>(stream), timer()));
}

moe_status moe_read_status(const void* fwd_ws, int32_t* out, void* stream) {
  if (!fwd_ws || !out) return MOE_ERR_NULL;
  hipStream_t hs = static_cast<hipStream_t>(stream);
  if (hipMemcpyAsync(out, fwd_ws, sizeof(int32_t), hipMemcpyDeviceToHost, hs) != hipSuccess)
    return MOE_ERR_LAUNCH;
  if (hipStreamSynchronize(hs) != hipSuccess) return MOE_ERR_LAUNCH;
  return MOE_OK;
}

moe_status moe_set_kernel_timing(int enable) {
  std::lock_guard<std::mutex> lk(g_timer_mu);
  g_timing = enable != 0;
  return MOE_OK;
}

moe_status moe_kernel_timing_collect(moe_kernel_time* out, int32_t max, int32_t* n_out) {
  std::lock_guard<std::mutex> lk(g_timer_mu);
  std::vector<moe_kernel_time> agg;
  moe_status st = MOE_OK;
  for (auto& r : g_timer.recs) {
    float ms = 0.f;
    if (!r.a || !r.b || hipEventSynchronize(r.b) != hipSuccess ||
        hipEventElapsedTime(&ms, r.a, r.b) != hipSuccess) {
      st = MOE_ERR_LAUNCH;
    }
    size_t i = 0;
    for (; i < agg.size(); ++i)
      if (r.name == agg[i].name) break;
    if (i == agg.size()) {
      moe_kernel_time kt;
      std::memset(&kt, 0, sizeof(kt));
      std::strncpy(kt.name, r.name.c_str(), sizeof(kt.name) - 1);
      agg.push_back(kt);
    }
    agg[i].launches += 1;
    agg[i].total_ms += ms;
    if (r.a) g_timer.pool.push_back(r.a);
    if (r.b) g_timer.pool.push_back(r.b);
  }
  g_timer.recs.clear();
  int32_t n = 0;
  for (size_t i = 0; i < agg.size() && n < max; ++i) out[n++] = agg[i];
  if (n_out) *n_out = n;
  return st;
}

}  // extern "C"
