// Drives the host checks of the operators around the recurrence under the
// sanitizers: one line "call short" a case, where `short` is the index of the
// buffer that is one byte too small (-1: none).  Prints each check's status.
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <vector>

#include "kda.h"
#include "kda_layer.h"
#include "kda_validate.h"

namespace {
int g_short = -1, g_next = 0;
uint8_t* fake() { return reinterpret_cast<uint8_t*>(uintptr_t(1) << 20) + (uintptr_t(g_next) << 36); }
size_t bytes(size_t need) { return need - (g_next++ == g_short ? 1 : 0); }
kda::Rows rows(size_t need, int64_t stride = 0) {
  uint8_t* p = fake();
  return {p, bytes(need), stride};
}
kda::Dst dst(size_t need) {
  uint8_t* p = fake();
  return {p, bytes(need)};
}

int prepare(bool backward, int32_t T, int32_t H, int32_t dtype, int64_t pad) {
  kda::PrepareArgs a{};
  a.T = T, a.H = H, a.K = 128, a.dtype = dtype, a.q_scale = 1.f, a.eps = 1e-6f;
  const size_t e = dtype == KDA_BF16 ? 2 : 4, row = size_t(H) * 128, t = size_t(T), o = backward ? e : 2;
  const int64_t s = int64_t(row) + pad;
  a.q_raw = rows(((t - 1) * s + row) * e, s);
  a.k_raw = rows(((t - 1) * s + row) * e, s);
  a.gate_raw = rows(((t - 1) * s + row) * e, s);
  a.beta_raw = rows(((t - 1) * (H + 3) + H) * e, H + 3);
  a.a_log = rows(size_t(H) * 4);
  a.dt_bias = rows(row * 4);
  a.q = dst(t * row * o), a.k = dst(t * row * o), a.g = dst(t * row * o), a.beta = dst(t * H * o);
  if (backward) {
    a.dq = rows(t * row * 4), a.dk = rows(t * row * 4), a.dg = rows(t * row * 4), a.dbeta = rows(t * H * 4);
    a.da_log = dst(size_t(H) * 4), a.ddt_bias = dst(row * 4);
    a.workspace = dst(kda::prepare_bwd_layout(T, H).total);
  }
  return kda::check_prepare(a, backward);
}

int norm(bool backward, int32_t T, int32_t H, int32_t V, int32_t dtype, int32_t o_format, int64_t pad) {
  kda::NormArgs a{};
  a.T = T, a.H = H, a.V = V, a.dtype = dtype, a.o_format = o_format, a.d_o_format = KDA_FP32;
  a.activation = KDA_ACT_SILU, a.eps = 1e-6f;
  const size_t e = dtype == KDA_BF16 ? 2 : 4, eo = o_format == KDA_BF16 ? 2 : 4, row = size_t(H) * V, n = row * T;
  const int64_t s = int64_t(row) + pad;
  a.o = rows(n * eo);
  a.gate = rows(((size_t(T) - 1) * s + row) * e, s);
  a.weight = rows(size_t(V) * 4);
  a.res_scale = rows(row * 4);
  if (!backward) {
    a.residual = rows(n * e);
    a.y = dst(n * e);
  } else {
    a.dy = rows(n * e);
    a.d_o = dst(n * 4), a.d_gate = dst(n * e), a.d_weight = dst(size_t(V) * 4), a.d_res_scale = dst(row * 4);
    a.workspace = dst(kda::norm_bwd_workspace(T, H, V));
  }
  return kda::check_norm(a, backward);
}

int scan(bool backward, const std::vector<int32_t>& cu, int32_t D, int32_t dtype, int32_t h_format) {
  kda_plan* plan = nullptr;
  if (kda_plan_segments(cu.data(), int32_t(cu.size()) - 1, 2, nullptr, &plan) != KDA_OK) return 1;
  kda::ScanArgs a{};
  a.plan = plan, a.D = D, a.dtype = dtype, a.h_format = h_format, a.tied = 1;
  const size_t e = dtype == KDA_BF16 ? 2 : 4, eh = h_format == KDA_BF16 ? 2 : 4, T = size_t(plan->T), n = T * D,
               state = size_t(plan->N) * D * 4;
  a.plan_dev = rows(plan->blob.size() * 4);
  a.x = rows(((T - 1) * (D + 5) + D) * e, D + 5);
  a.g = rows(n * e, D);
  a.initial_state = rows(state);
  if (!backward) {
    a.h = dst(n * eh), a.final_state = dst(state);
  } else {
    a.h_in = rows(n * eh), a.dh = rows(n * eh), a.d_final = rows(state);
    a.dx = dst(n * e), a.dg = dst(n * e), a.d_initial_state = dst(state);
  }
  const size_t ws = kda::scan_layout(plan->T, D).total;
  if (ws > 0) a.workspace = dst(ws);
  const int st = kda::check_scan(a, backward);
  kda_plan_destroy(plan);
  return st;
}

int scan_step(int32_t B, int32_t D, int32_t slots, int32_t dtype) {
  kda::ScanStepArgs a{};
  a.B = B, a.D = D, a.dtype = dtype, a.num_slots = slots;
  const size_t n = size_t(B) * D * (dtype == KDA_BF16 ? 2 : 4), pool = size_t(slots) * D * 4;
  a.x = rows(n), a.g = rows(n), a.slots = rows(size_t(B) * 4), a.state = rows(pool);
  a.state_out = dst(pool), a.h = dst(n);
  return kda::check_scan_step(a);
}

int step(int32_t B, int32_t H, int32_t slots, int32_t o_format) {
  kda::StepArgs a{};
  a.B = B, a.H = H, a.K = 128, a.V = 128, a.head_begin = 0, a.head_count = H, a.o_format = o_format, a.num_slots = slots;
  a.gate_lower_bound = -1.f;
  const size_t n = size_t(B) * H * 128, pool = size_t(slots) * H * 65536;
  a.q = rows(n * 2), a.k = rows(n * 2), a.v = rows(n * 2), a.g = rows(n * 2), a.beta = rows(size_t(B) * H * 2);
  a.slots = rows(size_t(B) * 4), a.state = rows(pool);
  a.state_out = dst(pool), a.o = dst(n * (o_format == KDA_BF16 ? 2 : 4));
  return kda::check_step(a);
}
}  // namespace

int main() {
  char call[32];
  while (std::scanf("%31s %d", call, &g_short) == 2) {
    g_next = 0;
    int st = 1;
    if (!std::strcmp(call, "prepare")) st = prepare(false, 7, 5, KDA_BF16, 8);
    if (!std::strcmp(call, "prepare_one")) st = prepare(false, 1, 1, KDA_FP32, 0);
    if (!std::strcmp(call, "prepare_bwd")) st = prepare(true, 7, 5, KDA_FP32, 4);
    if (!std::strcmp(call, "norm")) st = norm(false, 7, 3, 41, KDA_BF16, KDA_FP32, 1);
    if (!std::strcmp(call, "norm_bwd")) st = norm(true, 7, 3, 40, KDA_FP32, KDA_BF16, 0);
    if (!std::strcmp(call, "norm_wide")) st = norm(true, 2, 1, 8192, KDA_BF16, KDA_BF16, 3);
    if (!std::strcmp(call, "scan")) st = scan(false, {0, 3, 300}, 13, KDA_BF16, KDA_FP32);
    if (!std::strcmp(call, "scan_short")) st = scan(false, {0, 3, 10}, 13, KDA_FP32, KDA_BF16);
    if (!std::strcmp(call, "scan_bwd")) st = scan(true, {0, 3, 300}, 64, KDA_FP32, KDA_FP32);
    if (!std::strcmp(call, "scan_step")) st = scan_step(5, 9, 7, KDA_BF16);
    if (!std::strcmp(call, "step")) st = step(5, 2, 7, KDA_BF16);
    std::printf("%d %d\n", st, g_next);
  }
  return 0;
}
