// Drives the host checks of linear attention and of the norms and rotation before
// it under the sanitizers: one line "call short" a case, where `short` is the index
// of the buffer that is one byte too small (-1: none).  Prints each check's status
// and the number of its buffers.
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <vector>

#include "kda.h"
#include "kda_layer.h"
#include "kda_validate.h"

namespace {
int g_short = -1, g_next = 0;
uint8_t* fake() { return reinterpret_cast<uint8_t*>(uintptr_t(1) << 20) + (uintptr_t(g_next) << 40); }
size_t bytes(size_t need) { return need - (g_next++ == g_short ? 1 : 0); }
kda::Rows rows(size_t need, int64_t stride = 0) {
  uint8_t* p = fake();
  return {p, bytes(need), stride};
}
kda::Dst dst(size_t need) {
  uint8_t* p = fake();
  return {p, bytes(need)};
}

int rotate(bool backward, int32_t T, int32_t Hq, int32_t Hk, int32_t D, int32_t R, int32_t dtype, int64_t pad) {
  kda::RotateArgs a{};
  a.T = T, a.Hq = Hq, a.Hk = Hk, a.D = D, a.R = R, a.dtype = dtype, a.d_format = KDA_FP32, a.q_scale = 1.f, a.eps = 1e-6f;
  const size_t e = dtype == KDA_BF16 ? 2 : 4, t = size_t(T), nq = size_t(Hq) * D, nk = size_t(Hk) * D;
  a.q_raw = rows(((t - 1) * (nq + pad) + nq) * e, int64_t(nq) + pad);
  a.k_raw = rows(((t - 1) * (nk + pad) + nk) * e, int64_t(nk) + pad);
  a.positions = rows(t * 4), a.inv_freq = rows(size_t(R) / 2 * 4);
  a.q_weight = rows(size_t(D) * 4), a.k_weight = rows(size_t(D) * 4);
  a.q = dst(t * nq * e), a.k = dst(t * nk * e);
  if (backward) {
    a.dq = rows(t * nq * 4), a.dk = rows(t * nk * 4);
    a.dq_weight = dst(size_t(D) * 4), a.dk_weight = dst(size_t(D) * 4);
    a.workspace = dst(kda::rotate_bwd_workspace(T, D));
  }
  return kda::check_rotate(a, backward);
}

int linear(bool backward, const std::vector<int32_t>& cu, int32_t segments, int32_t H, int32_t Hq, int32_t K, int32_t V,
           int32_t g_dtype, int32_t format, bool fixed) {
  kda_plan* plan = nullptr;
  if (kda_plan_segments(cu.data(), int32_t(cu.size()) - 1, segments, nullptr, &plan) != KDA_OK) return 1;
  kda::LinearArgs a{};
  a.plan = plan, a.H = a.Hv = H, a.Hq = a.Hk = Hq, a.K = K, a.V = V, a.g_dtype = g_dtype, a.o_format = format;
  const size_t T = size_t(plan->T), e = format == KDA_BF16 ? 2 : 4, eg = g_dtype == KDA_BF16 ? 2 : 4, nq = size_t(Hq) * K,
               nv = size_t(H) * V, state = size_t(plan->N) * H * K * V * 4, ng = fixed ? size_t(H) : T * H;
  a.plan_dev = rows(plan->blob.size() * 4);
  a.q = rows(((T - 1) * (nq + 16) + nq) * 2, int64_t(nq) + 16);
  a.k = rows(T * nq * 2, int64_t(nq));
  a.v = rows(T * nv * 2, int64_t(nv));
  a.g = rows(ng * eg, fixed ? 0 : H);
  a.initial_state = rows(state);
  if (!backward) {
    a.o = dst(T * nv * e), a.final_state = dst(state);
  } else {
    a.d_o = rows(T * nv * 2), a.d_final = rows(state);
    a.dq = dst(T * nq * e), a.dk = dst(T * nq * e), a.dv = dst(T * nv * e), a.dg = dst(ng * eg);
    a.d_initial_state = dst(state);
  }
  const size_t ws = backward ? kda::linear_bwd_layout(a).total : kda::linear_layout(plan, H, K, V).total;
  if (ws > 0) a.workspace = dst(ws);
  const int st = kda::check_linear(a, backward);
  kda_plan_destroy(plan);
  return st;
}

int step(int32_t B, int32_t H, int32_t Hk, int32_t K, int32_t V, int32_t slots, int32_t o_format, bool fixed) {
  kda::LinearStepArgs a{};
  a.B = B, a.H = a.Hq = a.Hv = H, a.Hk = Hk, a.K = K, a.V = V, a.g_dtype = KDA_FP32, a.o_format = o_format, a.num_slots = slots;
  const size_t b = size_t(B), pool = size_t(slots) * H * K * V * 4;
  a.q = rows(b * H * K * 2), a.k = rows(b * Hk * K * 2), a.v = rows(b * H * V * 2);
  a.g = rows((fixed ? size_t(H) : b * H) * 4, fixed ? 0 : H);
  a.slots = rows(b * 4), a.state = rows(pool);
  a.state_out = dst(pool), a.o = dst(b * H * V * (o_format == KDA_BF16 ? 2 : 4));
  return kda::check_linear_step(a);
}
}  // namespace

int main() {
  char call[32];
  while (std::scanf("%31s %d", call, &g_short) == 2) {
    g_next = 0;
    int st = 1;
    if (!std::strcmp(call, "rotate")) st = rotate(false, 7, 5, 2, 96, 32, KDA_BF16, 8);
    if (!std::strcmp(call, "rotate_one")) st = rotate(false, 1, 1, 1, 8, 2, KDA_FP32, 0);
    if (!std::strcmp(call, "rotate_most")) st = rotate(false, 1 << 30, 1, 1, 256, 256, KDA_BF16, 1 << 20);
    if (!std::strcmp(call, "rotate_bwd")) st = rotate(true, 7, 5, 2, 96, 32, KDA_FP32, 8);
    if (!std::strcmp(call, "linear")) st = linear(false, {0, 7, 64, 300}, 3, 6, 2, 64, 40, KDA_FP32, KDA_BF16, false);
    if (!std::strcmp(call, "linear_uncut")) st = linear(false, {0, 1}, 1, 1, 1, 8, 8, KDA_BF16, KDA_FP32, true);
    if (!std::strcmp(call, "linear_most")) st = linear(false, {0, 1 << 30}, 16384, 16384, 4, 128, 128, KDA_FP32, KDA_FP32, false);
    if (!std::strcmp(call, "linear_bwd")) st = linear(true, {0, 7, 64, 300}, 3, 6, 2, 64, 40, KDA_BF16, KDA_FP32, false);
    if (!std::strcmp(call, "linear_bwd_fixed")) st = linear(true, {0, 5, 70}, 1, 3, 3, 128, 128, KDA_FP32, KDA_BF16, true);
    if (!std::strcmp(call, "step")) st = step(5, 6, 3, 64, 40, 9, KDA_BF16, false);
    if (!std::strcmp(call, "step_fixed")) st = step(1, 65535, 1, 128, 128, 1 << 7, KDA_FP32, true);
    std::printf("%d %d\n", st, g_next);
  }
  return 0;
}
