// C-ABI entry points of the operators around the recurrence: each packs its
// arguments, checks them on the host and launches.  An error returns a
// negative kda_status and enqueues nothing.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "kda.h"
#include "kda_layer.h"

extern "C" {

int kda_prepare_inputs(int32_t T, int32_t H, int32_t K, int32_t dtype,
                       const void* q_raw, size_t q_raw_bytes, int64_t q_raw_stride,
                       const void* k_raw, size_t k_raw_bytes, int64_t k_raw_stride,
                       const void* gate_raw, size_t gate_raw_bytes, int64_t gate_raw_stride,
                       const void* beta_raw, size_t beta_raw_bytes, int64_t beta_raw_stride,
                       const float* a_log, size_t a_log_bytes, const float* dt_bias, size_t dt_bias_bytes,
                       float q_scale, float eps,
                       uint16_t* q, size_t q_bytes, uint16_t* k, size_t k_bytes,
                       uint16_t* g, size_t g_bytes, uint16_t* beta, size_t beta_bytes, hipStream_t stream) {
  kda::PrepareArgs a{};
  a.T = T;
  a.H = H;
  a.K = K;
  a.dtype = dtype;
  a.q_raw = {q_raw, q_raw_bytes, q_raw_stride};
  a.k_raw = {k_raw, k_raw_bytes, k_raw_stride};
  a.gate_raw = {gate_raw, gate_raw_bytes, gate_raw_stride};
  a.beta_raw = {beta_raw, beta_raw_bytes, beta_raw_stride};
  a.a_log = {a_log, a_log_bytes, 0};
  a.dt_bias = {dt_bias, dt_bias_bytes, 0};
  a.q_scale = q_scale;
  a.eps = eps;
  a.q = {q, q_bytes};
  a.k = {k, k_bytes};
  a.g = {g, g_bytes};
  a.beta = {beta, beta_bytes};
  const int st = kda::check_prepare(a, false);
  return st != KDA_OK ? st : kda::launch_prepare(a, stream);
}

int kda_prepare_inputs_backward(int32_t T, int32_t H, int32_t K, int32_t dtype,
                                const void* q_raw, size_t q_raw_bytes, int64_t q_raw_stride,
                                const void* k_raw, size_t k_raw_bytes, int64_t k_raw_stride,
                                const void* gate_raw, size_t gate_raw_bytes, int64_t gate_raw_stride,
                                const void* beta_raw, size_t beta_raw_bytes, int64_t beta_raw_stride,
                                const float* a_log, size_t a_log_bytes, const float* dt_bias, size_t dt_bias_bytes,
                                float q_scale, float eps,
                                const float* dq, size_t dq_bytes, const float* dk, size_t dk_bytes,
                                const float* dg, size_t dg_bytes, const float* dbeta, size_t dbeta_bytes,
                                void* dq_raw, size_t dq_raw_bytes, void* dk_raw, size_t dk_raw_bytes,
                                void* dgate_raw, size_t dgate_raw_bytes, void* dbeta_raw, size_t dbeta_raw_bytes,
                                float* da_log, size_t da_log_bytes, float* ddt_bias, size_t ddt_bias_bytes,
                                void* workspace, size_t workspace_bytes, hipStream_t stream) {
  kda::PrepareArgs a{};
  a.T = T;
  a.H = H;
  a.K = K;
  a.dtype = dtype;
  a.q_raw = {q_raw, q_raw_bytes, q_raw_stride};
  a.k_raw = {k_raw, k_raw_bytes, k_raw_stride};
  a.gate_raw = {gate_raw, gate_raw_bytes, gate_raw_stride};
  a.beta_raw = {beta_raw, beta_raw_bytes, beta_raw_stride};
  a.a_log = {a_log, a_log_bytes, 0};
  a.dt_bias = {dt_bias, dt_bias_bytes, 0};
  a.q_scale = q_scale;
  a.eps = eps;
  a.dq = {dq, dq_bytes, 0};
  a.dk = {dk, dk_bytes, 0};
  a.dg = {dg, dg_bytes, 0};
  a.dbeta = {dbeta, dbeta_bytes, 0};
  a.q = {dq_raw, dq_raw_bytes};
  a.k = {dk_raw, dk_raw_bytes};
  a.g = {dgate_raw, dgate_raw_bytes};
  a.beta = {dbeta_raw, dbeta_raw_bytes};
  a.da_log = {da_log, da_log_bytes};
  a.ddt_bias = {ddt_bias, ddt_bias_bytes};
  a.workspace = {workspace, workspace_bytes};
  const int st = kda::check_prepare(a, true);
  return st != KDA_OK ? st : kda::launch_prepare_backward(a, stream);
}

size_t kda_prepare_inputs_backward_workspace_bytes(int32_t T, int32_t H, int32_t K) {
  if (T <= 0 || H <= 0 || H > 65535 || K != 128) return 0;
  return kda::prepare_bwd_layout(T, H).total;
}

int kda_qk_norm_rotate(int32_t T, int32_t Hq, int32_t Hk, int32_t D, int32_t R, int32_t dtype, int32_t interleaved,
                       const void* q_raw, size_t q_raw_bytes, int64_t q_raw_stride,
                       const void* k_raw, size_t k_raw_bytes, int64_t k_raw_stride,
                       const int32_t* positions, size_t positions_bytes,
                       const float* inv_freq, size_t inv_freq_bytes,
                       const float* q_weight, size_t q_weight_bytes, const float* k_weight, size_t k_weight_bytes,
                       float q_scale, float eps, void* q, size_t q_bytes, void* k, size_t k_bytes,
                       hipStream_t stream) {
  kda::RotateArgs a{};
  a.T = T;
  a.Hq = Hq;
  a.Hk = Hk;
  a.D = D;
  a.R = R;
  a.dtype = dtype;
  a.interleaved = interleaved;
  a.q_raw = {q_raw, q_raw_bytes, q_raw_stride};
  a.k_raw = {k_raw, k_raw_bytes, k_raw_stride};
  a.positions = {positions, positions_bytes, 0};
  a.inv_freq = {inv_freq, inv_freq_bytes, 0};
  a.q_weight = {q_weight, q_weight_bytes, 0};
  a.k_weight = {k_weight, k_weight_bytes, 0};
  a.q_scale = q_scale;
  a.eps = eps;
  a.q = {q, q_bytes};
  a.k = {k, k_bytes};
  const int st = kda::check_rotate(a, false);
  return st != KDA_OK ? st : kda::launch_rotate(a, stream);
}

int kda_qk_norm_rotate_backward(int32_t T, int32_t Hq, int32_t Hk, int32_t D, int32_t R, int32_t dtype, int32_t interleaved,
                                const void* q_raw, size_t q_raw_bytes, int64_t q_raw_stride,
                                const void* k_raw, size_t k_raw_bytes, int64_t k_raw_stride,
                                const int32_t* positions, size_t positions_bytes,
                                const float* inv_freq, size_t inv_freq_bytes,
                                const float* q_weight, size_t q_weight_bytes, const float* k_weight, size_t k_weight_bytes,
                                float q_scale, float eps,
                                const void* dq, size_t dq_bytes, const void* dk, size_t dk_bytes, int32_t d_format,
                                void* dq_raw, size_t dq_raw_bytes, void* dk_raw, size_t dk_raw_bytes,
                                float* dq_weight, size_t dq_weight_bytes, float* dk_weight, size_t dk_weight_bytes,
                                void* workspace, size_t workspace_bytes, hipStream_t stream) {
  kda::RotateArgs a{};
  a.T = T;
  a.Hq = Hq;
  a.Hk = Hk;
  a.D = D;
  a.R = R;
  a.dtype = dtype;
  a.interleaved = interleaved;
  a.q_raw = {q_raw, q_raw_bytes, q_raw_stride};
  a.k_raw = {k_raw, k_raw_bytes, k_raw_stride};
  a.positions = {positions, positions_bytes, 0};
  a.inv_freq = {inv_freq, inv_freq_bytes, 0};
  a.q_weight = {q_weight, q_weight_bytes, 0};
  a.k_weight = {k_weight, k_weight_bytes, 0};
  a.q_scale = q_scale;
  a.eps = eps;
  a.dq = {dq, dq_bytes, 0};
  a.dk = {dk, dk_bytes, 0};
  a.d_format = d_format;
  a.q = {dq_raw, dq_raw_bytes};
  a.k = {dk_raw, dk_raw_bytes};
  a.dq_weight = {dq_weight, dq_weight_bytes};
  a.dk_weight = {dk_weight, dk_weight_bytes};
  a.workspace = {workspace, workspace_bytes};
  const int st = kda::check_rotate(a, true);
  return st != KDA_OK ? st : kda::launch_rotate_backward(a, stream);
}

size_t kda_qk_norm_rotate_backward_workspace_bytes(int32_t T, int32_t D) {
  return T <= 0 || D <= 0 || D > 256 ? 0 : kda::rotate_bwd_workspace(T, D);
}

int kda_output_norm(int32_t T, int32_t H, int32_t V, const void* o, size_t o_bytes, int32_t o_format,
                    const void* gate, size_t gate_bytes, int64_t gate_stride, int32_t activation,
                    const float* weight, size_t weight_bytes, const float* res_scale, size_t res_scale_bytes,
                    const void* residual, size_t residual_bytes, int32_t dtype, float eps,
                    void* y, size_t y_bytes, hipStream_t stream) {
  kda::NormArgs a{};
  a.T = T;
  a.H = H;
  a.V = V;
  a.dtype = dtype;
  a.o_format = o_format;
  a.activation = activation;
  a.o = {o, o_bytes, 0};
  a.gate = {gate, gate_bytes, gate_stride};
  a.weight = {weight, weight_bytes, 0};
  a.res_scale = {res_scale, res_scale_bytes, 0};
  a.residual = {residual, residual_bytes, 0};
  a.eps = eps;
  a.y = {y, y_bytes};
  const int st = kda::check_norm(a, false);
  return st != KDA_OK ? st : kda::launch_norm(a, stream);
}

int kda_output_norm_backward(int32_t T, int32_t H, int32_t V, const void* dy, size_t dy_bytes,
                             const void* o, size_t o_bytes, int32_t o_format,
                             const void* gate, size_t gate_bytes, int64_t gate_stride, int32_t activation,
                             const float* weight, size_t weight_bytes,
                             const float* res_scale, size_t res_scale_bytes, int32_t dtype, float eps,
                             void* d_o, size_t d_o_bytes, int32_t d_o_format, void* d_gate, size_t d_gate_bytes,
                             float* d_weight, size_t d_weight_bytes,
                             float* d_res_scale, size_t d_res_scale_bytes,
                             void* workspace, size_t workspace_bytes, hipStream_t stream) {
  kda::NormArgs a{};
  a.T = T;
  a.H = H;
  a.V = V;
  a.dtype = dtype;
  a.o_format = o_format;
  a.activation = activation;
  a.d_o_format = d_o_format;
  a.dy = {dy, dy_bytes, 0};
  a.o = {o, o_bytes, 0};
  a.gate = {gate, gate_bytes, gate_stride};
  a.weight = {weight, weight_bytes, 0};
  a.res_scale = {res_scale, res_scale_bytes, 0};
  a.eps = eps;
  a.d_o = {d_o, d_o_bytes};
  a.d_gate = {d_gate, d_gate_bytes};
  a.d_weight = {d_weight, d_weight_bytes};
  a.d_res_scale = {d_res_scale, d_res_scale_bytes};
  a.workspace = {workspace, workspace_bytes};
  const int st = kda::check_norm(a, true);
  return st != KDA_OK ? st : kda::launch_norm_backward(a, stream);
}

size_t kda_output_norm_backward_workspace_bytes(int32_t T, int32_t H, int32_t V) {
  if (T <= 0 || H <= 0 || H > 65535 || V <= 0 || V > 8192 || static_cast<int64_t>(H) * V > (1 << 24)) return 0;
  return kda::norm_bwd_workspace(T, H, V);
}

int kda_scan_forward(const kda_plan* plan, const int32_t* plan_dev, size_t plan_dev_bytes, int32_t D, int32_t dtype,
                     const void* x, size_t x_bytes, int64_t x_stride, const void* g, size_t g_bytes, int64_t g_stride,
                     int32_t tied, const float* initial_state, size_t initial_state_bytes,
                     void* h, size_t h_bytes, int32_t h_format, float* final_state, size_t final_state_bytes,
                     void* workspace, size_t workspace_bytes, hipStream_t stream) {
  kda::ScanArgs a{};
  a.plan = plan;
  a.plan_dev = {plan_dev, plan_dev_bytes, 0};
  a.D = D;
  a.dtype = dtype;
  a.tied = tied;
  a.h_format = h_format;
  a.x = {x, x_bytes, x_stride};
  a.g = {g, g_bytes, g_stride};
  a.initial_state = {initial_state, initial_state_bytes, 0};
  a.h = {h, h_bytes};
  a.final_state = {final_state, final_state_bytes};
  a.workspace = {workspace, workspace_bytes};
  const int st = kda::check_scan(a, false);
  return st != KDA_OK ? st : kda::launch_scan(a, stream);
}

int kda_scan_backward(const kda_plan* plan, const int32_t* plan_dev, size_t plan_dev_bytes, int32_t D, int32_t dtype,
                      const void* x, size_t x_bytes, int64_t x_stride,
                      const void* g, size_t g_bytes, int64_t g_stride, int32_t tied,
                      const float* initial_state, size_t initial_state_bytes,
                      const void* h, size_t h_bytes, const void* dh, size_t dh_bytes, int32_t h_format,
                      const float* d_final, size_t d_final_bytes,
                      void* dx, size_t dx_bytes, void* dg, size_t dg_bytes,
                      float* d_initial_state, size_t d_initial_state_bytes,
                      void* workspace, size_t workspace_bytes, hipStream_t stream) {
  kda::ScanArgs a{};
  a.plan = plan;
  a.plan_dev = {plan_dev, plan_dev_bytes, 0};
  a.D = D;
  a.dtype = dtype;
  a.tied = tied;
  a.h_format = h_format;
  a.x = {x, x_bytes, x_stride};
  a.g = {g, g_bytes, g_stride};
  a.initial_state = {initial_state, initial_state_bytes, 0};
  a.h_in = {h, h_bytes, 0};
  a.dh = {dh, dh_bytes, 0};
  a.d_final = {d_final, d_final_bytes, 0};
  a.dx = {dx, dx_bytes};
  a.dg = {dg, dg_bytes};
  a.d_initial_state = {d_initial_state, d_initial_state_bytes};
  a.workspace = {workspace, workspace_bytes};
  const int st = kda::check_scan(a, true);
  return st != KDA_OK ? st : kda::launch_scan_backward(a, stream);
}

size_t kda_scan_workspace_bytes(const kda_plan* plan, int32_t D) {
  return plan == nullptr || D <= 0 || D > (1 << 20) ? 0 : kda::scan_layout(plan->T, D).total;
}

int kda_scan_step(int32_t B, int32_t D, int32_t dtype, const void* x, size_t x_bytes, const void* g, size_t g_bytes,
                  int32_t tied, const int32_t* slots, size_t slots_bytes, int32_t num_slots,
                  const float* state, size_t state_bytes, float* state_out, size_t state_out_bytes,
                  void* h, size_t h_bytes, hipStream_t stream) {
  kda::ScanStepArgs a{};
  a.B = B;
  a.D = D;
  a.dtype = dtype;
  a.tied = tied;
  a.num_slots = num_slots;
  a.x = {x, x_bytes, 0};
  a.g = {g, g_bytes, 0};
  a.slots = {slots, slots_bytes, 0};
  a.state = {state, state_bytes, 0};
  a.state_out = {state_out, state_out_bytes};
  a.h = {h, h_bytes};
  const int st = kda::check_scan_step(a);
  return st != KDA_OK ? st : kda::launch_scan_step(a, stream);
}

int kda_step(int32_t B, int32_t H, int32_t K, int32_t V, int32_t head_begin, int32_t head_count,
             const uint16_t* q, size_t q_bytes, const uint16_t* k, size_t k_bytes,
             const uint16_t* v, size_t v_bytes, const uint16_t* g, size_t g_bytes,
             const uint16_t* beta, size_t beta_bytes, float gate_lower_bound,
             const int32_t* slots, size_t slots_bytes, int32_t num_slots,
             const float* state, size_t state_bytes, float* state_out, size_t state_out_bytes,
             void* o, size_t o_bytes, int32_t o_format, hipStream_t stream) {
  kda::StepArgs a{};
  a.B = B;
  a.H = H;
  a.K = K;
  a.V = V;
  a.head_begin = head_begin;
  a.head_count = head_count;
  a.o_format = o_format;
  a.num_slots = num_slots;
  a.q = {q, q_bytes, 0};
  a.k = {k, k_bytes, 0};
  a.v = {v, v_bytes, 0};
  a.g = {g, g_bytes, 0};
  a.beta = {beta, beta_bytes, 0};
  a.gate_lower_bound = gate_lower_bound;
  a.slots = {slots, slots_bytes, 0};
  a.state = {state, state_bytes, 0};
  a.state_out = {state_out, state_out_bytes};
  a.o = {o, o_bytes};
  const int st = kda::check_step(a);
  return st != KDA_OK ? st : kda::launch_step(a, stream);
}

int kda_linear_forward(const kda_plan* plan, const int32_t* plan_dev, size_t plan_dev_bytes, int32_t H, int32_t Hq,
                       int32_t Hk, int32_t Hv, int32_t K, int32_t V, const uint16_t* q, size_t q_bytes, int64_t q_stride,
                       const uint16_t* k, size_t k_bytes, int64_t k_stride, const uint16_t* v, size_t v_bytes, int64_t v_stride,
                       const void* g, size_t g_bytes, int64_t g_stride, int32_t g_dtype,
                       const float* initial_state, size_t initial_state_bytes,
                       void* o, size_t o_bytes, int32_t o_format, float* final_state, size_t final_state_bytes,
                       void* workspace, size_t workspace_bytes, hipStream_t stream) {
  kda::LinearArgs a{};
  a.plan = plan;
  a.plan_dev = {plan_dev, plan_dev_bytes, 0};
  a.H = H;
  a.Hq = Hq;
  a.Hk = Hk;
  a.Hv = Hv;
  a.K = K;
  a.V = V;
  a.g_dtype = g_dtype;
  a.q = {q, q_bytes, q_stride};
  a.k = {k, k_bytes, k_stride};
  a.v = {v, v_bytes, v_stride};
  a.g = {g, g_bytes, g_stride};
  a.initial_state = {initial_state, initial_state_bytes, 0};
  a.o_format = o_format;
  a.o = {o, o_bytes};
  a.final_state = {final_state, final_state_bytes};
  a.workspace = {workspace, workspace_bytes};
  const int st = kda::check_linear(a, false);
  return st != KDA_OK ? st : kda::launch_linear(a, stream);
}

int kda_linear_backward(const kda_plan* plan, const int32_t* plan_dev, size_t plan_dev_bytes, int32_t H, int32_t Hq,
                        int32_t Hk, int32_t Hv, int32_t K, int32_t V, const uint16_t* q, size_t q_bytes, int64_t q_stride,
                        const uint16_t* k, size_t k_bytes, int64_t k_stride, const uint16_t* v, size_t v_bytes, int64_t v_stride,
                        const void* g, size_t g_bytes, int64_t g_stride, int32_t g_dtype,
                        const float* initial_state, size_t initial_state_bytes,
                        const uint16_t* d_o, size_t d_o_bytes, const float* d_final, size_t d_final_bytes,
                        void* dq, size_t dq_bytes, void* dk, size_t dk_bytes, void* dv, size_t dv_bytes,
                        int32_t grad_format, void* dg, size_t dg_bytes,
                        float* d_initial_state, size_t d_initial_state_bytes,
                        void* workspace, size_t workspace_bytes, hipStream_t stream) {
  kda::LinearArgs a{};
  a.plan = plan;
  a.plan_dev = {plan_dev, plan_dev_bytes, 0};
  a.H = H;
  a.Hq = Hq;
  a.Hk = Hk;
  a.Hv = Hv;
  a.K = K;
  a.V = V;
  a.g_dtype = g_dtype;
  a.q = {q, q_bytes, q_stride};
  a.k = {k, k_bytes, k_stride};
  a.v = {v, v_bytes, v_stride};
  a.g = {g, g_bytes, g_stride};
  a.initial_state = {initial_state, initial_state_bytes, 0};
  a.o_format = grad_format;
  a.d_o = {d_o, d_o_bytes, 0};
  a.d_final = {d_final, d_final_bytes, 0};
  a.dq = {dq, dq_bytes};
  a.dk = {dk, dk_bytes};
  a.dv = {dv, dv_bytes};
  a.dg = {dg, dg_bytes};
  a.d_initial_state = {d_initial_state, d_initial_state_bytes};
  a.workspace = {workspace, workspace_bytes};
  const int st = kda::check_linear(a, true);
  return st != KDA_OK ? st : kda::launch_linear_backward(a, stream);
}

size_t kda_linear_workspace_bytes(const kda_plan* plan, int32_t H, int32_t K, int32_t V) {
  kda::LinearArgs a{};
  a.plan = plan;
  a.H = a.Hq = a.Hk = a.Hv = H;
  a.K = K;
  a.V = V;
  const bool fits = kda::check_linear_sizes(a) == KDA_OK && kda::linear_grid_fits(a, false);
  return fits ? kda::linear_layout(plan, H, K, V).total : 0;
}

size_t kda_linear_backward_workspace_bytes(const kda_plan* plan, int32_t H, int32_t Hq, int32_t Hk, int32_t Hv, int32_t K,
                                           int32_t V) {
  kda::LinearArgs a{};
  a.plan = plan;
  a.H = H;
  a.Hq = Hq;
  a.Hk = Hk;
  a.Hv = Hv;
  a.K = K;
  a.V = V;
  const bool fits = kda::check_linear_sizes(a) == KDA_OK && kda::linear_grid_fits(a, true);
  return fits ? kda::linear_bwd_layout(a).total : 0;
}

int kda_linear_step(int32_t B, int32_t H, int32_t Hq, int32_t Hk, int32_t Hv, int32_t K, int32_t V,
                    const uint16_t* q, size_t q_bytes, const uint16_t* k, size_t k_bytes,
                    const uint16_t* v, size_t v_bytes, const void* g, size_t g_bytes, int64_t g_stride,
                    int32_t g_dtype, const int32_t* slots, size_t slots_bytes, int32_t num_slots,
                    const float* state, size_t state_bytes, float* state_out, size_t state_out_bytes,
                    void* o, size_t o_bytes, int32_t o_format, hipStream_t stream) {
  kda::LinearStepArgs a{};
  a.B = B;
  a.H = H;
  a.Hq = Hq;
  a.Hk = Hk;
  a.Hv = Hv;
  a.K = K;
  a.V = V;
  a.g_dtype = g_dtype;
  a.o_format = o_format;
  a.num_slots = num_slots;
  a.q = {q, q_bytes, 0};
  a.k = {k, k_bytes, 0};
  a.v = {v, v_bytes, 0};
  a.g = {g, g_bytes, g_stride};
  a.slots = {slots, slots_bytes, 0};
  a.state = {state, state_bytes, 0};
  a.state_out = {state_out, state_out_bytes};
  a.o = {o, o_bytes};
  const int st = kda::check_linear_step(a);
  return st != KDA_OK ? st : kda::launch_linear_step(a, stream);
}

}  // extern "C"
