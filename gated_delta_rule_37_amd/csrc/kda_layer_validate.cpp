// Host-side argument validation of the operators around the recurrence (no
// HIP calls): every check their entry points make before anything is
// enqueued, and the layouts of their workspaces.  Builds with a host compiler
// too (the sanitizer tests).
#include "kda_layer.h"

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "kda.h"
#include "kda_validate.h"

namespace kda {
namespace {

constexpr int32_t kMaxBatch = 1 << 20;
constexpr int32_t kMaxChannels = 1 << 20;
constexpr int32_t kMaxNormWidth = 8192;
constexpr int64_t kMaxNormRow = 1 << 24;   // H * V: the column sums' grid
constexpr int32_t kMaxHeads = 65535;
constexpr int64_t kMaxStride = (int64_t(1) << 31) - 1;   // 2^30 rows of it stay inside 64-bit byte counts

bool known_type(int32_t t) { return t == KDA_FP32 || t == KDA_BF16; }
size_t size_of(int32_t t) { return t == KDA_BF16 ? 2 : 4; }
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// The element stride of a tensor of rows: at least the row.
int check_stride(const Rows& r, int64_t row) {
  if (r.ptr == nullptr) return KDA_OK;   // reported with the other null pointers, or optional
  if (r.stride < row) return KDA_ERR_INVALID_ARG;
  return r.stride > kMaxStride ? KDA_ERR_UNSUPPORTED : KDA_OK;
}
size_t rows_need(const Rows& r, int32_t T, size_t row, size_t element) {
  return (static_cast<size_t>(T - 1) * static_cast<size_t>(r.stride) + row) * element;
}

int first_error(std::initializer_list<int> statuses) {
  for (int s : statuses) {
    if (s != KDA_OK) return s;
  }
  return KDA_OK;
}

bool overlap(const void* a, const void* b, size_t bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y ? y - x < bytes : x - y < bytes;
}

int check_workspace(const Dst& ws, size_t need) {
  if (need == 0) return KDA_OK;
  if (ws.ptr == nullptr) return KDA_ERR_INVALID_ARG;
  if (!aligned16(ws.ptr)) return KDA_ERR_MISALIGNED;
  return ws.bytes < need ? KDA_ERR_WORKSPACE_TOO_SMALL : KDA_OK;
}

// A batch of single tokens over state slots.
int check_slots(int32_t B, const Rows& slots, int32_t num_slots) {
  if (B <= 0 || num_slots <= 0) return KDA_ERR_INVALID_ARG;
  if (B > kMaxBatch) return KDA_ERR_UNSUPPORTED;
  return slots.ptr == nullptr && num_slots < B ? KDA_ERR_INVALID_ARG : KDA_OK;
}

int check_pool(const Rows& state, const Dst& state_out, size_t bytes) {
  return state.ptr != state_out.ptr && overlap(state.ptr, state_out.ptr, bytes) ? KDA_ERR_INVALID_ARG : KDA_OK;
}

}  // namespace

RowGrid row_grid(int64_t T, int64_t H, int32_t groups_per_block, int32_t max_blocks) {
  const int64_t rows = T * H;
  const int64_t want = (rows + groups_per_block - 1) / groups_per_block;   // one row a group
  const int64_t least = (H + groups_per_block - 1) / groups_per_block;     // one group a head
  RowGrid g;
  g.groups_per_block = groups_per_block;
  int64_t blocks = want < max_blocks ? want : max_blocks;
  if (blocks < least) blocks = least;
  g.blocks = static_cast<int32_t>(blocks);
  int64_t lanes = blocks * groups_per_block / H;
  if (lanes > T) lanes = T;
  g.lanes = static_cast<int32_t>(lanes);
  return g;
}

PrepareBwdLayout prepare_bwd_layout(int32_t T, int32_t H) {
  PrepareBwdLayout L;
  L.grid = row_grid(T, H, kPrepareGroups, kPrepareBwdBlocks);
  const size_t rows = static_cast<size_t>(L.grid.lanes) * static_cast<size_t>(H);
  L.bias = 0;
  L.decay = up256(rows * 128 * sizeof(float));
  L.total = L.decay + up256(rows * sizeof(float));
  return L;
}

// A row's last vectors leave lanes idle, so a row takes the smallest group that
// holds it; up to 1024 channels it stays inside a wave, where its sum needs no
// barrier.  Forward, bf16 o and residual, 268 MB in rows of V: V = 128 72 us (64
// lanes: 194), 256 70 (64 lanes: 110), 512 71 (256 lanes: 205), 1024 70 (256
// lanes: 117), 2048 73 (64 lanes of four vectors: 106), 4096 72, 8192 74 (256
// lanes of four vectors: 109).
NormShape norm_shape(int32_t V) {
  if (V <= 128) return {16, 1};
  if (V <= 256) return {32, 1};
  if (V <= 512) return {64, 1};
  if (V <= 1024) return {64, 2};
  if (V <= 2048) return {256, 1};
  if (V <= 4096) return {256, 2};
  return {512, 2};
}
// Backward: each workgroup leaves partial sums, so only as many as run at once
// and have enough in flight.  Two vectors a lane (154-178 registers): three
// workgroups a CU of 256 threads and one of 512; with 65536 rows of 1024 bf16
// channels 768 workgroups 114 us, 512 142, 1024 154, with rows of 8192 256
// workgroups 161, 512 166.  One vector (85-92 registers): four of bf16 o (2^26
// channels in rows of 128, 256, 512 and 2048: 1024 workgroups 109, 110, 111 and
// 113 us, 768 111, 114, 115 and 122), three of fp32 o, whose loads are twice as
// many (with a gate: 768 workgroups 181, 178, 179 and 182 us, 1024 183, 181, 181
// and 186, 512 191 to 206).
int32_t norm_bwd_blocks(const NormShape& s, int32_t o_format) {
  if (s.vectors == 1 && o_format == KDA_BF16) return 1024;
  return s.lanes == 512 ? 256 : 768;
}
int32_t norm_threads(const NormShape& s) { return s.lanes > kRowThreads ? s.lanes : kRowThreads; }

NormBwdLayout norm_bwd_layout(int32_t T, int32_t H, int32_t V, int32_t o_format) {
  const NormShape shape = norm_shape(V);
  NormBwdLayout L;
  L.grid = row_grid(T, H, norm_threads(shape) / shape.lanes, norm_bwd_blocks(shape, o_format));
  const size_t v = static_cast<size_t>(V) * sizeof(float);
  L.weight = 0;
  L.scale = up256(static_cast<size_t>(L.grid.blocks) * v);
  L.total = L.scale + up256(static_cast<size_t>(L.grid.lanes) * static_cast<size_t>(H) * v);
  return L;
}
// Of either format of o: bf16 has the more workgroups.
size_t norm_bwd_workspace(int32_t T, int32_t H, int32_t V) { return norm_bwd_layout(T, H, V, KDA_BF16).total; }

bool norm_whole_rows(const NormArgs& a) {
  return a.V % 8 == 0 && (a.gate.ptr == nullptr || a.gate.stride * static_cast<int64_t>(size_of(a.dtype)) % 16 == 0);
}

ScanLayout scan_layout(int32_t T, int32_t D) {
  ScanLayout L{};
  L.tiles = static_cast<int32_t>((static_cast<int64_t>(T) + kScanTile - 1) / kScanTile);
  L.columns = (D + kScanChannels - 1) / kScanChannels;
  if (L.tiles == 1) return L;
  const size_t cells = static_cast<size_t>(L.tiles) * static_cast<size_t>(L.columns) * kScanChannels;
  L.tickets = 0;
  L.maps = static_cast<size_t>(L.columns) * 128;
  L.states = L.maps + cells * 8;
  L.total = L.states + cells * 4;
  return L;
}

int check_prepare(const PrepareArgs& a, bool backward) {
  if (a.T <= 0 || a.H <= 0 || a.K <= 0) return KDA_ERR_INVALID_ARG;
  if (a.K != 128 || a.H > kMaxHeads || a.T > kMaxTokens) return KDA_ERR_UNSUPPORTED;
  if (!known_type(a.dtype)) return KDA_ERR_INVALID_ARG;
  if (!std::isfinite(a.q_scale) || !(a.eps > 0.f) || !std::isfinite(a.eps)) return KDA_ERR_INVALID_ARG;
  const size_t e = size_of(a.dtype), H = static_cast<size_t>(a.H), row = H * 128,
               n = static_cast<size_t>(a.T) * row, nb = static_cast<size_t>(a.T) * H;
  int st = first_error({check_stride(a.q_raw, row), check_stride(a.k_raw, row), check_stride(a.gate_raw, row),
                        check_stride(a.beta_raw, H)});
  if (st != KDA_OK) return st;
  if (backward && (a.dt_bias.ptr == nullptr) != (a.ddt_bias.ptr == nullptr)) return KDA_ERR_INVALID_ARG;
  const size_t out = backward ? e : 2;
  st = check_buffers({{a.q_raw.ptr, a.q_raw.bytes, rows_need(a.q_raw, a.T, row, e), false},
                      {a.k_raw.ptr, a.k_raw.bytes, rows_need(a.k_raw, a.T, row, e), false},
                      {a.gate_raw.ptr, a.gate_raw.bytes, rows_need(a.gate_raw, a.T, row, e), false},
                      {a.beta_raw.ptr, a.beta_raw.bytes, rows_need(a.beta_raw, a.T, H, e), false},
                      {a.a_log.ptr, a.a_log.bytes, H * 4, false},
                      {a.dt_bias.ptr, a.dt_bias.bytes, row * 4, true},
                      {a.dq.ptr, a.dq.bytes, n * 4, !backward},
                      {a.dk.ptr, a.dk.bytes, n * 4, !backward},
                      {a.dg.ptr, a.dg.bytes, n * 4, !backward},
                      {a.dbeta.ptr, a.dbeta.bytes, nb * 4, !backward},
                      {a.q.ptr, a.q.bytes, n * out, false},
                      {a.k.ptr, a.k.bytes, n * out, false},
                      {a.g.ptr, a.g.bytes, n * out, false},
                      {a.beta.ptr, a.beta.bytes, nb * out, false},
                      {a.da_log.ptr, a.da_log.bytes, H * 4, !backward},
                      {a.ddt_bias.ptr, a.ddt_bias.bytes, row * 4, true}});
  if (st != KDA_OK) return st;
  for (const Rows* r : {&a.q_raw, &a.k_raw, &a.gate_raw}) {
    if (r->stride * static_cast<int64_t>(e) % 16 != 0) return KDA_ERR_MISALIGNED;
  }
  return backward ? check_workspace(a.workspace, prepare_bwd_layout(a.T, a.H).total) : KDA_OK;
}

int check_norm(const NormArgs& a, bool backward) {
  if (a.T <= 0 || a.H <= 0 || a.V <= 0) return KDA_ERR_INVALID_ARG;
  if (a.V > kMaxNormWidth || a.H > kMaxHeads || a.T > kMaxTokens) return KDA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(a.H) * a.V > kMaxNormRow) return KDA_ERR_UNSUPPORTED;
  if (!known_type(a.dtype) || !known_type(a.o_format)) return KDA_ERR_INVALID_ARG;
  if (backward && !known_type(a.d_o_format)) return KDA_ERR_INVALID_ARG;
  if (a.activation != KDA_ACT_NONE && a.activation != KDA_ACT_SIGMOID && a.activation != KDA_ACT_SILU) {
    return KDA_ERR_INVALID_ARG;
  }
  if (!(a.eps > 0.f) || !std::isfinite(a.eps)) return KDA_ERR_INVALID_ARG;
  const bool gated = a.activation != KDA_ACT_NONE;
  if (gated != (a.gate.ptr != nullptr)) return KDA_ERR_INVALID_ARG;
  if (backward && (gated != (a.d_gate.ptr != nullptr) || (a.res_scale.ptr == nullptr) != (a.d_res_scale.ptr == nullptr))) {
    return KDA_ERR_INVALID_ARG;
  }
  const size_t e = size_of(a.dtype), row = static_cast<size_t>(a.H) * static_cast<size_t>(a.V),
               n = static_cast<size_t>(a.T) * row, V = static_cast<size_t>(a.V);
  int st = check_stride(a.gate, static_cast<int64_t>(row));
  if (st != KDA_OK) return st;
  st = check_buffers({{a.o.ptr, a.o.bytes, n * size_of(a.o_format), false},
                      {a.gate.ptr, a.gate.bytes, gated ? rows_need(a.gate, a.T, row, e) : 0, true},
                      {a.weight.ptr, a.weight.bytes, V * 4, false},
                      {a.res_scale.ptr, a.res_scale.bytes, row * 4, true},
                      {a.residual.ptr, a.residual.bytes, n * e, true},
                      {a.y.ptr, a.y.bytes, n * e, backward},
                      {a.dy.ptr, a.dy.bytes, n * e, !backward},
                      {a.d_o.ptr, a.d_o.bytes, n * (backward ? size_of(a.d_o_format) : 0), !backward},
                      {a.d_gate.ptr, a.d_gate.bytes, n * e, true},
                      {a.d_weight.ptr, a.d_weight.bytes, V * 4, !backward},
                      {a.d_res_scale.ptr, a.d_res_scale.bytes, row * 4, true}});
  if (st != KDA_OK) return st;
  return backward ? check_workspace(a.workspace, norm_bwd_workspace(a.T, a.H, a.V)) : KDA_OK;
}

int check_scan(const ScanArgs& a, bool backward) {
  if (a.plan == nullptr || a.plan_dev.ptr == nullptr || a.D <= 0) return KDA_ERR_INVALID_ARG;
  if (a.D > kMaxChannels) return KDA_ERR_UNSUPPORTED;
  if (!known_type(a.dtype) || !known_type(a.h_format) || (a.tied != 0 && a.tied != 1)) return KDA_ERR_INVALID_ARG;
  const bool need_x = !backward || a.tied != 0;
  const int32_t T = a.plan->T;
  const size_t D = static_cast<size_t>(a.D), e = size_of(a.dtype), n = static_cast<size_t>(T) * D,
               nh = n * size_of(a.h_format), state = static_cast<size_t>(a.plan->N) * D * 4;
  int st = first_error({need_x ? check_stride(a.x, a.D) : KDA_OK, check_stride(a.g, a.D)});
  if (st != KDA_OK) return st;
  if ((need_x && a.x.stride > kMaxScanStride) || a.g.stride > kMaxScanStride) return KDA_ERR_UNSUPPORTED;
  st = check_buffers({{a.plan_dev.ptr, a.plan_dev.bytes, a.plan->blob.size() * sizeof(int32_t), false},
                      {a.x.ptr, a.x.bytes, need_x ? rows_need(a.x, T, D, e) : 0, !need_x},
                      {a.g.ptr, a.g.bytes, rows_need(a.g, T, D, e), false},
                      {a.initial_state.ptr, a.initial_state.bytes, state, true},
                      {a.h.ptr, a.h.bytes, nh, backward},
                      {a.final_state.ptr, a.final_state.bytes, state, backward},
                      {a.h_in.ptr, a.h_in.bytes, nh, !backward},
                      {a.dh.ptr, a.dh.bytes, nh, !backward},
                      {a.d_final.ptr, a.d_final.bytes, state, true},
                      {a.dx.ptr, a.dx.bytes, n * e, !backward},
                      {a.dg.ptr, a.dg.bytes, n * e, !backward},
                      {a.d_initial_state.ptr, a.d_initial_state.bytes, state, true}});
  if (st != KDA_OK) return st;
  return check_workspace(a.workspace, scan_layout(a.plan->T, a.D).total);
}

int check_scan_step(const ScanStepArgs& a) {
  if (a.D <= 0) return KDA_ERR_INVALID_ARG;
  int st = check_slots(a.B, a.slots, a.num_slots);
  if (st != KDA_OK) return st;
  if (a.D > kMaxChannels) return KDA_ERR_UNSUPPORTED;
  if (!known_type(a.dtype) || (a.tied != 0 && a.tied != 1)) return KDA_ERR_INVALID_ARG;
  const size_t n = static_cast<size_t>(a.B) * static_cast<size_t>(a.D) * size_of(a.dtype),
               pool = static_cast<size_t>(a.num_slots) * static_cast<size_t>(a.D) * 4;
  st = check_buffers({{a.x.ptr, a.x.bytes, n, false},
                      {a.g.ptr, a.g.bytes, n, false},
                      {a.slots.ptr, a.slots.bytes, static_cast<size_t>(a.B) * 4, true},
                      {a.state.ptr, a.state.bytes, pool, false},
                      {a.state_out.ptr, a.state_out.bytes, pool, false},
                      {a.h.ptr, a.h.bytes, n, false}});
  return st != KDA_OK ? st : check_pool(a.state, a.state_out, pool);
}

int check_step(const StepArgs& a) {
  if (a.H <= 0 || a.K <= 0 || a.V <= 0) return KDA_ERR_INVALID_ARG;
  int st = check_slots(a.B, a.slots, a.num_slots);
  if (st != KDA_OK) return st;
  if (a.K != 128 || a.V != 128 || a.H > kMaxHeads) return KDA_ERR_UNSUPPORTED;
  st = check_heads(a.H, a.head_begin, a.head_count);
  if (st != KDA_OK) return st;
  if (a.o_format != KDA_O_FP32 && a.o_format != KDA_O_BF16) return KDA_ERR_INVALID_ARG;
  st = check_gate_bound(a.gate_lower_bound);
  if (st != KDA_OK) return st;
  const size_t rows = static_cast<size_t>(a.B) * static_cast<size_t>(a.H), n = rows * 128,
               pool = static_cast<size_t>(a.num_slots) * static_cast<size_t>(a.H) * 128 * 128 * 4;
  st = check_buffers({{a.q.ptr, a.q.bytes, n * 2, false},
                      {a.k.ptr, a.k.bytes, n * 2, false},
                      {a.v.ptr, a.v.bytes, n * 2, false},
                      {a.g.ptr, a.g.bytes, n * 2, false},
                      {a.beta.ptr, a.beta.bytes, rows * 2, false},
                      {a.slots.ptr, a.slots.bytes, static_cast<size_t>(a.B) * 4, true},
                      {a.state.ptr, a.state.bytes, pool, false},
                      {a.state_out.ptr, a.state_out.bytes, pool, false},
                      {a.o.ptr, a.o.bytes, n * size_of(a.o_format), false}});
  return st != KDA_OK ? st : check_pool(a.state, a.state_out, pool);
}

}  // namespace kda
