// Parameter blocks, host checks and launchers of the operators around the
// recurrence (input preparation, output norm, per-channel scan, single-token
// steps).  A launcher takes arguments that have passed its check and returns
// a kda_status.
#ifndef KDA_LAYER_H_
#define KDA_LAYER_H_

#include <cstddef>
#include <cstdint>

#include "kda_internal.h"

namespace kda {

// A tensor of token rows: dense rows `stride` elements apart.
struct Rows {
  const void* ptr;
  size_t bytes;
  int64_t stride;
};

struct Dst {
  void* ptr;
  size_t bytes;
};

struct PrepareArgs {
  int32_t T, H, K, dtype;
  Rows q_raw, k_raw, gate_raw, beta_raw;
  Rows a_log, dt_bias;               // FP32, stride unused
  float q_scale, eps;
  Dst q, k, g, beta;                 // forward: bf16; backward: gradients of the raw inputs (dtype)
  Rows dq, dk, dg, dbeta;            // backward only, FP32
  Dst da_log, ddt_bias, workspace;   // backward only
};

struct NormArgs {
  int32_t T, H, V, dtype, o_format, activation, d_o_format;
  Rows o, gate, weight, res_scale, residual, dy;
  float eps;
  Dst y;                                             // forward
  Dst d_o, d_gate, d_weight, d_res_scale, workspace; // backward
};

struct ScanArgs {
  const kda_plan* plan;
  Rows plan_dev;
  int32_t D, dtype, tied, h_format;
  Rows x, g, initial_state;
  Dst h, final_state, workspace;              // forward
  Rows h_in, dh, d_final;                     // backward
  Dst dx, dg, d_initial_state;
};

struct ScanStepArgs {
  int32_t B, D, dtype, tied, num_slots;
  Rows x, g, slots, state;
  Dst state_out, h;
};

struct StepArgs {
  int32_t B, H, K, V, head_begin, head_count, o_format, num_slots;
  Rows q, k, v, g, beta, slots, state;
  float gate_lower_bound;
  Dst state_out, o;
};

// Partial sums over tokens (the backward passes of the row-wise operators).
// A group of lanes takes rows (t, h) of one head: rows r, r + P H, r + 2 P H,
// ... for the P "lanes" of tokens; every group leaves one partial row.
//
// Work of a row-wise launch: threads per workgroup, workgroups, and P.
struct RowGrid {
  int32_t groups_per_block, blocks, lanes;   // lanes = P
};
RowGrid row_grid(int64_t T, int64_t H, int32_t groups_per_block, int32_t max_blocks);

constexpr int kRowThreads = 256;        // row-wise kernels
constexpr int64_t kStreamBytes = int64_t(256) << 20;   // the last-level cache: larger calls go past it
constexpr int kPrepareGroups = 16;      // 16-lane groups of 8 channels a workgroup
constexpr int kPrepareBwdBlocks = 512;  // backward grid at most: two workgroups a CU

struct PrepareBwdLayout {
  RowGrid grid;
  size_t bias, decay, total;   // byte offsets: [P][H][128] and [P][H] FP32
};
PrepareBwdLayout prepare_bwd_layout(int32_t T, int32_t H);

// The norm's lane group for rows of V channels: `lanes` threads a row, each
// with `vectors` vectors of 8 channels.
struct NormShape {
  int32_t lanes, vectors;
};
NormShape norm_shape(int32_t V);
int32_t norm_threads(const NormShape& shape);   // a workgroup's

struct NormBwdLayout {
  RowGrid grid;
  size_t weight, scale, total;   // byte offsets: [blocks][V] and [P][H][V] FP32
};
NormBwdLayout norm_bwd_layout(int32_t T, int32_t H, int32_t V, int32_t o_format);
size_t norm_bwd_workspace(int32_t T, int32_t H, int32_t V);
bool norm_whole_rows(const NormArgs& a);   // rows of whole, aligned 16-byte vectors

// The scan's tiles: kScanTile tokens of kScanChannels channels, one workgroup
// each.  More than one token tile need words of workspace in which tiles leave
// their maps (8 bytes a channel) and end states (4), and a ticket counter a
// channel block on a cache line of its own (byte offsets).
constexpr int kScanThreads = 256;
constexpr int kScanTile = 128;
constexpr int kScanChannels = 64;
constexpr int64_t kMaxScanStride = 1 << 22;   // byte offsets inside a tile stay below 2^32
struct ScanLayout {
  int32_t tiles, columns;
  size_t tickets, maps, states, total;
};
ScanLayout scan_layout(int32_t T, int32_t D);
// Whether a ticket names one of a channel block's tiles.  The words of a
// workspace that another call overwrites can hold anything, and a ticket is
// turned into addresses: one with the top bit set must not pass as negative.
constexpr bool is_tile(uint32_t ticket, int32_t tiles) { return ticket < static_cast<uint32_t>(tiles); }

int check_prepare(const PrepareArgs& a, bool backward);
int check_norm(const NormArgs& a, bool backward);
int check_scan(const ScanArgs& a, bool backward);
int check_scan_step(const ScanStepArgs& a);
int check_step(const StepArgs& a);

}  // namespace kda

#ifdef __HIPCC__
#include <hip/hip_runtime.h>
namespace kda {
// The status of the launch just made (kda_api.hip); KDA_ERR_HIP keeps the error.
int finish_launch();

int launch_prepare(const PrepareArgs& a, hipStream_t stream);
int launch_prepare_backward(const PrepareArgs& a, hipStream_t stream);
int launch_norm(const NormArgs& a, hipStream_t stream);
int launch_norm_backward(const NormArgs& a, hipStream_t stream);
int launch_scan(const ScanArgs& a, hipStream_t stream);
int launch_scan_backward(const ScanArgs& a, hipStream_t stream);
int launch_scan_step(const ScanStepArgs& a, hipStream_t stream);
int launch_step(const StepArgs& a, hipStream_t stream);
}  // namespace kda
#endif

#endif  // KDA_LAYER_H_
