// Parameter blocks, host checks and launchers of the operators around the
// recurrence (input preparation, norms and rotation of queries and keys, output
// norm, per-channel scan, linear attention, single-token steps).  A launcher takes arguments that have passed its check and returns
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

struct RotateArgs {
  int32_t T, Hq, Hk, D, R, dtype, interleaved, d_format;
  Rows q_raw, k_raw;
  Rows positions, inv_freq, q_weight, k_weight;   // int32; FP32; stride unused
  float q_scale, eps;
  Dst q, k;                                       // backward: gradients of the raw rows
  Rows dq, dk;                                    // backward only, d_format
  Dst dq_weight, dk_weight, workspace;
};

struct LinearStepArgs {
  int32_t B, H, Hq, Hk, Hv, K, V, g_dtype, o_format, num_slots;
  Rows q, k, v, g, slots, state;   // g.stride: H, or 0 for one g [H]
  Dst state_out, o;
};

struct LinearArgs {
  const kda_plan* plan;
  Rows plan_dev;
  int32_t H, Hq, Hk, Hv, K, V, g_dtype, o_format;   // backward: o_format is the gradients'
  Rows q, k, v, g;                                  // g.stride 0: one g [H]
  Rows initial_state;
  Dst o, final_state, workspace;                    // forward
  Rows d_o, d_final;                                // backward
  Dst dq, dk, dv, dg, d_initial_state;
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
// Norms and rotation, backward grid at most: three workgroups a CU (gradients of 8191
// x 32 heads 38 us, of 32768 x 40 170; 256 workgroups 68 and 349, 1536 43 and 180).
constexpr int kRotateBwdBlocks = 768;
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

// Work of the norms and rotation: `tiles` of `tokens` tokens, forward each by
// row_blocks workgroups, backward by `blocks` workgroups in all.
struct RotateGrid {
  int32_t tokens, tiles, row_blocks, blocks;
};
RotateGrid rotate_grid(const RotateArgs& a, bool backward);
size_t rotate_bwd_workspace(int32_t T, int32_t D);
bool rotate_whole_rows(const RotateArgs& a);   // pairs of whole, aligned 16-byte vectors

// Linear attention's workspace (byte offsets): the pieces' states and decays
// where a sequence is cut, [P][H][K][V] and [P][H] FP32.
struct LinearLayout {
  size_t states, decays, total;
};
LinearLayout linear_layout(const kda_plan* plan, int32_t H, int32_t K, int32_t V);
// How far apart the chunks inside a piece are whose states' product gives what passes
// by them for the gates' gradient.  Gradients of 16384 tokens x 32 heads in pieces of 16
// chunks: 734 us, with 16 (none inside) 720.  Gates' gradients of tokens 2^17 times
// smaller than those around them are within 3.8e-6 of their own norm, with 16 6.1e-6.
constexpr int kAnchorChunks = 8;
// Backward, behind those: the states' cotangents; of both passes the gates' gradient
// within the chunks [H][T] (at least 64 rows: then query_gates holds the 64 ranges' sums
// of a shared gate), four numbers at each chunk's border [T / 64 + 1 + F][H][4] (chunk c
// of fragment f in slot floor(begin_f / 64) + f + c), what passes by the chunk where the
// pass ends [F][H] and the states at the anchors [T / (64 kAnchorChunks)][H][K][V] (chunk
// c of fragment f in place floor(begin_f / (64 kAnchorChunks)) + c / kAnchorChunks - 1;
// none where no fragment has one); the fragments' sums of a shared gate [F][H]; and for
// each of q, k, v that heads share its gradient for every head [T][H][K] or [T][H][V].
// All FP32, divisions rounded down.
struct LinearBwdLayout {
  size_t states, cotangents, decays, query_gates, key_gates, query_border, key_border, query_by, key_by, sums, query_anchors,
      key_anchors, query_heads, key_heads, value_heads, total;
};
LinearBwdLayout linear_bwd_layout(const LinearArgs& a);

int check_prepare(const PrepareArgs& a, bool backward);
int check_rotate(const RotateArgs& a, bool backward);
int check_linear_sizes(const LinearArgs& a);
bool linear_grid_fits(const LinearArgs& a, bool backward);   // sizes that passed the check
int check_linear(const LinearArgs& a, bool backward);
int check_linear_step(const LinearStepArgs& a);
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
int launch_rotate(const RotateArgs& a, hipStream_t stream);
int launch_rotate_backward(const RotateArgs& a, hipStream_t stream);
int launch_linear(const LinearArgs& a, hipStream_t stream);
int launch_linear_backward(const LinearArgs& a, hipStream_t stream);
int launch_linear_step(const LinearStepArgs& a, hipStream_t stream);
int launch_norm(const NormArgs& a, hipStream_t stream);
int launch_norm_backward(const NormArgs& a, hipStream_t stream);
int launch_scan(const ScanArgs& a, hipStream_t stream);
int launch_scan_backward(const ScanArgs& a, hipStream_t stream);
int launch_scan_step(const ScanStepArgs& a, hipStream_t stream);
int launch_step(const StepArgs& a, hipStream_t stream);
}  // namespace kda
#endif

#endif  // KDA_LAYER_H_
