// Linear attention with a decay for each head over packed sequences
// (kda_linear_forward) and its gradients (kda_linear_backward): the passes of
// kda_linear_pass.h, the scan of the pieces' states between them, and the sums
// that shared heads and a shared gate need.
//
// A plan's pieces run in parallel.  Where a piece goes on within its sequence, its
// state comes from a first pass over the pieces' keys and values alone and an
// ordered scan: state_{r+1} = e^{G_r} state_r + update_r.
#include "kda_linear_pass.h"

#include <algorithm>

#include "kda.h"

namespace kda {

namespace {

// The state before every piece that goes on within its sequence and, with
// blockIdx.z 1, the cotangent after every piece whose sequence goes on, in place of
// the pieces' own updates.  A thread has four elements of one head's state.
__global__ __launch_bounds__(kRowThreads) void linear_scan_kernel(const int32_t* plan, BlobLayout L, int32_t P, int32_t H,
                                                                  int32_t quads, const float* decays, float* states,
                                                                  float* cotangents) {
  const bool rev = blockIdx.z != 0;
  const int32_t i = static_cast<int32_t>(blockIdx.x) * kRowThreads + static_cast<int32_t>(threadIdx.x);
  const int32_t head = static_cast<int32_t>(blockIdx.y);
  if (i >= quads) return;
  float* const own = (rev ? cotangents : states) + (static_cast<int64_t>(head) * quads + i) * 4;
  const int64_t step = static_cast<int64_t>(H) * quads * 4;
  f32x4 state = zero4();
  // eight pieces' updates in flight; those that were not made are read and dropped
  constexpr int kAhead = 8;
  for (int32_t n0 = 0; n0 < P; n0 += kAhead) {
    f32x4 update[kAhead];
    float decay[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int32_t n = min(n0 + i, P - 1), r = rev ? P - 1 - n : n;
      update[i] = ld4(own + r * step);
      decay[i] = decays[static_cast<int64_t>(r) * H + head];
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (n0 + i >= P) break;
      const int32_t r = rev ? P - 1 - n0 - i : n0 + i;
      const bool before = plan[L.seg_carry_in + r] != 0, after = r + 1 < P && plan[L.seg_carry_in + r + 1] != 0;
      const bool through = before && after && plan[L.seg_transition_live + r] != 0;
      const bool has = rev ? before : after;   // the piece's update was made
      if (rev ? after : before) st4(own + r * step, state);
      state = has ? (through ? decay[i] * state + update[i] : update[i]) : zero4();
    }
  }
}

// Sums of `share` neighbouring heads' rows [T, H, W] FP32 into [T, H / share, W], of
// as many gradients as have shared heads.
struct HeadSums {
  const float* in;
  void* out;
  int64_t quads;
  int32_t share, W;
};
__global__ __launch_bounds__(kRowThreads) void linear_heads_kernel(HeadSums a, HeadSums b, HeadSums c, int32_t out_fp32) {
  const HeadSums s = blockIdx.y == 0 ? a : blockIdx.y == 1 ? b : c;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x;
  if (i >= s.quads) return;
  const int64_t row = i * 4 / s.W, ch = i * 4 - row * s.W;
  f32x4 sum = ld4(s.in + row * s.share * s.W + ch);
  for (int32_t m = 1; m < s.share; ++m) sum += ld4(s.in + (row * s.share + m) * s.W + ch);
  if (out_fp32) {
    st4(static_cast<float*>(s.out) + i * 4, sum);
  } else {
    const u32x2 v = {pack_bf16(sum[0], sum[1]), pack_bf16(sum[2], sum[3])};
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(s.out) + i * 4) = v;
  }
}

// The gradient of a fragment's gates:
//     dg_t = pairs across t in its chunk + what the chunk's tokens from t on take from
//            before it + what those before t give to after it + what passes by it.
// What passes by a chunk c, by_c = e^{G_C} <cotangent after it, state before it>, is
// that product at the fragment's first and last chunk (from the passes) and at its
// anchors, every kAnchorChunks-th chunk.  Between two of them
//     by_c + given_c = by_{c+1} + taken_{c+1},
// as both are what passes the border between two chunks.  Such a step leaves an error
// of about 2^-23 |cotangent| |state| at that border (their norms), which would stay in
// all chunks behind it however little passes by those.  So it is taken from both
// anchors, |by_c| is held to e^{G_C} |cotangent after c| |state before c|, which is 0
// behind a gate that forgets all, and the chunk takes the side with the lesser error.
// [T, H], or with `sums` the fragment's sum of it.
constexpr int kGateGroups = 64 / kAnchorChunks;   // of the 64 chunks that are worked on at a time
__global__ __launch_bounds__(kRowThreads) void linear_gate_kernel(const int32_t* plan, BlobLayout L, int32_t T, int32_t H,
                                                                  int32_t KV, GateParts query, GateParts key, void* dg,
                                                                  int32_t dg_bf16, float* sums) {
  __shared__ float by[64];
  __shared__ float products[kGateGroups][kRowThreads / 64];
  __shared__ float total[kRowThreads / 64];
  const int32_t f = static_cast<int32_t>(blockIdx.x / static_cast<uint32_t>(H));
  const int32_t head = static_cast<int32_t>(blockIdx.x % static_cast<uint32_t>(H));
  const int32_t begin = plan[L.frag_begin + f], end = plan[L.frag_end + f];
  const int32_t chunks = (end - begin + kLinearChunk - 1) / kLinearChunk;
  const int64_t cell = static_cast<int64_t>(f) * H + head, slot = static_cast<int64_t>(begin / kLinearChunk) + f;
  const int lane = static_cast<int>(threadIdx.x) & 63, wave = static_cast<int>(threadIdx.x) >> 6;
  const bool back = lane >= 32;     // lanes 0 .. 31 go from an anchor on, 32 .. 63 from the next one back
  const int r = lane & 31;
  float sum = 0.f, next = 0.f;      // by of the chunk behind the 64
  for (int32_t from = (chunks - 1) / 64 * 64; from >= 0; from -= 64) {
    const int32_t to = min(from + 64, chunks);
#pragma unroll 1
    for (int n = 0; n < kGateGroups; ++n) {
      const int32_t c = from + n * kAnchorChunks;
      if (c == 0 || c + 1 >= chunks) continue;
      const int64_t at = (static_cast<int64_t>(begin / (kAnchorChunks * kLinearChunk) + c / kAnchorChunks - 1) * H + head) * KV;
      f32x4 dot = zero4();
#pragma unroll 4
      for (int32_t i = 4 * static_cast<int32_t>(threadIdx.x); i < KV; i += 4 * kRowThreads) {
        dot += ld4(query.anchors + at + i) * ld4(key.anchors + at + i);
      }
      const float part = sum64((dot[0] + dot[1]) + (dot[2] + dot[3]));
      if (lane == 0) products[n][wave] = part;
    }
    __syncthreads();
    const auto anchor = [&](int32_t c) {   // by of a chunk where it is a product
      if (c + 1 == chunks) return query.by[cell];
      if (c == 0) return key.by[cell];
      if (c == from + 64) return next;
      const float* part = products[(c - from) / kAnchorChunks];
      return query.border[(slot + c) * H + head][2] * ((part[0] + part[1]) + (part[2] + part[3]));
    };
#pragma unroll 1
    for (int n = wave; n < kGateGroups; n += kRowThreads / 64) {
      const int32_t a = from + n * kAnchorChunks, b = min(a + kAnchorChunks, chunks - 1), steps = b - a;
      if (a >= chunks) break;
      const int32_t c = back ? max(b - r, a) : min(a + r, b);
      const f32x4 first = query.border[(slot + c) * H + head], second = key.border[(slot + c) * H + head];
      const float taken = first[0], state = first[1], given = second[0], cotangent = second[1];
      // the border to the chunk of the lane before
      const float step = __shfl_up(back ? taken : given, 1) - (back ? given : taken);
      const float size = __shfl_up(back ? state : cotangent, 1) * (back ? cotangent : state);
      const float most = first[2] * state * cotangent;
      float x = anchor(back ? b : a), error = 0x1p-23f * most;
#pragma unroll 1
      for (int i = 1; i < steps; ++i) {
        const float x0 = __shfl_up(x, 1), error0 = __shfl_up(error, 1);
        if (r != i) continue;
        x = x0 + step;
        x = x > most ? most : x < -most ? -most : x;   // NaN stays
        error = error0 + 0x1p-23f * size;
        error = error > most ? most : error;
      }
      const int other = 32 + max(steps - r, 0);   // the same chunk from the other anchor
      const float y = __shfl(x, other), y_error = __shfl(error, other);
      const bool from_b = r > 0 && (r == steps || x != x || (y_error < error && y == y));
      if (!back && r <= steps && r < kAnchorChunks) by[a + r - from] = from_b ? y : x;
    }
    next = anchor(from);
    __syncthreads();
    for (int32_t c = from + wave; c < to; c += kRowThreads / 64) {
      const int32_t t = begin + c * kLinearChunk + lane;
      if (t >= end) continue;
      const int64_t at = static_cast<int64_t>(head) * T + t;
      const float d = query.tokens[at] + key.tokens[at] + by[c - from];
      sum += d;
      if (sums != nullptr) continue;
      if (dg_bf16) {
        static_cast<uint16_t*>(dg)[static_cast<int64_t>(t) * H + head] = static_cast<uint16_t>(pack_bf16(d, 0.f));
      } else {
        static_cast<float*>(dg)[static_cast<int64_t>(t) * H + head] = d;
      }
    }
    __syncthreads();
  }
  if (sums == nullptr) return;
  sum = sum64(sum);
  if (lane == 0) total[wave] = sum;
  __syncthreads();
  if (threadIdx.x == 0) sums[cell] = (total[0] + total[1]) + (total[2] + total[3]);
}

// Column sums of [rows][H] in FP32: a workgroup a head's range of rows, then the
// ranges' sums in order.
constexpr int kGateBlocks = 64;
__global__ __launch_bounds__(1024) void linear_columns_kernel(const float* in, int32_t rows, int32_t H, float* part) {
  __shared__ float sums[16][64];
  const int32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = static_cast<int32_t>(blockIdx.x) * 64 + lane;
  const int32_t per = (rows + kGateBlocks - 1) / kGateBlocks, first = static_cast<int32_t>(blockIdx.y) * per;
  const int32_t n = min(per, rows - first);
  float sum = col < H && n > 0 ? column_sum(in + static_cast<int64_t>(first) * H + col, H, wave, n) : 0.f;
  sums[wave][lane] = sum;
  __syncthreads();
  if (wave == 0 && col < H) {
    for (int i = 1; i < 16; ++i) sum += sums[i][lane];
    part[static_cast<int64_t>(blockIdx.y) * H + col] = sum;
  }
}
__global__ __launch_bounds__(kRowThreads) void linear_columns_sum_kernel(const float* part, int32_t H, void* dg,
                                                                         int32_t bf16_out) {
  const int32_t h = static_cast<int32_t>(blockIdx.x) * kRowThreads + static_cast<int32_t>(threadIdx.x);
  if (h >= H) return;
  float sum = 0.f;
  for (int i = 0; i < kGateBlocks; ++i) sum += part[static_cast<int64_t>(i) * H + h];
  if (bf16_out) {
    static_cast<uint16_t*>(dg)[h] = static_cast<uint16_t>(pack_bf16(sum, 0.f));
  } else {
    static_cast<float*>(dg)[h] = sum;
  }
}

template <int SS>
void (*linear_output_of(int32_t K, int32_t V))(LinearParams) {
  if (K > 64) return V > 64 ? linear_output_kernel<128, 128, SS, SS> : linear_output_kernel<128, 64, SS, SS>;
  return V > 64 ? linear_output_kernel<64, 128, SS, SS> : linear_output_kernel<64, 64, SS, SS>;
}

Tokens tokens_of(const Rows& r, int32_t H, int32_t heads, int32_t width) {
  return {static_cast<const uint16_t*>(r.ptr), r.stride, H / heads, width};
}

LinearParams pass_of(const LinearArgs& a, int32_t KW, int32_t VW) {
  LinearParams p{};
  p.plan = static_cast<const int32_t*>(a.plan_dev.ptr);
  p.L = a.plan->layout;
  p.T = a.plan->T;
  p.H = a.H;
  p.KW = KW;
  p.VW = VW;
  p.g = a.g.ptr;
  p.g_stride = a.g.stride;
  p.g_bf16 = a.g_dtype == KDA_BF16 ? 1 : 0;
  return p;
}

// The states before the pieces and, where asked for, the cotangents after them.
int launch_piece_states(const LinearArgs& a, float* states, float* decays, const Tokens* d_o, float* cotangents,
                        hipStream_t stream) {
  LinearParams p = pass_of(a, a.K, a.V);
  p.y = tokens_of(a.k, a.H, a.Hk, a.K);
  p.z = tokens_of(a.v, a.H, a.Hv, a.V);
  p.seq_state = static_cast<const float*>(a.initial_state.ptr);
  p.piece_out = states;
  p.decay_out = decays;
  LinearParams r = p;
  if (d_o != nullptr) {
    r.y = tokens_of(a.q, a.H, a.Hq, a.K);
    r.z = *d_o;
    r.seq_state = static_cast<const float*>(a.d_final.ptr);
    r.piece_out = cotangents;
    r.decay_out = nullptr;   // the same as p's
    r.reversed = 1;
  }
  void (*kernel)(LinearParams, LinearParams) =
      a.K > 64 ? (a.V > 64 ? linear_summary_kernel<128, 128> : linear_summary_kernel<128, 64>)
               : (a.V > 64 ? linear_summary_kernel<64, 128> : linear_summary_kernel<64, 64>);
  const uint32_t both = d_o != nullptr ? 2 : 1;
  (void)hipGetLastError();
  hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(a.plan->F) * static_cast<uint32_t>(a.H), both), dim3(kLinearThreads),
                     0, stream, p, r);
  const int st = finish_launch();
  if (st != KDA_OK) return st;
  const int32_t quads = a.K * a.V / 4;
  hipLaunchKernelGGL(linear_scan_kernel, dim3((quads + kRowThreads - 1) / kRowThreads, a.H, both), dim3(kRowThreads), 0, stream,
                     p.plan, a.plan->layout, a.plan->P, a.H, quads, decays, states, cotangents);
  return finish_launch();
}

}  // namespace

int launch_linear(const LinearArgs& a, hipStream_t stream) {
  if (!linear_grid_fits(a, false)) return KDA_ERR_UNSUPPORTED;
  const LinearLayout L = linear_layout(a.plan, a.H, a.K, a.V);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace.ptr);
  float *states = reinterpret_cast<float*>(ws + L.states), *decays = reinterpret_cast<float*>(ws + L.decays);
  if (a.plan->F > a.plan->N) {
    const int st = launch_piece_states(a, states, decays, nullptr, nullptr, stream);
    if (st != KDA_OK) return st;
  }
  LinearParams p = pass_of(a, a.K, a.V);
  p.x = tokens_of(a.q, a.H, a.Hq, a.K);
  p.y = tokens_of(a.k, a.H, a.Hk, a.K);
  p.z = tokens_of(a.v, a.H, a.Hv, a.V);
  p.seq_state = static_cast<const float*>(a.initial_state.ptr);
  p.piece_state = states;
  p.seq_out = static_cast<float*>(a.final_state.ptr);
  p.o = a.o.ptr;
  p.o_fp32 = a.o_format == KDA_FP32 ? 1 : 0;
  (void)hipGetLastError();
  hipLaunchKernelGGL(p.o_fp32 ? linear_output_of<3>(a.K, a.V) : linear_output_of<2>(a.K, a.V),
                     dim3(static_cast<uint32_t>(a.plan->F) * static_cast<uint32_t>(a.H)), dim3(kLinearThreads), 0, stream, p);
  return finish_launch();
}

int launch_linear_backward(const LinearArgs& a, hipStream_t stream) {
  if (!linear_grid_fits(a, true)) return KDA_ERR_UNSUPPORTED;
  const auto quads_of = [&](int32_t heads, int32_t width) {
    return heads == a.H ? 0 : static_cast<int64_t>(a.plan->T) * heads * width / 4;
  };
  const int64_t most = std::max({quads_of(a.Hq, a.K), quads_of(a.Hk, a.K), quads_of(a.Hv, a.V)});
  const LinearBwdLayout L = linear_bwd_layout(a);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace.ptr);
  auto at = [ws](size_t offset) { return reinterpret_cast<float*>(ws + offset); };
  const bool cut = a.plan->F > a.plan->N, fp32 = a.o_format == KDA_FP32, fixed = a.g.stride == 0;
  const Rows d_o = {a.d_o.ptr, a.d_o.bytes, static_cast<int64_t>(a.H) * a.V};
  const Tokens q = tokens_of(a.q, a.H, a.Hq, a.K), k = tokens_of(a.k, a.H, a.Hk, a.K), v = tokens_of(a.v, a.H, a.Hv, a.V),
               d = tokens_of(d_o, a.H, a.H, a.V);
  const float *h0 = static_cast<const float*>(a.initial_state.ptr), *d_final = static_cast<const float*>(a.d_final.ptr);
  int st = KDA_OK;
  if (cut) {
    st = launch_piece_states(a, at(L.states), at(L.decays), &d, at(L.cotangents), stream);
    if (st != KDA_OK) return st;
  }
  const int32_t F = a.plan->F;
  const uint32_t cells = static_cast<uint32_t>(F) * static_cast<uint32_t>(a.H);
  // heads that share a row are added in a launch of their own
  HeadSums sums[3] = {};
  int shared = 0;
  const auto out = [&](LinearParams& p, int32_t heads, const Dst& to, size_t offset) {
    const bool own = heads == a.H;
    p.o = own ? to.ptr : static_cast<void*>(at(offset));
    p.o_fp32 = fp32 || !own ? 1 : 0;
    if (own) return;
    sums[shared++] = {at(offset), to.ptr, quads_of(heads, p.VW), a.H / heads, p.VW};
  };
  LinearParams query = pass_of(a, a.V, a.K);
  query.transposed = 1;
  query.x = d;
  query.y = v;
  query.z = k;
  query.e = q;
  query.seq_state = h0;
  query.piece_state = at(L.states);
  query.gates = {at(L.query_gates), reinterpret_cast<f32x4*>(at(L.query_border)), at(L.query_by), at(L.query_anchors)};
  query.end_seq = d_final;
  query.end_piece = at(L.cotangents);
  out(query, a.Hq, a.dq, L.query_heads);
  LinearParams key = pass_of(a, a.V, a.K);
  key.transposed = 1;
  key.x = v;
  key.y = d;
  key.z = q;
  key.e = k;
  key.seq_state = d_final;
  key.piece_state = at(L.cotangents);
  key.gates = {at(L.key_gates), reinterpret_cast<f32x4*>(at(L.key_border)), at(L.key_by), at(L.key_anchors)};
  key.end_seq = h0;
  key.end_piece = at(L.states);
  out(key, a.Hk, a.dk, L.key_heads);
  LinearParams value = pass_of(a, a.K, a.V);
  value.x = k;
  value.y = q;
  value.z = d;
  value.seq_state = d_final;
  value.piece_state = at(L.cotangents);
  value.seq_out = static_cast<float*>(a.d_initial_state.ptr);
  out(value, a.Hv, a.dv, L.value_heads);

  (void)hipGetLastError();
  hipLaunchKernelGGL(fp32 ? linear_grad_fp32(a.K, a.V) : linear_grad_bf16(a.K, a.V), dim3(cells, 3), dim3(kLinearThreads), 0,
                     stream, query, key, value);
  hipLaunchKernelGGL(linear_gate_kernel, dim3(cells), dim3(kRowThreads), 0, stream, query.plan, query.L, a.plan->T, a.H,
                     a.K * a.V, query.gates, key.gates, a.dg.ptr, a.g_dtype == KDA_BF16 ? 1 : 0, fixed ? at(L.sums) : nullptr);
  if (fixed) {
    float* const part = at(L.query_gates);   // read by now
    hipLaunchKernelGGL(linear_columns_kernel, dim3((a.H + 63) / 64, kGateBlocks), dim3(1024), 0, stream, at(L.sums), F, a.H,
                       part);
    hipLaunchKernelGGL(linear_columns_sum_kernel, dim3((a.H + kRowThreads - 1) / kRowThreads), dim3(kRowThreads), 0, stream,
                       part, a.H, a.dg.ptr, a.g_dtype == KDA_BF16 ? 1 : 0);
  }
  if (shared > 0) {
    hipLaunchKernelGGL(linear_heads_kernel, dim3(static_cast<uint32_t>((most + kRowThreads - 1) / kRowThreads), shared),
                       dim3(kRowThreads), 0, stream, sums[0], sums[1], sums[2], fp32 ? 1 : 0);
  }
  return finish_launch();
}

}  // namespace kda
