// The norm after the recurrence with its gate and residual scale
// (kda_output_norm) and its gradients.
//
// Per (token, head) row of V channels, with r = (mean o^2 + eps)^(-1/2) and
// n = o r:
//   y = residual + s act(z) w n
// and for a cotangent dy, with m = dy act(z) n:
//   dn = dy s act(z) w,  d_o = r (dn - n mean(dn n)),  d_z = dy s w n act'(z),
//   dw = sum over rows of s m,  ds = w * (sum over tokens of m).
//
// A row stays in the registers of its lane group (16 lanes for a head of 128,
// up to a workgroup for 8192 channels): each element is read and written
// once, HBM bandwidth is the bound.  Rows whose width or stride is not a
// multiple of 16 bytes take the same vectors at any address, and what is left
// of the row one by one.  fp32 o, gate and y in bf16, 65536 x 32 heads of
// 128 forward 378 us, 5.7 TB/s; 8191 x 16 backward with every term 42 us, 5.6
// TB/s (part of it from the last-level cache), and 5 us for the sums over the
// rows (a large copy: 5.2 TB/s).
#include "kda_layer.h"
#include "kda_layer_device.h"

#include "kda.h"

namespace kda {
namespace {

struct NormParams {
  const void *o, *gate, *residual, *dy;
  int64_t gate_stride;
  const float *weight, *res_scale;
  float eps;
  int32_t T, H, V, lanes;   // lanes: P, the tokens in flight for one head
  int32_t activation;
  void *y, *d_o, *d_gate;
  float *weight_part, *scale_part;
};

// Threads of a workgroup: 256, or one row's.
template <int LANES>
constexpr int kThreads = LANES > kRowThreads ? LANES : kRowThreads;

// Sum over a lane group of LANES threads (16, 32, 64 or the whole workgroup).
template <int LANES>
__device__ __forceinline__ float group_sum(float x, float* scratch) {
  if constexpr (LANES == 16) return sum16(x);
  if constexpr (LANES == 32) return sum32(x);
  x = sum64(x);
  if constexpr (LANES > 64) {
    __syncthreads();   // the scratch's readers of the sum before
    if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = x;
    __syncthreads();
    x = (scratch[0] + scratch[1]) + (scratch[2] + scratch[3]);
    if constexpr (LANES == 512) x += (scratch[4] + scratch[5]) + (scratch[6] + scratch[7]);
  }
  return x;
}

__device__ __forceinline__ float act(int32_t activation, float z) {
  const float s = sigmoidf(z);
  return activation == KDA_ACT_SILU ? z * s : s;
}
__device__ __forceinline__ void act_and_slope(int32_t activation, float z, float& a, float& slope) {
  const Sigmoids s = sigmoids(z);
  const bool silu = activation == KDA_ACT_SILU;
  a = silu ? z * s.up : s.up;
  slope = s.up * (silu ? 1.f + z * s.down : s.down);
}

// One lane's share of a row: vectors j LANES + lane of j = 0..NV-1.  WHOLE:
// the row is aligned vectors; else they lie at any address and the last is
// taken element by element.
template <int LANES, int NV, bool WHOLE>
struct Share {
  int32_t lane, V;
  __device__ __forceinline__ int32_t at(int j) const { return (j * LANES + lane) * 8; }
  __device__ __forceinline__ bool has(int j) const { return at(j) < V; }
  __device__ __forceinline__ bool whole(int j) const { return WHOLE ? has(j) : at(j) + 8 <= V; }
};

// Elements of a row of `src`, or `fill` behind its end and where src is null.
template <bool STREAM = false, int LANES, int NV, bool WHOLE, typename E>
__device__ __forceinline__ void load_row(const Share<LANES, NV, WHOLE>& sh, const E* src, float fill, float (&x)[NV][8]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (src != nullptr && sh.whole(j)) {
      if constexpr (WHOLE) {
        load<8, STREAM>(src + sh.at(j), x[j]);
      } else {
        load8_any(src + sh.at(j), x[j]);
      }
      continue;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[j][i] = fill;
    if (!WHOLE && src != nullptr && sh.has(j)) {
#pragma unroll
      for (int i = 0; i < 7; ++i) {
        float e[1] = {fill};
        if (sh.at(j) + i < sh.V) load<1>(src + sh.at(j) + i, e);
        x[j][i] = e[0];
      }
    }
  }
}
template <bool STREAM = false, int LANES, int NV, bool WHOLE, typename E>
__device__ __forceinline__ void store_row(const Share<LANES, NV, WHOLE>& sh, E* dst, const float (&x)[NV][8]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (sh.whole(j)) {
      if constexpr (WHOLE) {
        store<8, STREAM>(dst + sh.at(j), x[j]);
      } else {
        store8_any(dst + sh.at(j), x[j]);
      }
    } else if (!WHOLE && sh.has(j)) {
#pragma unroll
      for (int i = 0; i < 7; ++i) {
        const float e[1] = {x[j][i]};
        if (sh.at(j) + i < sh.V) store<1>(dst + sh.at(j) + i, e);
      }
    }
  }
}

template <typename O, typename E, bool WHOLE, bool STREAM, int LANES, int NV>
__global__ __launch_bounds__(kThreads<LANES>) void norm_kernel(NormParams p) {
  __shared__ float scratch[8];
  constexpr int kGroups = kThreads<LANES> / LANES;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kGroups + threadIdx.x / LANES;
  const int64_t token = id / p.H, head = id - token * p.H;
  if (token >= p.lanes) return;   // whole groups, so whole workgroups where the group is one
  const Share<LANES, NV, WHOLE> sh{static_cast<int32_t>(threadIdx.x % LANES), p.V};
  float w[NV][8], s[NV][8];
  load_row(sh, p.weight, 0.f, w);
  load_row(sh, p.res_scale == nullptr ? nullptr : p.res_scale + head * p.V, 1.f, s);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[j][i] *= s[j][i];
  }
  const float inv = 1.f / static_cast<float>(p.V);
  for (int64_t t = token; t < p.T; t += p.lanes) {
    const int64_t row = (t * p.H + head) * p.V;
    float o[NV][8], z[NV][8], res[NV][8];
    load_row<STREAM>(sh, static_cast<const O*>(p.o) + row, 0.f, o);
    load_row<STREAM>(sh, p.gate == nullptr ? nullptr : static_cast<const E*>(p.gate) + t * p.gate_stride + head * p.V, 0.f, z);
    load_row<STREAM>(sh, p.residual == nullptr ? nullptr : static_cast<const E*>(p.residual) + row, 0.f, res);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += (o[j][i] * inv) * o[j][i];   // the sum without 1 / V could overflow
    }
    const float r = rsqrtf(group_sum<LANES>(sum, scratch) + p.eps);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float y = o[j][i] * r * w[j][i];
        if (p.activation != KDA_ACT_NONE) y *= act(p.activation, z[j][i]);
        o[j][i] = y + res[j][i];
      }
    }
    store_row<STREAM>(sh, static_cast<E*>(p.y) + row, o);
  }
}

template <typename O, typename E, typename G, bool WHOLE, int LANES, int NV>
__global__ __launch_bounds__(kThreads<LANES>) void norm_backward_kernel(NormParams p) {
  __shared__ float scratch[8];
  constexpr int kGroups = kThreads<LANES> / LANES;
  __shared__ __align__(16) float part[kGroups > 1 ? kGroups : 1][LANES * 8 * NV];
  const int32_t group = threadIdx.x / LANES;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kGroups + group;
  const int64_t token = id / p.H, head = id - token * p.H;
  const bool active = token < p.lanes;
  const Share<LANES, NV, WHOLE> sh{static_cast<int32_t>(threadIdx.x % LANES), p.V};
  float w[NV][8], s[NV][8], m[NV][8];
  load_row(sh, p.weight, 0.f, w);
  load_row(sh, p.res_scale == nullptr ? nullptr : p.res_scale + head * p.V, 1.f, s);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m[j][i] = 0.f;
  }
  const float inv = 1.f / static_cast<float>(p.V);
  for (int64_t t = active ? token : p.T; t < p.T; t += p.lanes) {
    const int64_t row = (t * p.H + head) * p.V;
    float o[NV][8], z[NV][8], dy[NV][8];
    load_row(sh, static_cast<const O*>(p.o) + row, 0.f, o);
    load_row(sh, static_cast<const E*>(p.dy) + row, 0.f, dy);
    load_row(sh, p.gate == nullptr ? nullptr : static_cast<const E*>(p.gate) + t * p.gate_stride + head * p.V, 0.f, z);
    float sum = 0.f, dot = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float a = 1.f, slope = 0.f;
        if (p.activation != KDA_ACT_NONE) act_and_slope(p.activation, z[j][i], a, slope);
        z[j][i] = dy[j][i] * s[j][i] * w[j][i] * slope;   // d_z / n
        dy[j][i] *= a;                                    // dy act(z)
        const float share = o[j][i] * inv;                // as in the forward
        sum += share * o[j][i];
        dot += dy[j][i] * s[j][i] * w[j][i] * share;      // mean of dn o
      }
    }
    const float r = rsqrtf(group_sum<LANES>(sum, scratch) + p.eps);
    const float c = group_sum<LANES>(dot, scratch) * r;   // mean(dn n)
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = o[j][i] * r;
        m[j][i] += dy[j][i] * n;
        z[j][i] *= n;
        o[j][i] = r * (dy[j][i] * s[j][i] * w[j][i] - n * c);
      }
    }
    store_row(sh, static_cast<G*>(p.d_o) + row, o);
    if (p.gate != nullptr) store_row(sh, static_cast<E*>(p.d_gate) + row, z);
  }
  // ds: this group's sum of m; dw: the workgroup's sum of s m, of an idle group
  // zeros whatever s is
  if (active && p.res_scale != nullptr) store_row(sh, p.scale_part + (token * p.H + head) * p.V, m);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m[j][i] = active ? m[j][i] * s[j][i] : 0.f;
  }
  if constexpr (kGroups == 1) {
    store_row(sh, p.weight_part + static_cast<int64_t>(blockIdx.x) * p.V, m);
  } else {
    store_row(sh, &part[group][0], m);
    __syncthreads();
    for (int32_t v = threadIdx.x; v < p.V; v += kThreads<LANES>) {
      float sum = 0.f;
      for (int i = 0; i < kGroups; ++i) sum += part[i][v];
      p.weight_part[static_cast<int64_t>(blockIdx.x) * p.V + v] = sum;
    }
  }
}

// Column sums of the partial rows, 64 columns a workgroup: d_weight over
// weight_part[blocks][V] (the first weight_blocks workgroups), d_res_scale
// over scale_part[lanes][H V], times the weight (the rest).
__global__ __launch_bounds__(1024) void norm_reduce_kernel(NormParams p, int32_t blocks, int32_t weight_blocks,
                                                           float* d_weight, float* d_res_scale) {
  __shared__ float part[16][64];
  const int32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, block = static_cast<int32_t>(blockIdx.x);
  const bool is_weight = block < weight_blocks;
  const int64_t columns = is_weight ? p.V : static_cast<int64_t>(p.H) * p.V;
  const int64_t col = static_cast<int64_t>(is_weight ? block : block - weight_blocks) * 64 + lane;
  const float* src = is_weight ? p.weight_part : p.scale_part;
  const int32_t rows = is_weight ? blocks : p.lanes;
  float sum = col < columns ? column_sum(src + col, columns, wave, rows) : 0.f;
  part[wave][lane] = sum;
  __syncthreads();
  if (wave == 0 && col < columns) {
    for (int i = 1; i < 16; ++i) sum += part[i][lane];
    if (is_weight) {
      d_weight[col] = sum;
    } else {
      d_res_scale[col] = sum * p.weight[col % p.V];
    }
  }
}

NormParams params_of(const NormArgs& a, const RowGrid& grid) {
  NormParams p{};
  p.o = a.o.ptr;
  p.gate = a.gate.ptr;
  p.residual = a.residual.ptr;
  p.dy = a.dy.ptr;
  p.gate_stride = a.gate.stride;
  p.weight = static_cast<const float*>(a.weight.ptr);
  p.res_scale = static_cast<const float*>(a.res_scale.ptr);
  p.eps = a.eps;
  p.T = a.T;
  p.H = a.H;
  p.V = a.V;
  p.lanes = grid.lanes;
  p.activation = a.activation;
  p.y = a.y.ptr;
  p.d_o = a.d_o.ptr;
  p.d_gate = a.d_gate.ptr;
  return p;
}

// Calls f with the lane group's shape as template arguments.
template <typename F>
void with_shape(const NormShape& s, F&& f) {
  if (s.lanes == 16) return f.template operator()<16, 1>();
  if (s.lanes == 32) return f.template operator()<32, 1>();
  if (s.lanes == 64 && s.vectors == 1) return f.template operator()<64, 1>();
  if (s.lanes == 64) return f.template operator()<64, 2>();
  if (s.lanes == 256 && s.vectors == 1) return f.template operator()<256, 1>();
  if (s.lanes == 256) return f.template operator()<256, 2>();
  return f.template operator()<512, 2>();
}

template <typename O, typename E>
struct LaunchForward {
  NormParams p;
  RowGrid grid;
  bool whole, past_caches;
  hipStream_t stream;
  template <int LANES, int NV>
  void operator()() const {
    void (*kernel)(NormParams) = !whole        ? norm_kernel<O, E, false, false, LANES, NV>
                                 : past_caches ? norm_kernel<O, E, true, true, LANES, NV>
                                               : norm_kernel<O, E, true, false, LANES, NV>;
    hipLaunchKernelGGL(kernel, dim3(grid.blocks), dim3(kThreads<LANES>), 0, stream, p);
  }
};
template <typename O, typename E, typename G>
struct LaunchBackward {
  NormParams p;
  RowGrid grid;
  bool whole;
  hipStream_t stream;
  template <int LANES, int NV>
  void operator()() const {
    void (*kernel)(NormParams) =
        whole ? norm_backward_kernel<O, E, G, true, LANES, NV> : norm_backward_kernel<O, E, G, false, LANES, NV>;
    hipLaunchKernelGGL(kernel, dim3(grid.blocks), dim3(kThreads<LANES>), 0, stream, p);
  }
};

constexpr int kNormBlocks = 1024;   // four workgroups a CU: 415 us at 65536 x 32 heads, 461 with eight

}  // namespace

int launch_norm(const NormArgs& a, hipStream_t stream) {
  const NormShape shape = norm_shape(a.V);
  const bool whole = norm_whole_rows(a);
  const RowGrid grid = row_grid(a.T, a.H, norm_threads(shape) / shape.lanes, kNormBlocks);
  const NormParams p = params_of(a, grid);
  (void)hipGetLastError();
  const bool o16 = a.o_format == KDA_BF16, e16 = a.dtype == KDA_BF16;
  // Gate, fp32 o, bf16: at 2.1 GB past the caches 381 us against 415, at 268 MB
  // 95 and 101, at 134 MB (a quarter of it from the cache) 27 and 25.
  const int64_t per = (o16 ? 2 : 4) + (e16 ? 2 : 4) * (1 + (a.gate.ptr != nullptr) + (a.residual.ptr != nullptr));
  const bool past = static_cast<int64_t>(a.T) * a.H * a.V * per >= kStreamBytes;
  if (o16 && e16) with_shape(shape, LaunchForward<bf16_t, bf16_t>{p, grid, whole, past, stream});
  if (o16 && !e16) with_shape(shape, LaunchForward<bf16_t, fp32_t>{p, grid, whole, past, stream});
  if (!o16 && e16) with_shape(shape, LaunchForward<fp32_t, bf16_t>{p, grid, whole, past, stream});
  if (!o16 && !e16) with_shape(shape, LaunchForward<fp32_t, fp32_t>{p, grid, whole, past, stream});
  return finish_launch();
}

int launch_norm_backward(const NormArgs& a, hipStream_t stream) {
  const NormShape shape = norm_shape(a.V);
  const bool whole = norm_whole_rows(a);
  const NormBwdLayout L = norm_bwd_layout(a.T, a.H, a.V, a.o_format);
  NormParams p = params_of(a, L.grid);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace.ptr);
  p.weight_part = reinterpret_cast<float*>(ws + L.weight);
  p.scale_part = reinterpret_cast<float*>(ws + L.scale);
  (void)hipGetLastError();
  const bool o16 = a.o_format == KDA_BF16, e16 = a.dtype == KDA_BF16, g16 = a.d_o_format == KDA_BF16;
  if (o16 && e16 && g16) with_shape(shape, LaunchBackward<bf16_t, bf16_t, bf16_t>{p, L.grid, whole, stream});
  if (o16 && e16 && !g16) with_shape(shape, LaunchBackward<bf16_t, bf16_t, fp32_t>{p, L.grid, whole, stream});
  if (o16 && !e16 && g16) with_shape(shape, LaunchBackward<bf16_t, fp32_t, bf16_t>{p, L.grid, whole, stream});
  if (o16 && !e16 && !g16) with_shape(shape, LaunchBackward<bf16_t, fp32_t, fp32_t>{p, L.grid, whole, stream});
  if (!o16 && e16 && g16) with_shape(shape, LaunchBackward<fp32_t, bf16_t, bf16_t>{p, L.grid, whole, stream});
  if (!o16 && e16 && !g16) with_shape(shape, LaunchBackward<fp32_t, bf16_t, fp32_t>{p, L.grid, whole, stream});
  if (!o16 && !e16 && g16) with_shape(shape, LaunchBackward<fp32_t, fp32_t, bf16_t>{p, L.grid, whole, stream});
  if (!o16 && !e16 && !g16) with_shape(shape, LaunchBackward<fp32_t, fp32_t, fp32_t>{p, L.grid, whole, stream});
  const int st = finish_launch();
  if (st != KDA_OK) return st;
  const int64_t weight_blocks = (a.V + 63) / 64;
  const int64_t scale_blocks = a.res_scale.ptr == nullptr ? 0 : (static_cast<int64_t>(a.H) * a.V + 63) / 64;
  hipLaunchKernelGGL(norm_reduce_kernel, dim3(static_cast<uint32_t>(weight_blocks + scale_blocks)), dim3(1024), 0,
                     stream, p, L.grid.blocks, static_cast<int32_t>(weight_blocks),
                     static_cast<float*>(a.d_weight.ptr), static_cast<float*>(a.d_res_scale.ptr));
  return finish_launch();
}

}  // namespace kda
