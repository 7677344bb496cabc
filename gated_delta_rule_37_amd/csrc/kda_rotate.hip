// The norms of queries and keys per head and their rotation by position
// (kda_qk_norm_rotate) and the gradients.
//
// Per (token, head) row x of D channels, all in FP32:
//   n = w x r, r = (mean x^2 + eps)^(-1/2), q also times q_scale
//   pairs (a, b) of the first R channels: a cos t - b sin t, a sin t + b cos t
// and for a cotangent d, with m = d turned by -t and times q_scale:
//   dw = sum m x r,  dx = r (w m - x r mean(w m x r)).
//
// The angle t = position * inv_freq reaches 10^6 radians, where FP32 keeps no
// digit of it: turns = position (inv_freq / 2 pi) in FP64, whose fraction is
// exact to 10^-10, then the sine and cosine of the FP32 fraction.  A workgroup
// makes them once for its tokens, in LDS, for all heads.
//
// A row is L lanes of 16 channels, held as 8 pairs, so that a rotation needs no
// other lane; a lane's two 16-byte loads are neighbouring channels where those
// are paired, else the two halves.  Both directions only stream, so HBM bounds
// them: 32768 tokens x 40 heads of 128 BF16 channels take 118 us (5.7 TB/s),
// gradients of 8191 x 32 heads 38 us and 4 for the sums over the tokens (201 MB),
// calls of up to 2048 tokens the host's 11.
#include "kda_layer.h"
#include "kda_layer_device.h"

#include "kda.h"

namespace kda {
namespace {

struct RotateParams {
  const void *q_raw, *k_raw;
  int64_t q_stride, k_stride;
  const int32_t* positions;
  const float *inv_freq, *q_weight, *k_weight;
  float q_scale, eps;
  int32_t T, Hq, Hk, D, R, tokens;   // tokens: a workgroup's at a time
  int32_t interleaved, tiles, row_blocks;
  void *q, *k;                       // forward: outputs; backward: gradients of the raw rows
  const void *dq, *dk;
  float* part;                       // backward: [blocks][2][D]
};

// Sum over the 4, 8 or 16 lanes of a row, the same bits in each.
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}
template <int L>
__device__ __forceinline__ float sum_lanes(float x) {
  x += dpp<0xb1>(x);                        // the lane beside
  x += dpp<0x4e>(x);                        // the pair beside
  if constexpr (L >= 8) x += dpp<0x141>(x); // the quad beside
  if constexpr (L >= 16) x += dpp<0x140>(x);
  return x;
}

// A lane's 8 pairs of a row of D channels.  WHOLE: pairs 8 lane .. 8 lane + 7 by
// 16-byte vectors; otherwise pairs lane, lane + L, ... one element at a time.
// Pair p is rotated if p < R / 2.
template <int L, bool WHOLE>
struct Pairs {
  int32_t lane, D, R;
  bool interleaved;

  __device__ __forceinline__ int32_t pair(int i) const { return WHOLE ? 8 * lane + i : lane + L * i; }
  __device__ __forceinline__ bool has(int i) const { return pair(i) < D / 2; }
  __device__ __forceinline__ bool turned(int i) const { return pair(i) < R / 2; }
  // the pair's channels; those behind R are paired in halves too
  __device__ __forceinline__ int32_t first(int32_t p) const {
    if (interleaved) return 2 * p;
    return p < R / 2 ? p : p + R / 2;
  }
  __device__ __forceinline__ int32_t second(int32_t p) const {
    if (interleaved) return 2 * p + 1;
    return p < R / 2 ? p + R / 2 : p + D / 2;
  }

  template <bool STREAM, typename E>
  __device__ __forceinline__ void load(const E* row, float (&a)[8], float (&b)[8]) const {
    if constexpr (WHOLE) {
      if (interleaved) {
        float x[8], y[8];
        kda::load<8, STREAM>(row + 16 * lane, x);
        kda::load<8, STREAM>(row + 16 * lane + 8, y);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = x[2 * i];
          b[i] = x[2 * i + 1];
          a[4 + i] = y[2 * i];
          b[4 + i] = y[2 * i + 1];
        }
      } else {
        kda::load<8, STREAM>(row + first(8 * lane), a);
        kda::load<8, STREAM>(row + second(8 * lane), b);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float x[1] = {0.f}, y[1] = {0.f};
        if (has(i)) {
          kda::load<1>(row + first(pair(i)), x);
          kda::load<1>(row + second(pair(i)), y);
        }
        a[i] = x[0];
        b[i] = y[0];
      }
    }
  }

  template <bool STREAM, typename E>
  __device__ __forceinline__ void store(E* row, const float (&a)[8], const float (&b)[8]) const {
    if constexpr (WHOLE) {
      if (interleaved) {
        float x[8], y[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[2 * i] = a[i];
          x[2 * i + 1] = b[i];
          y[2 * i] = a[4 + i];
          y[2 * i + 1] = b[4 + i];
        }
        kda::store<8, STREAM>(row + 16 * lane, x);
        kda::store<8, STREAM>(row + 16 * lane + 8, y);
      } else {
        kda::store<8, STREAM>(row + first(8 * lane), a);
        kda::store<8, STREAM>(row + second(8 * lane), b);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (has(i)) {
          const float x[1] = {a[i]}, y[1] = {b[i]};
          kda::store<1>(row + first(pair(i)), x);
          kda::store<1>(row + second(pair(i)), y);
        }
      }
    }
  }

  // a weight times `scale`, or `scale` itself
  __device__ __forceinline__ void weight(const float* w, float scale, float (&a)[8], float (&b)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = b[i] = 1.f;
    if (w != nullptr && (!WHOLE || has(0))) load<false>(w, a, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a[i] *= scale;
      b[i] *= scale;
    }
  }
};

constexpr int kMaxPairs = 128;

// Cosine and sine of the turns of tokens t0 .. t0 + tokens - 1.
__device__ __forceinline__ void make_angles(const RotateParams& p, int32_t t0, int32_t tokens, float2* table) {
  const int32_t half = p.R / 2;
  for (int32_t i = threadIdx.x; i < tokens * half; i += kRowThreads) {
    const int32_t t = i / half, f = i - t * half;
    if (t0 + t >= p.T) break;
    // 1 / (2 pi)
    double turns = static_cast<double>(p.positions[t0 + t]) * (static_cast<double>(p.inv_freq[f]) * 0.15915494309189535);
    turns -= rint(turns);
    float s, c;
    sincospif(static_cast<float>(2.0 * turns), &s, &c);
    table[t * kMaxPairs + f] = make_float2(c, s);
  }
}

// One row's place: token of the tile, head, and whether it is a query's.
struct Place {
  int32_t token, head;
  bool query;
};
__device__ __forceinline__ Place place_of(const RotateParams& p, int32_t r) {
  const int32_t heads = p.Hq + p.Hk;
  Place w;
  w.token = r / heads;
  const int32_t h = r - w.token * heads;
  w.query = h < p.Hq;
  w.head = w.query ? h : h - p.Hq;
  return w;
}

constexpr int kRotateTokens = 4;

template <typename E, int L, bool WHOLE, bool STREAM>
__global__ __launch_bounds__(kRowThreads) void rotate_kernel(RotateParams p) {
  __shared__ float2 table[kRotateTokens * kMaxPairs];
  constexpr int kGroups = kRowThreads / L;
  const int32_t tile = static_cast<int32_t>(blockIdx.x / static_cast<uint32_t>(p.row_blocks));
  const int32_t part = static_cast<int32_t>(blockIdx.x % static_cast<uint32_t>(p.row_blocks));
  const int32_t t0 = tile * p.tokens;
  const int32_t tokens = min(p.tokens, p.T - t0), rows = tokens * (p.Hq + p.Hk);
  make_angles(p, t0, tokens, table);
  const Pairs<L, WHOLE> lanes{static_cast<int32_t>(threadIdx.x) % L, p.D, p.R, p.interleaved != 0};
  const bool active = !WHOLE || lanes.has(0);
  float qa[8], qb[8], ka[8], kb[8];
  lanes.weight(p.q_weight, p.q_scale, qa, qb);
  lanes.weight(p.k_weight, 1.f, ka, kb);
  __syncthreads();
  const float inv_d = 1.f / static_cast<float>(p.D);
  const int32_t group = static_cast<int32_t>(threadIdx.x) / L;
  for (int32_t r = part * kGroups + group; r < rows; r += p.row_blocks * kGroups) {
    const Place w = place_of(p, r);
    const int64_t t = t0 + w.token;
    const E* in = w.query ? static_cast<const E*>(p.q_raw) + t * p.q_stride : static_cast<const E*>(p.k_raw) + t * p.k_stride;
    float a[8], b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = b[i] = 0.f;
    if (active) lanes.template load<STREAM>(in + static_cast<int64_t>(w.head) * p.D, a, b);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += a[i] * (a[i] * inv_d) + b[i] * (b[i] * inv_d);
    const float scale = rsqrtf(sum_lanes<L>(sum) + p.eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = a[i] * scale * (w.query ? qa[i] : ka[i]), y = b[i] * scale * (w.query ? qb[i] : kb[i]);
      const bool turn = lanes.turned(i);
      const float2 c = turn ? table[w.token * kMaxPairs + lanes.pair(i)] : make_float2(1.f, 0.f);
      a[i] = turn ? x * c.x - y * c.y : x;
      b[i] = turn ? x * c.y + y * c.x : y;
    }
    E* out = w.query ? static_cast<E*>(p.q) + (t * p.Hq + w.head) * p.D : static_cast<E*>(p.k) + (t * p.Hk + w.head) * p.D;
    if (active) lanes.template store<STREAM>(out, a, b);
  }
}

template <typename E, typename G, int L, bool WHOLE>
__global__ __launch_bounds__(kRowThreads) void rotate_backward_kernel(RotateParams p) {
  __shared__ float2 table[kRotateTokens * kMaxPairs];
  __shared__ float sums[kRowThreads / 64][2][2 * kMaxPairs];
  constexpr int kGroups = kRowThreads / L;
  const Pairs<L, WHOLE> lanes{static_cast<int32_t>(threadIdx.x) % L, p.D, p.R, p.interleaved != 0};
  const bool active = !WHOLE || lanes.has(0);
  float qa[8], qb[8], ka[8], kb[8];
  lanes.weight(p.q_weight, 1.f, qa, qb);
  lanes.weight(p.k_weight, 1.f, ka, kb);
  float wqa[8], wqb[8], wka[8], wkb[8];   // this lane's sums for the weights
#pragma unroll
  for (int i = 0; i < 8; ++i) wqa[i] = wqb[i] = wka[i] = wkb[i] = 0.f;
  const float inv_d = 1.f / static_cast<float>(p.D);
  const int32_t group = static_cast<int32_t>(threadIdx.x) / L;
  for (int32_t tile = static_cast<int32_t>(blockIdx.x); tile < p.tiles; tile += static_cast<int32_t>(gridDim.x)) {
    const int32_t t0 = tile * p.tokens;
    const int32_t tokens = min(p.tokens, p.T - t0), rows = tokens * (p.Hq + p.Hk);
    __syncthreads();   // the last tile's readers
    make_angles(p, t0, tokens, table);
    __syncthreads();
    for (int32_t r = group; r < rows; r += kGroups) {
      const Place w = place_of(p, r);
      const int64_t t = t0 + w.token;
      const E* in = w.query ? static_cast<const E*>(p.q_raw) + t * p.q_stride : static_cast<const E*>(p.k_raw) + t * p.k_stride;
      const int64_t at = w.query ? (t * p.Hq + w.head) * p.D : (t * p.Hk + w.head) * p.D;
      float a[8], b[8], da[8], db[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] = b[i] = da[i] = db[i] = 0.f;
      if (active) {
        lanes.template load<false>(in + static_cast<int64_t>(w.head) * p.D, a, b);
        lanes.template load<false>(static_cast<const G*>(w.query ? p.dq : p.dk) + at, da, db);
      }
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += a[i] * (a[i] * inv_d) + b[i] * (b[i] * inv_d);
      const float scale = rsqrtf(sum_lanes<L>(sum) + p.eps), s = w.query ? p.q_scale : 1.f;
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool turn = lanes.turned(i);
        const float2 c = turn ? table[w.token * kMaxPairs + lanes.pair(i)] : make_float2(1.f, 0.f);
        const float x = s * (turn ? da[i] * c.x + db[i] * c.y : da[i]), y = s * (turn ? db[i] * c.x - da[i] * c.y : db[i]);
        a[i] *= scale;   // x r first: the product x r^2 of a row near zero would overflow
        b[i] *= scale;
        if (w.query) {
          wqa[i] += x * a[i];
          wqb[i] += y * b[i];
        } else {
          wka[i] += x * a[i];
          wkb[i] += y * b[i];
        }
        da[i] = x * (w.query ? qa[i] : ka[i]);
        db[i] = y * (w.query ? qb[i] : kb[i]);
        dot += da[i] * (a[i] * inv_d) + db[i] * (b[i] * inv_d);
      }
      dot = sum_lanes<L>(dot);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        da[i] = scale * (da[i] - a[i] * dot);
        db[i] = scale * (db[i] - b[i] * dot);
      }
      if (active) lanes.template store<false>(static_cast<E*>(w.query ? p.q : p.k) + at, da, db);
    }
  }
  if (p.part == nullptr) return;
  // the groups of a wave, then the waves, in a fixed order
  const int32_t wave = threadIdx.x >> 6;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int m = L; m < 64; m *= 2) {
      wqa[i] += __shfl_xor(wqa[i], m);
      wqb[i] += __shfl_xor(wqb[i], m);
      wka[i] += __shfl_xor(wka[i], m);
      wkb[i] += __shfl_xor(wkb[i], m);
    }
    if ((threadIdx.x & 63) < L && lanes.has(i)) {
      const int32_t first = lanes.first(lanes.pair(i)), second = lanes.second(lanes.pair(i));
      sums[wave][0][first] = wqa[i];
      sums[wave][0][second] = wqb[i];
      sums[wave][1][first] = wka[i];
      sums[wave][1][second] = wkb[i];
    }
  }
  __syncthreads();
  float* out = p.part + static_cast<int64_t>(blockIdx.x) * 2 * p.D;
  for (int32_t c = threadIdx.x; c < 2 * p.D; c += kRowThreads) {
    const int32_t which = c >= p.D ? 1 : 0, ch = c - which * p.D;
    out[c] = (sums[0][which][ch] + sums[1][which][ch]) + (sums[2][which][ch] + sums[3][which][ch]);
  }
}

// The weights' gradients from the workgroups' sums: 64 columns a workgroup, 16
// waves take every sixteenth row.
__global__ __launch_bounds__(1024) void rotate_reduce_kernel(const float* part, int32_t blocks, int32_t D, float* dq_weight,
                                                             float* dk_weight) {
  __shared__ float sums[16][64];
  const int32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = static_cast<int32_t>(blockIdx.x) * 64 + lane;
  float sum = col < 2 * D ? column_sum(part + col, 2 * D, wave, blocks) : 0.f;
  sums[wave][lane] = sum;
  __syncthreads();
  if (wave == 0 && col < 2 * D) {
    for (int i = 1; i < 16; ++i) sum += sums[i][lane];
    float* out = col < D ? dq_weight : dk_weight;
    if (out != nullptr) out[col < D ? col : col - D] = sum;
  }
}

RotateParams params_of(const RotateArgs& a, const RotateGrid& grid) {
  RotateParams p{};
  p.q_raw = a.q_raw.ptr;
  p.k_raw = a.k_raw.ptr;
  p.q_stride = a.q_raw.stride;
  p.k_stride = a.k_raw.stride;
  p.positions = static_cast<const int32_t*>(a.positions.ptr);
  p.inv_freq = static_cast<const float*>(a.inv_freq.ptr);
  p.q_weight = static_cast<const float*>(a.q_weight.ptr);
  p.k_weight = static_cast<const float*>(a.k_weight.ptr);
  p.q_scale = a.q_scale;
  p.eps = a.eps;
  p.T = a.T;
  p.Hq = a.Hq;
  p.Hk = a.Hk;
  p.D = a.D;
  p.R = a.R;
  p.tokens = grid.tokens;
  p.interleaved = a.interleaved;
  p.tiles = grid.tiles;
  p.row_blocks = grid.row_blocks;
  p.q = a.q.ptr;
  p.k = a.k.ptr;
  return p;
}

template <typename E, bool STREAM>
void (*forward_of(int32_t D, bool whole))(RotateParams) {
  if (!whole) return rotate_kernel<E, 16, false, false>;
  return D <= 64 ? rotate_kernel<E, 4, true, STREAM> : D <= 128 ? rotate_kernel<E, 8, true, STREAM> : rotate_kernel<E, 16, true, STREAM>;
}
template <typename E, typename G>
void (*backward_of(int32_t D, bool whole))(RotateParams) {
  if (!whole) return rotate_backward_kernel<E, G, 16, false>;
  return D <= 64 ? rotate_backward_kernel<E, G, 4, true> : D <= 128 ? rotate_backward_kernel<E, G, 8, true>
                                                                    : rotate_backward_kernel<E, G, 16, true>;
}

}  // namespace

int launch_rotate(const RotateArgs& a, hipStream_t stream) {
  const RotateGrid grid = rotate_grid(a, false);
  const RotateParams p = params_of(a, grid);
  const bool whole = rotate_whole_rows(a), e16 = a.dtype == KDA_BF16;
  const bool past = static_cast<int64_t>(a.T) * (a.Hq + a.Hk) * a.D * (e16 ? 4 : 8) >= kStreamBytes;
  void (*kernel)(RotateParams) = e16 ? (past ? forward_of<bf16_t, true>(a.D, whole) : forward_of<bf16_t, false>(a.D, whole))
                                     : (past ? forward_of<fp32_t, true>(a.D, whole) : forward_of<fp32_t, false>(a.D, whole));
  const int64_t blocks = static_cast<int64_t>(grid.tiles) * grid.row_blocks;
  if (blocks * kRowThreads > 2147483647LL) return KDA_ERR_UNSUPPORTED;
  (void)hipGetLastError();
  hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(blocks)), dim3(kRowThreads), 0, stream, p);
  return finish_launch();
}

int launch_rotate_backward(const RotateArgs& a, hipStream_t stream) {
  const RotateGrid grid = rotate_grid(a, true);
  RotateParams p = params_of(a, grid);
  p.dq = a.dq.ptr;
  p.dk = a.dk.ptr;
  const bool weights = a.dq_weight.ptr != nullptr || a.dk_weight.ptr != nullptr;
  p.part = weights ? static_cast<float*>(a.workspace.ptr) : nullptr;
  const bool whole = rotate_whole_rows(a), e16 = a.dtype == KDA_BF16, d16 = a.d_format == KDA_BF16;
  void (*kernel)(RotateParams) = e16 ? (d16 ? backward_of<bf16_t, bf16_t>(a.D, whole) : backward_of<bf16_t, fp32_t>(a.D, whole))
                                     : (d16 ? backward_of<fp32_t, bf16_t>(a.D, whole) : backward_of<fp32_t, fp32_t>(a.D, whole));
  (void)hipGetLastError();
  hipLaunchKernelGGL(kernel, dim3(grid.blocks), dim3(kRowThreads), 0, stream, p);
  const int st = finish_launch();
  if (st != KDA_OK || !weights) return st;
  hipLaunchKernelGGL(rotate_reduce_kernel, dim3((2 * a.D + 63) / 64), dim3(1024), 0, stream, p.part, grid.blocks, a.D,
                     static_cast<float*>(a.dq_weight.ptr), static_cast<float*>(a.dk_weight.ptr));
  return finish_launch();
}

}  // namespace kda
