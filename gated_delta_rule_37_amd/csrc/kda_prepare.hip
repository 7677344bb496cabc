// The norms before the recurrence and its gates (kda_prepare_inputs) and
// their gradients.
//
// Per (token, head) row of 128 channels, all in FP32:
//   q = s x r, r = (sum x^2 + eps)^(-1/2); k the same with s = 1
//   g = -e^a softplus(z), z = gate + bias; beta = sigmoid(b)
// and for cotangents d of them
//   dx = s r (d - x r^2 sum(x d)),  dgate = -e^a d sigmoid(z),
//   da = sum d g,  dbias = sum over tokens of dgate,  db = d beta (1 - beta).
//
// A row is 16 lanes of 8 channels: one 16-byte load a tensor (bf16), the row
// sum four DPP rotations.  Neighbouring groups take neighbouring rows, and the
// step between a group's rows is a multiple of the heads, so that its head, and
// with it a_log and the bias, stays.  Both directions only stream: each element
// is read and written once, so HBM bandwidth bounds them.  bf16, 32768 x 32
// heads forward 317 us, 5.1 TB/s; 8191 x 16 backward 79 us, 5.1 TB/s, and 5 us
// for the sums over the tokens (a large copy: 5.2 TB/s).  fp32, 16384 x 32
// forward 227 us, 5.3 TB/s; 8191 x 16 backward 123 us with its sums, 4.9.
#include "kda_layer.h"
#include "kda_layer_device.h"

#include "kda.h"

namespace kda {
namespace {

struct PrepareParams {
  const void *q_raw, *k_raw, *gate_raw, *beta_raw;
  int64_t q_stride, k_stride, gate_stride, beta_stride;
  const float *a_log, *dt_bias;
  float q_scale, eps;
  int32_t T, H, lanes;   // lanes: P, the tokens in flight for one head
  void *q, *k, *g, *beta;
  const float *dq, *dk, *dg, *dbeta;
  float *bias_part, *decay_part;
};

// softplus(z) = max(z, 0) + log1p(t), t = e^-|z|, with log1p(t) =
// 2 atanh(s), s = t / (2 + t) <= 1/3: the odd series to s^15 leaves 2^-26, and
// no branch or cancellation loses relative precision where t is small.  EXACT:
// for a result in fp32 (the forward's is rounded to bf16: 316 us against 318 at
// 32768 x 32 heads).
template <bool EXACT>
__device__ __forceinline__ float softplusf(float z) {
  const float t = EXACT ? exact_exp(-fabsf(z)) : fast_exp(-fabsf(z)), s = t * __builtin_amdgcn_rcpf(2.f + t), w = s * s;
  float a = 1.f / 15.f;
  a = a * w + 1.f / 13.f;
  a = a * w + 1.f / 11.f;
  a = a * w + 1.f / 9.f;
  a = a * w + 1.f / 7.f;
  a = a * w + 1.f / 5.f;
  a = a * w + 1.f / 3.f;
  a = a * w + 1.f;
  return fmaxf(z, 0.f) + (s + s) * a;
}

// The row's lane group: row index within one step of the grid, its head and
// first token.
struct Group {
  int32_t lane, head, token;
  bool active;
};
__device__ __forceinline__ Group group_of(const PrepareParams& p) {
  Group w;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kPrepareGroups + (threadIdx.x >> 4);
  w.lane = threadIdx.x & 15;
  w.token = static_cast<int32_t>(id / p.H);
  w.head = static_cast<int32_t>(id - static_cast<int64_t>(w.token) * p.H);
  w.active = w.token < p.lanes;
  return w;
}

template <typename E, bool STREAM>
__global__ __launch_bounds__(kRowThreads) void prepare_kernel(PrepareParams p) {
  const Group w = group_of(p);
  if (!w.active) return;
  const int32_t c0 = w.lane * 8;
  const int64_t col = static_cast<int64_t>(w.head) * 128 + c0;
  const float rate = -exact_exp(p.a_log[w.head]);
  float bias[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (p.dt_bias != nullptr) load<8>(p.dt_bias + col, bias);
  for (int64_t t = w.token; t < p.T; t += p.lanes) {
    float q[8], k[8], z[8];
    load<8, STREAM>(static_cast<const E*>(p.q_raw) + t * p.q_stride + col, q);
    load<8, STREAM>(static_cast<const E*>(p.k_raw) + t * p.k_stride + col, k);
    load<8, STREAM>(static_cast<const E*>(p.gate_raw) + t * p.gate_stride + col, z);
    float b[1] = {0.f};
    if (w.lane == 0) load<1>(static_cast<const E*>(p.beta_raw) + t * p.beta_stride + w.head, b);
    float sq = 0.f, sk = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sq += q[i] * q[i];
      sk += k[i] * k[i];
    }
    const float rq = p.q_scale * rsqrtf(sum16(sq) + p.eps), rk = rsqrtf(sum16(sk) + p.eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      q[i] *= rq;
      k[i] *= rk;
      z[i] = rate * softplusf<false>(z[i] + bias[i]);
    }
    const int64_t row = t * p.H + w.head, out = row * 128 + c0;
    store<8, STREAM>(static_cast<bf16_t*>(p.q) + out, q);
    store<8, STREAM>(static_cast<bf16_t*>(p.k) + out, k);
    store<8, STREAM>(static_cast<bf16_t*>(p.g) + out, z);
    if (w.lane == 0) {
      b[0] = sigmoidf(b[0]);
      store<1>(static_cast<bf16_t*>(p.beta) + row, b);
    }
  }
}

template <typename E>
__global__ __launch_bounds__(kRowThreads) void prepare_backward_kernel(PrepareParams p) {
  const Group w = group_of(p);
  if (!w.active) return;
  const int32_t c0 = w.lane * 8;
  const int64_t col = static_cast<int64_t>(w.head) * 128 + c0;
  const float rate = -exact_exp(p.a_log[w.head]);
  float bias[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (p.dt_bias != nullptr) load<8>(p.dt_bias + col, bias);
  float sum_bias[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  float sum_decay = 0.f;
  for (int64_t t = w.token; t < p.T; t += p.lanes) {
    const int64_t row = t * p.H + w.head, at = row * 128 + c0;
    float q[8], k[8], z[8], dq[8], dk[8], dg[8];
    load<8>(static_cast<const E*>(p.q_raw) + t * p.q_stride + col, q);
    load<8>(static_cast<const E*>(p.k_raw) + t * p.k_stride + col, k);
    load<8>(static_cast<const E*>(p.gate_raw) + t * p.gate_stride + col, z);
    load<8>(p.dq + at, dq);
    load<8>(p.dk + at, dk);
    load<8>(p.dg + at, dg);
    float b[1] = {0.f}, db = 0.f;
    if (w.lane == 0) {
      load<1>(static_cast<const E*>(p.beta_raw) + t * p.beta_stride + w.head, b);
      db = p.dbeta[row];
    }
    float sq = 0.f, sk = 0.f, xq = 0.f, xk = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sq += q[i] * q[i];
      sk += k[i] * k[i];
      xq += q[i] * dq[i];
      xk += k[i] * dk[i];
    }
    const float rq = rsqrtf(sum16(sq) + p.eps), rk = rsqrtf(sum16(sk) + p.eps);
    // x r first: the product x r^2 of a row near zero would overflow
    const float pq = rq * sum16(xq), pk = rk * sum16(xk);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      dq[i] = p.q_scale * rq * (dq[i] - (q[i] * rq) * pq);
      dk[i] = rk * (dk[i] - (k[i] * rk) * pk);
      const float v = z[i] + bias[i];
      sum_decay += dg[i] * rate * softplusf<true>(v);
      dg[i] = dg[i] * rate * sigmoidf(v);
      sum_bias[i] += dg[i];
    }
    store<8>(static_cast<E*>(p.q) + at, dq);
    store<8>(static_cast<E*>(p.k) + at, dk);
    store<8>(static_cast<E*>(p.g) + at, dg);
    if (w.lane == 0) {
      const Sigmoids s = sigmoids(b[0]);
      b[0] = db * s.up * s.down;
      store<1>(static_cast<E*>(p.beta) + row, b);
    }
  }
  const int64_t part = static_cast<int64_t>(w.token) * p.H + w.head;
  store<8>(p.bias_part + part * 128 + c0, sum_bias);
  sum_decay = sum16(sum_decay);
  if (w.lane == 0) p.decay_part[part] = sum_decay;
}

// Sums of the partial rows: ddt_bias[h, c] over bias_part[p][h][c] (the first
// bias_blocks workgroups, 64 columns each), da_log[h] over decay_part[p][h]
// (the rest).  16 waves take every sixteenth partial row.
__global__ __launch_bounds__(1024) void prepare_reduce_kernel(const float* bias_part, const float* decay_part,
                                                              int32_t lanes, int32_t H, int32_t bias_blocks,
                                                              float* ddt_bias, float* da_log) {
  __shared__ float part[16][64];
  const int32_t block = static_cast<int32_t>(blockIdx.x), lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const bool is_bias = block < bias_blocks;
  const int64_t columns = is_bias ? static_cast<int64_t>(H) * 128 : H;
  const int64_t col = static_cast<int64_t>(is_bias ? block : block - bias_blocks) * 64 + lane;
  const float* src = is_bias ? bias_part : decay_part;
  float sum = col < columns ? column_sum(src + col, columns, wave, lanes) : 0.f;
  part[wave][lane] = sum;
  __syncthreads();
  if (wave == 0 && col < columns) {
    for (int i = 1; i < 16; ++i) sum += part[i][lane];
    (is_bias ? ddt_bias : da_log)[col] = sum;
  }
}

PrepareParams params_of(const PrepareArgs& a, const RowGrid& grid) {
  PrepareParams p{};
  p.q_raw = a.q_raw.ptr;
  p.k_raw = a.k_raw.ptr;
  p.gate_raw = a.gate_raw.ptr;
  p.beta_raw = a.beta_raw.ptr;
  p.q_stride = a.q_raw.stride;
  p.k_stride = a.k_raw.stride;
  p.gate_stride = a.gate_raw.stride;
  p.beta_stride = a.beta_raw.stride;
  p.a_log = static_cast<const float*>(a.a_log.ptr);
  p.dt_bias = static_cast<const float*>(a.dt_bias.ptr);
  p.q_scale = a.q_scale;
  p.eps = a.eps;
  p.T = a.T;
  p.H = a.H;
  p.lanes = grid.lanes;
  p.q = a.q.ptr;
  p.k = a.k.ptr;
  p.g = a.g.ptr;
  p.beta = a.beta.ptr;
  return p;
}

constexpr int kPrepareBlocks = 2048;

}  // namespace

int launch_prepare(const PrepareArgs& a, hipStream_t stream) {
  const RowGrid grid = row_grid(a.T, a.H, kPrepareGroups, kPrepareBlocks);
  const PrepareParams p = params_of(a, grid);
  // bf16: at 1.6 GB past the caches 317 us against 327, at 101 MB 44 and 38
  const bool e16 = a.dtype == KDA_BF16;
  const bool past = static_cast<int64_t>(a.T) * a.H * 384 * (e16 ? 4 : 6) >= kStreamBytes;
  void (*kernel)(PrepareParams) = e16 ? (past ? prepare_kernel<bf16_t, true> : prepare_kernel<bf16_t, false>)
                                      : (past ? prepare_kernel<fp32_t, true> : prepare_kernel<fp32_t, false>);
  (void)hipGetLastError();
  hipLaunchKernelGGL(kernel, dim3(grid.blocks), dim3(kRowThreads), 0, stream, p);
  return finish_launch();
}

int launch_prepare_backward(const PrepareArgs& a, hipStream_t stream) {
  const PrepareBwdLayout L = prepare_bwd_layout(a.T, a.H);
  PrepareParams p = params_of(a, L.grid);
  p.dq = static_cast<const float*>(a.dq.ptr);
  p.dk = static_cast<const float*>(a.dk.ptr);
  p.dg = static_cast<const float*>(a.dg.ptr);
  p.dbeta = static_cast<const float*>(a.dbeta.ptr);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace.ptr);
  p.bias_part = reinterpret_cast<float*>(ws + L.bias);
  p.decay_part = reinterpret_cast<float*>(ws + L.decay);
  (void)hipGetLastError();
  if (a.dtype == KDA_BF16) {
    hipLaunchKernelGGL(prepare_backward_kernel<bf16_t>, dim3(L.grid.blocks), dim3(kRowThreads), 0, stream, p);
  } else {
    hipLaunchKernelGGL(prepare_backward_kernel<fp32_t>, dim3(L.grid.blocks), dim3(kRowThreads), 0, stream, p);
  }
  const int st = finish_launch();
  if (st != KDA_OK) return st;
  const int32_t bias_blocks = a.ddt_bias.ptr != nullptr ? a.H * 2 : 0, decay_blocks = (a.H + 63) / 64;
  hipLaunchKernelGGL(prepare_reduce_kernel, dim3(bias_blocks + decay_blocks), dim3(1024), 0, stream, p.bias_part,
                     p.decay_part, L.grid.lanes, a.H, bias_blocks, static_cast<float*>(a.ddt_bias.ptr),
                     static_cast<float*>(a.da_log.ptr));
  return finish_launch();
}

}  // namespace kda
