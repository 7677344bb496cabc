// Linear attention with a decay for each head, single tokens over a pool of
// states (kda_linear_step): S' = e^g S + k v^T, o = S'^T q.
//
// S is read once, S' written once, and o is summed from the same registers:
// 8 K V bytes a (row, head), which HBM bandwidth bounds.  A workgroup of 256
// threads holds the whole state: a thread 4 columns of every `span`th row (at
// most 16 of them), so that neighbouring threads read neighbouring 16 bytes.  256
// rows x 32 heads of 128 x 128 take 199 us (some unused: 1.08 GB, 5.4 TB/s), one row
// of 4 heads the host's 11.
#include "kda_layer.h"
#include "kda_layer_device.h"

#include "kda.h"

namespace kda {
namespace {

struct LinearStepParams {
  const uint16_t *q, *k, *v;
  const void* g;
  SlotRows rows;
  const float* state;
  float* state_out;
  void* o;
  int32_t H, K, V, Hq, Hk, Hv, g_stride, g_bf16, o_bf16;
};

constexpr int kLinearStepThreads = 256;
constexpr int kStepRows = 16;

__global__ __launch_bounds__(kLinearStepThreads) void linear_step_kernel(LinearStepParams p) {
  __shared__ __align__(16) float key[2][128];                   // k, q of the row
  __shared__ __align__(16) f32x4 sums[kLinearStepThreads];      // the threads' parts of o
  __shared__ int32_t box;
  const int32_t b0 = static_cast<int32_t>(blockIdx.x / static_cast<uint32_t>(p.H));
  const int32_t head = static_cast<int32_t>(blockIdx.x % static_cast<uint32_t>(p.H));
  const int32_t slot = p.rows.own(b0);
  if (slot < 0) return;
  const int32_t quads = p.V / 4, span = kLinearStepThreads / quads, tid = static_cast<int32_t>(threadIdx.x);
  const int32_t row0 = tid / quads, col = (tid - row0 * quads) * 4;
  const bool active = row0 < span;
  const int64_t at = (static_cast<int64_t>(slot) * p.H + head) * (p.K * p.V) + row0 * p.V + col;
  f32x4 S[kStepRows];
#pragma unroll
  for (int i = 0; i < kStepRows; ++i) {
    S[i] = zero4();
    if (active && row0 + i * span < p.K) S[i] = ld4(p.state + at + i * span * p.V);
  }
  const int32_t hq = head / (p.H / p.Hq), hk = head / (p.H / p.Hk), hv = head / (p.H / p.Hv);
  for (int32_t b = b0; b < p.rows.B; b = p.rows.next(b, slot, &box)) {
    if (tid < p.K) {
      key[0][tid] = bf2f(p.k[(static_cast<int64_t>(b) * p.Hk + hk) * p.K + tid]);
    } else if (tid >= 128 && tid - 128 < p.K) {
      key[1][tid - 128] = bf2f(p.q[(static_cast<int64_t>(b) * p.Hq + hq) * p.K + tid - 128]);
    }
    const int64_t gi = static_cast<int64_t>(b) * p.g_stride + head;
    const float decay = exact_exp(p.g_bf16 ? bf2f(static_cast<const uint16_t*>(p.g)[gi]) : static_cast<const float*>(p.g)[gi]);
    f32x4 v = zero4();
    if (active) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = bf2f(p.v[(static_cast<int64_t>(b) * p.Hv + hv) * p.V + col + j]);
    }
    __syncthreads();
    f32x4 sum = zero4();
#pragma unroll
    for (int i = 0; i < kStepRows; ++i) {
      const int32_t r = row0 + i * span;
      if (active && r < p.K) {
        S[i] = decay * S[i] + key[0][r] * v;
        sum += key[1][r] * S[i];
      }
    }
    sums[tid] = sum;
    __syncthreads();
    // the parts of one column group, halved until one is left
    for (int32_t n = span; n > 1;) {
      const int32_t half = (n + 1) / 2;
      if (row0 < n - half) sums[tid] += sums[tid + half * quads];
      __syncthreads();
      n = half;
    }
    if (row0 == 0) {
      const f32x4 o = sums[tid];
      const int64_t out = (static_cast<int64_t>(b) * p.H + head) * p.V + col;
      if (p.o_bf16) {
        u32x2 w;
        w[0] = pack_bf16(o[0], o[1]);
        w[1] = pack_bf16(o[2], o[3]);
        *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p.o) + out) = w;
      } else {
        st4(static_cast<float*>(p.o) + out, o);
      }
    }
    if (p.rows.slots == nullptr) break;
  }
#pragma unroll
  for (int i = 0; i < kStepRows; ++i) {
    if (active && row0 + i * span < p.K) st4(p.state_out + at + i * span * p.V, S[i]);
  }
}

}  // namespace

int launch_linear_step(const LinearStepArgs& a, hipStream_t stream) {
  LinearStepParams p{};
  p.q = static_cast<const uint16_t*>(a.q.ptr);
  p.k = static_cast<const uint16_t*>(a.k.ptr);
  p.v = static_cast<const uint16_t*>(a.v.ptr);
  p.g = a.g.ptr;
  p.rows = {static_cast<const int32_t*>(a.slots.ptr), a.B, a.num_slots};
  p.state = static_cast<const float*>(a.state.ptr);
  p.state_out = static_cast<float*>(a.state_out.ptr);
  p.o = a.o.ptr;
  p.H = a.H;
  p.K = a.K;
  p.V = a.V;
  p.Hq = a.Hq;
  p.Hk = a.Hk;
  p.Hv = a.Hv;
  p.g_stride = static_cast<int32_t>(a.g.stride);
  p.g_bf16 = a.g_dtype == KDA_BF16 ? 1 : 0;
  p.o_bf16 = a.o_format == KDA_BF16 ? 1 : 0;
  const int64_t blocks = static_cast<int64_t>(a.B) * a.H;
  if (blocks * kLinearStepThreads > 2147483647LL) return KDA_ERR_UNSUPPORTED;
  (void)hipGetLastError();
  hipLaunchKernelGGL(linear_step_kernel, dim3(static_cast<uint32_t>(blocks)), dim3(kLinearStepThreads), 0, stream, p);
  return finish_launch();
}

}  // namespace kda
