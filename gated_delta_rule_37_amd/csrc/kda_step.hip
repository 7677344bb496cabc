// Single tokens over a pool of states: the KDA recurrence (kda_step) and the
// per-channel one (kda_scan_step).
//
// KDA, one token of one head with state S [K, V]:
//   S' = Diag(e^g) S,  u = beta (v - S'^T k),  S = S' + k u^T,
//   o = S^T q = S'^T q + (q . k) u,
// so S' is read once, both column sums come from the same registers, and S is
// written once: 64 KiB each way a (row, head), which HBM bandwidth bounds.
// A workgroup of 256 threads holds the whole state in registers: a thread has
// 4 columns of 16 rows, a wave's load covers two rows (1 KiB); four workgroups
// fit a CU, 256 KiB in flight.  256 rows x 32 heads 190 us, 5.7 TB/s (a large
// copy: 5.2); one row of 4 heads 4.8 us, 64 rows of 2048 channels 4.1 us (the
// latency of a launch, a load, two barriers and a store).
#include "kda_layer.h"
#include "kda_layer_device.h"

#include "kda.h"

namespace kda {
namespace {

// The rows of the batch that name one slot, in order.  The workgroups of the
// first such row work for all of them; the others have nothing to do.  Each
// workgroup reads the whole list, so that cost grows with the square of the
// rows: nothing up to 1024 of them, 65536 rows of 8 channels 1450 us against 32
// without slots.
struct SlotRows {
  const int32_t* slots;   // null: row b is slot b
  int32_t B, num_slots;

  // The slot of row b, or -1 where the row is unused or not its slot's first.
  // `box` is one int of shared memory; the whole workgroup calls.
  __device__ __forceinline__ int32_t own(int32_t b) const {
    if (slots == nullptr) return b;
    const int32_t slot = slots[b];
    if (slot < 0 || slot >= num_slots) return -1;
    int earlier = 0;
    for (int32_t j = threadIdx.x; j < b; j += blockDim.x) earlier |= slots[j] == slot;
    return __syncthreads_or(earlier) ? -1 : slot;
  }

  // The next row after b of the same slot, or B.
  __device__ __forceinline__ int32_t next(int32_t b, int32_t slot, int32_t* box) const {
    if (slots == nullptr) return B;
    __syncthreads();   // the readers of the last answer
    if (threadIdx.x == 0) *box = B;
    __syncthreads();
    for (int32_t j = b + 1 + threadIdx.x; j < B; j += blockDim.x) {
      if (slots[j] == slot) {
        atomicMin(box, j);
        break;
      }
    }
    __syncthreads();
    return *box;
  }
};

struct StepParams {
  const uint16_t *q, *k, *v, *g, *beta;
  SlotRows rows;
  const float* state;
  float* state_out;
  void* o;
  int32_t o_bf16, H, h0, hn;
  int32_t gate_floor_on;
  float gate_floor;
};

constexpr int kStepThreads = 256;

__global__ __launch_bounds__(kStepThreads) void step_kernel(StepParams p) {
  __shared__ __align__(16) float key[3][128];        // k, q, e^g of the row
  __shared__ __align__(16) float sums[4][2][128];    // the waves' parts of S'^T k and S'^T q
  __shared__ float dots[4];
  __shared__ int32_t box;
  const int32_t b0 = static_cast<int32_t>(blockIdx.x / static_cast<uint32_t>(p.hn));
  const int32_t head = p.h0 + static_cast<int32_t>(blockIdx.x % static_cast<uint32_t>(p.hn));
  const int32_t slot = p.rows.own(b0);
  if (slot < 0) return;
  const int32_t col = (threadIdx.x & 31) * 4, row0 = threadIdx.x >> 5, wave = threadIdx.x >> 6;
  const int64_t at = (static_cast<int64_t>(slot) * p.H + head) * (128 * 128) + row0 * 128 + col;
  f32x4 S[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) S[i] = ld4(p.state + at + i * 8 * 128);

  for (int32_t b = b0; b < p.rows.B; b = p.rows.next(b, slot, &box)) {
    const int64_t bh = static_cast<int64_t>(b) * p.H + head;
    if (threadIdx.x < 128) {
      const int64_t c = bh * 128 + threadIdx.x;
      float g = bf2f(p.g[c]);
      if (p.gate_floor_on) g = fmaxf(g, p.gate_floor);
      key[0][threadIdx.x] = bf2f(p.k[c]);
      key[1][threadIdx.x] = bf2f(p.q[c]);
      key[2][threadIdx.x] = exact_exp(g);
    }
    const float beta = bf2f(p.beta[bh]);
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = bf2f(p.v[bh * 128 + col + j]);
    __syncthreads();
    f32x4 sk = zero4(), sq = zero4();
    float qk = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int32_t r = row0 + 8 * i;
      const float k = key[0][r], q = key[1][r];
      S[i] *= key[2][r];
      sk += k * S[i];
      sq += q * S[i];
      qk += k * q;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      sk[j] += __shfl_xor(sk[j], 32);
      sq[j] += __shfl_xor(sq[j], 32);
    }
    qk += __shfl_xor(qk, 32);
    if ((threadIdx.x & 32) == 0) {
      st4(&sums[wave][0][col], sk);
      st4(&sums[wave][1][col], sq);
      if ((threadIdx.x & 63) == 0) dots[wave] = qk;
    }
    __syncthreads();
    sk = (ld4(&sums[0][0][col]) + ld4(&sums[1][0][col])) + (ld4(&sums[2][0][col]) + ld4(&sums[3][0][col]));
    sq = (ld4(&sums[0][1][col]) + ld4(&sums[1][1][col])) + (ld4(&sums[2][1][col]) + ld4(&sums[3][1][col]));
    qk = (dots[0] + dots[1]) + (dots[2] + dots[3]);
    f32x4 u;
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = beta * (v[j] - sk[j]);
#pragma unroll
    for (int i = 0; i < 16; ++i) S[i] += key[0][row0 + 8 * i] * u;
    if (row0 == 0) {
      sq += qk * u;
      if (p.o_bf16) {
        uint32_t* o = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o) + bh * 128 + col);
        o[0] = pack_bf16(sq[0], sq[1]);
        o[1] = pack_bf16(sq[2], sq[3]);
      } else {
        st4(static_cast<float*>(p.o) + bh * 128 + col, sq);
      }
    }
    if (p.rows.slots == nullptr) break;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) st4(p.state_out + at + i * 8 * 128, S[i]);
}

struct ScanStepParams {
  const void *x, *g;
  SlotRows rows;
  const float* state;
  float* state_out;
  void* h;
  int32_t D, tied, blocks;   // blocks: workgroups a row
};

constexpr int kScanStepThreads = 256;

template <typename E, int VEC>
__global__ __launch_bounds__(kScanStepThreads) void scan_step_kernel(ScanStepParams p) {
  __shared__ int32_t box;
  const int32_t b0 = static_cast<int32_t>(blockIdx.x / static_cast<uint32_t>(p.blocks));
  const int32_t slot = p.rows.own(b0);
  if (slot < 0) return;
  const int32_t d = (static_cast<int32_t>(blockIdx.x % static_cast<uint32_t>(p.blocks)) * kScanStepThreads + threadIdx.x) * VEC;
  const bool active = d < p.D;
  const int64_t at = static_cast<int64_t>(slot) * p.D + d;
  float h[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) h[i] = 0.f;
  if (active) load<VEC>(p.state + at, h);
  for (int32_t b = b0; b < p.rows.B; b = p.rows.next(b, slot, &box)) {
    const int64_t row = static_cast<int64_t>(b) * p.D + d;
    if (active) {
      float x[VEC], g[VEC];
      load<VEC>(static_cast<const E*>(p.x) + row, x);
      load<VEC>(static_cast<const E*>(p.g) + row, g);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float a = exact_exp(g[i]);
        h[i] = a * h[i] + (p.tied ? one_minus_exp(g[i], a) : 1.f) * x[i];
      }
      store<VEC>(static_cast<E*>(p.h) + row, h);
    }
    if (p.rows.slots == nullptr) break;
  }
  if (active) store<VEC>(p.state_out + at, h);
}

}  // namespace

int launch_step(const StepArgs& a, hipStream_t stream) {
  StepParams p{};
  p.q = static_cast<const uint16_t*>(a.q.ptr);
  p.k = static_cast<const uint16_t*>(a.k.ptr);
  p.v = static_cast<const uint16_t*>(a.v.ptr);
  p.g = static_cast<const uint16_t*>(a.g.ptr);
  p.beta = static_cast<const uint16_t*>(a.beta.ptr);
  p.rows = {static_cast<const int32_t*>(a.slots.ptr), a.B, a.num_slots};
  p.state = static_cast<const float*>(a.state.ptr);
  p.state_out = static_cast<float*>(a.state_out.ptr);
  p.o = a.o.ptr;
  p.o_bf16 = a.o_format == KDA_O_BF16 ? 1 : 0;
  p.H = a.H;
  p.h0 = a.head_begin;
  p.hn = a.head_count;
  p.gate_floor_on = a.gate_lower_bound > -INFINITY ? 1 : 0;
  p.gate_floor = a.gate_lower_bound;
  const int64_t blocks = static_cast<int64_t>(a.B) * a.head_count;
  if (blocks * kStepThreads > 2147483647LL) return KDA_ERR_UNSUPPORTED;
  (void)hipGetLastError();
  hipLaunchKernelGGL(step_kernel, dim3(static_cast<uint32_t>(blocks)), dim3(kStepThreads), 0, stream, p);
  return finish_launch();
}

int launch_scan_step(const ScanStepArgs& a, hipStream_t stream) {
  ScanStepParams p{};
  p.x = a.x.ptr;
  p.g = a.g.ptr;
  p.rows = {static_cast<const int32_t*>(a.slots.ptr), a.B, a.num_slots};
  p.state = static_cast<const float*>(a.state.ptr);
  p.state_out = static_cast<float*>(a.state_out.ptr);
  p.h = a.h.ptr;
  p.D = a.D;
  p.tied = a.tied;
  const int32_t vec = a.D % 8 == 0 ? 8 : 1;
  p.blocks = (a.D + kScanStepThreads * vec - 1) / (kScanStepThreads * vec);
  const int64_t blocks = static_cast<int64_t>(a.B) * p.blocks;
  if (blocks * kScanStepThreads > 2147483647LL) return KDA_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<uint32_t>(blocks)), threads(kScanStepThreads);
  (void)hipGetLastError();
  if (a.dtype == KDA_BF16) {
    if (vec == 8) {
      hipLaunchKernelGGL((scan_step_kernel<bf16_t, 8>), grid, threads, 0, stream, p);
    } else {
      hipLaunchKernelGGL((scan_step_kernel<bf16_t, 1>), grid, threads, 0, stream, p);
    }
  } else if (vec == 8) {
    hipLaunchKernelGGL((scan_step_kernel<fp32_t, 8>), grid, threads, 0, stream, p);
  } else {
    hipLaunchKernelGGL((scan_step_kernel<fp32_t, 1>), grid, threads, 0, stream, p);
  }
  return finish_launch();
}

}  // namespace kda
