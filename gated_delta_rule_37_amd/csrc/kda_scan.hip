// A gated linear recurrence with one state per channel over packed sequences
// (kda_scan_forward) and its gradients (kda_scan_backward):
//   h_t = a_t h_{t-1} + u_t,   a = e^g,  u = x or (1 - a) x
//   l_t = dh_t + a_{t+1} l_{t+1},  dx = l or (1 - a) l,  dg = l a (h_{t-1} - [tied] x)
//
// One thread walks one channel of one sequence, so that neighbouring threads
// read neighbouring channels.
#include "kda_layer.h"
#include "kda_layer_device.h"

#include "kda.h"

namespace kda {
namespace {

struct ScanParams {
  const int32_t* plan;
  BlobLayout L;
  int32_t T, N, F, D;
  int32_t tied;
  const void *x, *g;
  int64_t x_stride, g_stride;
  const float *initial_state, *d_final;
  void* h;
  float* final_state;
  const void *h_in, *dh;
  void *dx, *dg;
  float* d_initial_state;
};

// The first fragment of sequence n: n itself where no segment cuts a
// sequence, else found in the sorted frag_seq.
__device__ __forceinline__ int32_t first_fragment(const ScanParams& p, int32_t n) {
  if (p.F == p.N) return n;
  int32_t lo = 0, hi = p.F;
  while (lo < hi) {
    const int32_t mid = (lo + hi) >> 1;
    if (p.plan[p.L.frag_seq + mid] < n) {
      lo = mid + 1;
    } else {
      hi = mid;
    }
  }
  return lo;
}
__device__ __forceinline__ int32_t sequence_begin(const ScanParams& p, int32_t n) {
  return n >= p.N ? p.T : p.plan[p.L.frag_begin + first_fragment(p, n)];
}

constexpr int kScanThreads = 256;

template <typename E, typename O>
__global__ __launch_bounds__(kScanThreads) void scan_kernel(ScanParams p, int32_t blocks) {
  const int32_t n = static_cast<int32_t>(blockIdx.x / static_cast<uint32_t>(blocks));
  const int32_t d = static_cast<int32_t>(blockIdx.x % static_cast<uint32_t>(blocks)) * kScanThreads + threadIdx.x;
  if (d >= p.D) return;
  const int32_t begin = sequence_begin(p, n), end = sequence_begin(p, n + 1);
  float h[1] = {p.initial_state == nullptr ? 0.f : p.initial_state[static_cast<int64_t>(n) * p.D + d]};
  for (int64_t t = begin; t < end; ++t) {
    float x[1], g[1];
    load<1>(static_cast<const E*>(p.x) + t * p.x_stride + d, x);
    load<1>(static_cast<const E*>(p.g) + t * p.g_stride + d, g);
    h[0] = __expf(g[0]) * h[0] + (p.tied ? -expm1f(g[0]) : 1.f) * x[0];
    store<1>(static_cast<O*>(p.h) + t * p.D + d, h);
  }
  p.final_state[static_cast<int64_t>(n) * p.D + d] = h[0];
}

template <typename E, typename O>
__global__ __launch_bounds__(kScanThreads) void scan_backward_kernel(ScanParams p, int32_t blocks) {
  const int32_t n = static_cast<int32_t>(blockIdx.x / static_cast<uint32_t>(blocks));
  const int32_t d = static_cast<int32_t>(blockIdx.x % static_cast<uint32_t>(blocks)) * kScanThreads + threadIdx.x;
  if (d >= p.D) return;
  const int32_t begin = sequence_begin(p, n), end = sequence_begin(p, n + 1);
  const int64_t nd = static_cast<int64_t>(n) * p.D + d;
  float carry = p.d_final == nullptr ? 0.f : p.d_final[nd];   // a_{t+1} l_{t+1}
  const float first = p.initial_state == nullptr ? 0.f : p.initial_state[nd];
  for (int64_t t = end - 1; t >= begin; --t) {
    float x[1] = {0.f}, g[1], dh[1], before[1] = {first};
    load<1>(static_cast<const E*>(p.g) + t * p.g_stride + d, g);
    if (p.tied) load<1>(static_cast<const E*>(p.x) + t * p.x_stride + d, x);
    load<1>(static_cast<const O*>(p.dh) + t * p.D + d, dh);
    if (t > begin) load<1>(static_cast<const O*>(p.h_in) + (t - 1) * p.D + d, before);
    const float l = dh[0] + carry;
    carry = __expf(g[0]) * l;
    float dx[1] = {p.tied ? -expm1f(g[0]) * l : l}, dg[1] = {carry * (before[0] - x[0])};
    store<1>(static_cast<E*>(p.dx) + t * p.D + d, dx);
    store<1>(static_cast<E*>(p.dg) + t * p.D + d, dg);
  }
  if (p.d_initial_state != nullptr) p.d_initial_state[nd] = carry;
}

ScanParams params_of(const ScanArgs& a) {
  ScanParams p{};
  p.plan = static_cast<const int32_t*>(a.plan_dev.ptr);
  p.L = a.plan->layout;
  p.T = a.plan->T;
  p.N = a.plan->N;
  p.F = a.plan->F;
  p.D = a.D;
  p.tied = a.tied;
  p.x = a.x.ptr;
  p.g = a.g.ptr;
  p.x_stride = a.x.stride;
  p.g_stride = a.g.stride;
  p.initial_state = static_cast<const float*>(a.initial_state.ptr);
  p.d_final = static_cast<const float*>(a.d_final.ptr);
  p.h = a.h.ptr;
  p.final_state = static_cast<float*>(a.final_state.ptr);
  p.h_in = a.h_in.ptr;
  p.dh = a.dh.ptr;
  p.dx = a.dx.ptr;
  p.dg = a.dg.ptr;
  p.d_initial_state = static_cast<float*>(a.d_initial_state.ptr);
  return p;
}

template <typename F16E16, typename F32E16, typename F16E32, typename F32E32>
int dispatch(const ScanArgs& a, F16E16 k16, F32E16 k32, F16E32 k16e32, F32E32 k32e32, hipStream_t stream) {
  const ScanParams p = params_of(a);
  const int32_t blocks = (a.D + kScanThreads - 1) / kScanThreads;
  const int64_t total = static_cast<int64_t>(blocks) * p.N;
  if (total * kScanThreads > 2147483647LL) return KDA_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<uint32_t>(total)), threads(kScanThreads);
  const bool e16 = a.dtype == KDA_BF16, o16 = a.h_format == KDA_BF16;
  (void)hipGetLastError();
  if (e16 && o16) hipLaunchKernelGGL(k16, grid, threads, 0, stream, p, blocks);
  if (e16 && !o16) hipLaunchKernelGGL(k32, grid, threads, 0, stream, p, blocks);
  if (!e16 && o16) hipLaunchKernelGGL(k16e32, grid, threads, 0, stream, p, blocks);
  if (!e16 && !o16) hipLaunchKernelGGL(k32e32, grid, threads, 0, stream, p, blocks);
  return finish_launch();
}

}  // namespace

int launch_scan(const ScanArgs& a, hipStream_t stream) {
  return dispatch(a, scan_kernel<bf16_t, bf16_t>, scan_kernel<bf16_t, fp32_t>, scan_kernel<fp32_t, bf16_t>,
                  scan_kernel<fp32_t, fp32_t>, stream);
}

int launch_scan_backward(const ScanArgs& a, hipStream_t stream) {
  return dispatch(a, scan_backward_kernel<bf16_t, bf16_t>, scan_backward_kernel<bf16_t, fp32_t>,
                  scan_backward_kernel<fp32_t, bf16_t>, scan_backward_kernel<fp32_t, fp32_t>, stream);
}

}  // namespace kda
