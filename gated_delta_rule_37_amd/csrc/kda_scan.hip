// A gated linear recurrence with one state per channel over packed sequences
// (kda_scan_forward) and its gradients (kda_scan_backward):
//   h_t = a_t h_{t-1} + u_t,   a = e^g,  u = x or (1 - a) x.
// With c_t = a_t l_t the backward is the same recurrence from the other end,
//   c_t = a_t c_{t+1} + a_t dh_t,   l_t = dh_t + c_{t+1},
//   dx = l or (1 - a) l,   dg = c (h_{t-1} - [tied] x),   d_initial = c_1.
//
// A run of tokens is the map h -> A h + B, A the product of its decays and B
// its end state from zero; two neighbouring runs compose to
// (A2 A1, A2 B1 + B2).  A workgroup owns a few channels of one sequence and
// walks its tokens in tiles, the whole sequence's state never leaving it: a
// thread scans R tokens of VEC channels in registers, the threads' maps are
// composed across the wave by shuffles and across the waves through LDS, and
// every state follows as (state from zero) + (product of decays) * carry.  So
// each element is read and written once, HBM bandwidth being the bound.
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
  int32_t blocks, bundles;   // channel blocks, and bundles of them, of a unit
  int64_t total_bundles;
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

// A workgroup's work: sequence n, channels from `channel`, and its tokens.
// Workgroups go round the 8 XCDs in launch order; neighbouring channel blocks
// share cache lines, so a bundle of kBundle blocks stays on one XCD.
constexpr int kXcds = 8;
struct Unit {
  int32_t n, block, begin, end;
};
template <int BUNDLE>
__device__ __forceinline__ bool unit_of(const ScanParams& p, Unit& u) {
  const uint32_t id = blockIdx.x, xcd = id % kXcds, i = id / kXcds;
  const int64_t bundle = static_cast<int64_t>(i / BUNDLE) * kXcds + xcd;
  if (bundle >= p.total_bundles) return false;
  const int32_t seq = static_cast<int32_t>(bundle / p.bundles);
  u.block = static_cast<int32_t>(bundle - static_cast<int64_t>(seq) * p.bundles) * BUNDLE + static_cast<int32_t>(i % BUNDLE);
  if (u.block >= p.blocks) return false;
  u.n = seq;
  u.begin = sequence_begin(p, u.n);
  u.end = sequence_begin(p, u.n + 1);
  return true;
}

// LPR lanes of VEC channels each make a row; a thread takes R tokens.
template <int VEC_, int LPR_, int R_, int THREADS_>
struct Geometry {
  static constexpr int VEC = VEC_, LPR = LPR_, R = R_, THREADS = THREADS_;
  static constexpr int kWaves = THREADS / 64, kTile = THREADS / LPR * R, kChannels = LPR * VEC;
};

// Composes the maps (A, B) of the thread groups before this one in the wave:
// on return (A, B) is this group's own prefix without itself (the identity
// for the first), and (TA, TB) the whole wave's.  Groups are LPR lanes apart.
template <int VEC, int LPR>
__device__ __forceinline__ void wave_scan(float (&A)[VEC], float (&B)[VEC], float (&TA)[VEC], float (&TB)[VEC]) {
  const int32_t lane = threadIdx.x & 63;
#pragma unroll
  for (int off = LPR; off < 64; off *= 2) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const float a = __shfl_up(A[i], off), b = __shfl_up(B[i], off);
      if (lane >= off) {
        B[i] += A[i] * b;
        A[i] *= a;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    TA[i] = __shfl(A[i], 64 - LPR + lane % LPR);
    TB[i] = __shfl(B[i], 64 - LPR + lane % LPR);
    const float a = __shfl_up(A[i], LPR), b = __shfl_up(B[i], LPR);
    A[i] = lane >= LPR ? a : 1.f;
    B[i] = lane >= LPR ? b : 0.f;
  }
}

// The carry into this thread group, given its wave's prefix (A, B) and total
// (TA, TB), and the workgroup's carry moved on behind the tile.
template <typename G>
__device__ __forceinline__ void tile_carry(float (*box)[2][G::kChannels], const float (&A)[G::VEC],
                                           const float (&B)[G::VEC], const float (&TA)[G::VEC],
                                           const float (&TB)[G::VEC], float (&carry)[G::VEC], float (&in)[G::VEC]) {
  const int32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c0 = (lane % G::LPR) * G::VEC;
  if (lane < G::LPR) {
#pragma unroll
    for (int i = 0; i < G::VEC; ++i) {
      box[wave][0][c0 + i] = TA[i];
      box[wave][1][c0 + i] = TB[i];
    }
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < G::kWaves; ++w) {
    if (w == wave) {
#pragma unroll
      for (int i = 0; i < G::VEC; ++i) in[i] = A[i] * carry[i] + B[i];
    }
#pragma unroll
    for (int i = 0; i < G::VEC; ++i) carry[i] = box[w][0][c0 + i] * carry[i] + box[w][1][c0 + i];
  }
}

template <typename E, typename O, typename G>
__global__ __launch_bounds__(G::THREADS) void scan_kernel(ScanParams p) {
  constexpr int VEC = G::VEC, R = G::R;
  __shared__ __align__(16) float box[2][G::kWaves][2][G::kChannels];
  Unit u;
  if (!unit_of<4>(p, u)) return;
  const int32_t row = threadIdx.x / G::LPR * R;                                // first token in the tile
  const int32_t d = u.block * G::kChannels + (threadIdx.x % G::LPR) * VEC;
  const bool owner = d < p.D;
  const int32_t dl = owner ? d : p.D - VEC;                                    // a channel that can be read
  const E* x0 = static_cast<const E*>(p.x) + dl;
  const E* g0 = static_cast<const E*>(p.g) + dl;
  float carry[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) carry[i] = 0.f;
  if (p.initial_state != nullptr) load<VEC>(p.initial_state + static_cast<int64_t>(u.n) * p.D + dl, carry);

  RawVec<E, VEC> x[R], g[R];
  const auto fetch = [&](int32_t tile) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t t = min(tile + row + r, u.end - 1);
      load_raw<E, VEC>(x0 + t * p.x_stride, x[r]);
      load_raw<E, VEC>(g0 + t * p.g_stride, g[r]);
    }
  };
  fetch(u.begin);
  int parity = 0;
  for (int32_t tile = u.begin; tile < u.end; tile += G::kTile, parity ^= 1) {
    // states from zero and products of decays, in this thread's tokens
    float h[R][VEC], P[R][VEC], A[VEC], B[VEC], TA[VEC], TB[VEC], in[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      A[i] = 1.f;
      B[i] = 0.f;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool valid = tile + row + r < u.end;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float gi = element(g[r], i), xi = element(x[r], i);
        float a = __expf(gi);
        float v = p.tied ? one_minus_exp(gi, a) * xi : xi;
        a = valid ? a : 1.f;
        v = valid ? v : 0.f;
        B[i] = a * B[i] + v;
        A[i] *= a;
        h[r][i] = B[i];
        P[r][i] = A[i];
      }
    }
    if (tile + G::kTile < u.end) fetch(tile + G::kTile);
    wave_scan<VEC, G::LPR>(A, B, TA, TB);
    tile_carry<G>(box[parity], A, B, TA, TB, carry, in);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t t = tile + row + r;
#pragma unroll
      for (int i = 0; i < VEC; ++i) h[r][i] += P[r][i] * in[i];
      if (t < u.end && owner) store<VEC>(static_cast<O*>(p.h) + t * p.D + d, h[r]);
    }
  }
  if (threadIdx.x < G::LPR && owner) store<VEC>(p.final_state + static_cast<int64_t>(u.n) * p.D + d, carry);
}

// The backward: tiles from the sequence's end, row 0 of a tile its last token.
template <typename E, typename O, typename G>
__global__ __launch_bounds__(G::THREADS) void scan_backward_kernel(ScanParams p) {
  constexpr int VEC = G::VEC, R = G::R;
  __shared__ __align__(16) float box[2][G::kWaves][2][G::kChannels];
  Unit u;
  if (!unit_of<4>(p, u)) return;
  const int32_t row = threadIdx.x / G::LPR * R;
  const int32_t d = u.block * G::kChannels + (threadIdx.x % G::LPR) * VEC;
  const bool owner = d < p.D;
  const int32_t dl = owner ? d : p.D - VEC;
  const int64_t nd = static_cast<int64_t>(u.n) * p.D + dl;
  const E* x0 = static_cast<const E*>(p.x) + dl;
  const E* g0 = static_cast<const E*>(p.g) + dl;
  const O* h0 = static_cast<const O*>(p.h_in) + dl;
  const O* dh0 = static_cast<const O*>(p.dh) + dl;
  float carry[VEC], first[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) carry[i] = first[i] = 0.f;
  if (p.d_final != nullptr) load<VEC>(p.d_final + nd, carry);
  if (p.initial_state != nullptr) load<VEC>(p.initial_state + nd, first);

  RawVec<E, VEC> g[R];
  RawVec<O, VEC> dh[R];
  const auto fetch = [&](int32_t last) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t t = max(last - row - r, u.begin);
      load_raw<E, VEC>(g0 + t * p.g_stride, g[r]);
      load_raw<O, VEC>(dh0 + t * p.D, dh[r]);
    }
  };
  fetch(u.end - 1);
  int parity = 0;
  for (int32_t last = u.end - 1; last >= u.begin; last -= G::kTile, parity ^= 1) {
    // what this tile's outputs need besides the scan
    RawVec<E, VEC> x[R];
    RawVec<O, VEC> before[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t t = max(last - row - r, u.begin);
      load_raw<O, VEC>(h0 + max(t - 1, static_cast<int64_t>(u.begin)) * p.D, before[r]);
      if (p.tied) load_raw<E, VEC>(x0 + t * p.x_stride, x[r]);
    }
    float c[R][VEC], P[R][VEC], l[R][VEC], share[R][VEC], A[VEC], B[VEC], TA[VEC], TB[VEC], in[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      A[i] = 1.f;
      B[i] = 0.f;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool valid = last - row - r >= u.begin;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float gi = element(g[r], i);
        float a = __expf(gi), v = element(dh[r], i);
        share[r][i] = p.tied ? one_minus_exp(gi, a) : 1.f;
        l[r][i] = v;
        a = valid ? a : 1.f;
        v = valid ? v : 0.f;
        B[i] = valid ? a * (B[i] + v) : B[i];
        A[i] *= a;
        c[r][i] = B[i];
        P[r][i] = A[i];
      }
    }
    if (last - G::kTile >= u.begin) fetch(last - G::kTile);
    wave_scan<VEC, G::LPR>(A, B, TA, TB);
    tile_carry<G>(box[parity], A, B, TA, TB, carry, in);
    float next[VEC];   // c_{t+1}
#pragma unroll
    for (int i = 0; i < VEC; ++i) next[i] = in[i];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t t = last - row - r;
      float dx[VEC], dg[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        dx[i] = share[r][i] * (l[r][i] + next[i]);
        next[i] = c[r][i] + P[r][i] * in[i];
        const float h = t > u.begin ? element(before[r], i) : first[i];
        dg[i] = next[i] * (p.tied ? h - element(x[r], i) : h);
      }
      if (t >= u.begin && owner) {
        store<VEC>(static_cast<E*>(p.dx) + t * p.D + d, dx);
        store<VEC>(static_cast<E*>(p.dg) + t * p.D + d, dg);
      }
    }
  }
  if (p.d_initial_state != nullptr && threadIdx.x < G::LPR && owner) store<VEC>(p.d_initial_state + nd, carry);
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

template <typename G>
int launch(void (*kernel)(ScanParams), ScanParams p, hipStream_t stream) {
  p.blocks = (p.D + G::kChannels - 1) / G::kChannels;
  p.bundles = (p.blocks + 3) / 4;
  p.total_bundles = static_cast<int64_t>(p.bundles) * p.N;
  const int64_t grid = (p.total_bundles + kXcds - 1) / kXcds * kXcds * 4;
  if (grid * G::THREADS > 2147483647LL) return KDA_ERR_UNSUPPORTED;
  (void)hipGetLastError();
  hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(grid)), dim3(G::THREADS), 0, stream, p);
  return finish_launch();
}

// Rows of 16-byte pieces: whole vectors and strides.
bool vector_rows(const ScanArgs& a, bool with_x) {
  const int64_t per = a.dtype == KDA_BF16 ? 8 : 4;
  return a.D % 8 == 0 && a.g.stride % per == 0 && (!with_x || a.x.stride % per == 0);
}

using Vector = Geometry<4, 4, 8, 512>;
using VectorBackward = Geometry<4, 4, 4, 512>;
using Wide = Geometry<8, 2, 4, 512>;
using Scalar = Geometry<1, 16, 8, 512>;

}  // namespace

int launch_scan(const ScanArgs& a, hipStream_t stream) {
  const ScanParams p = params_of(a);
  const bool e16 = a.dtype == KDA_BF16, o16 = a.h_format == KDA_BF16;
  if (vector_rows(a, true)) {
    if (e16 && o16) return launch<Vector>(scan_kernel<bf16_t, bf16_t, Vector>, p, stream);
    if (e16) return launch<Vector>(scan_kernel<bf16_t, fp32_t, Vector>, p, stream);
    if (o16) return launch<Wide>(scan_kernel<fp32_t, bf16_t, Wide>, p, stream);
    return launch<Wide>(scan_kernel<fp32_t, fp32_t, Wide>, p, stream);
  }
  if (e16 && o16) return launch<Scalar>(scan_kernel<bf16_t, bf16_t, Scalar>, p, stream);
  if (e16) return launch<Scalar>(scan_kernel<bf16_t, fp32_t, Scalar>, p, stream);
  if (o16) return launch<Scalar>(scan_kernel<fp32_t, bf16_t, Scalar>, p, stream);
  return launch<Scalar>(scan_kernel<fp32_t, fp32_t, Scalar>, p, stream);
}

int launch_scan_backward(const ScanArgs& a, hipStream_t stream) {
  const ScanParams p = params_of(a);
  const bool e16 = a.dtype == KDA_BF16, o16 = a.h_format == KDA_BF16;
  if (vector_rows(a, a.tied != 0)) {
    if (e16 && o16) return launch<VectorBackward>(scan_backward_kernel<bf16_t, bf16_t, VectorBackward>, p, stream);
    if (e16) return launch<VectorBackward>(scan_backward_kernel<bf16_t, fp32_t, VectorBackward>, p, stream);
    if (o16) return launch<Wide>(scan_backward_kernel<fp32_t, bf16_t, Wide>, p, stream);
    return launch<Wide>(scan_backward_kernel<fp32_t, fp32_t, Wide>, p, stream);
  }
  if (e16 && o16) return launch<Scalar>(scan_backward_kernel<bf16_t, bf16_t, Scalar>, p, stream);
  if (e16) return launch<Scalar>(scan_backward_kernel<bf16_t, fp32_t, Scalar>, p, stream);
  if (o16) return launch<Scalar>(scan_backward_kernel<fp32_t, bf16_t, Scalar>, p, stream);
  return launch<Scalar>(scan_backward_kernel<fp32_t, fp32_t, Scalar>, p, stream);
}

}  // namespace kda
