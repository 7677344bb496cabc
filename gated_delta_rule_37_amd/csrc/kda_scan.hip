// A gated linear recurrence with one state per channel over packed sequences
// (kda_scan_forward) and its gradients (kda_scan_backward):
//   h_t = a_t h_{t-1} + u_t,   a = e^g,  u = x or (1 - a) x.
// With c_t = a_t l_t the backward is the same recurrence from the other end,
//   c_t = a_t c_{t+1} + a_t dh_t,   l_t = dh_t + c_{t+1},
//   dx = l or (1 - a) l,   dg = c (h_{t-1} - [tied] x),   d_initial = c_1.
//
// A run of tokens is the map h -> A h + B, A the product of its decays and B
// its end state from zero; two neighbouring runs compose to
// (A2 A1, A2 B1 + B2).  A sequence's first token is the constant map
// (0, a_1 h_0 + u_1), so packed sequences need nothing else.
//
// One pass: a workgroup keeps a tile of kScanTile tokens of 64 channels in
// registers (a 128-byte line of bf16 a row), scans it from zero, publishes its
// map, gets the state before its tile from the maps of the tiles before it
// (look_back), publishes the state behind it, and only then walks its tokens
// from that state and writes.  Each element is read and written once, so HBM
// bandwidth is the bound where there are many channel blocks of whole 128-byte
// lines: 65536 x 4096 bf16 forward (tied) 292-310 us, 5.2-5.5 TB/s, 32768 x 4096
// backward 234-242 us, 5.6 TB/s (a large copy: 5.2).  Few blocks are bound by the
// chain of look-backs (32768 x 64 forward 36 us, backward 38, 0.3 and 0.7 TB/s),
// rows whose lines two blocks share likely by fetching them twice (32768 x 4093
// 237 and 480 us, 3.4 TB/s).
//
// What was measured on the way, 65536 x 4096 forward: a thread walking a channel
// alone 31.6 ms; a workgroup owning 16 channels and walking the whole sequence
// 0.53 ms (32-byte rows, one workgroup a CU); tiles with look-back 0.41; keeping
// x and g instead of the states and products of decays, so that five workgroups
// fit a CU, 0.39; past the caches 0.363; the blocks' shift over the XCDs 0.310.
#include "kda_layer.h"
#include "kda_layer_device.h"

#include <type_traits>

#include "kda.h"

namespace kda {
namespace {

struct ScanParams {
  const int32_t* plan;
  BlobLayout L;
  int32_t T, N, F, D;
  const void *x, *g;
  int64_t x_stride, g_stride;
  const float *initial_state, *d_final;
  void* h;
  float* final_state;
  const void *h_in, *dh;
  void *dx, *dg;
  float* d_initial_state;
  int32_t tiles, columns;   // token tiles, channel blocks
  uint32_t* tickets;        // [columns] 32 words apart
  uint64_t* maps;           // [tiles][columns][64]: A, B of a tile
  uint32_t* states;         // [tiles][columns][64]: the state behind a tile
};

// LPR lanes of VEC channels make a row of 64 channels; a thread takes R
// tokens, so that every geometry has the same tile.  LOOK: see look_back;
// STREAM: past the caches.
template <int VEC_, int LPR_, int R_, int LOOK_, bool STREAM_>
struct Geometry {
  static constexpr int VEC = VEC_, LPR = LPR_, R = R_, LOOK = LOOK_;
  static constexpr bool STREAM = STREAM_;
  static_assert(VEC * LPR == kScanChannels && kScanThreads / LPR * R == kScanTile, "");
};
static_assert(kScanTile < kScanThreads, "a thread for each token boundary of a tile");

// The map (A, B) of h; a constant map (A = 0, as a sequence's start gives) is B
// whatever h is, so that an infinity or NaN stays in its own sequence.
__device__ __forceinline__ float apply(float A, float B, float h) { return A == 0.f ? B : __fmaf_rn(A, h, B); }
// The decay of a run that ends with one of decay a: 0 from a constant map on,
// where the product would keep a NaN or infinity of the sequence before.
__device__ __forceinline__ float decay_after(float A, float a) { return a == 0.f ? 0.f : A * a; }

// ------------------------------------------------ the tiles' maps and states
// Words that other workgroups wait for carry their own readiness: all ones
// until written (a NaN that no arithmetic here gives: NaNs are written as the
// canonical one).  So no ordering between words is needed, only agent-scope
// atomics, which reach past the XCDs' own L2 caches.
constexpr uint32_t kEmpty = 0xffffffffu;
__device__ __forceinline__ uint32_t float_bits(float x) { return x != x ? 0x7fc00000u : __float_as_uint(x); }

// The decay e^g of the scan over gates of type E and states stored as O.  In bf16
// throughout the hardware's exponential has to do, in both directions: 65536 x
// 4096 forward 292 us, with the exact one in both walks 320 (backward 235 and
// 238).  Gates near 0, which remember, lose nothing there, and a gate far below
// 0 scales what is left of the state by 1 + |g| units of 2^-24.
template <typename E, typename O>
__device__ __forceinline__ float decay_of(float g) {
  constexpr bool kBf16 = sizeof(E) == 2 && sizeof(O) == 2;
  return kBf16 ? fast_exp(g) : exact_exp(g);
}

// This workgroup's channel block; each block gets as many workgroups as there
// are tiles.  Workgroups go round the 8 XCDs in launch order: without the shift
// from round to round, an XCD would keep the same blocks where their number is
// a multiple of 8, lines 1 KiB apart, and use few of its L2's channels (65536 x
// 4096 forward: 310 us against 363).
__device__ __forceinline__ int32_t column_of(const ScanParams& p) {
  const uint32_t columns = static_cast<uint32_t>(p.columns), round = blockIdx.x / columns;
  return static_cast<int32_t>((blockIdx.x + 5 * round) % columns);
}

// The next tile of this workgroup's channel block.  Tickets are handed out in
// the order of the tiles, so every tile before this one belongs to a workgroup
// that already runs, and the oldest of them waits for nothing: all waits end.
__device__ __forceinline__ uint32_t take_ticket(const ScanParams& p, int32_t column, uint32_t* box) {
  if (p.tiles == 1) return 0u;
  if (threadIdx.x == 0) {
    *box = __hip_atomic_fetch_add(p.tickets + column * 32, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1u;
  }
  __syncthreads();
  return static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int32_t>(*box)));
}

__device__ __forceinline__ int64_t word_of(const ScanParams& p, int32_t tile, int32_t column) {
  return (static_cast<int64_t>(tile) * p.columns + column) * kScanChannels;
}

// The state before tile `tile`, for this wave's lane: channel `lane` of the
// block.  Looks at the LOOK tiles before it until, for every channel, one of
// them has its state and those after it their maps, then applies those maps in
// order: exactly what each of these tiles does itself, so the result does not
// depend on which states were there.  Polls are bounded, so that a workspace
// that another call overwrites gives wrong values, NaN or rows that stay
// unwritten (a ticket given twice or passed over), but no hang.
constexpr int kMaxPolls = 1 << 20;   // seconds; a wait takes microseconds
template <int LOOK>
__device__ __forceinline__ float look_back(const ScanParams& p, int32_t tile, int32_t column) {
  const int32_t lane = threadIdx.x & 63;
  for (int polls = 0; polls < kMaxPolls; ++polls) {
    uint32_t state[LOOK];
    uint64_t map[LOOK];
#pragma unroll
    for (int i = 0; i < LOOK; ++i) {
      const int64_t w = word_of(p, max(tile - 1 - i, 0), column);
      state[i] = __hip_atomic_load(p.states + w + lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      // the farthest tile's map would need a state behind the window
      map[i] = i < LOOK - 1 ? __hip_atomic_load(p.maps + w + lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0;
    }
    bool have = false;
    float h = 0.f;
#pragma unroll
    for (int i = LOOK - 1; i >= 0; --i) {
      if (i >= tile) continue;
      const uint32_t a = static_cast<uint32_t>(map[i]);
      if (state[i] != kEmpty) {
        h = __uint_as_float(state[i]);
        have = true;
      } else if (i == LOOK - 1 || a == kEmpty) {
        have = false;
      } else {
        h = apply(__uint_as_float(a), __uint_as_float(static_cast<uint32_t>(map[i] >> 32)), h);
      }
    }
    if (__ballot(!have) == 0) return h;
    __builtin_amdgcn_s_sleep(8);
  }
  return __uint_as_float(0x7fc00000u);
}

// ------------------------------------------------ sequence boundaries
// mark[i] = n + 1 where sequence n begins at token base + i, for i in
// [0, kScanTile], and N + 1 at the tokens' end; else 0.  Returns whether the
// tile has any.  The whole workgroup calls.
__device__ __forceinline__ bool mark_sequences(const ScanParams& p, int32_t base, int32_t* mark) {
  for (int32_t i = threadIdx.x; i <= kScanTile; i += kScanThreads) mark[i] = 0;
  // A thread looks at one fragment (the last at the tokens' end): of all, or,
  // where they are more than the threads, from the first in the tile on, which
  // no more than kScanTile + 1 can follow.  The search costs a chain of loads.
  int32_t lo = 0;
  if (p.F >= kScanThreads) {
    int32_t hi = p.F;
    while (lo < hi) {
      const int32_t mid = (lo + hi) >> 1;
      if (p.plan[p.L.frag_begin + mid] < base) {
        lo = mid + 1;
      } else {
        hi = mid;
      }
    }
  }
  __syncthreads();
  bool any = false;
  const int32_t f = lo + static_cast<int32_t>(threadIdx.x);
  if (f <= p.F) {
    const int32_t at = (f < p.F ? p.plan[p.L.frag_begin + f] : p.T) - base;
    if (at >= 0 && at <= kScanTile) {
      const bool carried = f < p.F && (p.plan[p.L.frag_flags + f] & kFragCarried) != 0;
      if (!carried) {
        mark[at] = f < p.F ? p.plan[p.L.frag_seq + f] + 1 : p.N + 1;
        any = true;
      }
    }
  }
  return __builtin_amdgcn_readfirstlane(__syncthreads_or(any)) != 0;   // a scalar: the callers' branches too
}

// ------------------------------------------------ composition in the tile
// A thread group is the LPR threads that share R tokens.
template <typename G>
struct TileLds {
  static constexpr int kGroups = kScanThreads / G::LPR;
  float map[kGroups][2][kScanChannels];   // the groups' maps
  float before[kGroups][kScanChannels];   // the states before the groups
  int32_t mark[kScanTile + 1];
  uint32_t ticket;
};

// Given the thread group's map (A, B), the state before it; publishes the
// tile's map and the state behind the tile.  The first wave works alone, a
// lane a channel, from group to group.
template <typename G>
__device__ __forceinline__ void tile_states(const ScanParams& p, int32_t tile, int32_t column, TileLds<G>& lds,
                                            const float (&A)[G::VEC], const float (&B)[G::VEC], float (&in)[G::VEC]) {
  constexpr int VEC = G::VEC, kGroups = TileLds<G>::kGroups;
  const int32_t lane = threadIdx.x & 63, group = threadIdx.x / G::LPR, c0 = (threadIdx.x % G::LPR) * VEC;
  store<VEC>(&lds.map[group][0][c0], A);
  store<VEC>(&lds.map[group][1][c0], B);
  __syncthreads();
  if (__builtin_amdgcn_readfirstlane(threadIdx.x >> 6) == 0) {
    float state = 0.f;
    if (p.tiles > 1) {
      float a = 1.f, b = 0.f;
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        const float ga = lds.map[i][0][lane];
        b = apply(ga, lds.map[i][1][lane], b);
        a = decay_after(a, ga);
      }
      const int64_t w = word_of(p, tile, column) + lane;
      if (tile > 0) {
        __hip_atomic_store(p.maps + w, static_cast<uint64_t>(float_bits(b)) << 32 | float_bits(a), __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
        state = look_back<G::LOOK>(p, tile, column);
      }
      __hip_atomic_store(p.states + w, float_bits(apply(a, b, state)), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      lds.before[i][lane] = state;
      state = apply(lds.map[i][0][lane], lds.map[i][1][lane], state);
    }
  }
  __syncthreads();
  load<VEC>(&lds.before[group][c0], in);
}

// A thread's rows of a tensor: an address that the whole workgroup shares and
// a 32-bit byte offset (kMaxScanStride keeps a tile's within 2^32), so that a
// row costs no address registers.
template <typename E>
struct Span {
  const char* base;   // token `from`, channel 0
  int64_t step;       // bytes from a token to the next
  __device__ __forceinline__ Span(const void* p, int64_t stride, int64_t from)
      : base(static_cast<const char*>(p) + from * stride * static_cast<int64_t>(sizeof(E))),
        step(stride * static_cast<int64_t>(sizeof(E))) {}
  __device__ __forceinline__ uint32_t offset(int32_t token, int32_t channel) const {
    return static_cast<uint32_t>(token) * static_cast<uint32_t>(step) + static_cast<uint32_t>(channel) * sizeof(E);
  }
  // `shift` tokens (the same for the workgroup) from the one at `offset`
  __device__ __forceinline__ E* at(uint32_t offset, int32_t shift) const {
    return reinterpret_cast<E*>(const_cast<char*>(base + shift * step) + offset);
  }
};

// Rows row, row + DIR, ... (tokens from the span's first) of channel dl; where
// not FULL, limited to [0, most].
template <int DIR, bool FULL, bool STREAM, int VEC, int R, typename E>
__device__ __forceinline__ void fetch_rows(const Span<E>& s, int32_t row, int32_t dl, int32_t most, RawVec<E, VEC> (&x)[R]) {
  const uint32_t off = s.offset(row, dl);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if constexpr (FULL) {
      load_raw<STREAM>(s.at(off, DIR * r), x[r]);
    } else {
      load_raw<STREAM>(s.at(s.offset(max(min(row + DIR * r, most), 0), dl), 0), x[r]);
    }
  }
}

template <typename F>
__device__ __forceinline__ void with_flag(bool flag, F&& f) {
  if (flag) {
    f(std::true_type{});
  } else {
    f(std::false_type{});
  }
}

// Row n of per-sequence states [N, D], or zeros where there are none.
template <int VEC>
__device__ __forceinline__ void load_state(const float* states, int32_t n, int32_t D, int32_t d, float (&x)[VEC]) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) x[i] = 0.f;
  if (states != nullptr) load<VEC>(states + static_cast<int64_t>(n) * D + d, x);
}

// Row r's map (a, v) after the map (A, B) of the rows before it.  Unless PLAIN:
// where a sequence begins (mark > 0, in the direction of the walk) it takes in
// that sequence's state (row mark - less of `states`) and is constant; a row
// that does not exist is the identity.
template <bool PLAIN, int VEC>
__device__ __forceinline__ void step_map(int r, int32_t mark, bool valid, const float* states, int32_t less, int32_t D,
                                         int32_t d, float (&a)[VEC], const float (&v)[VEC], float (&A)[VEC],
                                         float (&B)[VEC]) {
  float b[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) b[i] = v[i];
  if (!PLAIN) {
    if (!valid) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        a[i] = 1.f;
        b[i] = 0.f;
      }
    } else if (mark > 0) {
      float s[VEC];
      load_state(states, mark - less, D, d, s);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        b[i] += a[i] * s[i];
        a[i] = 0.f;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    B[i] = r == 0 ? b[i] : PLAIN ? a[i] * B[i] + b[i] : apply(a[i], b[i], B[i]);
    A[i] = r == 0 ? a[i] : PLAIN ? A[i] * a[i] : decay_after(A[i], a[i]);
    // row by row: composing all rows at the end would keep their maps in registers
    if (!PLAIN) asm volatile("" : "+v"(A[i]), "+v"(B[i]));
  }
}

template <typename E, typename O, typename G, bool TIED>
__global__ __launch_bounds__(kScanThreads) void scan_kernel(ScanParams p) {
  constexpr int VEC = G::VEC, R = G::R;
  __shared__ __align__(16) TileLds<G> lds;
  const int32_t column = column_of(p);
  const uint32_t ticket = take_ticket(p, column, &lds.ticket);
  if (!is_tile(ticket, p.tiles)) return;
  const int32_t tile = static_cast<int32_t>(ticket);
  const int32_t row = threadIdx.x / G::LPR * R;                                // first token in the tile
  const int32_t d = column * kScanChannels + (threadIdx.x % G::LPR) * VEC;
  const bool owner = d < p.D;
  // a vector inside the row: the last one shares channels with its neighbour,
  // which computes and writes the same values
  const int32_t dl = min(d, p.D - VEC);
  const int32_t begin = tile * kScanTile, left = min(p.T - begin, kScanTile);
  const Span<E> xs(p.x, p.x_stride, begin), gs(p.g, p.g_stride, begin);
  const Span<O> hs(p.h, p.D, begin);
  RawVec<E, VEC> x[R], g[R];
  with_flag(left == kScanTile, [&](auto full) {
    fetch_rows<1, full.value, G::STREAM>(gs, row, dl, left - 1, g);
    fetch_rows<1, full.value, G::STREAM>(xs, row, dl, left - 1, x);
  });
  const bool marked = mark_sequences(p, begin, lds.mark);
  const uint32_t out = hs.offset(row, dl);
  // PLAIN: a whole tile inside one sequence
  with_flag(left == kScanTile && !marked, [&](auto plain) {
    // the map of this thread's tokens
    constexpr bool kKeep = TIED && plain.value;   // u is kept, else x
    float u[R][VEC], A[VEC], B[VEC], h[VEC];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float a[VEC], v[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float gi = element(g[r], i);
        a[i] = decay_of<E, O>(gi);
        v[i] = TIED ? one_minus_exp(gi, a[i]) * element(x[r], i) : element(x[r], i);
        if (kKeep) u[r][i] = v[i];
      }
      step_map<plain.value>(r, lds.mark[row + r], row + r < left, p.initial_state, 1, p.D, dl, a, v, A, B);
    }
    tile_states<G>(p, tile, column, lds, A, B, h);
    // the states: decays again from g, which takes fewer registers than their values
#pragma unroll
    for (int r = 0; r < R; ++r) {
      forget(g[r]);
      if (!kKeep) forget(x[r]);
      if (!plain.value) {
        const int32_t start = lds.mark[row + r];
        if (start > 0 && row + r < left) load_state(p.initial_state, start - 1, p.D, dl, h);
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float gi = element(g[r], i), a = decay_of<E, O>(gi);
        float v = kKeep ? u[r][i] : element(x[r], i);
        if (TIED && !kKeep) v *= one_minus_exp(gi, a);
        h[i] = a * h[i] + v;
      }
      if (owner && (plain.value || row + r < left)) {
        store<VEC, G::STREAM>(hs.at(out, r), h);
        if (!plain.value) {
          const int32_t next = lds.mark[row + r + 1];   // the sequence after one that ends here
          if (next > 0) store<VEC>(p.final_state + static_cast<int64_t>(next - 2) * p.D + dl, h);
        }
      }
    }
  });
}

// The backward: tiles in order from the tokens' end, row 0 of a tile its last
// token.
template <typename E, typename O, typename G, bool TIED>
__global__ __launch_bounds__(kScanThreads) void scan_backward_kernel(ScanParams p) {
  constexpr int VEC = G::VEC, R = G::R;
  __shared__ __align__(16) TileLds<G> lds;
  const int32_t column = column_of(p);
  const uint32_t ticket = take_ticket(p, column, &lds.ticket);
  if (!is_tile(ticket, p.tiles)) return;
  const int32_t tile = static_cast<int32_t>(ticket);
  const int32_t row = threadIdx.x / G::LPR * R;
  const int32_t d = column * kScanChannels + (threadIdx.x % G::LPR) * VEC;
  const bool owner = d < p.D;
  const int32_t dl = min(d, p.D - VEC);   // as in the forward
  const int32_t end = p.T - tile * kScanTile, left = min(end, kScanTile), base = end - kScanTile;
  // tokens from the tile's first one; this thread's go down from `token`
  const int32_t from = max(base, 0), token = left - 1 - row;
  const Span<E> xs(p.x, p.x_stride, from), gs(p.g, p.g_stride, from), dxs(p.dx, p.D, from), dgs(p.dg, p.D, from);
  const Span<O> dhs(p.dh, p.D, from), hs(p.h_in, p.D, max(from - 1, 0));
  RawVec<E, VEC> x[R], g[R];
  RawVec<O, VEC> dh[R], before[R];                                      // before: h_{t-1}
  with_flag(base >= 1, [&](auto full) {
    fetch_rows<-1, full.value, G::STREAM>(gs, token, dl, left - 1, g);
    fetch_rows<-1, full.value, G::STREAM>(dhs, token, dl, left - 1, dh);
    if (TIED) fetch_rows<-1, full.value, G::STREAM>(xs, token, dl, left - 1, x);
    // token - 1 of the tensor; where there is none (the first token of all), that one
    fetch_rows<-1, full.value, G::STREAM>(hs, base >= 1 ? token : token - 1, dl, left - 1, before);
  });
  const bool marked = mark_sequences(p, base, lds.mark);
  const uint32_t out = dxs.offset(max(token, 0), dl);
  with_flag(base >= 1 && !marked, [&](auto plain) {
    float A[VEC], B[VEC], c[VEC];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float a[VEC], v[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        a[i] = decay_of<E, O>(element(g[r], i));
        v[i] = a[i] * element(dh[r], i);
      }
      // a sequence's last token: c = a (dh + d_final)
      step_map<plain.value>(r, lds.mark[kScanTile - row - r], row + r < left, p.d_final, 2, p.D, dl, a, v, A, B);
    }
    tile_states<G>(p, tile, column, lds, A, B, c);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool valid = plain.value || row + r < left;
      forget(g[r]);   // as in the forward
      forget(dh[r]);
      float hp[VEC], dx[VEC], dg[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) hp[i] = element(before[r], i);
      int32_t start = 0;
      if (!plain.value && valid) {
        start = lds.mark[kScanTile - 1 - row - r];
        if (start > 0) load_state(p.initial_state, start - 1, p.D, dl, hp);
        const int32_t next = lds.mark[kScanTile - row - r];
        if (next > 0) load_state(p.d_final, next - 2, p.D, dl, c);
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float gi = element(g[r], i), a = decay_of<E, O>(gi), l = element(dh[r], i) + c[i];
        dx[i] = TIED ? one_minus_exp(gi, a) * l : l;
        c[i] = a * l;
        dg[i] = c[i] * (TIED ? hp[i] - element(x[r], i) : hp[i]);
      }
      if (owner && valid) {
        store<VEC, G::STREAM>(dxs.at(out, -r), dx);
        store<VEC, G::STREAM>(dgs.at(out, -r), dg);
        if (start > 0 && p.d_initial_state != nullptr) {
          store<VEC>(p.d_initial_state + static_cast<int64_t>(start - 1) * p.D + dl, c);
        }
      }
    }
  });
}

// All ones over the tickets, maps and states of a call: n 16-byte words.
__global__ __launch_bounds__(256) void scan_clear_kernel(u32x4* words, int64_t n) {
  const u32x4 ones = {kEmpty, kEmpty, kEmpty, kEmpty};
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256) {
    words[i] = ones;
  }
}

template <typename E, typename O, typename G>
int run(ScanParams p, bool tied, bool backward, void* workspace, hipStream_t stream) {
  const ScanLayout L = scan_layout(p.T, p.D);
  p.tiles = L.tiles;
  p.columns = L.columns;
  const int64_t grid = static_cast<int64_t>(p.tiles) * p.columns;
  if (grid * kScanThreads > 4294967295LL) return KDA_ERR_UNSUPPORTED;
  (void)hipGetLastError();
  if (L.total > 0) {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.tickets = reinterpret_cast<uint32_t*>(ws + L.tickets);
    p.maps = reinterpret_cast<uint64_t*>(ws + L.maps);
    p.states = reinterpret_cast<uint32_t*>(ws + L.states);
    const int64_t words = static_cast<int64_t>(L.total / 16), blocks = (words + 255) / 256;
    hipLaunchKernelGGL(scan_clear_kernel, dim3(static_cast<uint32_t>(blocks < 2048 ? blocks : 2048)), dim3(256), 0, stream,
                       reinterpret_cast<u32x4*>(ws), words);
    const int st = finish_launch();
    if (st != KDA_OK) return st;
  }
  void (*kernel)(ScanParams) = backward ? (tied ? scan_backward_kernel<E, O, G, true> : scan_backward_kernel<E, O, G, false>)
                                        : (tied ? scan_kernel<E, O, G, true> : scan_kernel<E, O, G, false>);
  hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(grid)), dim3(kScanThreads), 0, stream, p);
  return finish_launch();
}

// Many tiles of a channel block are in flight where there are few blocks, and
// a wide window lets a state pass over more of them at once; where there are
// many, its registers cost more than it gives.  Forward, 32768 tokens, bf16, a
// window of 4 against one of 16: 4096 channels (64 blocks) 193 and 227 us,
// 2048 109 and 122, 1024 77 and 68, 512 65 and 44, 64 57 and 36.
constexpr int32_t kNarrowBlocks = 24;
using Vector = Geometry<4, 16, 8, 4, false>;         // rows of at least one 4-element vector
// The same from kStreamBytes on, if every row is whole 128-byte lines.  At
// 1.6 GB (65536 x 4096 forward) past the caches 364 us against 388, at 101 MB
// (4096 x 4096) 32 and 29; with lines that two rows share (32768 x 4093) 344
// and 269.
using VectorStream = Geometry<4, 16, 8, 4, true>;
using VectorNarrow = Geometry<4, 16, 8, 16, false>;  // of fewer than kNarrowBlocks blocks
using Scalar = Geometry<1, 64, 32, 16, false>;       // rows of up to three elements

template <typename G>
int run_types(const ScanArgs& a, bool backward, const ScanParams& p, hipStream_t stream) {
  const bool e16 = a.dtype == KDA_BF16, o16 = a.h_format == KDA_BF16, tied = a.tied != 0;
  if (e16 && o16) return run<bf16_t, bf16_t, G>(p, tied, backward, a.workspace.ptr, stream);
  if (e16) return run<bf16_t, fp32_t, G>(p, tied, backward, a.workspace.ptr, stream);
  if (o16) return run<fp32_t, bf16_t, G>(p, tied, backward, a.workspace.ptr, stream);
  return run<fp32_t, fp32_t, G>(p, tied, backward, a.workspace.ptr, stream);
}

int launch_either(const ScanArgs& a, bool backward, hipStream_t stream) {
  ScanParams p{};
  p.plan = static_cast<const int32_t*>(a.plan_dev.ptr);
  p.L = a.plan->layout;
  p.T = a.plan->T;
  p.N = a.plan->N;
  p.F = a.plan->F;
  p.D = a.D;
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
  if (a.D < Vector::VEC) return run_types<Scalar>(a, backward, p, stream);
  if (a.D < kNarrowBlocks * kScanChannels) return run_types<VectorNarrow>(a, backward, p, stream);
  const int64_t e = a.dtype == KDA_BF16 ? 2 : 4, eh = a.h_format == KDA_BF16 ? 2 : 4;
  const bool reads_x = !backward || a.tied != 0;
  const int64_t element = backward ? (a.tied != 0 ? 4 : 3) * e + 2 * eh : 2 * e + eh;
  // whole 128-byte lines in every row of every tensor
  const bool lines = a.D % 64 == 0 && a.g.stride % 64 == 0 && (!reads_x || a.x.stride % 64 == 0);
  if (lines && static_cast<int64_t>(p.T) * p.D * element >= kStreamBytes) {
    return run_types<VectorStream>(a, backward, p, stream);
  }
  return run_types<Vector>(a, backward, p, stream);
}

}  // namespace

int launch_scan(const ScanArgs& a, hipStream_t stream) { return launch_either(a, false, stream); }
int launch_scan_backward(const ScanArgs& a, hipStream_t stream) { return launch_either(a, true, stream); }

}  // namespace kda
