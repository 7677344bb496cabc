// One pass of linear attention with a decay for each head over a fragment's
// 64-token chunks, on the bf16 matrix cores.
//
// With queries x, keys y, values z, a state S [KD, VD] (rows: channels of y) and
// the prefix sums G of the chunk's gates, a forward pass has per chunk
//     out_i = sum_{j <= i} e^{G_i - G_j} (x_i . y_j) z_j + e^{G_i} S^T x_i
//     S    <- e^{G_C} S + sum_j e^{G_C - G_j} y_j z_j^T
// and a reversed one, which walks the chunks from the last to the first,
//     out_j = sum_{i >= j} e^{G_i - G_j} (x_j . y_i) z_i + e^{G_C - G_j} S^T x_j
//     S    <- e^{G_C} S + sum_i e^{G_i} y_i z_i^T.
// The operator is the forward pass of (q, k, v); of its gradients, dq is the
// forward pass of (do, v, k) with the state transposed, dk the reversed pass of
// (v, do, q) transposed, dv the reversed pass of (k, q, do).
//
// A workgroup is one fragment of one head, four waves.  A wave holds a quarter of
// S's columns in FP32 accumulators, tiles of 32 x 32 or, where VD is 64, 16 x 16; x,
// y, z of the chunk lie in LDS in bf16, exactly as they came.  Whatever is not exact
// in bf16 is split into bf16 parts (8 bits each): two of them leave 2^-16, three 2^-24
// of a factor.
//   * P = (x y^T) o decay: 16 x 16 tiles, a wave owns whole rows of tiles; its
//     parts go through LDS, as they are every wave's operand.  Two parts where the
//     output is BF16, three for FP32.
//   * out^T = S^T x^T + z^T P^T: transposed, so that a lane has one token and four
//     neighbouring channels.  S's accumulators are the matrix core's operand as
//     they are: its rows stand for channels in the order that makes a lane's k
//     slots eight neighbouring channels.  They are split in registers, in two parts
//     where only a BF16 output comes of it, in three for FP32 and for dq and dk, whose
//     products with q and k are the gates' gradient.
//   * S's update: z, read transposed, times its weights, split in registers, always
//     in three parts, as a state is FP32; y read transposed.
// The chunks come by copies from memory to LDS that take no registers: x of the next
// chunk after its last reader in this one, y into a second buffer a chunk ahead, z
// beside P, which does not need it.  80 KB of LDS and 256 registers, two workgroups
// a CU.
// Decays: a gate of a token enters with at least -160 in units of 2 (2^-160 is 0 in
// FP32), prefix sums are taken in FP64 and kept as a multiple of 2^-9 and the
// rest, so that the difference of two of them is exact however large they are.
//
// Measured at 128 x 128, in a row of launches at 2.0 GHz (in the first after a pause the
// clock falls to 1.5, with the same cycles and a third more time).  Forward, 65536 tokens
// x 32 heads: 230 us for the pieces' own updates (1.07 GB, 4.7 TB/s), 18 for their scan,
// 510 for the outputs (2.25 GB, 4.4 TB/s; the copies and stores of that pass alone take
// 476, its products alone 400 to 427; matrix cores busy 42 %, vector units 39 %).  The
// same with FP32 outputs, one workgroup a CU: 1164 in all for 813.  Gradients of 16384 x
// 32: 125 + 27 for both directions' pieces, 545 for the three passes, 28 for the gates.
// No unit bounds those passes: matrix cores are busy 30 %, vector units 40 %, LDS 20 %,
// and waves wait 43 % of their cycles, for barriers and copies that two workgroups a CU
// do not cover.  FP32 gradients 1090 in all for 742.  What the choices are worth, each
// when it was made: through registers instead of copies, with spills 974 (forward) and
// 1153 (gradients) for 825 and 769; 8 waves of 16 columns at this width 1035 for 905; 4
// waves of 16 columns where VD is 64 102 for 119 (24 sequences of 16384 x 16 in all); the
// gradients' passes in one launch 45 for 60 (1501 x 6); buffers' resources from the
// first lane and fewer addresses spilt (12 bytes are) 721 for 761 (16384 x 32);
// subtraction of parts by dot2 instructions, other schedulers, grouped schedules: the
// same.  Then exactness of the gates' gradient: 707 to 734 for what passes by a chunk,
// 746 with decays of 24 bits in it.
#ifndef KDA_LINEAR_PASS_H_
#define KDA_LINEAR_PASS_H_

#include <hip/hip_runtime.h>

#include <cstdint>

#include "kda_layer.h"
#include "kda_layer_device.h"

namespace kda {

// The next token's row is `stride` elements on; head h reads row head h / share,
// `width` elements.
struct Tokens {
  const uint16_t* p;
  int64_t stride;
  int32_t share, width;
};

// What a pass finds of the gates' gradient.
struct GateParts {
  float* tokens;   // [H][T], the pairs with one token in the chunk
  f32x4* border;   // [slot][H] what passes a border of the chunk (query: its first token's, key: its last's),
                   // the norm of the state there, the chunk's decay, nothing
  float* by;       // [fragment][H] what passes by the chunk where the pass ends
  float* anchors;  // [anchor][H][K][V] the state at that border of every kAnchorChunks-th chunk of a fragment
};

struct LinearParams {
  const int32_t* plan;
  BlobLayout L;
  int32_t T, H, KW, VW;         // tokens, heads, widths in use (KW <= KD, VW <= VD)
  Tokens x, y, z, e;            // e: q (kQuery) or k (kKey)
  const void* g;
  int64_t g_stride;
  int32_t g_bf16;
  int32_t transposed;           // states in memory are [VW][KW]
  int32_t reversed;             // kSummary
  const float* seq_state;       // where a sequence begins (reversed: ends), or null
  const float* piece_state;     // where a piece goes on: its own state before (reversed: after) it
  float* seq_out;               // at the other end, or null
  float *piece_out, *decay_out; // kSummary
  void* o;                      // [T, H, VW]
  int32_t o_fp32;
  GateParts gates;              // kQuery, kKey
  const float *end_seq, *end_piece;   // the states of the other gradient where this pass ends (seq: or null)
};

// kSummary: a fragment's own state and decay alone.  kQuery and kKey: also what
// queries and keys take and give of the gates' gradient.
enum LinearMode { kSummary, kOutput, kQuery, kKey };

constexpr int kLinearChunk = 64;
constexpr float kLeastGate = -160.f;

// 2^(high + low), high a multiple of 2^-9 and |low| at most that.  EXACT: what the sum
// lost in FP32, up to half a unit of 2^6, is worked in to first order, as in exact_exp,
// to 4 units of 2^-24 for 45; without it for what is used with 16 bits.
template <bool EXACT>
__device__ __forceinline__ float power2(float high, float low) {
  const float x = high + low, e = __builtin_amdgcn_exp2f(x);
  return EXACT ? __fmaf_rn(e, (low - (x - high)) * kLn2, e) : e;
}
__device__ __forceinline__ float power2(double x) {
  const float high = static_cast<float>(x), e = __builtin_amdgcn_exp2f(high);
  return __fmaf_rn(e, static_cast<float>(x - high) * kLn2, e);
}

// Tiles of 64 tokens, rows of W bf16 in 16-byte units; the unit's place is xored
// with bits of the row, so that 16 rows' units of one column, and 4 rows' 64
// bytes, lie on different banks.
template <int W>
__device__ __forceinline__ int row_bits(int row) {
  return W == 128 ? ((row & 3) << 2) | ((row >> 2) & 3) : (((row >> 1) & 1) << 2) | ((row >> 2) & 3);
}
template <int W>
__device__ __forceinline__ const bf16* unit_at(const bf16* tile, int row, int unit) {
  return tile + row * W + ((unit ^ row_bits<W>(row)) << 3);
}
template <int W>
__device__ __forceinline__ bf16* unit_at(bf16* tile, int row, int unit) {
  return const_cast<bf16*>(unit_at<W>(static_cast<const bf16*>(tile), row, unit));
}
// 8 bytes, volatile, so that two are not fused into one ds_read2_b64, which takes
// four times as long
__device__ __forceinline__ bf16x4 ld_piece(const bf16* p) { return *(lds_bf16x4*)(const_cast<bf16*>(p)); }
__device__ __forceinline__ bf16x8 ld_unit(const bf16* p) { return *reinterpret_cast<const bf16x8*>(p); }

// A buffer of `bytes` bytes from p on, for raw 32-bit accesses (the resource's last
// word says so): loads past it give zero and touch no memory, stores past it are
// dropped.  The resource is read from the first lane: where the compiler holds it in
// vector registers it would walk the lanes at each access.
constexpr int kRawBuffer = 0x00020000;
__device__ __forceinline__ auto buffer_of(const void* p, int64_t bytes) {
  const uint64_t at = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at)),
                 hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(static_cast<uint64_t>(hi) << 32 | lo), 0,
                                           __builtin_amdgcn_readfirstlane(static_cast<int>(bytes)), kRawBuffer);
}
constexpr uint32_t kOutside = 0x80000000u;   // no buffer is that long

// A thread's share of a tile on its way to LDS through registers.
template <int W>
struct Staged {
  static constexpr int kRows = 256 / (W / 8), kSteps = kLinearChunk / kRows;
  u32x4 r[kSteps];

  // Byte offset of the thread's first unit in the chunk's rows; columns behind the
  // width are outside.
  static __device__ __forceinline__ uint32_t offset(const Tokens& t) {
    const int row = static_cast<int>(threadIdx.x) / (W / 8), c = static_cast<int>(threadIdx.x) % (W / 8);
    return 8 * c < t.width ? static_cast<uint32_t>(row) * static_cast<uint32_t>(t.stride) * 2 + 16 * c : kOutside;
  }
  __device__ __forceinline__ void load(const Tokens& t, uint32_t at, int head, int64_t t0, int valid) {
    const auto rows = buffer_of(t.p + t0 * t.stride + static_cast<int64_t>(head / t.share) * t.width,
                                (valid - 1) * t.stride * 2 + t.width * 2);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      r[i] = __builtin_amdgcn_raw_buffer_load_b128(rows, at + i * (kRows * static_cast<uint32_t>(t.stride) * 2), 0, 0);
    }
  }
  __device__ __forceinline__ void store(bf16* tile) const {
    const int row = static_cast<int>(threadIdx.x) / (W / 8), c = static_cast<int>(threadIdx.x) % (W / 8);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) st4(unit_at<W>(tile, i * kRows + row, c), r[i]);
  }
};

// A tile on its way from memory to LDS without registers: a wave's copy moves 64
// 16-byte units to 1 KiB of LDS, lane after lane, so each lane takes the unit whose
// place its own is.
template <int W>
struct Copy {
  static constexpr int kRows = 64 / (W / 8);             // of a copy
  static constexpr int kSteps = kLinearChunk / kRows / 4;   // of a wave
  uint32_t at, step;

  __device__ __forceinline__ Copy(const Tokens& t, int wave, int lane)
      : step(kRows * 4 * static_cast<uint32_t>(t.stride) * 2) {
    const int row = wave * kRows + lane / (W / 8);
    const int c = (lane % (W / 8)) ^ row_bits<W>(row);   // the same bits 4 kRows rows on
    at = 8 * c < t.width ? static_cast<uint32_t>(row) * static_cast<uint32_t>(t.stride) * 2 + 16 * c : kOutside;
  }
  // rows behind `valid` become zero
  __device__ __forceinline__ void start(const Tokens& t, int head, int64_t t0, int valid, bf16* tile, int wave) const {
    const uint64_t base = reinterpret_cast<uint64_t>(t.p + t0 * t.stride + static_cast<int64_t>(head / t.share) * t.width);
    u32x4 rows;
    rows[0] = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(base));
    rows[1] = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(base >> 32) & 0xffffu);
    rows[2] = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>((valid - 1) * static_cast<int>(t.stride) * 2 + t.width * 2));
    rows[3] = kRawBuffer;
    typedef __attribute__((address_space(3))) bf16* Lds;
    const uint32_t lds = __builtin_amdgcn_readfirstlane(
        static_cast<uint32_t>(reinterpret_cast<uintptr_t>((Lds)tile)) + wave * 1024);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                   :: "s"(lds + i * 4096), "v"(at + i * step), "s"(rows) : "memory", "m0");
    }
  }
};
// Waits until at most N of the wave's last memory accesses are under way.
template <int N>
__device__ __forceinline__ void copies_done() {
  asm volatile("s_waitcnt vmcnt(%0)" :: "n"(N) : "memory");
}

// Eight tokens row0 .. row0 + 7 of column col0 + lane % 32 (col0, row0 multiples of
// 32 and 8).
template <int W>
__device__ __forceinline__ bf16x8 column_tokens(const bf16* tile, int row0, int col0, int lane) {
  const int s = lane & 15, unit = (col0 >> 3) + 2 * ((lane >> 4) & 1) + ((s & 3) >> 1), row = row0 + (s >> 2);
  return join8(lds_read_tr(unit_at<W>(tile, row, unit) + 4 * (s & 1)),
               lds_read_tr(unit_at<W>(tile, row + 4, unit) + 4 * (s & 1)));
}
// Eight tokens of column col0 + lane % 16.
template <int W>
__device__ __forceinline__ bf16x8 column16_tokens(const bf16* tile, int row0, int col0, int lane) {
  const int s = lane & 15, unit = (col0 >> 3) + ((s & 3) >> 1), row = row0 + (s >> 2);
  return join8(lds_read_tr(unit_at<W>(tile, row, unit) + 4 * (s & 1)),
               lds_read_tr(unit_at<W>(tile, row + 4, unit) + 4 * (s & 1)));
}
// 32 columns with the second and third four of every 16 columns exchanged: rows of the
// product are then S's rows as they are kept.
template <int W>
__device__ __forceinline__ bf16x8 slot_column_tokens(const bf16* tile, int row0, int col0, int lane) {
  const int s = lane & 15, n = ((s & 1) << 1) | ((s & 2) >> 1), row = row0 + (s >> 2);
  const int unit = (col0 >> 3) + 2 * ((lane >> 4) & 1) + (n >> 1);
  return join8(lds_read_tr(unit_at<W>(tile, row, unit) + 4 * (n & 1)),
               lds_read_tr(unit_at<W>(tile, row + 4, unit) + 4 * (n & 1)));
}

// Takes the pair h of bf16 from (a, b), exactly: x less its bf16 rounding is an FP32
// number.
__device__ __forceinline__ void minus(uint32_t h, float& a, float& b) {
  a -= __uint_as_float(h << 16);
  b -= __uint_as_float(h & 0xffff0000u);
}

// x as N bf16 parts, each the rest of those before it rounded.
template <int N>
__device__ __forceinline__ void split_parts(const float (&x)[8], bf16x8 (&part)[N]) {
  u32x4 w[N];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = x[2 * i], b = x[2 * i + 1];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const uint32_t h = pack_bf16(a, b);
      w[n][i] = h;
      if (n + 1 < N) minus(h, a, b);
    }
  }
#pragma unroll
  for (int n = 0; n < N; ++n) part[n] = __builtin_bit_cast(bf16x8, w[n]);
}

// P: out tokens i by tokens j of the sum, 32 x 32 blocks of the triangle's side
// that is not empty (block of i plus block of j), 16-byte units xored as above.
constexpr int kPartSize = 3 * 1024;
__device__ __forceinline__ bf16* p_unit(bf16* part, int block, int row, int unit) {
  return part + block * 1024 + row * 32 + ((unit ^ ((row >> 2) & 3)) << 3);
}

template <int KD, int VD, int PS, int MODE>
struct LinearSmem {
  static constexpr bool kOut = MODE != kSummary;
  __align__(16) bf16 x[kOut ? kLinearChunk * KD : 8];
  __align__(16) bf16 y[MODE == kQuery ? 1 : 2][kLinearChunk * KD];
  __align__(16) bf16 z[MODE == kSummary ? 2 : 1][kLinearChunk * VD];
  __align__(16) bf16 e[MODE == kQuery ? kLinearChunk * VD : 8];
  __align__(16) bf16 p[kOut ? PS * kPartSize : 8];
  struct Gates {
    __align__(16) float high[kLinearChunk], low[kLinearChunk], w_in[kLinearChunk];
    float whole;
  } gates[2];   // of this chunk and the next
  __align__(16) float pairs[MODE == kQuery ? 4 : 1][kLinearChunk];
  float dots[4][kLinearChunk];
  float by[4], squares[2][4];   // squares: of this chunk's state and the next's
};

// A wave's part of a state in memory: f(four neighbouring values of the tiles, their
// first row).  32 x 32 tiles hold rows in the order that makes a lane's k slots
// neighbouring channels, 16 x 16 tiles as they are.
template <int CW, typename Acc, int KT, typename F>
__device__ __forceinline__ void each_quad(Acc (&S)[KT], int lane, F f) {
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) {
    if constexpr (CW == 32) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f32x4 v = {S[kt][4 * q], S[kt][4 * q + 1], S[kt][4 * q + 2], S[kt][4 * q + 3]};
        f(v, 32 * kt + 16 * (q >> 1) + 8 * (lane >> 5) + 4 * (q & 1));
#pragma unroll
        for (int j = 0; j < 4; ++j) S[kt][4 * q + j] = v[j];
      }
    } else {
      f(S[kt], 16 * kt + 4 * (lane >> 4));
    }
    asm volatile("" ::: "memory");   // a tile's loads and addresses at a time
  }
}
__device__ __forceinline__ f32x4 load_quad(const LinearParams& p, const float* s, int row, int col) {
  if (p.transposed) return ld4(s + static_cast<int64_t>(col) * p.KW + row);
  f32x4 v;
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = s[(row + j) * p.VW + col];
  return v;
}
__device__ __forceinline__ void store_quad(const LinearParams& p, float* s, int row, int col, const f32x4 v) {
  if (p.transposed) {
    st4(s + static_cast<int64_t>(col) * p.KW + row, v);
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) s[(row + j) * p.VW + col] = v[j];
}

// The inclusive prefix sum over the wave's 64 lanes: within rows of 16 by row shifts,
// then each row's total broadcast to those behind it.  No lane needs another's address.
template <int CTRL, int ROWS>
__device__ __forceinline__ float from_lane(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, ROWS, 0xf, true));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float prefix_step(float x) {
  return x + from_lane<CTRL, ROWS>(x);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double prefix_step(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(b), CTRL, ROWS, 0xf, true),
                 hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(b >> 32), CTRL, ROWS, 0xf, true);
  return x + __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}
template <typename X>
__device__ __forceinline__ X wave_prefix(X x) {
  x = prefix_step<0x111, 0xf>(x);
  x = prefix_step<0x112, 0xf>(x);
  x = prefix_step<0x114, 0xf>(x);
  x = prefix_step<0x118, 0xf>(x);
  x = prefix_step<0x142, 0xa>(x);   // lane 15 to row 1, lane 47 to row 3
  return prefix_step<0x143, 0xc>(x);   // lane 31 to rows 2 and 3
}
__device__ __forceinline__ float last_lane(float x) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 63));
}

__device__ __forceinline__ f32x16 product(const bf16x8& a, const bf16x8& b, const f32x16& c) { return mfma(a, b, c); }
__device__ __forceinline__ f32x4 product(const bf16x8& a, const bf16x8& b, const f32x4& c) { return mfma16(a, b, c); }
template <int N>
struct LinearAcc;
template <>
struct LinearAcc<32> {
  typedef f32x16 type;
};
template <>
struct LinearAcc<16> {
  typedef f32x4 type;
};

template <int KD, int VD, int SS, int PS, bool REV, int MODE>
__device__ __forceinline__ void linear_pass(const LinearParams& p, LinearSmem<KD, VD, PS, MODE>& sm) {
  constexpr int CW = VD / 4, KT = KD / CW, OT = kLinearChunk / CW, US = 3;   // a wave's columns, tiles of S and of out
  constexpr bool kOut = MODE != kSummary;
  typedef typename LinearAcc<CW>::type Acc;
  const bool rev = MODE == kSummary ? p.reversed != 0 : REV;

  const int32_t f = p.plan[p.L.frag_order + static_cast<int32_t>(blockIdx.x / static_cast<uint32_t>(p.H))];
  const int32_t head = static_cast<int32_t>(blockIdx.x % static_cast<uint32_t>(p.H));
  const int32_t flags = p.plan[p.L.frag_flags + f], seg = p.plan[p.L.frag_seg + f], seq = p.plan[p.L.frag_seq + f];
  const int32_t begin = p.plan[p.L.frag_begin + f], end = p.plan[p.L.frag_end + f];
  const bool carried = (flags & kFragCarried) != 0, seq_end = (flags & kFragSeqEnd) != 0;
  // whether the pass starts (ends) at its sequence's own end, not at a cut
  const bool starts = rev ? seq_end : !carried, ends = rev ? !carried : seq_end;
  if (!kOut && ends) return;   // nothing goes on from here

  const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5, l16 = lane & 15, quad = lane >> 4;
  const int lcol = lane % CW, lrow = lane / CW;   // a tile's column, and which rows
  const int col = CW * wave + lcol;
  const int64_t size = static_cast<int64_t>(p.KW) * p.VW;

  Acc S[KT];
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) {
#pragma unroll
    for (int i = 0; i < CW * CW / 64; ++i) S[kt][i] = 0.f;
  }
  {
    const float* from = starts ? p.seq_state : kOut ? p.piece_state : nullptr;
    if (from != nullptr) {
      from += (static_cast<int64_t>(starts ? seq : seg) * p.H + head) * size;
      each_quad<CW>(S, lane, [&](f32x4& v, int row) {
        if (row < p.KW && col < p.VW) v = load_quad(p, from, row, col);
      });
    }
  }
  const int chunks = (end - begin + kLinearChunk - 1) / kLinearChunk;
  double total = 0.0;

  const Copy<KD> cx(p.x, wave, lane), cy(p.y, wave, lane);
  Staged<KD> sy;
  Staged<VD> sz;
  const uint32_t at_y = MODE == kQuery ? sy.offset(p.y) : 0, at_z = MODE == kQuery ? sz.offset(p.z) : 0;
  const Copy<VD> cz(p.z, wave, lane), ce(p.e, wave, lane);
  const uint32_t o_size = p.o_fp32 ? 4 : 2, o_row = static_cast<uint32_t>(p.H) * p.VW * o_size;
  const uint32_t at_key = lcol * static_cast<uint32_t>(p.e.stride) * 2 + (CW * wave + 4 * lrow) * 2;
  // first token of the chunk that is walked as number `it`, and its tokens
  const auto first_of = [&](int it) { return static_cast<int64_t>(begin) + (rev ? chunks - 1 - it : it) * kLinearChunk; };
  const auto valid_of = [&](int64_t t0) { return min(kLinearChunk, end - static_cast<int>(t0)); };
  const auto start_x = [&](int it) {
    if (!kOut || it >= chunks) return;
    const int64_t t0 = first_of(it);
    cx.start(p.x, head, t0, valid_of(t0), sm.x, wave);
    if (MODE == kQuery) ce.start(p.e, head, t0, valid_of(t0), sm.e, wave);
  };
  const auto start_y = [&](int it) {
    if (it >= chunks) return;
    const int64_t t0 = first_of(it);
    if constexpr (MODE == kQuery) {   // all four tiles are read to the chunk's end but x and e: no room for two of y
      sy.load(p.y, at_y, head, t0, valid_of(t0));
      sz.load(p.z, at_z, head, t0, valid_of(t0));
    } else {
      cy.start(p.y, head, t0, valid_of(t0), sm.y[it & 1], wave);
    }
  };
  const auto start_z = [&](int it) {
    const int64_t t0 = first_of(it);
    cz.start(p.z, head, t0, valid_of(t0), sm.z[kOut ? 0 : it & 1], wave);
  };
  // What comes through registers: wave 0's gates, two chunks ahead as their prefix
  // sums are made beside P, and for kKey a lane's channels of k.  The compiler does
  // not know of the copies, so it would wait for all of them before it uses such a
  // value; `landed` uses them where the copies before them have been waited for
  // anyway.
  uint32_t gate = 0;
  constexpr int kKeys = CW * CW / 256 * OT;   // a lane's quads of out
  u32x2 key[MODE == kKey ? kKeys : 1];
  const auto fetch_gate = [&](int it) {
    if (wave != 0 || it >= chunks) return;
    const int64_t t0 = first_of(it), size = p.g_bf16 ? 2 : 4;
    const auto rows = buffer_of(static_cast<const char*>(p.g) + (t0 * p.g_stride + head) * size,
                                (valid_of(t0) - 1) * p.g_stride * size + size);
    const uint32_t at = lane * static_cast<uint32_t>(p.g_stride) * static_cast<uint32_t>(size);
    if (p.g_bf16) {
      gate = static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(rows, at, 0, 0));
    } else {
      gate = __builtin_amdgcn_raw_buffer_load_b32(rows, at, 0, 0);
    }
  };
  const auto fetch_key = [&](int it) {
    if constexpr (MODE == kKey) {
      if (it >= chunks) return;
      const int64_t t0 = first_of(it);
      const int valid = valid_of(t0);
      const auto rows = buffer_of(p.e.p + t0 * p.e.stride + static_cast<int64_t>(head / p.e.share) * p.e.width,
                                  (valid - 1) * p.e.stride * 2 + p.e.width * 2);
#pragma unroll
      for (int n = 0; n < kKeys; ++n) {
        const int tile = n / (kKeys / OT), q = n % (kKeys / OT);
        const uint32_t at = at_key + CW * tile * static_cast<uint32_t>(p.e.stride) * 2 + 16 * q;
        key[n] = __builtin_amdgcn_raw_buffer_load_b64(rows, CW * wave + 8 * q + 4 * lrow < p.VW ? at : kOutside, 0, 0);
      }
    }
  };
  const auto landed = [&] {
    asm volatile("" : "+v"(gate));
    if constexpr (MODE == kKey) {
#pragma unroll
      for (int n = 0; n < kKeys; ++n) asm volatile("" : "+v"(key[n]));
    }
  };
  const auto make_gates = [&](int it) {
    if (wave != 0 || it >= chunks) return;
    auto& to = sm.gates[it & 1];
    const float g = lane < valid_of(first_of(it)) ? __uint_as_float(p.g_bf16 ? gate << 16 : gate) : 0.f;
    double G = static_cast<double>(g) * 1.4426950408889634074;
    if (G < kLeastGate) G = kLeastGate;   // NaN stays
    G = wave_prefix(G);
    const double last = __shfl(G, 63);
    const double high = rint(G * 512.0) * (1.0 / 512.0);
    to.high[lane] = static_cast<float>(high);
    to.low[lane] = static_cast<float>(G - high);
    to.w_in[lane] = power2(rev ? G : last - G);
    if (lane == 0) to.whole = power2(last);
    total += last;
  };
  fetch_gate(0);
  make_gates(0);
  fetch_gate(1);
  fetch_key(0);
  start_y(0);
  if (kOut) start_x(0);
  if (!kOut) start_z(0);
  // the squares of the state at chunk it's border, and there the anchor's copy of it,
  // where a chunk lies between the first and the last
  const auto measure = [&](int it) {
    if constexpr (MODE == kQuery || MODE == kKey) {
      if (chunks < 3) return;
      float squares = 0.f;
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
#pragma unroll
        for (int i = 0; i < CW * CW / 64; ++i) squares += S[kt][i] * S[kt][i];
      }
      squares = last_lane(wave_prefix(squares));
      if (lane == 0) sm.squares[it & 1][wave] = squares;
      const int c = rev ? chunks - 1 - it : it;
      if (it > 0 && c > 0 && c + 1 < chunks && c % kAnchorChunks == 0) {
        const int place = opaque(begin) / (kAnchorChunks * kLinearChunk) + c / kAnchorChunks - 1, at = opaque(col);
        float* const to = p.gates.anchors + (static_cast<int64_t>(place) * p.H + opaque(head)) * size;
        each_quad<CW>(S, opaque(lane), [&](f32x4& v, int row) {
          if (row < p.KW && at < p.VW) store_quad(p, to, row, at, v);
        });
      }
    }
  };
  measure(0);
  // What the first chunk needs; the others' is waited for at the end of the chunk
  // before, so that nothing that the compiler knows of is under way at the loop's
  // head: it would wait for it where the value is used, after the next copies.
  copies_done<0>();
  landed();

  for (int it = 0; it < chunks; ++it) {
    const int c = rev ? chunks - 1 - it : it;
    const int64_t t0 = begin + c * kLinearChunk;
    const int valid = min(kLinearChunk, end - static_cast<int>(t0));
    const int Y = MODE == kQuery ? 0 : it & 1, Z = kOut ? 0 : it & 1;
    const bool last = (MODE == kQuery || (MODE == kKey && chunks > 1)) && it + 1 == chunks;
    if constexpr (MODE == kQuery) {
      block_sync();   // the last chunk's readers
      sy.store(sm.y[0]);
      sz.store(sm.z[0]);
      copies_done<4>();   // x, e, while the last chunk's stores go on
      landed();
      block_sync();
    } else {
      block_sync();   // everyone's; and the last chunk's readers are done
      if (kOut) start_z(it);
    }
    start_y(it + 1);
    if (!kOut && it + 1 < chunks) start_z(it + 1);
    make_gates(it + 1);
    fetch_gate(it + 2);
    const auto& gates = sm.gates[it & 1];
    // kQuery: the addresses of what is read by columns are made anew, as all would not fit
    const int reader = MODE == kQuery ? opaque(lane) : lane;

    Acc out[OT];
    if constexpr (kOut) {
      // P: tiles of 16 out tokens (columns) by 16 tokens of the sum (rows)
      {
        const int a = wave;
        bf16x8 xf[KD / 32];
#pragma unroll
        for (int s = 0; s < KD / 32; ++s) xf[s] = ld_unit(unit_at<KD>(sm.x, 16 * a + l16, 4 * s + quad));
        const float high = gates.high[16 * a + l16], low = gates.low[16 * a + l16];
        float before = 0.f;   // kQuery: the pairs' sum over the tiles so far
        // the products of all four tiles, also where none is needed: other waves
        // need all of theirs meanwhile
        f32x4 acc[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          acc[b] = zero4();
#pragma unroll
          for (int s = 0; s < KD / 32; ++s) {
            acc[b] = mfma16(ld_unit(unit_at<KD>(sm.y[Y], 16 * b + l16, 4 * s + quad)), xf[s], acc[b]);
          }
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          if (REV ? b < (a & 2) : b > (a | 1)) continue;
          const int block = (a >> 1) + (b >> 1), row = 16 * (a & 1) + l16, unit = 2 * (b & 1) + (quad >> 1);
          if (REV ? b < a : b > a) {   // the empty corner of a block on the diagonal
            const bf16x4 zero = {0, 0, 0, 0};
#pragma unroll
            for (int s = 0; s < PS; ++s) {
              *reinterpret_cast<bf16x4*>(p_unit(sm.p + s * kPartSize, block, row, unit) + 4 * (quad & 1)) = zero;
            }
            continue;
          }
          const f32x4 high_j = ld4(gates.high + 16 * b + 4 * quad), low_j = ld4(gates.low + 16 * b + 4 * quad);
          float w[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            // FP32's 24 bits also for kQuery's pairs, which are the gates' gradient
            const float e = power2<PS == 3 || MODE == kQuery>(REV ? high_j[r] - high : high - high_j[r],
                                                              REV ? low_j[r] - low : low - low_j[r]);
            const int j = 4 * quad + r;
            const bool keep = a != b || (REV ? j >= l16 : j <= l16);
            w[r] = keep ? acc[b][r] * e : 0.f;
          }
          if constexpr (MODE == kQuery) {
            // pairs (i, j < i): sums over j < t for every t <= i of the tile, then over i
            f32x4 m = zero4();
#pragma unroll
            for (int s = 0; s < VD / 32; ++s) {
              m = mfma16(ld_unit(unit_at<VD>(sm.z[Z], 16 * b + l16, 4 * s + quad)),
                         ld_unit(unit_at<VD>(sm.e, 16 * a + l16, 4 * s + quad)), m);
            }
            float pair[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) pair[r] = a != b || 4 * quad + r < l16 ? m[r] * w[r] : 0.f;
            float incl = (pair[0] + pair[1]) + (pair[2] + pair[3]);
            float y = __shfl_up(incl, 16);
            if (quad >= 1) incl += y;
            y = __shfl_up(incl, 32);
            if (quad >= 2) incl += y;
            y = __shfl_up(incl, 16);
            float sum = before + (quad >= 1 ? y : 0.f);
            before += __shfl(incl, 48 + l16);
            f32x4 column;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              column[r] = sum16(a != b || 4 * quad + r <= l16 ? sum : 0.f);
              sum += pair[r];
            }
            if (l16 == 0) st4(&sm.pairs[a][16 * b + 4 * quad], column);
          }
          float left[4] = {w[0], w[1], w[2], w[3]};
#pragma unroll
          for (int s = 0; s < PS; ++s) {
            u32x2 h;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              h[i] = pack_bf16(left[2 * i], left[2 * i + 1]);
              if (s + 1 < PS) minus(h[i], left[2 * i], left[2 * i + 1]);
            }
            *reinterpret_cast<u32x2*>(p_unit(sm.p + s * kPartSize, block, row, unit) + 4 * (quad & 1)) = h;
          }
        }
      }
      // through the state
#pragma unroll
      for (int ib = 0; ib < OT; ++ib) {
#pragma unroll
        for (int i = 0; i < CW * CW / 64; ++i) out[ib][i] = 0.f;
      }
#pragma unroll
      for (int u = 0; u < KD * CW / 512; ++u) {   // 16 rows of S in 32 x 32 tiles, 32 in 16 x 16
        float v[8];
        if constexpr (CW == 32) {
          tile_kslots(S[u / 2], u % 2, v);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v[j] = S[2 * u][j];
            v[4 + j] = S[2 * u + 1][j];
          }
        }
        bf16x8 part[SS];
        split_parts<SS>(v, part);
#pragma unroll
        for (int ib = 0; ib < OT; ++ib) {
          const int row = CW * ib + lcol;
          bf16x8 xf;
          if constexpr (CW == 32) {
            xf = ld_unit(unit_at<KD>(sm.x, row, 2 * u + half));
          } else {   // channels 4 quad .. 4 quad + 3 of both tiles
            const bf16x4 lo = ld_piece(unit_at<KD>(sm.x, row, 4 * u + (quad >> 1)) + 4 * (quad & 1));
            const bf16x4 hi = ld_piece(unit_at<KD>(sm.x, row, 4 * u + 2 + (quad >> 1)) + 4 * (quad & 1));
            xf = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
          }
#pragma unroll
          for (int n = 0; n < SS; ++n) out[ib] = product(part[n], xf, out[ib]);
        }
      }
#pragma unroll
      for (int ib = 0; ib < OT; ++ib) {
        const float high = gates.high[CW * ib + lcol], low = gates.low[CW * ib + lcol];
        const float w = power2<SS == 3>(REV ? gates.high[63] - high : high, REV ? gates.low[63] - low : low);
#pragma unroll
        for (int i = 0; i < CW * CW / 64; ++i) out[ib][i] *= w;
      }
      if constexpr (MODE == kQuery || MODE == kKey) {
        // q . (dq through the state), k . (dk through the state)
#pragma unroll
        for (int ib = 0; ib < OT; ++ib) {
          const int t = CW * ib + lcol;
          float dot = 0.f;
#pragma unroll
          for (int q = 0; q < CW * CW / 256; ++q) {
            bf16x4 v;
            if constexpr (MODE == kQuery) {
              const int ch = CW * wave + 8 * q + 4 * lrow;
              v = ld_piece(unit_at<VD>(sm.e, t, ch >> 3) + (ch & 4));
            } else {
              v = __builtin_bit_cast(bf16x4, key[CW * CW / 256 * ib + q]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) dot += static_cast<float>(v[j]) * out[ib][4 * q + j];
          }
          dot = t < valid ? dot : 0.f;
          if (CW == 16) dot += __shfl_xor(dot, 16);
          dot += __shfl_xor(dot, 32);
          if (lrow == 0) sm.dots[wave][t] = dot;
        }
      }
      // What passes by the chunk, e^{G_C} <cotangent after it, state before it>, is a
      // dot product of states at both ends of the fragment, where the other state is
      // in memory, and at its anchors, where both passes leave theirs for
      // linear_gate_kernel
      if (last) {
        const float* with = ends ? p.end_seq : p.end_piece;
        float dot = 0.f;
        if (with != nullptr) {
          with += (static_cast<int64_t>(ends ? seq : seg) * p.H + head) * size;
          const int at = opaque(col);   // its addresses are not kept over the chunks
          each_quad<CW>(S, opaque(lane), [&](f32x4& v, int row) {
            if (row >= p.KW || at >= p.VW) return;
            const f32x4 w = load_quad(p, with, row, at);
#pragma unroll
            for (int j = 0; j < 4; ++j) dot += v[j] * w[j];
          });
        }
        dot = sum64(dot);
        if (lane == 0) sm.by[wave] = dot;
      }
      if constexpr (MODE != kQuery) {   // z; y's copies may go on
        if (it + 1 < chunks) {
          copies_done<Copy<KD>::kSteps>();
        } else {
          copies_done<0>();
        }
      }
      block_sync();   // P, dots, pairs and z are whole
      start_x(it + 1);
      fetch_key(it + 1);
    }

    // z by columns: 16 tokens a product with 32 x 32 tiles, 32 with 16 x 16
    constexpr int ZT = CW / 8;
    bf16x8 zf[ZT];
#pragma unroll
    for (int s = 0; s < ZT; ++s) {
      if constexpr (CW == 32) {
        zf[s] = column_tokens<VD>(sm.z[Z], 16 * s + 8 * half, 32 * wave, reader);
      } else {
        zf[s] = column16_tokens<VD>(sm.z[Z], 32 * s + 8 * quad, 16 * wave, reader);
      }
    }
    if constexpr (kOut) {
#pragma unroll
      for (int ib = 0; ib < OT; ++ib) {
#pragma unroll
        for (int s = 0; s < ZT; ++s) {
          const int ob = CW == 32 ? ib : ib >> 1, jb = CW == 32 ? s >> 1 : s;   // blocks of 32 tokens
          if (REV ? jb < ob : jb > ob) continue;
#pragma unroll
          for (int n = 0; n < PS; ++n) {
            const bf16* part = sm.p + n * kPartSize;
            const bf16x8 pf = CW == 32
                ? ld_unit(p_unit(const_cast<bf16*>(part), ob + jb, reader & 31, 2 * (s & 1) + (reader >> 5)))
                : ld_unit(p_unit(const_cast<bf16*>(part), ob + jb, 16 * (ib & 1) + (reader & 15), reader >> 4));
            out[ib] = product(zf[s], pf, out[ib]);
          }
        }
      }
    }
    // the state after the chunk
    const float whole = gates.whole;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
#pragma unroll
      for (int i = 0; i < CW * CW / 64; ++i) S[kt][i] *= whole;
    }
#pragma unroll
    for (int s = 0; s < ZT; ++s) {
      const int t = 512 / CW * s + 8 * lrow;   // the first of the lane's eight tokens
      const u32x4 raw = __builtin_bit_cast(u32x4, zf[s]);
      const f32x4 w0 = ld4(gates.w_in + t), w1 = ld4(gates.w_in + t + 4);
      float v[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(raw[i] << 16) * (i < 2 ? w0[2 * i] : w1[2 * i - 4]);
        v[2 * i + 1] = __uint_as_float(raw[i] & 0xffff0000u) * (i < 2 ? w0[2 * i + 1] : w1[2 * i - 3]);
      }
      bf16x8 part[US];
      split_parts<US>(v, part);
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        const bf16x8 yf = CW == 32 ? slot_column_tokens<KD>(sm.y[Y], t, 32 * kt, reader)
                                   : column16_tokens<KD>(sm.y[Y], t, 16 * kt, reader);
#pragma unroll
        for (int n = 0; n < US; ++n) S[kt] = product(yf, part[n], S[kt]);
      }
    }
    if constexpr (kOut) {
      // the lane's place, in kQuery and kKey also made anew for each chunk
      const int writer = MODE == kOutput ? lane : opaque(lane), ocol = writer % CW, orow = writer / CW;
      const uint32_t at_o = ocol * o_row + (CW * wave + 4 * orow) * o_size;
      // Four stores in every case, which the copies' wait counts, and the compiler's
      // for what came through registers; FP32 has four more.
      const auto rows = buffer_of(static_cast<char*>(p.o) + (t0 * p.H + head) * p.VW * o_size,
                                  static_cast<int64_t>(valid) * o_row);
      const bool wide = p.o_fp32 != 0;
#pragma unroll
      for (int ib = 0; ib < OT; ++ib) {
        const uint32_t base = at_o + CW * ib * o_row;
        if constexpr (CW == 16) {
          const u32x4 raw = __builtin_bit_cast(u32x4, out[ib]);
          const uint32_t at = CW * wave + 4 * orow < p.VW ? base : kOutside;
          u32x2 v = {pack_bf16(out[ib][0], out[ib][1]), pack_bf16(out[ib][2], out[ib][3])};
#pragma unroll
          for (int j = 0; j < 2; ++j) v[j] = wide ? raw[j] : v[j];
          __builtin_amdgcn_raw_buffer_store_b64(v, rows, at, 0, 0);
          if (wide) __builtin_amdgcn_raw_buffer_store_b64(u32x2{raw[2], raw[3]}, rows, at + 8, 0, 0);
        } else {
#pragma unroll
          for (int q = 0; q < 4; q += 2) {
            f32x4 quads[2];
#pragma unroll
            for (int j = 0; j < 8; ++j) quads[j / 4][j % 4] = out[ib][4 * q + j];
            // channels 0 .. 7 of 16 to the lower half's lane of a token, 8 .. 15 to the upper's
            u32x2 lo = {pack_bf16(quads[0][0], quads[0][1]), pack_bf16(quads[1][0], quads[1][1])};
            u32x2 hi = {pack_bf16(quads[0][2], quads[0][3]), pack_bf16(quads[1][2], quads[1][3])};
            lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(lo[0], lo[1], false, false));
            hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(hi[0], hi[1], false, false));
            u32x4 v = {lo[0], hi[0], lo[1], hi[1]};
            const u32x4 raw = __builtin_bit_cast(u32x4, quads[0]);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = wide ? raw[j] : v[j];
            // the lane's first channel: four from there on, and four from eight on, or eight
            const int ch = 32 * wave + 8 * q + (wide ? 4 : 8) * orow;
            const uint32_t at = base + 8 * q * o_size + (wide ? 0 : 8 * orow);
            __builtin_amdgcn_raw_buffer_store_b128(v, rows, ch < p.VW ? at : kOutside, 0, 0);
            if (wide) {
              const uint32_t next = ch + 8 < p.VW ? at + 32 : kOutside;
              __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, quads[1]), rows, next, 0, 0);
            }
          }
        }
      }
    }
    if constexpr (MODE == kQuery || MODE == kKey) {
      if (it + 1 < chunks) measure(it + 1);
      if (wave == 0) {
        // kQuery's sums run from the chunk's end
        const int token = MODE == kQuery ? 63 - opaque(lane) : opaque(lane);
        float dot = sm.dots[0][token];
#pragma unroll
        for (int w = 1; w < 4; ++w) dot += sm.dots[w][token];
        const float sums = wave_prefix(dot), border = last_lane(sums);
        float part;
        if constexpr (MODE == kQuery) {
          // pairs across t in the chunk, and what the tokens from t on take from before it
          part = 0.f;
#pragma unroll
          for (int a = 0; a < 4; ++a) part += token < 16 * (a + 1) ? sm.pairs[a][token] : 0.f;
          part += sums;
        } else {
          // what the tokens before t give to after the chunk: the lane before's (lane 0: 0)
          part = from_lane<0x138, 0xf>(sums);
        }
        if (token < valid) p.gates.tokens[static_cast<int64_t>(head) * p.T + t0 + token] = part;
        if (lane == 0) {
          const int at = opaque(head);
          // less than 2^-63 an element of the state leaves no square: at most 2^-56 in all
          const float* squares = sm.squares[it & 1];
          const float norm = sqrtf((squares[0] + squares[1]) + (squares[2] + squares[3])) + 0x1p-56f;
          p.gates.border[(static_cast<int64_t>(begin / kLinearChunk) + f + c) * p.H + at] = f32x4{border, norm, gates.whole, 0.f};
          if (last) {
            float by = sm.by[0];
#pragma unroll
            for (int w = 1; w < 4; ++w) by += sm.by[w];
            p.gates.by[static_cast<int64_t>(f) * p.H + at] = gates.whole * by;
          }
        }
      }
    }
    if constexpr (MODE != kQuery) {   // the next x and y (kSummary: y, z), while this chunk's stores go on
      copies_done<kOut ? 4 : 0>();
      landed();
    }
  }

  float* to = !kOut ? p.piece_out + (static_cast<int64_t>(seg) * p.H + head) * size
                    : p.seq_out != nullptr && ends ? p.seq_out + (static_cast<int64_t>(seq) * p.H + head) * size : nullptr;
  if (to != nullptr) {
    each_quad<CW>(S, lane, [&](f32x4& v, int row) {
      if (row < p.KW && col < p.VW) store_quad(p, to, row, col, v);
    });
  }
  if (!kOut && p.decay_out != nullptr && tid == 0) {
    p.decay_out[static_cast<int64_t>(seg) * p.H + head] = power2(total);
  }
}

constexpr int kLinearThreads = 256;
template <int KD, int VD, int SS, int PS>
__global__ __launch_bounds__(kLinearThreads, 2) void linear_output_kernel(LinearParams p) {
  __shared__ LinearSmem<KD, VD, PS, kOutput> sm;
  linear_pass<KD, VD, SS, PS, false, kOutput>(p, sm);
}
// The pieces' updates, and beside them those of their cotangents.
template <int KD, int VD>
__global__ __launch_bounds__(kLinearThreads, 2) void linear_summary_kernel(LinearParams p, LinearParams other) {
  __shared__ LinearSmem<KD, VD, 1, kSummary> sm;
  linear_pass<KD, VD, 1, 1, false, kSummary>(blockIdx.y == 0 ? p : other, sm);
}
// The three gradients beside one another: while the last workgroups of one end, those
// of the next begin, and a few short sequences' fill the GPU together.
template <int KD, int VD, int PS>
__global__ __launch_bounds__(kLinearThreads, 2) void linear_grad_kernel(LinearParams query, LinearParams key,
                                                                        LinearParams value) {
  __shared__ union {
    LinearSmem<VD, KD, PS, kQuery> query;
    LinearSmem<VD, KD, PS, kKey> key;
    LinearSmem<KD, VD, PS, kOutput> value;
  } sm;
  if (blockIdx.y == 0) {
    linear_pass<VD, KD, 3, PS, false, kQuery>(query, sm.query);
  } else if (blockIdx.y == 1) {
    linear_pass<VD, KD, 3, PS, true, kKey>(key, sm.key);
  } else {
    linear_pass<KD, VD, PS, PS, true, kOutput>(value, sm.value);
  }
}
typedef void (*LinearGrad)(LinearParams, LinearParams, LinearParams);
// KD and VD by the widths in use.
template <int PS>
LinearGrad linear_grad_of(int32_t K, int32_t V) {
  if (K > 64) return V > 64 ? linear_grad_kernel<128, 128, PS> : linear_grad_kernel<128, 64, PS>;
  return V > 64 ? linear_grad_kernel<64, 128, PS> : linear_grad_kernel<64, 64, PS>;
}
LinearGrad linear_grad_bf16(int32_t K, int32_t V);   // kda_linear_grad.hip
LinearGrad linear_grad_fp32(int32_t K, int32_t V);   // kda_linear_grad32.hip

}  // namespace kda

#endif  // KDA_LINEAR_PASS_H_
