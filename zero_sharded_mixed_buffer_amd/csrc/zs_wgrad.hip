// gfx950 kernels of the weight gradient from an 8-bit checkpoint (zs_act_wgrad):
//   dw[n][k] = base[n][k] + sum over tokens t of dy[t][n] * x8[t][k]
// on the matrix cores.
//
// Both operands are stored token by token, so the sum runs along their slow axis: a lane of
// the matrix instruction needs consecutive tokens of one column.  Tiles are staged in LDS as
// they lie in memory (a row per token) and read back through gfx950's transposing LDS loads,
// four tokens of one column per lane and load.  The checkpoint's codes become 2-byte values
// on the way into LDS, once per workgroup instead of once per wave.
//
// Where there are enough tiles the operations bound it, 2 * rows * cols * outs: 8192 tokens, 4096 ->
// 14336 in 0.80 ms (1.20 PFLOP/s; 0.82 added to a bf16 base), 4096 -> 4096 in 0.22 ms (1.24).  In
// turn with these, the library's bf16 product takes 0.94 ms (1.02) and 0.23 ms (1.21) on the
// token-major operands that a backward pass has, 0.63 ms (1.53) and 0.17 ms (1.67) if both are
// transposed before it.  The matrix cores are busy 60 % of the time and LDS 46 %, at the 1.7 to 1.8
// GHz that the card holds under this load.  Codes in int8 need five vector instructions for two
// values where e4m3 has one: 0.89 ms with a base.  With few tokens the launch's start and end are
// most of it: 512 tokens, 4096 -> 14336 take 0.10 ms where the bytes take 0.04, 64 tokens 0.06.
//
// Where the tiles do not fill the last round of CUs, those of it are split over the tokens; each
// split leaves its fp32 sums in the workspace and k_wgrad_fold adds them in token order: no
// atomics, the same result from call to call.

#include <algorithm>
#include <type_traits>

#include "zs_act_dev.h"

namespace zs {
namespace {

using namespace act;

typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8hf __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) v4s lds_v4s;

template <int DT>
__device__ __forceinline__ v16f mfma(const v8s& a, const v8s& b, const v16f& c) {
  if constexpr (DT == ZS_BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8hf, a), __builtin_bit_cast(v8hf, b), c, 0, 0, 0);
}

// An infinity in either half of a pair of fp16 values becomes the largest number: code * s may lie
// up to one code step past it although the source did not.  NaN stays.
__device__ __forceinline__ uint32_t fp16_range(uint32_t x) {
  typedef _Float16 v2h __attribute__((ext_vector_type(2)));
  const v2h top = {static_cast<_Float16>(65504.0f), static_cast<_Float16>(65504.0f)};
  return __builtin_bit_cast(
      uint32_t, __builtin_elementwise_maximum(__builtin_elementwise_minimum(__builtin_bit_cast(v2h, x), top), -top));
}

// Sixteen codes under scale byte b as 2-byte values in memory order, each rounded once to nearest
// even.  gfx950 converts a pair of e4m3 codes with a power-of-two scale in one instruction, which
// takes the scale from the exponent field alone, 0 (2^-127) and 255 (NaN) included.  The rounding
// changes nothing in bf16 down to its smallest normal number (a code has four significant bits, or
// seven), nor in fp16 for values that were fp16 numbers.
template <int DT, int CODE>
__device__ __forceinline__ void values16(const v4u& c, int b, v4u& lo, v4u& hi) {
  if constexpr (CODE == ZS_E4M3) {
    const float s = bits_f(static_cast<uint32_t>(b) << 23);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t x, y;
      if constexpr (DT == ZS_BF16) {
        x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[j], s, false));
        y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[j], s, true));
      } else {
        x = fp16_range(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[j], s, false)));
        y = fp16_range(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[j], s, true)));
      }
      (j < 2 ? lo : hi)[2 * (j & 1)] = x;
      (j < 2 ? lo : hi)[2 * (j & 1) + 1] = y;
    }
  } else {
    float f[8];
    const float s = scale_value(b);
    decode8<CODE>(v2u{c[0], c[1]}, s, f);
    lo = narrow8<DT>(f);
    decode8<CODE>(v2u{c[2], c[3]}, s, f);
    hi = narrow8<DT>(f);
    if constexpr (DT == ZS_FP16) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        lo[j] = fp16_range(lo[j]);
        hi[j] = fp16_range(hi[j]);
      }
    }
  }
}

// A workgroup's tile: WN x WK waves, each FN x FK matrix instructions of 32 x 32; a stage holds
// T tokens of both operands, and there are two of them in LDS.  The four rows that a transposing
// load takes 64 bytes of must lie on different banks.  Either 64 bytes of padding behind each row
// do that (PAD), or the 64-byte blocks of row r change places by block ^ (r % 4), which takes no
// LDS but an address register for each instruction of the tile.
template <int WN_, int WK_, int FN_, int FK_, int T_, bool PAD_>
struct Tile {
  static constexpr bool kPad = PAD_;
  static constexpr int WN = WN_, WK = WK_, FN = FN_, FK = FK_, T = T_;
  static constexpr int kThreads = WN * WK * 64;
  static constexpr int kN = WN * FN * 32, kK = WK * FK * 32;  // columns of dy, and of x8
  static constexpr int kPitchN = kN * 2 + (kPad ? 64 : 0), kPitchK = kK * 2 + (kPad ? 64 : 0);
  static constexpr int kOperandN = kPitchN * T;
  static constexpr int kBuffer = kOperandN + kPitchK * T;
  static constexpr int kLoadsN = T * kN / 8 / kThreads;   // 16-byte loads per thread: dy
  static constexpr int kLoadsK = T * kK / 16 / kThreads;  // and codes
  // the epilogue's strips: 32 rows of one wave's columns, at a pitch that puts the two half waves
  // of an accumulator store on different banks
  static constexpr int kStripPitch = (FN > FK ? FN : FK) * 32 + 8;
  static constexpr int kStrips = WN * WK * 32 * kStripPitch * 4;
  static constexpr int kLds = 2 * kBuffer > kStrips ? 2 * kBuffer : kStrips;
  static_assert(kLoadsN * kThreads * 8 == T * kN && kLoadsK * kThreads * 16 == T * kK, "whole loads");
  static_assert(kLds <= 163840, "LDS of a CU");
  // a thread's rows of a stage are equal modulo 4, so that its blocks change places alike
  static_assert(kThreads / (kN / 8) % 4 == 0 && kThreads / (kK / 16) % 4 == 0, "rows of a load");
  // byte of column `at` (in bytes) in row `row` of an operand
  static __device__ __forceinline__ int place(int row, int pitch, int at) {
    return row * pitch + (kPad ? at : (at ^ ((row & 3) * 64)));
  }
};

struct WgradTask {
  int64_t t0, t1;  // tokens
  int64_t n0, k0;  // first columns of dy and x8
};

template <class TL>
struct Stage {
  v4u a[TL::kLoadsN];
  v4u b[TL::kLoadsK];
  int scale[TL::kLoadsK];
};

// Tokens t .. t + T - 1 of the two operands into registers; tokens past the task's read as zero.
// Whole stages take plain loads: a uniform base per load and a lane offset that never changes.
// Loads that begin past the last column are left out; one that begins before and ends behind it
// takes the elements behind a row of dy along (padding, or the next row: a stage with the last row
// does not come here), which reach columns of the tile that are never stored.
template <class TL>
struct Fetcher {
  static constexpr int kPerRowN = TL::kN / 8, kPerRowK = TL::kK / 16;         // loads of a row
  static constexpr int kRowsN = TL::kThreads / kPerRowN, kRowsK = TL::kThreads / kPerRowK;  // rows of a load
  const WgradArgs& g;
  const WgradTask& w;
  int64_t padded;
  uint32_t off_n, off_k;     // off_k / 32 is the scale's offset
  bool whole, any_n, any_k;  // the tile lies inside; this lane's loads begin inside
  int64_t last;              // the first token that no plain stage may hold

  __device__ __forceinline__ Fetcher(const WgradArgs& g_, const WgradTask& w_) : g(g_), w(w_) {
    const int rn = threadIdx.x / kPerRowN, rk = threadIdx.x / kPerRowK;
    padded = act_padded(g.cols);
    off_n = static_cast<uint32_t>(rn * g.dy_stride + (threadIdx.x % kPerRowN) * 8) * 2;
    off_k = static_cast<uint32_t>(rk * padded + (threadIdx.x % kPerRowK) * 16);
    whole = w.n0 + TL::kN <= g.outs && w.k0 + TL::kK <= padded;
    any_n = w.n0 + static_cast<int64_t>(threadIdx.x % kPerRowN) * 8 < g.outs;
    any_k = w.k0 + static_cast<int64_t>(threadIdx.x % kPerRowK) * 16 < padded;
    last = whole || w.t1 < g.rows ? w.t1 : g.rows - 1;
    if (g.dy_stride >= (1 << 24) || padded >= (1 << 24) || g.dy_stride < 8) last = 0;  // offsets of 32 bits
  }

  __device__ __forceinline__ void operator()(int64_t t, Stage<TL>& st) const {
    if (t + TL::T <= last) {
      const char* pn = reinterpret_cast<const char*>(g.dy + t * g.dy_stride + w.n0);
      const uint8_t* pk = g.x8.codes + t * padded + w.k0;
      const uint8_t* ps = g.x8.scales + (t * padded + w.k0) / kActGroup;
      if (whole || any_n) {
#pragma unroll
        for (int u = 0; u < TL::kLoadsN; ++u)
          st.a[u] = *reinterpret_cast<const v4u_a2*>(pn + u * kRowsN * g.dy_stride * 2 + off_n);
      }
      if (whole || any_k) {
#pragma unroll
        for (int u = 0; u < TL::kLoadsK; ++u) {
          st.b[u] = *reinterpret_cast<const v4u*>(pk + u * kRowsK * padded + off_k);
          st.scale[u] = ps[u * kRowsK * (padded / kActGroup) + off_k / kActGroup];
        }
      }
      return;
    }
    // the seldom way: its addresses are worked out here each time, not kept over the main loop
    int id = threadIdx.x;
    asm volatile("" : "+v"(id));
#pragma unroll
    for (int u = 0; u < TL::kLoadsN; ++u) {
      const int64_t row = t + u * kRowsN + id / kPerRowN, col = w.n0 + (id % kPerRowN) * 8;
      const int64_t left = row < w.t1 ? g.outs - col : 0;
      st.a[u] = load8h(g.dy + row * g.dy_stride + col, left >= 8 ? 8 : left > 0 ? static_cast<int>(left) : 0);
    }
#pragma unroll
    for (int u = 0; u < TL::kLoadsK; ++u) {
      const int64_t row = t + u * kRowsK + id / kPerRowK, col = w.k0 + (id % kPerRowK) * 16;
      st.b[u] = v4u{0u, 0u, 0u, 0u};
      st.scale[u] = 0;
      if (row < w.t1 && col < padded) {
        st.b[u] = *reinterpret_cast<const v4u*>(g.x8.codes + row * padded + col);
        st.scale[u] = g.x8.scales[(row * padded + col) / kActGroup];
      }
    }
  }
};

// Part `part` of `parts` of a stage into LDS.
template <int DT, int CODE, class TL>
__device__ __forceinline__ void stage_to_lds(const Stage<TL>& st, char* buf, int part, int parts) {
  constexpr int kPerRowN = TL::kN / 8, kPerRowK = TL::kK / 16;
  constexpr int kRowsN = TL::kThreads / kPerRowN, kRowsK = TL::kThreads / kPerRowK;
  char* pn = buf + TL::place(threadIdx.x / kPerRowN, TL::kPitchN, threadIdx.x % kPerRowN * 16);
  char* pk = buf + TL::kOperandN + TL::place(threadIdx.x / kPerRowK, TL::kPitchK, threadIdx.x % kPerRowK * 32);
#pragma unroll
  for (int u = 0; u < TL::kLoadsN; ++u)
    if (u % parts == part) *reinterpret_cast<v4u*>(pn + u * kRowsN * TL::kPitchN) = st.a[u];
#pragma unroll
  for (int u = 0; u < TL::kLoadsK; ++u) {
    if (u % parts != part) continue;
    v4u lo, hi;
    values16<DT, CODE>(st.b[u], st.scale[u], lo, hi);
    *reinterpret_cast<v4u*>(pk + u * kRowsK * TL::kPitchK) = lo;
    *reinterpret_cast<v4u*>(pk + u * kRowsK * TL::kPitchK + 16) = hi;
  }
}

// Eight tokens of column (lane & 31) for one matrix instruction: lanes 0 .. 31 take tokens
// 0 .. 7 of the sixteen, lanes 32 .. 63 tokens 8 .. 15.  In each transposing load sixteen lanes
// read four rows of sixteen columns, four columns to a lane, and receive four rows of their
// own column.  `p` is the lane's address for the first load.
template <int PITCH>
__device__ __forceinline__ v8s read_operand(const char* p) {
  const v4s x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p));
  const v4s y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p + 4 * PITCH));
  return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Work units of a launch: the first `direct` tiles each as one workgroup over all tokens, the
// others in `splits` workgroups each, over `per` tokens.
struct WgradGrid {
  int32_t tiles_n, tiles_k, direct, splits;
  int64_t per;
};

// Eight sums of one row of the output, from column col on, cnt of them inside: added to the base
// and rounded once.
template <int DT>
__device__ __forceinline__ void write8(const WgradArgs& g, int64_t row, int64_t col, int cnt, float (&f)[8]) {
  const int64_t at = row * g.dw_stride + col;
  if (g.dw_dt == ZS_FP32) {
    float* p = static_cast<float*>(g.dw) + at;
    const float* base = static_cast<const float*>(g.base);
    if (cnt == 8) {
      v4u lo, hi;
      if (base != nullptr) {
        const v4u x = *reinterpret_cast<const v4u_a4*>(base + at), y = *reinterpret_cast<const v4u_a4*>(base + at + 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f[j] += bits_f(x[j]);
          f[4 + j] += bits_f(y[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        lo[j] = f_bits(f[j]);
        hi[j] = f_bits(f[4 + j]);
      }
      *reinterpret_cast<v4u_a4*>(p) = lo;
      *reinterpret_cast<v4u_a4*>(p + 4) = hi;
    } else {
#pragma unroll
      for (int j = 0; j < 7; ++j)
        if (j < cnt) p[j] = f[j] + (base != nullptr ? base[at + j] : 0.0f);
    }
    return;
  }
  if (g.base != nullptr) {
    float x[8];
    widen8<DT>(load8h(static_cast<const uint16_t*>(g.base) + at, cnt), x);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] += x[j];
  }
  store8h(static_cast<uint16_t*>(g.dw) + at, narrow8<DT>(f), cnt);
}

template <int DT, int CODE, class TL>
__global__ __launch_bounds__(TL::kThreads, 2) void k_wgrad(WgradArgs g, WgradGrid gr) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  // one contiguous run of units per XCD, of the direct tiles and of the split ones, so that
  // neighbouring tiles share their operands in its L2
  const int tiles = gr.tiles_n * gr.tiles_k;
  int tile, split = -1;
  if (blockIdx.x < static_cast<unsigned>(gr.direct)) {  // a multiple of the XCDs
    tile = blockIdx.x % kXcds * (gr.direct / kXcds) + blockIdx.x / kXcds;
  } else {
    const int units = (tiles - gr.direct) * gr.splits;
    const int b = blockIdx.x - gr.direct;
    const int unit = b % kXcds * ((units + kXcds - 1) / kXcds) + b / kXcds;
    if (unit >= units) return;
    // all tiles of one split before the next: they share its tokens
    tile = gr.direct + unit % (tiles - gr.direct);
    split = unit / (tiles - gr.direct);
  }
  WgradTask w;
  w.t0 = split < 0 ? 0 : split * gr.per;
  w.t1 = split < 0 || w.t0 + gr.per > g.rows ? g.rows : w.t0 + gr.per;
  w.n0 = int64_t(tile / gr.tiles_k) * TL::kN;
  w.k0 = int64_t(tile % gr.tiles_k) * TL::kK;

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wn = wave / TL::WK * TL::FN * 32, wk = wave % TL::WK * TL::FK * 32;  // the wave's part of the tile
  // addresses of the lane's transposing loads within a buffer for each instruction of the wave's
  // part; with padding they differ by constants
  const int lane_row = (lane >> 5) * 8 + ((lane & 15) >> 2), lane_col = ((lane >> 4) & 1) * 16 + (lane & 3) * 4;
  int at_n[TL::FN], at_k[TL::FK];
#pragma unroll
  for (int i = 0; i < TL::FN; ++i)
    at_n[i] = TL::kPad && i > 0 ? at_n[0] + i * 64 : TL::place(lane_row, TL::kPitchN, (wn + i * 32 + lane_col) * 2);
#pragma unroll
  for (int j = 0; j < TL::FK; ++j)
    at_k[j] = TL::kPad && j > 0 ? at_k[0] + j * 64
                                : TL::kOperandN + TL::place(lane_row, TL::kPitchK, (wk + j * 32 + lane_col) * 2);

  v16f acc[TL::FN][TL::FK];
#pragma unroll
  for (int i = 0; i < TL::FN; ++i)
#pragma unroll
    for (int j = 0; j < TL::FK; ++j) acc[i][j] = v16f(0.0f);

  struct Operands {
    v8s a[TL::FN], b[TL::FK];
  };
  auto read = [&](Operands& f, const char* buf, int step) {
#pragma unroll
    for (int i = 0; i < TL::FN; ++i) f.a[i] = read_operand<TL::kPitchN>(buf + at_n[i] + step * 16 * TL::kPitchN);
#pragma unroll
    for (int j = 0; j < TL::FK; ++j) f.b[j] = read_operand<TL::kPitchK>(buf + at_k[j] + step * 16 * TL::kPitchK);
  };
  auto multiply = [&](const Operands& f, int from = 0, int to = TL::FN) {
#pragma unroll
    for (int i = from; i < to; ++i)
#pragma unroll
      for (int j = 0; j < TL::FK; ++j) acc[i][j] = mfma<DT>(f.a[i], f.b[j], acc[i][j]);
  };
  // Between two matrix instructions: a share of the next step's LDS reads, of the conversions and
  // of the LDS writes, so that the matrix cores do not wait for any of them.
  auto interleave = [&](auto matrix, auto reads) {
    constexpr int kM = decltype(matrix)::value, kReads = decltype(reads)::value;
#pragma unroll
    for (int m = 0; m < kM; ++m) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                        // matrix
      __builtin_amdgcn_sched_group_barrier(0x100, (kReads + kM - 1) / kM, 0);  // LDS reads
      __builtin_amdgcn_sched_group_barrier(0x002, 6, 0);                        // vector
      __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);                        // LDS writes
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  constexpr std::integral_constant<int, TL::FN * TL::FK> kAll{};
  constexpr std::integral_constant<int, TL::FN * TL::FK / 2> kHalf{};
  constexpr std::integral_constant<int, 2 * (TL::FN + TL::FK)> kReads{};
  constexpr std::integral_constant<int, 0> kNone{};
  // One barrier per stage.  While stage i is multiplied from one LDS buffer, stage i + 1 goes from
  // registers into the other, whose readers passed the barrier of stage i - 1, during the first
  // step; then stage i + 2 sets out from memory.  The operands of a step are read during the step
  // before, the first ones of the next stage after the barrier, during the last step.  (Operands
  // read two or three steps ahead, or two stages under way from memory, change neither tile's time
  // by more than 2 %: neither LDS nor memory latency is what is left.)
  constexpr int kSteps = TL::T / 16;
  static_assert(kSteps % 2 == 0, "the operand sets alternate");
  const Fetcher<TL> fetch(g, w);
  const int64_t stages = (w.t1 - w.t0 + TL::T - 1) / TL::T;
  if (stages > 0) {
    Stage<TL> st{};
    Operands f[2];
    fetch(w.t0, st);
    stage_to_lds<DT, CODE, TL>(st, lds, 0, 1);
    if (stages > 1) fetch(w.t0 + TL::T, st);
    __syncthreads();
    read(f[0], lds, 0);
    char* cur = lds;
    char* other = lds + TL::kBuffer;
    for (int64_t i = 0; i + 1 < stages; ++i) {
      // the first step, in halves: the conversions of one are done before those of the other begin
      read(f[1], cur, 1);
      multiply(f[0], 0, TL::FN / 2);
      stage_to_lds<DT, CODE, TL>(st, other, 0, 2);
      interleave(kHalf, kReads);
      multiply(f[0], TL::FN / 2, TL::FN);
      stage_to_lds<DT, CODE, TL>(st, other, 1, 2);
      interleave(kHalf, kNone);
      if (i + 2 < stages) fetch(w.t0 + (i + 2) * TL::T, st);
#pragma unroll
      for (int step = 1; step + 1 < kSteps; ++step) {
        read(f[(step + 1) & 1], cur, step + 1);
        multiply(f[step & 1]);
        interleave(kAll, kReads);
      }
      __syncthreads();
      read(f[0], other, 0);
      multiply(f[(kSteps - 1) & 1]);
      interleave(kAll, kReads);
      char* x = cur;
      cur = other;
      other = x;
    }
#pragma unroll
    for (int step = 0; step < kSteps; ++step) {
      if (step + 1 < kSteps) read(f[(step + 1) & 1], cur, step + 1);
      multiply(f[step & 1]);
      interleave(kAll, kReads);
    }
    __syncthreads();  // the strips below reuse the buffers
  }

  // The sums leave through LDS, a strip of 32 output rows of the wave at a time, so that a lane
  // stores eight consecutive elements of a row.  Accumulator r of a lane is row
  // 8 * (r / 4) + 4 * (lane / 32) + r % 4 (dy's column), column lane % 32 (x8's column).
  float* strip = reinterpret_cast<float*>(lds) + wave * 32 * TL::kStripPitch;
  const int64_t out_rows = g.in_major ? g.cols : g.outs, out_cols = g.in_major ? g.outs : g.cols;
  const int64_t row0 = g.in_major ? w.k0 : w.n0, col0 = g.in_major ? w.n0 : w.k0;
  const int wave_row = g.in_major ? wk : wn, wave_col = g.in_major ? wn : wk;
  const int tile_cols = g.in_major ? TL::kN : TL::kK;
  // a split leaves its whole tile, row by row, in the workspace
  float* part = nullptr;
  if (split >= 0 && gr.splits > 1) part = g.partials + (int64_t(tile - gr.direct) * gr.splits + split) * (TL::kN * TL::kK);
  auto leave = [&](int index, int groups) {  // rows of the strip, `groups` eights of columns to a row
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    for (int q = lane; q < 32 * groups; q += 64) {
      const int r = q / groups, c = q % groups * 8;
      const v4u x = *reinterpret_cast<const v4u*>(strip + r * TL::kStripPitch + c);
      const v4u y = *reinterpret_cast<const v4u*>(strip + r * TL::kStripPitch + c + 4);
      const int tr = wave_row + index * 32 + r, tc = wave_col + c;
      if (part != nullptr) {
        v4u* p = reinterpret_cast<v4u*>(part + tr * tile_cols + tc);
        p[0] = x;
        p[1] = y;
        continue;
      }
      const int64_t row = row0 + tr, col = col0 + tc, left = out_cols - col;
      if (row >= out_rows || left <= 0) continue;
      float f[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[j] = bits_f(x[j]);
        f[4 + j] = bits_f(y[j]);
      }
      write8<DT>(g, row, col, left >= 8 ? 8 : static_cast<int>(left), f);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  };
  if (g.in_major) {
#pragma unroll
    for (int j = 0; j < TL::FK; ++j) {
#pragma unroll
      for (int i = 0; i < TL::FN; ++i)
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
          v4u x;
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = f_bits(acc[i][j][r + e]);
          *reinterpret_cast<v4u*>(strip + (lane & 31) * TL::kStripPitch + i * 32 + 2 * r + 4 * (lane >> 5)) = x;
        }
      leave(j, TL::FN * 4);
    }
  } else {
#pragma unroll
    for (int i = 0; i < TL::FN; ++i) {
#pragma unroll
      for (int j = 0; j < TL::FK; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          strip[(8 * (r / 4) + 4 * (lane >> 5) + r % 4) * TL::kStripPitch + j * 32 + (lane & 31)] = acc[i][j][r];
      leave(i, TL::FK * 4);
    }
  }
}

// The split tiles of dw: base + the splits' sums in token order, added in fp32 as one long sum
// would be, rounded once.  A thread takes eight consecutive elements.  Bound by memory: 128 large
// tiles in two splits, added to a bf16 base, take 16 us.
template <int DT, class TL>
__global__ __launch_bounds__(kThreads) void k_wgrad_fold(WgradArgs g, WgradGrid gr) {
  constexpr int kArea = TL::kN * TL::kK, kBlocks = kArea / 8 / kThreads;
  const int tile = blockIdx.x / kBlocks, e = (blockIdx.x % kBlocks * kThreads + threadIdx.x) * 8;
  const int tile_cols = g.in_major ? TL::kN : TL::kK;
  const int64_t n0 = int64_t((gr.direct + tile) / gr.tiles_k) * TL::kN, k0 = int64_t((gr.direct + tile) % gr.tiles_k) * TL::kK;
  const int64_t row = (g.in_major ? k0 : n0) + e / tile_cols, col = (g.in_major ? n0 : k0) + e % tile_cols;
  const int64_t left = (g.in_major ? g.outs : g.cols) - col;
  if (row >= (g.in_major ? g.cols : g.outs) || left <= 0) return;
  const float* p = g.partials + int64_t(tile) * gr.splits * kArea + e;
  float f[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int s = 0; s < gr.splits; ++s) {
    const v4u x = *reinterpret_cast<const v4u*>(p + int64_t(s) * kArea), y = *reinterpret_cast<const v4u*>(p + int64_t(s) * kArea + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[j] += bits_f(x[j]);
      f[4 + j] += bits_f(y[j]);
    }
  }
  write8<DT>(g, row, col, left >= 8 ? 8 : static_cast<int>(left), f);
}

// ------------------------------------------------------------------ launch choices

// Both tiles take stages of 64 tokens.  The large one, one workgroup of eight waves to a CU, reads
// half as many operand bytes from L2 and LDS for each product: 8192 x 4096 -> 4096 in 218 us against
// 314.  The small one, two workgroups of four waves to a CU, serves outputs with few large tiles:
// 1024 x 1024 -> 4096 in 18 us against 33, 16384 x 1024 -> 1024 in 50 against 53.  Four waves of 4 x 4 instructions, with less LDS traffic still, were slower than
// eight of 4 x 2 (298 us against 270, both before the interleaving below was in place).
using SmallTile = Tile<2, 2, 2, 2, 64, false>;  // 128 x 128
using LargeTile = Tile<2, 4, 4, 2, 64, true>;   // 256 x 256

struct WgradChoice {
  bool large;
  WgradGrid grid;
  int64_t workspace;
};

// Time of a launch in microseconds as a function of the tile, the tiles done directly and the
// splits of the others, from what the kernels measure on MI355X (256 CUs): a stage of the large
// tile, one workgroup to a CU, and of the small one, one or two to a CU; the start and end of
// a workgroup; the partial sums and the launch that folds them.  Of fourteen sizes from 128 x 64 ->
// 256 to 8192 x 4096 -> 14336 its choice is within 3 % of the best of all tiles and splits on twelve,
// 6 % off at 16384 x 1024 -> 1024 (53.5 us, 50.2 are possible) and 20 % at 1024 x 1024 -> 1024 (19.9,
// 16.6).  The bytes of dw and base are the same for every choice and not in it, so that it is no
// estimate of a short batch's time.
template <class TL>
double launch_cost(int64_t tiles, int64_t direct, int64_t splits, int64_t stages) {
  auto rounds = [&](int64_t units, int64_t n) {
    if (TL::kN == 256) return double((units + 255) / 256) * (n * 1.65 + (splits > 1 ? 8.0 : 6.0));
    const int64_t full = units / 512, rest = units % 512;
    return full * (n * 1.22 + 4.0) + (rest == 0 ? 0.0 : rest <= 256 ? n * 0.74 + 4.0 : n * 1.22 + 4.0);
  };
  double t = direct > 0 ? rounds(direct, stages) : 0.0;
  if (tiles > direct) t += rounds((tiles - direct) * splits, (stages + splits - 1) / splits);
  if (splits > 1) t += 4.0 + double(tiles - direct) * splits * (TL::kN * TL::kK) * 4 / 6.0e6;
  return t;
}

template <class TL>
void consider(int64_t rows, int64_t cols, int64_t outs, WgradChoice* best, double* cost) {
  constexpr int64_t kSlots = TL::kN == 256 ? 256 : 512;
  const int64_t tn = (outs + TL::kN - 1) / TL::kN, tk = (cols + TL::kK - 1) / TL::kK, tiles = tn * tk;
  const int64_t stages = std::max<int64_t>(1, (rows + TL::T - 1) / TL::T);
  const int64_t whole = tiles / kSlots * kSlots;
  for (int64_t s = 1; s <= 64; ++s) {
    const int64_t per = (stages + s - 1) / s;
    if (s > 1 && per < 4) break;
    if ((stages + per - 1) / per != s) continue;
    for (const int64_t direct : {int64_t(0), whole}) {
      if (s == 1 && direct != 0) continue;
      if (s > 1 && (tiles - direct) * s > 4 * kSlots) continue;  // splitting more than that only adds sums
      const double t = launch_cost<TL>(tiles, direct, s, stages);
      if (t >= *cost) continue;
      *cost = t;
      best->large = TL::kN == 256;
      best->grid = {static_cast<int32_t>(tn), static_cast<int32_t>(tk), static_cast<int32_t>(direct), static_cast<int32_t>(s),
                    per * TL::T};
      best->workspace = s == 1 ? 16 : (tiles - direct) * s * (TL::kN * TL::kK) * int64_t(sizeof(float));
    }
  }
}

WgradChoice choose(int64_t rows, int64_t cols, int64_t outs) {
  WgradChoice c{};
  double cost = 1e30;
  consider<LargeTile>(rows, cols, outs, &c, &cost);
  consider<SmallTile>(rows, cols, outs, &c, &cost);
  return c;
}

template <int DT, int CODE, class TL>
hipError_t wgrad_launch(const WgradArgs& a, const WgradGrid& gr, hipStream_t s) {
  const int64_t rest = int64_t(gr.tiles_n) * gr.tiles_k - gr.direct;
  if (TL::kLds > 65536) {
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_wgrad<DT, CODE, TL>),
                                       hipFuncAttributeMaxDynamicSharedMemorySize, TL::kLds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((k_wgrad<DT, CODE, TL>),
                     dim3(static_cast<unsigned>(gr.direct + launch_units(rest * gr.splits, kXcdWhole))),
                     dim3(TL::kThreads), TL::kLds, s, a, gr);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || gr.splits == 1) return e;
  hipLaunchKernelGGL((k_wgrad_fold<DT, TL>), dim3(static_cast<unsigned>(rest * (TL::kN * TL::kK / 8 / kThreads))),
                     dim3(kThreads), 0, s, a, gr);
  return hipGetLastError();
}

template <int DT, int CODE>
hipError_t wgrad_size(const WgradArgs& a, const WgradChoice& c, hipStream_t s) {
  return c.large ? wgrad_launch<DT, CODE, LargeTile>(a, c.grid, s) : wgrad_launch<DT, CODE, SmallTile>(a, c.grid, s);
}

template <int DT>
hipError_t wgrad_code(const WgradArgs& a, hipStream_t s) {
  const WgradChoice c = choose(a.rows, a.cols, a.outs);
  return a.x8.code == ZS_E4M3 ? wgrad_size<DT, ZS_E4M3>(a, c, s) : wgrad_size<DT, ZS_INT8>(a, c, s);
}

}  // namespace

int64_t wgrad_workspace(int64_t rows, int64_t cols, int64_t outs) {
  // the most workgroups of 512 threads that one launch holds, counted in the smaller tile (the
  // sides are bounded first so that nothing overflows)
  constexpr int64_t kMaxUnits = (int64_t(1) << 23) - 64;
  if (cols > (int64_t(1) << 30) || outs > (int64_t(1) << 30)) return -1;
  if (((outs + 127) / 128) * ((cols + 127) / 128) > kMaxUnits) return -1;
  return choose(rows, cols, outs).workspace;
}

hipError_t launch_wgrad(const WgradArgs& a, hipStream_t s) {
  return a.dy_dt == ZS_BF16 ? wgrad_code<ZS_BF16>(a, s) : wgrad_code<ZS_FP16>(a, s);
}

}  // namespace zs
