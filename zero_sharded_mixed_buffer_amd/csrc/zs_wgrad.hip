// gfx950 kernels of the weight gradient from an 8-bit checkpoint (zs_act_wgrad):
//   dw[n][k] = base[n][k] + sum over tokens t of dy[t][n] * x8[t][k]
// on the matrix cores.
//
// Both operands are stored token by token, so the sum runs along their slow axis: a lane of
// the matrix instruction needs consecutive tokens of one column.  Tiles are staged in LDS as
// they lie in memory (a row per token) and read back through gfx950's transposing LDS loads,
// four tokens of one column per lane and load.  The checkpoint's codes become 2-byte values
// (code * 2^k, exact) on the way into LDS, once per workgroup instead of once per wave.
//
// When the output has few tiles the tokens are split over several workgroups per tile; each
// leaves its fp32 sums in the workspace and k_wgrad_fold adds them in token order: no
// atomics, the same result from call to call.

#include <algorithm>

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

// Sixteen codes under scale byte b as 2-byte values in memory order.
template <int DT, int CODE>
__device__ __forceinline__ void values16(const v4u& c, int b, v4u& lo, v4u& hi) {
  float f[8];
  const float s = scale_value(b);
  decode8<CODE>(v2u{c[0], c[1]}, s, f);
  clamp8<DT>(f);
  lo = narrow8<DT>(f);
  decode8<CODE>(v2u{c[2], c[3]}, s, f);
  clamp8<DT>(f);
  hi = narrow8<DT>(f);
}

// A workgroup's tile: WN x WK waves, each FN x FK matrix instructions of 32 x 32; a stage holds
// T tokens of both operands, and there are two of them in LDS.
template <int WN_, int WK_, int FN_, int FK_, int T_>
struct Tile {
  static constexpr int WN = WN_, WK = WK_, FN = FN_, FK = FK_, T = T_;
  static constexpr int kThreads = WN * WK * 64;
  static constexpr int kN = WN * FN * 32, kK = WK * FK * 32;  // columns of dy, and of x8
  // 64 bytes behind each row put the four rows of a transposing load on different banks
  static constexpr int kPitchN = kN * 2 + 64, kPitchK = kK * 2 + 64;
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

// Tokens t .. t + T - 1 of the two operands into registers; what lies past the tokens or columns
// of the task reads as zero, and its memory is not touched.
template <class TL>
__device__ __forceinline__ void fetch(const WgradArgs& g, const WgradTask& w, int64_t t, Stage<TL>& st) {
  const int64_t padded = act_padded(g.cols);
  constexpr int kPerRowN = TL::kN / 8, kPerRowK = TL::kK / 16;
  const bool inside = t + TL::T <= w.t1 && w.n0 + TL::kN <= g.outs && w.k0 + TL::kK <= padded;
#pragma unroll
  for (int u = 0; u < TL::kLoadsN; ++u) {
    const int i = u * TL::kThreads + threadIdx.x;
    const int64_t row = t + i / kPerRowN, col = w.n0 + (i % kPerRowN) * 8;
    const uint16_t* p = g.dy + row * g.dy_stride + col;
    if (inside) {
      st.a[u] = *reinterpret_cast<const v4u_a2*>(p);
    } else {
      const int64_t left = g.outs - col;
      st.a[u] = load8h(p, row < w.t1 ? (left >= 8 ? 8 : left > 0 ? static_cast<int>(left) : 0) : 0);
    }
  }
#pragma unroll
  for (int u = 0; u < TL::kLoadsK; ++u) {
    const int i = u * TL::kThreads + threadIdx.x;
    const int64_t row = t + i / kPerRowK, col = w.k0 + (i % kPerRowK) * 16;
    const int64_t at = row * padded + col;
    if (inside || (row < w.t1 && col < padded)) {
      st.b[u] = *reinterpret_cast<const v4u*>(g.x8.codes + at);
      st.scale[u] = g.x8.scales[at / kActGroup];
    } else {
      st.b[u] = v4u{0u, 0u, 0u, 0u};
      st.scale[u] = 0;
    }
  }
}

template <int DT, int CODE, class TL>
__device__ __forceinline__ void stage_to_lds(const Stage<TL>& st, char* buf) {
  constexpr int kPerRowN = TL::kN / 8, kPerRowK = TL::kK / 16;
#pragma unroll
  for (int u = 0; u < TL::kLoadsN; ++u) {
    const int i = u * TL::kThreads + threadIdx.x;
    *reinterpret_cast<v4u*>(buf + (i / kPerRowN) * TL::kPitchN + (i % kPerRowN) * 16) = st.a[u];
  }
#pragma unroll
  for (int u = 0; u < TL::kLoadsK; ++u) {
    const int i = u * TL::kThreads + threadIdx.x;
    v4u lo, hi;
    values16<DT, CODE>(st.b[u], st.scale[u], lo, hi);
    char* p = buf + TL::kOperandN + (i / kPerRowK) * TL::kPitchK + (i % kPerRowK) * 32;
    *reinterpret_cast<v4u*>(p) = lo;
    *reinterpret_cast<v4u*>(p + 16) = hi;
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

__device__ __forceinline__ float load_dw(const void* p, int dt, int64_t i) {
  if (dt == ZS_FP32) return static_cast<const float*>(p)[i];
  const uint32_t b = static_cast<const uint16_t*>(p)[i];
  return dt == ZS_BF16 ? lo_f<ZS_BF16>(b) : lo_f<ZS_FP16>(b);
}
__device__ __forceinline__ void store_dw(void* p, int dt, int64_t i, float x) {
  if (dt == ZS_FP32)
    static_cast<float*>(p)[i] = x;
  else
    static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(dt == ZS_BF16 ? half_bits<ZS_BF16>(x) : half_bits<ZS_FP16>(x));
}

struct WgradGrid {
  int32_t tiles_n, tiles_k, splits;
  int64_t per;     // tokens per split
  int64_t pitch;   // row pitch of the partial sums, in elements
};

// Eight sums of one row of the output, from column col on, cnt of them inside: added to the base
// and rounded once, or left in fp32 among the partial sums.
template <int DT>
__device__ __forceinline__ void write8(const WgradArgs& g, float* part, int64_t stride, int64_t row, int64_t col, int cnt,
                                       float (&f)[8]) {
  const int64_t at = row * stride + col;
  if (part != nullptr || g.dw_dt == ZS_FP32) {
    float* p = (part != nullptr ? part : static_cast<float*>(g.dw)) + at;
    const float* base = part != nullptr ? nullptr : static_cast<const float*>(g.base);
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
__global__ __launch_bounds__(TL::kThreads, TL::FN* TL::FK >= 16 ? 1 : 2) void k_wgrad(WgradArgs g, WgradGrid gr) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  // one contiguous run of tiles per XCD, so that neighbouring tiles share their operands in its L2
  const int64_t units = int64_t(gr.tiles_n) * gr.tiles_k * gr.splits;
  const int64_t per_xcd = (units + kXcds - 1) / kXcds;
  const int64_t unit = (blockIdx.x % kXcds) * per_xcd + blockIdx.x / kXcds;
  if (unit >= units) return;
  const int64_t tiles = int64_t(gr.tiles_n) * gr.tiles_k;
  const int64_t split = unit / tiles, tile = unit % tiles;
  WgradTask w;
  w.t0 = split * gr.per;
  w.t1 = w.t0 + gr.per < g.rows ? w.t0 + gr.per : g.rows;
  w.n0 = tile / gr.tiles_k * TL::kN;
  w.k0 = tile % gr.tiles_k * TL::kK;

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wn = wave / TL::WK * TL::FN * 32, wk = wave % TL::WK * TL::FK * 32;  // the wave's part of the tile
  // address of the lane's transposing loads within an operand
  const int lane_row = (lane >> 5) * 8 + ((lane & 15) >> 2), lane_col = ((lane >> 4) & 1) * 16 + (lane & 3) * 4;
  const int at_n = lane_row * TL::kPitchN + (wn + lane_col) * 2;
  const int at_k = TL::kOperandN + lane_row * TL::kPitchK + (wk + lane_col) * 2;

  v16f acc[TL::FN][TL::FK];
#pragma unroll
  for (int i = 0; i < TL::FN; ++i)
#pragma unroll
    for (int j = 0; j < TL::FK; ++j) acc[i][j] = v16f(0.0f);

  Stage<TL> st;
  int turn = 0;
  if (w.t0 < w.t1) {
    fetch<TL>(g, w, w.t0, st);
    stage_to_lds<DT, CODE, TL>(st, lds);
  }
  __syncthreads();
  for (int64_t t = w.t0; t < w.t1; t += TL::T, turn ^= 1) {
    const bool more = t + TL::T < w.t1;
    if (more) fetch<TL>(g, w, t + TL::T, st);
    const char* buf = lds + turn * TL::kBuffer;
#pragma unroll
    for (int s = 0; s < TL::T / 16; ++s) {
      v8s a[TL::FN], b[TL::FK];
#pragma unroll
      for (int i = 0; i < TL::FN; ++i) a[i] = read_operand<TL::kPitchN>(buf + at_n + s * 16 * TL::kPitchN + i * 64);
#pragma unroll
      for (int j = 0; j < TL::FK; ++j) b[j] = read_operand<TL::kPitchK>(buf + at_k + s * 16 * TL::kPitchK + j * 64);
#pragma unroll
      for (int i = 0; i < TL::FN; ++i)
#pragma unroll
        for (int j = 0; j < TL::FK; ++j) acc[i][j] = mfma<DT>(a[i], b[j], acc[i][j]);
    }
    if (more) stage_to_lds<DT, CODE, TL>(st, lds + (turn ^ 1) * TL::kBuffer);
    __syncthreads();
  }

  // The sums leave through LDS, a strip of 32 output rows of the wave at a time, so that a lane
  // stores eight consecutive elements of a row.  Accumulator r of a lane is row
  // 8 * (r / 4) + 4 * (lane / 32) + r % 4 (dy's column), column lane % 32 (x8's column).
  float* strip = reinterpret_cast<float*>(lds) + wave * 32 * TL::kStripPitch;
  const int64_t out_rows = g.in_major ? g.cols : g.outs, out_cols = g.in_major ? g.outs : g.cols;
  float* part = gr.splits > 1 ? g.partials + split * out_rows * gr.pitch : nullptr;
  const int64_t stride = part != nullptr ? gr.pitch : g.dw_stride;
  const int64_t row0 = g.in_major ? w.k0 + wk : w.n0 + wn, col0 = g.in_major ? w.n0 + wn : w.k0 + wk;
  auto leave = [&](int index, int groups) {  // rows of the strip, `groups` eights of columns to a row
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    for (int q = lane; q < 32 * groups; q += 64) {
      const int r = q / groups, c = q % groups * 8;
      const int64_t row = row0 + index * 32 + r, col = col0 + c;
      const int64_t left = out_cols - col;
      if (row >= out_rows || left <= 0) continue;
      float f[8];
      const v4u x = *reinterpret_cast<const v4u*>(strip + r * TL::kStripPitch + c);
      const v4u y = *reinterpret_cast<const v4u*>(strip + r * TL::kStripPitch + c + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[j] = bits_f(x[j]);
        f[4 + j] = bits_f(y[j]);
      }
      write8<DT>(g, part, stride, row, col, left >= 8 ? 8 : static_cast<int>(left), f);
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

// dw = base + the splits' sums in token order, added in fp32 as one long sum would be.
__global__ __launch_bounds__(kThreads) void k_wgrad_fold(const float* __restrict__ partials, int32_t splits, int64_t rows,
                                                         int64_t cols, int64_t pitch, void* dw, const void* base, int dt,
                                                         int64_t dw_stride) {
  const int64_t quads = pitch / 4;
  const int64_t q = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (q >= rows * quads) return;
  const int64_t row = q / quads, col = q % quads * 4;
  float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = 0; s < splits; ++s) {
    const v4u x = *reinterpret_cast<const v4u*>(partials + (s * rows + row) * pitch + col);
#pragma unroll
    for (int j = 0; j < 4; ++j) t[j] += bits_f(x[j]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (col + j >= cols) break;
    const int64_t at = row * dw_stride + col + j;
    store_dw(dw, dt, at, t[j] + (base != nullptr ? load_dw(base, dt, at) : 0.0f));
  }
}

// ------------------------------------------------------------------ launch choices

using SmallTile = Tile<2, 2, 2, 2, 32>;  // 128 x 128
#ifndef ZS_LARGE
#define ZS_LARGE 2, 2, 4, 4, 64
#endif
using LargeTile = Tile<ZS_LARGE>;  // 256 x 256
constexpr int64_t kMaxUnits = (int64_t(1) << 23) - 64;  // workgroups of 512 threads in one launch

struct WgradChoice {
  bool large;
  WgradGrid grid;
};

WgradChoice choose(int64_t rows, int64_t cols, int64_t outs) {
  WgradChoice c{};
  auto count = [&](int64_t sn, int64_t sk) { return ((outs + sn - 1) / sn) * ((cols + sk - 1) / sk); };
  c.large = count(LargeTile::kN, LargeTile::kK) >= 192 && rows >= 512;
  const int64_t sn = c.large ? LargeTile::kN : SmallTile::kN, sk = c.large ? LargeTile::kK : SmallTile::kK;
  const int64_t step = c.large ? LargeTile::T : SmallTile::T;
  const int64_t n = count(sn, sk);
  int64_t splits = 1;
  if (!c.large && n < 512) {
    splits = std::min<int64_t>(768 / n, rows / (8 * step));  // three workgroups per CU, at least eight stages each
    splits = std::max<int64_t>(splits, 1);
  }
  const int64_t steps = std::max<int64_t>(1, (rows + step - 1) / step);
  const int64_t per = (steps + splits - 1) / splits;
  c.grid.tiles_n = static_cast<int32_t>((outs + sn - 1) / sn);
  c.grid.tiles_k = static_cast<int32_t>((cols + sk - 1) / sk);
  c.grid.splits = static_cast<int32_t>((steps + per - 1) / per);
  c.grid.per = per * step;
  return c;
}

template <int DT, int CODE, class TL>
hipError_t wgrad_launch(const WgradArgs& a, const WgradGrid& gr, hipStream_t s) {
  const int64_t units = int64_t(gr.tiles_n) * gr.tiles_k * gr.splits;
  if (TL::kLds > 65536) {
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_wgrad<DT, CODE, TL>),
                                       hipFuncAttributeMaxDynamicSharedMemorySize, TL::kLds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((k_wgrad<DT, CODE, TL>), dim3(static_cast<unsigned>(launch_units(units, kXcdWhole))),
                     dim3(TL::kThreads), TL::kLds, s, a, gr);
  return hipGetLastError();
}

template <int DT, int CODE>
hipError_t wgrad_size(const WgradArgs& a, const WgradChoice& c, hipStream_t s) {
  return c.large ? wgrad_launch<DT, CODE, LargeTile>(a, c.grid, s) : wgrad_launch<DT, CODE, SmallTile>(a, c.grid, s);
}

template <int DT>
hipError_t wgrad_code(const WgradArgs& a, const WgradChoice& c, hipStream_t s) {
  return a.x8.code == ZS_E4M3 ? wgrad_size<DT, ZS_E4M3>(a, c, s) : wgrad_size<DT, ZS_INT8>(a, c, s);
}

int64_t fold_pitch(int64_t row) { return (row + 3) / 4 * 4; }

}  // namespace

int64_t wgrad_workspace(int64_t rows, int64_t cols, int64_t outs) {
  // 128 x 128 tiles are the most there can be (sides are bounded first so that nothing overflows)
  if (cols > (int64_t(1) << 30) || outs > (int64_t(1) << 30)) return -1;
  if (((outs + 127) / 128) * ((cols + 127) / 128) > kMaxUnits / 2) return -1;
  const WgradChoice c = choose(rows, cols, outs);
  if (c.grid.splits == 1) return 16;
  // either orientation of dw: its rows are padded to whole groups of four
  return int64_t(4) * c.grid.splits * std::max(outs * fold_pitch(cols), cols * fold_pitch(outs));
}

hipError_t launch_wgrad(const WgradArgs& a, hipStream_t s) {
  WgradChoice c = choose(a.rows, a.cols, a.outs);
  const int64_t dw_rows = a.in_major ? a.cols : a.outs, dw_cols = a.in_major ? a.outs : a.cols;
  c.grid.pitch = fold_pitch(dw_cols);
  hipError_t e = a.dy_dt == ZS_BF16 ? wgrad_code<ZS_BF16>(a, c, s) : wgrad_code<ZS_FP16>(a, c, s);
  if (e != hipSuccess || c.grid.splits == 1) return e;
  const int64_t n = dw_rows * (c.grid.pitch / 4);
  hipLaunchKernelGGL(k_wgrad_fold, dim3(static_cast<unsigned>((n + kThreads - 1) / kThreads)), dim3(kThreads), 0, s,
                     a.partials, c.grid.splits, dw_rows, dw_cols, c.grid.pitch, a.dw, a.base, a.dw_dt, a.dw_stride);
  return hipGetLastError();
}

}  // namespace zs
