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

// A workgroup's tile: four waves, two by two, each F x F matrix instructions of 32 x 32; a
// stage holds T tokens of both operands.
template <int F, int T>
struct Tile {
  static constexpr int kSide = 2 * F * 32;          // columns of dy, and of x8
  static constexpr int kTokens = T;
  // 64 bytes behind each row put the four rows of a transposing load on different banks
  static constexpr int kPitch = kSide * 2 + 64;
  static constexpr int kOperand = kPitch * T;
  static constexpr int kBuffer = 2 * kOperand;
  static constexpr int kLds = 2 * kBuffer;          // double-buffered
  static constexpr int kLoadsA = T * kSide / 8 / kThreads;   // 16-byte loads per thread: dy
  static constexpr int kLoadsB = T * kSide / 16 / kThreads;  // and codes
};

struct WgradTask {
  int64_t t0, t1;  // tokens
  int64_t n0, k0;  // first columns of dy and x8
};

template <int DT, class TL>
struct Stage {
  v4u a[TL::kLoadsA];
  v4u b[TL::kLoadsB];
  int scale[TL::kLoadsB];
};

// Tokens t .. t + kTokens - 1 of the two operands into registers; what lies past the tokens or
// columns of the task reads as zero, and its memory is not touched.
template <int DT, class TL>
__device__ __forceinline__ void fetch(const WgradArgs& g, const WgradTask& w, int64_t t, Stage<DT, TL>& st) {
  const int64_t padded = act_padded(g.cols);
  constexpr int kPerRowA = TL::kSide / 8, kPerRowB = TL::kSide / 16;
  const bool inside = t + TL::kTokens <= w.t1 && w.n0 + TL::kSide <= g.outs && w.k0 + TL::kSide <= padded;
#pragma unroll
  for (int u = 0; u < TL::kLoadsA; ++u) {
    const int i = u * kThreads + threadIdx.x;
    const int64_t row = t + i / kPerRowA, col = w.n0 + (i % kPerRowA) * 8;
    const uint16_t* p = g.dy + row * g.dy_stride + col;
    if (inside) {
      st.a[u] = *reinterpret_cast<const v4u_a2*>(p);
    } else {
      const int64_t left = g.outs - col;
      st.a[u] = load8h(p, row < w.t1 ? (left >= 8 ? 8 : left > 0 ? static_cast<int>(left) : 0) : 0);
    }
  }
#pragma unroll
  for (int u = 0; u < TL::kLoadsB; ++u) {
    const int i = u * kThreads + threadIdx.x;
    const int64_t row = t + i / kPerRowB, col = w.k0 + (i % kPerRowB) * 16;
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
__device__ __forceinline__ void stage_to_lds(const Stage<DT, TL>& st, char* buf) {
  constexpr int kPerRowA = TL::kSide / 8, kPerRowB = TL::kSide / 16;
#pragma unroll
  for (int u = 0; u < TL::kLoadsA; ++u) {
    const int i = u * kThreads + threadIdx.x;
    *reinterpret_cast<v4u*>(buf + (i / kPerRowA) * TL::kPitch + (i % kPerRowA) * 16) = st.a[u];
  }
#pragma unroll
  for (int u = 0; u < TL::kLoadsB; ++u) {
    const int i = u * kThreads + threadIdx.x;
    v4u lo, hi;
    values16<DT, CODE>(st.b[u], st.scale[u], lo, hi);
    char* p = buf + TL::kOperand + (i / kPerRowB) * TL::kPitch + (i % kPerRowB) * 32;
    *reinterpret_cast<v4u*>(p) = lo;
    *reinterpret_cast<v4u*>(p + 16) = hi;
  }
}

// Eight tokens of column (lane & 31) for one matrix instruction: lanes 0 .. 31 take tokens
// 0 .. 7 of the sixteen, lanes 32 .. 63 tokens 8 .. 15.  In each transposing load sixteen lanes
// read four rows of sixteen columns, four columns to a lane, and receive four rows of their
// own column.  `p` is the lane's address for the first load.
template <class TL>
__device__ __forceinline__ v8s read_operand(const char* p) {
  const v4s x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p));
  const v4s y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p + 4 * TL::kPitch));
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

template <int DT, int CODE, int F, int T>
__global__ __launch_bounds__(kThreads, F >= 4 ? 1 : 2) void k_wgrad(WgradArgs g, WgradGrid gr) {
  using TL = Tile<F, T>;
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
  w.n0 = tile / gr.tiles_k * TL::kSide;
  w.k0 = tile % gr.tiles_k * TL::kSide;

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wn = (wave >> 1) * F * 32, wk = (wave & 1) * F * 32;  // the wave's part of the tile
  // address of the lane's transposing loads within an operand
  const int lane_at = ((lane >> 5) * 8 + ((lane & 15) >> 2)) * TL::kPitch + (((lane >> 4) & 1) * 16 + (lane & 3) * 4) * 2;

  v16f acc[F][F];
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < F; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  Stage<DT, TL> st;
  int turn = 0;
  if (w.t0 < w.t1) {
    fetch<DT, TL>(g, w, w.t0, st);
    stage_to_lds<DT, CODE, TL>(st, lds);
  }
  __syncthreads();
  for (int64_t t = w.t0; t < w.t1; t += T, turn ^= 1) {
    const bool more = t + T < w.t1;
    if (more) fetch<DT, TL>(g, w, t + T, st);
    const char* buf = lds + turn * TL::kBuffer + lane_at;
#pragma unroll
    for (int s = 0; s < T / 16; ++s) {
      v8s a[F], b[F];
#pragma unroll
      for (int i = 0; i < F; ++i) {
        a[i] = read_operand<TL>(buf + s * 16 * TL::kPitch + (wn + i * 32) * 2);
        b[i] = read_operand<TL>(buf + TL::kOperand + s * 16 * TL::kPitch + (wk + i * 32) * 2);
      }
#pragma unroll
      for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j) acc[i][j] = mfma<DT>(a[i], b[j], acc[i][j]);
    }
    if (more) stage_to_lds<DT, CODE, TL>(st, lds + (turn ^ 1) * TL::kBuffer);
    __syncthreads();
  }

  // Accumulator r of a lane is row 8 * (r / 4) + 4 * (lane / 32) + r % 4, column lane % 32.
  const bool partial = gr.splits > 1;
  const int64_t stride = partial ? gr.pitch : g.dw_stride;
  float* part = g.partials + split * (g.in_major ? g.cols : g.outs) * gr.pitch;
#pragma unroll
  for (int i = 0; i < F; ++i) {
#pragma unroll
    for (int j = 0; j < F; ++j) {
      const int64_t k = w.k0 + wk + j * 32 + (lane & 31);
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int64_t n = w.n0 + wn + i * 32 + 8 * (r / 4) + 4 * (lane >> 5) + r % 4;
        if (n >= g.outs || k >= g.cols) continue;
        const int64_t at = g.in_major ? k * stride + n : n * stride + k;
        const float x = acc[i][j][r];
        if (partial)
          part[at] = x;
        else
          store_dw(g.dw, g.dw_dt, at, x + (g.base != nullptr ? load_dw(g.base, g.dw_dt, at) : 0.0f));
      }
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

constexpr int kF = 2, kT = 32;
constexpr int64_t kMaxUnits = (int64_t(1) << 24) - 64;  // workgroups of 256 threads in one launch

WgradGrid choose(int64_t rows, int64_t cols, int64_t outs) {
  WgradGrid c{};
  constexpr int64_t side = Tile<kF, kT>::kSide;
  const int64_t tn = (outs + side - 1) / side, tk = (cols + side - 1) / side, n = tn * tk;
  int64_t splits = 1;
  if (n < 512) {
    splits = std::min<int64_t>(768 / n, rows / (8 * kT));  // three workgroups per CU, at least eight stages each
    splits = std::max<int64_t>(splits, 1);
  }
  const int64_t steps = std::max<int64_t>(1, (rows + kT - 1) / kT);
  const int64_t per = (steps + splits - 1) / splits;
  c.tiles_n = static_cast<int32_t>(tn);
  c.tiles_k = static_cast<int32_t>(tk);
  c.splits = static_cast<int32_t>((steps + per - 1) / per);
  c.per = per * kT;
  return c;
}

template <int DT, int CODE, int F, int T>
hipError_t wgrad_launch(const WgradArgs& a, const WgradGrid& gr, hipStream_t s) {
  using TL = Tile<F, T>;
  const int64_t units = int64_t(gr.tiles_n) * gr.tiles_k * gr.splits;
  const void* fn = reinterpret_cast<const void*>(&k_wgrad<DT, CODE, F, T>);
  if (TL::kLds > 65536) {
    hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, TL::kLds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((k_wgrad<DT, CODE, F, T>), dim3(static_cast<unsigned>(launch_units(units, kXcdWhole))),
                     dim3(kThreads), TL::kLds, s, a, gr);
  return hipGetLastError();
}

template <int DT>
hipError_t wgrad_code(const WgradArgs& a, const WgradGrid& c, hipStream_t s) {
  return a.x8.code == ZS_E4M3 ? wgrad_launch<DT, ZS_E4M3, kF, kT>(a, c, s) : wgrad_launch<DT, ZS_INT8, kF, kT>(a, c, s);
}

int64_t fold_pitch(int64_t row) { return (row + 3) / 4 * 4; }

}  // namespace

int64_t wgrad_workspace(int64_t rows, int64_t cols, int64_t outs) {
  // 128 x 128 tiles are the most there can be (sides are bounded first so that nothing overflows)
  if (cols > (int64_t(1) << 30) || outs > (int64_t(1) << 30)) return -1;
  if (((outs + 127) / 128) * ((cols + 127) / 128) > kMaxUnits / 2) return -1;
  const WgradGrid c = choose(rows, cols, outs);
  if (c.splits == 1) return 16;
  // either orientation of dw: its rows are padded to whole groups of four
  return int64_t(4) * c.splits * std::max(outs * fold_pitch(cols), cols * fold_pitch(outs));
}

hipError_t launch_wgrad(const WgradArgs& a, hipStream_t s) {
  WgradGrid c = choose(a.rows, a.cols, a.outs);
  const int64_t dw_rows = a.in_major ? a.cols : a.outs, dw_cols = a.in_major ? a.outs : a.cols;
  c.pitch = fold_pitch(dw_cols);
  hipError_t e = a.dy_dt == ZS_BF16 ? wgrad_code<ZS_BF16>(a, c, s) : wgrad_code<ZS_FP16>(a, c, s);
  if (e != hipSuccess || c.splits == 1) return e;
  const int64_t n = dw_rows * (c.pitch / 4);
  hipLaunchKernelGGL(k_wgrad_fold, dim3(static_cast<unsigned>((n + kThreads - 1) / kThreads)), dim3(kThreads), 0, s,
                     a.partials, c.splits, dw_rows, dw_cols, c.pitch, a.dw, a.base, a.dw_dt, a.dw_stride);
  return hipGetLastError();
}

}  // namespace zs
