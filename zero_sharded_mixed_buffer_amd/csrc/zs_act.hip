// gfx950 kernels of the 8-bit activation checkpoints and of the root-mean-square norm with
// its backward pass (zs_act.h).
//
// All of them stream HBM.  A lane owns chunks of eight consecutive columns (one 16-byte
// access of 2-byte data, one 8-byte access of codes), so four neighbouring lanes hold a group
// of 32 that shares a scale, and its largest magnitude is two quad permutes away.  A row of
// the norm stays in the registers of the lanes that own it between the statistics and the
// outputs: every input is read once.

#include "zs_act_dev.h"

namespace zs {
namespace {

using namespace act;

// ------------------------------------------------------------------ pack, unpack

// Task t of a matrix is chunk t % chunks_per_row of row t / chunks_per_row; a workgroup takes U * 256
// consecutive ones.  One wide division per workgroup finds its first row, a 32-bit one per chunk
// the others; a matrix without gaps is one long row and needs neither.
struct Tasks {
  int64_t row0;
  uint32_t rem0, chunks_per_row;
  bool one;
  __device__ __forceinline__ Tasks(int64_t first, int64_t ntasks, uint32_t cpr) : chunks_per_row(cpr) {
    one = ntasks <= cpr;
    if (one)
      row0 = 0;
    else if (ntasks <= 0xFFFFFFFFll)
      row0 = static_cast<uint32_t>(first) / cpr;
    else
      row0 = first / cpr;
    rem0 = static_cast<uint32_t>(first - row0 * cpr);
  }
  __device__ __forceinline__ void at(uint32_t k, int64_t* row, uint32_t* chunk) const {
    const uint32_t r = rem0 + k;
    const uint32_t d = one ? 0 : r / chunks_per_row;
    *row = row0 + d;
    *chunk = r - d * chunks_per_row;
  }
};

__device__ __forceinline__ int clamp_count(int64_t left) { return left >= 8 ? 8 : left > 0 ? static_cast<int>(left) : 0; }

// Reads 2 (or 4) bytes and writes 1.03 per element; bound by memory: 16384 x 14336 bf16 to e4m3 in
// 110 us, 6.5 TB/s, where a plain copy runs at 6.1.
template <int DT, int CODE, int U>
__global__ __launch_bounds__(kThreads) void k_act_pack(const void* __restrict__ src, int64_t stride, int64_t cols,
                                                       uint32_t chunks_per_row, int64_t ntasks,
                                                       uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const int64_t first = int64_t(blockIdx.x) * (U * kThreads);
  const Tasks tasks(first, ntasks, chunks_per_row);
  float f[U][8];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t k = u * kThreads + threadIdx.x;
    int64_t row;
    uint32_t chunk;
    tasks.at(k, &row, &chunk);
    const int cnt = first + k < ntasks ? clamp_count(cols - int64_t(chunk) * 8) : 0;
    const int64_t e = row * stride + int64_t(chunk) * 8;
    if constexpr (DT == ZS_FP32) {
      const float* p = static_cast<const float*>(src) + e;
#pragma unroll
      for (int j = 0; j < 8; ++j) f[u][j] = 0.0f;
      if (cnt == 8) {
        const v4u a = *reinterpret_cast<const v4u_a4*>(p);
        const v4u b = *reinterpret_cast<const v4u_a4*>(p + 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f[u][j] = bits_f(a[j]);
          f[u][4 + j] = bits_f(b[j]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 7; ++j)
          if (j < cnt) f[u][j] = p[j];
      }
    } else {
      widen8<DT>(load8h_nt(static_cast<const uint16_t*>(src) + e, cnt), f[u]);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t t = first + u * kThreads + threadIdx.x;
    if (t < ntasks) encode_store<CODE>(f[u], codes, scales, t);
  }
}

// The way back: 1.03 bytes read and 2 (or 4) written per element, 116 us at the same size, 6.1 TB/s.
template <int DT, int CODE, int U>
__global__ __launch_bounds__(kThreads) void k_act_unpack(const uint8_t* __restrict__ codes,
                                                         const uint8_t* __restrict__ scales, int64_t cols,
                                                         uint32_t chunks_per_row, int64_t ntasks,
                                                         void* __restrict__ dst, int64_t stride) {
  const int64_t first = int64_t(blockIdx.x) * (U * kThreads);
  const Tasks tasks(first, ntasks, chunks_per_row);
  v2u c[U];
  int b[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t t = first + u * kThreads + threadIdx.x;
    c[u] = v2u{0u, 0u};
    b[u] = 0;
    if (t < ntasks) {
      c[u] = __builtin_nontemporal_load(reinterpret_cast<const v2u*>(codes) + t);
      b[u] = scales[t >> 2];
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t k = u * kThreads + threadIdx.x;
    int64_t row;
    uint32_t chunk;
    tasks.at(k, &row, &chunk);
    const int cnt = first + k < ntasks ? clamp_count(cols - int64_t(chunk) * 8) : 0;
    if (cnt == 0) continue;
    const int64_t e = row * stride + int64_t(chunk) * 8;
    float f[8];
    decode8<CODE>(c[u], scale_value(b[u]), f);
    if constexpr (DT == ZS_FP32) {
      float* p = static_cast<float*>(dst) + e;
      if (cnt == 8) {
        v4u lo, hi;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          lo[j] = f_bits(f[j]);
          hi[j] = f_bits(f[4 + j]);
        }
        __builtin_nontemporal_store(lo, reinterpret_cast<v4u_a4*>(p));
        __builtin_nontemporal_store(hi, reinterpret_cast<v4u_a4*>(p + 4));
      } else {
#pragma unroll
        for (int j = 0; j < 7; ++j)
          if (j < cnt) p[j] = f[j];
      }
    } else {
      clamp8<DT>(f);
      store8h(static_cast<uint16_t*>(dst) + e, narrow8<DT>(f), cnt);
    }
  }
}

// ------------------------------------------------------------------ norm

// The value of the lane `16 - N` places further in the lane's row of sixteen, going round.
template <int N>
__device__ __forceinline__ uint32_t rotate16(uint32_t x) {
  return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x120 + N, 0xF, 0xF, true));
}
template <int N>
__device__ __forceinline__ float rotate16(float x) {
  return bits_f(rotate16<N>(f_bits(x)));
}
template <int N>
__device__ __forceinline__ double rotate16(double x) {
  const v2u w = __builtin_bit_cast(v2u, x);
  return __builtin_bit_cast(double, v2u{rotate16<N>(w[0]), rotate16<N>(w[1])});
}

// Sum over the LPR lanes of a row, the same in every lane: rotations by 8, 4, 2 and 1 inside
// sixteen lanes (each adds the same pairs in all lanes), butterflies across the wave, then the
// waves' sums in index order through LDS.  `slot` is LDS of LPR / 64 values that no earlier sum
// still reads.
template <int LPR, typename T>
__device__ __forceinline__ T row_sum(T x, T* slot) {
  x += rotate16<8>(x);
  x += rotate16<4>(x);
  x += rotate16<2>(x);
  x += rotate16<1>(x);
  if constexpr (LPR >= 64) {
    x += __shfl_xor(x, 16, 64);
    x += __shfl_xor(x, 32, 64);
  }
  if constexpr (LPR > 64) {
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x % LPR >> 6] = x;
    __syncthreads();
    x = slot[0];
#pragma unroll
    for (int i = 1; i < LPR / 64; ++i) x += slot[i];
  }
  return x;
}

template <int LPR>
constexpr int norm_block() {
  return LPR > kThreads ? LPR : kThreads;
}
// The backward pass takes shorter rows several at once: fewer rounds where there is one workgroup,
// fewer partial sums where there are many (16384 x 2048: 45.7 us with two rows to a workgroup, 49.2
// with one and twice the workgroups).
template <int LPR>
constexpr int backward_block() {
  return LPR > 512 ? LPR : 512;
}

// LPR lanes share a row, V chunks each (LPR * V * 8 >= cols), and take R rows.  The sum of squares
// is taken in fp64: it neither overflows for any finite fp16 or bf16 row nor depends on the row's
// length, and costs 16 operations per 16 bytes of the row.  Bound by memory where rows are long
// (16384 x 4096, residual and every output: 110 us, 6.1 TB/s); rows of 128 columns come to 80 % of
// that (131072 of them: 17 us), where those sums take about half of the vector units' time.
template <int DT, int LPR, int V, int R>
__global__ __launch_bounds__(norm_block<LPR>()) void k_rmsnorm(NormArgs a) {
  constexpr int kRows = norm_block<LPR>() / LPR;
  __shared__ double slot[LPR > 64 ? LPR / 64 : 1];
  static_assert(R == 1 || LPR <= 64, "a workgroup's rows share one slot");
  const int lane = threadIdx.x % LPR;
  const int64_t row0 = int64_t(blockIdx.x) * (kRows * R) + threadIdx.x / LPR;
  const int64_t chunks = act_padded(a.cols) / 8;
  v4u hb[R][V];
#pragma unroll
  for (int q = 0; q < R; ++q) {
    const int64_t row = row0 + q * kRows;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int col = (v * LPR + lane) * 8;
      hb[q][v] = load8h_nt(a.x + row * a.x_stride + col, row < a.rows ? clamp_count(a.cols - col) : 0);
    }
  }
  if (a.residual != nullptr) {
    v4u rb[R][V];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const int64_t row = row0 + q * kRows;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int col = (v * LPR + lane) * 8;
        rb[q][v] = load8h_nt(a.residual + row * a.residual_stride + col, row < a.rows ? clamp_count(a.cols - col) : 0);
      }
    }
#pragma unroll
    for (int q = 0; q < R; ++q)
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          hb[q][v][j] = pair_bits<DT>(lo_f<DT>(hb[q][v][j]) + lo_f<DT>(rb[q][v][j]),
                                      hi_f<DT>(hb[q][v][j]) + hi_f<DT>(rb[q][v][j]));
  }
  double sum[R];
#pragma unroll
  for (int q = 0; q < R; ++q) {
    sum[q] = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float f[8];
      widen8<DT>(hb[q][v], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[q] += static_cast<double>(f[j]) * static_cast<double>(f[j]);
    }
    sum[q] = row_sum<LPR>(sum[q], slot);
  }
#pragma unroll
  for (int q = 0; q < R; ++q) {
    const int64_t row = row0 + q * kRows;
    if (row >= a.rows) break;
    const float rstd = static_cast<float>(1.0 / sqrt(sum[q] / a.cols + a.eps));
    if (a.rstd != nullptr && lane == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int chunk = v * LPR + lane;
      const int col = chunk * 8;
      if (chunk >= chunks) continue;  // whole groups of four lanes leave together
      const int cnt = clamp_count(a.cols - col);
      float f[8];
      widen8<DT>(hb[q][v], f);
      if (a.h != nullptr) store8h(a.h + row * a.h_stride + col, hb[q][v], cnt);
      if (a.h8.codes != nullptr) {
        if (a.h8.code == ZS_E4M3)
          encode_store<ZS_E4M3>(f, a.h8.codes, a.h8.scales, row * chunks + chunk);
        else
          encode_store<ZS_INT8>(f, a.h8.codes, a.h8.scales, row * chunks + chunk);
      }
      if (a.y == nullptr && a.y8.codes == nullptr) continue;
      float w[8];
      widen8<DT>(load8h(a.weight + col, cnt), w);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = f[j] * rstd * w[j];  // zeros behind the row, unless all of it is NaN
      if (a.y != nullptr) store8h(a.y + row * a.y_stride + col, narrow8<DT>(f), cnt);
      if (a.y8.codes != nullptr) {
        if (a.y8.code == ZS_E4M3)
          encode_store<ZS_E4M3>(f, a.y8.codes, a.y8.scales, row * chunks + chunk);
        else
          encode_store<ZS_INT8>(f, a.y8.codes, a.y8.scales, row * chunks + chunk);
      }
    }
  }
}

// ------------------------------------------------------------------ norm, backward

__device__ __forceinline__ float load_any(const void* p, int dt, int64_t i) {
  if (dt == ZS_FP32) return static_cast<const float*>(p)[i];
  const uint32_t b = static_cast<const uint16_t*>(p)[i];
  return dt == ZS_BF16 ? lo_f<ZS_BF16>(b) : lo_f<ZS_FP16>(b);
}
__device__ __forceinline__ void store_any(void* p, int dt, int64_t i, float x) {
  if (dt == ZS_FP32)
    static_cast<float*>(p)[i] = x;
  else
    static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(dt == ZS_BF16 ? half_bits<ZS_BF16>(x) : half_bits<ZS_FP16>(x));
}

// What the norm's backward reads as h: 16-bit values, or a checkpoint of either code.
enum Saved : int { kSaved16 = 0, kSavedE4m3 = 1, kSavedInt8 = 2 };

// Workgroup b takes rows b * kRows + sub, then every (gridDim.x * kRows)-th, and keeps the sums
// of dy * xh of its columns in registers over all of them; they leave as one row of
// `partials`, which k_dweight adds up in row order.  Bound by memory: sixteen waves to a CU keep
// enough loads in flight (at 16384 x 4096 from an e4m3 checkpoint 82 us with the fold, 5.7 TB/s;
// with the next row's loads issued a row ahead, at the price of registers, 87, and with 256
// threads of two chunks to a row 91).
template <int DT, int SAVED, int LPR, int V>
__global__ __launch_bounds__(backward_block<LPR>(), 4) void k_rmsnorm_backward(NormBackwardArgs a) {
  constexpr int kBlock = backward_block<LPR>();
  constexpr int kRows = kBlock / LPR;
  __shared__ float slot[2][kRows][LPR > 64 ? LPR / 64 : 1];
  __shared__ float fold[kRows > 1 ? kRows : 1][kRows > 1 ? LPR * V * 8 : 1];
  const int sub = threadIdx.x / LPR;
  const int lane = threadIdx.x % LPR;
  const int64_t chunks = act_padded(a.cols) / 8;
  v4u w[V];
  int width[V];
  float acc[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int col = (v * LPR + lane) * 8;
    width[v] = clamp_count(a.cols - col);
    w[v] = load8h(a.weight + col, width[v]);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[v][j] = 0.0f;
  }
  struct Row {
    v4u dy[V], dh[V];
    v4u h[SAVED == kSaved16 ? V : 1];
    v2u code[SAVED == kSaved16 ? 1 : V];
    int byte[V];
    float rstd;
  };
  auto load = [&](Row& r, int64_t row) {
    const bool live = row < a.rows;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int chunk = v * LPR + lane;
      const int cnt = live ? width[v] : 0;
      r.dy[v] = load8h_nt(a.dy + row * a.dy_stride + chunk * 8, cnt);
      if constexpr (SAVED == kSaved16) {
        r.h[v] = load8h_nt(a.h + row * a.h_stride + chunk * 8, cnt);
      } else {
        r.code[v] = v2u{0u, 0u};
        r.byte[v] = 0;
        if (cnt > 0) {
          r.code[v] = __builtin_nontemporal_load(reinterpret_cast<const v2u*>(a.h8.codes) + row * chunks + chunk);
          r.byte[v] = a.h8.scales[(row * chunks + chunk) >> 2];
        }
      }
      r.dh[v] = a.dh != nullptr ? load8h_nt(a.dh + row * a.dh_stride + chunk * 8, cnt) : v4u{0u, 0u, 0u, 0u};
    }
    r.rstd = live ? a.rstd[row] : 0.0f;
  };
  // xh, dy and weight of chunk v in fp32.  A checkpoint's scale is a power of two, so that it and
  // rstd make one factor with one rounding.  Columns past the end hold zeros everywhere; where a NaN
  // scale covers them, live columns of the group make the row NaN anyway.
  auto widen = [&](const Row& r, int v, float (&xh)[8], float (&d)[8], float (&g)[8]) {
    if constexpr (SAVED == kSaved16) {
      widen8<DT>(r.h[v], xh);
#pragma unroll
      for (int j = 0; j < 8; ++j) xh[j] *= r.rstd;
    } else {
      decode8<SAVED == kSavedE4m3 ? ZS_E4M3 : ZS_INT8>(r.code[v], scale_value(r.byte[v]) * r.rstd, xh);
    }
    widen8<DT>(r.dy[v], d);
    widen8<DT>(w[v], g);
  };
  int turn = 0;
  const int64_t step = int64_t(gridDim.x) * kRows;
  for (int64_t row0 = int64_t(blockIdx.x) * kRows; row0 < a.rows; row0 += step, turn ^= 1) {
    const int64_t row = row0 + sub;
    Row r;
    load(r, row);
    float dot = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float xh[8], d[8], g[8];
      widen(r, v, xh, d, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float t = d[j] * xh[j];
        dot += t * g[j];
        acc[v][j] += t;
      }
    }
    dot = row_sum<LPR>(dot, slot[turn][sub]);
    const float mean = dot / static_cast<float>(a.cols);
    if (row >= a.rows) continue;
    // The row waits for its mean in packed form: without this the compiler keeps the widened
    // values over the reduction, at two to three times the registers.
#pragma unroll
    for (int v = 0; v < V; ++v) {
      asm volatile("" : "+v"(r.dy[v]), "+v"(w[v]));
      if constexpr (SAVED == kSaved16)
        asm volatile("" : "+v"(r.h[v]));
      else
        asm volatile("" : "+v"(r.code[v]));
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (width[v] == 0) continue;
      float xh[8], d[8], g[8], out[8];
      widen(r, v, xh, d, g);
      widen8<DT>(r.dh[v], out);
#pragma unroll
      for (int j = 0; j < 8; ++j) out[j] += r.rstd * (d[j] * g[j] - xh[j] * mean);
      store8h(a.dx + row * a.dx_stride + (v * LPR + lane) * 8, narrow8<DT>(out), width[v]);
    }
  }
  if (a.dweight == nullptr) return;
  const int64_t pitch = (int64_t(a.cols) + 7) / 8 * 8;
  if constexpr (kRows > 1) {
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) fold[sub][(v * LPR + lane) * 8 + j] = acc[v][j];
    __syncthreads();
    for (int c = threadIdx.x; c < a.cols; c += kBlock) {
      float t = fold[0][c];
#pragma unroll
      for (int i = 1; i < kRows; ++i) t += fold[i][c];
      if (gridDim.x == 1)
        store_any(a.dweight, a.dweight_dt, c, t + (a.base != nullptr ? load_any(a.base, a.dweight_dt, c) : 0.0f));
      else
        a.partials[int64_t(blockIdx.x) * pitch + c] = t;
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int col = (v * LPR + lane) * 8;
      if (width[v] == 0) continue;
      if (gridDim.x == 1) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < width[v])
            store_any(a.dweight, a.dweight_dt, col + j,
                      acc[v][j] + (a.base != nullptr ? load_any(a.base, a.dweight_dt, col + j) : 0.0f));
      } else {
        v4u lo, hi;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          lo[j] = f_bits(acc[v][j]);
          hi[j] = f_bits(acc[v][4 + j]);
        }
        v4u* p = reinterpret_cast<v4u*>(a.partials + int64_t(blockIdx.x) * pitch + col);
        p[0] = lo;
        p[1] = hi;
      }
    }
  }
}

// dweight = base + the sum of `count` partial rows, in a fixed order: 32 threads share a
// column, each adding every 32nd row, then the sums in index order, in fp64.  512 rows of 4096
// take 4.7 us.
constexpr int kFoldCols = 32, kFoldSlices = 32;
__global__ __launch_bounds__(kFoldCols* kFoldSlices) void k_dweight(const float* __restrict__ partials, int64_t count,
                                                                     int64_t pitch, int32_t cols, void* dweight, int dt,
                                                                     const void* base) {
  __shared__ double part[kFoldSlices][kFoldCols];
  const int c = threadIdx.x % kFoldCols, slice = threadIdx.x / kFoldCols;
  const int64_t col = int64_t(blockIdx.x) * kFoldCols + c;
  double t = 0.0;
  if (col < cols) {
#pragma unroll 8
    for (int64_t i = slice; i < count; i += kFoldSlices) t += static_cast<double>(partials[i * pitch + col]);
  }
  part[slice][c] = t;
  __syncthreads();
  if (slice == 0 && col < cols) {
#pragma unroll
    for (int i = 1; i < kFoldSlices; ++i) t += part[i][c];
    if (base != nullptr) t += static_cast<double>(load_any(base, dt, col));
    store_any(dweight, dt, col, static_cast<float>(t));
  }
}

// ------------------------------------------------------------------ launch choices

// Four chunks to a thread keep enough loads in flight on their own; with fewer than eight
// workgroups to a CU that way, one chunk to a thread spreads the work (4097 x 1003 int8: pack
// 7.6 -> 5.7 us, unpack 7.2 -> 4.9).
constexpr int64_t kFewChunks = int64_t(8) * 256 * 4 * kThreads;

template <int DT, int CODE, int U>
hipError_t pack_launch(const void* src, int64_t stride, int64_t cols, uint32_t cpr, int64_t n, const Act& act,
                       hipStream_t s) {
  hipLaunchKernelGGL((k_act_pack<DT, CODE, U>), dim3(static_cast<unsigned>((n + U * kThreads - 1) / (U * kThreads))),
                     dim3(kThreads), 0, s, src, stride, cols, cpr, n, act.codes, act.scales);
  return hipGetLastError();
}
template <int DT, int CODE>
hipError_t pack_size(const void* src, int64_t stride, int64_t cols, uint32_t cpr, int64_t n, const Act& act,
                     hipStream_t s) {
  return n < kFewChunks ? pack_launch<DT, CODE, 1>(src, stride, cols, cpr, n, act, s)
                        : pack_launch<DT, CODE, 4>(src, stride, cols, cpr, n, act, s);
}
template <int DT>
hipError_t pack_code(const void* src, int64_t stride, int64_t cols, uint32_t cpr, int64_t n, const Act& act,
                     hipStream_t s) {
  return act.code == ZS_E4M3 ? pack_size<DT, ZS_E4M3>(src, stride, cols, cpr, n, act, s)
                             : pack_size<DT, ZS_INT8>(src, stride, cols, cpr, n, act, s);
}

template <int DT, int CODE, int U>
hipError_t unpack_launch(const Act& act, int64_t cols, uint32_t cpr, int64_t n, void* dst, int64_t stride,
                         hipStream_t s) {
  hipLaunchKernelGGL((k_act_unpack<DT, CODE, U>), dim3(static_cast<unsigned>((n + U * kThreads - 1) / (U * kThreads))),
                     dim3(kThreads), 0, s, act.codes, act.scales, cols, cpr, n, dst, stride);
  return hipGetLastError();
}
template <int DT, int CODE>
hipError_t unpack_size(const Act& act, int64_t cols, uint32_t cpr, int64_t n, void* dst, int64_t stride, hipStream_t s) {
  return n < kFewChunks ? unpack_launch<DT, CODE, 1>(act, cols, cpr, n, dst, stride, s)
                        : unpack_launch<DT, CODE, 4>(act, cols, cpr, n, dst, stride, s);
}
template <int DT>
hipError_t unpack_code(const Act& act, int64_t cols, uint32_t cpr, int64_t n, void* dst, int64_t stride, hipStream_t s) {
  return act.code == ZS_E4M3 ? unpack_size<DT, ZS_E4M3>(act, cols, cpr, n, dst, stride, s)
                             : unpack_size<DT, ZS_INT8>(act, cols, cpr, n, dst, stride, s);
}

// A matrix without gaps between its rows, whole groups to a row, is one row.
void one_row(int64_t stride, int64_t* rows, int64_t* cols) {
  if (*rows > 1 && stride == *cols && *cols % kActPad == 0 && *cols / 8 <= (int64_t(1) << 31) / *rows) {
    *cols *= *rows;
    *rows = 1;
  }
}

template <int DT, int LPR, int V, int R = 1>
hipError_t norm_launch(const NormArgs& a, hipStream_t s) {
  constexpr int kBlock = norm_block<LPR>();
  constexpr int kRows = kBlock / LPR * R;
  hipLaunchKernelGGL((k_rmsnorm<DT, LPR, V, R>), dim3(static_cast<unsigned>((a.rows + kRows - 1) / kRows)), dim3(kBlock), 0,
                     s, a);
  return hipGetLastError();
}

// Lanes and chunks to a row.  Rows of up to 512 columns leave a lane one chunk; with many of them
// it takes two rows, for more loads in flight (131072 x 128: 17.8 us against 18.5 with one row and
// 19.4 with four).  Up to 1024 columns a wave takes a row without a barrier (16384 x 1024: 16.6 us
// against 24.0 with a workgroup to a row, half its lanes idle) where the rows fill the card that way
// (777 x 1003: 6.2 us against 5.7).  From there a workgroup takes a row:
// of 256 threads with two chunks each, except that with a residual, whose outputs too are twice as
// many, rows enough and most of the threads busy, 512 threads with one chunk are faster (16384 rows,
// all outputs: 4096 columns 110.6 us against 117.5, 3584 99.0 against 100.3, 3200 89.6 against
// 91.0, but 2688 77.5 against 76.3; with 16-bit outputs alone 85.9 against 88.1, 76.5 against 77.0,
// 70.5 against 68.1, 62.5 against 57.5; 4096 columns without a residual 64.9 against 57.1, 2048 rows
// 16.7 against 14.2).
template <int DT>
hipError_t norm_cols(const NormArgs& a, hipStream_t s) {
  const bool many = a.rows >= 32768;
  if (a.cols <= 128) return many ? norm_launch<DT, 16, 1, 2>(a, s) : norm_launch<DT, 16, 1>(a, s);
  if (a.cols <= 512) return many ? norm_launch<DT, 64, 1, 2>(a, s) : norm_launch<DT, 64, 1>(a, s);
  if (a.cols <= 1024 && a.rows >= 4096) return norm_launch<DT, 64, 2>(a, s);
  if (a.cols <= 2048) return norm_launch<DT, 256, 1>(a, s);
  if (a.cols <= 4096)
    return a.residual != nullptr && a.rows >= 8192 && a.cols > 3200 ? norm_launch<DT, 512, 1>(a, s)
                                                                    : norm_launch<DT, 256, 2>(a, s);
  if (a.cols <= 8192) return norm_launch<DT, 512, 2>(a, s);
  return norm_launch<DT, 1024, 2>(a, s);
}

int norm_rows_per_block(int64_t cols) { return cols <= 128 ? norm_block<16>() / 16 : cols <= 1024 ? norm_block<64>() / 64 : 1; }
int backward_rows_per_block(int64_t cols) {
  return cols <= 128 ? backward_block<16>() / 16 : cols <= 1024 ? backward_block<64>() / 64 : cols <= 2048 ? 2 : 1;
}

template <int DT, int SAVED, int LPR, int V>
hipError_t backward_launch(const NormBackwardArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((k_rmsnorm_backward<DT, SAVED, LPR, V>), dim3(static_cast<unsigned>(rmsnorm_partials(a.rows, a.cols))),
                     dim3(backward_block<LPR>()), 0, s, a);
  return hipGetLastError();
}

template <int DT, int SAVED>
hipError_t backward_cols(const NormBackwardArgs& a, hipStream_t s) {
  if (a.cols <= 128) return backward_launch<DT, SAVED, 16, 1>(a, s);
  if (a.cols <= 512) return backward_launch<DT, SAVED, 64, 1>(a, s);
  if (a.cols <= 1024) return backward_launch<DT, SAVED, 64, 2>(a, s);
  if (a.cols <= 2048) return backward_launch<DT, SAVED, 256, 1>(a, s);
  if (a.cols <= 4096) return backward_launch<DT, SAVED, 512, 1>(a, s);
  if (a.cols <= 8192) return backward_launch<DT, SAVED, 512, 2>(a, s);
  return backward_launch<DT, SAVED, 1024, 2>(a, s);
}

template <int DT>
hipError_t backward_saved(const NormBackwardArgs& a, hipStream_t s) {
  if (a.h != nullptr) return backward_cols<DT, kSaved16>(a, s);
  if (a.h8.code == ZS_E4M3) return backward_cols<DT, kSavedE4m3>(a, s);
  return backward_cols<DT, kSavedInt8>(a, s);
}

}  // namespace

hipError_t launch_act_pack(const void* src, int dt, int64_t stride, int64_t rows, int64_t cols, const Act& act,
                           hipStream_t s) {
  one_row(stride, &rows, &cols);
  const uint32_t cpr = static_cast<uint32_t>(act_padded(cols) / 8);
  const int64_t n = rows * cpr;
  if (n == 0) return hipSuccess;
  if (dt == ZS_BF16) return pack_code<ZS_BF16>(src, stride, cols, cpr, n, act, s);
  if (dt == ZS_FP16) return pack_code<ZS_FP16>(src, stride, cols, cpr, n, act, s);
  return pack_code<ZS_FP32>(src, stride, cols, cpr, n, act, s);
}

hipError_t launch_act_unpack(const Act& act, int64_t rows, int64_t cols, void* dst, int dt, int64_t stride,
                             hipStream_t s) {
  one_row(stride, &rows, &cols);
  const uint32_t cpr = static_cast<uint32_t>(act_padded(cols) / 8);
  const int64_t n = rows * cpr;
  if (n == 0) return hipSuccess;
  if (dt == ZS_BF16) return unpack_code<ZS_BF16>(act, cols, cpr, n, dst, stride, s);
  if (dt == ZS_FP16) return unpack_code<ZS_FP16>(act, cols, cpr, n, dst, stride, s);
  return unpack_code<ZS_FP32>(act, cols, cpr, n, dst, stride, s);
}

hipError_t launch_rmsnorm(const NormArgs& a, int dt, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  return dt == ZS_BF16 ? norm_cols<ZS_BF16>(a, s) : norm_cols<ZS_FP16>(a, s);
}

int64_t rmsnorm_max_rows(int64_t cols) {
  const int threads = cols <= 2048 ? 256 : cols <= 8192 ? 512 : 1024;
  return ((int64_t(1) << 32) / threads - 1) * norm_rows_per_block(cols);
}

int64_t rmsnorm_partials(int64_t rows, int64_t cols) {
  const int per = backward_rows_per_block(cols);
  const int64_t steps = (rows + per - 1) / per;
  // Up to eight rounds one workgroup does alone, with no partial sums and no second launch.
  // Otherwise as many workgroups as bring sixteen waves to every CU: more only add partial sums
  // (16384 x 4096, eight waves to one: 82 us with 512, 85 with 1024; 2048 x 16384, sixteen: 52 with
  // 256, 59 with 512).
  if (steps <= 8) return 1;
  const int64_t most = cols > 8192 ? 256 : 512;
  return steps < most ? steps : most;
}

hipError_t launch_rmsnorm_backward(const NormBackwardArgs& a, int dt, hipStream_t s) {
  hipError_t e = dt == ZS_BF16 ? backward_saved<ZS_BF16>(a, s) : backward_saved<ZS_FP16>(a, s);
  const int64_t parts = rmsnorm_partials(a.rows, a.cols);
  if (e != hipSuccess || a.dweight == nullptr || parts == 1) return e;
  const int64_t pitch = (int64_t(a.cols) + 7) / 8 * 8;
  hipLaunchKernelGGL(k_dweight, dim3(static_cast<unsigned>((a.cols + kFoldCols - 1) / kFoldCols)),
                     dim3(kFoldCols * kFoldSlices), 0, s,
                     a.partials, parts, pitch, a.cols, a.dweight, a.dweight_dt, a.base);
  return hipGetLastError();
}

}  // namespace zs
