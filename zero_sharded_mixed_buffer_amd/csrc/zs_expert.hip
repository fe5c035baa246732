// gfx950 kernels of the way of tokens to their experts and back: the stable order of the choices by
// expert (zs_route), the rows in that order (zs_expert_gather), and the weighted sum of a token's
// rows with its backward pass (zs_expert_combine, zs_expert_combine_backward).

#include <algorithm>

#include "zs_act_dev.h"

namespace zs {
namespace {

using namespace act;

// ------------------------------------------------------------------ order by expert

// Bound by latency: 32 choices take 4 us in one launch, 32768 5 + 7 us in two (17 in three, with a
// launch for the sums of all chunks).
//
// A counting sort that keeps the order of equal keys.  A wave takes kWaveChunk consecutive choices,
// 64 at a time in order.  A choice's place is the number of choices of smaller experts, plus those of
// its own expert in workgroups, waves and rounds before it, plus the lanes before it in its round: no
// atomics.  Choices that name no expert count as expert E.
constexpr int kWaveChunk = 256, kRounds = kWaveChunk / 64;

__device__ __forceinline__ int expert_of(const void* ids, int id_bytes, int64_t i, int experts) {
  const int64_t v = id_bytes == 8 ? static_cast<const int64_t*>(ids)[i] : static_cast<const int32_t*>(ids)[i];
  return v >= 0 && v < experts ? static_cast<int>(v) : experts;
}

// A lane's keys in the wave's rounds, -1 behind the last choice.
__device__ __forceinline__ void load_keys(const RouteArgs& g, int64_t first, int (&key)[kRounds]) {
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const int64_t at = first + i * 64 + (threadIdx.x & 63);
    key[i] = at < g.slots ? expert_of(g.ids, g.id_bytes, at, g.experts) : -1;
  }
}

// Lanes with the same key, among those that have one.
__device__ __forceinline__ uint64_t same_key(int key, int bits) {
  uint64_t mask = __ballot(key >= 0);
  for (int b = 0; b < bits; ++b) {
    const uint64_t set = __ballot((key >> b) & 1);
    mask &= (key >> b) & 1 ? set : ~set;
  }
  return mask;
}

__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// counts[e] += this wave's choices of each expert.
__device__ __forceinline__ void count_wave(const RouteArgs& g, const int (&key)[kRounds], int* counts) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const uint64_t mask = same_key(key[i], g.bits);
    if (key[i] >= 0 && (mask >> lane) == 1) counts[key[i]] += __popcll(mask);  // the last lane of a key
    wave_fence();
  }
}

__global__ __launch_bounds__(256) void k_route_count(RouteArgs g) {
  extern __shared__ int counts[];  // four waves of experts + 1
  const int keys = g.experts + 1, wave = threadIdx.x >> 6;
  int key[kRounds];
  load_keys(g, int64_t(blockIdx.x) * kRouteChunk + wave * kWaveChunk, key);
  for (int i = threadIdx.x; i < 4 * keys; i += 256) counts[i] = 0;
  __syncthreads();
  count_wave(g, key, counts + wave * keys);
  __syncthreads();
  for (int e = threadIdx.x; e < keys; e += 256)
    g.counts[int64_t(blockIdx.x) * keys + e] = counts[e] + counts[keys + e] + counts[2 * keys + e] + counts[3 * keys + e];
}

// One workgroup to an expert: its counts become the choices before each chunk; totals[e] is their sum.
__global__ __launch_bounds__(256) void k_route_scan(RouteArgs g) {
  __shared__ int sums[4];
  const int keys = g.experts + 1, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int before = 0;
  for (int64_t c = 0; c < g.chunks; c += 256) {
    int* p = g.counts + (c + threadIdx.x) * keys + blockIdx.x;
    const int n = c + threadIdx.x < g.chunks ? *p : 0;
    int sum = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(sum, d);
      if (lane >= d) sum += o;
    }
    if (lane == 63) sums[wave] = sum;
    __syncthreads();
    int front = before;
    for (int w = 0; w < wave; ++w) front += sums[w];
    if (c + threadIdx.x < g.chunks) *p = front + sum - n;
    before += sums[0] + sums[1] + sums[2] + sums[3];
    __syncthreads();
  }
  if (threadIdx.x == 0) g.totals[blockIdx.x] = before;
}

// Where the counts of the workgroups before this one come from: there is none (kAlone), from all
// workgroups' counts, which each adds up for itself (kFew), or from k_route_scan (kMany).
enum RouteWay { kAlone, kFew, kMany };
constexpr int64_t kFewChunks = 64;  // 65536 choices; what kFew adds up for itself then costs as much as the launch of a scan

template <RouteWay WAY, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void k_route_place(RouteArgs g) {
  extern __shared__ int counts[];  // waves of experts + 1, then the experts' first places, then the choices before this workgroup
  const int keys = g.experts + 1, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int* starts = counts + WAVES * keys;
  int* fronts = starts + keys;
  const int64_t first = int64_t(blockIdx.x) * (WAVES * kWaveChunk) + wave * kWaveChunk;
  int key[kRounds];
  load_keys(g, first, key);
  for (int i = threadIdx.x; i < WAVES * keys; i += WAVES * 64) counts[i] = 0;
  __syncthreads();
  count_wave(g, key, counts + wave * keys);
  __syncthreads();
  for (int e = threadIdx.x; e < keys; e += WAVES * 64) {  // this expert's choices in all, and before this workgroup
    int all = 0, front = 0;
    if constexpr (WAY == kAlone) {
      for (int w = 0; w < WAVES; ++w) all += counts[w * keys + e];
    } else if constexpr (WAY == kFew) {
#pragma unroll 8
      for (int c = 0; c < static_cast<int>(g.chunks); ++c) {
        const int n = g.counts[c * keys + e];
        all += n;
        if (c < static_cast<int>(blockIdx.x)) front += n;
      }
    } else {
      all = g.totals[e];
      front = g.counts[int64_t(blockIdx.x) * keys + e];
    }
    starts[e] = all;
    fronts[e] = front;
  }
  __syncthreads();
  if (wave == 0) {  // places before each expert
    int before = 0;
    for (int c = 0; c < keys; c += 64) {
      const int e = c + lane;
      const int n = e < keys ? starts[e] : 0;
      int sum = n;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(sum, d);
        if (lane >= d) sum += o;
      }
      if (e < keys) starts[e] = before + sum - n;
      if (blockIdx.x == 0 && e < g.experts) g.ends[e] = before + sum;
      before += __shfl(sum, 63);
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < keys; e += WAVES * 64) {
    int at = starts[e] + fronts[e];
    for (int w = 0; w < WAVES; ++w) {
      const int n = counts[w * keys + e];
      counts[w * keys + e] = at;
      at += n;
    }
  }
  __syncthreads();
  int* next = counts + wave * keys;
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const int64_t at = first + i * 64 + lane;
    const bool part = key[i] >= 0;
    const uint64_t mask = same_key(key[i], g.bits);
    const int place = part ? next[key[i]] + __popcll(mask & ((uint64_t(1) << lane) - 1)) : 0;
    wave_fence();
    if (part && (mask >> lane) == 1) next[key[i]] = place + 1;
    wave_fence();
    if (part) {
      const int slot = static_cast<int>(at);
      g.place[at] = key[i] < g.experts ? place : -1;
      g.slot[place] = key[i] < g.experts ? slot : -1 - slot;
    }
  }
}

// ------------------------------------------------------------------ rows

// Rows are moved 16 bytes to a lane (8 or 4 elements); a row's last piece may be short.  At any
// alignment.
template <int SIZE>
__device__ __forceinline__ v4u load_piece(const char* p, int64_t left) {  // left: elements from p on
  constexpr int kElems = 16 / SIZE;
  if (left >= kElems) return *reinterpret_cast<const v4u_a2*>(p);
  if constexpr (SIZE == 2) return load8h(reinterpret_cast<const uint16_t*>(p), static_cast<int>(left));
  v4u w = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int j = 0; j < 3; ++j)
    if (j < left) w[j] = reinterpret_cast<const uint32_t*>(p)[j];
  return w;
}
template <int SIZE>
__device__ __forceinline__ void store_piece(char* p, const v4u& w, int64_t left) {
  constexpr int kElems = 16 / SIZE;
  if (left >= kElems) {
    __builtin_nontemporal_store(w, reinterpret_cast<v4u_a2*>(p));
    return;
  }
  if constexpr (SIZE == 2) {
#pragma unroll
    for (int j = 0; j < 7; ++j)
      if (j < left) reinterpret_cast<uint16_t*>(p)[j] = static_cast<uint16_t>(w[j >> 1] >> ((j & 1) * 16));
  } else {
#pragma unroll
    for (int j = 0; j < 3; ++j)
      if (j < left) reinterpret_cast<uint32_t*>(p)[j] = w[j];
  }
}

template <int DT>
struct Piece {
  static constexpr int kSize = DT == ZS_FP32 ? 4 : 2, kElems = 16 / kSize;
  static __device__ __forceinline__ void widen(const v4u& w, float* f) {
    if constexpr (DT == ZS_FP32) {
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = bits_f(w[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[2 * j] = lo_f<DT>(w[j]);
        f[2 * j + 1] = hi_f<DT>(w[j]);
      }
    }
  }
  static __device__ __forceinline__ v4u narrow(const float* f) {
    v4u w;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = DT == ZS_FP32 ? f_bits(f[j]) : pair_bits<DT>(f[2 * j % kElems], f[(2 * j + 1) % kElems]);
    return w;
  }
};

// Bound by memory.  16384 x 4096 to two rows each: the gather takes 75 us (5.3 TB/s), the combination 67
// (6.0), its backward 122 (5.5).  Rows are written past the caches: through them 82, 76 and 128.
//
// A lane's next kAhead pieces of a row, loaded together: a load's latency, not its bytes, is what a
// short row costs.  Four instead of two were slower (routing and gather 109 us against 103).
constexpr int kAhead = 2;

// out[p] = x[slot[p] / choices], zeros where the slot names no choice of an expert.  A workgroup
// takes 1 << rows_log2 rows, as many lanes to each.
template <int SIZE>
__global__ __launch_bounds__(256) void k_gather(RowsArgs g) {
  constexpr int kElems = 16 / SIZE;
  const int per = 256 >> g.rows_log2;
  const int64_t p = (int64_t(blockIdx.x) << g.rows_log2) + threadIdx.x / per;
  if (p >= g.rows) return;
  const int slot = g.slot[p];
  const bool any = slot >= 0 && slot < g.rows;
  const char* src = static_cast<const char*>(g.x) + (any ? int64_t(slot / g.choices) * g.x_stride * SIZE : 0);
  char* dst = static_cast<char*>(g.out) + p * g.out_stride * SIZE;
  const int64_t step = int64_t(per) * kElems;
  for (int64_t c = int64_t(threadIdx.x % per) * kElems; c < g.cols; c += kAhead * step) {
    v4u w[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      w[u] = v4u{0u, 0u, 0u, 0u};
      if (any && c + u * step < g.cols) w[u] = load_piece<SIZE>(src + (c + u * step) * SIZE, g.cols - c - u * step);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (c + u * step < g.cols) store_piece<SIZE>(dst + (c + u * step) * SIZE, w[u], g.cols - c - u * step);
  }
}

// out[t] = sum over j of weights[t][j] * y[place[t][j]], in order of j, in fp32, rounded once.
template <int DT>
__global__ __launch_bounds__(256) void k_combine(RowsArgs g) {
  using P = Piece<DT>;
  const int per = 256 >> g.rows_log2;
  const int64_t t = (int64_t(blockIdx.x) << g.rows_log2) + threadIdx.x / per;
  if (t >= g.rows / g.choices) return;
  const int32_t* place = g.place + t * g.choices;
  const float* weights = g.weights != nullptr ? g.weights + t * g.choices : nullptr;
  const int64_t step = int64_t(per) * P::kElems;
  for (int64_t c = int64_t(threadIdx.x % per) * P::kElems; c < g.cols; c += kAhead * step) {
    float sum[kAhead][P::kElems];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int i = 0; i < P::kElems; ++i) sum[u][i] = 0.0f;
#pragma unroll 2
    for (int j = 0; j < g.choices; ++j) {
      const int p = place[j];
      if (p < 0 || p >= g.rows) continue;
      const float w = weights != nullptr ? weights[j] : 1.0f;
      const char* y = static_cast<const char*>(g.x) + (int64_t(p) * g.x_stride + c) * P::kSize;
      v4u v[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        v[u] = v4u{0u, 0u, 0u, 0u};
        if (c + u * step < g.cols) v[u] = load_piece<P::kSize>(y + u * step * P::kSize, g.cols - c - u * step);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        float f[P::kElems];
        P::widen(v[u], f);
#pragma unroll
        for (int i = 0; i < P::kElems; ++i) sum[u][i] += w * f[i];
      }
    }
    char* out = static_cast<char*>(g.out) + (t * g.out_stride + c) * P::kSize;
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (c + u * step < g.cols) store_piece<P::kSize>(out + u * step * P::kSize, P::narrow(sum[u]), g.cols - c - u * step);
  }
}

// For each token t and its choice j in row p = place[t][j]: dy[p] = weights[t][j] * dout[t],
// dweights[t][j] = sum over columns of dout[t] * y[p].  By tokens, so that dout is read from memory
// once and from the caches for the other choices; the token also clears those of its choices' worth
// of rows that hold no expert's choice.
template <int DT>
__global__ __launch_bounds__(256) void k_combine_backward(CombineBackwardArgs g) {
  using P = Piece<DT>;
  const int per = 256 >> g.rows_log2;
  const int64_t t = (int64_t(blockIdx.x) << g.rows_log2) + threadIdx.x / per;
  const int in_row = threadIdx.x % per;
  __shared__ float sums[4];
  const bool here = t * g.choices < g.rows;
  const int64_t step = int64_t(per) * P::kElems;
  const char* dout = static_cast<const char*>(g.dout) + (here ? t : 0) * g.dout_stride * P::kSize;
  for (int j = 0; j < g.choices; ++j) {
    const int64_t s = t * g.choices + j;
    int p = here ? g.place[s] : -1;
    const bool any = p >= 0 && p < g.rows;
    const float w = any && g.weights != nullptr ? g.weights[s] : 1.0f;
    float dot = 0.0f;
    if (any) {
      const char* y = static_cast<const char*>(g.y) + int64_t(p) * g.y_stride * P::kSize;
      char* dy = g.dy != nullptr ? static_cast<char*>(g.dy) + int64_t(p) * g.dy_stride * P::kSize : nullptr;
      for (int64_t c = int64_t(in_row) * P::kElems; c < g.cols; c += kAhead * step) {
        v4u a[kAhead], b[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          a[u] = b[u] = v4u{0u, 0u, 0u, 0u};
          const int64_t at = c + u * step;
          if (at < g.cols) {
            a[u] = load_piece<P::kSize>(dout + at * P::kSize, g.cols - at);
            if (g.dweights != nullptr) b[u] = load_piece<P::kSize>(y + at * P::kSize, g.cols - at);
          }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int64_t at = c + u * step;
          float d[P::kElems], f[P::kElems];
          P::widen(a[u], d);
          P::widen(b[u], f);
#pragma unroll
          for (int i = 0; i < P::kElems; ++i) {
            dot += d[i] * f[i];
            d[i] *= w;
          }
          if (dy != nullptr && at < g.cols) store_piece<P::kSize>(dy + at * P::kSize, P::narrow(d), g.cols - at);
        }
      }
    }
    if (g.dy != nullptr && here && g.slot[s] < 0) {
      char* dy = static_cast<char*>(g.dy) + s * g.dy_stride * P::kSize;
      for (int64_t c = int64_t(in_row) * P::kElems; c < g.cols; c += step)
        store_piece<P::kSize>(dy + c * P::kSize, v4u{0u, 0u, 0u, 0u}, g.cols - c);
    }
    if (g.dweights == nullptr) continue;
    // a row's lanes are a power of two: within a wave, or whole waves of one row
    for (int d = (per < 64 ? per : 64) / 2; d > 0; d >>= 1) dot += __shfl_xor(dot, d);
    if (per > 64) {
      __syncthreads();
      if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = dot;
      __syncthreads();
      const int w0 = threadIdx.x / per * (per / 64);
      dot = sums[w0];
      for (int v = 1; v < per / 64; ++v) dot += sums[w0 + v];
    }
    if (in_row == 0 && here) g.dweights[s] = dot;
  }
}

// Rows to a workgroup: as many lanes to a row as it has pieces, within 16 .. 256.
int rows_log2(int64_t cols, int elems) {
  const int64_t pieces = (cols + elems - 1) / elems;
  int lg = 0;
  while (lg < 4 && (256 >> lg) / 2 >= pieces) ++lg;
  return lg;
}

int64_t row_blocks(int64_t rows, int lg) { return (rows + (int64_t(1) << lg) - 1) >> lg; }

}  // namespace

int64_t expert_row_blocks(int64_t rows, int64_t cols, int dt) { return row_blocks(rows, rows_log2(cols, dt == ZS_FP32 ? 4 : 8)); }

int64_t route_workspace(int64_t slots, int experts) {
  const int64_t chunks = (slots + kRouteChunk - 1) / kRouteChunk;
  if (chunks <= 1) return 16;
  return (chunks + 1) * (int64_t(experts) + 1) * int64_t(sizeof(int32_t));
}

hipError_t launch_route(RouteArgs a, void* workspace, hipStream_t s) {
  const int keys = a.experts + 1;
  a.chunks = (a.slots + kRouteChunk - 1) / kRouteChunk;
  a.bits = 0;
  while ((1 << a.bits) < keys) ++a.bits;
  a.totals = static_cast<int32_t*>(workspace);
  a.counts = a.totals + keys;
  auto lds = [&](int waves) { return size_t(waves + 2) * keys * sizeof(int); };
  if (a.chunks <= 1) {
    hipLaunchKernelGGL((k_route_place<kAlone, 4>), dim3(1), dim3(256), lds(4), s, a);
    return hipGetLastError();
  }
  if (a.slots <= 16 * kWaveChunk && keys <= 512) {  // 36 KB of LDS
    hipLaunchKernelGGL((k_route_place<kAlone, 16>), dim3(1), dim3(1024), lds(16), s, a);
    return hipGetLastError();
  }
  const unsigned chunks = static_cast<unsigned>(a.chunks);
  hipLaunchKernelGGL(k_route_count, dim3(chunks), dim3(256), lds(4), s, a);
  if (a.chunks <= kFewChunks) {
    hipLaunchKernelGGL((k_route_place<kFew, 4>), dim3(chunks), dim3(256), lds(4), s, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(k_route_scan, dim3(static_cast<unsigned>(keys)), dim3(256), 0, s, a);
  hipLaunchKernelGGL((k_route_place<kMany, 4>), dim3(chunks), dim3(256), lds(4), s, a);
  return hipGetLastError();
}

hipError_t launch_expert_gather(RowsArgs a, int dt, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  a.rows_log2 = rows_log2(a.cols, dt == ZS_FP32 ? 4 : 8);
  const dim3 grid(static_cast<unsigned>(row_blocks(a.rows, a.rows_log2)));
  if (dt == ZS_FP32) hipLaunchKernelGGL((k_gather<4>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_gather<2>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_expert_combine(RowsArgs a, int dt, hipStream_t s) {
  const int64_t tokens = a.rows / a.choices;
  if (tokens == 0) return hipSuccess;
  a.rows_log2 = rows_log2(a.cols, dt == ZS_FP32 ? 4 : 8);
  const dim3 grid(static_cast<unsigned>(row_blocks(tokens, a.rows_log2)));
  if (dt == ZS_BF16) hipLaunchKernelGGL((k_combine<ZS_BF16>), grid, dim3(256), 0, s, a);
  else if (dt == ZS_FP16) hipLaunchKernelGGL((k_combine<ZS_FP16>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_combine<ZS_FP32>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_expert_combine_backward(CombineBackwardArgs a, int dt, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  a.rows_log2 = rows_log2(a.cols, dt == ZS_FP32 ? 4 : 8);
  const dim3 grid(static_cast<unsigned>(row_blocks(a.rows / a.choices, a.rows_log2)));
  if (dt == ZS_BF16) hipLaunchKernelGGL((k_combine_backward<ZS_BF16>), grid, dim3(256), 0, s, a);
  else if (dt == ZS_FP16) hipLaunchKernelGGL((k_combine_backward<ZS_FP16>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_combine_backward<ZS_FP32>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace zs
