// gfx950 kernels of the matrix products: a layer's products with an 8-bit weight (zs_product8), and
// the experts' products over groups of rows (zs_expert_product, zs_expert_wgrad):
//   c[m][n] = sum over k of a[m][k] * b[n][k]
// on the matrix cores, summed in fp32.  16-bit products are exact in it.  The 8-bit instructions align up to
// eight consecutive products to the largest and cut off what lies 2^-13 below it before they add the eight to
// the fp32 sum: up to 7 * 2^-13 of the largest for each eight, and measured over whole sums about 2^-15.6 of
// the result, where rounding it to fp16 takes 2^-12.2 (777 x 1003 -> 517: error against 64 bits 2.083e-4 of the
// norm, 2.074e-4 for the exact sum rounded once).  Without the cut, in bf16, the product runs at the 16-bit
// rate, at half the speed.
//
// An operand lies in memory with consecutive k (rows of m or n, "by rows"), or with consecutive m
// or n (rows of k, "by k").  A stage of the sum is 128 bytes of every row, a cache line: 64 values of
// k in 16 bits, 128 in 8.  Stages go from memory straight into LDS, 16 bytes to a lane, into two
// buffers in turn.  Such a load puts a wave's 64 pieces one after the other, so rows cannot be padded
// against bank conflicts: instead a lane fetches another piece of its row than its place says.
// Operands by rows are read back 16 bytes to a lane (sixteen lanes that read at once: sixteen rows,
// whose pieces lie on all 64 banks), operands by k through gfx950's transposing loads.
//
// Long sums are bound by the matrix cores and the clock that the card's power allows: 16384 x 4096 ->
// 14336 in 8 bits takes 801 us (2.40 PFLOP/s, matrix cores 57 % busy; the library with one scale for each
// whole matrix 770), in bf16 over eight experts 1590 (1.21, 74 %; over one 1462, the library 1380).  Short
// ones are bound by a tile's start and end: both gradients of 16 experts of 4096 x 448, 16384 rows, take
// 99 + 100 us where the operations take 86.  Few rows are bound by reading b: 1 x 4096 -> 14336 in 8 bits
// in 14 us (4.1 TB/s), 32 rows over 16 experts of 4096 x 448 in 15.

#include <algorithm>
#include <type_traits>

#include "zs_act_dev.h"

namespace zs {
namespace {

using namespace act;

typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8hf __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;
typedef __attribute__((address_space(3))) void lds_void;
typedef v4u v4u_a1 __attribute__((aligned(1)));

// A workgroup's tile: WM x WN waves, each FM x FN matrix instructions of 32 x 32; DEPTH stages in LDS.
template <int WM_, int WN_, int FM_, int FN_, int DEPTH_>
struct Tile {
  static constexpr int WM = WM_, WN = WN_, FM = FM_, FN = FN_, kStages = DEPTH_;
  static constexpr int kThreads = WM * WN * 64;
  static constexpr int kM = WM * FM * 32, kN = WN * FN * 32;
  // bytes of a stage of half of a's rows, and of b's
  static constexpr int kHalfM = kM / 2 * 128, kBufferN = kN * 128;
  static constexpr int kBuffers = kStages * (2 * kHalfM + kBufferN);
  static constexpr int kSegment = kM * 64;  // a's scales (8-bit operands): 64 bytes of each row, twice
  static constexpr int kStripPitch = FN * 32 + 8;  // the epilogue's strips, as in the weight gradient
  static constexpr int kStrips = WM * WN * 32 * kStripPitch * 4;
  static constexpr int lds(bool eight) {
    const int all = kBuffers + (eight ? 2 * kSegment : 0);
    return all > kStrips ? all : kStrips;
  }
  static_assert(lds(true) <= 163840, "LDS of a CU");
  static_assert((kStages & (kStages - 1)) == 0 && FM % 2 == 0 && kThreads % 64 == 0 && kM >= 128 && kN >= 128, "halves, and blocks that change places");
};

// ------------------------------------------------------------------ groups of rows

// Running sums or maxima (of numbers that are not negative) over a wave's lanes, through the data-parallel
// moves within and between rows of sixteen lanes.
template <bool MAX, int CTRL, int ROWS>
__device__ __forceinline__ int scan_step(int v) {
  const int o = __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
  return MAX ? (o > v ? o : v) : v + o;
}
template <bool MAX>
__device__ __forceinline__ int wave_scan(int v) {
  v = scan_step<MAX, 0x111, 0xF>(v);  // from one, two, four, eight lanes before, in the same row
  v = scan_step<MAX, 0x112, 0xF>(v);
  v = scan_step<MAX, 0x114, 0xF>(v);
  v = scan_step<MAX, 0x118, 0xF>(v);
  v = scan_step<MAX, 0x142, 0xA>(v);  // a row's last lane to the row behind it
  return scan_step<MAX, 0x143, 0xC>(v);
}

// Ends that run backwards or past the rows would lead out of the matrices: an end counts as the
// largest one up to it, within 0 .. rows.
struct Span {
  int64_t first, last;
  int group;
};

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// The span of rows of group e.
__device__ __forceinline__ Span group_span(const int32_t* ends, int e, int64_t rows) {
  const int lane = threadIdx.x & 63;
  int before = 0, upto = 0;
  for (int c = 0; c <= e; c += 64) {
    int v = c + lane <= e ? ends[c + lane] : 0;
    v = v < 0 ? 0 : v > rows ? static_cast<int>(rows) : v;
    const int all = __builtin_amdgcn_readlane(wave_scan<true>(v), 63);
    const int less = __builtin_amdgcn_readlane(wave_scan<true>(c + lane < e ? v : 0), 63);
    before = less > before ? less : before;
    upto = all > upto ? all : upto;
  }
  return {before, upto > before ? upto : before, e};
}

// 64 groups' rows from `top` on, one group to a lane: their tiles, and the tiles up to each.
struct GroupTiles {
  int start, end, tiles, upto;
};
__device__ __forceinline__ GroupTiles group_tiles(const int32_t* ends, int groups, bool rest, int64_t rows, int tile, int c, int top) {
  const int lane = threadIdx.x & 63;
  int v = c + lane < groups ? ends[c + lane] : c + lane == groups && rest ? static_cast<int>(rows) : 0;
  v = v < 0 ? 0 : v > rows ? static_cast<int>(rows) : v;
  v = wave_scan<true>(v);
  v = v > top ? v : top;
  const int start = __builtin_amdgcn_update_dpp(top, v, 0x138, 0xF, 0xF, false);  // the end of the lane before
  const int n = (v - start + tile - 1) / tile;
  return {start, v, n, wave_scan<false>(n)};
}

// Tiles of `tile` rows of all groups, one group after the other, and, where `rest`, of the rows behind
// the last one as one more group.  unit_of(their number) names one of them, or none with a number
// below 0: *s is its group, with the rows from the tile's first to the group's last.
template <class UnitOf>
__device__ __forceinline__ void find_tile(const int32_t* ends, int groups, bool rest, int64_t rows, int tile, UnitOf unit_of, Span* s) {
  if (ends == nullptr) {
    const int unit = unit_of(static_cast<int>((rows + tile - 1) / tile));
    *s = {int64_t(unit) * tile, rows, 0};
    return;
  }
  auto pick = [&](const GroupTiles& t, int unit, int c) {
    const int mine = unit - (t.upto - t.tiles);
    const uint64_t hit = __ballot(mine >= 0 && mine < t.tiles);
    if (hit == 0) return;
    const int at = __ffsll(static_cast<unsigned long long>(hit)) - 1;
    s->first = __builtin_amdgcn_readlane(t.start, at) + int64_t(__builtin_amdgcn_readlane(mine, at)) * tile;
    s->last = __builtin_amdgcn_readlane(t.end, at);
    s->group = c + at;
  };
  const int all = groups + (rest ? 1 : 0);
  if (all <= 64) {  // one look at the ends
    const GroupTiles t = group_tiles(ends, groups, rest, rows, tile, 0, 0);
    pick(t, unit_of(__builtin_amdgcn_readlane(t.upto, 63)), 0);
    return;
  }
  int tiles = 0, unit = 0;
  for (int pass = 0; pass < 2; ++pass) {  // count, then look
    int top = 0, before = 0;
    for (int c = 0; c < all; c += 64) {
      const GroupTiles t = group_tiles(ends, groups, rest, rows, tile, c, top);
      if (pass == 0) tiles += __builtin_amdgcn_readlane(t.upto, 63);
      else pick(t, unit - before, c);
      before += __builtin_amdgcn_readlane(t.upto, 63);
      top = __builtin_amdgcn_readlane(t.end, 63);
    }
    if (pass == 0) unit = unit_of(tiles);
  }
}

// ------------------------------------------------------------------ operands

template <int DT>
__device__ __forceinline__ v16f mfma(const v8s& a, const v8s& b, const v16f& c) {
  if constexpr (DT == ZS_BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8hf, a), __builtin_bit_cast(v8hf, b), c, 0, 0, 0);
}

// Elements k .. k + 7 of a row of `len` 2-byte elements, zeros behind the row's end: where the row ends
// among them, the row's last eight, moved down: one load and a few shifts instead of seven loads of
// single elements.
__device__ __forceinline__ v4u load8_row(const uint16_t* row, int64_t k, int64_t len) {
  if (len < 8) return load8h(row + k, len > k ? static_cast<int>(len - k) : 0);
  const int64_t from = k < len - 8 ? k : len - 8;
  const v4u w = *reinterpret_cast<const v4u_a2*>(row + from);
  if (k == from) return w;
  if (k >= len) return v4u{0u, 0u, 0u, 0u};
  return __builtin_bit_cast(v4u, __builtin_bit_cast(unsigned __int128, w) >> (16 * static_cast<int>(k - from)));
}

constexpr int64_t kFewUnits = 512;  // see few_rows
constexpr int kEight = 3;  // the operands' type beside ZS_BF16 and ZS_FP16: e4m3 codes

// One operand of a workgroup, or half of one: R rows of m or n, k from 0 to `depth` (elements).
// BY_K: k runs over memory rows.  Row r is the tile's row r, or, of a half, the r % RUN-th of the
// half's rows of wave row r / RUN: each wave finds half of its rows in either half.  `left` rows of
// the tile lie inside the matrix; the others repeat the last one and reach outputs that are never
// stored.  `stride` and offsets in bytes.
template <bool BY_K, int R, int RUN, int THREADS, int SIZE>
struct Operand {
  static constexpr int kLoads = R * 8 / THREADS;         // 16-byte pieces per thread and stage
  static constexpr int kPerRow = BY_K ? R / 8 : 8;       // pieces of a memory row
  static constexpr int kRows = THREADS / kPerRow;        // memory rows of one load of the workgroup
  static constexpr int kDepth = BY_K ? 64 : 128 / SIZE;  // k of a stage
  static constexpr int kBlocks = R >= 128 ? 4 : 2;       // by k: blocks of 64 bytes that change places
  static_assert(!BY_K || SIZE == 2, "8-bit operands lie by rows");
  static_assert(kLoads * THREADS == R * 8, "whole loads");
  static_assert(kRows % (BY_K ? 4 : 16) == 0, "a thread's pieces change places alike");
  const char* base;
  int64_t stride, depth, padded;
  int left, half;  // half: 0 or 1, -1 for a whole operand
  uint32_t off[kLoads];

  // which piece of its memory row a thread fetches
  static __device__ __forceinline__ int piece() {
    const int row = threadIdx.x / kPerRow, at = threadIdx.x % kPerRow;
    return BY_K ? ((at >> 2) ^ (row & (kBlocks - 1))) << 2 | (at & 3) : at ^ ((row >> 1) & 7);
  }
  __device__ __forceinline__ int tile_row(int r) const { return half < 0 ? r : r / RUN * (2 * RUN) + half * RUN + r % RUN; }
  // padded: bytes of a memory row that may be read (8-bit operands by rows)
  __device__ __forceinline__ Operand(const char* base_, int64_t stride_, int left_, int64_t depth_, int64_t padded_, int half_ = -1)
      : base(base_), stride(stride_), depth(depth_), padded(padded_), left(left_), half(half_) {
    int col = tile_row(piece() * 8);  // by k
    if (BY_K && col + 8 > left) col = left >= 8 ? left - 8 : 0;
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      int row = u * kRows + threadIdx.x / kPerRow;
      if (!BY_K) {
        row = tile_row(row);
        if (row >= left) row = left - 1;
      }
      off[u] = static_cast<uint32_t>(row) * static_cast<uint32_t>(stride) + (BY_K ? col * 2 : piece() * 16);
      asm volatile("" : "+v"(off[u]));  // one register, not half of a 64-bit product
    }
  }
  __device__ __forceinline__ const char* at(int64_t stage) const {
    return base + stage * (BY_K ? stride * kDepth : int64_t(128));
  }
  // Piece u of a whole stage, which begins at p, from memory to LDS.  (A buffer's base is scalar and
  // moves with the stage; the offsets stay.  Beside global loads to LDS the compiler would wait for all
  // LDS reads under way wherever one is needed.)
  __device__ __forceinline__ void direct(int u, const char* p, char* lds, int wave) const {
#ifdef __HIP_DEVICE_COMPILE__  // the host compiler knows no buffers
    const auto r = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p), 0, -1, 0x00027000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(lds + (u * THREADS + wave * 64) * 16), 16, off[u], 0, 0, 0);
#endif
  }
  // A stage into registers, at any alignment, with zeros outside.  OFTEN: one that lies inside takes the
  // offsets that `direct` has; the addresses of the others are worked out here.
  template <bool OFTEN = false>
  __device__ __forceinline__ void fetch(int64_t stage, v4u (&r)[kLoads]) const {
    if (OFTEN && SIZE == 2 && (stage + 1) * kDepth <= depth && stride < (1 << 24) && (!BY_K || left >= (half < 0 ? R : 2 * R))) {
      const char* p = at(stage);
#pragma unroll
      for (int u = 0; u < kLoads; ++u) r[u] = *reinterpret_cast<const v4u_a2*>(p + off[u]);
      return;
    }
    int id = threadIdx.x;
    asm volatile("" : "+v"(id));
    const int row0 = id / kPerRow, p = piece();
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      int64_t row = row0 + u * kRows;
      if constexpr (BY_K) {
        const int col = tile_row(p * 8);
        row += stage * kDepth;
        const int cnt = row < depth ? left - col : 0;
        r[u] = load8h(reinterpret_cast<const uint16_t*>(base + row * stride) + col, cnt >= 8 ? 8 : cnt > 0 ? cnt : 0);
        continue;
      }
      row = tile_row(static_cast<int>(row));
      if (row >= left) row = left - 1;
      if constexpr (SIZE == 1) {  // past the row's end: a piece of the same row, which meets zeros
        const int64_t byte = stage * 128 + p * 16;
        r[u] = *reinterpret_cast<const v4u*>(base + row * stride + (byte < padded ? byte : padded - 16));
      } else {
        r[u] = load8_row(reinterpret_cast<const uint16_t*>(base + row * stride), stage * kDepth + p * 8, depth);
      }
    }
  }
  static __device__ __forceinline__ void leave(const v4u (&r)[kLoads], char* lds) {
#pragma unroll
    for (int u = 0; u < kLoads; ++u) *reinterpret_cast<v4u*>(lds + (u * THREADS + threadIdx.x) * 16) = r[u];
  }
};

// How a lane reads the fragments of one operand from a buffer: fragment f holds 32 rows of m or n,
// quarter s of a stage 16 values of k in 16 bits (32 in 8): lanes 0 .. 31 the first of its two pieces,
// 32 .. 63 the second.
template <bool BY_K, int R, int F>
struct Reader {
  static constexpr int kPitch = BY_K ? R * 2 : 128;
  int at[BY_K ? F : 4], wave_at;
  __device__ __forceinline__ Reader(int first) {  // the wave's first row
    const int lane = threadIdx.x & 63;
    wave_at = BY_K ? 0 : first * 128;
    if constexpr (BY_K) {
      const int row = (lane >> 5) * 8 + ((lane & 15) >> 2), col = ((lane >> 4) & 1) * 16 + (lane & 3) * 4;
#pragma unroll
      for (int f = 0; f < F; ++f) at[f] = row * kPitch + (((first + f * 32 + col) * 2) ^ ((row & (R >= 128 ? 3 : 1)) * 64));
    } else {
#pragma unroll
      for (int s = 0; s < 4; ++s) at[s] = (lane & 31) * 128 + (((2 * s + (lane >> 5)) ^ ((lane >> 1) & 7)) * 16);
    }
  }
  __device__ __forceinline__ v8s operator()(const char* buf, int f, int s) const {
    if constexpr (BY_K) {
      const char* p = buf + at[f] + s * 16 * kPitch;
      const v4s x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p));
      const v4s y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p + 4 * kPitch));
      return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
      return *reinterpret_cast<const v8s*>(buf + wave_at + at[s] + f * 4096);
    }
  }
};

// Waits until at most N of the wave's loads are under way, and for its LDS reads and writes; the
// workgroup's barrier.
template <int N>
__device__ __forceinline__ void wait_loads() {
#ifdef __HIP_DEVICE_COMPILE__
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
#endif
}
__device__ __forceinline__ void wait_lds() {
#ifdef __HIP_DEVICE_COMPILE__
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#endif
}
__device__ __forceinline__ void meet() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// ------------------------------------------------------------------ the product

// Eight elements of the base from `at` on, cnt of them inside, as they lie in memory.
struct Base8 {
  v4u lo, hi;  // hi: of fp32
};
__device__ __forceinline__ Base8 load_base8(const ProductArgs& g, int64_t at, int cnt) {
  Base8 b = {{0u, 0u, 0u, 0u}, {0u, 0u, 0u, 0u}};
  if (g.c_dt != ZS_FP32) {
    b.lo = load8h(static_cast<const uint16_t*>(g.base) + at, cnt);
    return b;
  }
  const uint32_t* p = static_cast<const uint32_t*>(g.base) + at;
  if (cnt == 8) {
    b.lo = *reinterpret_cast<const v4u_a4*>(p);
    b.hi = *reinterpret_cast<const v4u_a4*>(p + 4);
  } else {
#pragma unroll
    for (int j = 0; j < 7; ++j)
      if (j < cnt) (j < 4 ? b.lo : b.hi)[j & 3] = p[j];
  }
  return b;
}

// Eight sums of a row of c, cnt of them inside: added to the base and rounded once.
__device__ __forceinline__ void write8(const ProductArgs& g, int64_t at, int cnt, const Base8& base, float (&f)[8]) {
  if (g.c_dt == ZS_FP32) {
    uint32_t* p = static_cast<uint32_t*>(g.c) + at;
    v4u lo, hi;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      lo[j] = f_bits(f[j] + bits_f(base.lo[j]));
      hi[j] = f_bits(f[4 + j] + bits_f(base.hi[j]));
    }
    if (cnt == 8) {
      *reinterpret_cast<v4u_a4*>(p) = lo;
      *reinterpret_cast<v4u_a4*>(p + 4) = hi;
    } else {
#pragma unroll
      for (int j = 0; j < 7; ++j)
        if (j < cnt) p[j] = (j < 4 ? lo : hi)[j & 3];
    }
    return;
  }
  uint16_t* p = static_cast<uint16_t*>(g.c) + at;
  float x[8];
  if (g.c_dt == ZS_BF16) widen8<ZS_BF16>(base.lo, x);
  else widen8<ZS_FP16>(base.lo, x);
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] += x[j];
  store8h(p, g.c_dt == ZS_BF16 ? narrow8<ZS_BF16>(f) : narrow8<ZS_FP16>(f), cnt);
}

// Unit u of a tiles_m x tiles_n grid in bands of eight rows of tiles, column by column: workgroups
// that run at the same time share rows of both operands in their XCD's L2.
__device__ __forceinline__ void banded(int u, int tiles_m, int tiles_n, int* m, int* n) {
  constexpr int kBand = 8;
  const int band = u / (kBand * tiles_n), in = u - band * kBand * tiles_n;
  const int high = tiles_m - band * kBand < kBand ? tiles_m - band * kBand : kBand;
  *n = in / high;
  *m = band * kBand + in - *n * high;
}

// KIND: ZS_BF16, ZS_FP16 or kEight.  AK, BK: operand a, b lies by k.  SUM_GROUPS: the groups divide
// k, and each has an output of its own (the weight gradient); otherwise they divide m, and each has
// a b of its own.  STAGED: stages pass through registers, for operands that are not aligned to
// whole words.
template <int KIND, bool AK, bool BK, bool SUM_GROUPS, bool STAGED, class TL>
__global__ __launch_bounds__(TL::kThreads, 2) void k_product(ProductArgs g) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  constexpr int kSize = KIND == kEight ? 1 : 2;
  using OpA = Operand<AK, TL::kM / 2, TL::FM * 16, TL::kThreads, kSize>;
  using OpB = Operand<BK, TL::kN, TL::kN, TL::kThreads, kSize>;
  constexpr int kDepth = OpA::kDepth;

  // one contiguous run of units per XCD
  const int tiles_n = static_cast<int>((g.n + TL::kN - 1) / TL::kN);
  Span s{0, 0, 0};
  int64_t m0, k0 = 0, depth = g.k;
  int tm = -1, tn = 0;
  auto unit_of = [&](int units) {  // this workgroup's, or -1
    const int run = (units + kXcds - 1) / kXcds, in_run = blockIdx.x / kXcds, unit = blockIdx.x % kXcds * run + in_run;
    return in_run < run && unit < units ? unit : -1;
  };
  if constexpr (SUM_GROUPS) {
    const int tiles_m = static_cast<int>((g.m + TL::kM - 1) / TL::kM);
    const int unit = unit_of(tiles_m * tiles_n * g.groups);
    if (unit < 0) return;
    const int e = unit / (tiles_m * tiles_n);
    s = group_span(g.ends, e, g.k);
    banded(unit - e * tiles_m * tiles_n, tiles_m, tiles_n, &tm, &tn);
    m0 = int64_t(tm) * TL::kM;
    k0 = s.first;
    depth = s.last - s.first;
  } else {
    find_tile(g.ends, g.groups, g.zero_rest, g.m, TL::kM,
              [&](int tiles_m) {
                const int unit = unit_of(tiles_m * tiles_n);
                if (unit >= 0) banded(unit, tiles_m, tiles_n, &tm, &tn);
                return tm;
              },
              &s);
    if (tm < 0) return;
    m0 = s.first;
    if (g.ends != nullptr && s.group == g.groups) depth = 0;  // rows behind the last group: zeros
  }
  const int64_t n0 = int64_t(tn) * TL::kN;
  const int64_t m_end = SUM_GROUPS ? g.m : s.last;
  const int left_m = static_cast<int>(m_end - m0 < TL::kM ? m_end - m0 : TL::kM);
  const int left_n = static_cast<int>(g.n - n0 < TL::kN ? g.n - n0 : TL::kN);
  // a group behind the last one has no b
  const int64_t b_at = SUM_GROUPS || depth == 0 ? 0 : s.group * g.b_group;
  const char* const a_base = static_cast<const char*>(g.a) + (AK ? k0 * g.a_stride + m0 : m0 * g.a_stride + k0) * kSize;
  const OpA op_a[2] = {{a_base, g.a_stride * kSize, left_m, depth, g.a_padded, 0}, {a_base, g.a_stride * kSize, left_m, depth, g.a_padded, 1}};
  const OpB op_b(static_cast<const char*>(g.b) + (b_at + (BK ? k0 * g.b_stride + n0 : n0 * g.b_stride + k0)) * kSize,
                 g.b_stride * kSize, left_n, depth, g.b_padded);

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / TL::WN * TL::FM * 32, wn = wave % TL::WN * TL::FN * 32;
  const Reader<AK, TL::kM / 2, TL::FM / 2> read_a(wm / 2);
  const Reader<BK, TL::kN, TL::FN> read_b(wn);

  v16f acc[TL::FM][TL::FN];
#pragma unroll
  for (int i = 0; i < TL::FM; ++i)
#pragma unroll
    for (int j = 0; j < TL::FN; ++j) acc[i][j] = v16f(0.0f);

  // Scales of 8-bit operands for a stage: a dword of four groups of 32 for each of a's rows, a byte for
  // b's block.  Lanes 32 .. 63 name those of the second and fourth group.  Those of a come through LDS,
  // a segment of sixteen stages (64 bytes of a row) at a time: read by each wave for its fragments, the
  // scattered dwords took as long as both operands.  The four pieces of a segment's row change places
  // by (row / 4) % 4.
  constexpr int kScales = KIND == kEight ? TL::FM : 1;
  constexpr int kPieces = TL::kM * 4 / TL::kThreads;
  struct Scales {
    int a[kScales], b;
  };
  char* const segments = lds + TL::kBuffers;
  const int64_t a_groups = g.a_padded / kActGroup;
  const uint8_t* b_scale = nullptr;
  if constexpr (KIND == kEight) b_scale = g.b_scales + (n0 + wn < g.n ? n0 + wn : g.n - 1) / 128 * g.b_scale_row;
  auto begin_segment = [&](int64_t segment) {
    if constexpr (KIND == kEight) {
      char* into = segments + (segment & 1) * TL::kSegment;
      const uint8_t* p = g.a_scales + m0 * a_groups + segment * 64;
      const int64_t left = a_groups - segment * 64;  // groups of the rows from here on
      int id = threadIdx.x;
      asm volatile("" : "+v"(id));
#pragma unroll
      for (int u = 0; u < kPieces; ++u) {
        int row = (u * TL::kThreads + id) / 4;
        const int at = ((id & 3) ^ ((row >> 2) & 3)) * 16;
        if (row >= left_m) row = left_m - 1;
        v4u w;
        if (at + 16 <= left) {
          w = *reinterpret_cast<const v4u_a1*>(p + row * a_groups + at);
        } else {  // groups past the row's end count as its last one: they meet zeros
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            w[q] = 0;
            for (int e = 0; e < 4; ++e) {
              const int64_t i = at + q * 4 + e < left ? at + q * 4 + e : left - 1;
              w[q] |= static_cast<uint32_t>(p[row * a_groups + i]) << (8 * e);
            }
          }
        }
        *reinterpret_cast<v4u*>(into + (u * TL::kThreads + id) * 16) = w;
      }
    }
  };
  const int scale_row = (wm + (lane & 31)) * 64, scale_turn = ((lane >> 2) & 3) * 16;
  auto read_scales = [&](int64_t stage, Scales& sc) {
    if constexpr (KIND == kEight) {
      const int q = static_cast<int>(stage) & 15;
      const char* p = segments + (static_cast<int>(stage >> 4) & 1) * TL::kSegment + scale_row + (((q >> 2) * 16) ^ scale_turn) + (q & 3) * 4;
#pragma unroll
      for (int i = 0; i < TL::FM; ++i)
        sc.a[i] = static_cast<int>(*reinterpret_cast<const uint32_t*>(p + i * 2048) >> (lane >> 5) * 8);
    }
  };

  // A stage is multiplied in four clusters: half h of the wave's rows of a with half q of the stage's
  // k, (0, 0), (0, 1), (1, 0), (1, 1).  b's fragments are read with the first two and kept.
  constexpr int kHalf = TL::FM / 2;
  constexpr bool kJoined = KIND != kEight;
  v8s fa[kJoined ? 2 : 1][kHalf][2], fb[2][TL::FN][2];
  auto multiply = [&](int h, int q, const v8s (&fa)[kHalf][2], const Scales& sc, auto odd) {
    if constexpr (KIND == kEight) {
      typedef short v16s __attribute__((ext_vector_type(16)));
#pragma unroll
      for (int i = 0; i < kHalf; ++i)
#pragma unroll
        for (int j = 0; j < TL::FN; ++j) {
          const v16s a = __builtin_shufflevector(fa[i][0], fa[i][1], 0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15);
          const v16s b = __builtin_shufflevector(fb[q][j][0], fb[q][j][1], 0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15);
          v16f& c = acc[h * kHalf + i][j];
          c = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(__builtin_bit_cast(v8i, a), __builtin_bit_cast(v8i, b), c, 0, 0,
                                                              2 * decltype(odd)::value, sc.a[h * kHalf + i], 0, sc.b);
        }
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < kHalf; ++i)
#pragma unroll
          for (int j = 0; j < TL::FN; ++j)
            acc[h * kHalf + i][j] = mfma<KIND>(fa[i][e], fb[q][j][e], acc[h * kHalf + i][j]);
    }
  };

  const int64_t stages = (depth + kDepth - 1) / kDepth;
  // stages that lie inside both operands; the others pass through registers
  const int64_t whole = STAGED ? 0 : KIND == kEight ? g.a_padded / 128 : depth / kDepth;
  constexpr int kBufs = TL::kStages;
  auto buffer_a = [&](int h, int64_t stage) { return lds + (kBufs * h + (static_cast<int>(stage) & (kBufs - 1))) * TL::kHalfM; };
  auto buffer_b = [&](int64_t stage) {
    return lds + 2 * kBufs * TL::kHalfM + (static_cast<int>(stage) & (kBufs - 1)) * TL::kBufferN;
  };
  // a stage of an operand into LDS: under way, or done where it takes registers
  auto begin = [&](const auto& op, int64_t stage, char* buf) {
    using Op = std::remove_cv_t<std::remove_reference_t<decltype(op)>>;
    if (stage < whole) {
      const char* p = op.at(stage);
#pragma unroll
      for (int u = 0; u < Op::kLoads; ++u) op.direct(u, p, buf, wave);
    } else {
      v4u t[Op::kLoads];
      op.fetch(stage, t);
      Op::leave(t, buf);
    }
  };
  // Two groups of waves take turns: while one reads its fragments and sends for later stages, the other,
  // one barrier ahead or behind, multiplies; each SIMD has a wave of both.  (Where waves are four to a
  // workgroup, two workgroups on a CU do that for each other, and the barriers within a half of a
  // stage are left out.)
  // A half of a, and b, are free once their clusters have been read, and a later stage goes there, i + 2
  // with two buffers: b and the first half from cluster 2 of stage i on, the second half in cluster 0 of
  // stage i + 1.  Each has a stage and a half of time.  A wave waits for its own pieces one cluster before they are read;
  // the barrier behind that makes it all waves'.
  constexpr bool kTurns = TL::kThreads == 512;
  static_assert(!STAGED || KIND != kEight, "8-bit operands are aligned");
  static_assert(!STAGED || kBufs == 2, "a stage in registers, one in LDS beside the present one");
  if (stages > 0) {
    constexpr std::integral_constant<int, 0> kZero{};
    constexpr std::integral_constant<int, 1> kOne{};
    Scales sc;
    int next_b_scale = 0;
    auto none = [] {};
    auto cluster = [&](int h, auto odd, const char* buf_a, const char* buf_b, auto around, auto after) {
      constexpr int kFirst = decltype(odd)::value, kLast = kJoined ? 1 : kFirst;
#pragma unroll
      for (int q = kFirst; q <= kLast; ++q) {
        if (h == 0) {
#pragma unroll
          for (int j = 0; j < TL::FN; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) fb[q][j][e] = read_b(buf_b, j, 2 * q + e);
        }
#pragma unroll
        for (int i = 0; i < kHalf; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) fa[q - kFirst][i][e] = read_a(buf_a, i, 2 * q + e);
      }
      around();
      wait_lds();
      if (kTurns) meet();
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int q = kFirst; q <= kLast; ++q) multiply(h, q, fa[q - kFirst], sc, odd);
      __builtin_amdgcn_s_setprio(0);
      after();
      if (kTurns || kLast == 1) meet();
    };
    for (int64_t i = 0; i < kBufs && i < stages; ++i) {
      begin(op_a[0], i, buffer_a(0, i));
      begin(op_b, i, buffer_b(i));
      if (i < kBufs - 1) begin(op_a[1], i, buffer_a(1, i));
    }
    begin_segment(0);
    if constexpr (KIND == kEight) next_b_scale = b_scale[0];
    wait_loads<0>();
    wait_lds();
    meet();
    if (kTurns && wave >= 4) meet();
    // MAIN: the new stages go straight to LDS
    v4u ra0[STAGED ? OpA::kLoads : 1], ra1[STAGED ? OpA::kLoads : 1], rb[STAGED ? OpB::kLoads : 1];
    auto one_stage = [&](int64_t i, auto main) {
      constexpr bool kMain = decltype(main)::value;
      constexpr int kA = OpA::kLoads, kB = OpB::kLoads;
      char* a0 = buffer_a(0, i);
      char* a1 = buffer_a(1, i);
      char* b = buffer_b(i);
      if constexpr (KIND == kEight) {
        if ((i & 15) == 8 && (i / 16 + 1) * 16 < stages) begin_segment(i / 16 + 1);
        read_scales(i, sc);
        sc.b = next_b_scale;
        if (kMain || i + 1 < stages) next_b_scale = b_scale[(i + 1) * g.b_scale_step];
      }
      const char* pa = op_a[0].at(i + kBufs);
      const char* pb = op_b.at(i + kBufs);
      auto send_a1 = [&] {
        if constexpr (kMain) {
          const char* p = op_a[1].at(i + kBufs - 1);
#pragma unroll
          for (int u = 0; u < kA; ++u) op_a[1].direct(u, p, buffer_a(1, i + kBufs - 1), wave);
        } else if constexpr (STAGED) {
          if (i + 1 < stages) op_a[1].template fetch<true>(i + 1, ra1);
        } else {
          if (i + kBufs - 1 < stages) begin(op_a[1], i + kBufs - 1, buffer_a(1, i + kBufs - 1));
        }
      };
      auto leave_a0_b = [&] {
        if constexpr (STAGED) {
          if (i > 0 && i + 1 < stages) {
            OpA::leave(ra0, buffer_a(0, i + 1));
            OpB::leave(rb, buffer_b(i + 1));
            wait_lds();
          }
        }
      };
      auto send_a0_b = [&](int from, int to) {  // pieces of b
        if constexpr (kMain) {
          if (from == 0) {
#pragma unroll
            for (int u = 0; u < kA; ++u) op_a[0].direct(u, pa, a0, wave);
          }
#pragma unroll
          for (int u = from; u < to; ++u) op_b.direct(u, pb, b, wave);
        } else if (from == 0 && i + kBufs < stages) {
          if constexpr (STAGED) {
            op_a[0].template fetch<true>(i + kBufs, ra0);
            op_b.template fetch<true>(i + kBufs, rb);
          } else {
            begin(op_a[0], i + kBufs, a0);
            begin(op_b, i + kBufs, b);
          }
        }
      };
      auto leave_a1 = [&] {
        if constexpr (STAGED) {
          if (i + 1 < stages) {
            OpA::leave(ra1, buffer_a(1, i + 1));
            wait_lds();
          }
        }
      };
      // how many pieces may be under way behind those that are waited for: the second half of a, then
      // the next stage's first half and b
      if constexpr (kJoined) {
        cluster(
            0, kZero, a0, b,
            [&] {
              if constexpr (!STAGED) wait_loads<kMain ? (kBufs - 1) * (kA + kB) + (kBufs - 2) * kA : 0>();
              send_a1();
            },
            leave_a0_b);
        cluster(
            1, kZero, a1, b,
            [&] {
              if constexpr (!STAGED) wait_loads<kMain ? (kBufs - 1) * kA + (kBufs - 2) * (kA + kB) : 0>();
              send_a0_b(0, kB);
            },
            leave_a1);
      } else {
        cluster(0, kZero, a0, b, send_a1, none);
        cluster(0, kOne, a0, b, [&] {
          wait_loads<kMain ? (kBufs - 1) * (kA + kB) + (kBufs - 1) * kA : 0>();
        }, none);
        cluster(1, kZero, a1, b, [&] { send_a0_b(0, kB / 2); }, none);
        cluster(1, kOne, a1, b, [&] {
          wait_loads<kMain ? kBufs * kA + kB / 2 + (kBufs - 2) * (kA + kB) : 0>();
          send_a0_b(kB / 2, kB);
        }, none);
      }
    };
    int64_t i = 0;
    for (; i + kBufs < whole; ++i) one_stage(i, std::true_type{});
    for (; i < stages; ++i) one_stage(i, std::false_type{});
    if (kTurns && wave < 4) meet();
    meet();  // the strips below reuse the buffers
  }

  // The sums leave through LDS, a strip of 32 rows of the wave at a time, so that a lane stores
  // eight consecutive elements of a row.  Accumulator r of a lane is row 8 * (r / 4) + 4 * (lane / 32)
  // + r % 4, column lane % 32.
  float* strip = reinterpret_cast<float*>(lds) + wave * 32 * TL::kStripPitch;
  const int64_t c_at = SUM_GROUPS ? s.group * g.c_group : 0;
  constexpr int kRounds = TL::FN * 2, kEights = TL::FN * 4;  // eights of columns of a strip's row
#pragma unroll
  for (int i = 0; i < TL::FM; ++i) {
    int64_t at[kRounds];
    int cnt[kRounds];
    Base8 base[kRounds];
#pragma unroll
    for (int u = 0; u < kRounds; ++u) {  // the base's elements set out together
      const int q = u * 64 + lane, tm = wm + i * 32 + q / kEights, col = wn + q % kEights * 8, left = left_n - col;
      at[u] = c_at + (m0 + tm) * g.c_stride + n0 + col;
      cnt[u] = tm >= left_m || left <= 0 ? 0 : left >= 8 ? 8 : left;
      base[u] = {{0u, 0u, 0u, 0u}, {0u, 0u, 0u, 0u}};
      if (g.base != nullptr && cnt[u] > 0) base[u] = load_base8(g, at[u], cnt[u]);
    }
#pragma unroll
    for (int j = 0; j < TL::FN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        strip[(8 * (r / 4) + 4 * (lane >> 5) + r % 4) * TL::kStripPitch + j * 32 + (lane & 31)] = acc[i][j][r];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int u = 0; u < kRounds; ++u) {
      const int q = u * 64 + lane;
      const float* from = strip + q / kEights * TL::kStripPitch + q % kEights * 8;
      const v4u x = *reinterpret_cast<const v4u*>(from), y = *reinterpret_cast<const v4u*>(from + 4);
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = bits_f(x[j]);
        v[4 + j] = bits_f(y[j]);
      }
      if (cnt[u] > 0) write8(g, at[u], cnt[u], base[u], v);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// ------------------------------------------------------------------ few rows

// Products of 16 * MF rows of a at a time, where reading b is most of it: a workgroup takes 16 * NF
// rows of b, each of its waves every WAVES-th piece of 128 bytes of k, and the waves' sums meet in
// LDS.  Operands go from memory into the matrix instructions' registers without LDS: a lane's row is
// lane % 16, and the order of k within a piece is free as long as both operands have the same, so
// that a lane takes 32 consecutive bytes (16-bit operands; for 8-bit ones the instruction's scales
// fix which).  Any alignment will do.
template <int KIND, int MF, int NF, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void k_few(ProductArgs g) {
  constexpr int kSize = KIND == kEight ? 1 : 2, kDepth = 128 / kSize, kWaves = WAVES, kAhead = MF * NF == 1 ? 4 : 2, kTileM = 16 * MF;
  __shared__ __attribute__((aligned(16))) v4f sums[kWaves][MF * NF][64];
  const int tiles_n = static_cast<int>((g.n + 16 * NF - 1) / (16 * NF));
  Span s{0, 0, 0};
  int tm = -1, tn = 0;
  find_tile(g.ends, g.groups, g.zero_rest, g.m, kTileM,
            [&](int tiles_m) {
              const int units = tiles_m * tiles_n, run = (units + kXcds - 1) / kXcds, in_run = blockIdx.x / kXcds;
              const int unit = blockIdx.x % kXcds * run + in_run;
              if (in_run < run && unit < units) {  // tiles of one n are neighbours
                tm = unit % tiles_m;
                tn = unit / tiles_m;
              }
              return tm;
            },
            &s);
  if (tm < 0) return;
  const int64_t m0 = s.first, n0 = int64_t(tn) * (16 * NF);
  const bool none = g.ends != nullptr && s.group == g.groups;  // rows behind the last group: zeros
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), row = lane & 15, part = lane >> 4;
  const int left_m = static_cast<int>(s.last - m0 < kTileM ? s.last - m0 : kTileM);

  v4f acc[MF][NF];
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j) acc[i][j] = v4f(0.0f);
  if (!none) {
    const int64_t a_groups = g.a_padded / kActGroup;
    const char* pa[MF];
    const uint8_t* a_scale[MF];
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const int64_t m = m0 + (i * 16 + row < left_m ? i * 16 + row : left_m - 1);
      pa[i] = static_cast<const char*>(g.a) + m * g.a_stride * kSize;
      a_scale[i] = KIND == kEight ? g.a_scales + m * a_groups + part : nullptr;
    }
    const char* pb[NF];
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      const int64_t n = n0 + j * 16 + row;
      pb[j] = static_cast<const char*>(g.b) + ((KIND == kEight ? 0 : s.group * g.b_group) + (n < g.n ? n : g.n - 1) * g.b_stride) * kSize;
    }
    const int first = part * (KIND == kEight ? 16 : 32), second = first + (KIND == kEight ? 64 : 16);  // bytes
    struct Piece {
      v4u a[MF][2], b[NF][2];
      int a_scale[MF], b_scale;
    };
    const uint8_t* b_scale = KIND == kEight ? g.b_scales + n0 / kWeightBlock * g.b_scale_row : nullptr;
    auto fetch = [&](int64_t at, Piece& p) {  // a whole piece
      const int64_t byte = at * 128;
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        p.a[i][0] = *reinterpret_cast<const v4u_a2*>(pa[i] + byte + first);
        p.a[i][1] = *reinterpret_cast<const v4u_a2*>(pa[i] + byte + second);
        if constexpr (KIND == kEight) p.a_scale[i] = a_scale[i][at * 4];
      }
#pragma unroll
      for (int j = 0; j < NF; ++j) {
        p.b[j][0] = __builtin_nontemporal_load(reinterpret_cast<const v4u_a2*>(pb[j] + byte + first));
        p.b[j][1] = __builtin_nontemporal_load(reinterpret_cast<const v4u_a2*>(pb[j] + byte + second));
      }
      if constexpr (KIND == kEight) p.b_scale = b_scale[at * g.b_scale_step];
    };
    auto fetch_last = [&](int64_t at, Piece& p) {
      if constexpr (KIND == kEight) {  // past the row of a: a piece of the same row, which meets zeros
        const int64_t byte = at * 128, top = g.a_padded - 16;
        const int64_t group = at * 4 + part < a_groups ? at * 4 : a_groups - 1 - part;
#pragma unroll
        for (int i = 0; i < MF; ++i) {
          p.a[i][0] = *reinterpret_cast<const v4u*>(pa[i] + (byte + first < top ? byte + first : top));
          p.a[i][1] = *reinterpret_cast<const v4u*>(pa[i] + (byte + second < top ? byte + second : top));
          p.a_scale[i] = a_scale[i][group];
        }
        p.b_scale = b_scale[at * g.b_scale_step];
#pragma unroll
        for (int j = 0; j < NF; ++j) {
          p.b[j][0] = *reinterpret_cast<const v4u*>(pb[j] + byte + first);
          p.b[j][1] = *reinterpret_cast<const v4u*>(pb[j] + byte + second);
        }
      } else {
        const int64_t k = at * kDepth + first / 2;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int i = 0; i < MF; ++i) p.a[i][e] = load8_row(reinterpret_cast<const uint16_t*>(pa[i]), k + 8 * e, g.k);
#pragma unroll
          for (int j = 0; j < NF; ++j) p.b[j][e] = load8_row(reinterpret_cast<const uint16_t*>(pb[j]), k + 8 * e, g.k);
        }
      }
    };
    auto multiply = [&](const Piece& p) {  // rows of the sums: b's, columns: a's
#pragma unroll
      for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j) {
          v4f& c = acc[i][j];
          if constexpr (KIND == kEight) {
            typedef unsigned int v8u __attribute__((ext_vector_type(8)));
            const v8u a = __builtin_shufflevector(p.a[i][0], p.a[i][1], 0, 1, 2, 3, 4, 5, 6, 7);
            const v8u b = __builtin_shufflevector(p.b[j][0], p.b[j][1], 0, 1, 2, 3, 4, 5, 6, 7);
            c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(__builtin_bit_cast(v8i, b), __builtin_bit_cast(v8i, a), c, 0, 0, 0,
                                                                 p.b_scale, 0, p.a_scale[i]);
          } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if constexpr (KIND == ZS_BF16)
                c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, p.b[j][e]), __builtin_bit_cast(v8bf, p.a[i][e]), c,
                                                            0, 0, 0);
              else
                c = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8hf, p.b[j][e]), __builtin_bit_cast(v8hf, p.a[i][e]), c, 0,
                                                           0, 0);
            }
          }
        }
    };
    const int64_t pieces = (g.k + kDepth - 1) / kDepth, whole = KIND == kEight ? g.a_padded / 128 : g.k / kDepth;
    int64_t at = wave;
    Piece p[kAhead];
    for (; at + (kAhead - 1) * kWaves < whole; at += kAhead * kWaves) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) fetch(at + u * kWaves, p[u]);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) multiply(p[u]);
    }
    for (; at < pieces; at += kWaves) {
      if (at < whole) fetch(at, p[0]);
      else fetch_last(at, p[0]);
      multiply(p[0]);
    }
  }
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j) sums[wave][i * NF + j][lane] = acc[i][j];
  __syncthreads();
  if (wave >= MF * NF) return;
  v4f sum = sums[0][wave][lane];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) sum += sums[w][wave][lane];
  // a lane has four consecutive columns of one of c's rows
  const int m = wave / NF * 16 + row;
  const int64_t n = n0 + wave % NF * 16 + part * 4, at = (m0 + m) * g.c_stride + n;
  if (m >= left_m) return;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if (n + r >= g.n) break;
    uint16_t* c = static_cast<uint16_t*>(g.c) + at + r;
    *c = static_cast<uint16_t>(g.c_dt == ZS_BF16 ? half_bits<ZS_BF16>(sum[r]) : half_bits<ZS_FP16>(sum[r]));
  }
}

template <int KIND, int MF>
hipError_t launch_few_rows(const ProductArgs& a, hipStream_t s) {
  const bool wide = product_units(a, false, 16 * MF, 32) >= 512;
  const int64_t units = product_units(a, false, 16 * MF, wide ? 32 : 16);
  constexpr int kWaves = 8;
  auto kernel = wide ? &k_few<KIND, MF, 2, kWaves> : &k_few<KIND, MF, 1, kWaves>;
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(launch_units(units, kXcdWhole))), dim3(kWaves * 64), 0, s, a);
  return hipGetLastError();
}

template <int KIND>
hipError_t launch_few(const ProductArgs& a, hipStream_t s) {
  return a.m <= 16 * int64_t(a.groups) ? launch_few_rows<KIND, 1>(a, s) : launch_few_rows<KIND, 2>(a, s);
}

// Whether k_few is the better way: past some 512 units its time goes with their number, while the tiles' time
// stays that of one tile's stages (0.65 us each) as long as there are no more tiles than CUs.  Both go with k
// alike, so the rule asks for the units alone.  Measured, us of k_few
// and of tiles: 8 bits 64 x 4096 -> 4096 (256 units) 18 and 22, 128 rows (512) 22 and 22, 256 (1024) 39 and 23;
// 128 x 14336 -> 4096 (512) 72 and 80, 256 (1024) 137 and 80; 512 x 1003 -> 517 (272) 8 and 12, 1024 (544) 11 and
// 12; 512 x 512 -> 2048 (1024) 9 and 9.  16 bits: one expert 64 x 4096 -> 4096 (384) 26 and 37, 128 (640) 34 and
// 38, 256 (1152) 63 and 39; 16 experts 512 x 4096 -> 448 (448) 29 and 37, 1024 (672) 41 and 38; 128 x 448 -> 4096
// (2560) 18 and 13; 256 x 1024 -> 1024 (768) 10 and 13, 1024 (1536) 21 and 15.  So it is off by up to 40 % between
// 512 and 1200 units of few stages or with many experts of few rows, which add a unit each.
bool few_rows(const ProductArgs& a) { return product_units(a, false, 32, 32) <= kFewUnits; }

using SmallTile = Tile<2, 2, 2, 2, 2>;  // 128 x 128, two workgroups to a CU
using LargeTile = Tile<2, 4, 4, 2, 2>;  // 256 x 256, one workgroup to a CU

// From how many large tiles on they are taken: below, too many CUs have none.  Measured, us with large and
// with small tiles, at any length of the sum alike.  8 bits, 2048, 3000 and 4096 rows (128, 192, 256 large tiles):
// 1024 -> 4096 22 and 15, 23 and 24, 23 and 27; 4096 -> 4096 52 and 39, 54 and 63, 60 and 72; 14336 -> 4096 146 and
// 109, 156 and 184, 178 and 215.  16 bits, one expert, the same rows: 448 -> 4096 19 and 13, 19 and 21, 21 and 25;
// 4096 -> 4096 71 and 64, 84 and 101, 102 and 125.  16384 rows over 16 experts of 4096 x 448: y (160) 74 and 64, dx
// (1280) 78 and 92, dw (512) 64 and 83; 8 of 1024 x 1024: y (288) 33 and 40, dw (128) 41 and 38; 7811 over 18 of
// 3200 x 4096: y (784) 226 and 263.  An expert's last tile counts as a whole one though half of it may be empty:
// 16384 rows over 64 experts of 1024 x 512 (256) take 27 and 22.
constexpr int64_t kLargeUnits = 192;

// ------------------------------------------------------------------ launch choices

template <int KIND, bool AK, bool BK, bool SUM_GROUPS, bool STAGED, class TL>
hipError_t launch_tile(const ProductArgs& a, hipStream_t s) {
  auto kernel = &k_product<KIND, AK, BK, SUM_GROUPS, STAGED, TL>;
  constexpr int kLds = TL::lds(KIND == kEight);
  if (kLds > 65536) {
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
    if (e != hipSuccess) return e;
  }
  const int64_t units = product_units(a, SUM_GROUPS, TL::kM, TL::kN);
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(launch_units(units, kXcdWhole))), dim3(TL::kThreads), kLds, s, a);
  return hipGetLastError();
}

// Whether an operand's stages can go straight to LDS: pieces at addresses of whole words, which such a
// load takes (7811 x 3156 -> 4096 over 18 experts 306 us, 520 through registers), offsets within a tile
// of 32 bits; by k also whole pieces at a row's end.
bool direct_rows(const void* p, int64_t stride, int64_t group) {
  return (reinterpret_cast<uintptr_t>(p) & 3) == 0 && stride % 2 == 0 && group % 2 == 0 && stride < (1 << 22);
}

template <int KIND, bool AK, bool BK, bool SUM_GROUPS>
hipError_t launch_sizes(const ProductArgs& a, hipStream_t s) {
  if constexpr (!AK && !BK && !SUM_GROUPS) {
    if (few_rows(a)) return launch_few<KIND>(a, s);
  }
  const bool direct = direct_rows(a.a, a.a_stride, 0) && direct_rows(a.b, a.b_stride, a.b_group) && (!AK || a.m % 8 == 0) &&
                      (!BK || a.n % 8 == 0);
  if (!direct) return launch_tile<KIND, AK, BK, SUM_GROUPS, true, SmallTile>(a, s);
  const int64_t per_group = SUM_GROUPS ? a.m : a.m / std::max(1, a.groups);
  if (per_group >= 192 && a.n >= 192 && product_units(a, SUM_GROUPS, LargeTile::kM, LargeTile::kN) >= kLargeUnits)
    return launch_tile<KIND, AK, BK, SUM_GROUPS, false, LargeTile>(a, s);
  return launch_tile<KIND, AK, BK, SUM_GROUPS, false, SmallTile>(a, s);
}

}  // namespace

int64_t product_units(const ProductArgs& a, bool sum_groups, int64_t tile_m, int64_t tile_n) {
  const int64_t tn = (a.n + tile_n - 1) / tile_n;
  if (sum_groups) return a.groups * ((a.m + tile_m - 1) / tile_m) * tn;
  // every group may end with a part of a tile
  return ((a.m + tile_m - 1) / tile_m + (a.ends != nullptr ? a.groups : 0)) * tn;
}

hipError_t launch_product8(const ProductArgs& a, hipStream_t s) {
  if (few_rows(a)) return launch_few<kEight>(a, s);
  if (product_units(a, false, LargeTile::kM, LargeTile::kN) >= kLargeUnits)
    return launch_tile<kEight, false, false, false, false, LargeTile>(a, s);
  return launch_tile<kEight, false, false, false, false, SmallTile>(a, s);
}

hipError_t launch_expert_product(const ProductArgs& a, int dt, bool in_major, hipStream_t s) {
  if (dt == ZS_BF16)
    return in_major ? launch_sizes<ZS_BF16, false, true, false>(a, s) : launch_sizes<ZS_BF16, false, false, false>(a, s);
  return in_major ? launch_sizes<ZS_FP16, false, true, false>(a, s) : launch_sizes<ZS_FP16, false, false, false>(a, s);
}

hipError_t launch_expert_wgrad(const ProductArgs& a, int dt, hipStream_t s) {
  return dt == ZS_BF16 ? launch_sizes<ZS_BF16, true, true, true>(a, s) : launch_sizes<ZS_FP16, true, true, true>(a, s);
}

// ------------------------------------------------------------------ weights in 8 bits

namespace {

// The codes of a weight, its transposed codes and its scales, one 128 x 128 block to a workgroup.  A
// thread holds two patches of four rows by eight columns, so that the four codes of a column leave
// as one word of the transposed block, which is turned in LDS.  Bound by memory: 14336 x 4096 in
// bf16 takes 42 us (5.6 TB/s), past the caches; 48 through them.
template <int DT>
__global__ __launch_bounds__(256) void k_weight8(const void* src, int64_t stride, int64_t outs, int64_t cols, uint8_t* codes,
                                                 uint8_t* codes_t, uint8_t* scales, int64_t blocks_n) {
  __shared__ __attribute__((aligned(16))) uint32_t turned[128 * 36];  // a column's 128 codes at a pitch of 144 bytes
  __shared__ uint32_t tops[4];
  const int64_t bo = blockIdx.x / blocks_n, bc = blockIdx.x % blocks_n;
  const int64_t pc = blocks_n * 128, pr = (outs + 127) / 128 * 128;
  const int patch_c = threadIdx.x % 16, patch_r = threadIdx.x / 16;  // rows patch_r * 4 and 64 + patch_r * 4
  const int64_t col = bc * 128 + patch_c * 8;
  const int64_t left = cols - col;
  const int cnt = left >= 8 ? 8 : left > 0 ? static_cast<int>(left) : 0;
  float f[2][4][8];
  float top = 0.0f;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int64_t row = bo * 128 + h * 64 + patch_r * 4 + r;
      const int n = row < outs ? cnt : 0;
      if constexpr (DT == ZS_FP32) {
        const float* p = static_cast<const float*>(src) + row * stride + col;
        if (n == 8) {
          const v4u x = *reinterpret_cast<const v4u_a4*>(p), y = *reinterpret_cast<const v4u_a4*>(p + 4);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            f[h][r][j] = bits_f(x[j]);
            f[h][r][4 + j] = bits_f(y[j]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) f[h][r][j] = j < n ? p[j] : 0.0f;
        }
      } else {
        widen8<DT>(load8h_nt(static_cast<const uint16_t*>(src) + row * stride + col, n), f[h][r]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) top = __builtin_elementwise_maximum(top, fabsf(f[h][r][j]));  // a NaN wins
    }
  uint32_t m = f_bits(top) & 0x7FFFFFFFu;
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const uint32_t o = __shfl_xor(m, d);
    m = o > m ? o : m;
  }
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 4; ++w) m = tops[w] > m ? tops[w] : m;
  const int b = scale_byte<ZS_E4M3>(m);
  if (threadIdx.x == 0) scales[bo * blocks_n + bc] = static_cast<uint8_t>(b);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    v2u c[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      c[r] = encode8<ZS_E4M3>(f[h][r], b);
      const int64_t row = bo * 128 + h * 64 + patch_r * 4 + r;
      if (row < outs) __builtin_nontemporal_store(c[r], reinterpret_cast<v2u*>(codes + row * pc + col));
    }
    if (codes_t != nullptr) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t w = 0;
#pragma unroll
        for (int r = 0; r < 4; ++r) w |= ((c[r][j >> 2] >> (j % 4 * 8)) & 0xFFu) << (8 * r);
        turned[(patch_c * 8 + j) * 36 + h * 16 + patch_r] = w;
      }
    }
  }
  if (codes_t == nullptr) return;
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int id = q * 256 + threadIdx.x, row = id / 8, at = id % 8;
    const int64_t c = bc * 128 + row;
    if (c < cols)
      __builtin_nontemporal_store(*reinterpret_cast<const v4u*>(turned + row * 36 + at * 4),
                                  reinterpret_cast<v4u*>(codes_t + c * pr + bo * 128 + at * 16));
  }
}

}  // namespace

hipError_t launch_weight8(const void* src, int dt, int64_t stride, int64_t outs, int64_t cols, uint8_t* codes, uint8_t* codes_t,
                          uint8_t* scales, hipStream_t s) {
  const int64_t blocks_n = (cols + 127) / 128, blocks = (outs + 127) / 128 * blocks_n;
  if (blocks == 0) return hipSuccess;
  auto kernel = dt == ZS_BF16 ? &k_weight8<ZS_BF16> : dt == ZS_FP16 ? &k_weight8<ZS_FP16> : &k_weight8<ZS_FP32>;
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, src, stride, outs, cols, codes, codes_t, scales,
                     blocks_n);
  return hipGetLastError();
}

}  // namespace zs
