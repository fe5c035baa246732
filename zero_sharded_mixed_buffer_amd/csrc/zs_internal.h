// Internal declarations shared by the host planner / ABI (zs_abi.cpp) and the gfx950
// kernels (zs_kernels.hip).  Not part of the public C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zs.h"

namespace zs {

// Streaming-kernel geometry.  Every streaming kernel launches one workgroup of 256 threads
// (four wave64s) per unit of work - no persistent grid-stride loops, which measured slower
// on MI355X for these pure streams.  A thread owns groups of 8 consecutive flat elements
// (one 16-byte access of 2-byte data, two of fp32), and every kernel covers one
// 4096-element tile per workgroup: kUnroll groups per thread in the unpack kernel, two in
// the pack and check passes (kPackBlock, which also leave one fp64 partial sum per
// workgroup), and the same elements regrouped as four-element quads in the AdamW kernel.
constexpr int kThreads = 256;
constexpr int kGroup = 8;
constexpr int kUnroll = 2;
constexpr int64_t kTile = int64_t(kThreads) * kGroup * kUnroll;
constexpr int64_t kPackBlock = int64_t(kThreads) * kGroup * 2;
constexpr int kLevel2 = 1024;  // first-level partial-sum workgroups of the two-level reduction
// A shard of at most this many tiles runs the AdamW kernel with four workgroups per tile.
constexpr int64_t kSplitTiles = 256;

// XCD-aware work order.  The dispatcher deals consecutive workgroups to the eight XCDs in
// turn.  Run length R: 0 keeps that order (XCD x gets every eighth unit); R > 0 gives each
// XCD runs of R consecutive units (the units of each group of 8R are dealt as eight runs);
// kXcdWhole gives each XCD one contiguous eighth of the range.
constexpr int kXcds = 8;
constexpr int64_t kXcdWhole = -1;
constexpr int64_t kXcdRunAdamw = 16;
constexpr int64_t kXcdRunPack = kXcdWhole;
constexpr int64_t kXcdRunCheck = kXcdWhole;
constexpr int64_t kXcdRunUnpack = kXcdWhole;
// Workgroups launched for `units` units of work in the order of run length `run`.
inline int64_t launch_units(int64_t units, int64_t run) {
  if (run == 0) return units;
  const int64_t group = kXcds * (run > 0 ? run : 1);
  return (units + group - 1) / group * group;
}

// Workgroups (and partial sums) of a pack or check pass over len elements.
__host__ __device__ inline int64_t reduction_blocks(int64_t len) { return (len + kPackBlock - 1) / kPackBlock; }

// Segment map of one flat range (a rank's shard or the whole buffer), in device memory.
// Segment i covers range-relative [seg_begin[i], seg_begin[i+1]) and lies inside tensor
// seg_tensor[i] (-1: alignment gap or tail padding) starting at element seg_local[i] of it.
// tile_first[k] is the segment holding the first element of tile k (k < ntiles) and
// tile_first[ntiles] = nseg - 1, so the segments meeting tile k are
// tile_first[k] .. tile_first[k+1].
struct DevMap {
  const int64_t* seg_begin;   // nseg + 1 entries, last = len
  const int64_t* seg_local;   // nseg
  const int32_t* seg_tensor;  // nseg
  const int32_t* tile_first;  // ntiles + 1
  const uint8_t* seg_nodecay;  // nseg flags (1: the segment's tensor takes no weight decay), or null
  int64_t len;
  int64_t ntiles;
  int32_t nseg;
};

// Device-resident state: the public host struct followed by internal scratch.
struct DevState {
  zs_state_host h;
  double raw_sumsq;  // sum of squares of the (still scaled) shard, fixed order
  double pad_;
};

// Per-step AdamW hyper-parameters passed by value to the kernel.
struct AdamwArgs {
  double lr, beta1, beta2, eps, weight_decay;
};

enum FlagMode : int { kFlagSet = 0, kFlagOr = 1 };

// Launchers (zs_kernels.hip).  Each enqueues on `s` and returns the launch status.
// launch_pack / launch_check write reduction_blocks(len) partial sums when partials != null;
// launch_reduce_finalize folds n partials (via level2 scratch of kLevel2 doubles when n is
// large) into the state's flag and local sum of squares.
// launch_pack covers flat elements [lo, hi) of the map's range (hi < 0: to its end).
hipError_t launch_pack(const DevMap& map, const uint64_t* src_ptrs, int src_dt, void* dst, int dst_dt, bool accumulate,
                       double* partials, hipStream_t s, int64_t lo = 0, int64_t hi = -1);
hipError_t launch_check(const void* shard, int64_t n, int dt, double* partials, hipStream_t s);
hipError_t launch_reduce_finalize(const double* partials, int64_t nparts, double* level2, DevState* st,
                                  const int32_t* ext, int mode, double* local_out, hipStream_t s);
hipError_t launch_norm_finalize(DevState* st, const double* rank_sumsq, int dp_world, int dp_rank,
                                double* local_out, double max_norm, hipStream_t s);
// The single-rank step's finalizers in one launch (after the same first-level fold as
// launch_reduce_finalize): flag and local sum of squares (set mode, no other ranks), norm
// and clip coefficient, a copy of the state to `pre`, then the scaler commit.  The AdamW
// launch of that step takes `pre` as its state.
hipError_t launch_step_finalize(const double* partials, int64_t nparts, double* level2, DevState* st,
                                DevState* pre, double max_norm, hipStream_t s);
// The allocation-free step (zs_step_flat_noalloc): its finalize reads and commits a bare
// zs_state_host in the caller's memory, and its workspace is a fixed device array of the
// library, one per GPU, holding kNoAllocMaxParts first-level partial sums: check passes of
// at most kNoAllocMaxParts * kPackBlock elements.
constexpr int64_t kNoAllocMaxParts = int64_t(1) << 21;
constexpr int kMaxDevices = 64;
struct NoAllocScratch {
  DevState* pre;
  double* level2;    // kLevel2 slots
  double* partials;  // kNoAllocMaxParts slots
};
// The calling thread's current device's scratch (its address is looked up once per device).
hipError_t noalloc_scratch(NoAllocScratch* out);
hipError_t launch_step_finalize_ext(const double* partials, int64_t nparts, double* level2, zs_state_host* st,
                                    DevState* pre, double max_norm, hipStream_t s);
hipError_t launch_adamw(const DevMap& map, const void* shard, int grad_dt, float* master, float* m, float* v,
                        const AdamwArgs& hp, const DevState* st, const uint64_t* param_ptrs, void* flat_out,
                        int param_dt, hipStream_t s);
hipError_t launch_unpack(const DevMap& map, const void* src, int src_dt, const uint64_t* dst_ptrs, int dst_dt,
                         const DevState* skip, hipStream_t s);
hipError_t launch_scaler_update(DevState* st, hipStream_t s);

// Bandwidth yardsticks (zs_probe.hip); sizes already checked: n a multiple of kTile, bytes a
// multiple of 4 * kTile.
hipError_t launch_probe_mix(const void* g, float* p, float* m, float* v, void* out, int64_t n, hipStream_t s);
hipError_t launch_probe_copy(const void* src, void* dst, int64_t bytes, hipStream_t s);
hipError_t launch_probe_read(const void* src, int64_t bytes, uint32_t* sink, hipStream_t s);
hipError_t launch_probe_write(void* dst, int64_t bytes, hipStream_t s);

// Activation operators (zs_act.hip, zs_wgrad.hip); every argument already checked.  A matrix
// is a base pointer and a row stride in elements.
struct Act {  // checkpoint arrays; code is a zs_code
  uint8_t* codes;
  uint8_t* scales;
  int code;
};
constexpr int64_t kActPad = 32;           // codes per row are a multiple of this
constexpr int64_t kNormMaxCols = 16384;   // 1024 threads with two chunks of eight columns each
__host__ __device__ inline int64_t act_padded(int64_t cols) { return (cols + kActPad - 1) / kActPad * kActPad; }
// Rows of one launch of the norm (its workgroups hold fewer than 2^32 threads).
int64_t rmsnorm_max_rows(int64_t cols);
// Eight-element chunks of one pack or unpack launch (four per thread, < 2^32 threads).
constexpr int64_t kActMaxChunks = ((int64_t(1) << 32) - 256) * 4;

hipError_t launch_act_pack(const void* src, int dt, int64_t stride, int64_t rows, int64_t cols, const Act& act,
                           hipStream_t s);
hipError_t launch_act_unpack(const Act& act, int64_t rows, int64_t cols, void* dst, int dt, int64_t stride,
                             hipStream_t s);

struct NormArgs {
  const uint16_t* x;
  const uint16_t* residual;  // or null
  const uint16_t* weight;
  uint16_t* h;  // or null
  uint16_t* y;  // or null
  float* rstd;  // or null
  int64_t x_stride, residual_stride, h_stride, y_stride;
  Act y8, h8;  // codes null: none
  int64_t rows;
  int32_t cols;
  double eps;
};
hipError_t launch_rmsnorm(const NormArgs& a, int dt, hipStream_t s);

struct NormBackwardArgs {
  const uint16_t* dy;
  const uint16_t* dh;  // or null
  const uint16_t* h;   // or null: h8
  Act h8;
  const uint16_t* weight;
  const float* rstd;
  uint16_t* dx;
  int64_t dy_stride, dh_stride, h_stride, dx_stride;
  int64_t rows;
  int32_t cols;
  void* dweight;  // or null
  const void* base;  // or null
  int dweight_dt;
  float* partials;  // rmsnorm_partials(rows, cols) rows of round_up(cols, 8) sums
};
// Workgroups of the backward pass, each leaving one row of partial weight-gradient sums.
int64_t rmsnorm_partials(int64_t rows, int64_t cols);
hipError_t launch_rmsnorm_backward(const NormBackwardArgs& a, int dt, hipStream_t s);

struct WgradArgs {
  Act x8;
  const uint16_t* dy;
  void* dw;
  const void* base;  // or null
  float* partials;
  int64_t rows, cols, outs, dy_stride, dw_stride;
  int dy_dt, dw_dt;
  bool in_major;
};
int64_t wgrad_workspace(int64_t rows, int64_t cols, int64_t outs);  // bytes; < 0: past one launch
hipError_t launch_wgrad(const WgradArgs& a, hipStream_t s);

// Products (zs_product.hip): c[m][n] = base + sum over k of a[m][k] * b[n][k], over groups of m
// (each with a b of its own) or of k (each with a c of its own).  Strides in elements.
struct ProductArgs {
  const void* a;
  const void* b;
  void* c;
  const void* base;         // or null
  const uint8_t* a_scales;  // of 8-bit operands
  const uint8_t* b_scales;
  const int32_t* ends;  // the groups' ends, or null: one group
  int64_t m, n, k;
  int64_t a_stride, b_stride, c_stride, b_group, c_group;
  int64_t a_padded, b_padded;  // codes of a row of 8-bit operands
  int64_t b_scale_row, b_scale_step;  // from one of b's blocks to the next, along its rows and along k
  int32_t groups;
  int32_t c_dt;
  bool zero_rest;  // rows behind the last group become zeros
};
// Workgroups of a launch with such tiles.
int64_t product_units(const ProductArgs& a, bool sum_groups, int64_t tile_m, int64_t tile_n);
constexpr int64_t kProductMaxUnits = (int64_t(1) << 23) - 64;  // workgroups of 512 threads of one launch
constexpr int64_t kProductTile = 128;                          // the smallest tile's sides
hipError_t launch_product8(const ProductArgs& a, hipStream_t s);
hipError_t launch_expert_product(const ProductArgs& a, int dt, bool in_major, hipStream_t s);
hipError_t launch_expert_wgrad(const ProductArgs& a, int dt, hipStream_t s);
constexpr int64_t kWeightBlock = 128;
constexpr int64_t kWeight8MaxSide = int64_t(1) << 23;  // 256 rows of codes within 32-bit offsets
hipError_t launch_weight8(const void* src, int dt, int64_t stride, int64_t outs, int64_t cols, uint8_t* codes, uint8_t* codes_t,
                          uint8_t* scales, hipStream_t s);

// Routing (zs_expert.hip).
constexpr int kRouteChunk = 1024;     // choices of a workgroup
constexpr int64_t kMaxExperts = 1024;
constexpr int64_t kMaxSlots = (int64_t(1) << 31) - 4096;
struct RouteArgs {
  const void* ids;
  int32_t* ends;
  int32_t* slot;
  int32_t* place;
  int32_t* totals;  // workspace: experts + 1, then as many for each chunk
  int32_t* counts;
  int64_t slots, chunks;
  int32_t experts, id_bytes, bits;
};
int64_t route_workspace(int64_t slots, int experts);
hipError_t launch_route(RouteArgs a, void* workspace, hipStream_t s);
struct RowsArgs {
  const void* x;
  void* out;
  const int32_t* slot;   // the gather's
  const int32_t* place;  // the combination's
  const float* weights;  // or null: ones
  int64_t rows, cols, x_stride, out_stride;  // rows: tokens * choices
  int32_t choices, rows_log2;
};
// Workgroups of the gather's launch over rows, or the combination's over tokens.
int64_t expert_row_blocks(int64_t rows, int64_t cols, int dt);
constexpr int64_t kExpertMaxBlocks = (int64_t(1) << 24) - 1;  // of 256 threads: a launch holds fewer than 2^32
hipError_t launch_expert_gather(RowsArgs a, int dt, hipStream_t s);
hipError_t launch_expert_combine(RowsArgs a, int dt, hipStream_t s);
struct CombineBackwardArgs {
  const void* dout;
  const void* y;         // or null: no dweights
  const int32_t* slot;
  const int32_t* place;
  const float* weights;  // or null: ones
  void* dy;              // or null
  float* dweights;       // or null
  int64_t rows, cols, dout_stride, y_stride, dy_stride;
  int32_t choices, rows_log2;
};
hipError_t launch_expert_combine_backward(CombineBackwardArgs a, int dt, hipStream_t s);

}  // namespace zs
