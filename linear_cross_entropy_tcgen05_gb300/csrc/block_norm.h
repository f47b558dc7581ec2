// block_norm.h -- parameter block and launchers of the block norm (norms after and before a
// transformer block fused with its gate and residual scale). Not part of the public ABI.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace flce {

// A row is worked on by threads of eight columns each, all in one block where they fit, beyond
// that the blocks of a cluster (up to 8) share the row.
constexpr int kBnMaxThreads = 640;
constexpr int kBnMaxCluster = 8;
constexpr int kBnSmemBytes = 220 << 10;  // shared memory for parameters and rows on their way in
constexpr int64_t kBnMaxD = 16384;

struct BlockNormShape {
  int cluster;          // blocks that share a row
  int threads_per_row;  // in one block; a multiple of 32
  int rows_per_block;   // row groups of a block, each with rows of its own
};

struct BlockNormParams {
  const void *x, *residual, *gate, *w1, *b1, *w2, *b2;  // 1: after the block, 2: before the next
  void *h, *y;
  float* stats;  // [N][4] mean1, rstd1, mean2, rstd2; null: not kept
  int64_t ld_x, ld_residual, ld_gate;
  int64_t N;
  int D;
  int64_t gate_group;  // rows per gate row
  int w1_dt, b1_dt, w2_dt, b2_dt;
  int gate_res_type;   // the gate has the residual's type (else x's)
  int act, layer;
  float eps, scale, w_off;
  // rows of a worker (row group), forward and backward
  int64_t chunk_rows;
  // backward
  const void *h_in, *dh, *dy;
  int64_t ld_dh, ld_dy;
  void *dx, *dres, *dgate;
  int64_t chunks, chunks_per_group, group_rows;  // chunks never cross a gate group
  int gate_full;                                 // a gate row for each row: dgate is written row by row
  // Partial sums of dw1, db1, dw2, db2 [blocks][D], or null; with gate groups the first two have a
  // row for each worker.
  float* part[4];
  float* part_gate;  // [chunks][D], or null (dgate written directly when a group is one chunk)
};

// What the code of a kernel has: the norm after the block, a gate (for groups of rows, or GATE_ROWS:
// for each row), and (FULL) the means of layer norms and biases. A kernel takes what has less at
// run time. WIDE: blocks of up to 640 threads. Sets without POST have kernels of their own for the backward's
// sake (N = 32768, D = 4096 bf16, without a norm after the block, own kernels and those with POST: layer
// norms 245 and 310 us, with gates for groups 273 and 359, with a gate for each row 364 and 617, RMS norms
// with one 344 and 373; forward 201 and 207, 208 and 213, 252 and 256, 232 and 218).
enum BnFeature : int { BN_POST = 1, BN_GATE = 2, BN_FULL = 4, BN_GATE_ROWS = 8, BN_WIDE = 16 };
// Threads of a block at most. 640 leave 96 registers for each: enough for the forward kernels
// of aligned rows in one block (the others would spill), but those with FULL are slower for it
// (N = 32768, D = 2048 bf16, layer norms, 16 gates: 147 us against 126), so they come in both.
constexpr int kBnThreads = 512;
__host__ __device__ constexpr int bn_max_threads(int feat, bool vec, bool clusters) {
  return vec && !clusters && (!(feat & BN_FULL) || (feat & BN_WIDE)) ? kBnMaxThreads : kBnThreads;
}
// Parameters that a kernel keeps in shared memory (the others have room for theirs in registers).
__host__ __device__ constexpr int bn_shared_params(int feat, bool backward) {
  if (!(feat & BN_FULL)) return 0;
  if (!backward) return 4;
  return feat & BN_POST ? 2 : 1;
}
// Values that each thread of a backward kernel keeps there for itself: a bias's sum, or both and a
// gate (with all of them in registers the kernel spills, to local memory for which there is
// no L1 left: 386 us against 210 at N = 16384, D = 2304).
__host__ __device__ constexpr int bn_own_params(int feat, bool backward) {
  if (!backward || !(feat & BN_POST) || !(feat & BN_FULL)) return 0;
  return feat & BN_GATE ? 3 : 1;
}

// Rows that a row group works on together at most: they share the latency of their sums. (Four in
// the forward pass measured slower: their copies come in bursts that leave the memory idle
// between them, N = 65536, D = 4096 bf16: 537 us against 431.)
constexpr int kBnRows = 2;
constexpr int kBnMaxBatches = 6;

// 16-byte planes a thread of one row: x and the residual, or x, dy, h and dh, and a full gate.
constexpr int bn_planes(int x_bytes, int residual_bytes, bool gate_full, bool backward) {
  return (x_bytes + residual_bytes) / 2 * (backward ? 2 : 1) + (gate_full ? residual_bytes / 2 : 0);
}

// Batches of rows on their way in: as many as fit beside the parameters, of one row where there
// is no room for two batches of two. At least two are needed: one in work, one landed.
struct BnRing {
  int per, batches, params_bytes;
};
// Bytes of a row of a ring. Unaligned rows have 16 bytes more for each warp's plane.
constexpr int kBnWarpPlane = 33 * 16;
constexpr int bn_row_bytes(int threads, int planes, bool vec) { return planes * (vec ? 16 * threads : threads / 32 * kBnWarpPlane); }
constexpr BnRing bn_ring(const BlockNormShape& s, int planes, bool vec, int feat, bool backward) {
  const int threads = s.threads_per_row * s.rows_per_block;
  BnRing r{kBnRows, 1, bn_shared_params(feat, backward) * 32 * s.threads_per_row + bn_own_params(feat, backward) * 32 * threads};
  const int room = kBnSmemBytes - r.params_bytes, row = bn_row_bytes(threads, planes, vec);
  if (room / (row * r.per) < 2) r.per = 1;
  r.batches = room / (row * r.per);
  if (r.batches > kBnMaxBatches) r.batches = kBnMaxBatches;
  return r;
}

// Bytes from a line of shared memory to the ring's first row. Half a line for the forward of two RMS norms over
// 16-bit rows alone: its copies take a line more each (which likely paces reads among writes; N = 65536,
// D = 4096: 361 us with none, 336 with 16 bytes, 357 with 48, 324 with 64; N = 32768, D = 5120: 228 and 204; up
// to D = 2048 the same). Other forward kernels lose by it (gates for each row 214 and 224 us, layer norms with
// gates 276 and 289) or nothing (fp32 rows), the backward 12%.
__host__ __device__ constexpr int bn_ring_shift(int x_bytes, int residual_bytes, bool vec, int feat, int cluster, bool backward) {
  return !backward && vec && cluster == 1 && feat == BN_POST && x_bytes == 2 && residual_bytes == 2 ? 64 : 0;
}

// The features of the kernel that a call with these takes: unaligned rows, and rows shared by
// clusters unless they have RMS norms alone, take the kernel that has everything, and so do wide
// blocks of the FULL ones.
constexpr int bn_kernel_features(int feat, bool vec, int cluster, bool wide) {
  const int all = feat & BN_GATE_ROWS ? BN_POST | BN_GATE | BN_FULL | BN_GATE_ROWS : BN_POST | BN_GATE | BN_FULL;
  if (wide && (feat & BN_FULL)) return all | BN_WIDE;
  return !vec || (cluster > 1 && (feat & (BN_GATE | BN_FULL))) ? all : feat;
}

// One for each pair of types (x's, then the residual's) and direction, each in a file of its own.
#define FLCE_BN_ENTRY(NAME) \
  cudaError_t NAME(const BlockNormParams& p, const BlockNormShape& s, bool vec, int feat, unsigned blocks, cudaStream_t stream)
FLCE_BN_ENTRY(bn_forward_bf16_bf16);
FLCE_BN_ENTRY(bn_backward_bf16_bf16);
FLCE_BN_ENTRY(bn_forward_bf16_f32);
FLCE_BN_ENTRY(bn_backward_bf16_f32);
FLCE_BN_ENTRY(bn_forward_f16_f16);
FLCE_BN_ENTRY(bn_backward_f16_f16);
FLCE_BN_ENTRY(bn_forward_f16_f32);
FLCE_BN_ENTRY(bn_backward_f16_f32);
FLCE_BN_ENTRY(bn_forward_f32_f32);
FLCE_BN_ENTRY(bn_backward_f32_f32);
#undef FLCE_BN_ENTRY

// out[s][j] = sum over rows of segment s of part[s * rows + r][j], for up to five arrays.
struct BnSum {
  const float* part;
  void* out;
  int64_t segments, rows;
  int dt;
};
struct BnSums {
  BnSum a[5];
  int n, D;
};
cudaError_t bn_column_sums(const BnSums& s, cudaStream_t stream);

}  // namespace flce
