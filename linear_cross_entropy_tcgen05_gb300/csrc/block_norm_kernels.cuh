// block_norm_kernels.cuh -- forward and backward kernels of the block norm.
//
//   u = x, or Norm(x; w1, b1)           h = residual + s act(gate) u          y = Norm(h; w2, b2)
//   Norm(v) = (v - mean) rstd (w + w_off) + b, mean = 0 for the RMS norm.
//
// Both passes are bound by memory: the forward reads x and the residual and writes h and y,
// the backward reads x, h, dh, dy and writes dx and the residual's gradient. A thread owns
// eight columns of every row that its row group works on, so each element is read once, stays
// in registers through the row's reductions, and the parameters and the sums of their
// gradients stay in registers from row to row. A block writes one partial sum for each
// parameter; a second kernel adds them in a fixed order, so the gradients do not depend on
// timing. Statistics and sums are in 32 bits; h and y are rounded once, y from the 32-bit h.
#pragma once

#include "block_norm.h"
#include "elem_io.cuh"
#include "flce_internal.h"
#include "sm103_ptx.cuh"

namespace flce {
namespace {

// Sums over the threads of a row. Two scratch buffers take turns, so one barrier a sum is
// enough: a buffer is written again only after the barrier of the sum between.
struct RowSum {
  float* buf;      // [2][kWords] of this row group
  float* clus;     // [2][kBnMaxCluster][2] of this block
  int nw, warp, lane, bar, threads, cluster, turn;
  static constexpr int kWords = 2 * kBnMaxThreads / 32;

  template <int NV> __device__ __forceinline__ void sum(float (&v)[NV]) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if (nw > 1) {
      float* b = buf + turn * kWords;
      if (lane == 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) b[warp * NV + i] = v[i];
      }
      named_barrier_sync(uint32_t(bar), uint32_t(threads));
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = 0.f;
      const int n4 = (nw * NV + 3) / 4;
      for (int w = 0; w < n4; ++w) {
        const float4 q = reinterpret_cast<const float4*>(b)[w];
        const int left = nw * NV - 4 * w;  // words past the last warp hold another sum's values
        if constexpr (NV == 1) {
          v[0] += (q.x + (left > 1 ? q.y : 0.f)) + ((left > 2 ? q.z : 0.f) + (left > 3 ? q.w : 0.f));
        } else {
          v[0] += q.x + (left > 2 ? q.z : 0.f);
          v[1] += q.y + (left > 2 ? q.w : 0.f);
        }
      }
    }
    if (cluster > 1) {
      float* c = clus + turn * (2 * kBnMaxCluster);
      const int tid = warp * 32 + lane;
      if (tid < cluster) {
        const uint32_t at = map_shared_to_rank(smem_addr(c + cluster_ctarank() * 2), uint32_t(tid));
#pragma unroll
        for (int i = 0; i < NV; ++i) st_shared_cluster_u32(at + 4 * i, __float_as_uint(v[i]));
      }
      cluster_sync_all();
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = 0.f;
      for (int r = 0; r < cluster; ++r)
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] += c[2 * r + i];
    }
    turn ^= 1;
  }
};

struct RowThread {
  int group, t, col;
  int64_t worker;
};

__device__ __forceinline__ RowThread row_thread(int threads_per_row, int cluster) {
  RowThread r;
  r.group = int(threadIdx.x) / threads_per_row;
  r.t = int(threadIdx.x) - r.group * threads_per_row;
  const int rank = cluster > 1 ? int(cluster_ctarank()) : 0;
  r.col = (rank * threads_per_row + r.t) * 8;
  const int groups = int(blockDim.x) / threads_per_row;
  r.worker = int64_t(int(blockIdx.x) / cluster) * groups + r.group;
  return r;
}

__device__ __forceinline__ float activate(float g, int act) {
  return act == 0 ? g : act == 1 ? 1.f / (1.f + expf(-g)) : tanhf(g);
}
// derivative of the activation, from its value
__device__ __forceinline__ float activate_d(float a, int act) {
  return act == 0 ? 1.f : act == 1 ? a * (1.f - a) : 1.f - a * a;
}

template <typename TX, typename TR, bool VEC>
__device__ __forceinline__ void load_gate(const BlockNormParams& p, int64_t grow, int col, float (&a)[8]) {
  if (p.gate_res_type)
    unpack8(load8<TR, VEC>(static_cast<const TR*>(p.gate) + grow * p.ld_gate, col, p.D), a);
  else
    unpack8(load8<TX, VEC>(static_cast<const TX*>(p.gate) + grow * p.ld_gate, col, p.D), a);
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = activate(a[i], p.act);
}

__device__ __forceinline__ void load_weight(const void* w, int dt, float off, int col, int D, float (&f)[8]) {
  load8_any(w, dt, 0, col, D, f);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = col + i < D ? f[i] + off : 0.f;
}

__device__ __forceinline__ float sum8(const float (&v)[8]) {
  return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
}

// mean (0 for the RMS norm) and 1 / sqrt(mean of the squared distances from it + eps); the
// distances are summed from the values themselves, so a large common offset costs nothing.
__device__ __forceinline__ void row_stats(const float (&v)[8], int col, int D, bool layer, float eps, float inv_d,
                                          RowSum& rs, float& mean, float& rstd) {
  mean = 0.f;
  if (layer) {
    float s[1] = {sum8(v)};
    rs.sum(s);
    mean = s[0] * inv_d;
  }
  float q[1] = {0.f};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float d = v[i] - mean;
    q[0] += col + i < D ? d * d : 0.f;
  }
  rs.sum(q);
  rstd = rsqrtf(q[0] * inv_d + eps);
}

__device__ __forceinline__ RowSum row_sum(float* scratch, const RowThread& r, int threads_per_row, int cluster) {
  RowSum rs;
  rs.clus = scratch;
  rs.buf = scratch + 4 * kBnMaxCluster + r.group * 2 * RowSum::kWords;
  rs.nw = threads_per_row / 32;
  rs.warp = r.t / 32;
  rs.lane = r.t % 32;
  rs.bar = 1 + r.group;
  rs.threads = threads_per_row;
  rs.cluster = cluster;
  rs.turn = 0;
  return rs;
}
constexpr int kRowSumWords = 4 * kBnMaxCluster + 8 * 2 * RowSum::kWords;  // at most 8 groups use barriers

template <typename TX, typename TR, bool VEC>
__global__ void __launch_bounds__(kBnMaxThreads)
    flce_block_norm_forward_kernel(const BlockNormParams p, int threads_per_row, int cluster) {
  __shared__ __align__(16) float scratch[kRowSumWords];
  const RowThread r = row_thread(threads_per_row, cluster);
  RowSum rs = row_sum(scratch, r, threads_per_row, cluster);
  if (cluster > 1) cluster_sync_all();
  const int col = r.col, D = p.D;
  const bool post = p.w1 != nullptr, pre = p.w2 != nullptr;
  float w1[8], b1[8], w2[8], b2[8], a[8];
  load_weight(p.w1, p.w1_dt, p.w_off, col, D, w1);
  load8_any(p.b1, p.b1_dt, 0, col, D, b1);
  load_weight(p.w2, p.w2_dt, p.w_off, col, D, w2);
  load8_any(p.b2, p.b2_dt, 0, col, D, b2);
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = 1.f;
  const float inv_d = 1.f / float(D);
  const int64_t lo = r.worker * p.chunk_rows;
  const int64_t hi = lo + p.chunk_rows < p.N ? lo + p.chunk_rows : p.N;
  int64_t gate_end = lo;  // first row whose gate is not in a[]
  for (int64_t row = lo; row < hi; ++row) {
    const Raw8<TX> rx = load8<TX, VEC>(static_cast<const TX*>(p.x) + row * p.ld_x, col, D);
    Raw8<TR> rr = raw_zero<TR>();
    if (p.residual != nullptr) rr = load8<TR, VEC>(static_cast<const TR*>(p.residual) + row * p.ld_residual, col, D);
    if (p.gate != nullptr && row >= gate_end) {
      const int64_t g = row / p.gate_group;
      load_gate<TX, TR, VEC>(p, g, col, a);
      gate_end = (g + 1) * p.gate_group;
    }
    float u[8], h[8];
    unpack8(rx, u);
    unpack8(rr, h);
    float m1 = 0.f, r1 = 0.f, m2 = 0.f, r2 = 0.f;
    if (post) {
      row_stats(u, col, D, p.layer, p.eps, inv_d, rs, m1, r1);
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = (u[i] - m1) * r1 * w1[i] + b1[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] += p.scale * (a[i] * u[i]);
    store8<TR, VEC>(static_cast<TR*>(p.h) + row * D, col, D, h);
    if (pre) {
      row_stats(h, col, D, p.layer, p.eps, inv_d, rs, m2, r2);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = (h[i] - m2) * r2 * w2[i] + b2[i];
      store8<TX, VEC>(static_cast<TX*>(p.y) + row * D, col, D, h);
    }
    if (p.stats != nullptr && col == 0) {
      p.stats[row] = m1;
      p.stats[p.N + row] = r1;
      p.stats[2 * p.N + row] = m2;
      p.stats[3 * p.N + row] = r2;
    }
  }
  if (cluster > 1) cluster_sync_all();  // no block leaves while another may still write to it
}

template <typename TX, typename TR, bool VEC, int FEAT>
__global__ void __launch_bounds__(kBnMaxThreads)
    flce_block_norm_backward_kernel(const BlockNormParams p, int threads_per_row, int cluster) {
  constexpr bool POST = (FEAT & BN_POST) != 0, GATE = (FEAT & BN_GATE) != 0, BIAS = (FEAT & BN_BIAS) != 0;
  __shared__ __align__(16) float scratch[kRowSumWords];
  extern __shared__ float fold[];  // [threads][8] when a block has several row groups
  const RowThread r = row_thread(threads_per_row, cluster);
  RowSum rs = row_sum(scratch, r, threads_per_row, cluster);
  if (cluster > 1) cluster_sync_all();
  const int col = r.col, D = p.D;
  const bool post = POST && p.w1 != nullptr, pre = p.w2 != nullptr, gate = GATE && p.gate != nullptr;
  float w1[8], w2[8], b1[8], a[8], dw1[8], db1[8], dw2[8], db2[8], dg[8];
  load_weight(p.w1, p.w1_dt, p.w_off, col, D, w1);
  load_weight(p.w2, p.w2_dt, p.w_off, col, D, w2);
  load8_any(p.b1, p.b1_dt, 0, col, D, b1);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a[i] = 1.f;
    dw1[i] = db1[i] = dw2[i] = db2[i] = dg[i] = 0.f;
  }
  const float inv_d = 1.f / float(D), inv_d0 = p.layer ? inv_d : 0.f;
  const int64_t workers = int64_t(int(gridDim.x) / cluster) * (int(blockDim.x) / threads_per_row);
  for (int64_t chunk = r.worker; chunk < p.chunks; chunk += workers) {
    const int64_t g = chunk / p.chunks_per_group, first = g * p.group_rows;
    const int64_t lo = first + (chunk - g * p.chunks_per_group) * p.chunk_rows;
    const int64_t end = first + p.group_rows;
    const int64_t hi = lo + p.chunk_rows < end ? lo + p.chunk_rows : end;
    if (gate && !p.gate_full) load_gate<TX, TR, VEC>(p, g, col, a);
    for (int64_t row = lo; row < hi; ++row) {
      const Raw8<TX> rx = load8<TX, VEC>(static_cast<const TX*>(p.x) + row * p.ld_x, col, D);
      Raw8<TR> rh = raw_zero<TR>(), rdh = raw_zero<TR>();
      Raw8<TX> rdy = raw_zero<TX>();
      if (pre) rh = load8<TR, VEC>(static_cast<const TR*>(p.h_in) + row * D, col, D);
      if (p.dh != nullptr) rdh = load8<TR, VEC>(static_cast<const TR*>(p.dh) + row * p.ld_dh, col, D);
      if (pre && p.dy != nullptr) rdy = load8<TX, VEC>(static_cast<const TX*>(p.dy) + row * p.ld_dy, col, D);
      if (gate && p.gate_full) load_gate<TX, TR, VEC>(p, row, col, a);
      float x[8], d[8];  // d: the gradient of h, then of u
      unpack8(rx, x);
      unpack8(rdh, d);
      if (pre) {
        const float m2 = p.stats[2 * p.N + row], r2 = p.stats[3 * p.N + row];
        float n[8], dy[8];
        unpack8(rh, n);
        unpack8(rdy, dy);
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          n[i] = (n[i] - m2) * r2;
          dw2[i] += dy[i] * n[i];
          if (BIAS) db2[i] += dy[i];
          dy[i] *= w2[i];
          s[0] += dy[i] * n[i];
          s[1] += dy[i];
        }
        if (p.layer) {
          rs.sum(s);
        } else {
          float one[1] = {s[0]};
          rs.sum(one);
          s[0] = one[0];
        }
        const float c0 = s[1] * inv_d0, c1 = s[0] * inv_d;
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] += r2 * (dy[i] - c0 - n[i] * c1);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (col + i >= D) d[i] = 0.f;
      if (p.dres != nullptr) store8<TR, VEC>(static_cast<TR*>(p.dres) + row * D, col, D, d);
      float m1 = 0.f, r1 = 1.f;
      if (post) {
        m1 = p.stats[row];
        r1 = p.stats[p.N + row];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (x[i] - m1) * r1;
      }
      if (gate) {
        float e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          e[i] = d[i] * (post ? x[i] * w1[i] + b1[i] : x[i]);
          d[i] *= p.scale * a[i];
        }
        if (p.gate_full) {
          if (p.dgate != nullptr) {
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] *= p.scale * activate_d(a[i], p.act);
            if (p.gate_res_type)
              store8<TR, VEC>(static_cast<TR*>(p.dgate) + row * D, col, D, e);
            else
              store8<TX, VEC>(static_cast<TX*>(p.dgate) + row * D, col, D, e);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) dg[i] += e[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] *= p.scale;
      }
      if (post) {
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dw1[i] += d[i] * x[i];
          if (BIAS) db1[i] += d[i];
          d[i] *= w1[i];
          s[0] += d[i] * x[i];
          s[1] += d[i];
        }
        if (p.layer) {
          rs.sum(s);
        } else {
          float one[1] = {s[0]};
          rs.sum(one);
          s[0] = one[0];
        }
        const float c0 = s[1] * inv_d0, c1 = s[0] * inv_d;
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = r1 * (d[i] - c0 - x[i] * c1);
      }
      if (p.dx != nullptr) store8<TX, VEC>(static_cast<TX*>(p.dx) + row * D, col, D, d);
    }
    if (gate && !p.gate_full && p.dgate != nullptr) {
#pragma unroll
      for (int i = 0; i < 8; ++i) dg[i] *= p.scale * activate_d(a[i], p.act);
      if (p.part_gate != nullptr)
        store8<float, VEC>(p.part_gate + chunk * D, col, D, dg);
      else if (p.gate_res_type)
        store8<TR, VEC>(static_cast<TR*>(p.dgate) + g * D, col, D, dg);
      else
        store8<TX, VEC>(static_cast<TX*>(p.dgate) + g * D, col, D, dg);
#pragma unroll
      for (int i = 0; i < 8; ++i) dg[i] = 0.f;
    }
  }
  // one partial sum a block and parameter: the block's row groups first
  const int groups = int(blockDim.x) / threads_per_row;
  const int64_t block = int64_t(int(blockIdx.x) / cluster);
  auto flush = [&](float* part, const float(&v)[8]) {
    if (part == nullptr) return;
    if (groups == 1) {
      store8<float, VEC>(part + block * D, col, D, v);
      return;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) fold[threadIdx.x * 8 + i] = v[i];
    __syncthreads();
    if (r.group == 0) {
      float s[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = 0.f;
      for (int q = 0; q < groups; ++q)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] += fold[(q * threads_per_row + r.t) * 8 + i];
      store8<float, VEC>(part + block * D, col, D, s);
    }
  };
  if (POST) flush(p.part[0], dw1);
  if (POST && BIAS) flush(p.part[1], db1);
  flush(p.part[2], dw2);
  if (BIAS) flush(p.part[3], db2);
  if (cluster > 1) cluster_sync_all();
}

template <typename K>
cudaError_t bn_launch(K kernel, const BlockNormParams& p, const BlockNormShape& s, unsigned blocks, size_t smem,
                      cudaStream_t stream) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(blocks * unsigned(s.cluster));
  c.blockDim = dim3(unsigned(s.threads_per_row * s.rows_per_block));
  c.dynamicSmemBytes = smem;
  c.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = unsigned(s.cluster);
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&c, kernel, p, s.threads_per_row, s.cluster);
  if (e == cudaSuccess) count_launch();
  return e;
}

template <typename TX, typename TR>
cudaError_t bn_forward_typed(const BlockNormParams& p, const BlockNormShape& s, bool vec, unsigned blocks,
                             cudaStream_t stream) {
  return vec ? bn_launch(flce_block_norm_forward_kernel<TX, TR, true>, p, s, blocks, 0, stream)
             : bn_launch(flce_block_norm_forward_kernel<TX, TR, false>, p, s, blocks, 0, stream);
}

template <typename TX, typename TR>
cudaError_t bn_backward_typed(const BlockNormParams& p, const BlockNormShape& s, bool vec, int feat, unsigned blocks,
                              cudaStream_t stream) {
  const size_t smem = s.rows_per_block > 1 ? size_t(s.threads_per_row) * s.rows_per_block * 8 * sizeof(float) : 0;
  // unaligned rows take the kernel with every accumulator
  if (!vec) return bn_launch(flce_block_norm_backward_kernel<TX, TR, false, BN_ALL>, p, s, blocks, smem, stream);
  switch (feat) {
    case 0: return bn_launch(flce_block_norm_backward_kernel<TX, TR, true, 0>, p, s, blocks, smem, stream);
    case 1: return bn_launch(flce_block_norm_backward_kernel<TX, TR, true, 1>, p, s, blocks, smem, stream);
    case 2: return bn_launch(flce_block_norm_backward_kernel<TX, TR, true, 2>, p, s, blocks, smem, stream);
    case 3: return bn_launch(flce_block_norm_backward_kernel<TX, TR, true, 3>, p, s, blocks, smem, stream);
    case 4: return bn_launch(flce_block_norm_backward_kernel<TX, TR, true, 4>, p, s, blocks, smem, stream);
    case 5: return bn_launch(flce_block_norm_backward_kernel<TX, TR, true, 5>, p, s, blocks, smem, stream);
    case 6: return bn_launch(flce_block_norm_backward_kernel<TX, TR, true, 6>, p, s, blocks, smem, stream);
    default: return bn_launch(flce_block_norm_backward_kernel<TX, TR, true, 7>, p, s, blocks, smem, stream);
  }
}

}  // namespace
}  // namespace flce
