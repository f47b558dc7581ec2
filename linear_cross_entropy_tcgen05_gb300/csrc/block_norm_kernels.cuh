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
//
// Measured (of 6.8 TB/s that a copy reaches): N = 65536, D = 4096 bf16, two RMS norms, forward 324 us (6.6
// TB/s), backward 479 us (6.7). N = 16384, D = 2304 bf16 with an fp32 residual, layer norms, 16 gate
// rows: 104 us (4.4), 194 us (3.5): latency and instructions, not memory. Rows shared by
// clusters, D = 16384: 394 us, 590 us (16384 rows, 5.5). Unaligned rows, D = 4095: bf16 2.6 and 2.2
// TB/s, fp32 4.0 and 3.0 (bound by instructions: 600 and 1000 for a warp's 256 columns).
#pragma once

#include <math_constants.h>

#include "block_norm.h"
#include "elem_io.cuh"
#include "flce_internal.h"
#include "sm103_ptx.cuh"

// The kernels' local functions: one that is not inlined would keep what it refers to in memory.
#define FLCE_INLINE __attribute__((always_inline))

namespace flce {
namespace {

// Rows are copied to shared memory (cp.async) some batches of kBnRows rows ahead. A batch has,
// for each of its rows and tensors, planes of 16 bytes a thread. Slots whose tensor or columns are
// not there are zeroed once and never copied to.
//
// VEC: a thread copies and reads only its own eight columns, so a batch is ready for it when its
// own copies are: no barrier. (Neighbouring lanes copying neighbouring 16 bytes of fp32 rows, to
// one another's places, measured slower: N = 65536, D = 4096, forward 952 us against 896.) Else the
// rows start anywhere in 16 bytes, which wide copies do not, and a warp copies its 256 columns
// together. fp32 elements go to their thread's place one by one. Of 16-bit ones, which are too
// small for that, the 33 aligned pieces that the columns touch are copied (a plane has 33),
// and when they have landed each thread shifts its own columns into its place (take and land; N =
// 32768, D = 4095 bf16, two RMS norms: forward 683 to 410 us, backward 1030 to 725 us against loads of
// single elements).
template <bool VEC> struct RowRing {
  uint32_t first, end;       // this thread's first plane of the ring's first batch, and past its last
  int plane;                 // bytes from a plane of the thread to the next
  int row_bytes;             // from a batch's row to its next; 0 where it has one, which is read in the next one's place
  uint32_t batch_bytes;

  __device__ __forceinline__ void init(char* smem, int planes, int batches, int rows) {
    const int warps = int(blockDim.x) / 32, warp = int(threadIdx.x) / 32, lane = int(threadIdx.x) % 32;
    plane = VEC ? 16 * int(blockDim.x) : kBnWarpPlane;
    const int row = VEC ? planes * plane : warps * planes * plane;
    row_bytes = rows > 1 ? row : 0;
    batch_bytes = uint32_t(rows * row);
    first = smem_addr(smem) + 16u * uint32_t(VEC ? int(threadIdx.x) : lane) + uint32_t(VEC ? 0 : warp * planes * plane);
    end = first + uint32_t(batches) * batch_bytes;
    for (uint32_t at = first; at < end; at += uint32_t(row))
      for (int i = 0; i < planes; ++i)
        asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(at + uint32_t(i * plane)), "r"(0) : "memory");
    if (!VEC) __syncwarp();
  }
  __device__ __forceinline__ uint32_t after(uint32_t batch) const {
    return batch + batch_bytes == end ? first : batch + batch_bytes;
  }
  // The first column of the warp's first thread.
  __device__ __forceinline__ static int warp_col(const Cols& cs) { return cs.col - 8 * (int(threadIdx.x) % 32); }
  // A row's columns into their planes; base: the tensor, whose first row may start within 16 bytes.
  // VEC: by threads whose columns are in the row, else by warps of which some are.
  template <typename T> __device__ __forceinline__ void copy(uint32_t to, int planes, const void* base, const T* row, const Cols& cs) const {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < int(sizeof(T)) / 2; ++i)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + uint32_t((planes + i) * plane)),
                     "l"(reinterpret_cast<const char*>(row + cs.col) + 16 * i)
                     : "memory");
    } else if constexpr (sizeof(T) == 4) {
      // each element to its thread's place: neighbouring lanes copy neighbouring columns
      const int lane = int(threadIdx.x) % 32, c = warp_col(cs) + lane;
      to += uint32_t((planes + lane % 8 / 4) * plane + 16 * (lane / 8) + 4 * (lane % 4) - 16 * lane);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + 32 * i < cs.D)
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + 64u * i), "l"(row + c + 32 * i) : "memory");
    } else {
      const int lane = int(threadIdx.x) % 32;
      const char* at = reinterpret_cast<const char*>(row + warp_col(cs));
      const int s = int(reinterpret_cast<uintptr_t>(at) & 15);
      const int columns = cs.D - warp_col(cs) < 256 ? cs.D - warp_col(cs) : 256;
      const int bytes = s + columns * int(sizeof(T)) - 16 * lane;  // from the lane's piece on
      at += 16 * lane - s;
      to += uint32_t(planes * plane);
      if (bytes > 0 && at < static_cast<const char*>(base)) {  // nothing before the tensor is read
        for (int e = s; e < (bytes < 16 ? bytes : 16); e += int(sizeof(T)))
          asm volatile("st.shared.u16 [%0], %1;" ::"r"(to + uint32_t(e)), "h"(*reinterpret_cast<const uint16_t*>(at + e)) : "memory");
      } else if (bytes > 0) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(at), "r"(bytes < 16 ? bytes : 16) : "memory");
      }
      if (lane == 0 && bytes > 512)  // the 33rd
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + 512u), "l"(at + 512), "r"(bytes - 512 < 16 ? bytes - 512 : 16)
                     : "memory");
    }
  }
  // Not VEC: the thread's own columns of a row of 16-bit elements that has landed; row: where it came
  // from. All lanes take before any puts them into its own place.
  template <typename T> __device__ __forceinline__ Raw8<T> take(uint32_t to, int planes, const T* row, const Cols& cs) const {
    Raw8<T> v = raw_zero<T>();
    if constexpr (sizeof(T) == 2) {
      const int s = int(reinterpret_cast<uintptr_t>(row + warp_col(cs)) & 15);
      const uint32_t at = to + uint32_t(planes * plane);
      uint32_t w[8], q[4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[4 * i]), "=r"(w[4 * i + 1]), "=r"(w[4 * i + 2]), "=r"(w[4 * i + 3])
                     : "r"(at + 16u * i));
      words_from<T>(s / 4, w, s & 2, q);
      if (cs.D - warp_col(cs) < 256) {  // the row's last warp: nothing past the row
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int left = cs.D - cs.col - 2 * i;  // columns of the row from this word on
          q[i] = left <= 0 ? 0 : left == 1 ? q[i] & 0xffffu : q[i];
        }
      }
      v.v[0] = make_uint4(q[0], q[1], q[2], q[3]);
    }
    return v;
  }
  template <typename T> __device__ __forceinline__ void land(uint32_t to, int planes, const Raw8<T>& v) const {
    if constexpr (sizeof(T) == 2)
      asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(to + uint32_t(planes * plane)), "r"(v.v[0].x), "r"(v.v[0].y),
                   "r"(v.v[0].z), "r"(v.v[0].w)
                   : "memory");
  }
  template <typename T> __device__ __forceinline__ void get(uint32_t batch, int r, int planes, float2 (&f)[4]) const {
    Raw8<T> v;
#pragma unroll
    for (int i = 0; i < int(sizeof(T)) / 2; ++i)
      asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(v.v[i].x), "=r"(v.v[i].y), "=r"(v.v[i].z), "=r"(v.v[i].w)
                   : "r"(batch + uint32_t(r * row_bytes + (planes + i) * plane)));
    unpack8(v, f);
  }
  __device__ __forceinline__ static void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  // Waits until all but the newest `left` batches have landed.
  __device__ __forceinline__ static void wait(int left) {
    switch (left) {
      case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
      case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
      case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
      case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
      case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
      default: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
    }
  }
};

// Address of a row (computed where it is used: pointers that are kept from row to row cost the
// registers that the sums need).
template <typename T> __device__ __forceinline__ const T* row_at(const void* base, int64_t row, int64_t ld) {
  return static_cast<const T*>(base) + row * ld;
}
template <typename T> __device__ __forceinline__ T* row_at(void* base, int64_t row, int64_t ld) {
  return static_cast<T*>(base) + row * ld;
}

// Sums over the threads of a row, of NV values at once (those of several rows: a sum is all
// latency, about 500 cycles of shuffles, a barrier and reads, so rows share it). Within a warp
// the values are spread over the lanes as they are added (NV / 2 + ... + 1 shuffles and one a
// step after that, instead of five a value). Two scratch buffers take turns, so one barrier a
// sum is enough: a buffer is written again only after the barrier of the sum between.
// CLUSTER: blocks share rows; code apart, for its registers.
template <bool CLUSTER> struct RowSum {
  float* buf;      // [2][kMaxValues * nw] of this row group
  float* clus;     // [2][kBnMaxCluster][4] of this block
  int nw, warp, lane, bar, threads, turn;
  int blocks;  // of the cluster
  static constexpr int kMaxValues = 8;

  // Sums over the warp: value i ends in lanes i * (32 / NV) ... of the result.
  template <int NV> __device__ __forceinline__ float scatter_sum(const float (&v)[NV]) const {
    static_assert(NV == 2 || NV == 4 || NV == 8, "values of a sum");
    float s[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i] = v[i];
    int o = 16;
#pragma unroll
    for (int n = NV; n > 1; n /= 2, o /= 2) {
      const bool high = (lane & o) != 0;
#pragma unroll
      for (int i = 0; i < n / 2; ++i) {
        const float give = high ? s[i] : s[i + n / 2], keep = high ? s[i + n / 2] : s[i];
        s[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
      }
    }
#pragma unroll
    for (int k = 16 / NV; k > 0; k >>= 1) s[0] += __shfl_xor_sync(0xffffffffu, s[0], k);
    return s[0];
  }

  template <int NV> __device__ __forceinline__ void sum(float (&v)[NV]) {
    const float mine = scatter_sum(v);
    if (nw > 1) {
      float* b = buf + (CLUSTER ? turn & 1 : turn) * (kMaxValues * nw);
      if (lane % (32 / NV) == 0) b[warp * NV + lane / (32 / NV)] = mine;
      named_barrier_sync(uint32_t(bar), uint32_t(threads));
      if constexpr (NV <= 4) {
        float2 lo = both(0.f), hi = both(0.f);
        const int n4 = nw * NV / 4;
#pragma unroll 4
        for (int w = 0; w < n4; ++w) {
          const float4 q = reinterpret_cast<const float4*>(b)[w];
          lo = add2(lo, make_float2(q.x, q.y));
          hi = add2(hi, make_float2(q.z, q.w));
        }
        // two values of an odd number of warps: the last one's (what follows is another sum's)
        if (NV == 2 && (nw & 1)) lo = add2(lo, reinterpret_cast<const float2*>(b)[nw - 1]);
        if constexpr (NV == 2) {
          v[0] = lo.x + hi.x;
          v[1] = lo.y + hi.y;
        } else {
          v[0] = lo.x;
          v[1] = lo.y;
          v[2] = hi.x;
          v[3] = hi.y;
        }
      } else {
        float2 s2[4] = {both(0.f), both(0.f), both(0.f), both(0.f)};
#pragma unroll 4
        for (int w = 0; w < nw; ++w) {
          const float4 q = reinterpret_cast<const float4*>(b)[2 * w], u = reinterpret_cast<const float4*>(b)[2 * w + 1];
          s2[0] = add2(s2[0], make_float2(q.x, q.y));
          s2[1] = add2(s2[1], make_float2(q.z, q.w));
          s2[2] = add2(s2[2], make_float2(u.x, u.y));
          s2[3] = add2(s2[3], make_float2(u.z, u.w));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[2 * i] = s2[i].x;
          v[2 * i + 1] = s2[i].y;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = __shfl_sync(0xffffffffu, mine, i * (32 / NV));
    }
    if constexpr (CLUSTER) exchange(v);
    turn = CLUSTER ? turn + 1 : turn ^ 1;
  }

  // Of the warps' column sums s and squared distances q from their own means (value i in lanes
  // i * (32 / NR) ...): the rows' means and the squared distances from those. A warp has 256
  // columns, but for one that has the row's last `part` ones. With c the first warp's mean, the
  // distances are sum q_w + n_w (m_w - c)^2, less n (mean - c)^2: one pass over the warps, and
  // c is near enough to the mean that the difference loses nothing to speak of.
  template <int NR> __device__ __forceinline__ void merge(float s, float q, float inv_d, float (&mean)[NR], float (&dist)[NR]) {
    static_assert(2 * NR <= kMaxValues, "values of a sum");
    if (nw > 1) {
      float* b = buf + (CLUSTER ? turn & 1 : turn) * (kMaxValues * nw);
      if (lane % (32 / NR) == 0) {
        const int i = lane / (32 / NR);
        float* at = b + warp * 2 * NR + (i / 2) * 4 + i % 2;
        at[0] = s;
        at[2] = q;
      }
      named_barrier_sync(uint32_t(bar), uint32_t(threads));
      float2 total[NR / 2], far[NR / 2], c[NR / 2];
      const float first_inv = inv_columns(0);
#pragma unroll
      for (int i = 0; i < NR / 2; ++i) {
        const float4 o = reinterpret_cast<const float4*>(b)[i];
        total[i] = far[i] = both(0.f);
        c[i] = mul2(make_float2(o.x, o.y), both(-first_inv));
      }
      auto add = [&](int w, float n, float inv_n) {
#pragma unroll
        for (int i = 0; i < NR / 2; ++i) {
          const float4 o = reinterpret_cast<const float4*>(b + w * 2 * NR)[i];
          const float2 m = fma2(make_float2(o.x, o.y), both(inv_n), c[i]);
          total[i] = add2(total[i], make_float2(o.x, o.y));
          far[i] = add2(far[i], fma2(mul2(m, both(n)), m, make_float2(o.z, o.w)));
        }
      };
#pragma unroll 3
      for (int w = 0; w < full; ++w) add(w, 256.f, 1.f / 256.f);
      if (part > 0) add(full, float(part), part_inv);
      const float n = CLUSTER ? block_columns(int(cluster_ctarank())) : float(D), inv_n = CLUSTER ? (n > 0.f ? 1.f / n : 0.f) : inv_d;
#pragma unroll
      for (int i = 0; i < NR / 2; ++i) {
        const float2 m = fma2(total[i], both(inv_n), c[i]);  // this block's mean, less c
        far[i] = fma2(mul2(m, both(-n)), m, far[i]);
        mean[2 * i] = total[i].x;
        mean[2 * i + 1] = total[i].y;
        dist[2 * i] = far[i].x;
        dist[2 * i + 1] = far[i].y;
      }
    } else {
      // one warp: its mean is the row's
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        mean[i] = __shfl_sync(0xffffffffu, s, i * (32 / NR));
        dist[i] = __shfl_sync(0xffffffffu, q, i * (32 / NR));
      }
    }
    if constexpr (CLUSTER) {
      float v[2 * NR];
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        v[i] = mean[i];
        v[NR + i] = dist[i];
      }
      const float* c;
      const bool ok = publish(v, c);
      float all[NR];
#pragma unroll
      for (int i = 0; i < NR; ++i) all[i] = dist[i] = ok ? 0.f : CUDART_NAN_F;
      for (int r = 0; r < blocks; ++r)
#pragma unroll
        for (int i = 0; i < NR; ++i) all[i] += c[kMaxValues * r + i];
      for (int r = 0; r < blocks; ++r) {
        const float n = block_columns(r), inv_n = n > 0.f ? 1.f / n : 0.f;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          const float d = c[kMaxValues * r + i] * inv_n - all[i] * inv_d;
          dist[i] += c[kMaxValues * r + NR + i] + n * d * d;
        }
      }
#pragma unroll
      for (int i = 0; i < NR; ++i) mean[i] = all[i];
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      mean[i] *= inv_d;
      dist[i] = dist[i] < 0.f ? 0.f : dist[i];  // (a NaN stays)
    }
    turn = CLUSTER ? turn + 1 : turn ^ 1;
  }
  // Columns of the row that block r of the cluster has.
  int D;
  __device__ __forceinline__ float block_columns(int r) const {
    const int most = 8 * threads, left = D - r * most;
    return float(left < 0 ? 0 : left < most ? left : most);
  }
  // Shows this block's values to the blocks of the blocks; c: all blocks' values. The values go
  // as stores that are counted on a barrier of the block that they go to, so nobody waits for
  // anything else: a cluster barrier would also wait until the row's stores to global memory are
  // visible (N = 32768, D = 8192 bf16: forward 491 us with it). A block sends the next but one
  // sum's values only after it has all blocks' of the next, which they send when they have read
  // these: two buffers and barriers are enough. Returns false after a wait of 2 s (never, unless a
  // block of the cluster is gone).
  template <int NV> __device__ __forceinline__ bool publish(const float (&v)[NV], const float*& c) {
    const int use = turn & 1, tid = warp * 32 + lane;
    uint64_t* done = reinterpret_cast<uint64_t*>(clus - 4) + use;
    float* mine = clus + use * (kMaxValues * kBnMaxCluster);
    if (tid == 0) mbar_arrive_expect_tx(done, uint32_t(blocks * NV * 4));
    if (tid < blocks) {
      const uint32_t at = map_shared_to_rank(smem_addr(mine + cluster_ctarank() * kMaxValues), uint32_t(tid));
      const uint32_t bar_at = map_shared_to_rank(smem_addr(done), uint32_t(tid));
#pragma unroll
      for (int i = 0; i < NV; i += 2) st_async_v2(at + 4 * i, __float_as_uint(v[i]), __float_as_uint(v[i + 1]), bar_at);
    }
    c = mine;
    const uint32_t a = smem_addr(done), parity = uint32_t(turn >> 1) & 1u;
    if (mbar_try_wait_acq_cluster(a, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait_acq_cluster(a, parity))
      if (global_timer_ns() - t0 > FLCE_WAIT_LIMIT_NS) return false;
    return true;
  }
  // Sums over the blocks of the cluster.
  template <int NV> __device__ __forceinline__ void exchange(float (&v)[NV]) {
    const float* c;
    const bool ok = publish(v, c);
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = ok ? 0.f : CUDART_NAN_F;
    for (int r = 0; r < blocks; ++r)
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] += c[kMaxValues * r + i];
  }
  // Columns of the block's warps: `full` warps have 256 and the next one has `part`.
  int full, part;
  float part_inv;
  __device__ __forceinline__ float inv_columns(int w) const {
    return w < full ? 1.f / 256.f : w == full ? part_inv : 0.f;
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

// The reciprocal instruction, for d of 1 and more: off by one step at most.
__device__ __forceinline__ float quick_rcp(float d) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  return r;
}
// QUICK: by that reciprocal. With a gate for each row the forward's divisions were a quarter of its time (N
// = 32768, D = 4096 bf16, layer norms: 427 to 312 us). The backward takes value and derivative of such a
// gate from one exponential and one quick reciprocal (702 us with a division and a (1 - a), 649 us so),
// but for values alone the division: eight of the other at once spill (649 to 883 us).
template <bool QUICK> __device__ __forceinline__ float activate(float g, int act) {
  if (act != 1) return tanhf(g);
  const float d = 1.f + expf(-g);
  return QUICK ? quick_rcp(d) : 1.f / d;
}
// Derivative of the activation, from its argument: with e = exp(-k |g|), k = 1 (sigmoid) or 2 (tanh), it is
// k^2 e / (1 + e)^2. From the value, a (1 - a) or 1 - a^2, a gate of 8 would lose half its bits and one
// of 17 all.
__device__ __forceinline__ float activate_d(float g, int act) {
  if (act == 0) return 1.f;
  const float e = expf(act == 1 ? -fabsf(g) : -2.f * fabsf(g)), r = quick_rcp(1.f + e);
  return act == 1 ? e * r * r : 4.f * e * r * r;
}

template <bool QUICK> __device__ __forceinline__ void activate8(float2 (&a)[4], int act) {
  if (act == 0) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = make_float2(activate<QUICK>(a[i].x, act), activate<QUICK>(a[i].y, act));
}
// derivatives of the activation, from its arguments
__device__ __forceinline__ void derive8(const float2 (&g)[4], int act, float2 (&da)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) da[i] = make_float2(activate_d(g[i].x, act), activate_d(g[i].y, act));
}

// both at once: a's arguments become values
__device__ __forceinline__ void activate_derive8(float2 (&a)[4], int act, float2 (&da)[4]) {
  auto one = [&](float& g, float& d) FLCE_INLINE {
    const float e = expf(act == 1 ? -fabsf(g) : -2.f * fabsf(g)), r = quick_rcp(1.f + e);
    d = act == 1 ? e * r * r : 4.f * e * r * r;
    g = act == 2 ? tanhf(g) : g < 0.f ? e * r : r;
  };
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    da[i] = both(1.f);
    if (act == 0) continue;
    one(a[i].x, da[i].x);
    one(a[i].y, da[i].y);
  }
}

template <typename TX, typename TR, bool VEC>
__device__ __forceinline__ void load_gate(const BlockNormParams& p, int64_t grow, const Cols& cs, float2 (&g)[4]) {
  if (p.gate_res_type)
    unpack8(load8<TR, VEC>(static_cast<const TR*>(p.gate) + grow * p.ld_gate, cs), g);
  else
    unpack8(load8<TX, VEC>(static_cast<const TX*>(p.gate) + grow * p.ld_gate, cs), g);
}

// Parameters (zero past the row and where there are none), w + off; read once a block.
template <bool VEC>
__device__ __forceinline__ void load_weight(const void* w, int dt, float off, const Cols& cs, float2 (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = both(0.f);
  if (w == nullptr || cs.col >= cs.D) return;
  if (dt == ELEM_F32)
    unpack8(load8<float, VEC>(static_cast<const float*>(w), cs), f);
  else if (dt == ELEM_BF16)
    unpack8(load8<__nv_bfloat16, VEC>(static_cast<const __nv_bfloat16*>(w), cs), f);
  else
    unpack8(load8<__half, VEC>(static_cast<const __half*>(w), cs), f);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    f[i] = VEC ? make_float2(f[i].x + off, f[i].y + off)
               : make_float2(cs.col + 2 * i < cs.D ? f[i].x + off : 0.f, cs.col + 2 * i + 1 < cs.D ? f[i].y + off : 0.f);
}

// Eight values in shared memory, in two planes: a parameter's for a thread of a row, in the
// kernels with more of them than registers, or a thread's own (a gate, a sum). Offsets are 32-bit
// and made where they are used: a spilled register costs more than they do.
__device__ __forceinline__ void shared_get(const char* smem, int at, int plane, float2 (&f)[4]) {
  const float4 a = *reinterpret_cast<const float4*>(smem + at), b = *reinterpret_cast<const float4*>(smem + at + plane);
  f[0] = make_float2(a.x, a.y);
  f[1] = make_float2(a.z, a.w);
  f[2] = make_float2(b.x, b.y);
  f[3] = make_float2(b.z, b.w);
}
__device__ __forceinline__ void shared_set(char* smem, int at, int plane, const float2 (&f)[4]) {
  *reinterpret_cast<float4*>(smem + at) = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
  *reinterpret_cast<float4*>(smem + at + plane) = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
}

__device__ __forceinline__ float sum8(const float2 (&v)[4]) {
  const float2 s = add2(add2(v[0], v[1]), add2(v[2], v[3]));
  return s.x + s.y;
}
__device__ __forceinline__ float dot8(const float2 (&a)[4], const float2 (&b)[4]) {
  const float2 s = add2(fma2(a[1], b[1], mul2(a[0], b[0])), fma2(a[3], b[3], mul2(a[2], b[2])));
  return s.x + s.y;
}
// Zeros in the columns past the row. VEC: a thread's columns are all in the row or all past it,
// and what it reads there is zero already, so this is for what a mean was taken from.
template <bool VEC> __device__ __forceinline__ void cut8(float2 (&v)[4], const Cols& cs) {
  if constexpr (VEC) {
    const float live = cs.col < cs.D ? 1.f : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], both(live));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = make_float2(cs.col + 2 * i < cs.D ? v[i].x : 0.f, cs.col + 2 * i + 1 < cs.D ? v[i].y : 0.f);
  }
}

// Scratch of the sums: two barriers and two buffers of a cluster's sums, two buffers of all
// warps' sums.
constexpr int kClusterWords = 4 + 2 * RowSum<false>::kMaxValues * kBnMaxCluster;
constexpr int kRowSumWords = kClusterWords + 2 * RowSum<false>::kMaxValues * kBnMaxThreads / 32;

template <bool CLUSTER>
__device__ __forceinline__ RowSum<CLUSTER> row_sum(float* scratch, const RowThread& r, int threads_per_row, int cluster, int D) {
  RowSum<CLUSTER> rs;
  rs.D = D;
  const int cols = D - (r.col - 8 * r.t), most = 8 * threads_per_row;  // columns from this block's first on
  rs.full = (cols < 0 ? 0 : cols < most ? cols : most) / 256;
  rs.part = cols < 0 || cols >= most ? 0 : cols % 256;
  rs.part_inv = rs.part > 0 ? 1.f / float(rs.part) : 0.f;
  rs.clus = scratch + 4;  // behind the cluster's two barriers
  rs.nw = threads_per_row / 32;
  rs.buf = scratch + kClusterWords + r.group * 2 * RowSum<false>::kMaxValues * rs.nw;
  for (int i = int(threadIdx.x); i < kRowSumWords; i += int(blockDim.x)) scratch[i] = 0.f;
  __syncthreads();
  if (CLUSTER && threadIdx.x == 0) {
    mbar_init(reinterpret_cast<uint64_t*>(scratch), 1);
    mbar_init(reinterpret_cast<uint64_t*>(scratch) + 1, 1);
    fence_barrier_init();  // for the other blocks, which the kernel's first cluster barrier waits for
  }
  rs.warp = r.t / 32;
  rs.lane = r.t % 32;
  rs.bar = 1 + r.group;
  rs.threads = threads_per_row;
  rs.blocks = cluster;
  rs.turn = 0;
  return rs;
}

// Means (0 for the RMS norm) and 1 / sqrt(mean of the squared distances from it + eps) of R
// rows; get(r, v) gives a row's eight values. A layer norm's warps first take the mean and the
// squared distances from it over their own columns, so one sum over the row's warps is enough
// and a large common offset costs no precision.
template <int R, bool VEC, bool LAYER, typename SUM, typename F>
__device__ __forceinline__ void row_stats(F&& get, const Cols& cs, bool layer, float eps, float inv_d, SUM& rs,
                                          float (&mean)[R], float (&rstd)[R]) {
  if (LAYER && layer) {
    const float inv_n = rs.inv_columns(rs.warp);
    float v1[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float2 v[4];
      get(r, v);
      v1[r] = sum8(v);
    }
    const float s = rs.scatter_sum(v1);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float2 v[4];
      get(r, v);
      const float m = __shfl_sync(0xffffffffu, s, r * (32 / R)) * inv_n;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = add2(v[i], both(-m));
      cut8<VEC>(v, cs);
      v1[r] = dot8(v, v);
    }
    const float q = rs.scatter_sum(v1);
    rs.merge(s, q, inv_d, mean, rstd);
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float2 v[4];
      get(r, v);
      mean[r] = 0.f;
      rstd[r] = dot8(v, v);
    }
    rs.sum(rstd);
  }
#pragma unroll
  for (int r = 0; r < R; ++r) rstd[r] = rsqrtf(rstd[r] * inv_d + eps);
}

// What a kernel's code has: the norm after the block, a gate (for groups of rows or for each), and
// (FULL) the means of layer norms and biases. A kernel takes what has less at run time.
template <typename TX, typename TR, bool VEC, bool CLUSTER, int FEAT>
__global__ void __launch_bounds__(bn_max_threads(FEAT, VEC, CLUSTER), 1)
    flce_block_norm_forward_kernel(const __grid_constant__ BlockNormParams p, int threads_per_row, int blocks_per_row, int batches, int per) {
  constexpr int R = kBnRows;
  const int cluster = CLUSTER ? blocks_per_row : 1;
  constexpr bool POST = (FEAT & BN_POST) != 0, GATE = (FEAT & BN_GATE) != 0, FULL = (FEAT & BN_FULL) != 0;
  __shared__ __align__(128) float scratch[kRowSumWords];
  // (aligned to lines: with planes across them every access takes one more, 12% of the backward)
  extern __shared__ __align__(128) char ring_smem[];
  constexpr int kX = 0, kR = sizeof(TX) / 2, kG = kR + sizeof(TR) / 2;  // planes of x, residual and full gate
  constexpr int kParams = bn_shared_params(FEAT, false);
  const RowThread r0 = row_thread(threads_per_row, cluster);
  RowSum<CLUSTER> rs = row_sum<CLUSTER>(scratch, r0, threads_per_row, cluster, p.D);
  const int col = r0.col, D = p.D;
  const Cols cs{col, D};
  // else a thread (or, where warps copy together, a warp) past the row, whose values are zero
  const bool copies = (VEC ? col : RowRing<VEC>::warp_col(cs)) < D;
  const bool post = POST && p.w1 != nullptr, pre = p.w2 != nullptr, gate = GATE && p.gate != nullptr;
  constexpr bool gate_full = GATE && (FEAT & BN_GATE_ROWS) != 0;  // a gate for each row, else for groups of rows
  const int lo = int(r0.worker * p.chunk_rows < p.N ? r0.worker * p.chunk_rows : p.N);
  const int hi = int(lo + p.chunk_rows < p.N ? lo + p.chunk_rows : p.N);
  RowRing<VEC> ring{};
  int next = lo;  // the row that is copied next
  auto fetch = [&](uint32_t at) FLCE_INLINE {
    if (!VEC) __syncwarp();  // the warp has read what was there
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (!copies || r >= per || next + r >= hi) continue;
      const uint32_t to = at + uint32_t(r * ring.row_bytes);
      ring.copy(to, kX, p.x, row_at<TX>(p.x, next + r, p.ld_x), cs);
      if (p.residual != nullptr) ring.copy(to, kR, p.residual, row_at<TR>(p.residual, next + r, p.ld_residual), cs);
      if (gate_full && p.gate_res_type) ring.copy(to, kG, p.gate, row_at<TR>(p.gate, next + r, p.ld_gate), cs);
      if (gate_full && !p.gate_res_type) ring.copy(to, kG, p.gate, row_at<TX>(p.gate, next + r, p.ld_gate), cs);
    }
    next += per;
    ring.commit();
  };
  // Waits for the batch in slot `at`, whose first row is `row`.
  auto arrive = [&](uint32_t at, int row) FLCE_INLINE {
    ring.wait(batches - 1);
    if constexpr (!VEC) {
      __syncwarp();
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (!copies || r >= per || row + r >= hi) continue;
        const uint32_t to = at + uint32_t(r * ring.row_bytes);
        Raw8<TR> res = raw_zero<TR>(), gr = raw_zero<TR>();
        Raw8<TX> gx = raw_zero<TX>();
        const Raw8<TX> x = ring.take(to, kX, row_at<TX>(p.x, row + r, p.ld_x), cs);
        if (p.residual != nullptr) res = ring.take(to, kR, row_at<TR>(p.residual, row + r, p.ld_residual), cs);
        if (gate_full && p.gate_res_type) gr = ring.take(to, kG, row_at<TR>(p.gate, row + r, p.ld_gate), cs);
        if (gate_full && !p.gate_res_type) gx = ring.take(to, kG, row_at<TX>(p.gate, row + r, p.ld_gate), cs);
        __syncwarp();
        ring.land(to, kX, x);
        if (p.residual != nullptr) ring.land(to, kR, res);
        if (gate_full && p.gate_res_type) ring.land(to, kG, gr);
        if (gate_full && !p.gate_res_type) ring.land(to, kG, gx);
      }
    }
  };
  constexpr int kShift = bn_ring_shift(sizeof(TX), sizeof(TR), VEC, FEAT, CLUSTER ? 2 : 1, false);
  ring.init(ring_smem + kShift + (FULL ? kParams * 32 * threads_per_row : 0), kG + (gate_full ? int(sizeof(TR)) / 2 : 0), batches, per);
  for (uint32_t at = ring.first; at != ring.end; at += ring.batch_bytes) fetch(at);
  if (CLUSTER) cluster_sync_all();
  // Without FULL, c is what a row's value after the first norm is multiplied by: w1 scale
  // act(gate). With it w1 scale and b1 scale are in shared memory, and c is act(gate).
  float2 w1[4], w2[4], c[4];
  const int t16 = 16 * r0.t, plane = 16 * threads_per_row;  // a parameter's values for this thread
  auto param = [&](int index, float2 (&f)[4]) FLCE_INLINE { shared_get(ring_smem, t16 + 2 * index * plane, plane, f); };
  auto set_param = [&](int index, const float2 (&f)[4]) FLCE_INLINE {
    if (r0.group == 0) shared_set(ring_smem, t16 + 2 * index * plane, plane, f);
  };
  constexpr int kW2 = 0, kB2 = 1, kW1 = 2, kB1 = 3;
  load_weight<VEC>(p.w1, p.w1_dt, p.w_off, cs, w1);
  load_weight<VEC>(p.w2, p.w2_dt, p.w_off, cs, w2);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w1[i] = post ? mul2(w1[i], both(p.scale)) : both(p.scale);
    c[i] = FULL ? both(1.f) : w1[i];
  }
  if (FULL) {
    float2 b[4];
    set_param(kW2, w2);
    set_param(kW1, w1);
    load_weight<VEC>(p.b2, p.b2_dt, 0.f, cs, b);
    set_param(kB2, b);
    load_weight<VEC>(p.b1, p.b1_dt, 0.f, cs, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = mul2(b[i], both(p.scale));
    set_param(kB1, b);
    __syncthreads();
  }
  auto set_gate = [&](const float2(&a)[4]) FLCE_INLINE {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = FULL ? a[i] : mul2(w1[i], a[i]);
  };
  const float inv_d = 1.f / float(D);
  int gate_end = lo;  // first row whose gate is not in c
  // The first norm of a batch and the second norm of the batch before it share a sum: the
  // latency of a batch is one sum, and what comes before and after it is independent work.
  uint32_t batch = ring.first;
  float m1[R], r1[R];
#pragma unroll
  for (int r = 0; r < R; ++r) m1[r] = 0.f, r1[r] = 1.f;
  if (lo < hi) {
    arrive(batch, lo);
    if (post) row_stats<R, VEC, FULL, RowSum<CLUSTER>>([&](int r, float2 (&v)[4]) { ring.template get<TX>(batch, r, kX, v); }, cs, p.layer, p.eps, inv_d, rs, m1, r1);
  }
  for (int row = lo; row < hi; row += per) {
    const bool second = per > 1 && row + 1 < hi;  // the last batch may have one row
    float2 h[R][4];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r > 0 && !second) {
#pragma unroll
        for (int i = 0; i < 4; ++i) h[r][i] = both(0.f);
        continue;
      }
      if (gate_full) {
        float2 a[4];
        if (p.gate_res_type)
          ring.template get<TR>(batch, r, kG, a);
        else
          ring.template get<TX>(batch, r, kG, a);
        activate8<true>(a, p.act);
        set_gate(a);
      } else if (gate && row + r >= gate_end) {
        const int g = (row + r) / int(p.gate_group);
        float2 a[4];
        load_gate<TX, TR, VEC>(p, g, cs, a);
        activate8<true>(a, p.act);
        set_gate(a);
        gate_end = int((g + 1) * p.gate_group);
      }
      float2 u[4];
      ring.template get<TX>(batch, r, kX, u);
      ring.template get<TR>(batch, r, kR, h[r]);
      if (FULL) {
        float2 w[4], b[4];
        param(kW1, w);
        param(kB1, b);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          u[i] = fma2(mul2(add2(u[i], both(-m1[r])), both(r1[r])), w[i], b[i]);
          h[r][i] = GATE ? fma2(u[i], c[i], h[r][i]) : add2(u[i], h[r][i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (POST) u[i] = mul2(u[i], both(r1[r]));
          h[r][i] = fma2(u[i], c[i], h[r][i]);
        }
      }
      store8<TR, VEC>(row_at<TR>(p.h, row + r, D), cs, h[r]);
    }
    float m2[R], r2[R], n1[R], k1[R];
#pragma unroll
    for (int r = 0; r < R; ++r) m2[r] = r2[r] = n1[r] = 0.f, k1[r] = 1.f;
    fetch(batch);
    batch = ring.after(batch);
    arrive(batch, row + per);
    auto get_h = [&](int r, float2 (&v)[4]) FLCE_INLINE {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = h[r][i];
    };
    if (post && pre) {
      float mean[2 * R], rstd[2 * R];
      row_stats<2 * R, VEC, FULL, RowSum<CLUSTER>>(
          [&](int r, float2 (&v)[4]) {
            if (r < R)
              get_h(r, v);
            else
              ring.template get<TX>(batch, r - R, kX, v);
          },
          cs, p.layer, p.eps, inv_d, rs, mean, rstd);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        m2[r] = mean[r];
        r2[r] = rstd[r];
        n1[r] = mean[R + r];
        k1[r] = rstd[R + r];
      }
    } else if (pre) {
      row_stats<R, VEC, FULL, RowSum<CLUSTER>>(get_h, cs, p.layer, p.eps, inv_d, rs, m2, r2);
    } else if (post) {
      row_stats<R, VEC, FULL, RowSum<CLUSTER>>([&](int r, float2 (&v)[4]) { ring.template get<TX>(batch, r, kX, v); }, cs, p.layer, p.eps, inv_d, rs, n1, k1);
    }
    if (pre) {
      float2 b2[4];
      if (FULL) {
        param(kW2, w2);
        param(kB2, b2);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (r > 0 && !second) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (FULL)
            h[r][i] = fma2(mul2(add2(h[r][i], both(-m2[r])), both(r2[r])), w2[i], b2[i]);
          else
            h[r][i] = mul2(mul2(h[r][i], both(r2[r])), w2[i]);
        }
        store8<TX, VEC>(row_at<TX>(p.y, row + r, D), cs, h[r]);
      }
    }
    if (p.stats != nullptr && col == 0) {
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (r == 0 || second) reinterpret_cast<float4*>(p.stats)[row + r] = make_float4(m1[r], r1[r], m2[r], r2[r]);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m1[r] = n1[r];
      r1[r] = k1[r];
    }
  }
  if (CLUSTER) cluster_sync_all();  // no block leaves while another may still write to it
}

// The rows that it reads are x and the stored h: with a 16-bit residual stream that is h rounded to it, while
// the statistics (and the forward's y) are of the unrounded one. The stream's gradient hardly sees it; the
// weight's gradient, a sum of dy n, has that rounding beside its own (bf16: 2.4e-3 off, 1.7e-3 without). A
// caller that wants neither keeps the stream in fp32.
// With n = (v - m) r and g = upstream * w, a norm's gradient is r (g - mean(g) - n mean(g n)) =
// r g - r mean(g) - (v - m) r^3 mean(g (v - m)): it is computed in the last form, from the row's
// own values, so a norm costs two sums in which no normalised row is formed.
template <typename TX, typename TR, bool VEC, bool CLUSTER, int FEAT>
__global__ void __launch_bounds__(kBnThreads, 1)
    flce_block_norm_backward_kernel(const __grid_constant__ BlockNormParams p, int threads_per_row, int blocks_per_row, int batches, int per) {
  constexpr int R = kBnRows;
  const int cluster = CLUSTER ? blocks_per_row : 1;
  constexpr bool POST = (FEAT & BN_POST) != 0, GATE = (FEAT & BN_GATE) != 0, FULL = (FEAT & BN_FULL) != 0;
  __shared__ __align__(128) float scratch[kRowSumWords];
  // (aligned to lines: with planes across them every access takes one more, 12% of the backward)
  extern __shared__ __align__(128) char ring_smem[];
  constexpr int kX = 0, kY = sizeof(TX) / 2, kH = 2 * kY, kDh = kH + sizeof(TR) / 2, kG = kDh + sizeof(TR) / 2;  // planes
  constexpr int kParams = bn_shared_params(FEAT, true);
  // in shared memory: a bias's sum, and with a gate that and both biases' sums
  constexpr bool OWN_B = POST && FULL, OWN_A = POST && GATE && FULL;
  const RowThread r0 = row_thread(threads_per_row, cluster);
  RowSum<CLUSTER> rs = row_sum<CLUSTER>(scratch, r0, threads_per_row, cluster, p.D);
  const int col = r0.col, D = p.D;
  const Cols cs{col, D};
  const bool post = POST && p.w1 != nullptr, pre = p.w2 != nullptr, gate = GATE && p.gate != nullptr;
  constexpr bool gate_full = GATE && (FEAT & BN_GATE_ROWS) != 0;  // a gate for each row, else for groups of rows
  const int workers = int(gridDim.x) / cluster * (int(blockDim.x) / threads_per_row);
  const bool live_col = col < D;
  const bool copies = (VEC ? col : RowRing<VEC>::warp_col(cs)) < D;
  // the worker's rows: chunk after chunk, once for the copies and once, behind them, for the work
  struct Rows {
    int chunk, row, hi;
  };
  auto open = [&](Rows& w) FLCE_INLINE {
    if (w.chunk >= p.chunks) return;
    const int group = w.chunk / int(p.chunks_per_group);
    const int first = group * int(p.group_rows), end = first + int(p.group_rows);
    w.row = first + (w.chunk - group * int(p.chunks_per_group)) * int(p.chunk_rows);
    w.hi = end - w.row < int(p.chunk_rows) ? end : w.row + int(p.chunk_rows);
  };
  RowRing<VEC> ring{};
  Rows ahead{int(r0.worker), 0, 0};
  open(ahead);
  // a batch's statistics: copied by the first lanes of each warp for the warp alone
  __shared__ __align__(16) float4 warp_stats[kBnThreads / 32][kBnMaxBatches][R];
  const float4* stats = reinterpret_cast<const float4*>(p.stats);
  const uint32_t stat_at = smem_addr(&warp_stats[threadIdx.x / 32][0][0]);
  int stat_slot = 0;
  auto fetch = [&](uint32_t at) FLCE_INLINE {
    if (ahead.chunk < p.chunks) {
      if (rs.lane < R) {  // the rows' statistics, for this warp
        const int row = ahead.row + (rs.lane < per && ahead.row + rs.lane < ahead.hi ? rs.lane : 0);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(stat_at + uint32_t(stat_slot * R + rs.lane) * 16u),
                     "l"(stats + row)
                     : "memory");
      }
      if (copies) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          if (r > 0 && (r >= per || ahead.row + r >= ahead.hi)) continue;
          const uint32_t to = at + uint32_t(r * ring.row_bytes);
          const int row = ahead.row + r;
          ring.copy(to, kX, p.x, row_at<TX>(p.x, row, p.ld_x), cs);
          if (pre) ring.copy(to, kH, p.h_in, row_at<TR>(p.h_in, row, D), cs);
          if (p.dh != nullptr) ring.copy(to, kDh, p.dh, row_at<TR>(p.dh, row, p.ld_dh), cs);
          if (pre && p.dy != nullptr) ring.copy(to, kY, p.dy, row_at<TX>(p.dy, row, p.ld_dy), cs);
          if (gate_full && p.gate_res_type) ring.copy(to, kG, p.gate, row_at<TR>(p.gate, row, p.ld_gate), cs);
          if (gate_full && !p.gate_res_type) ring.copy(to, kG, p.gate, row_at<TX>(p.gate, row, p.ld_gate), cs);
        }
      }
      ahead.row += per;
      if (ahead.row >= ahead.hi) {
        ahead.chunk += workers;
        open(ahead);
      }
    }
    ring.commit();
    stat_slot = stat_slot + 1 == batches ? 0 : stat_slot + 1;
  };
  // Waits until all but the newest `left` batches have landed, the last of them in slot `at`, rows w.
  auto arrive = [&](int left, uint32_t at, const Rows& w) FLCE_INLINE {
    ring.wait(left);
    __syncwarp();
    if constexpr (!VEC) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (!copies || (r > 0 && (r >= per || w.row + r >= w.hi))) continue;
        const uint32_t to = at + uint32_t(r * ring.row_bytes);
        const int row = w.row + r;
        {
          Raw8<TR> h = raw_zero<TR>();
          const Raw8<TX> x = ring.take(to, kX, row_at<TX>(p.x, row, p.ld_x), cs);
          if (pre) h = ring.take(to, kH, row_at<TR>(p.h_in, row, D), cs);
          __syncwarp();
          ring.land(to, kX, x);
          ring.land(to, kH, h);
        }
        Raw8<TR> dh = raw_zero<TR>();
        Raw8<TX> dy = raw_zero<TX>();
        if (p.dh != nullptr) dh = ring.take(to, kDh, row_at<TR>(p.dh, row, p.ld_dh), cs);
        if (pre && p.dy != nullptr) dy = ring.take(to, kY, row_at<TX>(p.dy, row, p.ld_dy), cs);
        __syncwarp();
        ring.land(to, kDh, dh);
        ring.land(to, kY, dy);
        if (gate_full && p.gate_res_type) {
          const Raw8<TR> g = ring.take(to, kG, row_at<TR>(p.gate, row, p.ld_gate), cs);
          __syncwarp();
          ring.land(to, kG, g);
        } else if (gate_full) {
          const Raw8<TX> g = ring.take(to, kG, row_at<TX>(p.gate, row, p.ld_gate), cs);
          __syncwarp();
          ring.land(to, kG, g);
        }
      }
    }
  };
  ring.init(ring_smem + kParams * 32 * threads_per_row + bn_own_params(FEAT, true) * 32 * int(blockDim.x),
            kG + (gate_full ? int(sizeof(TR)) / 2 : 0), batches, per);
  for (uint32_t at = ring.first; at != ring.end; at += ring.batch_bytes) fetch(at);
  if (CLUSTER) cluster_sync_all();
  float2 w1[4], w2[4], a[4], dw1[4], db1[4], dw2[4], db2[4];
  const int t16 = 16 * r0.t, plane = 16 * threads_per_row;  // a parameter's values for this thread
  auto param = [&](int index, float2 (&f)[4]) FLCE_INLINE { shared_get(ring_smem, t16 + 2 * index * plane, plane, f); };
  auto set_param = [&](int index, const float2 (&f)[4]) FLCE_INLINE {
    if (r0.group == 0) shared_set(ring_smem, t16 + 2 * index * plane, plane, f);
  };
  constexpr int kW2 = 0, kW1 = 1;
  // the thread's own values follow the parameters
  const int own_plane = 16 * int(blockDim.x), own_at = 2 * kParams * plane + 16 * int(threadIdx.x);
  auto own = [&](int index, float2 (&f)[4]) FLCE_INLINE { shared_get(ring_smem, own_at + 2 * index * own_plane, own_plane, f); };
  auto set_own = [&](int index, const float2 (&f)[4]) FLCE_INLINE {
    shared_set(ring_smem, own_at + 2 * index * own_plane, own_plane, f);
  };
  constexpr int kDb1 = 0, kA = 1, kDb2 = 2;
  load_weight<VEC>(p.w2, p.w2_dt, p.w_off, cs, w2);
  if (POST) load_weight<VEC>(p.w1, p.w1_dt, p.w_off, cs, w1);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = both(1.f);
    if (!post) w1[i] = both(1.f);
    dw1[i] = db1[i] = dw2[i] = db2[i] = both(0.f);
  }
  if (FULL) {
    set_param(kW2, w2);
    if (POST) set_param(kW1, w1);
    __syncthreads();
  }
  if (OWN_A) set_own(kDb2, db2);
  if (OWN_B) set_own(kDb1, db1);
  const float inv_d = 1.f / float(D), inv_d0 = p.layer ? inv_d : 0.f;
  const float live = live_col ? 1.f : 0.f;  // threads past the row: their values stay zero
  // values of row r of the batch in slot `at`
  auto get_x = [&](uint32_t at, int r, float m1, float2 (&v)[4]) FLCE_INLINE {
    ring.template get<TX>(at, r, kX, v);
    if (FULL && POST) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = add2(v[i], both(-m1));
    }
  };
  auto get_h = [&](uint32_t at, int r, float m2, float2 (&v)[4]) FLCE_INLINE {
    ring.template get<TR>(at, r, kH, v);
    if (FULL) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = add2(v[i], both(-m2));
    }
  };
  auto get_stats = [&](int slot, int r) FLCE_INLINE {
    float4 s = warp_stats[threadIdx.x / 32][slot][r];
    s.y = post ? s.y * live : live;
    s.w *= live;
    return s;
  };
  auto step = [&](Rows& w) FLCE_INLINE {
    w.row += per;
    if (w.row >= w.hi) {
      w.chunk += workers;
      open(w);
    }
  };
  // Sums of the second norm's gradient over the batch's rows: s1 of g (h - mean), s0 of g.
  auto second_norm = [&](uint32_t at, int slot, const Rows& w, float (&s1)[R], float (&s0)[R]) FLCE_INLINE {
    if (FULL) param(kW2, w2);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      s1[r] = s0[r] = 0.f;
      if (r > 0 && (r >= per || w.row + r >= w.hi)) continue;
      const float4 st = get_stats(slot, r);
      float2 n[4], g[4];
      get_h(at, r, st.z, n);
      ring.template get<TX>(at, r, kY, g);
#pragma unroll
      for (int i = 0; i < 4; ++i) g[i] = mul2(g[i], w2[i]);
      s1[r] = dot8(g, n);
      if (FULL) s0[r] = sum8(g);
    }
  };
  // A batch's sums of the first norm and the next batch's sums of the second share a sum over
  // the row's threads, so a batch costs the latency of one.
  auto total = [&](float (&t1)[R], float (&t0)[R], float (&s1)[R], float (&s0)[R]) FLCE_INLINE {
    constexpr int kOf = POST ? 2 : 1;
    float v[kOf * R * (FULL ? 2 : 1)];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      v[r] = s1[r];
      if (POST) v[R + r] = t1[r];
      if (FULL) v[kOf * R + r] = s0[r];
      if (FULL && POST) v[kOf * R + R + r] = t0[r];
    }
    rs.sum(v);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      s1[r] = v[r];
      if (POST) t1[r] = v[R + r];
      if (FULL) s0[r] = v[kOf * R + r];
      if (FULL && POST) t0[r] = v[kOf * R + R + r];
    }
  };
  Rows now{int(r0.worker), 0, 0};
  open(now);
  uint32_t batch = ring.first;
  int slot = 0;
  auto enter = [&](int chunk) FLCE_INLINE {  // a chunk has one gate row
    if (gate && !gate_full && chunk < p.chunks) {
      load_gate<TX, TR, VEC>(p, chunk / int(p.chunks_per_group), cs, a);
      activate8<false>(a, p.act);
      if (OWN_A) set_own(kA, a);
    }
  };
  enter(now.chunk);
  float s1[R], s0[R], t1[R], t0[R];
#pragma unroll
  for (int r = 0; r < R; ++r) s1[r] = s0[r] = t1[r] = t0[r] = 0.f;
  if (now.chunk < p.chunks && pre) {
    arrive(batches - 1, batch, now);
    second_norm(batch, slot, now, s1, s0);
    total(t1, t0, s1, s0);
  }
  while (now.chunk < p.chunks) {
    const int row = now.row;
    const bool second = per > 1 && row + 1 < now.hi;  // a chunk's last batch may have one row
    Rows next = now;
    step(next);
    if (!pre) arrive(batches - 1, batch, now);
    float2 d[R][4];  // the gradient of h, then what the first norm's gradient is taken of
    if (FULL && POST) param(kW1, w1);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      t1[r] = t0[r] = 0.f;
      if (r > 0 && !second) continue;
      const float4 st = get_stats(slot, r);
      ring.template get<TR>(batch, r, kDh, d[r]);
      if (pre) {
        float2 n[4], g[4];
        get_h(batch, r, st.z, n);
        ring.template get<TX>(batch, r, kY, g);
        if (FULL) param(kW2, w2);
        if (FULL) {
          if (OWN_A) own(kDb2, db2);
#pragma unroll
          for (int i = 0; i < 4; ++i) db2[i] = add2(db2[i], g[i]);
          if (OWN_A) set_own(kDb2, db2);
        }
        const float2 k1 = both(-(s1[r] * st.w * inv_d) * st.w * st.w), k0 = both(-st.w * (s0[r] * inv_d0)), k = both(st.w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          d[r][i] = fma2(n[i], k1, d[r][i]);
          if (FULL) d[r][i] = add2(d[r][i], k0);
          g[i] = mul2(g[i], k);
          d[r][i] = fma2(g[i], w2[i], d[r][i]);
          dw2[i] = fma2(g[i], n[i], dw2[i]);
        }
        if (!VEC && FULL) cut8<VEC>(d[r], cs);
      }
      if (p.dres != nullptr) store8<TR, VEC>(row_at<TR>(p.dres, row + r, D), cs, d[r]);
      float2 x[4];
      if (POST || GATE) get_x(batch, r, st.x, x);
      if (gate_full) {
        if (p.gate_res_type)
          ring.template get<TR>(batch, r, kG, a);
        else
          ring.template get<TX>(batch, r, kG, a);
        if (p.dgate == nullptr) {
          activate8<false>(a, p.act);
        } else {  // d u scale act', u = (x - m) r w1 + b1, or x
          float2 e[4], da[4];
          activate_derive8(a, p.act, da);
          if (FULL && post) load_weight<VEC>(p.b1, p.b1_dt, 0.f, cs, e);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float2 u = x[i];
            if (POST) u = mul2(mul2(u, both(st.y)), w1[i]);
            if (FULL && post) u = add2(u, e[i]);
            e[i] = mul2(mul2(u, d[r][i]), mul2(da[i], both(p.scale)));
          }
          if (p.gate_res_type)
            store8<TR, VEC>(static_cast<TR*>(p.dgate) + int64_t(row + r) * D, cs, e);
          else
            store8<TX, VEC>(static_cast<TX*>(p.dgate) + int64_t(row + r) * D, cs, e);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) d[r][i] = mul2(d[r][i], a[i]);
      }
      if (POST || GATE) {
        const float2 k = both(st.y);
#pragma unroll
        for (int i = 0; i < 4; ++i) dw1[i] = fma2(mul2(d[r][i], k), x[i], dw1[i]);
        if (OWN_B) own(kDb1, db1);
        if (FULL) {
#pragma unroll
          for (int i = 0; i < 4; ++i) db1[i] = add2(db1[i], d[r][i]);
        }
        if (OWN_B) set_own(kDb1, db1);
      }
      if (gate && !gate_full) {
        if (OWN_A) own(kA, a);
#pragma unroll
        for (int i = 0; i < 4; ++i) d[r][i] = mul2(d[r][i], a[i]);
      }
      if (post) {
#pragma unroll
        for (int i = 0; i < 4; ++i) d[r][i] = mul2(d[r][i], w1[i]);
        t1[r] = dot8(d[r], x);
        if (FULL) t0[r] = sum8(d[r]);
      }
    }
    const uint32_t batch_next = ring.after(batch);
    const int slot_next = slot + 1 == batches ? 0 : slot + 1;
    if (pre && next.chunk < p.chunks) {
      arrive(batches - 2, batch_next, next);
      second_norm(batch_next, slot_next, next, s1, s0);
    }
    if (pre || post) total(t1, t0, s1, s0);
    if (p.dx != nullptr) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (r > 0 && !second) continue;
        if (post) {
          const float4 st = get_stats(slot, r);
          float2 x[4];
          get_x(batch, r, st.x, x);
          const float s = st.y * p.scale;
          const float2 k1 = both(-(t1[r] * st.y * inv_d) * st.y * s), k0 = both(-s * (t0[r] * inv_d0)), k = both(s);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (FULL)
              d[r][i] = fma2(d[r][i], k, fma2(x[i], k1, k0));
            else
              d[r][i] = fma2(d[r][i], k, mul2(x[i], k1));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) d[r][i] = mul2(d[r][i], both(p.scale));
        }
        store8<TX, VEC>(row_at<TX>(p.dx, row + r, D), cs, d[r]);
      }
    }
    __syncwarp();  // the warp has read the batch's statistics
    fetch(batch);
    // The end of a gate group's chunk. With P = sum of d n and Q = sum of d over its rows (d before
    // the gate, n = (x - m) r), the gate's gradient is (w1 P + b1 Q) scale act', and the chunk's
    // part of w1's and b1's is scale a P and scale a Q.
    if (gate && !gate_full && next.chunk != now.chunk) {
      float2 e[4], q[4];
      if (OWN_B) own(kDb1, db1);
      if (FULL && POST) param(kW1, w1);
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] = mul2(dw1[i], w1[i]);
      if (FULL && POST) {
        load_weight<VEC>(p.b1, p.b1_dt, 0.f, cs, q);
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = fma2(db1[i], q[i], e[i]);
      }
      load_gate<TX, TR, VEC>(p, now.chunk / int(p.chunks_per_group), cs, q);
      derive8(q, p.act, q);
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] = mul2(e[i], mul2(q[i], both(p.scale)));
      if (OWN_A) own(kA, a);
      if (p.dgate == nullptr) {
      } else if (p.part_gate != nullptr) {
        store8<float, VEC>(p.part_gate + int64_t(now.chunk) * D, cs, e);
      } else if (p.gate_res_type) {
        store8<TR, VEC>(static_cast<TR*>(p.dgate) + int64_t(now.chunk / int(p.chunks_per_group)) * D, cs, e);
      } else {
        store8<TX, VEC>(static_cast<TX*>(p.dgate) + int64_t(now.chunk / int(p.chunks_per_group)) * D, cs, e);
      }
      // the worker's sums of w1 and b1 over its chunks are in the workspace
      auto add_part = [&](float* part, const float2 (&v)[4]) FLCE_INLINE {
        if (part == nullptr) return;
        float* at = part + r0.worker * D;
        float2 sum[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] = both(0.f);
        if (now.chunk != int(r0.worker)) unpack8(load8<float, VEC>(at, cs), sum);
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] = fma2(v[i], mul2(a[i], both(p.scale)), sum[i]);
        store8<float, VEC>(at, cs, sum);
      };
      if (POST) add_part(p.part[0], dw1);
      if (POST && FULL) add_part(p.part[1], db1);
#pragma unroll
      for (int i = 0; i < 4; ++i) dw1[i] = db1[i] = both(0.f);
      if (OWN_B) set_own(kDb1, db1);
    }
    if (next.chunk != now.chunk) enter(next.chunk);
    batch = batch_next;
    slot = slot_next;
    now = next;
  }
  // one partial sum a block and parameter: the block's row groups first
  const int groups = int(blockDim.x) / threads_per_row;
  const int64_t block = int64_t(int(blockIdx.x) / cluster);
  // every copy has been waited for but the empty ones past the last row: the room is free
  float2* fold = reinterpret_cast<float2*>(ring_smem);  // [threads][4]
  auto flush = [&](float* part, const float2(&v)[4], float scale) FLCE_INLINE {
    if (part == nullptr) return;
    float2 s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = v[i];
    if (groups > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) fold[threadIdx.x * 4 + i] = v[i];
      __syncthreads();
      if (r0.group != 0) return;
      for (int q = 1; q < groups; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = add2(s[i], fold[(q * threads_per_row + r0.t) * 4 + i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = mul2(s[i], both(scale));
    store8<float, VEC>(part + block * D, cs, s);
  };
  if (OWN_A) own(kDb2, db2);
  if (OWN_B) {
    own(kDb1, db1);
    __syncthreads();  // the sums' room is used again
  }
  if (!gate || gate_full) {
    if (POST) flush(p.part[0], dw1, p.scale);
    if (POST && FULL) flush(p.part[1], db1, p.scale);
  } else if (r0.worker >= p.chunks) {  // a worker without a chunk: its sums are zero
    if (POST && p.part[0] != nullptr) store8<float, VEC>(p.part[0] + r0.worker * D, cs, dw1);
    if (POST && FULL && p.part[1] != nullptr) store8<float, VEC>(p.part[1] + r0.worker * D, cs, dw1);
  }
  flush(p.part[2], dw2, 1.f);
  if (FULL) flush(p.part[3], db2, 1.f);
  if (CLUSTER) cluster_sync_all();
}

template <typename K>
cudaError_t bn_launch(K kernel, const BlockNormParams& p, const BlockNormShape& s, unsigned blocks, int planes, int shift, bool vec,
                      int feat, bool backward, cudaStream_t stream) {
  const int threads = s.threads_per_row * s.rows_per_block;
  const BnRing r = bn_ring(s, planes, vec, feat, backward);
  size_t smem = size_t(shift) + size_t(r.params_bytes) + size_t(bn_row_bytes(threads, planes, vec)) * r.per * r.batches;
  if (smem < size_t(threads) * 32) smem = size_t(threads) * 32;  // row groups add up their sums in it
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBnSmemBytes + 128);  // (with its shift)
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(blocks * unsigned(s.cluster));
  c.blockDim = dim3(unsigned(threads));
  c.dynamicSmemBytes = smem;
  c.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = unsigned(s.cluster);
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = 1;
  e = cudaLaunchKernelEx(&c, kernel, p, s.threads_per_row, s.cluster, r.batches, r.per);
  if (e == cudaSuccess) count_launch();
  return e;
}

// The kernel of a feature set (as bn_kernel_features gives it); the argument: more of one row a block.
#define FLCE_BN_CASE(VEC, CLUSTER, FEAT) \
  case FEAT:                                                                                                          \
    return bn_launch(KERNEL<TX, TR, VEC, CLUSTER, FEAT>, p, s, blocks, planes,                                        \
                     bn_ring_shift(sizeof(TX), sizeof(TR), VEC, FEAT, s.cluster, BACKWARD), VEC, FEAT, BACKWARD, stream)
#define FLCE_BN_WIDE_CASES FLCE_BN_CASE(true, false, 23); FLCE_BN_CASE(true, false, 31)
#define FLCE_BN_DISPATCH(...)                                                               \
  const int planes = bn_planes(int(sizeof(TX)), int(sizeof(TR)), p.gate_full, BACKWARD);    \
  if (!vec && s.cluster > 1) {                                                              \
    switch (feat) { FLCE_BN_CASE(false, true, 7); FLCE_BN_CASE(false, true, 15); }          \
  } else if (!vec) {                                                                        \
    switch (feat) { FLCE_BN_CASE(false, false, 7); FLCE_BN_CASE(false, false, 15); }        \
  } else if (s.cluster > 1) {                                                               \
    switch (feat) {                                                                         \
      FLCE_BN_CASE(true, true, 0);                                                          \
      FLCE_BN_CASE(true, true, 1);                                                          \
      FLCE_BN_CASE(true, true, 7);                                                          \
      FLCE_BN_CASE(true, true, 15);                                                         \
    }                                                                                       \
  } else {                                                                                  \
    switch (feat) {                                                                         \
      FLCE_BN_CASE(true, false, 0);                                                         \
      FLCE_BN_CASE(true, false, 1);                                                         \
      FLCE_BN_CASE(true, false, 2);                                                         \
      FLCE_BN_CASE(true, false, 3);                                                         \
      FLCE_BN_CASE(true, false, 4);                                                         \
      FLCE_BN_CASE(true, false, 5);                                                         \
      FLCE_BN_CASE(true, false, 6);                                                         \
      FLCE_BN_CASE(true, false, 7);                                                         \
      FLCE_BN_CASE(true, false, 10);                                                        \
      FLCE_BN_CASE(true, false, 11);                                                        \
      FLCE_BN_CASE(true, false, 14);                                                        \
      FLCE_BN_CASE(true, false, 15);                                                        \
      __VA_ARGS__;                                                                          \
    }                                                                                       \
  }                                                                                         \
  return cudaErrorInvalidValue

}  // namespace
}  // namespace flce
