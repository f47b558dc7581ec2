// flce_block_norm.cu -- entry points of the block norm (include/flce.h): argument checks, how
// rows are shared out, the launch sequence, and the kernel that adds the parameter gradients'
// partial sums.
#include <cmath>
#include <cstdio>

#include "block_norm.h"
#include "elem_io.cuh"
#include "flce_host.h"
#include "flce_internal.h"

namespace flce {
namespace {

// Rows are shared out for 152 SMs (GB300) whatever the device says, so that the workspace
// size is a function of the sizes alone.
constexpr int kSms = 152;

constexpr int kBnFewThreads = 256;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

BlockNormShape bn_shape(int64_t D, int max_threads) {
  BlockNormShape s{};
  const int64_t threads = cdiv(D, 8);
  s.cluster = 1;
  while (threads > int64_t(max_threads) * s.cluster) s.cluster *= 2;
  s.threads_per_row = int(cdiv(cdiv(threads, s.cluster), 32) * 32);
  s.rows_per_block = s.cluster > 1 ? 1 : max_threads / s.threads_per_row;
  return s;
}

// Blocks (or clusters) that stay on the device together, one block an SM: the rows on their way
// in fill its shared memory. Clusters lie within a group of SMs, so not every SM is in one
// (cudaOccupancyMaxActiveClusters gives 76, 36 and 15 on GB300).
int64_t bn_resident(const BlockNormShape& s) {
  return s.cluster == 1 ? kSms : s.cluster == 2 ? kSms / 2 : s.cluster == 4 ? 36 : 15;
}

// How a call's rows are shared out, and the features of its kernel. Wide blocks are taken by rows
// that 512 threads would share in clusters, and by FULL kernels where they have room for more
// rows, if there are rows for more (N = 32768, D = 5120 bf16: 204 us against 297 in clusters; N =
// 16384, D = 2304, layer norms: 106 us against 122; but N = 48, D = 5120: 12.5 us against 11.3; and
// RMS norms at N = 32768, D = 2560: 126 us against 117). Blocks have half as many threads where
// rows of 512 would leave no room for two batches of them (fp32 rows of 4096 columns with a
// gate for each), so that clusters share them.
struct BnKernel {
  BlockNormShape shape;
  int max_threads, feat;
};
BnKernel bn_pick(const flce_block_norm_desc* d, bool vec, int feat, bool backward) {
  const int planes = bn_planes(elem_bytes(d->x_dtype), elem_bytes(d->residual_dtype), d->gate && d->gate_rows == d->N, backward);
  auto fits = [&](const BlockNormShape& s, int f) { return bn_ring(s, planes, vec, f, backward).batches >= 2; };
  const BlockNormShape s = bn_shape(d->D, kBnThreads);
  if (!backward && vec) {
    const BlockNormShape w = bn_shape(d->D, kBnMaxThreads);
    const int f = bn_kernel_features(feat, vec, 1, true);
    if (w.cluster == 1 && (s.cluster > 1 || ((feat & BN_FULL) && w.rows_per_block > s.rows_per_block)) &&
        d->N > bn_resident(s) * s.rows_per_block && fits(w, f))
      return BnKernel{w, kBnMaxThreads, f};
  }
  const int f = bn_kernel_features(feat, vec, s.cluster, false);
  if (fits(s, f)) return BnKernel{s, kBnThreads, f};
  const BlockNormShape few = bn_shape(d->D, kBnFewThreads);
  return BnKernel{few, kBnFewThreads, bn_kernel_features(feat, vec, few.cluster, false)};
}

struct BwdPlan {
  BlockNormShape shape;
  int64_t blocks, chunks, chunks_per_group, chunk_rows, group_rows;
  int64_t first_rows;  // partial sums of the first norm's parameters
  bool gate_parts;
  size_t part[4], part_gate, total;
};

// Rows of a gate group are split into chunks, chunks are dealt to the workers (row groups of
// blocks) in turn. Among splits that keep the partial sums of the gate's gradient small the
// one with the shortest longest worker is taken. A worker keeps its sums over at least four
// rows, so that the partial sums stay small beside the rows.
BwdPlan bwd_plan(int64_t N, int64_t D, int64_t gate_rows, int max_threads) {
  BwdPlan p{};
  p.shape = bn_shape(D, max_threads);
  const int64_t groups = gate_rows == 0 || gate_rows == N ? 1 : gate_rows;  // a full gate needs no sums
  p.group_rows = N / groups;
  int64_t blocks = bn_resident(p.shape);
  const int64_t need = cdiv(cdiv(N, 4), p.shape.rows_per_block);
  p.blocks = blocks < need ? blocks : need;
  const int64_t workers = p.blocks * p.shape.rows_per_block;
  // a worker takes one to four chunks: the split whose longest worker is shortest
  int64_t best = -1;
  for (int64_t rounds = 1; rounds <= 4; ++rounds) {
    int64_t k = rounds * workers / groups;
    k = k < 1 ? rounds : k < p.group_rows ? k : p.group_rows;
    const int64_t rows = cdiv(p.group_rows, k), per = cdiv(p.group_rows, rows);
    const int64_t cost = cdiv(groups * per, workers) * rows;
    if (best < 0 || cost < best) {
      best = cost;
      p.chunks_per_group = per;
      p.chunk_rows = rows;
    }
    if (groups == 1) break;  // one chunk a worker is even already
  }
  p.chunks = groups * p.chunks_per_group;
  p.gate_parts = gate_rows > 0 && gate_rows != N && p.chunks_per_group > 1;
  size_t o = 0;
  p.first_rows = gate_rows > 0 && gate_rows != N ? workers : p.blocks;
  for (int i = 0; i < 4; ++i) {
    p.part[i] = o;
    o += api_align256(size_t(i < 2 ? p.first_rows : p.blocks) * size_t(D) * sizeof(float));
  }
  p.part_gate = o;
  if (p.gate_parts) o += api_align256(size_t(p.chunks) * size_t(D) * sizeof(float));
  p.total = o;
  return p;
}

bool dtype_ok(int dt) { return dt >= 0 && dt <= 2; }

// The largest power of two that every row of a [.., D] buffer is aligned to is at least `a`.
bool rows_aligned(const void* p, int64_t ld, int dt, uintptr_t a) {
  return api_aligned(p, a) && (uint64_t(ld) * uint64_t(elem_bytes(dt))) % a == 0;
}
bool rows_vec(const void* p, int64_t ld, int dt) { return p == nullptr || rows_aligned(p, ld, dt, 8 * elem_bytes(dt)); }

flce_status bad(const char* what, const char* why) {
  api_note_error(what, why);
  return FLCE_ERR_INVALID_ARG;
}

flce_status check_desc(const flce_block_norm_desc* d) {
  if (!d) return bad("desc", "is null");
  if (d->N < 1 || d->D < 1) return bad("desc", "N and D must be at least 1");
  if (d->N >= (int64_t(1) << 30) || d->D > kBnMaxD) return FLCE_ERR_TOO_LARGE;
  if (!d->x) return bad("x", "is null");
  const int dts[] = {d->x_dtype, d->residual_dtype, d->gate_dtype, d->post_weight_dtype, d->post_bias_dtype,
                     d->weight_dtype, d->bias_dtype};
  for (int dt : dts)
    if (!dtype_ok(dt)) return bad("desc", "unknown dtype");
  if (d->residual_dtype != d->x_dtype && d->residual_dtype != FLCE_DTYPE_F32)
    return bad("residual_dtype", "must be x's type or fp32");
  if (d->norm != FLCE_NORM_RMS && d->norm != FLCE_NORM_LAYER) return bad("norm", "unknown norm");
  if (d->gate_activation < 0 || d->gate_activation > 2) return bad("gate_activation", "unknown activation");
  if (!(d->eps >= 0.f) || std::isinf(d->eps)) return bad("eps", "must be finite and not negative");
  if (!std::isfinite(d->scale) || !std::isfinite(d->weight_offset)) return bad("scale", "must be finite");
  if ((d->gate != nullptr) != (d->gate_rows > 0)) return bad("gate_rows", "is 0 without a gate, else its rows");
  if (d->gate_rows < 0 || d->gate_rows > d->N || (d->gate && d->N % d->gate_rows != 0))
    return bad("gate_rows", "must divide N");
  if (d->gate && d->gate_dtype != d->x_dtype && d->gate_dtype != d->residual_dtype)
    return bad("gate_dtype", "must be x's or the residual's type");
  if ((d->post_bias && !d->post_weight) || (d->bias && !d->weight)) return bad("bias", "needs its weight");
  if (d->ld_x < d->D || (d->residual && d->ld_residual < d->D) || (d->gate && d->ld_gate < d->D))
    return bad("ld", "row strides must be at least D");
  const struct { const void* p; int dt; } ptrs[] = {
      {d->x, d->x_dtype}, {d->residual, d->residual_dtype}, {d->gate, d->gate_dtype},
      {d->post_weight, d->post_weight_dtype}, {d->post_bias, d->post_bias_dtype}, {d->weight, d->weight_dtype},
      {d->bias, d->bias_dtype}};
  for (const auto& q : ptrs)
    if (!api_aligned(q.p, uintptr_t(elem_bytes(q.dt)))) return FLCE_ERR_ALIGNMENT;
  return FLCE_OK;
}

flce_status check_desc_memory(int dev, const flce_block_norm_desc* d) {
  const struct { const char* name; const void* p; } ptrs[] = {
      {"x", d->x}, {"residual", d->residual}, {"gate", d->gate}, {"post_weight", d->post_weight},
      {"post_bias", d->post_bias}, {"weight", d->weight}, {"bias", d->bias}};
  for (const auto& q : ptrs) {
    const flce_status st = api_check_memory(dev, q.name, q.p);
    if (st != FLCE_OK) return st;
  }
  return FLCE_OK;
}

BlockNormParams bn_params(const flce_block_norm_desc* d) {
  BlockNormParams p{};
  p.x = d->x;
  p.residual = d->residual;
  p.gate = d->gate;
  p.w1 = d->post_weight;
  p.b1 = d->post_bias;
  p.w2 = d->weight;
  p.b2 = d->bias;
  p.ld_x = d->ld_x;
  p.ld_residual = d->ld_residual;
  p.ld_gate = d->ld_gate;
  p.N = d->N;
  p.D = int(d->D);
  p.gate_group = d->gate ? d->N / d->gate_rows : d->N;
  p.w1_dt = d->post_weight_dtype;
  p.b1_dt = d->post_bias_dtype;
  p.w2_dt = d->weight_dtype;
  p.b2_dt = d->bias_dtype;
  p.gate_res_type = d->gate_dtype == d->residual_dtype;
  p.gate_full = d->gate != nullptr && d->gate_rows == d->N;
  p.act = d->gate_activation;
  p.layer = d->norm == FLCE_NORM_LAYER;
  p.eps = d->eps;
  p.scale = d->scale;
  p.w_off = d->weight_offset;
  return p;
}

int bn_features(const flce_block_norm_desc* d) {
  return (d->post_weight ? BN_POST : 0) | (d->gate ? BN_GATE : 0) | (d->gate && d->gate_rows == d->N ? BN_GATE_ROWS : 0) |
         (d->norm == FLCE_NORM_LAYER || d->post_bias || d->bias ? BN_FULL : 0);
}

bool desc_vec(const flce_block_norm_desc* d) {
  return d->D % 8 == 0 && rows_vec(d->x, d->ld_x, d->x_dtype) && rows_vec(d->residual, d->ld_residual, d->residual_dtype) &&
         rows_vec(d->gate, d->ld_gate, d->gate_dtype) && rows_vec(d->post_weight, 8, d->post_weight_dtype) &&
         rows_vec(d->post_bias, 8, d->post_bias_dtype) && rows_vec(d->weight, 8, d->weight_dtype) &&
         rows_vec(d->bias, 8, d->bias_dtype);
}

// Column sums of the partial sums: 32 columns a block, 32 threads down the rows of each, then
// one adds the 32. It reads what the backward kernel wrote a moment ago (from L2) and is bound by
// the latency of a column's loads: 7 us for 152 partial sums of two parameters, D = 4096, 11 us
// with biases and gates, of a backward pass of 130 and 180 us.
constexpr int kSumRows = 32;

__global__ void __launch_bounds__(32 * kSumRows) flce_block_norm_sums_kernel(const BnSums s) {
  __shared__ float part[kSumRows][33];
  const BnSum a = s.a[blockIdx.z];
  const int lane = int(threadIdx.x) % 32, ty = int(threadIdx.x) / 32;
  const int col = int(blockIdx.x) * 32 + lane;
  for (int64_t seg = blockIdx.y; seg < a.segments; seg += gridDim.y) {
    float v = 0.f;
    if (col < s.D) {
      const float* at = a.part + seg * a.rows * s.D + col;
#pragma unroll 5
      for (int64_t r = ty; r < a.rows; r += kSumRows) v += at[r * s.D];
    }
    part[ty][lane] = v;
    __syncthreads();
    if (ty == 0 && col < s.D) {
      float t = 0.f;
#pragma unroll
      for (int i = 0; i < kSumRows; ++i) t += part[i][lane];
      store_any(a.out, a.dt, seg * s.D + col, t);
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t bn_column_sums(const BnSums& s, cudaStream_t stream) {
  if (s.n == 0) return cudaSuccess;
  int64_t segments = 1;
  for (int i = 0; i < s.n; ++i) segments = s.a[i].segments > segments ? s.a[i].segments : segments;
  const dim3 grid(unsigned((s.D + 31) / 32), unsigned(segments < 1024 ? segments : 1024), unsigned(s.n));
  flce_block_norm_sums_kernel<<<grid, 32 * kSumRows, 0, stream>>>(s);
  count_launch();
  return cudaGetLastError();
}

}  // namespace flce

using namespace flce;

extern "C" {

size_t flce_block_norm_workspace_size(int64_t N, int64_t D, int64_t gate_rows) {
  if (N < 1 || D < 1 || N >= (int64_t(1) << 30) || D > kBnMaxD || gate_rows < 0 || gate_rows > N) return 0;
  if (gate_rows > 0 && N % gate_rows != 0) return 0;
  const size_t a = bwd_plan(N, D, gate_rows, kBnThreads).total;
  const size_t b = bwd_plan(N, D, gate_rows, kBnFewThreads).total;
  return a > b ? a : b;
}

flce_status flce_block_norm_forward(const flce_block_norm_desc* d, void* h, void* y, float* stats,
                                    struct CUstream_st* stream) {
  flce_status st = check_desc(d);
  if (st != FLCE_OK) return st;
  if (!h) return bad("h", "is null");
  if ((y != nullptr) != (d->weight != nullptr)) return bad("y", "is given exactly when weight is");
  if (h == d->residual && d->ld_residual != d->D && d->N > 1)  // its rows would be written over ones still to be read
    return bad("h", "in the residual's buffer, the residual's row stride must be D");
  if (!api_aligned(h, uintptr_t(elem_bytes(d->residual_dtype))) || !api_aligned(y, uintptr_t(elem_bytes(d->x_dtype))) ||
      !api_aligned(stats, 16))
    return FLCE_ERR_ALIGNMENT;
  int sms = 0, dev = -1;
  if ((st = api_device(&sms, &dev)) != FLCE_OK || (st = check_desc_memory(dev, d)) != FLCE_OK ||
      (st = api_check_memory(dev, "h", h)) != FLCE_OK || (st = api_check_memory(dev, "y", y)) != FLCE_OK ||
      (st = api_check_memory(dev, "stats", stats)) != FLCE_OK)
    return st;
  BlockNormParams p = bn_params(d);
  p.h = h;
  p.y = y;
  p.stats = stats;
  const bool vec = desc_vec(d) && rows_vec(h, d->D, d->residual_dtype) && rows_vec(y, d->D, d->x_dtype);
  const BnKernel k = bn_pick(d, vec, bn_features(d), false);
  const BlockNormShape& s = k.shape;
  const int64_t need = cdiv(d->N, s.rows_per_block), resident = bn_resident(s);
  int64_t blocks = need < resident ? need : resident;
  p.chunk_rows = cdiv(d->N, blocks * s.rows_per_block);
  blocks = cdiv(cdiv(d->N, p.chunk_rows), s.rows_per_block);
  const bool f32 = d->residual_dtype == FLCE_DTYPE_F32;
  const auto fn = d->x_dtype == FLCE_DTYPE_BF16  ? (f32 ? bn_forward_bf16_f32 : bn_forward_bf16_bf16)
                  : d->x_dtype == FLCE_DTYPE_F16 ? (f32 ? bn_forward_f16_f32 : bn_forward_f16_f16)
                                                 : bn_forward_f32_f32;
  return api_cuda("block norm forward", fn(p, s, vec, k.feat, unsigned(blocks), reinterpret_cast<cudaStream_t>(stream)));
}

flce_status flce_block_norm_backward(const flce_block_norm_desc* d, const void* h, const float* stats, const void* dh,
                                     int64_t ld_dh, const void* dy, int64_t ld_dy, const flce_block_norm_grads* g,
                                     void* workspace, size_t ws_bytes, struct CUstream_st* stream_) {
  flce_status st = check_desc(d);
  if (st != FLCE_OK) return st;
  if (!g) return bad("grads", "is null");
  if (!h || !stats) return bad("h", "the forward's h and stats are needed");
  if (!dh && !dy) return bad("dh", "dh or dy is needed");
  if (dy && !d->weight) return bad("dy", "without a weight there is no y");
  if ((dh && ld_dh < d->D) || (dy && ld_dy < d->D)) return bad("ld", "row strides must be at least D");
  if ((g->dgate && !d->gate) || (g->dpost_weight && !d->post_weight) || (g->dpost_bias && !d->post_bias) ||
      (g->dweight && !d->weight) || (g->dbias && !d->bias))
    return bad("grads", "a gradient of an input that is not there");
  const int er = elem_bytes(d->residual_dtype), ex = elem_bytes(d->x_dtype);
  if (!api_aligned(h, er) || !api_aligned(dh, er) || !api_aligned(g->dresidual, er) || !api_aligned(dy, ex) ||
      !api_aligned(g->dx, ex) || !api_aligned(stats, 16) || !api_aligned(g->dgate, elem_bytes(d->gate_dtype)) ||
      !api_aligned(g->dpost_weight, elem_bytes(d->post_weight_dtype)) ||
      !api_aligned(g->dpost_bias, elem_bytes(d->post_bias_dtype)) ||
      !api_aligned(g->dweight, elem_bytes(d->weight_dtype)) || !api_aligned(g->dbias, elem_bytes(d->bias_dtype)) ||
      !api_aligned(workspace, 256))
    return FLCE_ERR_ALIGNMENT;
  if (!workspace) return bad("workspace", "is null");
  if (ws_bytes < flce_block_norm_workspace_size(d->N, d->D, d->gate_rows)) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  int sms = 0, dev = -1;
  if ((st = api_device(&sms, &dev)) != FLCE_OK || (st = check_desc_memory(dev, d)) != FLCE_OK) return st;
  const struct { const char* name; const void* p; } ptrs[] = {
      {"h", h}, {"stats", stats}, {"dh", dh}, {"dy", dy}, {"dx", g->dx}, {"dresidual", g->dresidual},
      {"dgate", g->dgate}, {"dpost_weight", g->dpost_weight}, {"dpost_bias", g->dpost_bias}, {"dweight", g->dweight},
      {"dbias", g->dbias}, {"workspace", workspace}};
  for (const auto& q : ptrs)
    if ((st = api_check_memory(dev, q.name, q.p)) != FLCE_OK) return st;
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  const bool vec = desc_vec(d) && rows_vec(h, d->D, d->residual_dtype) && rows_vec(dh, ld_dh, d->residual_dtype) &&
                   rows_vec(dy, ld_dy, d->x_dtype) && rows_vec(g->dx, d->D, d->x_dtype) &&
                   rows_vec(g->dresidual, d->D, d->residual_dtype) && rows_vec(g->dgate, d->D, d->gate_dtype);
  const BnKernel k = bn_pick(d, vec, bn_features(d), true);
  const BwdPlan plan = bwd_plan(d->N, d->D, d->gate_rows, k.max_threads);
  char* ws = static_cast<char*>(workspace);
  BlockNormParams p = bn_params(d);
  p.stats = const_cast<float*>(stats);
  p.h_in = h;
  p.dh = dh;
  p.dy = dy;
  p.ld_dh = ld_dh;
  p.ld_dy = ld_dy;
  p.dx = g->dx;
  p.dres = g->dresidual;
  p.dgate = g->dgate;
  p.chunks = plan.chunks;
  p.chunks_per_group = plan.chunks_per_group;
  p.chunk_rows = plan.chunk_rows;
  p.group_rows = plan.group_rows;
  p.part_gate = g->dgate && plan.gate_parts ? reinterpret_cast<float*>(ws + plan.part_gate) : nullptr;
  BnSums sums{};
  sums.D = int(d->D);
  const struct { void* out; int dt; } params[4] = {{g->dpost_weight, d->post_weight_dtype}, {g->dpost_bias, d->post_bias_dtype},
                                                   {g->dweight, d->weight_dtype}, {g->dbias, d->bias_dtype}};
  for (int i = 0; i < 4; ++i) {
    if (!params[i].out) continue;
    p.part[i] = reinterpret_cast<float*>(ws + plan.part[i]);
    sums.a[sums.n++] = BnSum{p.part[i], params[i].out, 1, i < 2 ? plan.first_rows : plan.blocks, params[i].dt};
  }
  if (p.part_gate) sums.a[sums.n++] = BnSum{p.part_gate, g->dgate, d->gate_rows, plan.chunks_per_group, d->gate_dtype};
  const bool f32 = d->residual_dtype == FLCE_DTYPE_F32;
  const auto fn = d->x_dtype == FLCE_DTYPE_BF16  ? (f32 ? bn_backward_bf16_f32 : bn_backward_bf16_bf16)
                  : d->x_dtype == FLCE_DTYPE_F16 ? (f32 ? bn_backward_f16_f32 : bn_backward_f16_f16)
                                                 : bn_backward_f32_f32;
  st = api_cuda("block norm backward", fn(p, plan.shape, vec, k.feat, unsigned(plan.blocks), stream));
  if (st != FLCE_OK) return st;
  return api_cuda("block norm sums", bn_column_sums(sums, stream));
}

}  // extern "C"
