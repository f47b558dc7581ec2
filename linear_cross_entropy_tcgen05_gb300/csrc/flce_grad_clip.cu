// flce_grad_clip.cu -- global gradient norm over many tensors, and clipping (include/flce.h):
//
//   total = |s| (sum g^2)^(1/2), or |s| max |g|        out = g s min(1, max_norm / (total + eps))
//
// Bound by memory: one read for the norm, then a read and a write for the scaling (measured on
// 525 M fp32 values: 302 us and 650 us, 6.9 and 6.5 TB/s). Two
// kernels over the same list of chunks, whatever the number of tensors: their addresses go to
// the device as kernel parameters (no copy, no table kept between calls). The first writes one
// partial sum a block; every block of the second adds all partial sums in the same fixed order
// (a few hundred numbers from L2) and so knows the factor without a third launch or an atomic.
#include <cfloat>
#include <cmath>

#include "elem_io.cuh"
#include "flce_host.h"
#include "flce_internal.h"

namespace flce {
namespace {

constexpr int kClipThreads = 256;
// Persistent blocks of one launch, at most: those that stay on the device together. (Eight an SM
// do not: the last of them begin when the others end, 525 M fp32 values 1065 us against 945.)
constexpr int kClipPerSm = 4, kClipBlocks = 152 * kClipPerSm;
constexpr int kFewTensors = 60, kManyTensors = 900;
// Gradients that the scaling finds in L2 (129 MB) after the norm's pass: it takes the chunks in
// the opposite order, and what went before them, like what it writes, leaves L2 first (218 M bf16
// values into fp32: 290 us with none kept, 280 us with 60 MB, the same with 100).
constexpr int64_t kClipKeepBytes = int64_t(60) << 20;

struct ClipTensor {
  const void* grad;
  void* out;
  int64_t n;
  int first;  // its first chunk
  int16_t dt, out_dt;
};

// Tables of two sizes: the parameters of a launch are copied with it, and most calls are small.
template <int CAP> struct ClipTable {
  ClipTensor t[CAP];
  int count, chunks;
  int chunk_elems;  // a multiple of 8 * kClipThreads
  int keep;         // last chunks of the norm's pass that stay in L2 for the scaling's
  int inf_norm;
  float max_norm, eps, scale;
  double* part;        // this launch's partial sums
  const double* parts; // the call's partial sums, n_parts of them
  int n_parts;
  float* total;
};

template <typename TB> __device__ __forceinline__ int find_tensor(const TB& tb, int chunk) {
  int lo = 0, hi = tb.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tb.t[mid].first <= chunk) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Elements of the vector before the tensor's first: chunks start at vector boundaries of memory.
__device__ __forceinline__ int misalign(const void* p, int bytes) {
  return int((reinterpret_cast<uintptr_t>(p) & uintptr_t(8 * bytes - 1)) / bytes);
}

template <typename T> __device__ __forceinline__ Raw8<T> clip_load(const T* g, int64_t e, int64_t n) {
  if (e >= 0 && e + 8 <= n) return raw_load(g + e);
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = e + i >= 0 && e + i < n ? to_f32(g[e + i]) : 0.f;
  return pack8<T>(f);
}

// A thread's vectors of a chunk, a batch of them (128 bytes) in flight at a time. Those of a chunk
// that lies within its tensor need no checks. STREAM: they leave L2 first.
template <typename T, bool STREAM, typename F>
__device__ __forceinline__ void each_vector(const T* g, int64_t n, int64_t e0, int elems, F&& f) {
  constexpr int kClipBatch = 16 / sizeof(T);
  const bool inner = e0 >= 0 && e0 + elems <= n && elems % (8 * kClipThreads * kClipBatch) == 0;
  if (inner) {
    const T* at = g + e0 + threadIdx.x * 8;
    for (int v = 0; v < elems; v += 8 * kClipThreads * kClipBatch) {
      Raw8<T> r[kClipBatch];
#pragma unroll
      for (int k = 0; k < kClipBatch; ++k) {
        const T* p = at + v + k * 8 * kClipThreads;
        r[k] = STREAM ? raw_load_stream(p) : raw_load(p);
      }
#pragma unroll
      for (int k = 0; k < kClipBatch; ++k) f(r[k], e0 + v + k * 8 * kClipThreads + int(threadIdx.x) * 8);
    }
    return;
  }
  for (int v = int(threadIdx.x) * 8; v < elems; v += kClipThreads * 8) f(clip_load(g, e0 + v, n), e0 + v);
}

// Squares of a chunk in 32 bits (at most 64 of a thread, in four sums of 16), chunks in 64 bits. Where a thread's
// 32-bit sum may have lost something (overflow, or squares below the normal range) it takes
// its values once more in 64 bits.
template <typename T, bool STREAM>
__device__ __forceinline__ double chunk_squares(const T* g, int64_t n, int64_t e0, int elems) {
  float2 s[2] = {both(0.f), both(0.f)};
  uint32_t any = 0;
  constexpr uint32_t kMagnitude = sizeof(T) == 2 ? 0x7fff7fffu : 0x7fffffffu;
  each_vector<T, STREAM>(g, n, e0, elems, [&](const Raw8<T>& r, int64_t) {
    float2 f[4];
    unpack8(r, f);
#pragma unroll
    for (const uint4& q : r.v) any |= q.x | q.y | q.z | q.w;
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i & 1] = fma2(f[i], f[i], s[i & 1]);
  });
  const float sum = (s[0].x + s[0].y) + (s[1].x + s[1].y);
  if (sum > 1e-20f && sum < 1e30f) return double(sum);
  if ((any & kMagnitude) == 0) return 0.0;
  double d = 0.0;
  for (int v = int(threadIdx.x) * 8; v < elems; v += kClipThreads * 8) {
    float f[8];
    unpack8(clip_load(g, e0 + v, n), f);
    for (int i = 0; i < 8; ++i) d += double(f[i]) * double(f[i]);
  }
  return d;
}

// Largest magnitude as the bits of a float: NaN is above infinity, so it stays visible.
template <typename T, bool STREAM>
__device__ __forceinline__ uint32_t chunk_largest(const T* g, int64_t n, int64_t e0, int elems) {
  uint32_t m = 0;
  each_vector<T, STREAM>(g, n, e0, elems, [&](const Raw8<T>& r, int64_t) {
    float f[8];
    unpack8(r, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
  });
  return m;
}

template <typename T>
__device__ __forceinline__ void chunk_norm(const T* g, int64_t n, int64_t e0, int elems, bool inf_norm, bool stream,
                                           double& sum, uint32_t& largest) {
  if (inf_norm)
    largest = max(largest, stream ? chunk_largest<T, true>(g, n, e0, elems) : chunk_largest<T, false>(g, n, e0, elems));
  else
    sum += stream ? chunk_squares<T, true>(g, n, e0, elems) : chunk_squares<T, false>(g, n, e0, elems);
}

// Fixed-order sum (or largest, NaN above all) over the block; every thread gets it.
__device__ __forceinline__ double block_combine(double v, bool largest) {
  __shared__ double sh[kClipThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double w = __shfl_xor_sync(0xffffffffu, v, o);
    v = largest ? (w > v || w != w ? w : v) : v + w;
  }
  if (threadIdx.x % 32 == 0) sh[threadIdx.x / 32] = v;
  __syncthreads();
  v = sh[0];
  for (int i = 1; i < kClipThreads / 32; ++i) v = largest ? (sh[i] > v || sh[i] != sh[i] ? sh[i] : v) : v + sh[i];
  __syncthreads();
  return v;
}

template <int CAP>
__global__ void __launch_bounds__(kClipThreads, kClipPerSm) flce_grad_norm_kernel(const __grid_constant__ ClipTable<CAP> tb) {
  double sum = 0.0;
  uint32_t largest = 0;
  for (int c = int(blockIdx.x); c < tb.chunks; c += int(gridDim.x)) {
    const ClipTensor& t = tb.t[find_tensor(tb, c)];
    const int64_t e0 = int64_t(c - t.first) * tb.chunk_elems - misalign(t.grad, elem_bytes(t.dt));
    const int64_t left = t.n - e0;
    const int elems = int(left < tb.chunk_elems ? left : tb.chunk_elems);
    const bool stream = c < tb.chunks - tb.keep;
    if (t.dt == ELEM_F32)
      chunk_norm(static_cast<const float*>(t.grad), t.n, e0, elems, tb.inf_norm, stream, sum, largest);
    else if (t.dt == ELEM_BF16)
      chunk_norm(static_cast<const __nv_bfloat16*>(t.grad), t.n, e0, elems, tb.inf_norm, stream, sum, largest);
    else
      chunk_norm(static_cast<const __half*>(t.grad), t.n, e0, elems, tb.inf_norm, stream, sum, largest);
  }
  const double v = block_combine(tb.inf_norm ? double(__uint_as_float(largest)) : sum, tb.inf_norm);
  if (threadIdx.x == 0) tb.part[blockIdx.x] = v;
}

// What the gradients are multiplied with: f, and then tail. A factor below fp32's normal range (gradients
// near the end of that range, clipped to a small norm) keeps its bits as f 2^-100; else tail is 1.
struct ClipFactor {
  float f, tail;
};

// The total norm and the factor of the gradients, the same in every block.
template <typename TB> __device__ __forceinline__ ClipFactor clip_factor(const TB& tb, float* total) {
  double v = 0.0;
  for (int i = int(threadIdx.x); i < tb.n_parts; i += kClipThreads) {
    const double w = tb.parts[i];
    v = tb.inf_norm ? (w > v || w != w ? w : v) : v + w;
  }
  v = block_combine(v, tb.inf_norm);
  const double norm = (tb.inf_norm ? v : sqrt(v)) * fabs(double(tb.scale));
  *total = float(norm);
  double c = double(tb.max_norm) / (norm + double(tb.eps));
  if (!(c <= 1.0)) c = norm != norm ? norm : 1.0;  // 0 / 0 and inf / inf leave the gradients alone
  c *= double(tb.scale);
  const bool small = fabs(c) < double(FLT_MIN) && c != 0.0;
  return small ? ClipFactor{float(c * 0x1p100), 0x1p-100f} : ClipFactor{float(c), 1.f};
}

template <typename T, typename TO>
__device__ __forceinline__ void chunk_scale(const T* g, TO* out, int64_t n, int64_t e0, int elems, ClipFactor f) {
  const bool same = misalign(out, sizeof(TO)) == misalign(g, sizeof(T));
  each_vector<T, false>(g, n, e0, elems, [&](const Raw8<T>& r, int64_t e) {
    float2 x[4];
    unpack8(r, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = mul2(x[i], both(f.f));
    if (f.tail != 1.f) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = mul2(x[i], both(f.tail));
    }
    if (same && e >= 0 && e + 8 <= n) {
      raw_store_stream(out + e, pack8<TO>(x));
    } else {
      const float y[8] = {x[0].x, x[0].y, x[1].x, x[1].y, x[2].x, x[2].y, x[3].x, x[3].y};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e + i >= 0 && e + i < n) out[e + i] = from_f32<TO>(y[i]);
    }
  });
}

template <typename T>
__device__ __forceinline__ void chunk_scale_to(const ClipTensor& t, int64_t e0, int elems, ClipFactor f) {
  const T* g = static_cast<const T*>(t.grad);
  if (t.out_dt == ELEM_F32)
    chunk_scale(g, static_cast<float*>(t.out), t.n, e0, elems, f);
  else if (t.out_dt == ELEM_BF16)
    chunk_scale(g, static_cast<__nv_bfloat16*>(t.out), t.n, e0, elems, f);
  else
    chunk_scale(g, static_cast<__half*>(t.out), t.n, e0, elems, f);
}

template <int CAP>
__global__ void __launch_bounds__(kClipThreads, kClipPerSm) flce_grad_scale_kernel(const __grid_constant__ ClipTable<CAP> tb) {
  float total;
  const ClipFactor f = clip_factor(tb, &total);
  if (blockIdx.x == 0 && threadIdx.x == 0 && tb.total != nullptr) *tb.total = total;
  // a block's chunks of the norm's pass in the opposite order: the last are still in L2, on the
  // side of the device that it is on
  const int grid = int(gridDim.x), b = int(blockIdx.x);
  for (int c = b + (tb.chunks - 1 - b) / grid * grid; b < tb.chunks && c >= 0; c -= grid) {
    const ClipTensor& t = tb.t[find_tensor(tb, c)];
    if (t.out == nullptr || (f.f == 1.f && f.tail == 1.f && t.out == t.grad)) continue;  // nothing to change
    const int64_t e0 = int64_t(c - t.first) * tb.chunk_elems - misalign(t.grad, elem_bytes(t.dt));
    const int64_t left = t.n - e0;
    const int elems = int(left < tb.chunk_elems ? left : tb.chunk_elems);
    if (t.dt == ELEM_F32)
      chunk_scale_to<float>(t, e0, elems, f);
    else if (t.dt == ELEM_BF16)
      chunk_scale_to<__nv_bfloat16>(t, e0, elems, f);
    else
      chunk_scale_to<__half>(t, e0, elems, f);
  }
}

struct ClipCall {
  const flce_grad_tensor* tensors;
  int64_t count;
  int inf_norm;
  float max_norm, eps, scale;
  float* total;
  double* parts;
  bool scaling;
  int bytes;  // of the largest element
  cudaStream_t stream;
};

// Elements of a chunk: small enough that every SM gets some, at most 64 a thread.
int pick_chunk(int64_t total) {
  int elems = 8 * kClipThreads;
  while (elems < 64 * kClipThreads && total > int64_t(elems) * 2 * kClipBlocks) elems *= 2;
  return elems;
}

int64_t clip_chunks(const flce_grad_tensor& t, int elems) {
  const int b = elem_bytes(t.dtype);
  const int mis = int((reinterpret_cast<uintptr_t>(t.grad) & uintptr_t(8 * b - 1)) / b);
  return t.n == 0 ? 0 : (t.n + mis + elems - 1) / elems;
}

// Runs the norm kernel (pass 0) or the scaling kernel (pass 1) over the tensors, CAP at a time.
template <int CAP> flce_status clip_pass(const ClipCall& c, int elems, int pass, int* n_parts) {
  int parts = 0;
  int64_t i = 0;
  do {
    ClipTable<CAP> tb;
    tb.count = 0;
    int64_t chunks = 0;
    for (; i < c.count && tb.count < CAP; ++i) {
      const flce_grad_tensor& t = c.tensors[i];
      const int64_t k = clip_chunks(t, elems);
      if (k == 0) continue;
      if (chunks + k > (int64_t(1) << 30)) break;
      tb.t[tb.count++] = ClipTensor{t.grad, t.out, t.n, int(chunks), int16_t(t.dtype), int16_t(t.out_dtype)};
      chunks += k;
    }
    tb.chunks = int(chunks);
    tb.chunk_elems = elems;
    tb.inf_norm = c.inf_norm;
    tb.keep = c.scaling ? int(kClipKeepBytes / (int64_t(elems) * c.bytes)) : 0;
    tb.max_norm = c.max_norm;
    tb.eps = c.eps;
    tb.scale = c.scale;
    tb.parts = c.parts;
    tb.part = c.parts + parts;
    tb.n_parts = *n_parts;
    tb.total = pass == 1 && (i >= c.count) ? c.total : nullptr;
    const int64_t want = pass == 1 && !c.scaling ? 1 : chunks;
    const unsigned blocks = unsigned(want < 1 ? 1 : want < kClipBlocks ? want : kClipBlocks);
    if (pass == 1 && !c.scaling) tb.chunks = 0;
    if (pass == 0)
      flce_grad_norm_kernel<CAP><<<blocks, kClipThreads, 0, c.stream>>>(tb);
    else if (c.scaling || tb.total != nullptr)
      flce_grad_scale_kernel<CAP><<<blocks, kClipThreads, 0, c.stream>>>(tb);
    if (pass == 0 || c.scaling || tb.total != nullptr) count_launch();
    const flce_status st = api_cuda("gradient norm", cudaGetLastError());
    if (st != FLCE_OK) return st;
    parts += int(blocks);
  } while (i < c.count);
  if (pass == 0) *n_parts = parts;
  return FLCE_OK;
}

flce_status bad(const char* what, const char* why) {
  api_note_error(what, why);
  return FLCE_ERR_INVALID_ARG;
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" {

size_t flce_clip_grad_norm_workspace_size(int64_t count) {
  if (count < 0 || count > (int64_t(1) << 24)) return 0;
  // a launch takes at least kFewTensors tensors (or 2^30 chunks, more than a device holds)
  return api_align256(size_t(count / kFewTensors + 2) * kClipBlocks * sizeof(double));
}

flce_status flce_clip_grad_norm(const flce_grad_tensor* tensors, int64_t count, float max_norm, float norm_type,
                                float eps, float grad_scale, float* total_norm, void* workspace, size_t ws_bytes,
                                struct CUstream_st* stream) {
  if (count < 0 || (count > 0 && !tensors)) return bad("tensors", "is null or has a negative count");
  if (count > (int64_t(1) << 24)) return FLCE_ERR_TOO_LARGE;
  if (!(norm_type == 2.f) && !(std::isinf(norm_type) && norm_type > 0.f)) return bad("norm_type", "must be 2 or infinity");
  if (!(max_norm >= 0.f)) return bad("max_norm", "must not be negative");
  if (!(eps >= 0.f) || std::isinf(eps)) return bad("eps", "must be finite and not negative");
  if (!std::isfinite(grad_scale)) return bad("grad_scale", "must be finite");
  if (!total_norm || !workspace) return bad("total_norm", "total_norm and the workspace are needed");
  if (!api_aligned(total_norm, 4) || !api_aligned(workspace, 256)) return FLCE_ERR_ALIGNMENT;
  int64_t total = 0;
  bool scaling = false;
  int bytes = 2;
  for (int64_t i = 0; i < count; ++i) {
    const flce_grad_tensor& t = tensors[i];
    if (t.n < 0) return bad("tensors", "a negative number of elements");
    if (t.n >= (int64_t(1) << 40)) return FLCE_ERR_TOO_LARGE;
    if (t.dtype < 0 || t.dtype > 2 || t.out_dtype < 0 || t.out_dtype > 2) return bad("tensors", "unknown dtype");
    if (t.n == 0) continue;
    if (!t.grad) return bad("tensors", "a gradient is null");
    if (t.out == t.grad && t.dtype != t.out_dtype) return bad("tensors", "in place, the types must be equal");
    if (!api_aligned(t.grad, uintptr_t(elem_bytes(t.dtype))) || !api_aligned(t.out, uintptr_t(elem_bytes(t.out_dtype))))
      return FLCE_ERR_ALIGNMENT;
    total += t.n;
    scaling |= t.out != nullptr;
    if (t.dtype == FLCE_DTYPE_F32) bytes = 4;
  }
  if (ws_bytes < flce_clip_grad_norm_workspace_size(count)) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  int sms = 0, dev = -1;
  flce_status st = api_device(&sms, &dev);
  if (st != FLCE_OK) return st;
  if ((st = api_check_memory(dev, "total_norm", total_norm)) != FLCE_OK ||
      (st = api_check_memory(dev, "workspace", workspace)) != FLCE_OK)
    return st;
  for (int64_t i = 0; i < count; ++i) {
    if (tensors[i].n == 0) continue;
    if ((st = api_check_memory(dev, "gradient", tensors[i].grad)) != FLCE_OK) return st;
    if (tensors[i].out != tensors[i].grad && (st = api_check_memory(dev, "clipped gradient", tensors[i].out)) != FLCE_OK)
      return st;
  }
  const ClipCall c{tensors, count, std::isinf(norm_type), max_norm, eps, grad_scale, total_norm,
                   static_cast<double*>(workspace), scaling, bytes, reinterpret_cast<cudaStream_t>(stream)};
  const int elems = pick_chunk(total);
  int n_parts = 0;
  for (int pass = 0; pass < 2; ++pass) {
    st = count <= kFewTensors ? clip_pass<kFewTensors>(c, elems, pass, &n_parts)
                              : clip_pass<kManyTensors>(c, elems, pass, &n_parts);
    if (st != FLCE_OK) return st;
  }
  return FLCE_OK;
}

}  // extern "C"
