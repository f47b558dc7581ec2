// flce_beam.cu -- a beam-search step (include/flce.h): selection over beams and vocabulary, and
// the reordering of the states that go with the beams.
//
// Selection: s[b, k, v] = score[b, k] + z[b, k, v] - lse_v z[b, k, :], the M best of K V, the
// lowest flat index first where they are equal. Bound by reading the logits once: a block takes a
// segment of a row into registers, from which it gets the segment's maximum and sum of
// exponentials and its M best logits (a row's order is its logits' order); a second kernel
// joins the segments and beams of a request. The order between beams depends on their lse, so
// segments are joined and scores compared in 64 bits.
//
// Reordering: out[.., b K + j, ..] = in[.., b K + parent[b, j], ..] for any number of tensors in
// one launch. A thread reads the same few bytes of all K beams before it writes any of them, so
// it works in place, without a second buffer; in place a beam that is its own parent costs nothing.
#include <cmath>

#include <math_constants.h>

#include "elem_io.cuh"
#include "flce_host.h"
#include "flce_internal.h"

namespace flce {
namespace {

constexpr int kBeamThreads = 256;
constexpr int kMaxBeams = 32, kMaxSelect = 64;
constexpr int kListCap = 512;  // candidates that are ranked against one another
constexpr float kLog2e = 1.4426950408889634f;

// Order-preserving bits of a float: larger value, larger bits.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t b) {
  return __uint_as_float(b & 0x80000000u ? b & 0x7fffffffu : ~b);
}
__device__ __forceinline__ uint64_t ordered64(double v) {
  const uint64_t b = uint64_t(__double_as_longlong(v == 0.0 ? 0.0 : v));  // -0 and 0 are equal
  return b >> 63 ? ~b : b | (uint64_t(1) << 63);
}
__device__ __forceinline__ double unordered64(uint64_t b) {
  return __longlong_as_double(int64_t(b >> 63 ? b & ~(uint64_t(1) << 63) : ~b));
}

// A candidate inside a row: the logit's ordered bits, then the complement of the token, so that
// of equal logits the lower token is the larger key. Zero is no candidate.
__device__ __forceinline__ uint64_t logit_key(float z, uint32_t token) {
  return (uint64_t(ordered(z == 0.f ? 0.f : z)) << 32) | uint32_t(~token);  // -0 and 0 are equal
}

struct SelectParams {
  const void* logits;
  int64_t ld_batch, ld_beam;
  const float* scores;
  const uint8_t* finished;
  int B, K, V, M;
  int segments, pad_token;
  float2* seg_stat;   // [B K][segments] maximum, sum of exp(z - maximum)
  uint64_t* seg_best; // [B K][segments][M] keys, descending, 0 past the segment's candidates
  float* out_scores;
  int32_t *out_parents, *out_tokens;
};

// The `need`-th largest of `n` values (n <= kBeamThreads, all distinct or zero) from the first n
// threads' values: each counts the larger ones.
template <typename KEY> __device__ __forceinline__ void rank_among(const KEY* keys, int n, int need, KEY* out) {
  const int i = int(threadIdx.x);
  if (i < n) {
    const KEY mine = keys[i];
    int above = 0;
    for (int j = 0; j < n; ++j) above += keys[j] > mine || (keys[j] == mine && j < i) ? 1 : 0;
    if (above == need - 1) *out = mine;
  }
}

// Groups of lanes whose maxima give the threshold: about twice as many as candidates wanted, so
// that about 1.4 M random values reach it.
__device__ __forceinline__ int group_lanes(int M) {
  int lanes = 32;  // 8 warps: 8 groups of 32 lanes ... 256 of one
  while (lanes > 1 && (kBeamThreads / lanes) < 2 * M) lanes >>= 1;
  return lanes;
}

template <typename T, int NV>
__global__ void __launch_bounds__(kBeamThreads) flce_beam_rows_kernel(const SelectParams p) {
  __shared__ float s_group[kBeamThreads];
  __shared__ float s_max[kBeamThreads / 32], s_sum[kBeamThreads / 32];
  __shared__ float s_least;
  __shared__ int s_count;
  __shared__ uint64_t s_list[kListCap];
  const int row = int(blockIdx.y), seg = int(blockIdx.x), tid = int(threadIdx.x);
  const int b = row / p.K, k = row - b * p.K;
  if (p.finished != nullptr && p.finished[row]) return;  // its only candidate needs no logits
  const T* z = static_cast<const T*>(p.logits) + int64_t(b) * p.ld_batch + int64_t(k) * p.ld_beam;
  const int mis = int((reinterpret_cast<uintptr_t>(z) & uintptr_t(8 * sizeof(T) - 1)) / sizeof(T));
  constexpr int kSeg = kBeamThreads * 8 * NV;
  const int e0 = seg * kSeg - mis + tid * 8;  // of this thread's first vector; the others follow kBeamThreads vectors apart
  Raw8<T> raw[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = e0 + j * kBeamThreads * 8;
    if (e >= 0 && e + 8 <= p.V) {
      raw[j] = raw_load(z + e);
    } else {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = e + i >= 0 && e + i < p.V ? to_f32(z[e + i]) : -CUDART_INF_F;
      raw[j] = pack8<T>(f);
    }
  }
  if (tid == 0) s_count = 0;
  float m = -CUDART_INF_F;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float f[8];
    unpack8(raw[j], f);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, f[i]);
  }
  float sum = 0.f;
  if (m != -CUDART_INF_F) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float f[8];
      unpack8(raw[j], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += exp2f((f[i] - m) * kLog2e);
    }
  } else {
    // fmaxf passes over NaN: a thread of NaN and -inf alone would miss it
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float f[8];
      unpack8(raw[j], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += f[i] != f[i] ? f[i] : 0.f;
    }
  }
  // maximum and sum of the warp, then of the block; group maxima on the way
  const int lanes = group_lanes(p.M);
  float wm = m;
  if (lanes == 1) s_group[tid] = wm;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, o));
    if (lanes == 2 * o && tid % lanes == 0) s_group[tid / lanes] = wm;
  }
  float ws = m == -CUDART_INF_F ? sum : sum * exp2f((m - wm) * kLog2e);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, o);
  if (tid % 32 == 0) {
    s_max[tid / 32] = wm;
    s_sum[tid / 32] = ws;
  }
  __syncthreads();
  rank_among(s_group, kBeamThreads / lanes, p.M, &s_least);
  const int64_t at = int64_t(row) * p.segments + seg;
  if (tid == kBeamThreads - 1) {
    float bm = s_max[0], bs = 0.f;
    for (int w = 1; w < kBeamThreads / 32; ++w) bm = fmaxf(bm, s_max[w]);
    for (int w = 0; w < kBeamThreads / 32; ++w) bs += s_max[w] == -CUDART_INF_F ? s_sum[w] : s_sum[w] * exp2f((s_max[w] - bm) * kLog2e);
    p.seg_stat[at] = make_float2(bm, bs);
  }
  __syncthreads();
  const float least = s_least;
  if (!(m < least)) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float f[8];
      unpack8(raw[j], f);
      const int e = e0 + j * kBeamThreads * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (!(f[i] < least) && e + i >= 0 && e + i < p.V) {
          const int n = atomicAdd(&s_count, 1);  // the order of the list does not matter: it is ranked
          if (n < kListCap) s_list[n] = logit_key(f[i], uint32_t(e + i));
        }
    }
  }
  __syncthreads();
  const int count = s_count;
  uint64_t* best = p.seg_best + at * p.M;
  if (count <= kListCap) {
    for (int i = tid; i < count; i += kBeamThreads) {
      const uint64_t mine = s_list[i];
      int above = 0;
      for (int j = 0; j < count; ++j) above += s_list[j] > mine ? 1 : 0;
      if (above < p.M) best[above] = mine;
    }
    for (int i = count + tid; i < p.M; i += kBeamThreads) best[i] = 0;
    return;
  }
  // many equal or sorted values: the M best one after the other
  uint64_t below = ~uint64_t(0);
  for (int n = 0; n < p.M; ++n) {
    uint64_t mine = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float f[8];
      unpack8(raw[j], f);
      const int e = e0 + j * kBeamThreads * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e + i >= 0 && e + i < p.V) {
          const uint64_t key = logit_key(f[i], uint32_t(e + i));
          mine = key < below && key > mine ? key : mine;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const uint64_t other = __shfl_xor_sync(0xffffffffu, mine, o);
      mine = other > mine ? other : mine;
    }
    __syncthreads();
    if (tid % 32 == 0) s_list[tid / 32] = mine;
    __syncthreads();
    for (int w = 0; w < kBeamThreads / 32; ++w) mine = s_list[w] > mine ? s_list[w] : mine;
    if (tid == 0) best[n] = mine;
    below = mine;
  }
}

// A candidate of a request: ordered bits of its score, then the lower flat index.
struct Candidate {
  uint64_t score;
  uint32_t row, token;
};
__device__ __forceinline__ bool better(const Candidate& a, const Candidate& b) {
  return a.score != b.score ? a.score > b.score : a.row != b.row ? a.row < b.row : a.token < b.token;
}
__device__ __forceinline__ Candidate no_candidate() { return Candidate{0, ~0u, ~0u}; }
__device__ __forceinline__ Candidate shuffle_best(Candidate c, int o) {
  Candidate d;
  d.score = __shfl_xor_sync(0xffffffffu, c.score, o);
  d.row = __shfl_xor_sync(0xffffffffu, c.row, o);
  d.token = __shfl_xor_sync(0xffffffffu, c.token, o);
  return better(d, c) ? d : c;
}

constexpr uint64_t kMinusInf = 0x000fffffffffffffull;  // ordered64(-inf)

// One block a request: lse of its beams, then the M best of their segments' best.
__global__ void __launch_bounds__(kBeamThreads) flce_beam_join_kernel(const SelectParams p) {
  __shared__ double s_base[kMaxBeams];  // score - lse; NaN: the beam has no candidate
  __shared__ int s_dead[kMaxBeams];     // 0 live, 1 no candidate, 2 finished
  __shared__ Candidate s_group[kBeamThreads], s_list[kListCap];
  __shared__ Candidate s_least;
  __shared__ int s_count;
  const int b = int(blockIdx.x), tid = int(threadIdx.x), warp = tid / 32, lane = tid % 32;
  for (int k = warp; k < p.K; k += kBeamThreads / 32) {
    const int64_t row = int64_t(b) * p.K + k;
    const float score = p.scores[row];
    if (p.finished != nullptr && p.finished[row]) {
      if (lane == 0) {
        s_base[k] = double(score);
        s_dead[k] = isfinite(score) ? 2 : 1;
      }
      continue;
    }
    const float2* st = p.seg_stat + row * p.segments;
    float m = -CUDART_INF_F;
    for (int s = lane; s < p.segments; s += 32) m = fmaxf(m, st[s].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    double sum = 0.0;
    for (int s = lane; s < p.segments; s += 32) {
      const float2 v = st[s];
      sum += double(v.x == -CUDART_INF_F ? v.y : v.y * expf(v.x - m));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) {
      const double lse = double(m) + log(sum);
      s_base[k] = double(score) - lse;
      s_dead[k] = isfinite(score) && isfinite(lse) ? 0 : 1;
    }
  }
  if (tid == 0) s_count = 0;
  __syncthreads();
  // candidate j of list l: a live beam's segments have their M best, a beam that is finished
  // or has none a list of its own (its padding token, then the lowest tokens at -inf)
  const int lists = p.K * p.segments;
  auto candidate = [&](int l, int j) {
    const int k = l / p.segments, s = l - k * p.segments;
    if (s_dead[k] == 0) {
      const uint64_t key = p.seg_best[((int64_t(b) * p.K + k) * p.segments + s) * p.M + j];
      if (key == 0) return no_candidate();
      const float z = unordered(uint32_t(key >> 32));
      const double v = z == -CUDART_INF_F ? -CUDART_INF : s_base[k] + double(z);
      return Candidate{ordered64(v), uint32_t(k), ~uint32_t(key)};
    }
    if (s > 0 || j >= p.V) return no_candidate();
    if (s_dead[k] == 1) return Candidate{kMinusInf, uint32_t(k), uint32_t(j)};
    if (j == 0) return Candidate{ordered64(s_base[k]), uint32_t(k), uint32_t(p.pad_token)};
    return Candidate{kMinusInf, uint32_t(k), uint32_t(j - 1 < p.pad_token ? j - 1 : j)};
  };
  Candidate mine = no_candidate();
  for (int l = tid; l < lists; l += kBeamThreads) {
    const Candidate c = candidate(l, 0);
    if (better(c, mine)) mine = c;
  }
  Candidate g = mine;
  const int lanes = group_lanes(p.M), groups = kBeamThreads / lanes;
  if (lanes == 1) s_group[tid] = g;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    g = shuffle_best(g, o);
    if (lanes == 2 * o && tid % lanes == 0) s_group[tid / lanes] = g;
  }
  __syncthreads();
  if (tid < groups) {
    const Candidate c = s_group[tid];
    int above = 0;
    for (int j = 0; j < groups; ++j) above += better(s_group[j], c) || (j < tid && !better(c, s_group[j])) ? 1 : 0;
    if (above == p.M - 1) s_least = c;
  }
  __syncthreads();
  const Candidate least = s_least;
  for (int l = tid; l < lists; l += kBeamThreads)
    for (int j = 0; j < p.M; ++j) {
      const Candidate c = candidate(l, j);
      if (c.score == 0 || better(least, c)) break;  // lists descend
      const int n = atomicAdd(&s_count, 1);
      if (n < kListCap) s_list[n] = c;
    }
  __syncthreads();
  const int count = s_count;
  auto put = [&](int n, const Candidate& c) {
    const int64_t o = int64_t(b) * p.M + n;
    p.out_scores[o] = float(unordered64(c.score));
    p.out_parents[o] = int32_t(c.row);
    p.out_tokens[o] = int32_t(c.token);
  };
  if (count <= kListCap) {
    for (int i = tid; i < count; i += kBeamThreads) {
      const Candidate c = s_list[i];
      int above = 0;
      for (int j = 0; j < count; ++j) above += better(s_list[j], c) ? 1 : 0;
      if (above < p.M) put(above, c);
    }
    return;
  }
  Candidate last{~uint64_t(0), 0, 0};
  for (int n = 0; n < p.M; ++n) {
    mine = no_candidate();
    for (int l = tid; l < lists; l += kBeamThreads)
      for (int j = 0; j < p.M; ++j) {
        const Candidate c = candidate(l, j);
        if (c.score == 0) break;
        if (!better(last, c)) continue;
        if (better(c, mine)) mine = c;
        break;
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine = shuffle_best(mine, o);
    __syncthreads();
    if (lane == 0) s_group[warp] = mine;
    __syncthreads();
    for (int w = 0; w < kBeamThreads / 32; ++w)
      if (better(s_group[w], mine)) mine = s_group[w];
    if (tid == 0) put(n, mine);
    last = mine;
  }
}

// Vectors of eight logits a thread: the more, the fewer segments to join, as long as there are
// blocks enough for the device.
int pick_vectors(int64_t rows, int64_t V) {
  for (int nv = 4; nv > 1; nv /= 2)
    if (rows * ((V + kBeamThreads * 8 * nv - 1) / (kBeamThreads * 8 * nv)) >= 152 * 4) return nv;
  return 1;
}

int64_t select_segments(int64_t rows, int64_t V) {
  const int64_t seg = int64_t(kBeamThreads) * 8 * pick_vectors(rows, V);
  return (V + 7 + seg - 1) / seg;  // a misaligned row starts up to seven elements into its first vector
}

template <typename T> cudaError_t launch_rows(const SelectParams& p, int nv, cudaStream_t stream) {
  const dim3 grid(unsigned(p.segments), unsigned(p.B * p.K));
  if (nv == 4)
    flce_beam_rows_kernel<T, 4><<<grid, kBeamThreads, 0, stream>>>(p);
  else if (nv == 2)
    flce_beam_rows_kernel<T, 2><<<grid, kBeamThreads, 0, stream>>>(p);
  else
    flce_beam_rows_kernel<T, 1><<<grid, kBeamThreads, 0, stream>>>(p);
  count_launch();
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------------
// Reordering
// ---------------------------------------------------------------------------------
// Tensors of one launch. Their descriptors are kernel parameters, which are copied with the
// launch: most calls have few.
constexpr int kFewStates = 6, kManyStates = 64;
constexpr int kOuter = 4;

struct StateDesc {
  const char* src;
  char* dst;
  int64_t beam_src, beam_dst;
  int64_t size[kOuter], stride_src[kOuter], stride_dst[kOuter];
  int64_t cols;     // inner columns of `width` bytes
  int64_t tiles;    // tiles of a request
  int64_t first;    // first tile of the launch
  int width;        // 16, 4 or 1
  int in_place;
};

template <int CAP> struct ReorderParams {
  StateDesc s[CAP];
  int count, B, K;
  const int32_t* parents;
  int64_t ld_parents;
};

template <typename W, int KMAX>
__device__ __forceinline__ void reorder_column(const StateDesc& s, int K, int b, int64_t c, const int* parent) {
  int64_t outer = c / s.cols, off_src = 0, off_dst = 0;
  const int64_t inner = (c - outer * s.cols) * int64_t(sizeof(W));
#pragma unroll
  for (int d = kOuter - 1; d >= 0; --d) {
    if (s.size[d] == 1) continue;
    const int64_t q = outer / s.size[d], i = outer - q * s.size[d];
    off_src += i * s.stride_src[d];
    off_dst += i * s.stride_dst[d];
    outer = q;
  }
  const char* src = s.src + off_src + int64_t(b) * K * s.beam_src + inner;
  char* dst = s.dst + off_dst + int64_t(b) * K * s.beam_dst + inner;
  W v[KMAX];
#pragma unroll
  for (int j = 0; j < KMAX; ++j)
    if (j < K && !(s.in_place && parent[j] == j)) v[j] = *reinterpret_cast<const W*>(src + parent[j] * s.beam_src);
#pragma unroll
  for (int j = 0; j < KMAX; ++j)
    if (j < K && !(s.in_place && parent[j] == j)) *reinterpret_cast<W*>(dst + j * s.beam_dst) = v[j];
}

template <int KMAX, int CAP>
__global__ void __launch_bounds__(kBeamThreads) flce_beam_reorder_kernel(const __grid_constant__ ReorderParams<CAP> p) {
  __shared__ int parent[kMaxBeams];
  int lo = 0, hi = p.count - 1;
  const int64_t tile = blockIdx.x;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.s[mid].first <= tile) lo = mid; else hi = mid - 1;
  }
  const StateDesc& s = p.s[lo];
  const int64_t t = tile - s.first;
  const int b = int(t / s.tiles);
  if (int(threadIdx.x) < p.K) {
    const int j = int(threadIdx.x), k = p.parents[b * p.ld_parents + j];
    parent[j] = k >= 0 && k < p.K ? k : j;  // no beam of this request: the state stays where it is
  }
  __syncthreads();
  int64_t total = s.cols;
#pragma unroll
  for (int d = 0; d < kOuter; ++d) total *= s.size[d];
  const int64_t c = (t - int64_t(b) * s.tiles) * kBeamThreads + threadIdx.x;
  if (c >= total) return;
  if (s.width == 16)
    reorder_column<uint4, KMAX>(s, p.K, b, c, parent);
  else if (s.width == 4)
    reorder_column<uint32_t, KMAX>(s, p.K, b, c, parent);
  else
    reorder_column<uint8_t, KMAX>(s, p.K, b, c, parent);
}

flce_status bad(const char* what, const char* why) {
  api_note_error(what, why);
  return FLCE_ERR_INVALID_ARG;
}

template <int CAP>
flce_status reorder_states(const flce_beam_state* states, int64_t count, const int32_t* parents, int64_t ld_parents,
                           int64_t B, int64_t K, cudaStream_t stream) {
  for (int64_t i = 0; i < count;) {
    ReorderParams<CAP> p;
    p.count = 0;
    p.B = int(B);
    p.K = int(K);
    p.parents = parents;
    p.ld_parents = ld_parents;
    int64_t tiles = 0;
    for (; i < count && p.count < CAP; ++i) {
      const flce_beam_state& s = states[i];
      StateDesc d{};
      d.src = static_cast<const char*>(s.src);
      d.dst = static_cast<char*>(s.dst);
      d.beam_src = s.beam_stride_src;
      d.beam_dst = s.beam_stride_dst;
      d.in_place = s.src == s.dst;
      uint64_t bits = uint64_t(reinterpret_cast<uintptr_t>(s.src) | reinterpret_cast<uintptr_t>(s.dst)) |
                      uint64_t(s.beam_stride_src) | uint64_t(s.beam_stride_dst) | uint64_t(s.inner_bytes);
      int64_t outer = 1;
      for (int k = 0; k < kOuter; ++k) {
        d.size[k] = s.outer_size[k];
        d.stride_src[k] = s.outer_stride_src[k];
        d.stride_dst[k] = s.outer_stride_dst[k];
        if (s.outer_size[k] > 1) bits |= uint64_t(s.outer_stride_src[k]) | uint64_t(s.outer_stride_dst[k]);
        outer *= s.outer_size[k];
      }
      d.width = bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 1;
      d.cols = s.inner_bytes / d.width;
      if (outer == 0 || d.cols == 0) continue;
      d.tiles = (outer * d.cols + kBeamThreads - 1) / kBeamThreads;
      if (tiles + B * d.tiles > 0x7fffffff) {
        if (p.count == 0) return FLCE_ERR_TOO_LARGE;
        break;
      }
      d.first = tiles;
      tiles += B * d.tiles;
      p.s[p.count++] = d;
    }
    if (p.count == 0) continue;
    const unsigned grid = unsigned(tiles);
    if (K <= 4)
      flce_beam_reorder_kernel<4, CAP><<<grid, kBeamThreads, 0, stream>>>(p);
    else if (K <= 8)
      flce_beam_reorder_kernel<8, CAP><<<grid, kBeamThreads, 0, stream>>>(p);
    else if (K <= 16)
      flce_beam_reorder_kernel<16, CAP><<<grid, kBeamThreads, 0, stream>>>(p);
    else
      flce_beam_reorder_kernel<32, CAP><<<grid, kBeamThreads, 0, stream>>>(p);
    count_launch();
    const flce_status st = api_cuda("beam reorder", cudaGetLastError());
    if (st != FLCE_OK) return st;
  }
  return FLCE_OK;
}

struct SelectLayout {
  size_t best, total;
};
SelectLayout select_layout(int64_t rows, int64_t V, int64_t M) {
  SelectLayout l{};
  const size_t n = size_t(rows) * size_t(select_segments(rows, V));
  l.best = api_align256(n * sizeof(float2));
  l.total = l.best + api_align256(n * size_t(M) * sizeof(uint64_t));
  return l;
}

bool select_sizes_ok(int64_t B, int64_t K, int64_t V, int64_t M) {
  return B >= 1 && K >= 1 && V >= 1 && M >= 1 && B <= 65535 && K <= kMaxBeams && B * K <= 65535 &&
         V < (int64_t(1) << 30) && M <= kMaxSelect;
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" {

size_t flce_beam_select_workspace_size(int64_t B, int64_t K, int64_t V, int64_t M) {
  if (!select_sizes_ok(B, K, V, M)) return 0;
  return select_layout(B * K, V, M).total;
}

flce_status flce_beam_select(const void* logits, int32_t dtype, int64_t B, int64_t K, int64_t V, int64_t ld_batch,
                             int64_t ld_beam, const float* scores, const uint8_t* finished, int32_t pad_token,
                             int64_t M, float* out_scores, int32_t* out_parents, int32_t* out_tokens, void* workspace,
                             size_t ws_bytes, struct CUstream_st* stream_) {
  if (!logits || !scores || !out_scores || !out_parents || !out_tokens || !workspace) return bad("buffer", "is null");
  if (B < 1 || K < 1 || V < 1 || M < 1) return bad("size", "B, K, V and M must be at least 1");
  if (!select_sizes_ok(B, K, V, M)) return FLCE_ERR_TOO_LARGE;
  if (M > K * V) return bad("M", "there are only K V candidates");
  if (dtype < 0 || dtype > 2) return bad("dtype", "unknown dtype");
  if (ld_beam < V && K > 1) return bad("ld_beam", "must be at least V");
  if (ld_batch < 0 || (B > 1 && ld_batch < V)) return bad("ld_batch", "must be at least V");
  if (finished && (pad_token < 0 || pad_token >= V)) return bad("pad_token", "must be a token of the vocabulary");
  if (!api_aligned(logits, uintptr_t(elem_bytes(dtype))) || !api_aligned(scores, 4) || !api_aligned(out_scores, 4) ||
      !api_aligned(out_parents, 4) || !api_aligned(out_tokens, 4) || !api_aligned(workspace, 256))
    return FLCE_ERR_ALIGNMENT;
  const SelectLayout l = select_layout(B * K, V, M);
  if (ws_bytes < l.total) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  int sms = 0, dev = -1;
  flce_status st = api_device(&sms, &dev);
  if (st != FLCE_OK) return st;
  const struct { const char* name; const void* p; } ptrs[] = {
      {"logits", logits}, {"scores", scores}, {"finished", finished}, {"out_scores", out_scores},
      {"out_parents", out_parents}, {"out_tokens", out_tokens}, {"workspace", workspace}};
  for (const auto& q : ptrs)
    if ((st = api_check_memory(dev, q.name, q.p)) != FLCE_OK) return st;
  SelectParams p{};
  p.logits = logits;
  p.ld_batch = ld_batch;
  p.ld_beam = ld_beam;
  p.scores = scores;
  p.finished = finished;
  p.B = int(B);
  p.K = int(K);
  p.V = int(V);
  p.M = int(M);
  p.segments = int(select_segments(B * K, V));
  p.pad_token = pad_token;
  p.seg_stat = reinterpret_cast<float2*>(workspace);
  p.seg_best = reinterpret_cast<uint64_t*>(static_cast<char*>(workspace) + l.best);
  p.out_scores = out_scores;
  p.out_parents = out_parents;
  p.out_tokens = out_tokens;
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  const int nv = pick_vectors(B * K, V);
  const cudaError_t e = dtype == FLCE_DTYPE_F32    ? launch_rows<float>(p, nv, stream)
                        : dtype == FLCE_DTYPE_BF16 ? launch_rows<__nv_bfloat16>(p, nv, stream)
                                                   : launch_rows<__half>(p, nv, stream);
  if ((st = api_cuda("beam rows", e)) != FLCE_OK) return st;
  flce_beam_join_kernel<<<unsigned(B), kBeamThreads, 0, stream>>>(p);
  count_launch();
  return api_cuda("beam join", cudaGetLastError());
}

flce_status flce_beam_reorder(const flce_beam_state* states, int64_t count, const int32_t* parents, int64_t ld_parents,
                              int64_t B, int64_t K, struct CUstream_st* stream_) {
  if (count < 0 || (count > 0 && !states)) return bad("states", "is null or has a negative count");
  if (!parents) return bad("parents", "is null");
  if (B < 1 || K < 1) return bad("size", "B and K must be at least 1");
  if (B > (int64_t(1) << 20) || K > kMaxBeams || count > (int64_t(1) << 20)) return FLCE_ERR_TOO_LARGE;
  if (ld_parents < K && B > 1) return bad("ld_parents", "must be at least K");
  if (!api_aligned(parents, 4)) return FLCE_ERR_ALIGNMENT;
  for (int64_t i = 0; i < count; ++i) {
    const flce_beam_state& s = states[i];
    if (s.inner_bytes < 0) return bad("states", "a negative size");
    for (int d = 0; d < kOuter; ++d)
      if (s.outer_size[d] < 0) return bad("states", "a negative size");
    if (!s.src || !s.dst) return bad("states", "a state is null");
    if (s.src == s.dst) {
      bool same = s.beam_stride_src == s.beam_stride_dst;
      for (int d = 0; d < kOuter; ++d)
        same = same && (s.outer_size[d] <= 1 || s.outer_stride_src[d] == s.outer_stride_dst[d]);
      if (!same) return bad("states", "in place, the strides must be equal");
    }
  }
  int sms = 0, dev = -1;
  flce_status st = api_device(&sms, &dev);
  if (st != FLCE_OK) return st;
  if ((st = api_check_memory(dev, "parents", parents)) != FLCE_OK) return st;
  for (int64_t i = 0; i < count; ++i) {
    if ((st = api_check_memory(dev, "state", states[i].src)) != FLCE_OK) return st;
    if (states[i].dst != states[i].src && (st = api_check_memory(dev, "reordered state", states[i].dst)) != FLCE_OK) return st;
  }
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  return count <= kFewStates ? reorder_states<kFewStates>(states, count, parents, ld_parents, B, K, stream)
                             : reorder_states<kManyStates>(states, count, parents, ld_parents, B, K, stream);
}

}  // extern "C"
