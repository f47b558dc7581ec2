// flce_beam.cu -- a beam-search step (include/flce.h): selection over beams and vocabulary, and
// the reordering of the states that go with the beams.
//
// Selection: s[b, k, v] = score[b, k] + z[b, k, v] - lse_v z[b, k, :], the M best of K V, the
// lowest flat index first where they are equal. With m the row's maximum and S = sum exp(z - m) it is
// formed as (z - m) + (score - log S): m + log S would lose log S, and the score with it, in a row whose
// logits are all masked with the type's lowest value (or near any other large one). Bound by reading the logits once, so that pass
// selects nothing: it leaves the maximum and the sum of exponentials of every piece of a row. One
// block a request then finds from the maxima a threshold that M candidates reach, and looks for
// them in the few pieces that can have any (from L2). The order between beams depends on their
// lse, so sums are joined and scores compared in 64 bits. (Selecting in every segment in the first
// pass took 101 us for 256 rows of 256000 bf16 logits, half of it waiting at barriers.)
//
// Reordering: out[.., b K + j, ..] = in[.., b K + parent[b, j], ..] for any number of tensors in
// one launch. A thread reads the same few bytes of all K beams before it writes any of them, so
// it works in place, without a second buffer; in place a beam that is its own parent costs nothing.
// Bound by memory: a cache of 128 beams and 1.07 GB in 191 us, 82% of the DRAM's time (parents that
// several beams share are read once).
#include <cfloat>
#include <cmath>

#include <math_constants.h>

#include "elem_io.cuh"
#include "flce_host.h"
#include "flce_internal.h"

namespace flce {
namespace {

constexpr int kBeamThreads = 256, kJoinThreads = 512;
constexpr int kMaxBeams = 32, kMaxSelect = 64;
constexpr int kListCap = 2048;   // candidates that are ranked against one another
constexpr int kBorderList = 512;  // of them, where there are more, those that a threshold is taken from
constexpr int kPiecesCap = 2048;  // pieces that may have some
constexpr float kLog2e = 1.4426950408889634f;

// 2^x; results below the normal range, beside a largest term of 1, are 0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Order-preserving bits of a score: larger value, larger bits. Zero is below every score.
__device__ __forceinline__ uint64_t ordered64(double v) {
  const uint64_t b = uint64_t(__double_as_longlong(v == 0.0 ? 0.0 : v));  // -0 and 0 are equal
  return b >> 63 ? ~b : b | (uint64_t(1) << 63);
}
__device__ __forceinline__ double unordered64(uint64_t b) {
  return __longlong_as_double(int64_t(b >> 63 ? b & ~(uint64_t(1) << 63) : ~b));
}

struct SelectParams {
  const void* logits;
  int64_t ld_batch, ld_beam;
  const float* scores;
  const uint8_t* finished;
  int B, K, V, M;
  int pieces;      // of a row
  int pad_token;
  float2* stat;    // [B K][pieces] maximum, sum of exp(z - maximum)
  float* out_scores;
  int32_t *out_parents, *out_tokens;
};

// A lane's vectors of a piece: NV of eight logits, 256 apart; -inf past the row. Pieces and vectors are
// counted from the row's first logit wherever it is in memory, so that equal rows have equal sums to
// the last bit, and equal beams exact ties.
template <typename T, int NV> struct Piece {
  static constexpr int kPer = 16 / sizeof(T), kParts = 8 / kPer;  // logits of 16 bytes, and those of a vector
  Raw8<T> raw[NV];
  int e0;  // the first logit of the lane's first vector
  // Whether 16-byte loads of the row are aligned from its first logit on.
  __device__ __forceinline__ static bool aligned(const T* z) {
    return (reinterpret_cast<uintptr_t>(z) & uintptr_t(8 * sizeof(T) - 1)) == 0;
  }
  __device__ __forceinline__ void load_aligned(const T* z, int V) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e = e0 + j * 256;
      if (e + 8 <= V)
        raw[j] = raw_load(z + e);
      else
        load_each(z, V, j);
    }
  }
  __device__ __forceinline__ void load_each(const T* z, int V, int j) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = e0 + j * 256 + i < V ? to_f32(z[e0 + j * 256 + i]) : -CUDART_INF_F;
    raw[j] = pack8<T>(f);
  }
  // For a few pieces.
  __device__ __forceinline__ void load(const T* z, int V, int piece, int lane) {
    e0 = piece * 256 * NV + lane * 8;
    if (aligned(z)) {
      load_aligned(z, V);
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) load_each(z, V, j);
    }
  }
  // For all pieces of a row, by whole warps. The vectors of an unaligned row are shifted out of the
  // aligned pieces of 16 bytes around them: a lane loads those that its first logits are in and has the
  // last from the next lane, the last lane from the first one's next vector. (512 x 4 rows of 50257 bf16
  // logits, with the join: 72 us; 62 with pieces that begin where memory's vectors do, whose sums
  // differed in their last bits between equal rows, and so put equal beams in any order; 109 with bounds
  // checked load by load.)
  __device__ __forceinline__ void load_all(const T* z, int V, int piece, int lane) {
    e0 = piece * 256 * NV + lane * 8;
    if (aligned(z)) return load_aligned(z, V);
    const int bytes = int(reinterpret_cast<uintptr_t>(z) & 15), ahead = bytes / int(sizeof(T));
    uint4 v[NV * kParts + 1];
    const T* at = z + e0 - ahead;
    if (piece > 0 && (piece + 1) * 256 * NV + kPer <= V) {
#pragma unroll
      for (int i = 0; i < NV * kParts; ++i) v[i] = *reinterpret_cast<const uint4*>(at + i / kParts * 256 + i % kParts * kPer);
      v[NV * kParts] = lane == 0 ? *reinterpret_cast<const uint4*>(at + NV * 256) : make_uint4(0u, 0u, 0u, 0u);
    } else {
#pragma unroll
      for (int i = 0; i <= NV * kParts; ++i) {
        const int e = e0 - ahead + i / kParts * 256 + i % kParts * kPer;
        float f[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = k < kPer && e + k >= 0 && e + k < V ? to_f32(z[e + k]) : -CUDART_INF_F;
        v[i] = pack8<T>(f).v[0];
      }
    }
    switch (bytes / 4) {
      case 0: shift<0>(v, lane, bytes & 2); break;
      case 1: shift<1>(v, lane, bytes & 2); break;
      case 2: shift<2>(v, lane, bytes & 2); break;
      default: shift<3>(v, lane, bytes & 2); break;
    }
  }
  template <int BY> __device__ __forceinline__ void shift(const uint4 (&v)[NV * kParts + 1], int lane, int half) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const uint4 &own = v[j * kParts], &next = v[(j + 1) * kParts];
      const uint32_t give[4] = {lane == 0 ? next.x : own.x, lane == 0 ? next.y : own.y, lane == 0 ? next.z : own.z,
                                lane == 0 ? next.w : own.w};
      uint32_t w[4 * kParts + 4], q[4 * kParts];
#pragma unroll
      for (int i = 0; i < kParts; ++i) {
        const uint4& p = v[j * kParts + i];
        w[4 * i] = p.x, w[4 * i + 1] = p.y, w[4 * i + 2] = p.z, w[4 * i + 3] = p.w;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) w[4 * kParts + i] = i <= BY ? __shfl_sync(0xffffffffu, give[i], (lane + 1) % 32) : 0u;
      words_from<BY, T>(w, half, q);
#pragma unroll
      for (int i = 0; i < kParts; ++i) raw[j].v[i] = make_uint4(q[4 * i], q[4 * i + 1], q[4 * i + 2], q[4 * i + 3]);
    }
  }
};

template <typename T> __device__ __forceinline__ const T* row_of(const SelectParams& p, int b, int k) {
  return static_cast<const T*>(p.logits) + int64_t(b) * p.ld_batch + int64_t(k) * p.ld_beam;
}

// The pass over the logits: a warp takes a piece of 256 NV of them into registers, and its maximum
// and sum of exponentials out. Nothing is selected here, so no warp waits for another: bound by
// memory and, for 16-bit logits, nearly as much by the exponentials (16 a clock and SM). 256 rows of
// 256000 bf16 logits: 24 us, 5.5 TB/s.
template <typename T, int NV>
__global__ void __launch_bounds__(kBeamThreads) flce_beam_rows_kernel(const SelectParams p) {
  const int row = int(blockIdx.y), piece = int(blockIdx.x) * (kBeamThreads / 32) + int(threadIdx.x) / 32;
  const int lane = int(threadIdx.x) % 32;
  if (piece >= p.pieces) return;
  if (p.finished != nullptr && p.finished[row]) return;  // its only candidate needs no logits
  const int b = row / p.K;
  Piece<T, NV> z;
  z.load_all(row_of<T>(p, b, row - b * p.K), p.V, piece, lane);
  float m = -CUDART_INF_F;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float2 f[4];
    unpack8(z.raw[j], f);
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(f[i].x, f[i].y));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  // (x - m) log2 e and not x log2 e - m log2 e: the largest term is 1 exactly. A piece of -inf alone
  // has the sum 0; a NaN or +inf makes it NaN (fmaxf passes over a NaN, the sum does not).
  const float base = m == -CUDART_INF_F ? 0.f : m;
  float2 s2 = both(0.f);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float2 f[4];
    unpack8(z.raw[j], f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 d = mul2(add2(f[i], both(-base)), both(kLog2e));
      s2 = add2(s2, make_float2(ex2(d.x), ex2(d.y)));
    }
  }
  float s = s2.x + s2.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) p.stat[int64_t(row) * p.pieces + piece] = make_float2(m, s);
}

enum BeamState : int { BEAM_LIVE = 0, BEAM_NONE = 1, BEAM_FINISHED = 2 };

// One block a request. lse of its beams; a threshold that at least M candidates reach, from the
// maxima of disjoint sets of them (the M-th largest of such maxima does); the candidates that reach
// it, from the few pieces whose maximum does; and their ranks among one another. The threshold
// and the test against it are in 32 bits with a margin, the scores and the order in 64. All of it
// is latency: 8 us for one request of four beams, 20 us for 16 beams of 256000 tokens and 32
// candidates (512 threads; 33 us with 256). More equal or sorted logits than the list holds take
// some passes more over the pieces that have them (4 requests of 8 beams of 128256 equal ones: 95 us
// with the pass over the logits).
template <typename T, int NV>
__global__ void __launch_bounds__(kJoinThreads) flce_beam_join_kernel(const SelectParams p) {
  constexpr int kWarps = kJoinThreads / 32;
  __shared__ float s_part_max[kMaxBeams];  // at least as many as warps
  __shared__ double s_part_sum[kMaxBeams];
  __shared__ double s_base[kMaxBeams];  // score - log S, or a finished beam's score
  __shared__ float s_base32[kMaxBeams], s_top[kMaxBeams];  // and the row's maximum
  __shared__ int s_state[kMaxBeams], s_beam[kMaxBeams], s_n_live, s_n_done;
  __shared__ __align__(16) float s_set[kJoinThreads];
  __shared__ float s_least;
  __shared__ double s_border;
  __shared__ int s_pieces[kPiecesCap];
  __shared__ int s_n_pieces, s_count;
  __shared__ __align__(16) uint64_t s_score[kListCap], s_place[kListCap];  // place: beam, then token
  const int b = int(blockIdx.x), tid = int(threadIdx.x), warp = tid / 32, lane = tid % 32;
  const float2* stat = p.stat + int64_t(b) * p.K * p.pieces;
  // a beam's pieces are shared by the warps that there are for it
  const int per_beam = kWarps > p.K ? kWarps / p.K : 1;
  for (int u = warp; u < p.K * per_beam; u += kWarps) {
    const int k = u / per_beam, first = (u - k * per_beam) * 32 + lane;
    if (p.finished != nullptr && p.finished[int64_t(b) * p.K + k]) continue;
    const float2* st = stat + k * p.pieces;
    float m = -CUDART_INF_F;
#pragma unroll 4
    for (int s = first; s < p.pieces; s += 32 * per_beam) m = fmaxf(m, st[s].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    double sum = 0.0;
#pragma unroll 4
    for (int s = first; s < p.pieces; s += 32 * per_beam) {
      const float2 v = st[s];
      sum += double(v.x == -CUDART_INF_F ? v.y : v.y * ex2((v.x - m) * kLog2e));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) {
      s_part_max[u] = m;
      s_part_sum[u] = sum;
    }
  }
  __syncthreads();
  if (warp == 0) {
    int state = BEAM_NONE;
    if (lane < p.K) {
      const int k = lane;
      const int64_t row = int64_t(b) * p.K + k;
      const float score = p.scores[row];
      double base = double(score);
      if (p.finished == nullptr || !p.finished[row]) {
        float m = -CUDART_INF_F;
        for (int w = 0; w < per_beam; ++w) m = fmaxf(m, s_part_max[k * per_beam + w]);
        double sum = 0.0;
        for (int w = 0; w < per_beam; ++w) {
          const float x = s_part_max[k * per_beam + w];
          sum += x == -CUDART_INF_F ? s_part_sum[k * per_beam + w] : s_part_sum[k * per_beam + w] * double(ex2((x - m) * kLog2e));
        }
        const double log_sum = log(sum);
        base -= log_sum;
        s_top[k] = m;
        if (isfinite(score) && isfinite(m) && isfinite(log_sum)) state = BEAM_LIVE;
      } else if (isfinite(score)) {
        state = BEAM_FINISHED;
      }
      s_base[k] = base;
      s_base32[k] = float(fmin(fmax(base, -double(FLT_MAX)), double(FLT_MAX)));
      s_state[k] = state;
    }
    // the live beams, then the finished ones
    const uint32_t live = __ballot_sync(0xffffffffu, state == BEAM_LIVE), done = __ballot_sync(0xffffffffu, state == BEAM_FINISHED);
    const uint32_t below = (1u << lane) - 1;
    if (state == BEAM_LIVE) s_beam[__popc(live & below)] = lane;
    if (state == BEAM_FINISHED) s_beam[__popc(live) + __popc(done & below)] = lane;
    if (lane == 0) {
      s_n_live = __popc(live);
      s_n_done = __popc(done);
    }
  }
  if (tid == 0) s_n_pieces = s_count = 0;
  __syncthreads();
  // a live beam's candidate of logit z
  auto value32 = [&](int k, float z) { return s_base32[k] + (z - s_top[k]); };
  auto value64 = [&](int k, float z) { return s_base[k] + (double(z) - double(s_top[k])); };
  // What the maxima are known of: the live beams' pieces, then the finished beams. (Beams without a
  // candidate are not among them: at a request's first step all but one are.)
  const int live_pieces = s_n_live * p.pieces, all = live_pieces + s_n_done;
  auto piece_best = [&](int i) {
    if (i >= live_pieces) return s_base32[s_beam[s_n_live + i - live_pieces]];
    const int l = i / p.pieces, k = s_beam[l];
    return value32(k, stat[k * p.pieces + (i - l * p.pieces)].x);
  };
  // Each thread's set: some of these, or where they are few, tokens. Sets of neighbouring lanes are
  // joined to about twice as many as candidates wanted: about 1.4 M random values reach the M-th
  // largest of 2 M maxima. Each has pieces of every beam: a beam that is far ahead of the others has
  // all the candidates, and with its pieces in a few sets the threshold would be another's
  // (16 requests of 8 beams, 128256 random logits, scores of deviation 1: 1.2 ms).
  float best = -CUDART_INF_F, size = 0.f;
  const bool by_piece = all >= 4 * p.M;
  const int values = by_piece ? all : p.V, active = values < kJoinThreads ? values : kJoinThreads;
  int lanes = 1;
  while (active / lanes >= 4 * p.M && lanes < 32) lanes *= 2;
  const int sets = kJoinThreads / lanes, first_piece = tid % lanes * sets + tid / lanes;
  if (by_piece) {
    for (int i = first_piece; i < all; i += kJoinThreads) best = fmaxf(best, piece_best(i));
  } else {
    if (tid < s_n_done) best = piece_best(live_pieces + tid);
    for (int l = 0; l < s_n_live; ++l) {
      const int k = s_beam[l];
      const T* z = row_of<T>(p, b, k);
      float m = -CUDART_INF_F;
      for (int v = tid; v < p.V; v += kJoinThreads) m = fmaxf(m, to_f32(z[v]));
      best = fmaxf(best, value32(k, m));
    }
  }
  for (int k = lane; k < p.K; k += 32)
    if (s_state[k] != BEAM_NONE) size = fmaxf(size, fabsf(s_base32[k]));
  if (lanes == 1) s_set[tid] = best;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
    size = fmaxf(size, __shfl_xor_sync(0xffffffffu, size, o));
    if (lanes == 2 * o && tid % lanes == 0) s_set[tid / lanes] = best;
  }
  __syncthreads();
  if (tid < sets) {
    const float mine = s_set[tid];
    int above = 0;
#pragma unroll 4
    for (int j = 0; j < sets; j += 4) {
      const float4 q = *reinterpret_cast<const float4*>(s_set + j);
      above += int(q.x > mine || (q.x == mine && j < tid)) + int(q.y > mine || (q.y == mine && j + 1 < tid)) +
               int(q.z > mine || (q.z == mine && j + 2 < tid)) + int(q.w > mine || (q.w == mine && j + 3 < tid));
    }
    if (above == p.M - 1) {
      // base, difference and their sum are rounded once each, and the difference is at most the sum
      // and the base: 16 steps of these are ample
      const float v = mine - 16.f * 0x1p-24f * (fabsf(mine) + 2.f * size);
      s_least = v == v ? v : -CUDART_INF_F;
    }
  }
  __syncthreads();
  const float least = s_least;
  auto wanted = [&](float v) { return v >= least && v > -CUDART_INF_F; };
  auto add = [&](double score, int k, int token) {
    const int n = atomicAdd(&s_count, 1);  // the order of the list does not matter: it is ranked
    if (n < kListCap) {
      s_score[n] = ordered64(score);
      s_place[n] = uint64_t(k) << 32 | uint32_t(token);
    }
  };
  if (tid < p.K && s_state[tid] == BEAM_FINISHED && wanted(s_base32[tid])) add(s_base[tid], tid, p.pad_token);
  for (int i = tid; i < live_pieces; i += kJoinThreads)
    if (wanted(piece_best(i))) {
      const int n = atomicAdd(&s_n_pieces, 1);
      if (n < kPiecesCap) s_pieces[n] = i;
    }
  __syncthreads();
  // every candidate of a piece that is wanted, to f(score, beam, token); by one warp
  auto scan = [&](int i, auto&& f) {
    const int l = i / p.pieces, k = s_beam[l];
    Piece<T, NV> z;
    z.load(row_of<T>(p, b, k), p.V, i - l * p.pieces, lane);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float v[8];
      unpack8(z.raw[j], v);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (wanted(value32(k, v[e]))) f(value64(k, v[e]), k, z.e0 + j * 256 + e);
    }
  };
  // more candidates than the list holds: which ones it has does not matter then
  auto full = [&]() { return *reinterpret_cast<volatile int*>(&s_count) > kListCap; };
  const int n_pieces = s_n_pieces;
  if (n_pieces <= kPiecesCap) {
    for (int i = warp; i < n_pieces && !full(); i += kWarps) scan(s_pieces[i], add);
  } else {
    for (int i = warp; i < live_pieces && !full(); i += kWarps)
      if (wanted(piece_best(i))) scan(i, add);
  }
  __syncthreads();
  int count = s_count;
  const int64_t out = int64_t(b) * p.M;
  auto put = [&](int n, uint64_t score, uint64_t place) {
    p.out_scores[out + n] = float(unordered64(score));
    p.out_parents[out + n] = int32_t(place >> 32);
    p.out_tokens[out + n] = int32_t(uint32_t(place));
  };
  // f(i, those above it) for each of the list's n candidates
  auto each_rank = [&](int n, auto&& f) {
    // four threads count those above a candidate, every fourth of the list each
    const int part = tid % 4;
    for (int i = tid / 4; i < (n + 7) / 8 * 8; i += kJoinThreads / 4) {  // whole warps: they shuffle
      const uint64_t score = i < n ? s_score[i] : ~uint64_t(0), place = i < n ? s_place[i] : 0;
      int above = 0;
#pragma unroll 4
      for (int j = part; j < n; j += 4)
        above += int(s_score[j] > score) + int(s_score[j] == score && s_place[j] < place);
      above += __shfl_xor_sync(0xffffffffu, above, 1);
      above += __shfl_xor_sync(0xffffffffu, above, 2);
      if (part == 0 && i < n) f(i, above);
    }
  };
  // Thousands reach the threshold (a mask of the type's lowest value that leaves few tokens, sorted or
  // equal logits, a beam of few pieces far ahead). The M-th best of some in the list, whichever these
  // are, is a threshold too; those above it are listed, until they fit. At least the others that
  // it was taken from are not above it, so this ends.
  bool border_set = false;
  double border = 0.0;
  while (count > kListCap) {
    each_rank(kBorderList, [&](int i, int above) {
      if (above == p.M - 1) s_border = unordered64(s_score[i]);
    });
    __syncthreads();
    border = s_border;
    border_set = true;
    if (tid == 0) s_count = 0;
    __syncthreads();
    if (tid < p.K && s_state[tid] == BEAM_FINISHED && s_base[tid] > border) add(s_base[tid], tid, p.pad_token);
    for (int i = warp; i < live_pieces && !full(); i += kWarps) {
      const int l = i / p.pieces, k = s_beam[l];
      if (value64(k, stat[k * p.pieces + (i - l * p.pieces)].x) <= border) continue;
      scan(i, [&](double score, int beam, int token) {
        if (score > border) add(score, beam, token);
      });
    }
    __syncthreads();
    count = s_count;
  }
  each_rank(count, [&](int i, int above) {
    if (above < p.M) put(above, s_score[i], s_place[i]);
  });
  if (warp != 0 || count >= p.M) return;
  int have = count;
  if (border_set) {
    // as many at the threshold as are wanted, lowest index first
    auto take = [&](uint32_t mine, int k, int token) {  // bits of a lane's eight tokens from `token` on
      int before = __popc(mine), total = before;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, total, o);
        if (lane >= o) total += v;
      }
      int n = have + total - before;
      for (int e = 0; e < 8; ++e)
        if (mine >> e & 1) {
          if (n < p.M) put(n, ordered64(border), uint64_t(k) << 32 | uint32_t(token + e));
          ++n;
        }
      have += __shfl_sync(0xffffffffu, total, 31);
    };
    for (int k = 0; k < p.K && have < p.M; ++k) {
      if (s_state[k] == BEAM_FINISHED) take(lane == 0 && s_base[k] == border ? 1u : 0u, k, p.pad_token);
      if (s_state[k] != BEAM_LIVE) continue;
      for (int p0 = 0; p0 < p.pieces && have < p.M; p0 += 32) {
        const int piece = p0 + lane;
        const bool has = piece < p.pieces && value64(k, stat[k * p.pieces + piece].x) >= border;
        for (uint32_t todo = __ballot_sync(0xffffffffu, has); todo != 0 && have < p.M; todo &= todo - 1) {
          Piece<T, NV> z;
          z.load(row_of<T>(p, b, k), p.V, p0 + __ffs(int(todo)) - 1, lane);
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            float v[8];
            unpack8(z.raw[j], v);
            uint32_t mine = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (v[e] > -CUDART_INF_F && value64(k, v[e]) == border) mine |= 1u << e;
            take(mine, k, z.e0 + j * 256);
          }
        }
      }
    }
    return;
  }
  // What is no candidate fills the rest, lowest index first: all tokens of a beam without any, all but
  // the padding of a finished one, the masked ones of a live one (with scores of -inf, or, under
  // two masks of the type's lowest value, of less than fp32 has).
  for (int k = 0; k < p.K && have < p.M; ++k) {
    const T* z = row_of<T>(p, b, k);
    for (int v0 = 0; v0 < p.V && have < p.M; v0 += 32) {
      const int v = v0 + lane;
      bool none = v < p.V;
      if (none && s_state[k] == BEAM_FINISHED) none = v != p.pad_token;
      if (none && s_state[k] == BEAM_LIVE) none = !(value32(k, to_f32(z[v])) > -CUDART_INF_F);
      const uint32_t who = __ballot_sync(0xffffffffu, none);
      const int n = have + __popc(who & ((1u << lane) - 1));
      if (none && n < p.M) put(n, ordered64(-CUDART_INF), uint64_t(k) << 32 | uint32_t(v));
      have += __popc(who);
    }
  }
}

// Vectors of eight logits a lane: the more, the fewer pieces, as long as there are warps enough for
// the device.
int pick_vectors(int64_t rows, int64_t V) {
  for (int nv = 4; nv > 1; nv /= 2)
    if (rows * ((V + 256 * nv - 1) / (256 * nv)) >= 152 * 32) return nv;
  return 1;
}

int64_t select_pieces(int64_t rows, int64_t V) {
  const int64_t piece = 256 * pick_vectors(rows, V);
  return (V + piece - 1) / piece;
}

template <typename T, int NV> cudaError_t launch_select(const SelectParams& p, cudaStream_t stream) {
  const dim3 grid(unsigned((p.pieces + kBeamThreads / 32 - 1) / (kBeamThreads / 32)), unsigned(p.B * p.K));
  flce_beam_rows_kernel<T, NV><<<grid, kBeamThreads, 0, stream>>>(p);
  count_launch();
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  flce_beam_join_kernel<T, NV><<<unsigned(p.B), kJoinThreads, 0, stream>>>(p);
  count_launch();
  return cudaGetLastError();
}

template <typename T> cudaError_t launch_select_typed(const SelectParams& p, int nv, cudaStream_t stream) {
  return nv == 4 ? launch_select<T, 4>(p, stream) : nv == 2 ? launch_select<T, 2>(p, stream) : launch_select<T, 1>(p, stream);
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
  return api_align256(size_t(B * K) * size_t(select_pieces(B * K, V)) * sizeof(float2));
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
  if (ws_bytes < flce_beam_select_workspace_size(B, K, V, M)) return FLCE_ERR_WORKSPACE_TOO_SMALL;
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
  p.pieces = int(select_pieces(B * K, V));
  p.pad_token = pad_token;
  p.stat = reinterpret_cast<float2*>(workspace);
  p.out_scores = out_scores;
  p.out_parents = out_parents;
  p.out_tokens = out_tokens;
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  const int nv = pick_vectors(B * K, V);
  const cudaError_t e = dtype == FLCE_DTYPE_F32    ? launch_select_typed<float>(p, nv, stream)
                        : dtype == FLCE_DTYPE_BF16 ? launch_select_typed<__nv_bfloat16>(p, nv, stream)
                                                   : launch_select_typed<__half>(p, nv, stream);
  return api_cuda("beam select", e);
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
