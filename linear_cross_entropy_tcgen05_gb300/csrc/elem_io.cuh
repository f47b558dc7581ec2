// elem_io.cuh -- loads, stores and conversions of runs of eight elements (bf16, f16 or
// fp32) shared by the kernels around the loss (block norm, gradient clipping, beam search).
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace flce {

// Element types, as flce_dtype in include/flce.h.
enum ElemType : int { ELEM_BF16 = 0, ELEM_F16 = 1, ELEM_F32 = 2 };

__host__ __device__ constexpr int elem_bytes(int dt) { return dt == ELEM_F32 ? 4 : 2; }

template <typename T> struct ElemOf;
template <> struct ElemOf<__nv_bfloat16> { static constexpr int code = ELEM_BF16; };
template <> struct ElemOf<__half> { static constexpr int code = ELEM_F16; };
template <> struct ElemOf<float> { static constexpr int code = ELEM_F32; };

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }

// Eight consecutive elements as they sit in memory.
template <typename T> struct Raw8 { uint4 v[sizeof(T) / 2]; };

template <typename T> __device__ __forceinline__ Raw8<T> raw_zero() {
  Raw8<T> r;
#pragma unroll
  for (auto& q : r.v) q = make_uint4(0u, 0u, 0u, 0u);
  return r;
}

// One 16-byte load (16-bit types) or one 32-byte load (fp32): p is aligned to eight elements.
template <typename T> __device__ __forceinline__ Raw8<T> raw_load(const T* p) {
  Raw8<T> r;
  if constexpr (sizeof(T) == 2) {
    r.v[0] = *reinterpret_cast<const uint4*>(p);
  } else {
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r.v[0].x), "=r"(r.v[0].y), "=r"(r.v[0].z), "=r"(r.v[0].w), "=r"(r.v[1].x), "=r"(r.v[1].y),
                   "=r"(r.v[1].z), "=r"(r.v[1].w)
                 : "l"(p));
  }
  return r;
}

template <typename T> __device__ __forceinline__ void raw_store(T* p, const Raw8<T>& r) {
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(p) = r.v[0];
  } else {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r.v[0].x), "r"(r.v[0].y),
                 "r"(r.v[0].z), "r"(r.v[0].w), "r"(r.v[1].x), "r"(r.v[1].y), "r"(r.v[1].z), "r"(r.v[1].w)
                 : "memory");
  }
}

// The same for what is not read again soon: first to leave L2.
template <typename T> __device__ __forceinline__ Raw8<T> raw_load_stream(const T* p) {
  Raw8<T> r;
  if constexpr (sizeof(T) == 2) {
    r.v[0] = __ldcs(reinterpret_cast<const uint4*>(p));
  } else {
    asm volatile("ld.global.L2::evict_first.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r.v[0].x), "=r"(r.v[0].y), "=r"(r.v[0].z), "=r"(r.v[0].w), "=r"(r.v[1].x), "=r"(r.v[1].y),
                   "=r"(r.v[1].z), "=r"(r.v[1].w)
                 : "l"(p));
  }
  return r;
}

template <typename T> __device__ __forceinline__ void raw_store_stream(T* p, const Raw8<T>& r) {
  if constexpr (sizeof(T) == 2) {
    __stcs(reinterpret_cast<uint4*>(p), r.v[0]);
  } else {
    asm volatile("st.global.L2::evict_first.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r.v[0].x),
                 "r"(r.v[0].y), "r"(r.v[0].z), "r"(r.v[0].w), "r"(r.v[1].x), "r"(r.v[1].y), "r"(r.v[1].z), "r"(r.v[1].w)
                 : "memory");
  }
}

__device__ __forceinline__ float2 unpack2(uint32_t w, __nv_bfloat16) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 unpack2(uint32_t w, __half) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __nv_bfloat16) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __half) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <typename T> __device__ __forceinline__ void unpack8(const Raw8<T>& r, float (&f)[8]) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = unpack2(w[i], T());
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f[4 * i] = __uint_as_float(r.v[i].x);
      f[4 * i + 1] = __uint_as_float(r.v[i].y);
      f[4 * i + 2] = __uint_as_float(r.v[i].z);
      f[4 * i + 3] = __uint_as_float(r.v[i].w);
    }
  }
}

template <typename T> __device__ __forceinline__ Raw8<T> pack8(const float (&f)[8]) {
  Raw8<T> r;
  if constexpr (sizeof(T) == 2) {
    r.v[0] = make_uint4(pack2(f[0], f[1], T()), pack2(f[2], f[3], T()), pack2(f[4], f[5], T()), pack2(f[6], f[7], T()));
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      r.v[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), __float_as_uint(f[4 * i + 2]),
                          __float_as_uint(f[4 * i + 3]));
  }
  return r;
}

// Two fp32 values in a register pair, worked on by one instruction (f32x2).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

template <typename T> __device__ __forceinline__ void unpack8(const Raw8<T>& r, float2 (&f)[4]) {
  if constexpr (sizeof(T) == 2) {
    f[0] = unpack2(r.v[0].x, T());
    f[1] = unpack2(r.v[0].y, T());
    f[2] = unpack2(r.v[0].z, T());
    f[3] = unpack2(r.v[0].w, T());
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f[2 * i] = make_float2(__uint_as_float(r.v[i].x), __uint_as_float(r.v[i].y));
      f[2 * i + 1] = make_float2(__uint_as_float(r.v[i].z), __uint_as_float(r.v[i].w));
    }
  }
}
template <typename T> __device__ __forceinline__ Raw8<T> pack8(const float2 (&f)[4]) {
  const float g[8] = {f[0].x, f[0].y, f[1].x, f[1].y, f[2].x, f[2].y, f[3].x, f[3].y};
  return pack8<T>(g);
}

// A thread's eight columns of a row of D. VEC: rows are aligned to eight elements and D is a multiple
// of eight, so they are one access and all in the row or all past it. Columns past the row read as
// zero and are not written.
struct Cols {
  int col, D;
};

template <typename T, bool VEC> __device__ __forceinline__ Raw8<T> load8(const T* row, const Cols& c) {
  if constexpr (VEC) {
    return c.col < c.D ? raw_load(row + c.col) : raw_zero<T>();
  } else {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = c.col + i < c.D ? to_f32(row[c.col + i]) : 0.f;
    return pack8<T>(f);
  }
}

// out = the words that begin 4 by + half bytes (half: 0 or 2) after w's first; what is past w is zero.
// `by` is the same for a whole warp, so it chooses between copies of the code that name the
// words, instead of choosing between words.
template <int BY, typename T, int N, int M>
__device__ __forceinline__ void words_from(const uint32_t (&w)[N], int half, uint32_t (&out)[M]) {
#pragma unroll
  for (int i = 0; i < M; ++i) {
    const uint32_t a = i + BY < N ? w[i + BY < N ? i + BY : 0] : 0u, b = i + BY + 1 < N ? w[i + BY + 1 < N ? i + BY + 1 : 0] : 0u;
    out[i] = sizeof(T) == 4 ? a : __funnelshift_r(a, b, 8 * half);
  }
}
template <typename T, int N, int M>
__device__ __forceinline__ void words_from(int by, const uint32_t (&w)[N], int half, uint32_t (&out)[M]) {
  switch (by) {
    case 0: words_from<0, T>(w, half, out); break;
    case 1: words_from<1, T>(w, half, out); break;
    case 2: words_from<2, T>(w, half, out); break;
    case 3: words_from<3, T>(w, half, out); break;
    default: words_from<4, T>(w, half, out); break;
  }
}

// Bytes first ... end - 1 of an aligned 16 that are in w.
template <typename T> __device__ __forceinline__ void store_part(char* at, const uint32_t* w, int first, int end) {
#pragma unroll
  for (int i = 0; i < 16 / int(sizeof(T)); ++i) {
    const int b = i * int(sizeof(T));
    if (b < first || b >= end) continue;
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<uint32_t*>(at + b) = w[i];
    else
      *reinterpret_cast<uint16_t*>(at + b) = uint16_t(i & 1 ? w[i / 2] >> 16 : w[i / 2]);
  }
}

// Eight columns of a thread, neighbouring threads with neighbouring ones. Not VEC: called by whole
// warps. The row's start is anywhere in 16 bytes, so a thread writes the aligned pieces that end in
// its own, with what it lacks of the first from the thread before it.
template <typename T, bool VEC> __device__ __forceinline__ void store8(T* row, const Cols& c, const float2 (&f)[4]) {
  const Raw8<T> raw = pack8<T>(f);
  if constexpr (VEC) {
    if (c.col < c.D) raw_store(row + c.col, raw);
  } else {
    constexpr int kPieces = int(sizeof(T)) / 2, kWords = 4 * kPieces;
    const int lane = int(threadIdx.x) % 32;
    char* at = reinterpret_cast<char*>(row + c.col);
    const int s = int(reinterpret_cast<uintptr_t>(at) & 15);
    at -= s;
    uint32_t w[kWords + 4], out[kWords + 4];  // the 16 bytes before the thread's own, and its own
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      w[4 + 4 * i] = raw.v[i].x;
      w[5 + 4 * i] = raw.v[i].y;
      w[6 + 4 * i] = raw.v[i].z;
      w[7 + 4 * i] = raw.v[i].w;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __shfl_up_sync(0xffffffffu, w[kWords + i], 1);
    words_from<T>((16 - s) / 4, w, s & 2, out);
    // bytes of the thread's pieces that are in the row, from the first piece on
    const int end = (c.D - c.col) * int(sizeof(T)) + s;
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      if (end - 16 * i >= 16 && (i > 0 || lane > 0 || s == 0))
        *reinterpret_cast<uint4*>(at + 16 * i) = make_uint4(out[4 * i], out[4 * i + 1], out[4 * i + 2], out[4 * i + 3]);
    // pieces that are not whole: the warp's first, its last (up to the next warp's first), the row's last
    if (lane == 0 && s > 0 && end > s) store_part<T>(at, out, s, end);
    const int left = end - 16 * kPieces;
    if (lane == 31 && s > 0 && left > 0) {
      store_part<T>(at + 16 * kPieces, out + kWords, 0, left < s ? left : s);
    } else if (left < 0 && end > 0) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        if (end - 16 * i > 0 && end - 16 * i < 16 && (i > 0 || lane > 0 || s == 0)) store_part<T>(at + 16 * i, out + 4 * i, 0, end - 16 * i);
    }
  }
}

// One element of a type known at run time only.
__device__ __forceinline__ void store_any(void* base, int dt, int64_t k, float v) {
  if (dt == ELEM_F32)
    static_cast<float*>(base)[k] = v;
  else if (dt == ELEM_BF16)
    static_cast<__nv_bfloat16*>(base)[k] = __float2bfloat16_rn(v);
  else
    static_cast<__half*>(base)[k] = __float2half_rn(v);
}

}  // namespace flce
