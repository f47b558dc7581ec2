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

// A thread's eight columns of a row of D: col, col + 1, ... where rows are aligned to eight elements
// and D is a multiple of eight (VEC: one access), else col, col + step, ... with neighbouring
// threads on neighbouring columns. Columns past the row read as zero and are not written.
struct Cols {
  int col, step, D;
  bool kept;  // a kernel with registers to spare keeps the offsets
  __device__ __forceinline__ int at(int i) const { return col + i * step; }
  // The same columns, to the compiler others: kept from one tensor to the next, their eight
  // offsets and addresses cost the registers that the sums need.
  __device__ __forceinline__ Cols afresh() const {
    Cols c = *this;
    if (!kept) asm("" : "+r"(c.col), "+r"(c.step));
    return c;
  }
};

template <typename T, bool VEC> __device__ __forceinline__ Raw8<T> load8(const T* row, const Cols& c) {
  if constexpr (VEC) {
    return c.col < c.D ? raw_load(row + c.col) : raw_zero<T>();
  } else {
    float f[8];
    const Cols d = c.afresh();
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = d.at(i) < d.D ? to_f32(row[d.at(i)]) : 0.f;
    return pack8<T>(f);
  }
}

template <typename T, bool VEC> __device__ __forceinline__ void store8(T* row, const Cols& c, const float2 (&f)[4]) {
  if constexpr (VEC) {
    if (c.col < c.D) raw_store(row + c.col, pack8<T>(f));
  } else {
    const float g[8] = {f[0].x, f[0].y, f[1].x, f[1].y, f[2].x, f[2].y, f[3].x, f[3].y};
    const Cols d = c.afresh();
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (d.at(i) < d.D) row[d.at(i)] = from_f32<T>(g[i]);
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
