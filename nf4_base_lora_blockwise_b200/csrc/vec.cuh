// vec.cuh -- vectors of VEC consecutive bf16 or fp32 elements between global memory and fp32
// registers, for the elementwise and row-wise kernels.  VEC * sizeof(T) is one access of up to 16
// bytes, or two of 16 (8 fp32 elements); pointers are aligned to it.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace qlora {

__device__ __forceinline__ float2 bf16x2_floats(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t floats_bf16x2(float a, float b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}

template <int VEC>
__device__ __forceinline__ void load_vec(const __nv_bfloat16* p, float (&f)[VEC]) {
  static_assert(VEC == 8 || VEC == 4 || VEC == 2 || VEC == 1, "vector width");
  if constexpr (VEC == 8) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = bf16x2_floats(w[i]);
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  } else if constexpr (VEC == 4) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    const float2 a = bf16x2_floats(v.x), b = bf16x2_floats(v.y);
    f[0] = a.x;
    f[1] = a.y;
    f[2] = b.x;
    f[3] = b.y;
  } else if constexpr (VEC == 2) {
    const float2 t = bf16x2_floats(*reinterpret_cast<const uint32_t*>(p));
    f[0] = t.x;
    f[1] = t.y;
  } else {
    f[0] = __bfloat162float(*p);
  }
}

template <int VEC>
__device__ __forceinline__ void load_vec(const float* p, float (&f)[VEC]) {
  static_assert(VEC == 8 || VEC == 4 || VEC == 2 || VEC == 1, "vector width");
  if constexpr (VEC >= 4) {
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
      const float4 v = reinterpret_cast<const float4*>(p)[i];
      f[4 * i] = v.x;
      f[4 * i + 1] = v.y;
      f[4 * i + 2] = v.z;
      f[4 * i + 3] = v.w;
    }
  } else if constexpr (VEC == 2) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    f[0] = v.x;
    f[1] = v.y;
  } else {
    f[0] = *p;
  }
}

template <int VEC>
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&f)[VEC]) {
  if constexpr (VEC == 8) {
    uint4 v;
    v.x = floats_bf16x2(f[0], f[1]);
    v.y = floats_bf16x2(f[2], f[3]);
    v.z = floats_bf16x2(f[4], f[5]);
    v.w = floats_bf16x2(f[6], f[7]);
    *reinterpret_cast<uint4*>(p) = v;
  } else if constexpr (VEC == 4) {
    *reinterpret_cast<uint2*>(p) = make_uint2(floats_bf16x2(f[0], f[1]), floats_bf16x2(f[2], f[3]));
  } else if constexpr (VEC == 2) {
    *reinterpret_cast<uint32_t*>(p) = floats_bf16x2(f[0], f[1]);
  } else {
    *p = __float2bfloat16_rn(f[0]);
  }
}

template <int VEC>
__device__ __forceinline__ void store_vec(float* p, const float (&f)[VEC]) {
  if constexpr (VEC >= 4) {
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i)
      reinterpret_cast<float4*>(p)[i] =
          make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
  } else if constexpr (VEC == 2) {
    *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
  } else {
    *p = f[0];
  }
}

// VEC elements at index i of an array that is fp32 when `f32`, else bf16.
template <int VEC>
__device__ __forceinline__ void load_either(const void* base, bool f32, int64_t i,
                                            float (&f)[VEC]) {
  if (f32)
    load_vec<VEC>(static_cast<const float*>(base) + i, f);
  else
    load_vec<VEC>(static_cast<const __nv_bfloat16*>(base) + i, f);
}
__device__ __forceinline__ float load_either1(const void* base, bool f32, int64_t i) {
  return f32 ? static_cast<const float*>(base)[i]
             : __bfloat162float(static_cast<const __nv_bfloat16*>(base)[i]);
}

// Two fp32 values in one register pair, with the rounding of the scalar operations.
using f2 = unsigned long long;
__device__ __forceinline__ f2 pair(float a, float b) {
  f2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ f2 pair_bits(uint32_t a, uint32_t b) {
  f2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ float2 split(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ f2 both(float a) { return pair(a, a); }
__device__ __forceinline__ float sum2(f2 v) {
  const float2 t = split(v);
  return t.x + t.y;
}
__device__ __forceinline__ uint32_t pack_bf16(f2 v) {
  const float2 t = split(v);
  return floats_bf16x2(t.x, t.y);
}
__device__ __forceinline__ f2 unpack_bf16(uint32_t w) { return pair_bits(w << 16, w & 0xFFFF0000u); }

}  // namespace qlora
