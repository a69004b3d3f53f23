// Element types of the operators around the layer: conversions between bf16 /
// fp16 / fp32 storage and fp32 registers, 16 bytes at a time or one by one.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "common.cuh"

namespace moe {

// Programmatic dependent launch: lets the next launch begin, and waits for the end
// of the one in front (at once where the launches are not chained).
MOE_DEV void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
MOE_DEV void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Two fp32 values in one 64-bit register pair: one instruction works on both
// (fma / mul / add.rn.f32x2), each half rounded as its scalar form.
typedef unsigned long long f32x2;
MOE_DEV f32x2 f2_of(float lo, float hi) {
  f32x2 v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
MOE_DEV f32x2 f2_both(float x) { return f2_of(x, x); }
MOE_DEV void f2_split(f32x2 v, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
MOE_DEV float f2_sum(f32x2 v) {
  float lo, hi;
  f2_split(v, lo, hi);
  return lo + hi;
}
MOE_DEV f32x2 f2_fma(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
MOE_DEV f32x2 f2_mul(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

template <typename T>
struct Elem;

// 16 bytes as fp32 pairs (VEC / 2 of them) and back.
template <typename T>
MOE_DEV void unpack_pairs(const uint4 &q, f32x2 *p) {
  float v[Elem<T>::VEC];
  Elem<T>::unpack(q, v);
#pragma unroll
  for (int k = 0; k < Elem<T>::VEC / 2; ++k) p[k] = f2_of(v[2 * k], v[2 * k + 1]);
}
template <typename T>
MOE_DEV uint4 pack_pairs(const f32x2 *p) {
  float v[Elem<T>::VEC];
#pragma unroll
  for (int k = 0; k < Elem<T>::VEC / 2; ++k) f2_split(p[k], v[2 * k], v[2 * k + 1]);
  return Elem<T>::pack(v);
}

template <>
struct Elem<__nv_bfloat16> {
  static constexpr int VEC = 8;
  MOE_DEV static void unpack(const uint4 &q, float *v) {
    v[0] = bf16lo(q.x); v[1] = bf16hi(q.x);
    v[2] = bf16lo(q.y); v[3] = bf16hi(q.y);
    v[4] = bf16lo(q.z); v[5] = bf16hi(q.z);
    v[6] = bf16lo(q.w); v[7] = bf16hi(q.w);
  }
  MOE_DEV static uint32_t pack2(float lo, float hi) { return pack_bf16x2(lo, hi); }
  MOE_DEV static uint4 pack(const float *v) {
    return make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
  }
  MOE_DEV static float to(__nv_bfloat16 x) { return __bfloat162float(x); }
  MOE_DEV static __nv_bfloat16 from(float x) { return __float2bfloat16_rn(x); }
};

template <>
struct Elem<__half> {
  static constexpr int VEC = 8;
  MOE_DEV static void unpack2(uint32_t w, float *v) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    v[0] = f.x;
    v[1] = f.y;
  }
  MOE_DEV static void unpack(const uint4 &q, float *v) {
    unpack2(q.x, v);
    unpack2(q.y, v + 2);
    unpack2(q.z, v + 4);
    unpack2(q.w, v + 6);
  }
  MOE_DEV static uint32_t pack2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
  MOE_DEV static uint4 pack(const float *v) {
    return make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
  }
  MOE_DEV static float to(__half x) { return __half2float(x); }
  MOE_DEV static __half from(float x) { return __float2half_rn(x); }
};

template <>
struct Elem<float> {
  static constexpr int VEC = 4;
  MOE_DEV static void unpack(const uint4 &q, float *v) {
    v[0] = __uint_as_float(q.x);
    v[1] = __uint_as_float(q.y);
    v[2] = __uint_as_float(q.z);
    v[3] = __uint_as_float(q.w);
  }
  MOE_DEV static uint4 pack(const float *v) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
  MOE_DEV static float to(float x) { return x; }
  MOE_DEV static float from(float x) { return x; }
};

// Streaming 16-byte accesses: read once / written once, so they do not displace
// what is used again (weights, column sums) from L1 and L2.
MOE_DEV uint4 ld_stream(const void *p) { return __ldcs(reinterpret_cast<const uint4 *>(p)); }
MOE_DEV void st_stream(void *p, const uint4 &v) { __stcs(reinterpret_cast<uint4 *>(p), v); }

inline __host__ __device__ int elem_bytes(int elem) { return elem == MOE_ELEM_FP32 ? 4 : 2; }

}  // namespace moe
