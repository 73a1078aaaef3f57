// packed.cuh -- two fp32 values in a register pair, and bf16 pieces taken apart into such pairs.
#pragma once
#include "common.cuh"

namespace fp4 {
namespace {

// two fp32 values in a register pair, each lane's operation rounded to nearest as the scalar one
__device__ __forceinline__ uint64_t pair_of(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ uint64_t pair_of(float v) { return pair_of(__float_as_uint(v), __float_as_uint(v)); }
__device__ __forceinline__ float lo_of(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi_of(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float r;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint64_t widen(uint32_t bf16x2) { return pair_of(bf16x2 << 16, bf16x2 & 0xFFFF0000u); }
__device__ __forceinline__ uint4 narrow(const uint64_t* h) {
  return make_uint4(pack_bf16x2_rn(lo_of(h[0]), hi_of(h[0])), pack_bf16x2_rn(lo_of(h[1]), hi_of(h[1])),
                    pack_bf16x2_rn(lo_of(h[2]), hi_of(h[2])), pack_bf16x2_rn(lo_of(h[3]), hi_of(h[3])));
}

}  // namespace
}  // namespace fp4
