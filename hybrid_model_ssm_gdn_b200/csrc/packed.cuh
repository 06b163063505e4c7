// packed.cuh -- pairs of fp32 values in one 64-bit register, two operations an instruction (sm_100a).
#pragma once

#include "common.cuh"

namespace rssm {

struct f2 {
  unsigned long long v;
};
__device__ __forceinline__ f2 pack2(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ f2 pack2(uint32_t a, uint32_t b) { return pack2(__uint_as_float(a), __uint_as_float(b)); }
__device__ __forceinline__ void unpack2(f2 p, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p.v)); }
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ f2 sub2(f2 a, f2 b) {
  f2 r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// the two bf16 pieces of a pair: hi = RN(v), lo = RN(v - hi), |v - hi - lo| <= 2^-17 |v|
__device__ __forceinline__ void cut2(f2 v, uint32_t &hi, uint32_t &lo) {
  float a, b;
  unpack2(v, a, b);
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  hi = *reinterpret_cast<const uint32_t *>(&h);
  unpack2(sub2(v, pack2(hi << 16, hi & 0xffff0000u)), a, b);
  const __nv_bfloat162 l = __floats2bfloat162_rn(a, b);
  lo = *reinterpret_cast<const uint32_t *>(&l);
}

// The three bf16 pieces of a pair, each to nearest, exact in all: 8 bits of what those before it left.  (12.8 issue cycles of
// a scheduler; 16.2 with pieces that are masked off, since the masks' instructions are no cheaper than the conversions.)
__device__ __forceinline__ void cut3(f2 v, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
  float a, b;
  unpack2(v, a, b);
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  hi = *reinterpret_cast<const uint32_t *>(&h);
  const f2 left = sub2(v, pack2(hi << 16, hi & 0xffff0000u));
  unpack2(left, a, b);
  const __nv_bfloat162 m = __floats2bfloat162_rn(a, b);
  mid = *reinterpret_cast<const uint32_t *>(&m);
  unpack2(sub2(left, pack2(mid << 16, mid & 0xffff0000u)), a, b);
  const __nv_bfloat162 l = __floats2bfloat162_rn(a, b);
  lo = *reinterpret_cast<const uint32_t *>(&l);
}

}  // namespace rssm
