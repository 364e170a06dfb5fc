// Element and eight-element access to rows of bf16 or fp32 at any element
// address (gfx950 takes unaligned vector accesses): the bandwidth-bound
// kernels of the token-slice norm and the linear layer.
#pragma once
#include "tpm_device.hpp"

namespace tpm {

namespace {

__device__ __forceinline__ float ld_f(const void* p, bool f32, int64_t i) {
  return f32 ? ((const float*)p)[i] : bf16_to_f32(((const uint16_t*)p)[i]);
}
__device__ __forceinline__ void st_f(void* p, bool f32, int64_t i, float v) {
  if (f32) ((float*)p)[i] = v;
  else ((uint16_t*)p)[i] = f32_to_bf16_rne(v);
}

typedef i32x4 i32x4_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef i32x2 i32x2_any __attribute__((aligned(1)));
typedef uint32_t u32_any __attribute__((aligned(1)));

template <bool F32>
struct Raw8 {   // eight elements as loaded
  i32x4 a, b;   // (b: fp32 only)
};
template <bool F32>
__device__ __forceinline__ Raw8<F32> load8(const void* p, int64_t i) {
  Raw8<F32> r;
  if constexpr (F32) {
    r.a = __builtin_bit_cast(i32x4, __builtin_nontemporal_load((const f32x4_any*)((const float*)p + i)));
    r.b = __builtin_bit_cast(i32x4, __builtin_nontemporal_load((const f32x4_any*)((const float*)p + i + 4)));
  } else {
    r.a = __builtin_nontemporal_load((const i32x4_any*)((const uint16_t*)p + i));
  }
  return r;
}
template <bool F32>
__device__ __forceinline__ void widen8(const Raw8<F32>& r, float (&v)[8]) {
  if constexpr (F32) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = __int_as_float(r.a[e]);
      v[4 + e] = __int_as_float(r.b[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = __uint_as_float((uint32_t)r.a[e] << 16);
      v[2 * e + 1] = __uint_as_float((uint32_t)r.a[e] & 0xFFFF0000u);
    }
  }
}
// gamma or bias: read again for every row, from the caches
__device__ __forceinline__ void param8(const void* p, bool f32, int64_t i, float (&v)[8]) {
  if (f32) {
    const f32x4 a = *(const f32x4_any*)((const float*)p + i), b = *(const f32x4_any*)((const float*)p + i + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = a[e];
      v[4 + e] = b[e];
    }
  } else {
    Raw8<false> r;
    r.a = *(const i32x4_any*)((const uint16_t*)p + i);
    widen8<false>(r, v);
  }
}
template <bool F32>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&v)[8], int shift) {
  if (__builtin_expect(shift != 0, 0)) {
#pragma unroll
    for (int e = 1; e < 8; ++e)
      if (e >= shift) st_f(p, F32, i + e, v[e]);
    return;
  }
  if constexpr (F32) {
    *(f32x4_any*)((float*)p + i) = f32x4{v[0], v[1], v[2], v[3]};
    *(f32x4_any*)((float*)p + i + 4) = f32x4{v[4], v[5], v[6], v[7]};
  } else {
    i32x4 o;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = (int)pack_bf16x2(v[2 * e], v[2 * e + 1]);
    *(i32x4_any*)((uint16_t*)p + i) = o;
  }
}
__device__ __forceinline__ void codes8(uint8_t* p, const float (&y)[8], int shift) {
  const uint32_t lo = fp8x4<false>(y[0], y[1], y[2], y[3]), hi = fp8x4<false>(y[4], y[5], y[6], y[7]);
  if (__builtin_expect(shift != 0, 0)) {
#pragma unroll
    for (int e = 1; e < 8; ++e)
      if (e >= shift) p[e] = (uint8_t)((e < 4 ? lo : hi) >> (8 * (e & 3)));
    return;
  }
  *(i32x2_any*)p = i32x2{(int)lo, (int)hi};
}
}  // namespace

// out[c] = sum over g < G of src[g, c] for the 64 columns from c0, by a
// work-group of WAVES waves: a wave's lanes read 256 contiguous bytes of every
// WAVES-th row, and the wave sums are added in wave order.  red: WAVES * 64
// floats of LDS.
template <int WAVES>
__device__ __forceinline__ void sum_columns(const float* src, int G, int64_t D, int64_t c0, float* red, float* out) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = c0 + lane;
  float s = 0.f;
  if (c < D) {
#pragma unroll 8
    for (int g = wave; g < G; g += WAVES) s += src[(int64_t)g * D + c];
  }
  red[wave * 64 + lane] = s;
  __syncthreads();
  if (wave == 0 && c < D) {
    for (int w = 1; w < WAVES; ++w) s += red[w * 64 + lane];
    out[c] = s;
  }
}

}  // namespace tpm
