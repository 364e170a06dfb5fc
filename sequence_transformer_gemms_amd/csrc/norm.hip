// Root-mean-square norm of a token slice with the residual's addition, and
// its backward, for gfx950.
//
// Under tensor-sequence parallelism a rank owns rows/T of the tokens between
// a row-parallel product and the next column-parallel one ("Tensor
// parallelism" algorithm page and "Tensor and sequence parallelism":
// normalisation and residual on s/T tokens).  Per row of D values:
//
//   forward   v = sum_t P_t + bias + residual;  r = 1 / sqrt(mean(v^2) + eps)
//             h = v (stored);  y = v r gamma
//   backward  dy = sum_t dP_t;  x = h r;  g = dy gamma
//             dh = r (g - x mean(g x)) + dres
//             dgamma = sum_rows dy x;  dbias = sum_rows dh
//
// The row-parallel bias enters here, once, after the sum over ranks ("Tensor
// parallelism", section "Pitfalls": added on every rank it would count T
// times).  v, the row sums and both column sums are held in fp32; y is
// computed from the unrounded v, so h and y are each rounded once.
#include "tpm_device.hpp"
#include "tpm_internal.hpp"

namespace tpm {

namespace {

__device__ __forceinline__ float ld_f(const void* p, bool f32, int64_t i) {
  return f32 ? ((const float*)p)[i] : bf16_to_f32(((const uint16_t*)p)[i]);
}
__device__ __forceinline__ void st_f(void* p, bool f32, int64_t i, float v) {
  if (f32) ((float*)p)[i] = v;
  else ((uint16_t*)p)[i] = f32_to_bf16_rne(v);
}

// Sum over the work-group (any whole number of waves up to 16), the same
// value in every thread: shuffles within a wave, then the wave sums in wave
// order.  red: 16 floats of LDS; two calls in a row need different ones.
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  const int waves = (blockDim.x + 63) >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < waves; ++w) s += red[w];
  return s;
}

// amax of the work-group's values into *amax (fp32 bits; non-negative floats
// order as integers), one atomic per work-group.
__device__ __forceinline__ void block_amax_to(float* amax, float v, float* red) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < (int)((blockDim.x + 63) >> 6); ++w) v = fmaxf(v, red[w]);
    atomicMax((unsigned int*)amax, __float_as_uint(v));
  }
}

// Padding rows of the MXFP8 scale records (rows up to the next multiple of
// 32) hold exponent 0, as mx_swizzle leaves them.  One thread per byte.
__device__ __forceinline__ void pad_mx_rows(const NormParams& p) {
  const int kb = (int)(p.D / 32);
  const int64_t pad = (p.rows + 31) / 32 * 32 - p.rows;
  for (int64_t i = threadIdx.x; i < pad * kb; i += blockDim.x)
    p.y_mx[mx_scale_offset((uint32_t)(p.rows + i / kb), (uint32_t)(i % kb), (uint32_t)(p.D / 128))] = 0;
}

// ------------------------------------------------------------ any shape
// One work-group per row, one element per thread at a time, two passes over
// the row's inputs (the second reads them again, mostly from the caches, so
// that a row of any length needs no storage).  h is stored in the second
// pass, after the element's last read: h may be the residual's buffer.
__device__ __forceinline__ float sum_in(const NormParams& p, int64_t row, int64_t c) {
  float v = 0.f;
  for (int t = 0; t < p.T; ++t) v += ld_f(p.x, p.x_f32, t * p.x_stride + row * p.ldx + c);
  if (p.bias) v += ld_f(p.bias, p.g_f32, c);
  if (p.res) v += ld_f(p.res, p.h_f32, row * p.ldr + c);
  return v;
}

__global__ void __launch_bounds__(256) norm_fwd_any(const NormParams p) {
  __shared__ float red[2][16];
  float lmax = 0.f;
  const float q_inv = p.y_scale ? 1.0f / *p.y_scale : 1.0f;
  int par = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, par ^= 1) {
    float ss = 0.f;
    for (int64_t c = threadIdx.x; c < p.D; c += 256) {
      const float v = sum_in(p, row, c);
      ss = fmaf(v, v, ss);
    }
    const float r = 1.0f / sqrtf(block_sum(ss, red[par]) / (float)p.D + p.eps);
    if (p.rstd && threadIdx.x == 0) p.rstd[row] = r;
    for (int64_t c = threadIdx.x; c < p.D; c += 256) {
      const float v = sum_in(p, row, c);
      if (p.h) st_f(p.h, p.h_f32, row * p.ldh + c, v);
      const float y = v * r * ld_f(p.gamma, p.g_f32, c);
      if (p.y_kind == NORM_Y_MX) {
        // D % 128 == 0: the 32 lanes of a block are all inside the row
        float m = fabsf(y);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
        const int E = max((int)((__float_as_uint(m) >> 23) & 0xFFu) - 8, 0);
        ((uint8_t*)p.y)[row * p.ldy + c] = f32_to_e4m3_rne_sat(y * __uint_as_float((uint32_t)(254 - E) << 23));
        if ((c & 31) == 0) p.y_mx[mx_scale_offset((uint32_t)row, (uint32_t)(c >> 5), (uint32_t)(p.D / 128))] = (uint8_t)E;
      } else if (p.y_kind == NORM_Y_E4M3) {
        lmax = fmaxf(lmax, fabsf(y));
        ((uint8_t*)p.y)[row * p.ldy + c] = f32_to_e4m3_rne_sat(y * q_inv);
      } else {
        st_f(p.y, p.y_kind == NORM_Y_F32, row * p.ldy + c, y);
      }
    }
  }
  if (p.y_kind == NORM_Y_MX && blockIdx.x == 0) pad_mx_rows(p);
  if (p.amax) {
    __syncthreads();
    block_amax_to(p.amax, lmax, red[0]);
  }
}

// One row after the other; thread c % 256 owns the columns' sums, which go
// to this work-group's row of the partial sums (read back and added to, in
// L2, from row to row).
__global__ void __launch_bounds__(256) norm_bwd_any(const NormParams p) {
  __shared__ float red[2][16];
  float* pg = p.part;                                          // [G][D] dgamma, then [G][D] dbias
  float* pb = p.part + (int64_t)gridDim.x * p.D;
  const int64_t own = (int64_t)blockIdx.x * p.D;
  int par = 0;
  bool first = true;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, par ^= 1) {
    const float r = p.rstd[row];
    float gx = 0.f;
    for (int64_t c = threadIdx.x; c < p.D; c += 256) {
      float dy = 0.f;
      for (int t = 0; t < p.T; ++t) dy += ld_f(p.x, p.x_f32, t * p.x_stride + row * p.ldx + c);
      const float x = ld_f(p.h, p.h_f32, row * p.ldh + c) * r;
      gx = fmaf(dy * ld_f(p.gamma, p.g_f32, c), x, gx);
    }
    const float m = block_sum(gx, red[par]) / (float)p.D;
    for (int64_t c = threadIdx.x; c < p.D; c += 256) {
      float dy = 0.f;
      for (int t = 0; t < p.T; ++t) dy += ld_f(p.x, p.x_f32, t * p.x_stride + row * p.ldx + c);
      const float x = ld_f(p.h, p.h_f32, row * p.ldh + c) * r;
      float dh = r * (dy * ld_f(p.gamma, p.g_f32, c) - x * m);
      if (p.res) dh += ld_f(p.res, p.h_f32, row * p.ldr + c);
      st_f(p.y, p.y_kind == NORM_Y_F32, row * p.ldy + c, dh);
      if (p.dgamma) pg[own + c] = (first ? 0.f : pg[own + c]) + dy * x;
      if (p.dbias) pb[own + c] = (first ? 0.f : pb[own + c]) + dh;
    }
    first = false;
  }
}

// dgamma and dbias: the work-groups' partial column sums added in work-group
// order, one column per thread.
__global__ void __launch_bounds__(256) norm_bwd_columns(const NormParams p, int G) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= p.D) return;
  for (int which = 0; which < 2; ++which) {
    float* out = which ? p.dbias : p.dgamma;
    if (!out) continue;
    const float* src = p.part + (which ? (int64_t)G * p.D : 0) + c;
    float s = 0.f;
    for (int g = 0; g < G; ++g) s += src[(int64_t)g * p.D];
    out[c] = s;
  }
}

}  // namespace

// Work-groups of the backward: each sums its rows' column contributions, so
// their number fixes the order of the column sums.  It depends on the shape
// alone, never on the stream.
int norm_bwd_groups(int64_t rows, int64_t) { return (int)std::min<int64_t>(rows, 256); }

hipError_t launch_norm_fwd(const NormParams& p, hipStream_t s) {
  const int grid = (int)std::min<int64_t>(p.rows, 4096);
  norm_fwd_any<<<grid, 256, 0, s>>>(p);
  return hipGetLastError();
}

hipError_t launch_norm_bwd(const NormParams& p, hipStream_t s) {
  const int G = norm_bwd_groups(p.rows, p.D);
  norm_bwd_any<<<G, 256, 0, s>>>(p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || (!p.dgamma && !p.dbias)) return e;
  norm_bwd_columns<<<(unsigned)((p.D + 255) / 256), 256, 0, s>>>(p, G);
  return hipGetLastError();
}

}  // namespace tpm
