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
#include <algorithm>
#include <type_traits>

#include "row_vec.hpp"
#include "tpm_internal.hpp"

namespace tpm {

namespace {

// widest rows held in the registers of 1024 threads: 4 chunks of 8 each, 2 in
// the backward, which also holds two column sums per column
constexpr int64_t kNormMaxFwd = 32768, kNormMaxBwd = 16384;

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

// 1 / sqrt(mean(v^2) + eps) to 48 bits, as hi + lo, and v r gamma rounded
// once.  For the 8-bit outputs, where a value next to a code's boundary falls
// on the other side by any error: at 8192 rows of 16384, 48 of 134M codes are
// not those of the exact values, 78 with r and the products in plain fp32,
// for 190 against 186 us.
__device__ __forceinline__ float row_factor(float ss, const NormParams& p, float& lo) {
  const double r = 1.0 / sqrt((double)ss / (double)p.D + (double)p.eps);
  lo = (float)(r - (double)(float)r);
  return (float)r;
}
__device__ __forceinline__ float scaled(float v, float r, float r_lo, float gamma) {
  const float x = v * r;
  // (an infinite gamma times a zero correction would be NaN)
  return fmaf(x, gamma, fmaf(v, r_lo, fmaf(v, r, -x)) * __builtin_amdgcn_fmed3f(gamma, -3e38f, 3e38f));
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
    float r_lo;
    const float r = row_factor(block_sum(ss, red[par]), p, r_lo);
    if (p.rstd && threadIdx.x == 0) p.rstd[row] = r;
    for (int64_t c = threadIdx.x; c < p.D; c += 256) {
      const float v = sum_in(p, row, c);
      if (p.h) st_f(p.h, p.h_f32, row * p.ldh + c, v);
      const float y = scaled(v, r, r_lo, ld_f(p.gamma, p.g_f32, c));
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

// ------------------------------------------------------ a row in registers
// A thread holds V chunks of eight consecutive columns of its row, chunk u at
// column 8 (u * NT + t) for thread t of the row's NT, so every load and store
// of a wave covers contiguous memory and each input is read once.  Loads and
// stores move 16 bytes at any element address (gfx950 takes unaligned vector
// accesses), so rows of odd width or stride run here too: where D % 8 != 0
// the row's last chunk is loaded from column D - 8, `shift` of its elements
// belong to the chunk before it, are zeroed, and are not stored.
// v += the partials t .. T - 1 of one chunk at `at`, fp32 in ascending t, up to
// B loads in flight; sum_partials: v = all of them
template <bool F32, int B>
__device__ __forceinline__ void add_partials(const NormParams& p, int64_t at, int t, float (&v)[8]) {
#pragma unroll 1
  for (; t < p.T; t += B) {
    Raw8<F32> q[B];
#pragma unroll
    for (int k = 0; k < B; ++k)
      if (t + k < p.T) q[k] = load8<F32>(p.x, at + (int64_t)(t + k) * p.x_stride);
#pragma unroll
    for (int k = 0; k < B; ++k)
      if (t + k < p.T) {
        float w[8];
        widen8<F32>(q[k], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += w[e];
      }
  }
}

template <bool F32, int B>
__device__ __forceinline__ void sum_partials(const NormParams& p, int64_t at, float (&v)[8]) {
  widen8<F32>(load8<F32>(p.x, at), v);
  add_partials<F32, B>(p, at, 1, v);
}

// Sum over the `waves` (1 .. 16) waves of a row, whose first wave in the
// work-group is `first`.  Every thread of the work-group calls it.
__device__ __forceinline__ float row_sum(float v, int first, int waves, float* red) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < waves; ++w) s += red[first + w];
  return s;
}

// chunk u of thread t: its first column, or -1 past the row's end; the
// elements below `shift` are the previous chunk's
__device__ __forceinline__ int chunk_at(int u, int NT, int t, int D, int& shift) {
  const int c = 8 * (u * NT + t);
  shift = 0;
  if (c + 8 <= D) return c;
  shift = c + 8 - D;
  return c < D ? D - 8 : -1;
}
__device__ __forceinline__ void drop(float (&v)[8], int shift) {
  if (shift)
#pragma unroll
    for (int e = 0; e < 7; ++e) v[e] = e < shift ? 0.f : v[e];
}

// FP8: y in one of the two 8-bit forms (a kernel of its own: the encoders'
// NaN path would cost the other one half its registers).
template <bool XF, bool HF, int V, bool FP8>
__global__ void __launch_bounds__(1024, 4) norm_fwd_vec(const NormParams p, int NT) {
  __shared__ float red[2][16];
  const int slots = blockDim.x / NT;                  // rows of the work-group
  const int slot = threadIdx.x / NT;
  int t = threadIdx.x - slot * NT;
  const int waves = NT >> 6, wave0 = slot * waves;
  const int D = (int)p.D;
  const float q_inv = FP8 && p.y_scale ? 1.0f / *p.y_scale : 1.0f;
  const float inv_d = 1.0f / (float)D;
  float lmax = 0.f;
  int par = 0;
  // (the loop bound is the work-group's: every thread meets the barriers)
  for (int64_t row0 = (int64_t)blockIdx.x * slots; row0 < p.rows; row0 += (int64_t)gridDim.x * slots, par ^= 1) {
    const int64_t row = row0 + slot;
    const bool live = row < p.rows;
    asm volatile("" : "+v"(t));   // column offsets are formed per row, not kept for every array
    float v[V][8];
    float ss = 0.f;
#pragma unroll
    for (int u = 0; u < V; ++u) {
      int shift;
      const int c = chunk_at(u, NT, t, D, shift);
      if (live && c >= 0) {
        Raw8<HF> rr;
        if (p.res) rr = load8<HF>(p.res, row * p.ldr + c);
        sum_partials<XF, 4>(p, row * p.ldx + c, v[u]);
        if (p.bias) {
          float w[8];
          param8(p.bias, p.g_f32, c, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[u][e] += w[e];
        }
        if (p.res) {
          float w[8];
          widen8<HF>(rr, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[u][e] += w[e];
        }
        drop(v[u], shift);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(v[u][e], v[u][e], ss);
      }
    }
    float r, r_lo = 0.f;
    if constexpr (FP8) r = row_factor(row_sum(ss, wave0, waves, red[par]), p, r_lo);
    else r = 1.0f / sqrtf(row_sum(ss, wave0, waves, red[par]) * inv_d + p.eps);
    if (!live) continue;
    if (p.rstd && t == 0) p.rstd[row] = r;
#pragma unroll
    for (int u = 0; u < V; ++u) {
      int shift;
      const int c = chunk_at(u, NT, t, D, shift);
      if (c < 0) continue;
      float y[8];
      param8(p.gamma, p.g_f32, c, y);
      if (p.h) store8<HF>(p.h, row * p.ldh + c, v[u], shift);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if constexpr (FP8) y[e] = scaled(v[u][e], r, r_lo, y[e]);
        else y[e] = v[u][e] * r * y[e];
      }
      if constexpr (!FP8) {
        if (p.y_kind == NORM_Y_F32) store8<true>(p.y, row * p.ldy + c, y, shift);
        else store8<false>(p.y, row * p.ldy + c, y, shift);
      } else if (p.y_kind == NORM_Y_E4M3) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          lmax = fmaxf(lmax, fabsf(y[e]));
          y[e] *= q_inv;
        }
        codes8((uint8_t*)p.y + row * p.ldy + c, y, shift);
      } else {
        // a 32-column block is four lanes (D % 128 == 0: all inside the row)
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          m = fmaxf(m, fabsf(y[e]));
        }
        m = fmaxf(m, __shfl_xor(m, 1, 64));
        m = fmaxf(m, __shfl_xor(m, 2, 64));
        const int E = max((int)((__float_as_uint(m) >> 23) & 0xFFu) - 8, 0);
        const float inv = __uint_as_float((uint32_t)(254 - E) << 23);   // 2^(127 - E)
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] *= inv;
        codes8((uint8_t*)p.y + row * p.ldy + c, y, 0);
        // the four scales of 128 columns are one dword of the row's record
        uint32_t w = (uint32_t)E << (8 * ((threadIdx.x >> 2) & 3));
        w |= (uint32_t)__shfl_xor((int)w, 4, 64);
        w |= (uint32_t)__shfl_xor((int)w, 8, 64);
        if ((threadIdx.x & 15) == 0)
          *(u32_any*)(p.y_mx + mx_scale_offset((uint32_t)row, (uint32_t)(c >> 5), (uint32_t)(D >> 7))) = w;
      }
    }
  }
  if constexpr (FP8) {
    if (p.y_kind == NORM_Y_MX && blockIdx.x == 0) pad_mx_rows(p);
    if (p.amax) {
      __syncthreads();
      block_amax_to(p.amax, lmax, red[0]);
    }
  }
}

// Backward.  A work-group holds blockDim / NT rows at a time and walks the
// rows with a stride; each thread keeps the dgamma and dbias sums of its own
// columns over all the rows it sees.  At the end the row slots' sums are
// added in LDS and leave as one row of partial sums per work-group.  With one
// chunk a thread, the next row's h, dres and first partials are loaded before
// this row's sum, whose barrier they would otherwise wait behind (T = 8, rows
// 1024, D 8192: 41 us, 44.6 without; fp32, T = 1, rows and D 8192: 209 and 232);
// more than two partials ahead gain nothing (42).
template <bool XF, bool HF, int V>
__global__ void __launch_bounds__(1024) norm_bwd_vec(const NormParams p, int NT) {
  __shared__ float red[2][16];
  __shared__ float cols[8192 * V];   // [slot][V * NT * 8]
  const int slots = blockDim.x / NT;
  const int slot = threadIdx.x / NT;
  int t = threadIdx.x - slot * NT;
  const int waves = NT >> 6, wave0 = slot * waves;
  const int D = (int)p.D;
  float sg[V][8], sb[V][8];
#pragma unroll
  for (int u = 0; u < V; ++u)
#pragma unroll
    for (int e = 0; e < 8; ++e) sg[u][e] = sb[u][e] = 0.f;
  const float inv_d = 1.0f / (float)D;
  int par = 0;
  constexpr int AHEAD = 2;
  Raw8<XF> nx[AHEAD];   // V == 1: the next row's
  Raw8<HF> nh, nd;
  float nr = 0.f;
  auto ahead = [&](int64_t row) {
    int shift;
    const int c = chunk_at(0, NT, t, D, shift);
    if (row >= p.rows || c < 0) return;
    nh = load8<HF>(p.h, row * p.ldh + c);
    if (p.res) nd = load8<HF>(p.res, row * p.ldr + c);
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (k < p.T) nx[k] = load8<XF>(p.x, row * p.ldx + c + k * p.x_stride);
    nr = p.rstd[row];
  };
  if (V == 1) ahead((int64_t)blockIdx.x * slots + slot);
  for (int64_t row0 = (int64_t)blockIdx.x * slots; row0 < p.rows; row0 += (int64_t)gridDim.x * slots, par ^= 1) {
    const int64_t row = row0 + slot;
    const bool live = row < p.rows;
    asm volatile("" : "+v"(t));   // column offsets are formed per row, not kept for every array
    float dy[V][8];
    Raw8<HF> hh[V], dres[V];
    float gx = 0.f;
    const float r = V == 1 ? nr : live ? p.rstd[row] : 0.f;
#pragma unroll
    for (int u = 0; u < V; ++u) {
      int shift;
      const int c = chunk_at(u, NT, t, D, shift);
      if (live && c >= 0) {
        float g[8], x[8];
        if constexpr (V == 1) {
          hh[u] = nh;
          dres[u] = nd;
          widen8<XF>(nx[0], dy[u]);
#pragma unroll
          for (int k = 1; k < AHEAD; ++k)
            if (k < p.T) {
              widen8<XF>(nx[k], x);
#pragma unroll
              for (int e = 0; e < 8; ++e) dy[u][e] += x[e];
            }
          add_partials<XF, XF ? 2 : 4>(p, row * p.ldx + c, AHEAD, dy[u]);
        } else {
          hh[u] = load8<HF>(p.h, row * p.ldh + c);
          if (p.res) dres[u] = load8<HF>(p.res, row * p.ldr + c);
          sum_partials<XF, XF ? 2 : 4>(p, row * p.ldx + c, dy[u]);
        }
        param8(p.gamma, p.g_f32, c, g);
        drop(dy[u], shift);
        widen8<HF>(hh[u], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] *= r;
          sg[u][e] = fmaf(dy[u][e], x[e], sg[u][e]);
          dy[u][e] *= g[e];
          gx = fmaf(dy[u][e], x[e], gx);
        }
      }
    }
    if (V == 1) ahead(row + (int64_t)gridDim.x * slots);
    const float m = row_sum(gx, wave0, waves, red[par]) * inv_d;
    if (!live) continue;
#pragma unroll
    for (int u = 0; u < V; ++u) {
      int shift;
      const int c = chunk_at(u, NT, t, D, shift);
      if (c < 0) continue;
      float dh[8], x[8];
      widen8<HF>(hh[u], x);
#pragma unroll
      for (int e = 0; e < 8; ++e) dh[e] = r * (dy[u][e] - x[e] * r * m);
      if (p.res) {
        widen8<HF>(dres[u], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) dh[e] += x[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sb[u][e] += dh[e];
      if (p.y_kind == NORM_Y_F32) store8<true>(p.y, row * p.ldy + c, dh, shift);
      else store8<false>(p.y, row * p.ldy + c, dh, shift);
    }
  }
  for (int which = 0; which < 2; ++which) {
    if (!(which ? p.dbias : p.dgamma)) continue;
    float* out = p.part + ((int64_t)which * gridDim.x + blockIdx.x) * p.D;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < V; ++u) {
      int shift;
      const int c = chunk_at(u, NT, t, D, shift);
      if (c < 0) continue;
      float* to = slots == 1 ? out : cols + slot * (V * NT * 8);
      store8<true>(to, c, which ? sb[u] : sg[u], shift);
    }
    if (slots == 1) continue;
    __syncthreads();
    for (int k = threadIdx.x; k < D; k += blockDim.x) {
      float s = 0.f;
      for (int i = 0; i < slots; ++i) s += cols[i * (V * NT * 8) + k];
      out[k] = s;
    }
  }
}

// Column sums of fp32 partial rows: out0 of src [G, D], and out1 of the [G, D]
// behind it (either may be null).  256 work-groups of 16 waves at D = 8192
// with both sums.
__global__ void __launch_bounds__(1024) column_sums(const float* part, int G, int64_t D, float* out0, float* out1) {
  __shared__ float red[16 * 64];
  const bool second = blockIdx.y == 1 || !out0;
  sum_columns<16>(part + (second ? (int64_t)G * D : 0), G, D, (int64_t)blockIdx.x * 64, red, second ? out1 : out0);
}

}  // namespace

// The most work-groups of the backward.  Each sums its rows' column
// contributions, so their number fixes the order of the column sums; it depends
// on the shape and the types alone, never on the stream or the arrays.  1024
// threads per CU either way: 512 work-groups of 512 threads where each sees
// eight rows or more (rows 8192, D 8192: 98 us, 104 with 256 of 1024), 256 of
// 1024 where the partial sums' own traffic counts (T = 8, rows 1024, D 8192: 41
// us and 48; rows 8192, D 16384: 201 and 210).
// whole waves that cover D columns at V chunks of 8 a thread
static int row_threads(int64_t D, int V) { return (int)((D + 512 * V - 1) / (512 * V)) * 64; }

// Rows of NT threads that a work-group of the backward holds, and the most
// work-groups.  Each sums its rows' column contributions, so their number
// fixes the order of the column sums; it depends on the shape and the types
// alone, never on the stream or the arrays.  Up to 1024 threads per CU either
// way: two work-groups of about 512 where each sees eight rows or more (rows
// 8192, D 8192: 98 us, 104 with 256 of 1024; D 7000 99 and 106), one of 1024 where
// rows of three, five or six waves would leave more of a CU idle (rows 20000, D
// 4099 159 and 198; 16384 x 2560 80 and 84), where the partial sums' own traffic
// counts (T = 8, rows 1024, D 8192: 41 us and 48), and for wide rows (8192 x 16384
// 201 and 210).
static int bwd_slots(int64_t rows, int64_t D, int NT) {
  const int w = NT / 64;
  const bool two = rows >= 4096 && D <= 8192 && (16 % w == 0 || w == 7);
  return std::max(1, (two ? 8 : 16) / w);
}
static int bwd_groups(int64_t rows, int64_t D, int NT) {
  const int threads = NT * bwd_slots(rows, D, NT);
  return (int)std::min<int64_t>(rows, rows >= 4096 && D <= 8192 && threads <= 512 ? 512 : 256);
}
int norm_bwd_groups(int64_t rows, int64_t D) {
  return D > kNormMaxBwd ? (int)std::min<int64_t>(rows, 256)
                         : std::max(bwd_groups(rows, D, row_threads(D, 1)), bwd_groups(rows, D, row_threads(D, 2)));
}

template <class F>
static void with_types(const NormParams& p, F&& f) {
  using T = std::true_type;
  using N = std::false_type;
  if (p.x_f32 && p.h_f32) f(T{}, T{});
  else if (p.x_f32) f(T{}, N{});
  else if (p.h_f32) f(N{}, T{});
  else f(N{}, N{});
}
template <class F>
static void with_chunks(int V, F&& f) {
  if (V == 1) f(std::integral_constant<int, 1>{});
  else if (V == 2) f(std::integral_constant<int, 2>{});
  else f(std::integral_constant<int, 4>{});
}

hipError_t launch_norm_fwd(const NormParams& p, hipStream_t s) {
  if (p.D < 8 || p.D > kNormMaxFwd) {
    norm_fwd_any<<<(int)std::min<int64_t>(p.rows, 4096), 256, 0, s>>>(p);
    return hipGetLastError();
  }
  // Chunks per thread.  Few rows: one, the most threads on each row.  Else
  // more bytes in flight per row and more rows per CU: rows 1024, D 8192, T = 8
  // 33 us with four, 37 with two, 43 with one; rows 8192, D 8192, T = 1 85 us
  // with two, 94 with four, 116 with one; rows 8192, D 16384 198 us with four,
  // 210 with two (e4m3 191 and 222).
  int V = p.rows < 512 ? 1 : (p.T >= 4 || p.D > 8192) ? 4 : 2;
  while (p.D > 8192 * V) V *= 2;
  const int NT = row_threads(p.D, V);
  const int threads = std::max(1, 256 / NT) * NT;
  const int slots = threads / NT;
  // bf16 and fp32 outputs: every row a work-group of its own, whatever number
  // of them a CU holds (rows 8192, D 8192 85 us, 100 with a grid of 2048 threads
  // per CU; 16384 x 6000 150 and 167; 16384 x 2560 58 and 70; 2048 x 8192 29 both).
  // 8-bit outputs: 1024 threads per CU, which are resident together, because
  // the amax and the encoders' code are paid per work-group (16384 x 8192 e4m3 190
  // us, 224 with one row each; 10000 x 1300 42 and 71, 45 with 2048 threads).
  const bool fp8 = p.y_kind == NORM_Y_E4M3 || p.y_kind == NORM_Y_MX;
  const int64_t most = fp8 ? 256 * (1024 / threads) : (int64_t(1) << 31) / threads;
  const int grid = (int)std::min<int64_t>((p.rows + slots - 1) / slots, most);
  with_chunks(V, [&](auto vc) {
    with_types(p, [&](auto xf, auto hf) {
      constexpr bool XF = decltype(xf)::value, HF = decltype(hf)::value;
      constexpr int V = decltype(vc)::value;
      if (fp8) norm_fwd_vec<XF, HF, V, true><<<grid, threads, 0, s>>>(p, NT);
      else norm_fwd_vec<XF, HF, V, false><<<grid, threads, 0, s>>>(p, NT);
    });
  });
  return hipGetLastError();
}

hipError_t launch_norm_bwd(const NormParams& p, hipStream_t s) {
  int G = norm_bwd_groups(p.rows, p.D);
  if (p.D < 8 || p.D > kNormMaxBwd) {
    norm_bwd_any<<<G, 256, 0, s>>>(p);
  } else {
    // Two chunks per thread; one where that leaves the registers for all the
    // loads of many partials, or of fp32 arrays, and of the next row (T = 8, rows
    // 1024, D 8192: 41 us, 48 with two; fp32, T = 2, rows 1001, D 4099: 27 and
    // 37), and for few rows, which then get work-groups of their own (rows 100,
    // D 8192: 12 us and 17).
    const bool few = p.rows <= 256;
    const int V = p.D <= 8192 && (p.x_f32 || p.h_f32 || p.T >= 4 || few) ? 1 : 2;
    const int NT = row_threads(p.D, V);
    const int slots = few ? 1 : bwd_slots(p.rows, p.D, NT);
    if (!few) G = (int)std::min<int64_t>(bwd_groups(p.rows, p.D, NT), (p.rows + slots - 1) / slots);
    const int threads = slots * NT;
    with_types(p, [&](auto xf, auto hf) {
      constexpr bool XF = decltype(xf)::value, HF = decltype(hf)::value;
      if (V == 1) norm_bwd_vec<XF, HF, 1><<<G, threads, 0, s>>>(p, NT);
      else norm_bwd_vec<XF, HF, 2><<<G, threads, 0, s>>>(p, NT);
    });
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return launch_column_sums(p.part, G, p.D, p.dgamma, p.dbias, s);
}

hipError_t launch_column_sums(const float* part, int G, int64_t D, float* out0, float* out1, hipStream_t s) {
  if (D == 0 || (!out0 && !out1)) return hipSuccess;
  const dim3 grid((unsigned)((D + 63) / 64), out0 && out1 ? 2 : 1);
  column_sums<<<grid, 1024, 0, s>>>(part, G, D, out0, out1);
  return hipGetLastError();
}

}  // namespace tpm
