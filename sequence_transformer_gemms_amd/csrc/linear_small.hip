// The linear layer's kernels beside the 256 x 256 tile program: few rows (a
// decoding step), shapes and alignments that are no whole 16-byte chunks, fp32
// on the matrix cores; and the elementwise part of its backward.
#include <algorithm>
#include <type_traits>

#include "row_vec.hpp"
#include "tpm_internal.hpp"

namespace tpm {

namespace {

__device__ __forceinline__ float scale_of(const GemmParams& p) {
  float s = 1.f;
  if (p.a_scale) s *= *p.a_scale;
  if (p.b_scale) s *= *p.b_scale;
  return s;
}

// Epilogue of one element: z = v + bias kept in aux, Y = act(z) + residual.
template <int ACT>
__device__ __forceinline__ void finish_one(const GemmParams& p, float v, int64_t row, int64_t col) {
  if (p.bias) v += ld_f(p.bias, p.bias_f32, col);
  if (p.aux) st_f(p.aux, p.aux_f32, row * p.ldaux + col, v);
  v = act_fwd_c<ACT>(v);
  if (p.resid) v += ld_f(p.resid, p.y_f32, row * p.ldr + col);
  st_f(p.Y, p.y_f32, row * p.ldy + col, v);
}

// K-range partial sums [splits, M, N] added in ascending order, then the epilogue.
__global__ void __launch_bounds__(256) finish_splits(const GemmParams p) {
  const float scale = scale_of(p);
  const int64_t total = (int64_t)p.M * p.N;
  with_act(p.act, [&](auto ac) {
    constexpr int ACT = decltype(ac)::value;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
      float s = 0.f;
#pragma unroll 8
      for (int sp = 0; sp < p.splits; ++sp) s += p.partial[sp * total + i];
      const int64_t row = i / p.N;
      finish_one<ACT>(p, s * scale, row, i - row * p.N);
    }
  });
}

// n (1 .. 7) elements at i, zeros behind them
__device__ __forceinline__ i32x4 load_some(const uint16_t* p, int64_t i, int n) {
  i32x4 w = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) w[e >> 1] |= (int)((uint32_t)p[i + e] << (16 * (e & 1)));
  return w;
}

// --------------------------------------------------------------- few rows
// Y of up to 16 rows at a time.  The weight is the traffic: each of its
// 16-byte chunks is loaded once per 16 rows, straight into registers.  A
// work-group of four waves owns 64 columns and a K range, 256 of K per step;
// a lane holds 8 k x 8 columns of W per step (eight loads; a wave's loads
// cover whole 128-byte lines in either layout of W) and for each row of X
// reads its eight k from LDS and does 32 two-term dot products.  The lanes'
// and waves' sums are joined at the end, the K ranges' by finish_splits.
typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));
__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2v, a), __builtin_bit_cast(bf16x2v, b), c, false);
}

template <int MT, bool WK>
__global__ void __launch_bounds__(256) linear_rows(const GemmParams p) {
  __shared__ __attribute__((aligned(16))) uint16_t xs[MT][kRowsStep];
  __shared__ float red[4][MT][kRowsTile];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n0 = blockIdx.x * kRowsTile, split = blockIdx.y, m0 = blockIdx.z * kRowsBlock;
  const int rows = min(MT, p.M - m0);
  const uint16_t* X = (const uint16_t*)p.A;
  const uint16_t* W = (const uint16_t*)p.B;
  const int steps = (p.K + kRowsStep - 1) / kRowsStep;
  const int s0 = split * p.ksteps_per_split, s1 = min(steps, s0 + p.ksteps_per_split);
  // this lane's 8 k (within the step) and its 8 columns: column cb + i
  const int k_lane = 64 * wave + 8 * (WK ? lane & 7 : lane >> 3);
  const int c_lane = 8 * (WK ? lane >> 3 : lane & 7);
  const int cb = WK ? n0 + c_lane : min(n0 + c_lane, p.N - 8);   // (a last chunk of fewer columns is loaded from N - 8)
  float acc[MT][8];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[m][i] = 0.f;

  auto load_w = [&](int s, i32x4 (&w)[8]) {
    const int k = s * kRowsStep + k_lane;
    if (s >= s1) return;
    if ((s + 1) * kRowsStep <= p.K) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t at = WK ? (int64_t)min(cb + i, p.N - 1) * p.ldb + k : (int64_t)(k + i) * p.ldb + cb;
        w[i] = __builtin_nontemporal_load((const i32x4_any*)(W + at));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        w[i] = i32x4{0, 0, 0, 0};
        if constexpr (WK) {
          const int n = min(8, p.K - k);
          const int64_t at = (int64_t)min(cb + i, p.N - 1) * p.ldb + k;
          if (n == 8) w[i] = __builtin_nontemporal_load((const i32x4_any*)(W + at));
          else if (n > 0) w[i] = load_some(W, at, n);
        } else {
          if (k + i < p.K) w[i] = __builtin_nontemporal_load((const i32x4_any*)(W + (int64_t)(k + i) * p.ldb + cb));
        }
      }
    }
  };
  auto load_x = [&](int s, uint16_t (&x)[MT]) {
    const int k = s * kRowsStep + (int)threadIdx.x;
#pragma unroll
    for (int m = 0; m < MT; ++m) x[m] = (s < s1 && k < p.K && m < rows) ? X[(int64_t)(m0 + m) * p.lda + k] : (uint16_t)0;
  };

  i32x4 w[2][8];
  uint16_t xr[MT];
  load_x(s0, xr);
  load_w(s0, w[0]);
  auto step = [&](int s, i32x4 (&cur)[8], i32x4 (&next)[8]) {
    __syncthreads();   // the previous step's reads of xs are done
#pragma unroll
    for (int m = 0; m < MT; ++m) xs[m][threadIdx.x] = xr[m];
    __syncthreads();
    load_x(s + 1, xr);
    load_w(s + 1, next);
    if constexpr (!WK) {
      // (row 2j, row 2j + 1) pairs of each column, in place: cur[2j] takes
      // columns 0-3, cur[2j + 1] columns 4-7
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const i32x4 a = cur[2 * j], b = cur[2 * j + 1];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const uint32_t lo = __builtin_amdgcn_perm((uint32_t)b[h], (uint32_t)a[h], 0x05040100u);
          const uint32_t hi = __builtin_amdgcn_perm((uint32_t)b[h], (uint32_t)a[h], 0x07060302u);
          if (h < 2) {
            cur[2 * j][2 * h] = (int)lo;
            cur[2 * j][2 * h + 1] = (int)hi;
          } else {
            cur[2 * j + 1][2 * h - 4] = (int)lo;
            cur[2 * j + 1][2 * h - 3] = (int)hi;
          }
        }
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const i32x4 x = *(const i32x4*)&xs[m][k_lane];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          acc[m][i] = dot2((uint32_t)(WK ? cur[i][j] : cur[2 * j + (i >> 2)][i & 3]), (uint32_t)x[j], acc[m][i]);
    }
  };
  for (int s = s0; s < s1; s += 2) {
    step(s, w[0], w[1]);
    if (s + 1 < s1) step(s + 1, w[1], w[0]);
  }
  // Sum over the eight lanes that share columns (they differ in three lane
  // bits), halving the columns a lane keeps at each exchange.
#pragma unroll
  for (int m = 0; m < MT; ++m) {
#pragma unroll
    for (int b = 0; b < 3; ++b) {
      const int bit = (WK ? 4 : 32) >> b, half = 4 >> b;
      const bool up = (lane & bit) != 0;
#pragma unroll
      for (int i = 0; i < half; ++i) {
        const float keep = up ? acc[m][i + half] : acc[m][i], give = up ? acc[m][i] : acc[m][i + half];
        acc[m][i] = keep + __shfl_xor(give, bit, 64);
      }
    }
    const int q = WK ? lane & 7 : lane >> 3;   // the column this lane kept
    const int col = cb + q;
    if (col >= n0 + c_lane) red[wave][m][col - n0] = acc[m][0];
  }
  __syncthreads();
  const float scale = scale_of(p);
  for (int i = threadIdx.x; i < rows * kRowsTile; i += 256) {
    const int m = i / kRowsTile, c = i - m * kRowsTile;
    if (n0 + c >= p.N) continue;
    const float s = ((red[0][m][c] + red[1][m][c]) + red[2][m][c]) + red[3][m][c];
    if (p.splits > 1) p.partial[((int64_t)split * p.M + m0 + m) * p.N + n0 + c] = s;
    else with_act(p.act, [&](auto ac) { finish_one<decltype(ac)::value>(p, s * scale, m0 + m, n0 + c); });
  }
}

// -------------------------------------------------------------- any shape
// 128 x 128 tile per work-group of four waves (64 x 64 each, 2 x 2 MFMAs of
// 32 x 32), K steps of 128 bytes (64 bf16, 32 fp32) through a double buffer in
// LDS; the next step's chunks are loaded into registers while the current one
// is multiplied.  Chunks of 16 bytes at any element address; what lies past an
// edge is zero.  bf16: the LDS tiles keep each operand's order in memory
// (K-major rows of 128 bytes, MN-major rows of 256), and MN-major fragments
// are transposed by the LDS read (ds_read_b64_tr_b16).  fp32
// (v_mfma_f32_32x32x2_f32): a lane reads four k of its row at once and feeds
// four MFMAs; A and B agree on the order of k, which the sum does not mind.
typedef __attribute__((address_space(3))) i16x4 lds_i16x4_t;

template <bool F32>
struct AnyTile {
  static constexpr int E = F32 ? 4 : 8;             // elements of a chunk
  static constexpr int KS = F32 ? 32 : 64;          // K of a step
  static constexpr int BYTES = kAnyTile * 128;      // LDS bytes of one operand tile
  static constexpr int MN_CHUNKS = kAnyTile / E;    // chunks of an MN-major row
};

// LDS byte address of chunk c of row r: rows of 128 bytes (K-major) or of
// MN_CHUNKS chunks (MN-major), swizzled so that the rows of one read differ
// in their banks.
template <bool F32, bool KM>
__device__ __forceinline__ uint32_t any_at(uint32_t r, uint32_t c) {
  if constexpr (KM) return r * 128u + ((c ^ ((r ^ (r >> 3)) & 7u)) << 4);
  else return r * (AnyTile<F32>::MN_CHUNKS * 16u) + ((F32 ? c : c ^ ((r & 3u) << 2)) << 4);
}

template <bool F32, bool KM>
__device__ __forceinline__ void any_load(const void* base, int64_t ld, int mn0, int mn_end, int k0, int k_end,
                                         i32x4 (&q)[4]) {
  using T = AnyTile<F32>;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int P = j * 256 + (int)threadIdx.x;
    int r, e, n;       // row in memory, first element of the chunk, elements of it inside
    bool in;
    if constexpr (KM) {
      r = mn0 + (P >> 3);
      e = k0 + (P & 7) * T::E;
      n = k_end - e;
      in = r < mn_end;
    } else {
      r = k0 + P / T::MN_CHUNKS;
      e = mn0 + (P % T::MN_CHUNKS) * T::E;
      n = mn_end - e;
      in = r < k_end;
    }
    q[j] = i32x4{0, 0, 0, 0};
    if (!in || n <= 0) continue;
    const int64_t at = (int64_t)r * ld + e;
    if (n >= T::E) {
      if constexpr (F32) q[j] = __builtin_bit_cast(i32x4, *(const f32x4_any*)((const float*)base + at));
      else q[j] = *(const i32x4_any*)((const uint16_t*)base + at);
    } else if constexpr (F32) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) q[j][i] = ((const int*)base)[at + i];
    } else {
      q[j] = load_some((const uint16_t*)base, at, n);
    }
  }
}
template <bool F32, bool KM>
__device__ __forceinline__ void any_store(char* tile, const i32x4 (&q)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t P = (uint32_t)(j * 256 + (int)threadIdx.x);
    const uint32_t r = KM ? P >> 3 : P / AnyTile<F32>::MN_CHUNKS, c = KM ? P & 7u : P % AnyTile<F32>::MN_CHUNKS;
    *(i32x4*)(tile + any_at<F32, KM>(r, c)) = q[j];
  }
}
// bf16: the 32 x 16 fragment of rows rb.., k 16 kk .. +15
template <bool KM>
__device__ __forceinline__ bf16x8 any_frag(const char* tile, int rb, int kk) {
  const int lane = threadIdx.x & 63;
  if constexpr (KM) {
    return *(const bf16x8*)(tile + any_at<false, true>((uint32_t)(rb + (lane & 31)), (uint32_t)(2 * kk + (lane >> 5))));
  } else {
    const int g = lane >> 4, j = lane & 15;
    const uint32_t mn = (uint32_t)(rb + 16 * (g & 1) + 4 * (j & 3));
    i16x4 h[2];
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const uint32_t k = (uint32_t)(16 * kk + 8 * (g >> 1) + 4 * hh + (j >> 2));
      h[hh] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_i16x4_t*)((lds_void*)(tile + any_at<false, false>(k, mn >> 3) + 2u * (mn & 7u))));
    }
    typedef short i16x8 __attribute__((ext_vector_type(8)));
    const i16x8 v = {h[0][0], h[0][1], h[0][2], h[0][3], h[1][0], h[1][1], h[1][2], h[1][3]};
    return __builtin_bit_cast(bf16x8, v);
  }
}
// fp32: row rb + lane % 32, k 8 q + 4 (lane / 32) + 0..3
template <bool KM>
__device__ __forceinline__ f32x4 any_quad(const char* tile, int rb, int q) {
  const int lane = threadIdx.x & 63;
  const uint32_t r = (uint32_t)(rb + (lane & 31)), h = (uint32_t)(lane >> 5);
  if constexpr (KM) {
    return *(const f32x4*)(tile + any_at<true, true>(r, 2u * (uint32_t)q + h));
  } else {
    f32x4 v;
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i)
      v[i] = *(const float*)(tile + any_at<true, false>(8u * (uint32_t)q + 4u * h + i, r >> 2) + 4u * (r & 3u));
    return v;
  }
}

template <bool F32, bool AK, bool BK>
__global__ void __launch_bounds__(256) linear_any(const GemmParams p, int nt) {
  using T = AnyTile<F32>;
  __shared__ __attribute__((aligned(1024))) char smem[2][2][T::BYTES];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int m0 = (int)(blockIdx.x / nt) * kAnyTile, n0 = (int)(blockIdx.x % nt) * kAnyTile, split = blockIdx.y;
  const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64;
  const int steps = (p.K + T::KS - 1) / T::KS;
  const int s0 = split * p.ksteps_per_split, s1 = min(steps, s0 + p.ksteps_per_split);
  f32x16 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
  i32x4 qa[4], qb[4];
  if (s0 < s1) {
    any_load<F32, AK>(p.A, p.lda, m0, p.M, s0 * T::KS, p.K, qa);
    any_load<F32, BK>(p.B, p.ldb, n0, p.N, s0 * T::KS, p.K, qb);
  }
  for (int s = s0; s < s1; ++s) {
    char* ta = smem[(s - s0) & 1][0];
    char* tb = smem[(s - s0) & 1][1];
    any_store<F32, AK>(ta, qa);
    any_store<F32, BK>(tb, qb);
    // one barrier a step: a wave that stores into this buffer again, two
    // steps on, has passed the next step's barrier, before which every wave
    // finished reading it
    __syncthreads();
    if (s + 1 < s1) {
      any_load<F32, AK>(p.A, p.lda, m0, p.M, (s + 1) * T::KS, p.K, qa);
      any_load<F32, BK>(p.B, p.ldb, n0, p.N, (s + 1) * T::KS, p.K, qb);
    }
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      if constexpr (F32) {
        f32x4 a[2], b[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          a[i] = any_quad<AK>(ta, wm + 32 * i, kk);
          b[i] = any_quad<BK>(tb, wn + 32 * i, kk);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(b[j][e], a[i][e], acc[i][j], 0, 0, 0);
      } else {
        bf16x8 a[2], b[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          a[i] = any_frag<AK>(ta, wm + 32 * i, kk);
          b[i] = any_frag<BK>(tb, wn + 32 * i, kk);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b[j], a[i], acc[i][j], 0, 0, 0);
      }
    }
  }
  // lane l: row l % 32, columns 8 q + 4 (l / 32) + 0..3 of each 32 x 32 block
  const float scale = scale_of(p);
  with_act(p.act, [&](auto ac) {
    constexpr int ACT = decltype(ac)::value;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = m0 + wm + 32 * i + (lane & 31);
      if (row >= p.M) continue;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int col = n0 + wn + 32 * j + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
          if (col >= p.N) continue;
          if (p.splits > 1) p.partial[((int64_t)split * p.M + row) * p.N + col] = acc[i][j][e];
          else finish_one<ACT>(p, acc[i][j][e] * scale, row, col);
        }
    }
  });
}

// ---------------------------------------------------- backward, elementwise
// dZ = dY act'(Z) and the column sums of the unrounded dZ: a work-group takes
// 512 columns (64 chunks of eight) of a band of rows, four rows at a time;
// the four rows' sums are joined in LDS, the bands' by column_sums.  Bound by
// reading dY and Z and writing dZ once.
template <bool F32>
__global__ void __launch_bounds__(256) dact_columns(const void* dY, int64_t lddy, const void* Z, int64_t ldz, int act,
                                                    int64_t M, int64_t N, int64_t band, void* dZ, float* part) {
  __shared__ float red[4][512];
  const int chunk = threadIdx.x & 63, sub = threadIdx.x >> 6;
  const int64_t c0 = (int64_t)blockIdx.x * 512 + 8 * chunk;
  const int n = (int)std::min<int64_t>(8, N - c0);       // columns of the chunk inside the matrix
  const int64_t r1 = std::min<int64_t>(M, (blockIdx.y + 1) * band);
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  with_act(act, [&](auto ac) {
    constexpr int ACT = decltype(ac)::value;
    for (int64_t r = blockIdx.y * band + sub; r < r1; r += 4) {
      if (n == 8) {
        float g[8];
        const Raw8<F32> gy = load8<F32>(dY, r * lddy + c0);
        if (Z) {
          float z[8];
          const Raw8<F32> zz = load8<F32>(Z, r * ldz + c0);
          widen8<F32>(gy, g);
          widen8<F32>(zz, z);
#pragma unroll
          for (int e = 0; e < 8; ++e) g[e] *= act_grad_c<ACT>(z[e]);
          store8<F32>(dZ, r * N + c0, g, 0);
        } else {
          widen8<F32>(gy, g);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += g[e];
      } else {
#pragma unroll
        for (int e = 0; e < 7; ++e) {
          if (e >= n) continue;
          float g = ld_f(dY, F32, r * lddy + c0 + e);
          if (Z) {
            g *= act_grad_c<ACT>(ld_f(Z, F32, r * ldz + c0 + e));
            st_f(dZ, F32, r * N + c0 + e, g);
          }
          sum[e] += g;
        }
      }
    }
  });
  if (!part) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) red[sub][8 * chunk + e] = sum[e];
  __syncthreads();
  for (int k = threadIdx.x; k < 512; k += 256) {
    const int64_t c = (int64_t)blockIdx.x * 512 + k;
    if (c < N) part[blockIdx.y * N + c] = ((red[0][k] + red[1][k]) + red[2][k]) + red[3][k];
  }
}

hipError_t launch_finish(const GemmParams& p, hipStream_t s) {
  if (p.splits <= 1) return hipSuccess;
  finish_splits<<<(int)std::min<int64_t>(((int64_t)p.M * p.N + 255) / 256, 8192), 256, 0, s>>>(p);
  return hipGetLastError();
}

template <bool WK>
hipError_t rows_of(const GemmParams& p, hipStream_t s) {
  const dim3 grid((p.N + kRowsTile - 1) / kRowsTile, p.splits, (p.M + kRowsBlock - 1) / kRowsBlock);
  if (p.M <= 1) linear_rows<1, WK><<<grid, 256, 0, s>>>(p);
  else if (p.M <= 2) linear_rows<2, WK><<<grid, 256, 0, s>>>(p);
  else if (p.M <= 4) linear_rows<4, WK><<<grid, 256, 0, s>>>(p);
  else if (p.M <= 8) linear_rows<8, WK><<<grid, 256, 0, s>>>(p);
  else linear_rows<16, WK><<<grid, 256, 0, s>>>(p);
  return hipGetLastError();
}

template <bool F32>
hipError_t any_of(const GemmParams& p, bool ta, bool tb, hipStream_t s) {
  const int nt = (p.N + kAnyTile - 1) / kAnyTile;
  const dim3 grid((unsigned)(((p.M + kAnyTile - 1) / kAnyTile) * nt), p.splits);
  if (!ta && tb) linear_any<F32, true, true><<<grid, 256, 0, s>>>(p, nt);
  else if (!ta) linear_any<F32, true, false><<<grid, 256, 0, s>>>(p, nt);
  else if (tb) linear_any<F32, false, true><<<grid, 256, 0, s>>>(p, nt);
  else linear_any<F32, false, false><<<grid, 256, 0, s>>>(p, nt);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_rows(const GemmParams& p, bool w_kmajor, hipStream_t s) {
  hipError_t e = w_kmajor ? rows_of<true>(p, s) : rows_of<false>(p, s);
  return e == hipSuccess ? launch_finish(p, s) : e;
}

hipError_t launch_linear_any(const GemmParams& p, bool trans_a, bool trans_b, hipStream_t s) {
  hipError_t e = p.a_dt == 0 ? any_of<true>(p, trans_a, trans_b, s) : any_of<false>(p, trans_a, trans_b, s);
  return e == hipSuccess ? launch_finish(p, s) : e;
}

// Bands of rows of dact_columns: about 2048 work-groups, at least eight rows each.
int dact_bands(int64_t M, int64_t N) {
  const int64_t strips = std::max<int64_t>(1, (N + 511) / 512);
  return (int)std::max<int64_t>(1, std::min<int64_t>((2048 + strips - 1) / strips, (M + 7) / 8));
}

hipError_t launch_dact_columns(const void* dY, int64_t lddy, const void* Z, int64_t ldz, bool f32, int act, int64_t M,
                               int64_t N, void* dZ, float* part, int bands, hipStream_t s) {
  const int64_t band = (M + bands - 1) / bands;
  const dim3 grid((unsigned)((N + 511) / 512), (unsigned)bands);
  if (f32) dact_columns<true><<<grid, 256, 0, s>>>(dY, lddy, Z, ldz, act, M, N, band, dZ, part);
  else dact_columns<false><<<grid, 256, 0, s>>>(dY, lddy, Z, ldz, act, M, N, band, dZ, part);
  return hipGetLastError();
}

}  // namespace tpm
