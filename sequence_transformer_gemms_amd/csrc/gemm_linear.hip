// Forward of one linear layer on the matrix cores, with bias, activation and
// residual in the epilogue: Y = act(X W + bias) + residual.  The tile program
// of gemm_tile.hpp with the epilogue lin_oct, and the finalisation passes of
// split K ranges.
#include "gemm_tile.hpp"

namespace tpm {

namespace {

template <bool FP8, bool BKM, int NW>
__global__ void __launch_bounds__(64 * NW, 1) linear_kernel(const GemmParams p) {
  __shared__ __attribute__((aligned(1024))) char smem[Layout<NW>::SMEM];
  // chunk-gated: this XCD's caches are invalidated once, before any operand
  // is loaded; a chunk's rows are only loaded after its flag is seen
  if (p.ready) __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  for (int u = blockIdx.x; u < p.units; u += gridDim.x)
    run_unit<FP8, true, BKM, NW, false, false, 0, true, true>(p, map_unit(p, u), smem);
}

__device__ __forceinline__ float scale_of(const GemmParams& p) {
  float s = 1.f;
  if (p.a_scale) s *= *p.a_scale;
  if (p.b_scale) s *= *p.b_scale;
  return s;
}

// Eight summed columns of a split tile: scale, then the epilogue.
template <int ACT>
__device__ __forceinline__ void finish_oct(const GemmParams& p, const f32x4& a0, const f32x4& a1, float scale, int row,
                                           int col) {
  float bias[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (p.bias) load_oct(p.bias, 0, p.bias_f32, 0, col, bias);
  float v[8] = {a0[0] * scale, a0[1] * scale, a0[2] * scale, a0[3] * scale,
                a1[0] * scale, a1[1] * scale, a1[2] * scale, a1[3] * scale};
  lin_oct<ACT, LK_ANY>(p, v, bias, row, col);
}

// K-range partial sums [splits, M, N] added in ascending order, eight columns a lane.
__global__ void __launch_bounds__(256) linear_splitk_finish(const GemmParams p) {
  const float scale = scale_of(p);
  const int64_t n8 = p.N / 8, total = (int64_t)p.M * n8, plane = (int64_t)p.M * p.N;
  with_act(p.act, [&](auto ac) {
    constexpr int ACT = decltype(ac)::value;
    for (int64_t w = (int64_t)blockIdx.x * 256 + threadIdx.x; w < total; w += (int64_t)gridDim.x * 256) {
      const int row = (int)(w / n8), col = (int)(w - (int64_t)row * n8) * 8;
      const float* src = p.partial + (int64_t)row * p.N + col;
      f32x4 a0 = __builtin_nontemporal_load((const f32x4*)src), a1 = __builtin_nontemporal_load((const f32x4*)src + 1);
      for (int sp = 1; sp < p.splits; ++sp) {
        a0 += __builtin_nontemporal_load((const f32x4*)(src + sp * plane));
        a1 += __builtin_nontemporal_load((const f32x4*)(src + sp * plane) + 1);
      }
      finish_oct<ACT>(p, a0, a1, scale, row, col);
    }
  });
}

// The tail tiles' pieces [piece][tile][256][256], one work-group per 64 rows.
__global__ void __launch_bounds__(256) linear_tail_finish(const GemmParams p) {
  const float scale = scale_of(p);
  const int t = blockIdx.x >> 2;
  const Tile tl = tail_tile(p, t);
  const int r0 = (blockIdx.x & 3) * 64 + (threadIdx.x >> 5), c = (threadIdx.x & 31) * 8;
  const int col = tl.n0 + c;
  const int64_t piece = (int64_t)p.tail_tiles * BM * BN;
  with_act(p.act, [&](auto ac) {
    constexpr int ACT = decltype(ac)::value;
#pragma unroll 2
    for (int i = 0; i < 8; ++i) {
      const int r = r0 + 8 * i, row = tl.m0 + r;
      if (row >= tl.m_end || col >= p.N) continue;
      const float* src = p.partial + ((int64_t)t * BM + r) * BN + c;
      f32x4 a0 = __builtin_nontemporal_load((const f32x4*)src), a1 = __builtin_nontemporal_load((const f32x4*)src + 1);
      for (int sp = 1; sp < p.tail_pieces; ++sp) {
        a0 += __builtin_nontemporal_load((const f32x4*)(src + sp * piece));
        a1 += __builtin_nontemporal_load((const f32x4*)(src + sp * piece) + 1);
      }
      finish_oct<ACT>(p, a0, a1, scale, row, col);
    }
  });
}

}  // namespace

hipError_t launch_linear(const GemmParams& p, bool fp8, bool w_kmajor, int grid, hipStream_t s) {
  if (fp8 && !w_kmajor) return hipErrorInvalidValue;  // rejected on the host first
  if (fp8) linear_kernel<true, true, 4><<<grid, 256, 0, s>>>(p);
  else if (w_kmajor) linear_kernel<false, true, 8><<<grid, 512, 0, s>>>(p);
  else linear_kernel<false, false, 8><<<grid, 512, 0, s>>>(p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (p.splits > 1)
    linear_splitk_finish<<<(int)std::min<int64_t>(((int64_t)p.M * (p.N / 8) + 255) / 256, 4096), 256, 0, s>>>(p);
  else if (p.tail_pieces > 1)
    linear_tail_finish<<<p.tail_tiles * 4, 256, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace tpm
