// Kernels and launchers of the persistent MFMA GEMM (the tile program is
// gemm_tile.hpp): one GEMM, two paired GEMMs, and the finalisation passes of
// split K ranges.
#include "gemm_tile.hpp"

namespace tpm {

namespace {

template <bool FP8, bool AK, bool BKM, int NW, bool GATED = false, bool MX = false, int F8F = 0>
__global__ void __launch_bounds__(64 * NW, 1) gemm_kernel(const GemmParams p) {
  __shared__ __attribute__((aligned(1024))) char smem[Layout<NW>::SMEM];
  // Chunk-gated GEMM: invalidate this XCD's caches once, before any
  // operand is loaded.  A row of chunk c is only ever loaded after
  // ready[c] has been seen set, and the producer publishes the data before
  // the flag (release), so no cache can hold a stale copy of it afterwards:
  // the per-chunk wait needs no further invalidation (which would throw away
  // every tile's cached operands on each chunk arrival).
  if (p.ready) __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  for (int u = blockIdx.x; u < p.units; u += gridDim.x)
    run_unit<FP8, AK, BKM, NW, GATED, MX, F8F>(p, map_unit(p, u), smem);
}

// Two independent bf16 GEMMs in one persistent launch (the weight and the
// input gradient of a linear layer, which read the same dY): each XCD
// (work-groups congruent mod 8) owns a contiguous eighth of each GEMM's
// logical units, those of GEMM FIRST listed first, and its work-groups take
// units from that list through a per-XCD ticket counter (queue[x], zero at
// launch), so that the longer units start first and the shorter ones fill
// in behind them.  Every unit is computed whole by the work-group that
// takes it, so results do not depend on which one does.  A work-group
// leaves the first GEMM's loop for good once its ticket passes that GEMM's
// units, so the two loops (and their loop-invariant registers) never
// overlap.
template <int NW, bool AK0, bool BK0, bool AK1, bool BK1, int FIRST>
__global__ void __launch_bounds__(64 * NW, 1) gemm_pair_kernel(const GemmParams p0, const GemmParams p1,
                                                              uint32_t* queue) {
  // the ticket word is a control word of the ring (a __shared__ variable of
  // its own makes the compiler wait for all LDS DMA before every LDS read of
  // the K loop); tickets are taken between work units, with no load in flight
  __shared__ __attribute__((aligned(1024))) char smem[Layout<NW>::SMEM];
  volatile int* ticket_word = reinterpret_cast<volatile int*>(smem + CTRL_TICKET);
  const int x = blockIdx.x & 7;
  const int n0 = p0.units, n1 = p1.units;
  const int b0 = (int)((int64_t)x * n0 / 8), c0 = (int)((int64_t)(x + 1) * n0 / 8) - b0;
  const int b1 = (int)((int64_t)x * n1 / 8), c1 = (int)((int64_t)(x + 1) * n1 / 8) - b1;
  // (every thread reads a ticket before thread 0 can take the next one:
  // the unit's body passes several work-group barriers)
  auto take = [&]() {
    if (threadIdx.x == 0) *ticket_word = (int)atomicAdd(queue + x, 1u);
    __syncthreads();
    return *ticket_word;
  };
  int i = take();
  if constexpr (FIRST == 0) {
    for (; i < c0; i = take()) run_unit<false, AK0, BK0, NW, false, false, 0, true>(p0, logical_unit(p0, b0 + i), smem);
    for (; i < c0 + c1; i = take()) run_unit<false, AK1, BK1, NW, false, false, 0, false>(p1, logical_unit(p1, b1 + i - c0), smem);
  } else {
    for (; i < c1; i = take()) run_unit<false, AK1, BK1, NW, false, false, 0, false>(p1, logical_unit(p1, b1 + i), smem);
    for (; i < c0 + c1; i = take()) run_unit<false, AK0, BK0, NW, false, false, 0, true>(p0, logical_unit(p0, b0 + i - c1), smem);
  }
}


// The epilogue of 8 summed values in a finalisation pass: the fp8 output of
// delayed scaling as the GEMM kernel writes it (pre-activation saved as
// bf16, codes e4m3(act(v) * fp32(1 / s)), amax of act(v)), else epi_oct.
template <int ACT>
__device__ __forceinline__ void finalize_oct(const GemmParams& p, float (&v)[8], int row, int col, float& lmax) {
  if (p.y_q_scale) {
    const float inv = 1.0f / *p.y_q_scale;
    if (p.aux) store_oct(p.aux, p.ldaux, false, row, col, v);
    float q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float h = act_fwd_c<ACT>(v[e]);
      lmax = fmaxf(lmax, fabsf(h));
      q[e] = h * inv;
    }
    *(uint2*)((uint8_t*)p.Y + (int64_t)row * p.ldy + col) =
        make_uint2(fp8x4<false>(q[0], q[1], q[2], q[3]), fp8x4<false>(q[4], q[5], q[6], q[7]));
    return;
  }
  epi_oct<ACT>(p, v, row, col, lmax);
}

// Split-K finalisation: Y = epilogue(scale * sum_{s=0}^{S-1} partial_s),
// summed in ascending s (deterministic), 8 consecutive columns per lane.
__global__ void __launch_bounds__(256) splitk_finalize(const GemmParams p) {
  float scale = 1.f;
  if (p.a_scale) scale *= *p.a_scale;
  if (p.b_scale) scale *= *p.b_scale;
  const int64_t n8 = p.N / 8;
  const int64_t total = (int64_t)p.M * n8;
  const int64_t plane = (int64_t)p.M * p.N;
  float lmax = 0.f;
  with_act(p.act, [&](auto ac) {
  constexpr int ACT = decltype(ac)::value;
  for (int64_t w = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; w < total; w += (int64_t)gridDim.x * blockDim.x) {
    const int row = (int)(w / n8);
    const int col = (int)(w - (int64_t)row * n8) * 8;
    const float* src = p.partial + (int64_t)row * p.N + col;
    f32x4 a0 = __builtin_nontemporal_load((const f32x4*)src);
    f32x4 a1 = __builtin_nontemporal_load((const f32x4*)src + 1);
    for (int sp = 1; sp < p.splits; ++sp) {
      a0 += __builtin_nontemporal_load((const f32x4*)(src + sp * plane));
      a1 += __builtin_nontemporal_load((const f32x4*)(src + sp * plane) + 1);
    }
    float v[8] = {a0[0] * scale, a0[1] * scale, a0[2] * scale, a0[3] * scale,
                  a1[0] * scale, a1[1] * scale, a1[2] * scale, a1[3] * scale};
    finalize_oct<ACT>(p, v, row, col, lmax);
  }
  });
  if (p.amax) block_amax(p.amax, lmax);
}

// Tail finalisation: each tail tile's pieces summed in ascending piece order
// (deterministic), scaled, then the epilogue; one work-group per 64 rows of a
// tail tile, 8 rows at a time, 8 consecutive columns per lane.
constexpr int kTailRows = 64;
__global__ void __launch_bounds__(256) tail_finalize(const GemmParams p) {
  float scale = 1.f;
  if (p.a_scale) scale *= *p.a_scale;
  if (p.b_scale) scale *= *p.b_scale;
  constexpr int BLOCKS_PER_TILE = BM / kTailRows;
  const int t = blockIdx.x / BLOCKS_PER_TILE;
  const int r0 = (blockIdx.x - t * BLOCKS_PER_TILE) * kTailRows + (threadIdx.x >> 5);
  const int c = (threadIdx.x & 31) * 8;
  const Tile tl = tail_tile(p, t);
  const int col = tl.n0 + c;
  const int64_t piece = (int64_t)p.tail_tiles * BM * BN;
  float lmax = 0.f;
  with_act(p.act, [&](auto ac) {
    constexpr int ACT = decltype(ac)::value;
#pragma unroll 2
    for (int i = 0; i < kTailRows / 8; ++i) {
      const int r = r0 + 8 * i;
      const int row = tl.m0 + r;
      if (row < tl.m_end && col < p.N) {
        const float* src = p.partial + ((int64_t)t * BM + r) * BN + c;
        f32x4 a0 = __builtin_nontemporal_load((const f32x4*)src);
        f32x4 a1 = __builtin_nontemporal_load((const f32x4*)src + 1);
        for (int sp = 1; sp < p.tail_pieces; ++sp) {
          a0 += __builtin_nontemporal_load((const f32x4*)(src + sp * piece));
          a1 += __builtin_nontemporal_load((const f32x4*)(src + sp * piece) + 1);
        }
        float v[8] = {a0[0] * scale, a0[1] * scale, a0[2] * scale, a0[3] * scale,
                      a1[0] * scale, a1[1] * scale, a1[2] * scale, a1[3] * scale};
        finalize_oct<ACT>(p, v, row, col, lmax);
      }
    }
  });
  if (p.amax) block_amax(p.amax, lmax);
}

}  // namespace

static hipError_t finalize_if_split(const GemmParams& p, hipStream_t s) {
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (p.splits > 1) {
    int64_t work = (int64_t)p.M * (p.N / 8);
    int64_t blocks = (work + 255) / 256;
    if (blocks > 4096) blocks = 4096;
    splitk_finalize<<<(int)blocks, 256, 0, s>>>(p);
  } else if (p.tail_pieces > 1) {
    tail_finalize<<<p.tail_tiles * (BM / kTailRows), 256, 0, s>>>(p);
  } else {
    return hipSuccess;
  }
  return hipGetLastError();
}

// bf16: 8 waves (two per SIMD, 128 x 64 each).  fp8: 4 waves (128 x 128
// each): two fp8 fragment sets of a 128 x 64 wave do not fit next to its
// accumulators in the registers of one of two waves per SIMD.
#ifndef TPM_GEMM_WAVES_BF16
#define TPM_GEMM_WAVES_BF16 8
#endif
#ifndef TPM_GEMM_WAVES_FP8
#define TPM_GEMM_WAVES_FP8 4
#endif
constexpr int kWaves = TPM_GEMM_WAVES_BF16, kWaves8 = TPM_GEMM_WAVES_FP8;
constexpr int kThreads = 64 * kWaves, kThreads8 = 64 * kWaves8;

hipError_t launch_gemm_bf16(const GemmParams& p, bool a_kmajor, bool b_kmajor, int grid, hipStream_t s) {
  if (p.epi == EPI_GATED) {
    if (!a_kmajor || b_kmajor || p.splits != 1) return hipErrorInvalidValue;  // rejected on the host first
    gemm_kernel<false, true, false, 8, true><<<grid, 512, 0, s>>>(p);
    return hipGetLastError();
  }
  if (a_kmajor && !b_kmajor) gemm_kernel<false, true, false, kWaves><<<grid, kThreads, 0, s>>>(p);
  else if (a_kmajor && b_kmajor) gemm_kernel<false, true, true, kWaves><<<grid, kThreads, 0, s>>>(p);
  else if (!a_kmajor && !b_kmajor) gemm_kernel<false, false, false, kWaves><<<grid, kThreads, 0, s>>>(p);
  else gemm_kernel<false, false, true, kWaves><<<grid, kThreads, 0, s>>>(p);
  return finalize_if_split(p, s);
}

hipError_t launch_gemm_pair_bf16(const GemmParams& p0, bool a0_kmajor, bool b0_kmajor, const GemmParams& p1,
                                 bool a1_kmajor, bool b1_kmajor, int first, uint32_t* queue, int grid, hipStream_t s) {
  // instantiated for a linear layer's backward: dW = X^T dY (both operands
  // MN-major) and dX = dY W^T (both K-major)
  if (a0_kmajor || b0_kmajor || !a1_kmajor || !b1_kmajor) return hipErrorInvalidValue;  // rejected on the host first
  if (first == 0) gemm_pair_kernel<kWaves, false, false, true, true, 0><<<grid, kThreads, 0, s>>>(p0, p1, queue);
  else gemm_pair_kernel<kWaves, false, false, true, true, 1><<<grid, kThreads, 0, s>>>(p0, p1, queue);
  hipError_t e = finalize_if_split(p0, s);
  if (e != hipSuccess) return e;
  return finalize_if_split(p1, s);
}

hipError_t launch_gemm_fp8(const GemmParams& p, bool a_kmajor, bool b_kmajor, int grid, hipStream_t s) {
  if (!a_kmajor || !b_kmajor) return hipErrorInvalidValue;  // rejected on the host first
  if (p.a_mx) gemm_kernel<true, true, true, kWaves8, false, true><<<grid, kThreads8, 0, s>>>(p);
  else if (p.f8fmt == 1) gemm_kernel<true, true, true, kWaves8, false, false, 1><<<grid, kThreads8, 0, s>>>(p);
  else if (p.f8fmt == 2) gemm_kernel<true, true, true, kWaves8, false, false, 2><<<grid, kThreads8, 0, s>>>(p);
  else if (p.f8fmt == 0) gemm_kernel<true, true, true, kWaves8><<<grid, kThreads8, 0, s>>>(p);
  else return hipErrorInvalidValue;  // both operands e5m2: rejected on the host first
  return finalize_if_split(p, s);
}

}  // namespace tpm
