// The linear layer's kernel beside the 256 x 256 tile program, for few rows (a
// decoding step), small products, shapes and alignments that are no whole
// 16-byte chunks, and fp32; and the elementwise part of its backward.
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

// Four consecutive elements at i, of which n (1 .. 4) are inside the row.
__device__ __forceinline__ f32x4 load4(const void* p, bool f32, int64_t i, int n) {
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  if (n == 4 && f32) return *(const f32x4_any*)((const float*)p + i);
  if (n == 4) {
    const i32x2 w = *(const i32x2_any*)((const uint16_t*)p + i);
    return f32x4{__uint_as_float((uint32_t)w[0] << 16), __uint_as_float((uint32_t)w[0] & 0xFFFF0000u),
                 __uint_as_float((uint32_t)w[1] << 16), __uint_as_float((uint32_t)w[1] & 0xFFFF0000u)};
  }
#pragma unroll
  for (int e = 0; e < 3; ++e)
    if (e < n) v[e] = ld_f(p, f32, i + e);
  return v;
}
__device__ __forceinline__ void store4(void* p, bool f32, int64_t i, int n, const f32x4& v) {
  if (n == 4 && f32) {
    *(f32x4_any*)((float*)p + i) = v;
  } else if (n == 4) {
    *(i32x2_any*)((uint16_t*)p + i) = i32x2{(int)pack_bf16x2(v[0], v[1]), (int)pack_bf16x2(v[2], v[3])};
  } else {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (e < n) st_f(p, f32, i + e, v[e]);
  }
}

// Epilogue of four columns: z = v + bias kept in aux, Y = act(z) + residual r.
__device__ __forceinline__ f32x4 bias4(const GemmParams& p, int64_t col) {
  return p.bias ? load4(p.bias, p.bias_f32, col, (int)std::min<int64_t>(4, p.N - col)) : f32x4{0.f, 0.f, 0.f, 0.f};
}
__device__ __forceinline__ f32x4 resid4(const GemmParams& p, int64_t row, int64_t col) {
  return p.resid ? load4(p.resid, p.y_f32, row * p.ldr + col, (int)std::min<int64_t>(4, p.N - col))
                 : f32x4{0.f, 0.f, 0.f, 0.f};
}
template <int ACT>
__device__ __forceinline__ void finish4(const GemmParams& p, f32x4 v, const f32x4& r, int64_t row, int64_t col) {
  const int n = (int)std::min<int64_t>(4, p.N - col);
  if (p.aux) store4(p.aux, p.aux_f32, row * p.ldaux + col, n, v);
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = act_fwd_c<ACT>(v[e]);
  store4(p.Y, p.y_f32, row * p.ldy + col, n, v + r);
}

// Sums of the K ranges, in ascending order, then the epilogue.  The partial sums
// are laid out by tile, part[range][tile][MB][128]; only the rows inside the
// matrix are written and read; 32 threads take the 128 columns of a row.  Up to
// eight ranges: a work-group takes eight rows.  More (a decoding step has tens):
// it takes one row, and eight times 32 threads add every eighth range, few
// dependent loads each, whose sums are added in order.
constexpr int kFinishRows = 8;
template <int MB>
__device__ __forceinline__ void finish_unit(const GemmParams& p, int u, f32x4 (&red)[8][32]) {
  const int q = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const bool many = p.splits > kFinishRows;
  const int strip = u % p.nt, row = many ? u / p.nt : u / p.nt * kFinishRows + slice, col = strip * kAnyTile + 4 * q;
  const int tile = strip * p.mt_per_group + row / MB;
  const f32x4* src = (const f32x4*)(p.partial + ((int64_t)tile * MB + row % MB) * kAnyTile) + q;
  const int64_t range = (int64_t)p.total_tiles * MB * kAnyTile / 4;
  const float scale = scale_of(p);
  f32x4 s = {0.f, 0.f, 0.f, 0.f}, bias = s, r = s;
  if (many) {
#pragma unroll 4
    for (int i = slice; i < p.splits; i += 8) s += src[i * range];
    red[slice][q] = s;
    __syncthreads();
    if (slice != 0 || col >= p.N) return;
    bias = bias4(p, col);
    r = resid4(p, row, col);
#pragma unroll
    for (int i = 1; i < 8; ++i) s += red[i][q];
  } else {
    if (row >= p.M || col >= p.N) return;
    bias = bias4(p, col);
    r = resid4(p, row, col);
#pragma unroll
    for (int i = 0; i < kFinishRows; ++i)
      if (i < p.splits) s += src[i * range];
  }
  s = s * scale + bias;
  with_act(p.act, [&](auto ac) { finish4<decltype(ac)::value>(p, s, r, row, col); });
}
template <int MB>
__global__ void __launch_bounds__(256) finish_ranges(const GemmParams p) {
  __shared__ f32x4 red[8][32];
  finish_unit<MB>(p, blockIdx.x, red);
}
// of two products: the first n0 work-groups are p0's
template <int MB>
__global__ void __launch_bounds__(256) finish_ranges_pair(const GemmParams p0, const GemmParams p1, int n0) {
  __shared__ f32x4 red[8][32];
  if ((int)blockIdx.x < n0) finish_unit<MB>(p0, blockIdx.x, red);
  else finish_unit<MB>(p1, (int)blockIdx.x - n0, red);
}

// -------------------------------------------------------------- any shape
// MB x 128 tile (MB = 128, 64 or 32 rows) per work-group of four waves, MFMAs
// of 32 x 32, K steps of 128 bytes (64 bf16, 32 fp32, 128 e4m3) through a double buffer
// in LDS; the next step's chunks are loaded into registers while the current
// one is multiplied.  Chunks of 16 bytes at any element address; what lies
// past an edge is zero.  bf16: the LDS tiles keep each operand's order in memory
// (K-major rows of 128 bytes, MN-major rows of 256), and MN-major fragments
// are transposed by the LDS read (ds_read_b64_tr_b16).  fp32
// (v_mfma_f32_32x32x2_f32): a lane reads four k of its row at once and feeds
// four MFMAs; A and B agree on the order of k, which the sum does not mind.
// e4m3 (v_mfma_f32_32x32x64_f8f6f4, both operands K-major) likewise.
typedef __attribute__((address_space(3))) i16x4 lds_i16x4_t;
typedef i32x4 i32x4_bytes __attribute__((aligned(1)));

enum { TY_F32 = 0, TY_BF16 = 1, TY_E4M3 = 2 };      // (the library's dtype codes)
template <int TY>
struct AnyTile {
  static constexpr int ESZ = TY == TY_F32 ? 4 : TY == TY_BF16 ? 2 : 1;
  static constexpr int E = 16 / ESZ;                // elements of a chunk
  static constexpr int KS = 128 / ESZ;              // K of a step
};

// LDS byte address of chunk c of row r of an operand tile of ROWS rows: rows of
// 128 bytes (K-major) or of ROWS / E chunks (MN-major), swizzled so that the
// rows of one read differ in their banks.
template <int TY, bool KM, int ROWS>
__device__ __forceinline__ uint32_t any_at(uint32_t r, uint32_t c) {
  constexpr uint32_t RC = ROWS / AnyTile<TY>::E;
  if constexpr (KM) return r * 128u + ((c ^ ((r ^ (r >> 3)) & 7u)) << 4);
  else return r * (RC * 16u) + ((TY == TY_F32 ? c : c ^ (((r & 3u) << 2) & (RC - 1u))) << 4);
}

// One thread's chunks of an operand tile of ROWS rows: ROWS / 32 of them, all
// in the same columns of memory, chunk j a uniform distance behind the first.
// K-major: operand rows line + 32 j, k from `first`; MN-major: k from line + j *
// LINES, operand rows from `first`.  A chunk that crosses the row's end is loaded
// so that it ends there and shifted into place when it is stored to LDS; rows
// narrower than a chunk are gathered element by element.
template <int TY, bool KM, int ROWS>
struct AnyOperand {
  static constexpr int E = AnyTile<TY>::E, KS = AnyTile<TY>::KS, ESZ = AnyTile<TY>::ESZ, N = ROWS / 32;
  static constexpr int RC = KM ? 8 : ROWS / E;             // chunks of a tile's memory row
  static constexpr int LINES = 256 / RC;                   // memory rows between chunks
  const char* p;       // chunk 0 of step 0
  int64_t ld;          // bytes
  int line, first;     // of step 0
  int lines, width;    // memory rows, and elements of a row
  __device__ __forceinline__ AnyOperand(const void* base, int64_t ld_, int mn0, int mn_end, int K) {
    line = (KM ? mn0 : 0) + (int)threadIdx.x / RC;
    first = (KM ? 0 : mn0) + (int)threadIdx.x % RC * E;
    lines = KM ? mn_end : K;
    width = KM ? K : mn_end;
    ld = ld_ * ESZ;
    p = (const char*)base + line * ld + (int64_t)first * ESZ;
  }
  // elements of step s's chunks inside the row (more than E: all of them)
  __device__ __forceinline__ int inside(int s) const { return width - first - (KM ? s * KS : 0); }
  __device__ __forceinline__ void load(int s, i32x4 (&q)[N]) const {
    const int l = line + (KM ? 0 : s * KS), n = inside(s);
    const char* at = p + (KM ? (int64_t)s * 128 : (int64_t)s * KS * ld) - (n < E ? (E - n) * ESZ : 0);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      q[j] = i32x4{0, 0, 0, 0};
      if (n <= 0 || l + j * LINES >= lines) continue;
      if (width >= E) {
        q[j] = *(const i32x4_bytes*)(at + j * LINES * ld);
      } else {   // (first = 0 here: the row is elements 0 .. n - 1)
        uint64_t w[2] = {0, 0};
#pragma unroll 1
        for (int e = 0; e < n; ++e) {
          const char* x = at + (E - n + e) * ESZ + j * LINES * ld;
          const uint64_t v = ESZ == 4 ? *(const uint32_t*)x : ESZ == 2 ? *(const uint16_t*)x : *(const uint8_t*)x;
          w[e * ESZ >> 3] |= v << (e * ESZ * 8 & 63);
        }
        q[j] = i32x4{(int)w[0], (int)(w[0] >> 32), (int)w[1], (int)(w[1] >> 32)};
      }
    }
  }
  __device__ __forceinline__ void store(int s, char* tile, i32x4 (&q)[N]) const {
    const int n = inside(s);
    if (__builtin_expect(n < E && n > 0 && width >= E, 0)) {
      int bits = (E - n) * ESZ * 8;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        uint64_t lo = (uint64_t)(uint32_t)q[j][0] | (uint64_t)(uint32_t)q[j][1] << 32;
        uint64_t hi = (uint64_t)(uint32_t)q[j][2] | (uint64_t)(uint32_t)q[j][3] << 32;
        const bool far = bits >= 64;
        lo = far ? hi : lo;
        hi = far ? 0 : hi;
        const int b = bits & 63;
        lo = (lo >> b) | (b ? hi << (64 - b) : 0);
        hi >>= b;
        q[j] = i32x4{(int)lo, (int)(lo >> 32), (int)hi, (int)(hi >> 32)};
      }
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const uint32_t P = (uint32_t)(j * 256 + (int)threadIdx.x);
      *(i32x4*)(tile + any_at<TY, KM, ROWS>(P / RC, P % RC)) = q[j];
    }
  }
};
// bf16: the 32 x 16 fragment of rows rb.., k 16 kk .. +15
template <bool KM, int ROWS>
__device__ __forceinline__ bf16x8 any_frag(const char* tile, int rb, int kk) {
  const int lane = threadIdx.x & 63;
  if constexpr (KM) {
    return *(const bf16x8*)(tile + any_at<TY_BF16, true, ROWS>((uint32_t)(rb + (lane & 31)), (uint32_t)(2 * kk + (lane >> 5))));
  } else {
    const int g = lane >> 4, j = lane & 15;
    const uint32_t mn = (uint32_t)(rb + 16 * (g & 1) + 4 * (j & 3));
    i16x4 h[2];
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const uint32_t k = (uint32_t)(16 * kk + 8 * (g >> 1) + 4 * hh + (j >> 2));
      h[hh] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_i16x4_t*)((lds_void*)(tile + any_at<TY_BF16, false, ROWS>(k, mn >> 3) + 2u * (mn & 7u))));
    }
    typedef short i16x8 __attribute__((ext_vector_type(8)));
    const i16x8 v = {h[0][0], h[0][1], h[0][2], h[0][3], h[1][0], h[1][1], h[1][2], h[1][3]};
    return __builtin_bit_cast(bf16x8, v);
  }
}
// fp32: row rb + lane % 32, k 8 q + 4 (lane / 32) + 0..3
template <bool KM, int ROWS>
__device__ __forceinline__ f32x4 any_quad(const char* tile, int rb, int q) {
  const int lane = threadIdx.x & 63;
  const uint32_t r = (uint32_t)(rb + (lane & 31)), h = (uint32_t)(lane >> 5);
  if constexpr (KM) {
    return *(const f32x4*)(tile + any_at<TY_F32, true, ROWS>(r, 2u * (uint32_t)q + h));
  } else {
    f32x4 v;
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i)
      v[i] = *(const float*)(tile + any_at<TY_F32, false, ROWS>(8u * (uint32_t)q + 4u * h + i, r >> 2) + 4u * (r & 3u));
    return v;
  }
}

// e4m3, K-major: row rb + lane % 32, two chunks of 16 of the 64 k of half kk
template <int ROWS>
__device__ __forceinline__ i32x8 any_frag8(const char* tile, int rb, int kk) {
  const int lane = threadIdx.x & 63;
  const uint32_t r = (uint32_t)(rb + (lane & 31)), c = (uint32_t)(4 * kk + (lane >> 5));
  const i32x4 lo = *(const i32x4*)(tile + any_at<TY_E4M3, true, ROWS>(r, c));
  const i32x4 hi = *(const i32x4*)(tile + any_at<TY_E4M3, true, ROWS>(r, c + 2u));
  return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}

// Where a strip has several row tiles, units of one XCD (work-group ids
// congruent mod 8) are made contiguous in the logical order, in which the row
// tiles follow each other: they read the same K range of the same columns of B
// through that XCD's L2 (M 256, K 8192, N 1280: 24 -> 23 us, N 8192: 75 -> 71).
// With one row tile B is read once anyway, and neighbouring strips at the same
// time from neighbouring addresses (M = 1, N 8192: 25 us, 27 remapped).
__device__ __forceinline__ int xcd_unit(const GemmParams& p, int i) {
  const int per = p.units >> 3;
  return p.mt_per_group > 1 && i < 8 * per ? (i & 7) * per + (i >> 3) : i;
}

// Unit u of p: K range u / tiles of tile u % tiles; tile t: row tile t % rows of
// strip t / rows.
template <int MB>
constexpr int kAnyLds = 2 * (MB + kAnyTile) * 128;
template <int TY, bool AK, bool BK, int MB>
__device__ __forceinline__ void any_unit(const GemmParams& p, int u, char* __restrict__ smem) {
  using T = AnyTile<TY>;
  // waves along N, and the 32 x 32 MFMA tiles of a wave
  constexpr int WN = MB == 32 ? 4 : 2, FM = MB == 128 ? 2 : 1, FN = MB == 32 ? 1 : 2;
  constexpr int A_BYTES = MB * 128, HALF = kAnyLds<MB> / 2;
  static_assert(MB * kAnyTile * 4 <= kAnyLds<MB>, "the sums fit the staging block");
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int tiles = p.total_tiles, split = u / tiles, tile = u - split * tiles;
  const int strip = tile / p.mt_per_group;
  const int m0 = (tile - strip * p.mt_per_group) * MB, n0 = strip * kAnyTile;
  const int wm = (wave / WN) * 32 * FM, wn = (wave % WN) * 32 * FN;
  const int steps = (p.K + T::KS - 1) / T::KS;
  const int s0 = split * p.ksteps_per_split, s1 = min(steps, s0 + p.ksteps_per_split);
  f32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
  // (two steps ahead: a step's multiplications are much shorter than a load)
  i32x4 qa[2][MB / 32], qb[2][4];
  const AnyOperand<TY, AK, MB> oa(p.A, p.lda, m0, p.M, p.K);
  const AnyOperand<TY, BK, 128> ob(p.B, p.ldb, n0, p.N, p.K);
  auto fetch = [&](int s, i32x4 (&a)[MB / 32], i32x4 (&b)[4]) {
    if (s >= s1) return;
    oa.load(s, a);
    ob.load(s, b);
  };
  auto step = [&](int s, char* ta, i32x4 (&a_next)[MB / 32], i32x4 (&b_next)[4]) {
    char* tb = ta + A_BYTES;
    oa.store(s, ta, a_next);
    ob.store(s, tb, b_next);
    // one barrier a step: a wave that stores into this buffer again, two
    // steps on, has passed the next step's barrier, before which every wave
    // finished reading it
    __syncthreads();
    fetch(s + 2, a_next, b_next);
#pragma unroll
    for (int kk = 0; kk < (TY == TY_E4M3 ? 2 : 4); ++kk) {
      if constexpr (TY == TY_E4M3) {
        i32x8 a[FM], b[FN];
#pragma unroll
        for (int i = 0; i < FM; ++i) a[i] = any_frag8<MB>(ta, wm + 32 * i, kk);
#pragma unroll
        for (int j = 0; j < FN; ++j) b[j] = any_frag8<128>(tb, wn + 32 * j, kk);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a[i], b[j], acc[i][j], 0, 0, 0, 0, 0, 0);
      } else if constexpr (TY == TY_F32) {
        f32x4 a[FM], b[FN];
#pragma unroll
        for (int i = 0; i < FM; ++i) a[i] = any_quad<AK, MB>(ta, wm + 32 * i, kk);
#pragma unroll
        for (int j = 0; j < FN; ++j) b[j] = any_quad<BK, 128>(tb, wn + 32 * j, kk);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i][e], b[j][e], acc[i][j], 0, 0, 0);
      } else {
        bf16x8 a[FM], b[FN];
#pragma unroll
        for (int i = 0; i < FM; ++i) a[i] = any_frag<AK, MB>(ta, wm + 32 * i, kk);
#pragma unroll
        for (int j = 0; j < FN; ++j) b[j] = any_frag<BK, 128>(tb, wn + 32 * j, kk);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
      }
    }
  };
  fetch(s0, qa[0], qb[0]);
  fetch(s0 + 1, qa[1], qb[1]);
  for (int s = s0; s < s1; s += 2) {
    step(s, smem, qa[0], qb[0]);
    if (s + 1 < s1) step(s + 1, smem + HALF, qa[1], qb[1]);
  }
  // Lane l holds column l % 32 and rows 8 q + 4 (l / 32) + 0..3 of each MFMA
  // tile.  The sums go through LDS and one compact loop over rows of 128
  // columns, four per thread: whole rows of 512 bytes in every store, and
  // little code, which each work-group fetches to run once.
  float* out = (float*)smem;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e)
        out[(wm + 32 * i + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3)) * kAnyTile + wn + 32 * j + (lane & 31)] = acc[i][j][e];
  __syncthreads();
  const int quads = min(MB, p.M - m0) * (kAnyTile / 4);
  if (p.splits > 1) {
    f32x4* to = (f32x4*)(p.partial + (int64_t)u * (MB * kAnyTile));
#pragma unroll 1
    for (int i = threadIdx.x; i < quads; i += 256) to[i] = *(const f32x4*)(out + 4 * i);
    return;
  }
  const float scale = scale_of(p);
  const int col = n0 + 4 * (threadIdx.x & 31);
  if (col >= p.N) return;
  const f32x4 bias = bias4(p, col);
  with_act(p.act, [&](auto ac) {
    // (four rows at a time: the residual's loads are in flight together)
#pragma unroll 1
    for (int i = threadIdx.x; i < quads; i += 1024) {
      f32x4 r[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i + 256 * u < quads) r[u] = resid4(p, m0 + (i >> 5) + 8 * u, col);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i + 256 * u < quads)
          finish4<decltype(ac)::value>(p, *(const f32x4*)(out + 4 * i + 1024 * u) * scale + bias, r[u],
                                       m0 + (i >> 5) + 8 * u, col);
    }
  });
}

template <int TY, bool BK, int MB>
__global__ void __launch_bounds__(256, 2) linear_any(const GemmParams p) {
  __shared__ __attribute__((aligned(1024))) char smem[kAnyLds<MB>];
  any_unit<TY, true, BK, MB>(p, xcd_unit(p, blockIdx.x), smem);
}

// The two products of a linear layer's backward in one launch (both are short
// where this kernel serves them): dW (p0, both operands MN-major), then dX (p1,
// both K-major), then the bands' column sums: beside the products instead of a
// launch of their own (fp32, M = 515, N = 771, K = 259: 24.5 us for the whole
// call against 27.4; bf16 64 x 512 x 512 11.0 and 13.0).
template <int TY, int MB>
__global__ void __launch_bounds__(256, 2) linear_any_pair(const GemmParams p0, const GemmParams p1, const BandSums b) {
  __shared__ __attribute__((aligned(1024))) char smem[kAnyLds<MB>];
  const int unit = (int)blockIdx.x - p0.units;
  if (unit < 0) any_unit<TY, false, false, MB>(p0, xcd_unit(p0, blockIdx.x), smem);
  else if (unit < p1.units) any_unit<TY, true, true, MB>(p1, xcd_unit(p1, unit), smem);
  else sum_columns<4>(b.bands, b.count, b.N, (int64_t)(unit - p1.units) * 64, (float*)smem, b.out);
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
  int64_t c0 = (int64_t)blockIdx.x * 512 + 8 * chunk;
  // a last chunk of fewer columns is loaded from N - 8: its first `shift`
  // elements are the chunk's before it (rows of fewer than eight: one by one)
  const int n = (int)std::min<int64_t>(8, N - c0), shift = N >= 8 && n > 0 ? 8 - n : 0;
  const int64_t r1 = std::min<int64_t>(M, (blockIdx.y + 1) * band);
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  c0 -= shift;
  with_act(act, [&](auto ac) {
    constexpr int ACT = decltype(ac)::value;
    if (N >= 8 && n > 0) {
      for (int64_t r = blockIdx.y * band + sub; r < r1; r += 4) {
        float g[8];
        const Raw8<F32> gy = load8<F32>(dY, r * lddy + c0);
        if (Z) {
          float z[8];
          const Raw8<F32> zz = load8<F32>(Z, r * ldz + c0);
          widen8<F32>(gy, g);
          widen8<F32>(zz, z);
#pragma unroll
          for (int e = 0; e < 8; ++e) g[e] *= act_grad_c<ACT>(z[e]);
          store8<F32>(dZ, r * N + c0, g, shift);
        } else {
          widen8<F32>(gy, g);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += g[e];
      }
    } else if (chunk < n) {   // N < 8: thread `chunk` takes column `chunk`
      for (int64_t r = blockIdx.y * band + sub; r < r1; r += 4) {
        float g = ld_f(dY, F32, r * lddy + chunk);
        if (Z) {
          g *= act_grad_c<ACT>(ld_f(Z, F32, r * ldz + chunk));
          st_f(dZ, F32, r * N + chunk, g);
        }
        sum[0] += g;
      }
    }
  });
  if (!part) return;
  if (N >= 8) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (n > 0 && e >= shift) red[sub][8 * chunk + e - shift] = sum[e];
  } else if (chunk < 8) {
    red[sub][chunk] = sum[0];
  }
  __syncthreads();
  for (int k = threadIdx.x; k < 512; k += 256) {
    const int64_t c = (int64_t)blockIdx.x * 512 + k;
    if (c < N) part[blockIdx.y * N + c] = ((red[0][k] + red[1][k]) + red[2][k]) + red[3][k];
  }
}

template <class F>
void with_tile(int mb, F&& f) {
  if (mb == 32) f(std::integral_constant<int, 32>{});
  else if (mb == 64) f(std::integral_constant<int, 64>{});
  else f(std::integral_constant<int, kAnyTile>{});
}

// work-groups of the finalisation (finish_unit)
unsigned finish_groups(const GemmParams& p) {
  const int rows = p.splits > kFinishRows ? p.M : (p.M + kFinishRows - 1) / kFinishRows;
  return p.splits > 1 ? (unsigned)rows * (unsigned)p.nt : 0u;
}

}  // namespace

hipError_t launch_linear_any(const GemmParams& p, int mb, bool w_kmajor, hipStream_t s) {
  hipError_t e = hipSuccess;
  with_tile(mb, [&](auto mc) {
    constexpr int MB = decltype(mc)::value;
    if (p.a_dt == TY_E4M3) {
      if (!w_kmajor) { e = hipErrorInvalidValue; return; }  // rejected on the host first
      linear_any<TY_E4M3, true, MB><<<p.units, 256, 0, s>>>(p);
    } else if (p.a_dt == TY_F32) {
      if (w_kmajor) linear_any<TY_F32, true, MB><<<p.units, 256, 0, s>>>(p);
      else linear_any<TY_F32, false, MB><<<p.units, 256, 0, s>>>(p);
    } else {
      if (w_kmajor) linear_any<TY_BF16, true, MB><<<p.units, 256, 0, s>>>(p);
      else linear_any<TY_BF16, false, MB><<<p.units, 256, 0, s>>>(p);
    }
    e = hipGetLastError();
    if (e != hipSuccess || p.splits <= 1) return;
    finish_ranges<MB><<<finish_groups(p), 256, 0, s>>>(p);
    e = hipGetLastError();
  });
  return e;
}

hipError_t launch_linear_any_pair(const GemmParams& p_dw, const GemmParams& p_dx, const BandSums& b, int mb, hipStream_t s) {
  hipError_t e = hipSuccess;
  with_tile(mb, [&](auto mc) {
    constexpr int MB = decltype(mc)::value;
    const unsigned sums = b.out ? (unsigned)((b.N + 63) / 64) : 0u;
    const unsigned grid = (unsigned)p_dw.units + (unsigned)p_dx.units + sums;
    if (grid == 0) return;
    if (p_dw.a_dt == TY_F32) linear_any_pair<TY_F32, MB><<<grid, 256, 0, s>>>(p_dw, p_dx, b);
    else linear_any_pair<TY_BF16, MB><<<grid, 256, 0, s>>>(p_dw, p_dx, b);
    e = hipGetLastError();
    const unsigned n0 = finish_groups(p_dw), n1 = finish_groups(p_dx);
    if (e != hipSuccess || n0 + n1 == 0) return;
    finish_ranges_pair<MB><<<n0 + n1, 256, 0, s>>>(p_dw, p_dx, (int)n0);
    e = hipGetLastError();
  });
  return e;
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
