// k_wgrad.hip - the weight gradient of a linear layer whose input was saved in
// 8 bits: dw = dy^T z on the matrix cores, the tokens being the summed axis.
//
// Both operands lie in memory with the summed axis outermost. Tiles [tokens,
// columns] go into shared memory as they lie, dy's as it is and the codes
// converted to dy's type on the way, and ds_read_b64_tr_b16 gives each lane
// the values of one column at four tokens, which is what a matrix instruction
// takes; which of its 16 places a token has does not matter, as long as both
// operands agree.
#include "dev_act.h"

namespace ps {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
#define LOCAL __attribute__((address_space(3)))

constexpr int kStep = 32;      // tokens in shared memory at a time
constexpr int kThreads = 256;  // four waves

// Tiles of the result: rows (columns of dy) by columns (of z), and how the four
// waves share it.
template <int N_, int K_, int WN_, int WK_>
struct Shape {
  static constexpr int N = N_, K = K_, WN = WN_, WK = WK_;
  static constexpr int FN = N / WN / 32, FK = K / WK / 32;   // 32 x 32 results of a wave
  static_assert(WN * WK == 4 && FN * WN * 32 == N && FK * WK * 32 == K, "four waves");
};
using Large = Shape<256, 256, 2, 2>;
using Middle = Shape<128, 128, 2, 2>;
using FewRows = Shape<32, 256, 1, 4>;
using FewCols = Shape<256, 32, 4, 1>;

// Place of a 16-byte chunk q of row t in a tile of W 16-bit columns. A transposing
// read takes four rows at the same 64 bytes; the exchange puts them on
// different banks.
template <int W>
__device__ __forceinline__ int chunk_at(int t, int q) {
  constexpr int kRows = W >= 128 ? 1 : 128 / W;   // rows in the 256 bytes of all banks
  return t * (W / 8) + (q ^ (4 * ((t / kRows) & (4 / kRows - 1))));
}

// A fragment of 16 tokens and 32 columns from column c on: tokens 0-3 and 8-11
// on lanes 0-31, 4-7 and 12-15 on the others.
template <int W>
__device__ __forceinline__ s16x8 fragment(const uint16_t* tile, int t0, int c, int lane) {
  const int t = t0 + (lane / 32) * 4 + (lane & 15) / 4;
  const int col = c + (lane & 16) + (lane & 3) * 4;
  const int o0 = chunk_at<W>(t, col / 8) * 8 + (col & 4), o1 = chunk_at<W>(t + 8, col / 8) * 8 + (col & 4);
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LOCAL s16x4*)(tile + o0));
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LOCAL s16x4*)(tile + o1));
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

template <int TYPE>
__device__ __forceinline__ f32x16 mfma(s16x8 a, s16x8 b, f32x16 c) {
  if (TYPE == PS_TYPE_BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// How many elements there are from (t, col) to the end of a matrix of `rows`
// rows, eight at most, none behind the last row. Columns past the row's end
// read the next row: they only reach results that are not stored.
__device__ __forceinline__ int left_from(int64_t t, int64_t rows, int64_t ld, int col, int cols) {
  if (t >= rows) return 0;
  const int64_t left = (rows - 1 - t) * ld + cols - col;
  return left >= 8 ? 8 : (int)left;
}

// One result to memory: dw = mul acc + add db [+ dw].
__device__ __forceinline__ void store_dw(const WgradArgs& p, int n, int k, float acc) {
  if (p.mul) acc *= p.mul[k];
  if (p.add) acc = __builtin_fmaf(p.add[k], p.db_sum[n], acc);
  const int64_t o = (int64_t)n * p.lddw + k;
  if (p.dw_type == PS_TYPE_F32) {
    float* d = (float*)p.dw + o;
    *d = p.accumulate ? *d + acc : acc;
  } else if (p.dw_type == PS_TYPE_BF16) {
    uint16_t* d = (uint16_t*)p.dw + o;
    if (p.accumulate) acc += bf16_lo(*d);
    *d = (uint16_t)round2<PS_TYPE_BF16>(acc, 0.0f);
  } else {
    _Float16* d = (_Float16*)p.dw + o;
    if (p.accumulate) acc += (float)*d;
    *d = (_Float16)acc;
  }
}

template <int TYPE, class S>
__global__ __launch_bounds__(kThreads) void k_wgrad(WgradArgs p) {
  __shared__ __attribute__((aligned(16))) uint16_t lds[2][kStep * (S::N + S::K)];
  const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
  const int tiles = p.cut.tiles_n * p.cut.tiles_k;
  const int split = blockIdx.x / tiles, tile = blockIdx.x % tiles;
  const int n0 = tile % p.cut.tiles_n * S::N, k0 = tile / p.cut.tiles_n * S::K;
  const int64_t first = (int64_t)split * p.cut.per_split;
  const int64_t end = min(first + p.cut.per_split, p.tokens);
  const int wn = wave / S::WK * (S::FN * 32), wk = wave % S::WK * (S::FK * 32);
  const int k_blocks = (p.k + kActBlock - 1) / kActBlock;

  constexpr int kA = (kStep * S::N / 8 + kThreads - 1) / kThreads, kB = (kStep * S::K / 8 + kThreads - 1) / kThreads;
  Raw8<TYPE> ra[kA];
  u32x2_any rb[kB];
  float sb[kB];
  auto fetch = [&](int64_t t0) {
#pragma unroll
    for (int i = 0; i < kA; ++i) {
      const int c = i * kThreads + threadIdx.x, q = c % (S::N / 8);
      const int64_t t = t0 + c / (S::N / 8);
      const int left = c < kStep * S::N / 8 && t < end ? left_from(t, p.tokens, p.lddy, n0 + q * 8, p.n) : 0;
      ra[i] = load8<TYPE, false>(p.dy, t * p.lddy + n0 + q * 8, left);
    }
#pragma unroll
    for (int i = 0; i < kB; ++i) {
      const int c = i * kThreads + threadIdx.x, q = c % (S::K / 8);
      const int64_t t = t0 + c / (S::K / 8);
      const int left = c < kStep * S::K / 8 && t < end ? left_from(t, p.tokens, p.k, k0 + q * 8, p.k) : 0;
      rb[i] = load_codes8(p.code, t * p.k + k0 + q * 8, left);
      const int block = min((k0 + q * 8) / kActBlock, k_blocks - 1);
      sb[i] = p.scale && left > 0 ? p.scale[t * k_blocks + block] : 1.0f;
    }
  };
  auto place = [&](uint16_t* tile_a, uint16_t* tile_b) {
#pragma unroll
    for (int i = 0; i < kA; ++i) {
      const int c = i * kThreads + threadIdx.x;
      if (c < kStep * S::N / 8) *(u32x4*)(tile_a + chunk_at<S::N>(c / (S::N / 8), c % (S::N / 8)) * 8) = ra[i].w[0];
    }
#pragma unroll
    for (int i = 0; i < kB; ++i) {
      const int c = i * kThreads + threadIdx.x;
      float v[8];
      codes_to_f32(rb[i], v);
      u32x4 w;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = round2<TYPE>(v[2 * j] * sb[i], v[2 * j + 1] * sb[i]);
      if (c < kStep * S::K / 8) *(u32x4*)(tile_b + chunk_at<S::K>(c / (S::K / 8), c % (S::K / 8)) * 8) = w;
    }
  };

  f32x16 acc[S::FN][S::FK];
#pragma unroll
  for (int i = 0; i < S::FN; ++i)
#pragma unroll
    for (int j = 0; j < S::FK; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;

  int buf = 0;
  if (first < end) {
    fetch(first);
    place(lds[0], lds[0] + kStep * S::N);
  }
  __syncthreads();
  for (int64_t t = first; t < end; t += kStep) {
    const bool more = t + kStep < end;
    if (more) fetch(t + kStep);
    const uint16_t *ta = lds[buf], *tb = ta + kStep * S::N;
#pragma unroll
    for (int u = 0; u < kStep; u += 16) {
      s16x8 a[S::FN], b[S::FK];
#pragma unroll
      for (int i = 0; i < S::FN; ++i) a[i] = fragment<S::N>(ta, u, wn + i * 32, lane);
#pragma unroll
      for (int j = 0; j < S::FK; ++j) b[j] = fragment<S::K>(tb, u, wk + j * 32, lane);
#pragma unroll
      for (int i = 0; i < S::FN; ++i)
#pragma unroll
        for (int j = 0; j < S::FK; ++j) acc[i][j] = mfma<TYPE>(a[i], b[j], acc[i][j]);
    }
    buf ^= 1;
    if (more) place(lds[buf], lds[buf] + kStep * S::N);
    __syncthreads();
  }

  // Result e of a 32 x 32 product: row 8 (e / 4) + 4 (lane / 32) + e % 4, column lane % 32.
#pragma unroll
  for (int i = 0; i < S::FN; ++i)
#pragma unroll
    for (int j = 0; j < S::FK; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int n = n0 + wn + i * 32 + 8 * (e / 4) + 4 * (lane / 32) + e % 4, k = k0 + wk + j * 32 + lane % 32;
        if (n >= p.n || k >= p.k) continue;
        if (p.cut.splits > 1)
          p.part[((int64_t)split * p.n + n) * p.k + k] = acc[i][j][e];
        else
          store_dw(p, n, k, acc[i][j][e]);
      }
}

// The splits' partial results added up in order.
__global__ __launch_bounds__(kThreads) void k_wgrad_join(WgradArgs p) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x, size = (int64_t)p.n * p.k;
  if (i >= size) return;
  float s = p.part[i];
  for (int j = 1; j < p.cut.splits; ++j) s += p.part[j * size + i];
  store_dw(p, (int)(i / p.k), (int)(i % p.k), s);
}

// Sums of dy over a strip of tokens: 256 columns a workgroup, eight on a lane,
// every eighth token on a group of lanes.
template <int TYPE>
__global__ __launch_bounds__(kThreads) void k_column_sums(WgradArgs p) {
  __shared__ float lds[8][256];
  const int q = threadIdx.x % 32, group = threadIdx.x / 32;
  const int col = blockIdx.x * 256 + q * 8;
  const int64_t first = (int64_t)blockIdx.y * p.cut.per_strip, end = min(first + p.cut.per_strip, p.tokens);
  float s[8] = {};
  for (int64_t t = first + group; t < end; t += 8) {
    float v[8];
    widen8<TYPE>(load8<TYPE, false>(p.dy, t * p.lddy + col, p.n - col), v);
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] += v[j];
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) lds[group][q * 8 + j] = s[j];
  __syncthreads();
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= p.n) return;
  float total = lds[0][threadIdx.x];
#pragma unroll
  for (int g = 1; g < 8; ++g) total += lds[g][threadIdx.x];
  p.db_part[(int64_t)blockIdx.y * p.n + c] = total;
}

__global__ __launch_bounds__(kThreads) void k_column_join(WgradArgs p) {
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= p.n) return;
  float s = 0;
  for (int i = 0; i < p.cut.strips; ++i) s += p.db_part[(int64_t)i * p.n + c];
  if (p.add) p.db_sum[c] = s;
  if (p.db) p.db[c] = p.accumulate ? p.db[c] + s : s;
}

template <int TYPE, class S>
void product(const WgradArgs& p, hipStream_t s) {
  hipLaunchKernelGGL((k_wgrad<TYPE, S>), dim3(p.cut.tiles_n * p.cut.tiles_k * p.cut.splits), dim3(kThreads), 0, s, p);
}

template <int TYPE>
ps_status product(const WgradArgs& p, hipStream_t s) {
  if (p.db || p.add) {
    if (p.cut.strips) hipLaunchKernelGGL(k_column_sums<TYPE>, dim3((p.n + 255) / 256, p.cut.strips), dim3(kThreads), 0, s, p);
    if (ps_status st = hip_check(hipGetLastError(), "k_column_sums launch")) return st;
    hipLaunchKernelGGL(k_column_join, dim3((p.n + kThreads - 1) / kThreads), dim3(kThreads), 0, s, p);
    if (ps_status st = hip_check(hipGetLastError(), "k_column_join launch")) return st;
  }
  switch (p.cut.kind) {
    case 0: product<TYPE, Large>(p, s); break;
    case 1: product<TYPE, Middle>(p, s); break;
    case 2: product<TYPE, FewRows>(p, s); break;
    default: product<TYPE, FewCols>(p, s); break;
  }
  if (ps_status st = hip_check(hipGetLastError(), "k_wgrad launch")) return st;
  if (p.cut.splits > 1) {
    const int64_t size = (int64_t)p.n * p.k;
    hipLaunchKernelGGL(k_wgrad_join, dim3((uint32_t)((size + kThreads - 1) / kThreads)), dim3(kThreads), 0, s, p);
    return hip_check(hipGetLastError(), "k_wgrad_join launch");
  }
  return PS_OK;
}

}  // namespace

WgradCut wgrad_cut(int64_t tokens, int64_t n, int64_t k) {
  static const int kN[] = {Large::N, Middle::N, FewRows::N, FewCols::N}, kK[] = {Large::K, Middle::K, FewRows::K, FewCols::K};
  WgradCut c = {};
  c.kind = n <= 32 ? 2 : k <= 32 ? 3 : n >= 1024 && k >= 1024 ? 0 : 1;
  c.tiles_n = (int32_t)((n + kN[c.kind] - 1) / kN[c.kind]);
  c.tiles_k = (int32_t)((k + kK[c.kind] - 1) / kK[c.kind]);
  const int64_t tiles = (int64_t)c.tiles_n * c.tiles_k;
  // enough workgroups for the 256 compute units, but 256 tokens or more for each
  const int64_t want = tiles >= 256 ? 1 : (256 + tiles - 1) / tiles;
  const int64_t most = tokens < 512 ? 1 : tokens / 256;
  c.splits = (int32_t)(want < most ? want : most);
  c.per_split = ((tokens + c.splits - 1) / c.splits + kStep - 1) / kStep * kStep;
  if (c.per_split) c.splits = (int32_t)((tokens + c.per_split - 1) / c.per_split);
  c.per_strip = tokens < 64 * 64 ? 64 : (tokens + 63) / 64;
  c.strips = (int32_t)((tokens + c.per_strip - 1) / c.per_strip);
  if (c.splits < 1) c.splits = 1;
  return c;
}

ps_status launch_wgrad(const WgradArgs& p, hipStream_t s) {
  return p.dy_type == PS_TYPE_BF16 ? product<PS_TYPE_BF16>(p, s) : product<PS_TYPE_F16>(p, s);
}

}  // namespace ps
