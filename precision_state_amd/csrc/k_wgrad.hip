// k_wgrad.hip - the weight gradient of a linear layer whose input was saved in
// 8 bits: dw = dy^T z on the matrix cores, the tokens being the summed axis.
//
// Both operands lie in memory with the summed axis outermost, and go into shared
// memory as they lie, the codes as bytes. Transposing reads
// (ds_read_b64_tr_b16, ds_read_b64_tr_b8) give each lane eight tokens of one
// column, which is what a matrix instruction takes, and the codes become bf16
// or fp16 between that read and the instruction, in the shadow of the matrix
// instructions before. 16384 tokens, 11008 x 4096: 1175 to 1260 us (1.17 to 1.26
// PFLOP/s); the matrix units are busy 72% of the time, and shared memory's
// bandwidth and the last round of tiles bound the rest. The largest tiles take all
// 256 registers and keep 2 to 23 more in scratch memory (with scales 2, with the
// column sums too 8; without scales 9 and 23).
#include <type_traits>

#include "dev_act.h"

namespace ps {
namespace {

typedef __bf16 bf16pair __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
#define LOCAL __attribute__((address_space(3)))

constexpr int kThreads = 256;   // of the join

// Tiles of the result: rows (columns of dy) by columns (of z), how the waves share
// it, and the tokens in shared memory at a time.
template <int N_, int K_, int WN_, int WK_, int STEP_>
struct Shape {
  static constexpr int N = N_, K = K_, WN = WN_, WK = WK_, STEP = STEP_;
  static constexpr int FN = N / WN / 32, FK = K / WK / 32;   // 32 x 32 results of a wave
  static constexpr int THREADS = 64 * WN * WK;
  static_assert(FN * WN * 32 == N && FK * WK * 32 == K, "whole products");
  // one buffer of shared memory: dy, codes, scales [STEP][blocks of 128]
  static constexpr int KB = (K + kActBlock - 1) / kActBlock;
  static constexpr int DY = STEP * N * 2, CODE = STEP * K, BYTES = DY + CODE + STEP * KB * 4;
};
using Large = Shape<256, 256, 2, 4, 64>;
using Middle = Shape<128, 128, 2, 2, 64>;
using FewRows = Shape<32, 256, 1, 4, 64>;
using FewCols = Shape<256, 32, 4, 1, 64>;

// Where 16-byte chunk q of row t lies in a tile of rows of W bytes. A
// transposing read takes R rows of G bytes each at the same place for half a
// wave (64 bytes of four rows, 32 of eight); exchanging the chunks by row puts
// them on different banks.
template <int W, int G>
__device__ __forceinline__ int chunk_at(int t, int q) {
  constexpr int kRows = W >= 256 ? 1 : 256 / W, kParts = (W >= 256 ? 256 : W) / G;
  return t * W + 16 * (q ^ (G / 16 * ((t / kRows) & (kParts - 1))));
}

// dy at 16 tokens and 32 columns: tokens 0-7 on lanes 0-31, 8-15 on the others.
template <int W>
__device__ __forceinline__ s16x8 dy_fragment(const char* tile, int t0, int c, int lane) {
  const int t = t0 + (lane / 32) * 8 + (lane & 15) / 4, col = c + (lane & 16) + (lane & 3) * 4;
  const int o = chunk_at<2 * W, 64>(t, col / 8) + (col & 4) * 2;
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LOCAL s16x4*)(tile + o));
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LOCAL s16x4*)(tile + o + 4 * 2 * W));
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// The codes at the same tokens, 32 columns.
template <int W>
__device__ __forceinline__ i32x2 code_fragment(const char* tile, int t0, int c, int lane) {
  const int t = t0 + (lane / 32) * 8 + (lane & 15) / 2, col = c + (lane & 16) + (lane & 1) * 8;
  return __builtin_amdgcn_ds_read_tr8_b64_v2i32((LOCAL i32x2*)(tile + chunk_at<W, 32>(t, col / 16) + (col & 8)));
}

// Eight codes, and their tokens' scales, as the values that are multiplied.
// Without scales one conversion makes two values; with them the product is
// formed in fp32 and rounded, which loses nothing if a scale is a power of two.
template <int TYPE, bool SCALED>
__device__ __forceinline__ s16x8 values(i32x2 c, const float* s) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (SCALED) {
      const f32x2 v = i & 1 ? __builtin_amdgcn_cvt_pk_f32_fp8(c[i / 2], true) : __builtin_amdgcn_cvt_pk_f32_fp8(c[i / 2], false);
      w[i] = round2<TYPE>(v.x * s[2 * i], v.y * s[2 * i + 1]);
    } else if (TYPE == PS_TYPE_BF16) {
      const bf16x2 v = i & 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i / 2], 1.0f, true)
                             : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i / 2], 1.0f, false);
      w[i] = __builtin_bit_cast(uint32_t, v);
    } else {
      const f16x2 v = i & 1 ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[i / 2], 1.0f, true)
                            : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[i / 2], 1.0f, false);
      w[i] = __builtin_bit_cast(uint32_t, v);
    }
  }
  return __builtin_bit_cast(s16x8, w);
}

// A block's scale as codes are multiplied by it. The code of a finite fp16 x from
// 63488 on stands for 2^16, which fp16 does not hold: with scales that reach so far
// made smaller by a little more than half a step of fp16 at a power of two, that
// product rounds to 65504. Of the others, powers of two round to the value one step
// below (2^-11 of it: no more than a rounding may be off), the rest as they would
// have, since a code's four bits leave them less than half a step away (1.875 / 2
// of it at most); greater ones are infinite as before. It is done where a lane has
// one scale of a step, not for each value between the matrix instructions. bf16
// reaches as far as fp32: only an x of 3.3e38 and more leaves it, and with it dw.
template <int TYPE>
__device__ __forceinline__ float scale_for(float s) {
  return TYPE == PS_TYPE_F16 && s >= 0x1p8f ? s * (1.0f - 0x1p-12f - 0x1p-20f) : s;
}

template <int TYPE>
__device__ __forceinline__ f32x16 mfma(s16x8 a, s16x8 b, f32x16 c) {
  if (TYPE == PS_TYPE_BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// s and the sum of eight values, two to an instruction (products with 1 in fp32).
template <int TYPE>
__device__ __forceinline__ float add_eight(s16x8 a, float s) {
  const u32x4 w = __builtin_bit_cast(u32x4, a);
  float r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t pair = w[i];
    if (TYPE == PS_TYPE_BF16)
      r[i] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16pair, pair), __builtin_bit_cast(bf16pair, 0x3F803F80u), i & 1 ? r[i - 1] : 0.0f, false);
    else
      r[i] = __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, pair), __builtin_bit_cast(f16x2, 0x3C003C00u), i & 1 ? r[i - 1] : 0.0f, false);
  }
  return s + (r[1] + r[3]);
}

// The 16 bytes from (t, at) of a matrix of `rows` rows of `width` bytes, `pitch`
// apart; those behind the matrix are 0 and not read.
__device__ __forceinline__ u32x4 load16_guarded(const char* base, int64_t t, int64_t rows, int64_t pitch, int at, int width) {
  const int64_t left = t < rows ? (rows - 1 - t) * pitch + width - at : 0;
  if (left >= 16) return *(const GLOBAL u32x4_byte*)(base + t * pitch + at);
  uint64_t lo = 0, hi = 0;
#pragma unroll 1
  for (int j = 0; j < left; ++j) {
    const uint64_t byte = (uint64_t)((const GLOBAL uint8_t*)base)[t * pitch + at + j] << (8 * (j & 7));
    if (j < 8)
      lo |= byte;
    else
      hi |= byte;
  }
  return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// How many rows `span` bytes can be loaded of, from byte `at` of the row on,
// without passing the end of the matrix. Bytes past a row's end are the next
// row's: they only reach results that are not stored.
__device__ __forceinline__ int64_t safe_rows(int64_t rows, int64_t pitch, int64_t at, int64_t span, int64_t width) {
  const int64_t over = at + span - width;
  return over <= 0 ? rows : max((int64_t)0, rows - (over + pitch - 1) / pitch);
}

// Four results of a row to memory, `left` of them inside: dw = mul acc + add db [+ dw].
__device__ __forceinline__ void store_dw(const WgradArgs& p, int n, int k, int left, f32x4 acc, float db) {
  if (left <= 0) return;
  const int64_t o = (int64_t)n * p.lddw + k;
  float v[8] = {acc[0], acc[1], acc[2], acc[3], 0, 0, 0, 0};
  if (left >= 4) {
    f32x4_any* f = (f32x4_any*)((float*)p.dw + o);
    u32x2_any* h = (u32x2_any*)((uint16_t*)p.dw + o);
    if (p.mul || p.add || p.accumulate) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (p.mul) v[i] *= p.mul[k + i];
        if (p.add) v[i] = __builtin_fmaf(p.add[k + i], db, v[i]);
      }
      if (p.accumulate) {
        float was[8];
        if (p.dw_type == PS_TYPE_F32) {
          const f32x4 w = *f;
#pragma unroll
          for (int i = 0; i < 4; ++i) was[i] = w[i];
        } else if (p.dw_type == PS_TYPE_BF16) {
          widen8<PS_TYPE_BF16>(Raw8<PS_TYPE_BF16>{{{(*h)[0], (*h)[1], 0, 0}}}, Cols<kWhole>(0, 8), was);
        } else {
          widen8<PS_TYPE_F16>(Raw8<PS_TYPE_F16>{{{(*h)[0], (*h)[1], 0, 0}}}, Cols<kWhole>(0, 8), was);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += was[i];
      }
    }
    if (p.dw_type == PS_TYPE_F32)
      *f = f32x4{v[0], v[1], v[2], v[3]};
    else if (p.dw_type == PS_TYPE_BF16)
      *h = u32x2_any{round2<PS_TYPE_BF16>(v[0], v[1]), round2<PS_TYPE_BF16>(v[2], v[3])};
    else
      *h = u32x2_any{round2<PS_TYPE_F16>(v[0], v[1]), round2<PS_TYPE_F16>(v[2], v[3])};
    return;
  }
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    if (i >= left) continue;
    if (p.mul) v[i] *= p.mul[k + i];
    if (p.add) v[i] = __builtin_fmaf(p.add[k + i], db, v[i]);
    if (p.dw_type == PS_TYPE_F32) {
      float* d = (float*)p.dw + o + i;
      *d = p.accumulate ? *d + v[i] : v[i];
    } else if (p.dw_type == PS_TYPE_BF16) {
      uint16_t* d = (uint16_t*)p.dw + o + i;
      *d = (uint16_t)round2<PS_TYPE_BF16>(p.accumulate ? v[i] + bf16_lo(*d) : v[i], 0.0f);
    } else {
      _Float16* d = (_Float16*)p.dw + o + i;
      *d = (_Float16)(p.accumulate ? v[i] + (float)*d : v[i]);
    }
  }
}

// Which tile a workgroup takes. Workgroups go to the XCDs in turn, each with an
// L2 of its own; this gives the 32 of an XCD that run together (one to a compute
// unit) eight by four neighbouring tiles, which share their rows of dy and codes.
struct Tile {
  int split, n, k;
  __device__ __forceinline__ Tile(const WgradCut& c) {
    constexpr int kGroup = 4;   // tiles of codes side by side
    const uint32_t total = gridDim.x, wg = blockIdx.x, round = kXcdCount * 32;
    uint32_t o = wg;
    if (wg < total / round * round) {
      o = xcd_item<32>(wg, total);
    } else {   // the last round, as far as it can be shared out evenly
      const uint32_t base = total / round * round, each = (total - base) / kXcdCount, i = wg - base;
      if (i < each * kXcdCount) o = base + i % kXcdCount * each + i / kXcdCount;
    }
    const int tiles = c.tiles_n * c.tiles_k;
    split = o / tiles;
    o -= split * tiles;
    const int group = o / (kGroup * c.tiles_n), wide = min(kGroup, c.tiles_k - group * kGroup);
    o -= group * kGroup * c.tiles_n;
    n = o / wide;
    k = group * kGroup + o % wide;
  }
};

// SUMS: the column sums of dy too, for db or add.
template <int TYPE, bool SCALED, bool SUMS, class S>
__global__ __launch_bounds__(S::THREADS, S::THREADS / 256) void k_wgrad(WgradArgs p) {
  __shared__ __attribute__((aligned(16))) char lds[2 * S::BYTES];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const Tile tile(p.cut);
  const int split = __builtin_amdgcn_readfirstlane(tile.split), n0 = __builtin_amdgcn_readfirstlane(tile.n) * S::N;
  const int k0 = __builtin_amdgcn_readfirstlane(tile.k) * S::K;
  const int tokens = (int)p.tokens, first = split * (int)p.cut.per_split, end = min(first + (int)p.cut.per_split, tokens);
  const int wn = wave / S::WK * (S::FN * 32), wk = wave % S::WK * (S::FK * 32);
  const int k_blocks = (p.k + kActBlock - 1) / kActBlock;
  const int safe = min(end, (int)min(safe_rows(tokens, p.lddy * 2, n0 * 2, S::N * 2, p.n * 2),
                                     safe_rows(tokens, p.k, k0, S::K, p.k)));

  // The next step's tiles on their way: registers between a load and a write. A
  // lane takes the same columns of every kPassA-th or kPassB-th row.
  constexpr int kRowA = S::N / 8, kRowB = S::K / 16;   // chunks of 16 bytes of a row
  constexpr int kPassA = S::THREADS / kRowA, kPassB = S::THREADS / kRowB;
  constexpr int kA = (S::STEP + kPassA - 1) / kPassA, kB = (S::STEP + kPassB - 1) / kPassB;
  static_assert(kA * kPassA == S::STEP && (kB * kPassB == S::STEP || kB == 1), "whole passes");
  static_assert(S::THREADS % (S::STEP * S::KB) == 0, "every scale taken as often");
  const int ta = threadIdx.x / kRowA, qa = threadIdx.x % kRowA, tb = threadIdx.x / kRowB, qb = threadIdx.x % kRowB;
  const bool has_b = kB * kPassB == S::STEP || tb < S::STEP;
  const uint32_t from_a = (uint32_t)ta * (uint32_t)(2 * p.lddy) + qa * 16, from_b = (uint32_t)tb * (uint32_t)p.k + qb * 16;
  const int to_a = chunk_at<2 * S::N, 64>(ta, qa), to_b = S::DY + chunk_at<S::K, 32>(tb, qb);
  // a scale for each lane; those too many take the same ones again, which costs less than a branch
  const int ts = (int)threadIdx.x % (S::STEP * S::KB) / S::KB, qs = threadIdx.x % S::KB;
  const int scale_block = min(k0 / kActBlock + qs, k_blocks - 1), to_s = S::DY + S::CODE + (qs * S::STEP + ts) * 4;
  u32x4 ra[kA], rb[kB];
  float rs = 0;
  auto load_a = [&](int i, int t0) __attribute__((always_inline)) {
    const GLOBAL char* row = scalar_pointer((GLOBAL char*)p.dy + (int64_t)(t0 + i * kPassA) * (2 * p.lddy) + 2 * n0);
    ra[i] = *(const GLOBAL u32x4_any*)(row + from_a);
  };
  auto load_b = [&](int i, int t0) __attribute__((always_inline)) {
    const GLOBAL char* row = scalar_pointer((GLOBAL char*)p.code + (int64_t)(t0 + i * kPassB) * p.k + k0);
    if (has_b) rb[i] = *(const GLOBAL u32x4_byte*)(row + from_b);
  };
  auto load_s = [&](int t0) __attribute__((always_inline)) {
    if (SCALED) rs = p.scale[(int64_t)(t0 + ts) * k_blocks + scale_block];
  };
  // The i-th part of three: what was loaded goes to the buffer, and the same rows
  // of the step after are loaded.
  // The scales go with the first part, but those of fp16, which scale_for makes
  // wait, with the last one (16384 x 8192 x 8192 2093 -> 2043 us; with the column
  // sums 2077 -> 2091, so not there).
  constexpr int U = S::STEP / 16, kParts = U - 1, kScalePart = TYPE == PS_TYPE_F16 && !SUMS ? kParts - 1 : 0;
  auto renew = [&](char* buf, int part, int t0) __attribute__((always_inline)) {
#pragma unroll
    for (int i = part * kA / kParts; i < (part + 1) * kA / kParts; ++i) {
      *(u32x4*)(buf + to_a + i * kPassA * 2 * S::N) = ra[i];
      load_a(i, t0);
    }
#pragma unroll
    for (int i = part * kB / kParts; i < (part + 1) * kB / kParts; ++i) {
      if (has_b) *(u32x4*)(buf + to_b + i * kPassB * S::K) = rb[i];
      load_b(i, t0);
    }
    if (part == kScalePart) {
      if (SCALED) *(float*)(buf + to_s) = scale_for<TYPE>(rs);
      load_s(t0);
    }
  };
  // The same for a step at the end of the split or of the matrices.
  auto load_and_place = [&](char* buf, int t0) __attribute__((always_inline)) {
#pragma unroll 1
    for (int i = 0; i < kA; ++i) {
      const int64_t t = t0 + i * kPassA + ta;
      const u32x4 w = load16_guarded((const char*)p.dy, t, t < end ? p.tokens : 0, 2 * p.lddy, 2 * n0 + qa * 16, 2 * p.n);
      *(u32x4*)(buf + to_a + i * kPassA * 2 * S::N) = w;
    }
#pragma unroll 1
    for (int i = 0; i < kB; ++i) {
      const int64_t t = t0 + i * kPassB + tb;
      if (has_b)
        *(u32x4*)(buf + to_b + i * kPassB * S::K) =
            load16_guarded((const char*)p.code, t, t < end ? p.tokens : 0, p.k, k0 + qb * 16, p.k);
    }
    const int64_t t = t0 + ts;
    if (SCALED) *(float*)(buf + to_s) = t < end ? scale_for<TYPE>(p.scale[t * k_blocks + scale_block]) : 0.0f;
  };

  f32x16 acc[S::FN][S::FK];
#pragma unroll
  for (int i = 0; i < S::FN; ++i)
#pragma unroll
    for (int j = 0; j < S::FK; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;

  float sums[S::FN] = {};   // of a lane's column, over its half of the tokens
  constexpr int kSets = SCALED ? 1 : 2;   // of fragments: with the scales two of them leave too few registers
  s16x8 a[kSets][S::FN];
  i32x2 b[kSets][S::FK];
  f32x4 sc[2];
  auto read = [&](const char* buf, int u, int to) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < S::FN; ++i) a[to][i] = dy_fragment<S::N>(buf, u, wn + i * 32, lane);
#pragma unroll
    for (int j = 0; j < S::FK; ++j) b[to][j] = code_fragment<S::K>(buf + S::DY, u, wk + j * 32, lane);
    if (SCALED) {
      const float* s = (const float*)(buf + S::DY + S::CODE) + wk / kActBlock * S::STEP + u + lane / 32 * 8;
      sc[0] = *(const f32x4*)s;
      sc[1] = *(const f32x4*)(s + 4);
    }
  };
  // Only the tiles at the first columns add up dy, or all if each needs the sums.
  const bool adds = SUMS && (k0 == 0 || (p.add && p.cut.splits == 1));
  auto multiply = [&](int from, auto sum) __attribute__((always_inline)) {
    float s[8];
    if (SCALED) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = sc[i / 4][i % 4];
    }
#pragma unroll
    for (int j = 0; j < S::FK; ++j) {
      const s16x8 v = values<TYPE, SCALED>(b[from][j], s);
#pragma unroll
      for (int i = 0; i < S::FN; ++i) acc[i][j] = mfma<TYPE>(a[from][i], v, acc[i][j]);
    }
    if (decltype(sum)::value) {
#pragma unroll
      for (int i = 0; i < S::FN; ++i) sums[i] = add_eight<TYPE>(a[from][i], sums[i]);
    }
  };

  // Two buffers: while one is multiplied the other is filled with the tiles that
  // were loaded a step before. The fragments of 16 tokens are read ahead of the
  // matrix instructions that use them, the first ones of a step before the last 16
  // tokens of the step before are multiplied. The last steps load and place the
  // last tiles again, so that no branch cuts a step.
  const int whole = __builtin_amdgcn_readfirstlane(first + (safe > first ? (safe - first) / S::STEP * S::STEP : 0));
  const int last = whole - S::STEP;
  auto step = [&](char* cur, char* nxt, int t, auto sum) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (kSets == 1) read(cur, u * 16, 0);
      if (kSets == 2 && u + 1 == U) __syncthreads();
      if (kSets == 2) read(u + 1 < U ? cur : nxt, (u + 1) % U * 16, (u + 1) & 1);
      if (u + 1 < U) renew(nxt, u, min(t + 2 * S::STEP, last));
      __builtin_amdgcn_s_setprio(1);
      multiply(kSets == 1 ? 0 : u & 1, sum);
      __builtin_amdgcn_s_setprio(0);
      if (kSets == 1 && u + 1 == U) __syncthreads();
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto steps = [&](auto sum) __attribute__((always_inline)) {
    char *one = lds, *two = lds + S::BYTES;
#pragma unroll
    for (int i = 0; i < kA; ++i) load_a(i, first);
#pragma unroll
    for (int i = 0; i < kB; ++i) load_b(i, first);
    load_s(first);
#pragma unroll
    for (int u = 0; u < kParts; ++u) renew(one, u, min(first + S::STEP, last));
    __syncthreads();
    if (kSets == 2) read(one, 0, 0);
    int t = first;
    for (; t + S::STEP < whole; t += 2 * S::STEP) {
      step(one, two, t, sum);
      step(two, one, t + S::STEP, sum);
    }
    if (t < whole) step(one, two, t, sum);
  };
  if (first < whole) {
    if (adds)
      steps(std::integral_constant<bool, SUMS>());
    else
      steps(std::false_type());
  }
  for (int t = whole; t < end; t += S::STEP) {
    __syncthreads();
    load_and_place(lds, t);
    __syncthreads();
#pragma unroll 1
    for (int u = 0; u < S::STEP; u += 16) {
      read(lds, u, 0);
      multiply(0, std::integral_constant<bool, SUMS>());
    }
  }

  // Result e of a 32 x 32 product is row 8 (e / 4) + 4 (lane / 32) + e % 4, column
  // lane % 32. A wave's 32 rows go through its part of shared memory, so that
  // rows are stored four columns a lane.
  constexpr int kSide = S::FK < 2 ? S::FK : 2, kCols = kSide * 32, kLanes = kCols / 4;   // products side by side
  static_assert(S::THREADS / 64 * 32 * kCols * 4 + S::N * 4 <= 2 * S::BYTES, "a part for each wave, and the column sums");
  float* part = (float*)lds + wave * (32 * kCols);
  float* db = (float*)(lds + 2 * S::BYTES) - S::N;   // behind the parts
  if (SUMS) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < S::FN; ++i) {
      const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(sums[i]), __float_as_uint(sums[i]), false, false);
      const float s = __uint_as_float(x[0]) + __uint_as_float(x[1]);
      if (wave % S::WK == 0 && lane < 32) db[wn + i * 32 + lane] = s;
    }
    __syncthreads();
    if (threadIdx.x < S::N) {
      const float s = db[threadIdx.x];
      const int n = n0 + threadIdx.x;
      if (k0 == 0 && n < p.n) {
        if (p.cut.splits > 1)
          p.db_part[(int64_t)split * p.n + n] = s;
        else if (p.db)
          p.db[n] = p.accumulate ? p.db[n] + s : s;
      }
    }
  }
#pragma unroll
  for (int x = 0; x < S::FN * S::FK / kSide; ++x) {
    const int i = x % S::FN, j0 = x / S::FN * kSide;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kSide; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e)
        part[(8 * (e / 4) + 4 * (lane / 32) + e % 4) * kCols + j * 32 + lane % 32] = acc[i][j0 + j][e];
    __syncthreads();
#pragma unroll 1
    for (int c = lane; c < 32 * kLanes; c += 64) {
      const int row = wn + i * 32 + c / kLanes, n = n0 + row, k = k0 + wk + j0 * 32 + c % kLanes * 4;
      if (n >= p.n) break;
      const f32x4 v = *(const f32x4*)(part + c * 4);
      if (p.cut.splits > 1) {
        float* d = p.part + ((int64_t)split * p.n + n) * p.k + k;
        if (p.k - k >= 4) {
          *(f32x4_any*)d = v;
        } else {
#pragma unroll
          for (int x = 0; x < 3; ++x)
            if (k + x < p.k) d[x] = v[x];
        }
      } else {
        store_dw(p, n, k, p.k - k, v, SUMS ? db[row] : 0.0f);
      }
    }
  }
}

// The splits' partial results added up in order, four columns of a row a lane;
// behind them db, one of its values a lane.
__global__ __launch_bounds__(kThreads) void k_wgrad_join(WgradArgs p) {
  const int quads = (p.k + 3) / 4;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x, size = (int64_t)p.n * p.k;
  auto db_of = [&](int n) {
    float s = 0;
#pragma unroll 8
    for (int j = 0; j < p.cut.splits; ++j) s += p.db_part[(int64_t)j * p.n + n];
    return s;
  };
  if (i >= (int64_t)p.n * quads) {
    const int64_t n = i - (int64_t)p.n * quads;
    if (!p.db || n >= p.n) return;
    const float s = db_of((int)n);
    p.db[n] = p.accumulate ? p.db[n] + s : s;
    return;
  }
  const int n = (int)(i / quads), k = (int)(i % quads) * 4, left = p.k - k;
  const float* d = p.part + (int64_t)n * p.k + k;
  f32x4 s = {0, 0, 0, 0};
  if (left >= 4) {
#pragma unroll 8
    for (int j = 0; j < p.cut.splits; ++j) s += *(const f32x4_any*)(d + j * size);
  } else {
    for (int j = 0; j < p.cut.splits; ++j)
#pragma unroll
      for (int x = 0; x < 3; ++x)
        if (x < left) s[x] += d[j * size + x];
  }
  store_dw(p, n, k, left, s, p.add ? db_of(n) : 0.0f);
}

template <int TYPE, class S>
void product(const WgradArgs& p, hipStream_t s) {
  const dim3 grid(p.cut.tiles_n * p.cut.tiles_k * p.cut.splits);
  const bool sums = p.db || p.add;
  if (p.scale && sums)
    hipLaunchKernelGGL((k_wgrad<TYPE, true, true, S>), grid, dim3(S::THREADS), 0, s, p);
  else if (p.scale)
    hipLaunchKernelGGL((k_wgrad<TYPE, true, false, S>), grid, dim3(S::THREADS), 0, s, p);
  else if (sums)
    hipLaunchKernelGGL((k_wgrad<TYPE, false, true, S>), grid, dim3(S::THREADS), 0, s, p);
  else
    hipLaunchKernelGGL((k_wgrad<TYPE, false, false, S>), grid, dim3(S::THREADS), 0, s, p);
}

template <int TYPE>
ps_status product(const WgradArgs& p, hipStream_t s) {
  switch (p.cut.kind) {
    case 0: product<TYPE, Large>(p, s); break;
    case 1: product<TYPE, Middle>(p, s); break;
    case 2: product<TYPE, FewRows>(p, s); break;
    default: product<TYPE, FewCols>(p, s); break;
  }
  if (ps_status st = hip_check(hipGetLastError(), "k_wgrad launch")) return st;
  if (p.cut.splits > 1) {
    const int64_t lanes = (int64_t)p.n * ((p.k + 3) / 4) + (p.db ? p.n : 0);
    hipLaunchKernelGGL(k_wgrad_join, dim3((uint32_t)((lanes + kThreads - 1) / kThreads)), dim3(kThreads), 0, s, p);
    return hip_check(hipGetLastError(), "k_wgrad_join launch");
  }
  return PS_OK;
}

}  // namespace

WgradCut wgrad_cut(int64_t tokens, int64_t n, int64_t k) {
  constexpr int kStep = 64;
  static const int kN[] = {Large::N, Middle::N, FewRows::N, FewCols::N}, kK[] = {Large::K, Middle::K, FewRows::K, FewCols::K};
  WgradCut c = {};
  c.kind = n <= 32 ? 2 : k <= 32 ? 3 : n >= 1024 && k >= 1024 ? 0 : 1;
  c.tiles_n = (int32_t)((n + kN[c.kind] - 1) / kN[c.kind]);
  c.tiles_k = (int32_t)((k + kK[c.kind] - 1) / kK[c.kind]);
  const int64_t tiles = (int64_t)c.tiles_n * c.tiles_k;
  // enough workgroups for the 256 compute units, but 128 tokens or more for each
  const int64_t want = tiles >= 256 ? 1 : (256 + tiles - 1) / tiles;
  const int64_t most = tokens < 256 ? 1 : tokens / 128;
  c.splits = (int32_t)(want < most ? want : most);
  c.per_split = ((tokens + c.splits - 1) / c.splits + kStep - 1) / kStep * kStep;   // whole steps
  if (c.per_split) c.splits = (int32_t)((tokens + c.per_split - 1) / c.per_split);
  if (c.splits < 1) c.splits = 1;
  return c;
}

ps_status launch_wgrad(const WgradArgs& p, hipStream_t s) {
  return p.dy_type == PS_TYPE_BF16 ? product<PS_TYPE_BF16>(p, s) : product<PS_TYPE_F16>(p, s);
}

}  // namespace ps
