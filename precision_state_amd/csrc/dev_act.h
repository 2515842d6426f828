// dev_act.h - gfx950 device helpers of the activation checkpoints: eight
// consecutive values of a row at any alignment, vectors of any type, sums over
// a wave.
#pragma once

#include "dev_adamw.h"
#include "ps_act.h"

namespace ps {

// The hardware reads and writes global memory at any byte address; these types
// let the compiler use the widest access for data aligned to its element only.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32_any __attribute__((aligned(1)));
typedef uint16_t u16_any __attribute__((aligned(1)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32x4_byte __attribute__((ext_vector_type(4), aligned(1)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// A grid dimension holds less than 2^32 lanes: `n` workgroups, and those that fill
// up the last of its rows, numbered blockIdx.y * gridDim.x + blockIdx.x < 2^31.
inline dim3 grid_2d(uint32_t n) {
  constexpr uint32_t kMost = 1u << 20;
  return n <= kMost ? dim3(n) : dim3(kMost, (n + kMost - 1) / kMost);
}

__device__ __forceinline__ uint32_t div_by(uint32_t u, const FastDiv& f) { return (uint32_t)(((uint64_t)u * f.m) >> f.s); }

// Eight values of a row as they lie in memory.
template <int TYPE>
struct Raw8 {
  u32x4 w[TYPE == PS_TYPE_F32 ? 2 : 1];   // [1] is there for fp32 only
};
template <int TYPE>
constexpr int kBytes = TYPE == PS_TYPE_F32 ? 4 : 2;

// 128 bits shifted down by 0 < n < 128.
__device__ __forceinline__ u32x4 shift_down(u32x4 w, int n) {
  uint64_t lo = (uint64_t)w[1] << 32 | w[0], hi = (uint64_t)w[3] << 32 | w[2];
  if (n >= 64) {
    lo = hi;
    hi = 0;
  }
  n &= 63;
  lo = lo >> n | (hi << 1) << (63 - n);
  hi >>= n;
  return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// Eight columns of a row, those from `col` on, of which `left` exist (none if
// left <= 0). END says how rows end: at a multiple of eight (kWhole); anywhere
// (kPart), where a lane with fewer than eight loads the row's last eight, which
// widen8 moves into place, so that every lane loads alike: no branch around a
// load, and no lane whose row ends costs more; or before eight (kShort), loaded
// one by one. kEvery is for rows of which every lane of the team has eight.
enum { kWhole = 0, kPart = 1, kShort = 2, kEvery = 3 };
inline int end_of(int cols) { return cols < 8 ? kShort : cols % 8 ? kPart : kWhole; }
template <int END>
struct Cols {
  int left, start;
  __device__ __forceinline__ Cols(int col, int cols)
      : left(END == kEvery ? 8 : cols - col),
        start(END == kShort || END == kEvery ? col : __builtin_elementwise_min(col, cols - 8)) {}
};

template <int TYPE, bool STREAM = true, int END>
__device__ __forceinline__ Raw8<TYPE> load8(const GLOBAL char* row, const Cols<END>& c) {
  Raw8<TYPE> r = {};
  if (END != kShort) {
    const GLOBAL u32x4_any* p = (const GLOBAL u32x4_any*)(row + (uint32_t)(c.start * kBytes<TYPE>));
#pragma unroll
    for (int i = 0; i < (int)sizeof(r.w) / 16; ++i) r.w[i] = STREAM ? (u32x4)__builtin_nontemporal_load(p + i) : (u32x4)p[i];
    return r;
  }
  // each pushes the ones before it down, so that they end where widen8 expects them
#pragma unroll 1
  for (int j = 0; j < c.left; ++j) {
    if (TYPE == PS_TYPE_F32) {
      u32x4& top = r.w[TYPE == PS_TYPE_F32 ? 1 : 0];
      r.w[0] = u32x4{r.w[0][1], r.w[0][2], r.w[0][3], top[0]};
      top = u32x4{top[1], top[2], top[3], ((const GLOBAL uint32_t*)row)[c.start + j]};
    } else {
      r.w[0] = shift_down(r.w[0], 16);
      r.w[0][3] |= (uint32_t)((const GLOBAL uint16_t*)row)[c.start + j] << 16;
    }
  }
  return r;
}

template <int TYPE, int END>
__device__ __forceinline__ void widen8(Raw8<TYPE> r, const Cols<END>& c, float* d) {
  if (c.left < (END == kWhole ? 1 : 8)) {
    const int k = 8 - c.left;
    if (c.left <= 0) {
      r = Raw8<TYPE>{};
    } else if (TYPE == PS_TYPE_F32) {
      if (k & 4) {
        r.w[0] = r.w[1];
        r.w[1] = u32x4{0, 0, 0, 0};
      }
      if (k & 2) {
        r.w[0] = u32x4{r.w[0][2], r.w[0][3], r.w[1][0], r.w[1][1]};
        r.w[1] = u32x4{r.w[1][2], r.w[1][3], 0, 0};
      }
      if (k & 1) {
        r.w[0] = u32x4{r.w[0][1], r.w[0][2], r.w[0][3], r.w[1][0]};
        r.w[1] = u32x4{r.w[1][1], r.w[1][2], r.w[1][3], 0};
      }
    } else {
      r.w[0] = shift_down(r.w[0], 16 * k);
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (TYPE == PS_TYPE_F32) {
      d[j] = __uint_as_float(r.w[j / 4][j % 4]);
    } else if (TYPE == PS_TYPE_BF16) {
      d[j] = j & 1 ? bf16_hi(r.w[0][j / 2]) : bf16_lo(r.w[0][j / 2]);
    } else {
      const uint32_t w = r.w[0][j / 2];
      const f16x2 h = __builtin_bit_cast(f16x2, w);
      d[j] = (float)h[j & 1];
    }
  }
}

template <int TYPE>
__device__ __forceinline__ uint32_t round2(float a, float b) {
  const f32x2 v = {a, b};
  if (TYPE == PS_TYPE_BF16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
}

// Eight values to columns col .. of a row, those that exist; `c.left` may be made less.
// Those of fp32 are two accesses, each of half of every 32 bytes, which the L2
// joins: a hint to stream them past it costs up to 40% (16384 x 12288 decoded to
// fp32 203 -> 286 us), where 16-bit values gain by it.
template <int TYPE, bool STREAM = true, int END>
__device__ __forceinline__ void store8(GLOBAL char* row, int col, const Cols<END>& c, const float* s) {
  const int left = c.left;
  if (left <= 0) return;
  Raw8<TYPE> r;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (TYPE == PS_TYPE_F32)
      r.w[j / 4][j % 4] = __float_as_uint(s[j]);
    else if (j % 2 == 0)
      r.w[0][j / 2] = round2<TYPE>(s[j], s[j + 1]);
  }
  GLOBAL char* at = row + (uint32_t)(col * kBytes<TYPE>);
  if (END == kWhole || left >= 8) {
    GLOBAL u32x4_any* p = (GLOBAL u32x4_any*)at;
#pragma unroll
    for (int i = 0; i < (int)sizeof(r.w) / 16; ++i) {
      if (STREAM && TYPE != PS_TYPE_F32)
        __builtin_nontemporal_store((u32x4_any)r.w[i], p + i);
      else
        p[i] = r.w[i];
    }
    return;
  }
  // the end of a row: four, two and one of what is left
  if (TYPE == PS_TYPE_F32) {
    if (left & 4) {
      *(GLOBAL u32x4_any*)at = r.w[0];
      r.w[0] = r.w[TYPE == PS_TYPE_F32 ? 1 : 0];
      at += 16;
    }
    if (left & 2) {
      *(GLOBAL u32x2_any*)at = u32x2_any{r.w[0][0], r.w[0][1]};
      r.w[0][0] = r.w[0][2];
      at += 8;
    }
    if (left & 1) *(GLOBAL uint32_t*)at = r.w[0][0];
  } else {
    if (left & 4) {
      *(GLOBAL u32x2_any*)at = u32x2_any{r.w[0][0], r.w[0][1]};
      r.w[0][0] = r.w[0][2];
      r.w[0][1] = r.w[0][3];
      at += 8;
    }
    if (left & 2) {
      *(GLOBAL u32_any*)at = r.w[0][0];
      r.w[0][0] = r.w[0][1];
      at += 4;
    }
    if (left & 1) *(GLOBAL uint16_t*)at = (uint16_t)r.w[0][0];
  }
}

// Eight codes, as load8.
template <int END>
__device__ __forceinline__ u32x2_any load_codes8(const GLOBAL char* row, const Cols<END>& c) {
  if (END != kShort) return __builtin_nontemporal_load((const GLOBAL u32x2_any*)(row + (uint32_t)c.start));
  uint64_t w = 0;
#pragma unroll 1
  for (int j = 0; j < c.left; ++j) w = w >> 8 | (uint64_t)((const GLOBAL uint8_t*)row)[c.start + j] << 56;
  return u32x2_any{(uint32_t)w, (uint32_t)(w >> 32)};
}

template <int END>
__device__ __forceinline__ void store_codes8(GLOBAL char* row, int col, const Cols<END>& at8, u32x2_any c) {
  const int left = at8.left;
  if (left <= 0) return;
  if (END == kWhole || left >= 8) {
    __builtin_nontemporal_store(c, (GLOBAL u32x2_any*)(row + (uint32_t)col));
    return;
  }
  GLOBAL char* at = row + (uint32_t)col;
  uint32_t w = c[0];
  if (left & 4) {
    *(GLOBAL u32_any*)at = w;
    w = c[1];
    at += 4;
  }
  if (left & 2) {
    *(GLOBAL u16_any*)at = (uint16_t)w;
    w >>= 16;
    at += 2;
  }
  if (left & 1) *at = (char)w;
}

// Row r of a matrix whose rows are ld elements, or bytes, apart. Global pointers
// from here on: a uniform one with a lane's 32-bit offset is one access.
template <int TYPE>
__device__ __forceinline__ GLOBAL char* row_of(const void* p, int64_t r, int64_t ld) {
  return (GLOBAL char*)p + r * ld * kBytes<TYPE>;
}
// The same for a row that the whole workgroup or wave is at, held in scalar registers.
__device__ __forceinline__ GLOBAL char* scalar_pointer(GLOBAL char* p) {
  uint64_t u = (uint64_t)p;
  asm("" : "+s"(u));   // no instruction: keeps the lane's offset out of it
  return (GLOBAL char*)u;
}
__device__ __forceinline__ GLOBAL char* codes_of(const uint8_t* p, int64_t r, int64_t ld) { return (GLOBAL char*)p + r * ld; }

template <int END>
__device__ __forceinline__ void codes_to_f32(u32x2_any c, const Cols<END>& at, float* d) {
  if (at.left < (END == kWhole ? 1 : 8)) {
    const uint64_t w = at.left > 0 ? ((uint64_t)c[1] << 32 | c[0]) >> (8 * (8 - at.left)) : 0;
    c = u32x2_any{(uint32_t)w, (uint32_t)(w >> 32)};
  }
  e4m3_unpack4(c[0], d);
  e4m3_unpack4(c[1], d + 4);
}

// Decoded values, codes times scale. The code of a finite x may be rounded up to
// what its type does not hold: 2^16 of an fp16 x from 63488 on, and of others
// 2^128, infinite in fp32, from 1.9375 * 2^127 on. Those are the type's largest
// value, which is the nearer one to x too. Greater products (an fp16 result from
// values of another type) overflow as they would in any conversion. Only scales
// from 2^8 or 2^120 on reach so far, and SKIP passes other blocks by: that is for
// kernels with as much arithmetic as memory traffic (8192 x 11008, one 16-bit input,
// slope of SiLU or tanh's GELU 71.5 to 74.5 -> 71 us; 524288 x 64 bf16 decoded,
// where half of the lanes have nothing, 23.1 -> 22.0); the others are better off
// without a branch (fp32, two inputs: 323 -> 300 us).
template <int TYPE, bool SKIP>
__device__ __forceinline__ void decode8(float* d, float s) {
  constexpr float kFrom = TYPE == PS_TYPE_F16 ? 0x1p8f : 0x1p120f;
  constexpr float kPast = TYPE == PS_TYPE_F16 ? 0x1p16f : __builtin_inff();
  constexpr float kMost = TYPE == PS_TYPE_F16 ? 65504.0f : TYPE == PS_TYPE_BF16 ? 0x1.FEp127f : 0x1.FFFFFEp127f;
#pragma unroll
  for (int j = 0; j < 8; ++j) d[j] *= s;
  if (SKIP && !(s >= kFrom)) return;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (__builtin_fabsf(d[j]) == kPast) d[j] = __builtin_copysignf(kMost, d[j]);
}

// Eight values of a vector of any type (uniform), kept in the caches: loaded, and
// later widened, so that several vectors are under way at a time.
typedef Raw8<PS_TYPE_F32> RawVec;
template <int END>
__device__ __forceinline__ RawVec load_vec(const void* v, int type, int64_t first, const Cols<END>& c) {
  RawVec r;
  if (type == PS_TYPE_F32)
    r = load8<PS_TYPE_F32, false>(scalar_pointer(row_of<PS_TYPE_F32>(v, first, 1)), c);
  else
    r.w[0] = load8<PS_TYPE_BF16, false>(scalar_pointer(row_of<PS_TYPE_BF16>(v, first, 1)), c).w[0];
  return r;
}
template <int END>
__device__ __forceinline__ void widen_vec(const RawVec& r, int type, const Cols<END>& c, float* d) {
  if (type == PS_TYPE_F32)
    widen8<PS_TYPE_F32>(r, c, d);
  else if (type == PS_TYPE_BF16)
    widen8<PS_TYPE_BF16>(Raw8<PS_TYPE_BF16>{{r.w[0]}}, c, d);
  else
    widen8<PS_TYPE_F16>(Raw8<PS_TYPE_F16>{{r.w[0]}}, c, d);
}

// Codes and scale of a block of 128 values, eight on each of a DPP row's 16
// lanes. The scale comes from the finite values; the conversion makes NaN of the
// others (checked on the GPU).
__device__ __forceinline__ u32x2_any encode_block(const float* x, float& s) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t u = __float_as_uint(x[j]) & 0x7FFFFFFFu;
    top = __builtin_elementwise_max(top, u < 0x7F800000u ? u : 0u);
  }
  top = __builtin_elementwise_max(top, dpp_u32<0xB1>(top));
  top = __builtin_elementwise_max(top, dpp_u32<0x4E>(top));
  top = __builtin_elementwise_max(top, dpp_u32<0x141>(top));
  top = __builtin_elementwise_max(top, dpp_u32<0x140>(top));
  float inv;
  e4m3_scale(top, s, inv);
  u32x2_any c;
  c[0] = e4m3_pack4(x, s);
  c[1] = e4m3_pack4(x + 4, s);
  return c;
}

// Sums over a DPP row's 16 lanes and over the wave, on every lane, always in the
// same order.
__device__ __forceinline__ float row16_sum(float x) {
  x += dpp<0xB1>(x);
  x += dpp<0x4E>(x);
  x += dpp<0x141>(x);
  x += dpp<0x140>(x);
  return x;
}

__device__ __forceinline__ float wave_sum(float x) {
  x = row16_sum(x);
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

}  // namespace ps
