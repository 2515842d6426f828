// k_adamw.hip - AdamW over a plan's tensors with fp32 or e4m3 moments, the
// global gradient norm, and the e4m3 moment codec.
//
// Every kernel here streams its arrays through once and is bound by HBM, or by
// the vector units where random bits are drawn. Step: one work item of 512
// elements (two moment blocks) is one 64-lane wave in a workgroup of its own;
// the item's tensor is found by a binary search over scalar loads.
#include "dev_adamw.h"
#include "ps_adamw.h"

namespace ps {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// Constant address space: wave-uniform reads through it are scalar loads. The
// tables are written between kernels only.
#define CONSTANT __attribute__((address_space(4)))

template <class T>
__device__ __forceinline__ T ld_const(const T* p) {
  uint64_t w[sizeof(T) / 8];
  static_assert(sizeof(T) % 8 == 0, "whole words");
#pragma unroll
  for (int k = 0; k < (int)(sizeof(T) / 8); ++k) w[k] = ((const CONSTANT uint64_t*)p)[k];
  T t;
  __builtin_memcpy(&t, w, sizeof(T));
  return t;
}

typedef GLOBAL char* gptr;   // an address in HBM: a wave-uniform one in it keeps the lane offsets at 32 bits

template <class T>
__device__ __forceinline__ gptr global(T* p) { return (gptr)(GLOBAL T*)p; }
template <class T>
__device__ __forceinline__ gptr global(const T* p) { return (gptr)(GLOBAL T*)p; }

template <class V>
__device__ __forceinline__ V ld_nt(gptr p) {
  return __builtin_nontemporal_load((const GLOBAL V*)p);
}
template <class V>
__device__ __forceinline__ void st_nt(gptr p, V v) {
  __builtin_nontemporal_store(v, (GLOBAL V*)p);
}

// ---------------------------------------------------------------------------
// R consecutive elements (4 or 8) of a run that starts `off` elements behind a
// wave-uniform pointer with `left` elements behind it; R divides off, and the
// addresses are R-element aligned. FULL: all of them exist. Otherwise elements
// at `left` and beyond read as zero and are not written.
// ---------------------------------------------------------------------------
template <int R, bool FULL>
__device__ __forceinline__ void ld_f32(gptr p, uint32_t off, uint32_t left, float* d) {
  const gptr q = p + off * 4u;
  if (FULL || off + R <= left) {
#pragma unroll
    for (int k = 0; k < R; k += 4) {
      const f32x4 a = ld_nt<f32x4>(q + 4 * k);
      d[k] = a.x; d[k + 1] = a.y; d[k + 2] = a.z; d[k + 3] = a.w;
    }
    return;
  }
  for (int j = 0; j < R; ++j) d[j] = off + j < left ? ((const GLOBAL float*)q)[j] : 0.0f;
}

template <int R, bool FULL>
__device__ __forceinline__ void st_f32(gptr p, uint32_t off, uint32_t left, const float* s) {
  const gptr q = p + off * 4u;
  if (FULL || off + R <= left) {
#pragma unroll
    for (int k = 0; k < R; k += 4) st_nt(q + 4 * k, f32x4{s[k], s[k + 1], s[k + 2], s[k + 3]});
    return;
  }
  for (int j = 0; j < R; ++j)
    if (off + j < left) ((GLOBAL float*)q)[j] = s[j];
}

template <int R, bool FULL>
__device__ __forceinline__ void ld_u16(gptr p, uint32_t off, uint32_t left, uint32_t* d) {
  const gptr q = p + off * 2u;
  if (FULL || off + R <= left) {
    if (R == 8) {
      const u32x4 a = ld_nt<u32x4>(q);
      d[0] = a.x; d[1] = a.y; d[2] = a.z; d[3] = a.w;
    } else {
      const u32x2 a = ld_nt<u32x2>(q);
      d[0] = a.x; d[1] = a.y;
    }
    return;
  }
  for (int j = 0; j < R / 2; ++j) {
    const uint32_t lo = off + 2 * j < left ? ((const GLOBAL uint16_t*)q)[2 * j] : 0u;
    const uint32_t hi = off + 2 * j + 1 < left ? ((const GLOBAL uint16_t*)q)[2 * j + 1] : 0u;
    d[j] = lo | (hi << 16);
  }
}

template <int R, bool FULL>
__device__ __forceinline__ void st_u16(gptr p, uint32_t off, uint32_t left, const uint32_t* s) {
  const gptr q = p + off * 2u;
  if (FULL || off + R <= left) {
    if (R == 8)
      st_nt(q, u32x4{s[0], s[1], s[2], s[3]});
    else
      st_nt(q, u32x2{s[0], s[1]});
    return;
  }
  for (int j = 0; j < R; ++j)
    if (off + j < left) ((GLOBAL uint16_t*)q)[j] = (uint16_t)(s[j >> 1] >> (16 * (j & 1)));
}

template <int R, bool FULL>
__device__ __forceinline__ void ld_u8(gptr p, uint32_t off, uint32_t left, uint32_t* d) {
  const gptr q = p + off;
  if (FULL || off + R <= left) {
    if (R == 8) {
      const u32x2 a = ld_nt<u32x2>(q);
      d[0] = a.x; d[1] = a.y;
    } else {
      d[0] = ld_nt<uint32_t>(q);
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < R / 4; ++k) d[k] = 0u;
  for (int j = 0; j < R; ++j)
    if (off + j < left) d[j >> 2] |= (uint32_t)((const GLOBAL uint8_t*)q)[j] << (8 * (j & 3));
}

template <int R, bool FULL>
__device__ __forceinline__ void st_u8(gptr p, uint32_t off, uint32_t left, const uint32_t* s) {
  const gptr q = p + off;
  if (FULL || off + R <= left) {
    if (R == 8)
      st_nt(q, u32x2{s[0], s[1]});
    else
      st_nt(q, s[0]);
    return;
  }
  for (int j = 0; j < R; ++j)
    if (off + j < left) ((GLOBAL uint8_t*)q)[j] = (uint8_t)(s[j >> 2] >> (8 * (j & 3)));
}

// Eight 16-bit floats (bf16, or fp16 if `half`) as fp32.
template <int N>
__device__ __forceinline__ void unpack(const uint32_t* w, bool half, float* d) {
  if (half) {
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
      const f16x2 h = __builtin_bit_cast(f16x2, w[j]);
      d[2 * j] = (float)h.x;
      d[2 * j + 1] = (float)h.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
      d[2 * j] = bf16_lo(w[j]);
      d[2 * j + 1] = bf16_hi(w[j]);
    }
  }
}

// Eight fp32 values rounded to nearest even as bf16, or fp16 if `half`.
template <int N>
__device__ __forceinline__ void pack(const float* s, bool half, uint32_t* w) {
  if (half) {
#pragma unroll
    for (int j = 0; j < N / 2; ++j)
      w[j] = __builtin_bit_cast(uint32_t, f16x2{(_Float16)s[2 * j], (_Float16)s[2 * j + 1]});
  } else {
#pragma unroll
    for (int j = 0; j < N / 2; ++j)
      w[j] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)s[2 * j], (__bf16)s[2 * j + 1]});
  }
}

// ---------------------------------------------------------------------------
// step
// ---------------------------------------------------------------------------

constexpr uint32_t kVStream = 0x80000000u;   // second moment's random streams: list index + 2^31

// Lane layout of a kind: fp32 arrays (moments, or the weights beside 8-bit
// moments) are read best by runs of 4, bf16 weights with 8-bit moments by runs
// of 8. Layer of 202M parameters, fp32 weights, bf16 gradients and copy: fp32
// moments 963 us by 4, 1130 us by 8; e4m3 moments 578 us by 4, 632 us by 8.
// bf16 weights with residual and e4m3 moments, 514M: 1131 us by 8, 1146 us by 4.
constexpr bool quad_lanes(int kind) { return !(kind & kAwE4m3) || !(kind & kAwBf16); }

// Waves a SIMD runs at once, held down on purpose: with fewer waves in flight
// the streams' reads and writes meet less in HBM, and as long as the
// arithmetic stays hidden that is worth more than latency. The 202M layer with
// fp32 moments took 1020, 890, 920, 946, 953 and 995 us at 1, 2, 3, 4, 5 and 8
// waves; 298M bf16 weights rounded stochastically, fp32 moments 1020, 1039 and 1061
// us at 2, 3 and 4; 514M bf16 weights with e4m3 moments 1459, 1188, 1138, 1150 and
// 1180 us at 2, 3, 4, 5 and 8: about 15 KB of loads in flight a SIMD for all. Where
// weights are rounded stochastically beside e4m3 moments, integer work for the
// random bits fills the vector units and wants as many waves as have registers (42M
// parameters, both rounded so: 87, 83, 79 and 77 us at 4, 5, 6 and 7 waves; 8 spill,
// 83 us). Each row was measured in turn on one card with the arithmetic of its
// time; cards differ by up to 3%.
constexpr int waves_of(int kind, int split) {
  return !(kind & kAwE4m3) ? 2 : (kind & kAwBf16) && split == PS_SPLIT_STOCHASTIC ? 7 : 4;
}

// Each XCD takes runs of this many consecutive items. At the waves above runs
// of 256 to 1024 measured alike, 64 and 2048 2-4% slower.
constexpr uint32_t kAwXcdChunk = 512;

// A lane's 8 elements of a work item. QUAD: two runs of 4, one in each block,
// so that 64 lanes read 1 KiB of fp32 in one contiguous access. Else one run of
// 8, 32 lanes to a block. p0 is the item's first element of an array.
template <bool QUAD, bool FULL>
struct Lane {
  static constexpr int R = QUAD ? 4 : 8;
  static constexpr int kBlocks = QUAD ? 2 : 1;
  static constexpr int block_of(int j) { return QUAD ? j / 4 : 0; }
  uint32_t off, left;
  __device__ __forceinline__ Lane(uint32_t left_) : off(threadIdx.x * R), left(left_) {}
#define PS_EACH(CALL, D)                                                                 \
  {                                                                                      \
    CALL<R, FULL>(p0, off, left, d);                                                     \
    if (QUAD) CALL<R, FULL>(p0, off + 256, left, d + D);                                 \
  }
  __device__ __forceinline__ void load_f32(gptr p0, float* d) const PS_EACH(ld_f32, 4)
  __device__ __forceinline__ void store_f32(gptr p0, const float* d) const PS_EACH(st_f32, 4)
  __device__ __forceinline__ void load_u16(gptr p0, uint32_t* d) const PS_EACH(ld_u16, 2)
  __device__ __forceinline__ void store_u16(gptr p0, const uint32_t* d) const PS_EACH(st_u16, 2)
  __device__ __forceinline__ void load_u8(gptr p0, uint32_t* d) const PS_EACH(ld_u8, 1)
  __device__ __forceinline__ void store_u8(gptr p0, const uint32_t* d) const PS_EACH(st_u8, 1)
#undef PS_EACH
  // Block b of the lane: its index in the item, and whether it has elements.
  __device__ __forceinline__ uint32_t block(int b) const { return QUAD ? (uint32_t)b : threadIdx.x >> 5; }
  __device__ __forceinline__ bool exists(int b) const { return FULL || block(b) * kBlock < left; }
  __device__ __forceinline__ uint32_t block_max(uint32_t x) const { return QUAD ? wave_max_u32(x) : row32_max_u32(x); }
  __device__ __forceinline__ bool leads() const { return (threadIdx.x & (QUAD ? 63 : 31)) == 0; }
};

// Random bits of a lane's two quads: outputs e/4 of the stream (dev_common.h).
// The stream's start and the item's part of the counter are wave-uniform.
template <bool QUAD>
__device__ __forceinline__ void random_quads(const AwScalars& c, uint32_t tid, int64_t elem0, uint64_t* z) {
  const uint64_t base = sr_stream(c.sr_seed, c.sr_step, tid) + ((uint64_t)(elem0 >> 2) + 1) * kGolden;
  const uint64_t x = base + (uint64_t)(threadIdx.x * (QUAD ? 1 : 2)) * kGolden;
  z[0] = splitmix64_mix(x);
  z[1] = splitmix64_mix(x + (QUAD ? 64 : 1) * kGolden);
}

// The item's elements elem0 .. elem0 + left - 1 of the tensor, left <= 512.
template <int KIND, int SPLIT, bool NADAM, bool FULL>
__device__ __forceinline__ void adamw_item(const AwRec& T, int64_t elem0, uint32_t left, const AwScalars& c, float mul,
                                           const AwRun& run) {
  constexpr bool BF = KIND & kAwBf16, G32 = KIND & kAwGrad32, E8 = KIND & kAwE4m3, CP = KIND & kAwCopy;
  constexpr bool SR = BF && SPLIT == PS_SPLIT_STOCHASTIC;
  constexpr bool QUAD = quad_lanes(KIND);
  using L = Lane<QUAD, FULL>;
  const L at(left);
  const gptr wp = global((char*)T.w) + elem0 * (BF ? 2 : 4);
  const gptr lp = global((char*)T.lo) + elem0 * 2;
  const gptr gp = global((const char*)T.g) + elem0 * (G32 ? 4 : 2);
  const gptr mp = global((char*)T.m) + elem0 * (E8 ? 1 : 4);
  const gptr vp = global((char*)T.v) + elem0 * (E8 ? 1 : 4);
  GLOBAL float* const msp = (GLOBAL float*)T.ms + (elem0 >> 8);
  GLOBAL float* const vsp = (GLOBAL float*)T.vs + (elem0 >> 8);

  float g[8], w[8], m[8], v[8];
  uint32_t gw[4], hw[4], lw[4], mc[2], vc[2];
  float ms[2] = {0.0f, 0.0f}, vs[2] = {0.0f, 0.0f};
  if (G32)
    at.load_f32(gp, g);
  else
    at.load_u16(gp, gw);
  if (E8) {
    at.load_u8(mp, mc);
    at.load_u8(vp, vc);
#pragma unroll
    for (int b = 0; b < L::kBlocks; ++b)
      if (at.exists(b)) {
        ms[b] = msp[at.block(b)];
        vs[b] = vsp[at.block(b)];
      }
  } else {
    at.load_f32(mp, m);
    at.load_f32(vp, v);
  }
  if (BF) {
    at.load_u16(wp, hw);
    if (!SR) at.load_u16(lp, lw);
  } else {
    at.load_f32(wp, w);
  }

  if (!G32) unpack<8>(gw, T.gtype == PS_TYPE_F16, g);
  if (E8) {
    // The whole scale counts, as in ps_decode_fp8: the conversion that takes a
    // scale reads only its exponent. (It saves 0.5 of 75.2 us for 42M weights and
    // second moments rounded stochastically, and nothing for the other kinds.)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      e4m3_unpack4(mc[q], m + 4 * q);
      e4m3_unpack4(vc[q], v + 4 * q);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int b = L::block_of(j);
      m[j] = m[j] * ms[b];
      const float r = v[j] * vs[b];
      v[j] = r * r;
    }
  }

  // Moments, and what decides whether the fast square root and quotient hold
  // for the whole wave: the least and largest v and |numerator| above zero.
  uint32_t mx_v[2] = {0u, 0u}, least_v = ~0u, least_a = ~0u;
  float mx_m[2] = {0.0f, 0.0f}, mx_a = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int b = L::block_of(j);
    const float gj = g[j] * mul;
    m[j] = c.B1 * m[j] + c.C1 * gj;
    v[j] = c.B2 * v[j] + c.C2 * (gj * gj);
    mx_v[b] = __builtin_elementwise_max(mx_v[b], __float_as_uint(v[j]));
    least_v = __builtin_elementwise_min(least_v, __float_as_uint(v[j]) - 1u);
    if (E8 || !NADAM) mx_m[b] = __builtin_fmaxf(mx_m[b], __builtin_fabsf(m[j]));
    if (NADAM) {
      g[j] = c.AG * gj + c.AM * m[j];   // the numerator
      mx_a = __builtin_fmaxf(mx_a, __builtin_fabsf(g[j]));
    }
    least_a = __builtin_elementwise_min(least_a, (__float_as_uint(NADAM ? g[j] : m[j]) << 1) - 1u);
  }
  if (!NADAM) mx_a = __builtin_fmaxf(mx_m[0], mx_m[1]);
  // v: 0 or in [2^-96, 2^60); a: 0 or |a| in [2^-60, 2^60). With EPS in
  // [2^-60, 2^58] and RS2 <= 2^28 (run.fast) d stays in [2^-60, 2^60].
  const bool out = least_v < ((127u - 96u) << 23) - 1u || least_a < ((127u - 60u) << 24) - 1u ||
                   __builtin_elementwise_max(mx_v[0], mx_v[1]) >= ((127u + 60u) << 23) || !(mx_a < 0x1p60f);
  const bool fast = run.fast && __builtin_amdgcn_ballot_w64(out) == 0;
  if (BF) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      w[j] = SR ? ((j & 1) ? bf16_hi(hw[j >> 1]) : bf16_lo(hw[j >> 1]))
                : __uint_as_float(join_pair_elem<SPLIT>(hw[j >> 1], lw[j >> 1], j & 1));
  }
  float vv[8];
  if (!E8) {
#pragma unroll
    for (int j = 0; j < 8; ++j) vv[j] = v[j];
  }
  if (fast) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = sqrt_fast(v[j]);
      const float q = div_fast(NADAM ? g[j] : m[j], v[j] * c.RS2 + c.EPS);
      w[j] = w[j] - ((NADAM ? q : c.A * q) + c.CWD * w[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      __builtin_amdgcn_sched_barrier(0);   // one element at a time: the rare path needs no registers of its own
      v[j] = __builtin_sqrtf(v[j]);
      const float q = (NADAM ? g[j] : m[j]) / (v[j] * c.RS2 + c.EPS);
      w[j] = w[j] - ((NADAM ? q : c.A * q) + c.CWD * w[j]);
    }
  }

  if (BF) {
    uint32_t oh[4], ol[4];
    if (SR) {
      uint64_t z[2];
      random_quads<QUAD>(c, T.tid, elem0, z);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        oh[q] = sr_pair(__float_as_uint(w[2 * q]), __float_as_uint(w[2 * q + 1]), random16(z[q >> 1], 2 * (q & 1)),
                        random16(z[q >> 1], 2 * (q & 1) + 1));
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        split_pair<SPLIT>(__float_as_uint(w[2 * q]), __float_as_uint(w[2 * q + 1]), oh[q], ol[q]);
      at.store_u16(lp, ol);
    }
    at.store_u16(wp, oh);
  } else {
    at.store_f32(wp, w);
    if (CP) {
      uint32_t oc[4];
      pack<8>(w, T.ctype == PS_TYPE_F16, oc);
      at.store_u16(global((char*)T.copy) + elem0 * 2, oc);
    }
  }
  if (!E8) {
    at.store_f32(mp, m);
    at.store_f32(vp, vv);
    return;
  }

  // Block scales: the largest |m|, and the root of the largest v, which is the
  // largest root.
  float sm[2], sv[2], inv_m[2], inv_v[2];
#pragma unroll
  for (int b = 0; b < L::kBlocks; ++b) {
    e4m3_scale(at.block_max(__float_as_uint(mx_m[b])), sm[b], inv_m[b]);
    const float top = __uint_as_float(at.block_max(mx_v[b]));
    e4m3_scale(__float_as_uint(fast ? sqrt_fast(top) : __builtin_sqrtf(top)), sv[b], inv_v[b]);
  }
  const uint32_t om[2] = {e4m3_pack4(m, sm[0]), e4m3_pack4(m + 4, sm[L::block_of(4)])};
  at.store_u8(mp, om);

  // Roots below 2^-6 of their scale, rare, take the general form; so do blocks
  // of zeros. The others are cut as they are: no root above zero is subnormal
  // (the least is 2^-74.5), so the scale moves only their exponent.
  bool small = false;
#pragma unroll
  for (int b = 0; b < L::kBlocks; ++b) {
    float least = v[4 * b];
#pragma unroll
    for (int j = 1; j < 8 / L::kBlocks; ++j) least = __builtin_fminf(least, v[4 * b + j]);
    small |= least < 0x1p-6f * sv[b];
  }
  small = __builtin_amdgcn_ballot_w64(small) != 0;
  uint64_t z[2] = {0u, 0u};
  if (run.round_sr) random_quads<QUAD>(c, T.tid | kVStream, elem0, z);
  uint32_t ov[2];
  if (!small) {
    if (run.round_sr) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = e4m3_cut(v[j], z[j >> 2], j & 3);
    }
    ov[0] = e4m3_pack4(v, sv[0]);
    ov[1] = e4m3_pack4(v + 4, sv[L::block_of(4)]);
  } else {
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      y[j] = v[j] * inv_v[L::block_of(j)];
      if (run.round_sr) y[j] = e4m3_stochastic(y[j], z[j >> 2], j & 3);
      y[j] = v[j] > 0.0f ? __builtin_fmaxf(y[j], kMinCode) : y[j];
    }
    ov[0] = e4m3_pack4(y);
    ov[1] = e4m3_pack4(y + 4);
  }
  at.store_u8(vp, ov);
#pragma unroll
  for (int b = 0; b < L::kBlocks; ++b)
    if (at.leads() && at.exists(b)) {
      msp[at.block(b)] = sm[b];
      vsp[at.block(b)] = sv[b];
    }
}

// Index of the record that owns work item `item` (prefix ends, wave-uniform).
__device__ __forceinline__ int find(const uint32_t* ends, int n, uint32_t item) {
  const CONSTANT uint32_t* end = (const CONSTANT uint32_t*)ends;
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (end[mid] > item)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// One step of one kind of tensors. 202M fp32 weights with bf16 gradients and
// copy and fp32 moments take 898 us (6.3 TB/s), 514M bf16 weights with residuals and
// e4m3 moments 1150 us (6.3 TB/s), both bound by HBM; 42M bf16 weights with e4m3
// moments, both rounded stochastically, 75 us (5.6 TB/s), bound by the vector units.
template <int KIND, int SPLIT, bool NADAM>
__global__ __launch_bounds__(64) __attribute__((amdgpu_waves_per_eu(
    waves_of(KIND, SPLIT), waves_of(KIND, SPLIT)))) void k_adamw_step(AwTable t, AwGroups sc, AwRun run) {
  const uint32_t item = xcd_item<kAwXcdChunk>(blockIdx.x, gridDim.x);
  const int i = find(t.item_end, t.n, item);
  const AwRec T = ld_const(t.recs + i);
  if (!T.g) return;
  float mul = 1.0f;
  if (run.clipped) {
    const CONSTANT ps_adamw_control* ctl = (const CONSTANT ps_adamw_control*)run.ctl;
    if (ctl->skip) return;
    mul = ctl->grad_mul;
  }
  const uint32_t begin = i ? t.item_end[i - 1] : 0u;
  const AwScalars c = run.dev_sc ? ld_const(run.dev_sc + T.group) : sc.g[T.group];
  const int64_t elem0 = (int64_t)(item - begin) * kAwItemElems;
  const int64_t left = T.n - elem0;
  if (left >= kAwItemElems)
    adamw_item<KIND, SPLIT, NADAM, true>(T, elem0, kAwItemElems, c, mul, run);
  else
    adamw_item<KIND, SPLIT, NADAM, false>(T, elem0, (uint32_t)left, c, mul, run);
}

// Step counted on the device: one lane per group computes the update's scalars
// in double, as the host does for a step number.
__global__ __launch_bounds__(64) void k_adamw_tick(ps_adamw_control* ctl, AwScalars* sc, AwTick hp, int n_groups,
                                                   int clipped) {
  if (clipped && ctl->skip) return;
  const int64_t t = ctl->step + 1;
  const float lr_mul = ctl->lr_mul;
  __syncthreads();   // every lane has read the old step
  const int i = (int)threadIdx.x;
  if (i == 0) ctl->step = t;
  if (i >= n_groups) return;
  const double lr = hp.lr[i] * (double)lr_mul, b1 = hp.beta1[i], b2 = hp.beta2[i];
  AwScalars c;
  c.B1 = (float)b1;
  c.C1 = (float)(1.0 - b1);
  c.B2 = (float)b2;
  c.C2 = (float)(1.0 - b2);
  c.EPS = (float)hp.eps[i];
  c.A = (float)(lr / (1.0 - pow(b1, (double)t)));
  c.RS2 = (float)(1.0 / sqrt(1.0 - pow(b2, (double)t)));
  c.AG = 0.0f;
  c.AM = 0.0f;
  c.CWD = (float)(lr * hp.wd[i]);
  c.sr_step = (uint32_t)t;
  c.pad = 0;
  c.sr_seed = hp.seed[i];
  sc[i] = c;
}

// ---------------------------------------------------------------------------
// gradient norm
// ---------------------------------------------------------------------------

constexpr int kNormThreads = 256;
static_assert(kNormCounts < kNormThreads, "one thread clears each count");

// Sum of the workgroup's values in lane order; valid in thread 0.
__device__ __forceinline__ double block_sum(double x) {
  __shared__ double part[kNormThreads / 64];
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) x += __shfl_down(x, d, 64);
  __syncthreads();   // a sum before this one has been read
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < kNormThreads / 64; ++i) s += part[i];
  return s;
}

// Adds the squares of eight gradients to four sums.
__device__ __forceinline__ void add_squares(const float* g, double* s) {
#pragma unroll
  for (int j = 0; j < 8; ++j) s[j & 3] = __builtin_fma((double)g[j], (double)g[j], s[j & 3]);
}

template <bool KEEP, class V>
__device__ __forceinline__ V ld_norm(gptr p) {
  return KEEP ? *(const GLOBAL V*)p : ld_nt<V>(p);
}

// A whole chunk's squares: every load is under way before the first is used,
// and `meanwhile` runs while they are. KEEP: the loads may stay in the caches.
template <bool KEEP, class F>
__device__ __forceinline__ void chunk_squares(gptr p, bool f32, bool half, double* s, F meanwhile) {
  constexpr int kLoads = kNormChunk / (8 * kNormThreads);   // of 8 elements
  if (f32) {
    f32x4 x[2 * kLoads];
#pragma unroll
    for (int k = 0; k < 2 * kLoads; ++k) x[k] = ld_norm<KEEP, f32x4>(p + (threadIdx.x * 16u + k * (16u * kNormThreads)));
    meanwhile();
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      const float g[8] = {x[2 * k].x,     x[2 * k].y,     x[2 * k].z,     x[2 * k].w,
                          x[2 * k + 1].x, x[2 * k + 1].y, x[2 * k + 1].z, x[2 * k + 1].w};
      add_squares(g, s);
    }
  } else {
    u32x4 x[kLoads];
#pragma unroll
    for (int k = 0; k < kLoads; ++k) x[k] = ld_norm<KEEP, u32x4>(p + (threadIdx.x * 16u + k * (16u * kNormThreads)));
    meanwhile();
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
      float g[8];
      unpack<8>(w, half, g);
      add_squares(g, s);
    }
  }
}

// Where a chunk's gradients are; left = 0 behind the last chunk and where a
// tensor has none.
struct Chunk {
  gptr p;
  uint32_t left;
  int32_t gtype;
};
__device__ __forceinline__ Chunk norm_chunk(const AwNormTable& t, uint32_t chunk) {
  if (chunk >= t.chunks) return Chunk{nullptr, 0, 0};
  const int i = find(t.chunk_end, t.n, chunk);
  const AwNormRec T = ld_const(t.recs + i);
  const uint32_t begin = i ? ((const CONSTANT uint32_t*)t.chunk_end)[i - 1] : 0u;
  const int64_t e0 = (int64_t)(chunk - begin) * kNormChunk, left = T.n - e0;
  return Chunk{global((const char*)T.g) + e0 * (T.gtype == PS_TYPE_F32 ? 4 : 2),
               T.g ? (uint32_t)(left < kNormChunk ? left : kNormChunk) : 0u, T.gtype};
}

// Workgroup b sums the squares of the chunks b, b + gridDim.x, ... in double:
// no finite gradient's square overflows or vanishes there, and a sum that is
// not finite says that a gradient is not. The workgroup that comes last adds
// the partial sums, in index order whichever it is, and writes the control
// block, so that there is one launch.
//
// The gradients' last kNormKeepBytes, of whole chunks, are read without the
// non-temporal hint and stay in the last-level cache (norm_keep.h); the step,
// whose own streams carry the hint, finds them there (norm and step of a 202M
// layer with e4m3 moments: 576, 560, 553 and 549 us for 0, 128, 192 and 256 MiB).
// The others carry it: without any the norm of 514M fp32 gradients takes 335 us,
// with all 296, with these 299; 42M bf16 gradients, which are all kept, take
// 18 us for the 16.9 below.
//
// The last one is found by counting: each workgroup counts on one of kNormCounts
// addresses, the last of those on a common one. (An address takes about 10 ns
// for a count: 2048 workgroups on a single one took 36 us for 42M bf16 gradients,
// a second launch for the sum 18.0 us, this 17.8 us, and 17.2 us with 1024
// workgroups of equal shares; 64 tensors of 8192 5.3, 7.0 and 4.9 us.) A chunk's
// record is looked up while the loads of the one before are under way: 16.9 us,
// and 296 us for 514M fp32 gradients, 301 us without. Partial sums and counts
// cross XCDs: they go through agent-scope atomics, which write through
// the XCD's L2, and a workgroup counts when its partial sum has arrived (a
// release per workgroup, which writes the whole L2 back, cost 70 us more). The
// last workgroup sets the counts back to 0.
__global__ __launch_bounds__(kNormThreads) void k_grad_norm(AwNormTable t, double* partials, uint32_t* counts,
                                                            ps_adamw_control* ctl, double max_norm, double grad_scale) {
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  uint32_t chunk = blockIdx.x;
  Chunk at = norm_chunk(t, chunk);
  while (chunk < t.chunks) {
    const Chunk now = at;
    const bool keep = chunk >= t.keep_from;
    chunk += gridDim.x;
    auto next = [&] { at = norm_chunk(t, chunk); };
    const bool f32 = now.gtype == PS_TYPE_F32, half = now.gtype == PS_TYPE_F16;
    const gptr p = now.p;
    if (now.left == kNormChunk) {
      if (keep)
        chunk_squares<true>(p, f32, half, s, next);
      else
        chunk_squares<false>(p, f32, half, s, next);
      continue;
    }
    next();
    const uint32_t left = now.left;
    for (uint32_t off = threadIdx.x * 8; off < left; off += 8 * kNormThreads) {
      float g[8];
      if (f32) {
        ld_f32<8, false>(p, off, left, g);
      } else {
        uint32_t w[4];
        ld_u16<8, false>(p, off, left, w);
        unpack<8>(w, half, g);
      }
      add_squares(g, s);
    }
  }
  double sum = block_sum((s[0] + s[1]) + (s[2] + s[3]));
  const uint32_t n = gridDim.x;
  if (n > 1) {
    __shared__ bool last;
    if (threadIdx.x == 0) {
      __hip_atomic_store(partials + blockIdx.x, sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      const uint32_t c = blockIdx.x % kNormCounts;
      const uint32_t of_c = (n - c + kNormCounts - 1) / kNormCounts, of_all = n < kNormCounts ? n : kNormCounts;
      last = __hip_atomic_fetch_add(counts + (1 + c) * kNormCountStride, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                 of_c - 1 &&
             __hip_atomic_fetch_add(counts, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == of_all - 1;
    }
    __syncthreads();
    if (!last) return;
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    sum = 0.0;
    for (uint32_t i = threadIdx.x; i < n; i += kNormThreads)
      sum += __hip_atomic_load(partials + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    sum = block_sum(sum);
    if (threadIdx.x <= kNormCounts) counts[threadIdx.x * kNormCountStride] = 0;
  }
  if (threadIdx.x != 0) return;
  const double norm = grad_scale * sqrt(sum);
  const bool skip = !(norm <= 1.7976931348623157e308);   // infinite or NaN
  const double clip = max_norm / (norm + 1e-6);
  ctl->norm = (float)norm;
  ctl->grad_mul = skip ? 0.0f : (float)(grad_scale * (clip < 1.0 ? clip : 1.0));
  ctl->skip = skip ? 1u : 0u;
  if (skip) ctl->skipped += 1;
}

struct GradChunk {
  const void* g[kAwGrads];
};

// Gradient pointers of list indices base .. base+n-1 into their records.
__global__ __launch_bounds__(64) void k_set_grads(AwRec* recs, AwNormRec* nrecs, const uint32_t* slot, GradChunk c, int n) {
  const int i = (int)(blockIdx.x * 64 + threadIdx.x);
  if (i >= n) return;
  const uint32_t a = slot[2 * i], b = slot[2 * i + 1];
  if (a) recs[a - 1].g = c.g[i];
  if (b) nrecs[b - 1].g = c.g[i];
}

// ---------------------------------------------------------------------------
// e4m3 codec, on the step's items and its lanes by runs of 4. Bound by HBM.
// ---------------------------------------------------------------------------

// The encoder's wave takes this many items: 150M second moments 124 us with one,
// 116 us with two (6.5 TB/s).
constexpr int kEncodeItems = 2;

// REP consecutive items, every load under way before the first use. The least
// value above zero decides for the wave whether the fast root holds.
template <int KIND, int REP, bool FULL>
__device__ __forceinline__ void encode_items(gptr x, gptr code, GLOBAL float* scale, uint32_t left) {
  using L = Lane<true, FULL>;
  float y[REP][8];
#pragma unroll
  for (int i = 0; i < REP; ++i) L(left).load_f32(x + i * (kAwItemElems * 4), y[i]);
#pragma unroll
  for (int i = 0; i < REP; ++i) {
    const L at(left);
    float* const v = y[i];
    uint32_t mx[2] = {0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j) mx[j / 4] = __builtin_elementwise_max(mx[j / 4], __float_as_uint(v[j]) & 0x7FFFFFFFu);
    float s[2], inv[2];
    float top[2] = {__uint_as_float(at.block_max(mx[0])), __uint_as_float(at.block_max(mx[1]))};
    if (KIND == PS_MOMENT_UNSIGNED) {
      uint32_t least = ~0u;
#pragma unroll
      for (int j = 0; j < 8; ++j) least = __builtin_elementwise_min(least, __float_as_uint(v[j]) - 1u);
      if (__builtin_amdgcn_ballot_w64(least < ((127u - 96u) << 23) - 1u) == 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = sqrt_fast(v[j]);
        top[0] = sqrt_fast(top[0]);                     // the largest root
        top[1] = sqrt_fast(top[1]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __builtin_sqrtf(v[j]);
        top[0] = __builtin_sqrtf(top[0]);
        top[1] = __builtin_sqrtf(top[1]);
      }
    }
    e4m3_scale(__float_as_uint(top[0]), s[0], inv[0]);
    e4m3_scale(__float_as_uint(top[1]), s[1], inv[1]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float q = v[j] * inv[j / 4];
      v[j] = KIND == PS_MOMENT_UNSIGNED && v[j] > 0.0f ? __builtin_fmaxf(q, kMinCode) : q;
    }
    const uint32_t c[2] = {e4m3_pack4(v), e4m3_pack4(v + 4)};
    at.store_u8(code + i * kAwItemElems, c);
#pragma unroll
    for (int b = 0; b < 2; ++b)
      if (at.leads() && at.exists(b)) scale[2 * i + b] = s[b];
  }
}

template <int KIND>
__global__ __launch_bounds__(64) void k_encode_fp8(const float* x, uint8_t* code, float* scale, int64_t n) {
  const int64_t e0 = (int64_t)xcd_item<kAwXcdChunk>(blockIdx.x, gridDim.x) * (kEncodeItems * kAwItemElems);
  gptr xp = global((const char*)x) + e0 * 4, cp = global((char*)code) + e0;
  GLOBAL float* sp = (GLOBAL float*)scale + (e0 >> 8);
  if (n - e0 >= kEncodeItems * kAwItemElems) {
    encode_items<KIND, kEncodeItems, true>(xp, cp, sp, kAwItemElems);
    return;
  }
  for (int64_t left = n - e0; left > 0; left -= kAwItemElems) {
    encode_items<KIND, 1, false>(xp, cp, sp, (uint32_t)(left < kAwItemElems ? left : kAwItemElems));
    xp += kAwItemElems * 4;
    cp += kAwItemElems;
    sp += kAwItemElems / kBlock;
  }
}

template <int KIND, bool FULL>
__device__ __forceinline__ void decode_item(gptr code, const GLOBAL float* scale, gptr x, uint32_t left) {
  using L = Lane<true, FULL>;
  const L at(left);
  uint32_t c[2];
  at.load_u8(code, c);
  float s[2] = {0.0f, 0.0f};
#pragma unroll
  for (int b = 0; b < L::kBlocks; ++b)
    if (at.exists(b)) s[b] = scale[at.block(b)];
  float y[8];
  e4m3_unpack4(c[0], y);
  e4m3_unpack4(c[1], y + 4);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    y[j] = y[j] * s[L::block_of(j)];
    if (KIND == PS_MOMENT_UNSIGNED) y[j] = y[j] * y[j];
  }
  at.store_f32(x, y);
}

template <int KIND>
__global__ __launch_bounds__(64) void k_decode_fp8(const uint8_t* code, const float* scale, float* x, int64_t n) {
  const int64_t e0 = (int64_t)xcd_item<kAwXcdChunk>(blockIdx.x, gridDim.x) * kAwItemElems;
  const gptr xp = global((char*)x) + e0 * 4, cp = global((const char*)code) + e0;
  const GLOBAL float* const sp = (const GLOBAL float*)scale + (e0 >> 8);
  if (n - e0 >= kAwItemElems)
    decode_item<KIND, true>(cp, sp, xp, kAwItemElems);
  else
    decode_item<KIND, false>(cp, sp, xp, (uint32_t)(n - e0));
}

template <int KIND, int SPLIT>
ps_status launch_t(const AwTable& t, uint32_t items, const AwGroups& sc, const AwRun& run, hipStream_t s) {
  if (run.nadam)
    hipLaunchKernelGGL((k_adamw_step<KIND, SPLIT, true>), dim3(items), dim3(64), 0, s, t, sc, run);
  else
    hipLaunchKernelGGL((k_adamw_step<KIND, SPLIT, false>), dim3(items), dim3(64), 0, s, t, sc, run);
  return hip_check(hipGetLastError(), "k_adamw_step launch");
}

}  // namespace

ps_status launch_adamw_step(int kind, int split, const AwTable& t, uint32_t items, const AwGroups& sc, const AwRun& run,
                            hipStream_t s) {
  switch (kind) {
#define PS_KIND(K) \
  case K: return launch_t<K, PS_SPLIT_TRUNC>(t, items, sc, run, s);
#define PS_KIND_BF16(K)                                                                          \
  case K:                                                                                        \
    return split == PS_SPLIT_STOCHASTIC     ? launch_t<K, PS_SPLIT_STOCHASTIC>(t, items, sc, run, s)   \
           : split == PS_SPLIT_NEAREST_AWAY ? launch_t<K, PS_SPLIT_NEAREST_AWAY>(t, items, sc, run, s) \
                                            : launch_t<K, PS_SPLIT_TRUNC>(t, items, sc, run, s);
    PS_KIND(0)
    PS_KIND(kAwGrad32)
    PS_KIND(kAwE4m3)
    PS_KIND(kAwGrad32 | kAwE4m3)
    PS_KIND(kAwCopy)
    PS_KIND(kAwGrad32 | kAwCopy)
    PS_KIND(kAwE4m3 | kAwCopy)
    PS_KIND(kAwGrad32 | kAwE4m3 | kAwCopy)
    PS_KIND_BF16(kAwBf16)
    PS_KIND_BF16(kAwBf16 | kAwGrad32)
    PS_KIND_BF16(kAwBf16 | kAwE4m3)
    PS_KIND_BF16(kAwBf16 | kAwGrad32 | kAwE4m3)
#undef PS_KIND
#undef PS_KIND_BF16
  }
  return fail(PS_ERR_UNSUPPORTED, "no kernel for tensor kind %d", kind);
}

ps_status launch_adamw_tick(ps_adamw_control* ctl, AwScalars* sc, const AwTick& hp, int n_groups, int clipped,
                            hipStream_t s) {
  hipLaunchKernelGGL(k_adamw_tick, dim3(1), dim3(64), 0, s, ctl, sc, hp, n_groups, clipped);
  return hip_check(hipGetLastError(), "k_adamw_tick launch");
}

ps_status launch_grad_norm(const AwNormTable& t, double* partials, uint32_t* counts, ps_adamw_control* ctl,
                           double max_norm, double grad_scale, hipStream_t s) {
  // every workgroup the same number of chunks, the last ones one less
  const uint32_t rounds = (t.chunks + kNormMaxWg - 1) / kNormMaxWg;
  const uint32_t wgs = rounds ? (t.chunks + rounds - 1) / rounds : 0;
  hipLaunchKernelGGL(k_grad_norm, dim3(wgs ? wgs : 1), dim3(kNormThreads), 0, s, t, partials, counts, ctl, max_norm,
                     grad_scale);
  return hip_check(hipGetLastError(), "k_grad_norm launch");
}

ps_status launch_set_grads(AwRec* recs, AwNormRec* nrecs, const uint32_t* slot, const void* const* grads, int32_t n,
                           hipStream_t s) {
  for (int32_t i = 0; i < n; i += kAwGrads) {
    const int k = n - i < kAwGrads ? n - i : kAwGrads;
    GradChunk c = {};
    for (int j = 0; j < k; ++j) c.g[j] = grads[i + j];
    hipLaunchKernelGGL(k_set_grads, dim3((k + 63) / 64), dim3(64), 0, s, recs, nrecs, slot + 2 * (size_t)i, c, k);
    if (ps_status st = hip_check(hipGetLastError(), "k_set_grads launch")) return st;
  }
  return PS_OK;
}

// Codec launches cover at most kCodecMax elements each (a launch has fewer
// than 2^32 lanes); longer arrays take several.
constexpr int64_t kCodecMax = (int64_t)kAwItemElems << 25;

ps_status launch_encode_fp8(const float* x, uint8_t* code, float* scale, int64_t n, int kind, hipStream_t s) {
  for (int64_t o = 0; o < n; o += kCodecMax) {
    const int64_t k = n - o < kCodecMax ? n - o : kCodecMax;
    const dim3 grid((uint32_t)((k + kEncodeItems * kAwItemElems - 1) / (kEncodeItems * kAwItemElems)));
    if (kind == PS_MOMENT_SIGNED)
      hipLaunchKernelGGL(k_encode_fp8<PS_MOMENT_SIGNED>, grid, dim3(64), 0, s, x + o, code + o,
                         scale + o / kBlock, k);
    else
      hipLaunchKernelGGL(k_encode_fp8<PS_MOMENT_UNSIGNED>, grid, dim3(64), 0, s, x + o, code + o,
                         scale + o / kBlock, k);
    if (ps_status st = hip_check(hipGetLastError(), "k_encode_fp8 launch")) return st;
  }
  return PS_OK;
}

ps_status launch_decode_fp8(const uint8_t* code, const float* scale, float* x, int64_t n, int kind, hipStream_t s) {
  for (int64_t o = 0; o < n; o += kCodecMax) {
    const int64_t k = n - o < kCodecMax ? n - o : kCodecMax;
    const dim3 grid((uint32_t)((k + kAwItemElems - 1) / kAwItemElems));
    if (kind == PS_MOMENT_SIGNED)
      hipLaunchKernelGGL(k_decode_fp8<PS_MOMENT_SIGNED>, grid, dim3(64), 0, s, code + o, scale + o / kBlock,
                         x + o, k);
    else
      hipLaunchKernelGGL(k_decode_fp8<PS_MOMENT_UNSIGNED>, grid, dim3(64), 0, s, code + o,
                         scale + o / kBlock, x + o, k);
    if (ps_status st = hip_check(hipGetLastError(), "k_decode_fp8 launch")) return st;
  }
  return PS_OK;
}

}  // namespace ps
