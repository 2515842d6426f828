// k_adamw.hip - AdamW over a plan's tensors with fp32 or e4m3 moments, the
// global gradient norm, and the e4m3 moment codec.
//
// Step: one work item of 512 elements is one 64-lane wave; a moment block of
// 256 elements belongs to 32 lanes, 8 consecutive elements each.
#include "dev_common.h"
#include "ps_internal.h"

namespace ps {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

template <class V>
__device__ __forceinline__ V ld_nt(const void* p) {
  return __builtin_nontemporal_load((const GLOBAL V*)p);
}
template <class V>
__device__ __forceinline__ void st_nt(void* p, V v) {
  __builtin_nontemporal_store(v, (GLOBAL V*)p);
}

// ---------------------------------------------------------------------------
// Eight consecutive elements e .. e+7 of an array of n; elements at n and
// beyond read as zero and are not written.
// ---------------------------------------------------------------------------

__device__ __forceinline__ void ld8_f32(const void* p, int64_t e, int64_t n, float* d) {
  const float* q = (const float*)p + e;
  if (e + 8 <= n) {
    const f32x4 a = ld_nt<f32x4>(q), b = ld_nt<f32x4>(q + 4);
    d[0] = a.x; d[1] = a.y; d[2] = a.z; d[3] = a.w;
    d[4] = b.x; d[5] = b.y; d[6] = b.z; d[7] = b.w;
    return;
  }
  for (int j = 0; j < 8; ++j) d[j] = e + j < n ? ((const GLOBAL float*)q)[j] : 0.0f;
}

__device__ __forceinline__ void st8_f32(void* p, int64_t e, int64_t n, const float* s) {
  float* q = (float*)p + e;
  if (e + 8 <= n) {
    st_nt(q, f32x4{s[0], s[1], s[2], s[3]});
    st_nt(q + 4, f32x4{s[4], s[5], s[6], s[7]});
    return;
  }
  for (int j = 0; j < 8; ++j)
    if (e + j < n) ((GLOBAL float*)q)[j] = s[j];
}

__device__ __forceinline__ void ld8_u16(const void* p, int64_t e, int64_t n, uint32_t* d) {
  const uint16_t* q = (const uint16_t*)p + e;
  if (e + 8 <= n) {
    const u32x4 a = ld_nt<u32x4>(q);
    d[0] = a.x; d[1] = a.y; d[2] = a.z; d[3] = a.w;
    return;
  }
  for (int j = 0; j < 4; ++j) {
    const uint32_t lo = e + 2 * j < n ? ((const GLOBAL uint16_t*)q)[2 * j] : 0u;
    const uint32_t hi = e + 2 * j + 1 < n ? ((const GLOBAL uint16_t*)q)[2 * j + 1] : 0u;
    d[j] = lo | (hi << 16);
  }
}

__device__ __forceinline__ void st8_u16(void* p, int64_t e, int64_t n, const uint32_t* s) {
  uint16_t* q = (uint16_t*)p + e;
  if (e + 8 <= n) {
    st_nt(q, u32x4{s[0], s[1], s[2], s[3]});
    return;
  }
  for (int j = 0; j < 8; ++j)
    if (e + j < n) ((GLOBAL uint16_t*)q)[j] = (uint16_t)(s[j >> 1] >> (16 * (j & 1)));
}

__device__ __forceinline__ void ld8_u8(const void* p, int64_t e, int64_t n, uint32_t* d) {
  const uint8_t* q = (const uint8_t*)p + e;
  if (e + 8 <= n) {
    const u32x2 a = ld_nt<u32x2>(q);
    d[0] = a.x; d[1] = a.y;
    return;
  }
  d[0] = d[1] = 0u;
  for (int j = 0; j < 8; ++j)
    if (e + j < n) d[j >> 2] |= (uint32_t)((const GLOBAL uint8_t*)q)[j] << (8 * (j & 3));
}

__device__ __forceinline__ void st8_u8(void* p, int64_t e, int64_t n, const uint32_t* s) {
  uint8_t* q = (uint8_t*)p + e;
  if (e + 8 <= n) {
    st_nt(q, u32x2{s[0], s[1]});
    return;
  }
  for (int j = 0; j < 8; ++j)
    if (e + j < n) ((GLOBAL uint8_t*)q)[j] = (uint8_t)(s[j >> 2] >> (8 * (j & 3)));
}

// Eight 16-bit floats (bf16, or fp16 if `half`) as fp32.
__device__ __forceinline__ void unpack8(const uint32_t* w, bool half, float* d) {
  if (half) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const f16x2 h = __builtin_bit_cast(f16x2, w[j]);
      d[2 * j] = (float)h.x;
      d[2 * j + 1] = (float)h.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      d[2 * j] = bf16_lo(w[j]);
      d[2 * j + 1] = bf16_hi(w[j]);
    }
  }
}

// Eight fp32 values rounded to nearest even as bf16, or fp16 if `half`.
__device__ __forceinline__ void pack8(const float* s, bool half, uint32_t* w) {
  if (half) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = __builtin_bit_cast(uint32_t, f16x2{(_Float16)s[2 * j], (_Float16)s[2 * j + 1]});
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)s[2 * j], (__bf16)s[2 * j + 1]});
  }
}

// ---------------------------------------------------------------------------
// e4m3 moments. The block's scale is the smallest power of two s >= 2^-126
// with max <= 448 s (448 = 1.75 * 2^8 is the largest e4m3 value): adding the
// mantissa bits above 1.75 carries into the exponent exactly when the
// mantissa is larger than 1.75. Scaling by a power of two is exact, so a code
// is one rounding of the moment, and the hardware conversion makes it.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void e4m3_scale(uint32_t max_bits, float& s, float& inv) {
  const int e = __builtin_elementwise_max((int)((max_bits + 0x1FFFFFu) >> 23) - 8, 1);
  s = __uint_as_float((uint32_t)e << 23);
  inv = __uint_as_float((uint32_t)(254 - e) << 23);
}

__device__ __forceinline__ void e4m3_unpack4(uint32_t c, float* d) {
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
  d[0] = a.x; d[1] = a.y; d[2] = b.x; d[3] = b.y;
}

__device__ __forceinline__ uint32_t e4m3_pack4(const float* y) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], lo, true);
}

constexpr float kMinCode = 0x1p-9f;   // smallest e4m3 value above zero

// y in [0, 448] cut to e4m3 after adding 16 random bits below its last kept
// place: values of 2^-6 and more keep 3 mantissa bits; smaller ones keep the
// places of 2^-6, which adding 2^-6 lines up.
__device__ __forceinline__ float e4m3_stochastic(float y, uint32_t r16) {
  const bool small = y < 0x1p-6f;
  const float z = small ? y + 0x1p-6f : y;
  const float q = __uint_as_float((__float_as_uint(z) + (r16 << 4)) & 0xFFF00000u);
  return small ? q - 0x1p-6f : q;
}

// ---------------------------------------------------------------------------
// step
// ---------------------------------------------------------------------------

constexpr uint32_t kVStream = 0x80000000u;   // second moment's random streams: list index + 2^31

template <int KIND, bool SR>
__device__ __forceinline__ void adamw_item(const AwRec& T, int64_t elem0, const AwScalars& c, float mul, const AwRun& run) {
  constexpr bool BF = KIND & kAwBf16, G32 = KIND & kAwGrad32, E8 = KIND & kAwE4m3, CP = KIND & kAwCopy;
  const int lane = (int)threadIdx.x;
  const int64_t n = T.n;
  const int64_t e = elem0 + lane * 8;
  const int64_t blk = (elem0 >> 8) + (lane >> 5);

  float g[8], w[8], m[8], v[8];
  uint32_t gw[4], hw[4], lw[4], mc[2], vc[2];
  float ms = 0.0f, vs = 0.0f;
  if (G32)
    ld8_f32(T.g, e, n, g);
  else
    ld8_u16(T.g, e, n, gw);
  if (E8) {
    ld8_u8(T.m, e, n, mc);
    ld8_u8(T.v, e, n, vc);
    if (blk * kBlock < n) {
      ms = ((const GLOBAL float*)T.ms)[blk];
      vs = ((const GLOBAL float*)T.vs)[blk];
    }
  } else {
    ld8_f32(T.m, e, n, m);
    ld8_f32(T.v, e, n, v);
  }
  if (BF) {
    ld8_u16(T.w, e, n, hw);
    if (!SR) ld8_u16(T.lo, e, n, lw);
  } else {
    ld8_f32(T.w, e, n, w);
  }

  if (!G32) unpack8(gw, T.gtype == PS_TYPE_F16, g);
  if (E8) {
    e4m3_unpack4(mc[0], m);
    e4m3_unpack4(mc[1], m + 4);
    e4m3_unpack4(vc[0], v);
    e4m3_unpack4(vc[1], v + 4);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[j] = m[j] * ms;
      const float r = v[j] * vs;
      v[j] = r * r;
    }
  }
  if (BF) {
    const uint32_t carry = run.nearest ? 0x8000u : 0u;   // nearest-away split: the residual's top bit was carried into hi
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (SR) {
        w[j] = (j & 1) ? bf16_hi(hw[j >> 1]) : bf16_lo(hw[j >> 1]);
      } else {
        const uint32_t b = perm(hw[j >> 1], lw[j >> 1], (j & 1) ? kSelHiHalves : kSelLoHalves);
        w[j] = __uint_as_float(b - ((b & carry) << 1));
      }
    }
  }

  float r[8];
  uint32_t mx_m = 0u, mx_r = 0u;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float gj = g[j] * mul;
    m[j] = c.B1 * m[j] + c.C1 * gj;
    v[j] = c.B2 * v[j] + c.C2 * (gj * gj);
    r[j] = __builtin_sqrtf(v[j]);
    const float d = r[j] * c.RS2 + c.EPS;
    float u = run.nadam ? (c.AG * gj + c.AM * m[j]) / d : c.A * (m[j] / d);
    u = u + c.CWD * w[j];
    w[j] = w[j] - u;
    if (E8) {
      mx_m = __builtin_elementwise_max(mx_m, __float_as_uint(m[j]) & 0x7FFFFFFFu);
      mx_r = __builtin_elementwise_max(mx_r, __float_as_uint(r[j]));
    }
  }

  if (BF) {
    uint32_t oh[4], ol[4];
    if (SR) {
      uint64_t rnd[2];
      sr_bits8(sr_stream(c.sr_seed, c.sr_step, T.tid), e, rnd);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t b = (uint32_t)(rnd[q >> 1] >> (32 * (q & 1)));
        oh[q] = sr_pair(__float_as_uint(w[2 * q]), __float_as_uint(w[2 * q + 1]), b & 0xFFFFu, b >> 16);
      }
    } else {
      const uint32_t carry = run.nearest ? 0x8000u : 0u;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t a = __float_as_uint(w[2 * q]), b = __float_as_uint(w[2 * q + 1]);
        ol[q] = perm(b, a, kSelLoHalves);
        oh[q] = perm(b + carry, a + carry, kSelHiHalves);
      }
      st8_u16(T.lo, e, n, ol);
    }
    st8_u16(T.w, e, n, oh);
  } else {
    st8_f32(T.w, e, n, w);
    if (CP) {
      uint32_t oc[4];
      pack8(w, T.ctype == PS_TYPE_F16, oc);
      st8_u16(T.copy, e, n, oc);
    }
  }

  if (!E8) {
    st8_f32(T.m, e, n, m);
    st8_f32(T.v, e, n, v);
    return;
  }
  float sm, inv_m, sv, inv_v;
  e4m3_scale(row32_max_u32(mx_m), sm, inv_m);
  e4m3_scale(row32_max_u32(mx_r), sv, inv_v);
  float y[8];
  uint64_t rnd[2] = {0u, 0u};
  if (run.round_sr) sr_bits8(sr_stream(c.sr_seed, c.sr_step, T.tid | kVStream), e, rnd);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    m[j] = m[j] * inv_m;
    y[j] = r[j] * inv_v;
    if (run.round_sr) y[j] = e4m3_stochastic(y[j], (uint32_t)(rnd[j >> 2] >> (16 * (j & 3))) & 0xFFFFu);
    y[j] = r[j] > 0.0f ? __builtin_fmaxf(y[j], kMinCode) : y[j];
  }
  const uint32_t om[2] = {e4m3_pack4(m), e4m3_pack4(m + 4)}, ov[2] = {e4m3_pack4(y), e4m3_pack4(y + 4)};
  st8_u8(T.m, e, n, om);
  st8_u8(T.v, e, n, ov);
  if ((lane & 31) == 0 && blk * kBlock < n) {
    ((GLOBAL float*)T.ms)[blk] = sm;
    ((GLOBAL float*)T.vs)[blk] = sv;
  }
}

// Index of the record that owns work item `item` (prefix ends, wave-uniform).
__device__ __forceinline__ int find(const uint32_t* end, int n, uint32_t item) {
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

template <int KIND, bool SR>
__global__ __launch_bounds__(64) void k_adamw_step(AwTable t, AwGroups sc, AwRun run) {
  const uint32_t item = xcd_item<>(blockIdx.x, gridDim.x);
  const int i = find(t.item_end, t.n, item);
  const AwRec& T = t.recs[i];
  if (!T.g) return;
  float mul = 1.0f;
  if (run.clipped) {
    if (run.ctl->skip) return;
    mul = run.ctl->grad_mul;
  }
  const uint32_t begin = i ? t.item_end[i - 1] : 0u;
  const AwScalars c = run.dev_sc ? run.dev_sc[T.group] : sc.g[T.group];
  adamw_item<KIND, SR>(T, (int64_t)(item - begin) * kAwItemElems, c, mul, run);
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

// Sum of the workgroup's values in lane order; valid in thread 0.
__device__ __forceinline__ double block_sum(double x) {
  __shared__ double part[kNormThreads / 64];
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) x += __shfl_down(x, d, 64);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < kNormThreads / 64; ++i) s += part[i];
  return s;
}

// Workgroup b sums the squares of the chunks b, b + gridDim.x, ... in double:
// no finite gradient's square overflows or vanishes there, and a sum that is
// not finite says that a gradient is not.
__global__ __launch_bounds__(kNormThreads) void k_grad_sumsq(AwNormTable t, double* partials) {
  double s0 = 0.0, s1 = 0.0;
  for (uint32_t chunk = blockIdx.x; chunk < t.chunks; chunk += gridDim.x) {
    const int i = find(t.chunk_end, t.n, chunk);
    const AwNormRec& T = t.recs[i];
    if (!T.g) continue;
    const uint32_t begin = i ? t.chunk_end[i - 1] : 0u;
    const int64_t e0 = (int64_t)(chunk - begin) * kNormChunk + threadIdx.x * 8;
#pragma unroll
    for (int k = 0; k < kNormChunk / (8 * kNormThreads); ++k) {
      const int64_t e = e0 + k * (8 * kNormThreads);
      if (e >= T.n) break;
      float g[8];
      if (T.gtype == PS_TYPE_F32) {
        ld8_f32(T.g, e, T.n, g);
      } else {
        uint32_t w[4];
        ld8_u16(T.g, e, T.n, w);
        unpack8(w, T.gtype == PS_TYPE_F16, g);
      }
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        s0 = __builtin_fma((double)g[j], (double)g[j], s0);
        s1 = __builtin_fma((double)g[j + 1], (double)g[j + 1], s1);
      }
    }
  }
  const double s = block_sum(s0 + s1);
  if (threadIdx.x == 0) partials[blockIdx.x] = s;
}

__global__ __launch_bounds__(kNormThreads) void k_grad_norm(const double* partials, uint32_t n, ps_adamw_control* ctl,
                                                            double max_norm, double grad_scale) {
  double s = 0.0;
  for (uint32_t i = threadIdx.x; i < n; i += kNormThreads) s += partials[i];
  s = block_sum(s);
  if (threadIdx.x != 0) return;
  const double norm = grad_scale * sqrt(s);
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
// e4m3 codec: one wave per 512 elements, laid out as the step's items
// ---------------------------------------------------------------------------
constexpr int kCodecThreads = 256;
constexpr int kCodecElems = kCodecThreads * 8;

template <int KIND>
__global__ __launch_bounds__(kCodecThreads) void k_encode_fp8(const float* __restrict__ x, uint8_t* __restrict__ code,
                                                              float* __restrict__ scale, int64_t n) {
  const int64_t e = (int64_t)blockIdx.x * kCodecElems + threadIdx.x * 8;
  float y[8];
  ld8_f32(x, e, n, y);
  uint32_t mx = 0u;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (KIND == PS_MOMENT_UNSIGNED) y[j] = __builtin_sqrtf(y[j]);
    mx = __builtin_elementwise_max(mx, __float_as_uint(y[j]) & 0x7FFFFFFFu);
  }
  float s, inv;
  e4m3_scale(row32_max_u32(mx), s, inv);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float q = y[j] * inv;
    y[j] = KIND == PS_MOMENT_UNSIGNED && y[j] > 0.0f ? __builtin_fmaxf(q, kMinCode) : q;
  }
  const uint32_t c[2] = {e4m3_pack4(y), e4m3_pack4(y + 4)};
  st8_u8(code, e, n, c);
  if ((threadIdx.x & 31) == 0 && e < n) ((GLOBAL float*)scale)[e >> 8] = s;
}

template <int KIND>
__global__ __launch_bounds__(kCodecThreads) void k_decode_fp8(const uint8_t* __restrict__ code,
                                                              const float* __restrict__ scale, float* __restrict__ x,
                                                              int64_t n) {
  const int64_t e = (int64_t)blockIdx.x * kCodecElems + threadIdx.x * 8;
  if (e >= n) return;
  uint32_t c[2];
  float y[8];
  ld8_u8(code, e, n, c);
  const float s = ((const GLOBAL float*)scale)[e >> 8];
  e4m3_unpack4(c[0], y);
  e4m3_unpack4(c[1], y + 4);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    y[j] = y[j] * s;
    if (KIND == PS_MOMENT_UNSIGNED) y[j] = y[j] * y[j];
  }
  st8_f32(x, e, n, y);
}

template <int KIND, bool SR>
ps_status launch_t(const AwTable& t, uint32_t items, const AwGroups& sc, const AwRun& run, hipStream_t s) {
  hipLaunchKernelGGL((k_adamw_step<KIND, SR>), dim3(items), dim3(64), 0, s, t, sc, run);
  return hip_check(hipGetLastError(), "k_adamw_step launch");
}

}  // namespace

ps_status launch_adamw_step(int kind, bool sr, const AwTable& t, uint32_t items, const AwGroups& sc, const AwRun& run,
                            hipStream_t s) {
  switch (kind) {
#define PS_KIND(K) \
  case K: return launch_t<K, false>(t, items, sc, run, s);
#define PS_KIND_BF16(K) \
  case K: return sr ? launch_t<K, true>(t, items, sc, run, s) : launch_t<K, false>(t, items, sc, run, s);
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

ps_status launch_grad_norm(const AwNormTable& t, double* partials, ps_adamw_control* ctl, double max_norm,
                           double grad_scale, hipStream_t s) {
  const uint32_t wgs = t.chunks < (uint32_t)kNormMaxWg ? t.chunks : (uint32_t)kNormMaxWg;
  if (wgs) {
    hipLaunchKernelGGL(k_grad_sumsq, dim3(wgs), dim3(kNormThreads), 0, s, t, partials);
    if (ps_status st = hip_check(hipGetLastError(), "k_grad_sumsq launch")) return st;
  }
  hipLaunchKernelGGL(k_grad_norm, dim3(1), dim3(kNormThreads), 0, s, partials, wgs, ctl, max_norm, grad_scale);
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
constexpr int64_t kCodecMax = (int64_t)kCodecElems << 23;

ps_status launch_encode_fp8(const float* x, uint8_t* code, float* scale, int64_t n, int kind, hipStream_t s) {
  for (int64_t o = 0; o < n; o += kCodecMax) {
    const int64_t k = n - o < kCodecMax ? n - o : kCodecMax;
    const dim3 grid((uint32_t)((k + kCodecElems - 1) / kCodecElems));
    if (kind == PS_MOMENT_SIGNED)
      hipLaunchKernelGGL(k_encode_fp8<PS_MOMENT_SIGNED>, grid, dim3(kCodecThreads), 0, s, x + o, code + o,
                         scale + o / kBlock, k);
    else
      hipLaunchKernelGGL(k_encode_fp8<PS_MOMENT_UNSIGNED>, grid, dim3(kCodecThreads), 0, s, x + o, code + o,
                         scale + o / kBlock, k);
    if (ps_status st = hip_check(hipGetLastError(), "k_encode_fp8 launch")) return st;
  }
  return PS_OK;
}

ps_status launch_decode_fp8(const uint8_t* code, const float* scale, float* x, int64_t n, int kind, hipStream_t s) {
  for (int64_t o = 0; o < n; o += kCodecMax) {
    const int64_t k = n - o < kCodecMax ? n - o : kCodecMax;
    const dim3 grid((uint32_t)((k + kCodecElems - 1) / kCodecElems));
    if (kind == PS_MOMENT_SIGNED)
      hipLaunchKernelGGL(k_decode_fp8<PS_MOMENT_SIGNED>, grid, dim3(kCodecThreads), 0, s, code + o, scale + o / kBlock,
                         x + o, k);
    else
      hipLaunchKernelGGL(k_decode_fp8<PS_MOMENT_UNSIGNED>, grid, dim3(kCodecThreads), 0, s, code + o,
                         scale + o / kBlock, x + o, k);
    if (ps_status st = hip_check(hipGetLastError(), "k_decode_fp8 launch")) return st;
  }
  return PS_OK;
}

}  // namespace ps
