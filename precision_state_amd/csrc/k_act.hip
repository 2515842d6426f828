// k_act.hip - the codec of saved activations, and the activation of a
// feed-forward layer with its inputs saved in 8 bits: forward, and backward
// from the codes.
//
// A block of 128 columns lies on 16 lanes, eight values each: its largest value
// is a DPP maximum inside the row of lanes, and a lane's loads and stores of
// 16-bit values are 16 bytes wide. Every call is one pass over its data, which
// bounds it: 16384 x 12288 bf16 encoded in 93 us (6.6 TB/s), gated SiLU of 8192 x
// 11008 forward in 116 us and backward, with its output once more, in 146 (6.2).
#include "dev_act.h"

namespace ps {
namespace {

constexpr int kThreads = 256;
constexpr int kTeams = kThreads / 16;   // blocks that a workgroup handles at a time

// The lane's place in unit u. Lanes of units that do not exist load from the
// last one and store nothing.
template <int END>
struct Place {
  int64_t row;
  int col;
  bool in;
  Cols<END> c;
  __device__ __forceinline__ Place(const ActGrid& g, uint32_t u) : c(0, 0) {
    in = u < g.units;
    u = in ? u : g.units - 1;
    const uint32_t r = div_by(u, g.nb);
    row = r;
    col = (int)(u - r * g.nb.d) * kActBlock + (int)(threadIdx.x & 15) * 8;
    c = Cols<END>(col, g.cols);
  }
  __device__ __forceinline__ Cols<END> to_store() const {
    Cols<END> s = c;
    if (!in) s.left = 0;
    return s;
  }
};

__device__ __forceinline__ uint32_t unit_of(int k, int per) {
  return ((blockIdx.y * gridDim.x + blockIdx.x) * per + k) * (uint32_t)kTeams + threadIdx.x / 16;
}

template <int TYPE, int END, int K>
__global__ __launch_bounds__(kThreads) void k_encode_act(ActGrid g, const void* x, int64_t ld, uint8_t* code, float* scale) {
  Raw8<TYPE> raw[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const Place<END> p(g, unit_of(k, K));
    raw[k] = load8<TYPE>(row_of<TYPE>(x, p.row, ld), p.c);
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const uint32_t u = unit_of(k, K);
    const Place<END> p(g, u);
    float v[8], s;
    widen8<TYPE>(raw[k], p.c, v);
    const u32x2_any c = encode_block(v, s);
    store_codes8(codes_of(code, p.row, g.cols), p.col, p.to_store(), c);
    if (p.in && (threadIdx.x & 15) == 0) scale[u] = s;
  }
}

template <int TYPE, int END, int K>
__global__ __launch_bounds__(kThreads) void k_decode_act(ActGrid g, const uint8_t* code, const float* scale, void* x,
                                                         int64_t ld) {
  u32x2_any c[K];
  float s[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const uint32_t u = unit_of(k, K);
    const Place<END> p(g, u);
    c[k] = load_codes8(codes_of(code, p.row, g.cols), p.c);
    s[k] = scale[p.in ? u : g.units - 1];
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const Place<END> p(g, unit_of(k, K));
    float v[8];
    codes_to_f32(c[k], p.c, v);
    decode8<TYPE, TYPE != PS_TYPE_F32>(v, s[k]);
    store8<TYPE>(row_of<TYPE>(x, p.row, ld), p.col, p.to_store(), v);
  }
}

// f(a) and f'(a). Each is a times a probability q: the logistic function for
// SILU, Phi for GELU, and for its tanh form (1 + tanh u) / 2, which is the
// logistic function of 2 u and loses nothing where tanh u comes near -1.
// Phi(-z) exp(z^2 / 2) for z >= 0 falls like 1 / z; in t = 1 / (1 + 0.35 z) it is
// t times a polynomial (the form of Hastings, Approximations for Digital
// Computers, 1955), fitted here: a relative error of 3.2e-8, and 5.9e-8 with the
// coefficients in fp32, up to z = 14.5, beyond which the exponential is 0 in fp32.
// That is one rounding; f' is off by 5e-8 in the 2-norm for normal a, which is that
// of its fp32 steps (a fit to the rounded coefficients, 3.4e-8, gains 1% of it).
// The exponential serves f' too (the math library's erfc: 8192 x 11008 bf16
// forward 132 us, this 78).
template <int ACT>
__device__ __forceinline__ void activation(float a, float& f, float& slope) {
  constexpr float kLog2e = 1.44269504f;
  if (ACT == PS_ACT_GELU) {
    constexpr float kP[] = {0.139621302f, 0.139863521f, 0.119821213f, 0.105552793f, -0.0232130159f,
                            0.159320623f, -0.255839765f, 0.144031256f, -0.0291579515f};
    const float z = fminf(__builtin_fabsf(a), 14.5f);
    const float e = __builtin_amdgcn_exp2f(z * z * (-0.5f * kLog2e)), t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.35f, z, 1.0f));
    float w = kP[8];
#pragma unroll
    for (int i = 7; i >= 0; --i) w = __builtin_fmaf(w, t, kP[i]);
    w *= t * e;
    const float q = a < 0.0f ? w : 1.0f - w;
    f = a * q;
    slope = __builtin_fmaf(a * 0.39894228f, e, q);
    return;
  }
  constexpr float c = 0.79788456f, c3 = 0.044715f;
  const float z = __builtin_amdgcn_fmed3f(a, -64.0f, 64.0f);   // q is 0 or 1 there, and z^2 stays finite
  const float u = ACT == PS_ACT_SILU ? a : 2.0f * c * z * __builtin_fmaf(c3, z * z, 1.0f);
  const float du = ACT == PS_ACT_SILU ? 1.0f : 2.0f * c * __builtin_fmaf(3.0f * c3, z * z, 1.0f);
  // 1 - q is e q, which keeps its places where q is next to 1 and f and du are large
  // (1 - q itself: slopes of tanh's form off by up to 2.0e-6, so by 2.1e-7); e is
  // infinite where q is 0
  const float e = __builtin_amdgcn_exp2f(u * -kLog2e), q = __builtin_amdgcn_rcpf(1.0f + e);
  f = a * q;
  slope = __builtin_fmaf(f * (__builtin_amdgcn_fmed3f(e, 0.0f, 0x1p126f) * q), du, q);
}

template <int TYPE, int ACT, bool GATED, bool SAVE, int END>
__global__ __launch_bounds__(kThreads) void k_glu_forward(ActGrid g, GluArgs t) {
  const uint32_t u = unit_of(0, 1);
  const Place<END> p(g, u);
  const Raw8<TYPE> ra = load8<TYPE>(row_of<TYPE>(t.a, p.row, t.lda), p.c);
  float a[8], b[8], o[8], s;
  if (GATED) widen8<TYPE>(load8<TYPE>(row_of<TYPE>(t.b, p.row, t.ldb), p.c), p.c, b);
  widen8<TYPE>(ra, p.c, a);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float slope;
    activation<ACT>(a[j], o[j], slope);
    if (GATED) o[j] *= b[j];
  }
  store8<TYPE>(row_of<TYPE>(t.out, p.row, t.ldo), p.col, p.to_store(), o);
  if (!SAVE) return;
  const bool writes = p.in && (threadIdx.x & 15) == 0;
  const u32x2_any c = encode_block(a, s);
  store_codes8(codes_of(t.a_code, p.row, g.cols), p.col, p.to_store(), c);
  if (writes) t.a_scale[u] = s;
  if (!GATED) return;
  const u32x2_any d = encode_block(b, s);
  store_codes8(codes_of(t.b_code, p.row, g.cols), p.col, p.to_store(), d);
  if (writes) t.b_scale[u] = s;
}

template <int TYPE, int ACT, bool GATED, int END>
__global__ __launch_bounds__(kThreads) void k_glu_backward(ActGrid g, GluArgs t) {
  const uint32_t u = unit_of(0, 1);
  const Place<END> p(g, u);
  const uint32_t at = p.in ? u : g.units - 1;
  const Raw8<TYPE> rd = load8<TYPE>(row_of<TYPE>(t.dout, p.row, t.ldd), p.c);
  const u32x2_any ca = load_codes8(codes_of(t.a_code, p.row, g.cols), p.c);
  const float sa = t.a_scale[at];
  float d[8], a[8], b[8], da[8], db[8], o[8], sb;
  if (GATED) {
    const u32x2_any cb = load_codes8(codes_of(t.b_code, p.row, g.cols), p.c);
    sb = t.b_scale[at];
    codes_to_f32(cb, p.c, b);
  }
  codes_to_f32(ca, p.c, a);
  decode8<TYPE, !GATED && TYPE != PS_TYPE_F32>(a, sa);
  if (GATED) decode8<TYPE, false>(b, sb);
  widen8<TYPE>(rd, p.c, d);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float f, slope;
    activation<ACT>(a[j], f, slope);
    if (GATED) {
      db[j] = d[j] * f;
      da[j] = d[j] * b[j] * slope;
      o[j] = f * b[j];
    } else {
      da[j] = d[j] * slope;
      o[j] = f;
    }
  }
  store8<TYPE>(row_of<TYPE>(t.da, p.row, t.lda), p.col, p.to_store(), da);
  if (GATED) store8<TYPE>(row_of<TYPE>(t.db, p.row, t.ldb), p.col, p.to_store(), db);
  if (t.out) store8<TYPE>(row_of<TYPE>(t.out, p.row, t.ldo), p.col, p.to_store(), o);
}

dim3 grid_of(const ActGrid& g, int k) { return grid_2d((g.units + kTeams * k - 1) / (kTeams * k)); }

// The codec's lanes have a part of two blocks (16384 x 12288 bf16 encoded in 93 us;
// with one block 105, with four 97), those of the activations, which have two to
// three streams more, of one (8192 x 11008 gated, forward 118 us and backward 143;
// with two blocks 122 and 151, with four 124 and 156).
constexpr int kCodecBlocks = 2;

template <int TYPE, int ACT, int END>
ps_status glu_forward(const ActGrid& g, const GluArgs& p, hipStream_t s) {
  const bool save = p.a_code != nullptr;
  const dim3 grid = grid_of(g, 1), wg(kThreads);
  if (p.b && save)
    hipLaunchKernelGGL((k_glu_forward<TYPE, ACT, true, true, END>), grid, wg, 0, s, g, p);
  else if (p.b)
    hipLaunchKernelGGL((k_glu_forward<TYPE, ACT, true, false, END>), grid, wg, 0, s, g, p);
  else if (save)
    hipLaunchKernelGGL((k_glu_forward<TYPE, ACT, false, true, END>), grid, wg, 0, s, g, p);
  else
    hipLaunchKernelGGL((k_glu_forward<TYPE, ACT, false, false, END>), grid, wg, 0, s, g, p);
  return hip_check(hipGetLastError(), "k_glu_forward launch");
}

template <int TYPE, int ACT, int END>
ps_status glu_backward(const ActGrid& g, const GluArgs& p, hipStream_t s) {
  if (p.b_code)
    hipLaunchKernelGGL((k_glu_backward<TYPE, ACT, true, END>), grid_of(g, 1), dim3(kThreads), 0, s, g, p);
  else
    hipLaunchKernelGGL((k_glu_backward<TYPE, ACT, false, END>), grid_of(g, 1), dim3(kThreads), 0, s, g, p);
  return hip_check(hipGetLastError(), "k_glu_backward launch");
}

template <int TYPE, int ACT>
ps_status glu(bool forward, const ActGrid& g, const GluArgs& p, hipStream_t s) {
  switch (end_of(g.cols)) {
    case kWhole: return forward ? glu_forward<TYPE, ACT, kWhole>(g, p, s) : glu_backward<TYPE, ACT, kWhole>(g, p, s);
    case kPart: return forward ? glu_forward<TYPE, ACT, kPart>(g, p, s) : glu_backward<TYPE, ACT, kPart>(g, p, s);
    default: return forward ? glu_forward<TYPE, ACT, kShort>(g, p, s) : glu_backward<TYPE, ACT, kShort>(g, p, s);
  }
}

template <int TYPE>
ps_status glu(bool forward, const ActGrid& g, int act, const GluArgs& p, hipStream_t s) {
  switch (act) {
    case PS_ACT_SILU: return glu<TYPE, PS_ACT_SILU>(forward, g, p, s);
    case PS_ACT_GELU: return glu<TYPE, PS_ACT_GELU>(forward, g, p, s);
    default: return glu<TYPE, PS_ACT_GELU_TANH>(forward, g, p, s);
  }
}

ps_status glu(bool forward, const ActGrid& g, int type, int act, const GluArgs& p, hipStream_t s) {
  switch (type) {
    case PS_TYPE_F32: return glu<PS_TYPE_F32>(forward, g, act, p, s);
    case PS_TYPE_BF16: return glu<PS_TYPE_BF16>(forward, g, act, p, s);
    default: return glu<PS_TYPE_F16>(forward, g, act, p, s);
  }
}

template <int TYPE>
ps_status encode(const ActGrid& g, const void* x, int64_t ld, uint8_t* code, float* scale, hipStream_t s) {
  const dim3 grid = grid_of(g, kCodecBlocks), wg(kThreads);
  switch (end_of(g.cols)) {
    case kWhole: hipLaunchKernelGGL((k_encode_act<TYPE, kWhole, kCodecBlocks>), grid, wg, 0, s, g, x, ld, code, scale); break;
    case kPart: hipLaunchKernelGGL((k_encode_act<TYPE, kPart, kCodecBlocks>), grid, wg, 0, s, g, x, ld, code, scale); break;
    default: hipLaunchKernelGGL((k_encode_act<TYPE, kShort, kCodecBlocks>), grid, wg, 0, s, g, x, ld, code, scale); break;
  }
  return hip_check(hipGetLastError(), "k_encode_act launch");
}

template <int TYPE>
ps_status decode(const ActGrid& g, const uint8_t* code, const float* scale, void* x, int64_t ld, hipStream_t s) {
  const dim3 grid = grid_of(g, kCodecBlocks), wg(kThreads);
  switch (end_of(g.cols)) {
    case kWhole: hipLaunchKernelGGL((k_decode_act<TYPE, kWhole, kCodecBlocks>), grid, wg, 0, s, g, code, scale, x, ld); break;
    case kPart: hipLaunchKernelGGL((k_decode_act<TYPE, kPart, kCodecBlocks>), grid, wg, 0, s, g, code, scale, x, ld); break;
    default: hipLaunchKernelGGL((k_decode_act<TYPE, kShort, kCodecBlocks>), grid, wg, 0, s, g, code, scale, x, ld); break;
  }
  return hip_check(hipGetLastError(), "k_decode_act launch");
}

}  // namespace

ps_status launch_encode_act(const ActGrid& g, int type, const void* x, int64_t ld, uint8_t* code, float* scale,
                            hipStream_t s) {
  switch (type) {
    case PS_TYPE_F32: return encode<PS_TYPE_F32>(g, x, ld, code, scale, s);
    case PS_TYPE_BF16: return encode<PS_TYPE_BF16>(g, x, ld, code, scale, s);
    default: return encode<PS_TYPE_F16>(g, x, ld, code, scale, s);
  }
}

ps_status launch_decode_act(const ActGrid& g, int type, const uint8_t* code, const float* scale, void* x, int64_t ld,
                            hipStream_t s) {
  switch (type) {
    case PS_TYPE_F32: return decode<PS_TYPE_F32>(g, code, scale, x, ld, s);
    case PS_TYPE_BF16: return decode<PS_TYPE_BF16>(g, code, scale, x, ld, s);
    default: return decode<PS_TYPE_F16>(g, code, scale, x, ld, s);
  }
}

ps_status launch_glu_forward(const ActGrid& g, int type, int act, const GluArgs& p, hipStream_t s) {
  return glu(true, g, type, act, p, s);
}

ps_status launch_glu_backward(const ActGrid& g, int type, int act, const GluArgs& p, hipStream_t s) {
  return glu(false, g, type, act, p, s);
}

}  // namespace ps
