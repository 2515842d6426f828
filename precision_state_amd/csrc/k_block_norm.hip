// k_block_norm.hip - the norms after a block and before the next one, with the
// gate, the residual scale and the residual sum between them, and their
// backward pass from 8-bit normalised values.
//
// A row is held in registers by one team of lanes from its first load to its
// last store, so that means, the residual sum, both norms and the codes cost
// one pass over memory. The variance of a LayerNorm is the mean square about
// the mean (a second reduction over registers), not a difference of sums.
#include "dev_act.h"

namespace ps {
namespace {

// Sums of a team of NT lanes, on every lane: a wave's alone, or those of its
// waves through shared memory. `turn` alternates between two places, so that
// one barrier a sum is enough.
template <int NT, int N>
struct TeamSum {
  static constexpr int kWaves = NT / 64;
  float (*lds)[kWaves][N];
  int turn = 0;
  __device__ __forceinline__ void operator()(float* v) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
    if (NT == 64) return;
    const int wave = threadIdx.x / 64;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) lds[turn][wave][i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = lds[turn][0][i];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) s += lds[turn][w][i];
      v[i] = s;
    }
    turn ^= 1;
  }
};

// The segment of a row: the last one that starts at or before it; -1 if there
// is none or it ends before the row. Reads seg_start[0 .. n] only, whatever it
// holds.
__device__ __forceinline__ int find_seg(const int32_t* start, int n, int row) {
  int lo = 0, hi = n;   // start[lo] <= row < start[hi], once that holds
  if (row < start[0] || row >= start[n]) return -1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (start[mid] <= row)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int64_t seg_offset(const NormArgs& p, uint32_t by_seg, int seg) {
  return p.flags & by_seg ? (int64_t)seg * p.cols : 0;
}


// z[0 .. V-1][8] of a row becomes its normalised values; the factor r is returned.
template <int NT, int V, class Sum>
__device__ __forceinline__ float normalise(const NormArgs& p, int kind, float eps, int lane, Sum& sum, float (*z)[8]) {
  float s[1];
  if (kind == PS_NORM_LAYER) {
    s[0] = 0;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) s[0] += z[v][j];
    sum(s);
    const float mean = s[0] * p.inv_cols;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) z[v][j] = (v * NT + lane) * 8 + j < p.cols ? z[v][j] - mean : 0.0f;
  }
  s[0] = 0;
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int j = 0; j < 8; ++j) s[0] = __builtin_fmaf(z[v][j], z[v][j], s[0]);
  sum(s);
  const float r = 1.0f / __builtin_sqrtf(__builtin_fmaf(s[0], p.inv_cols, eps));
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int j = 0; j < 8; ++j) z[v][j] *= r;
  return r;
}

__device__ __forceinline__ u32x2_any pack_codes(const float* z) {
  u32x2_any c;
  c[0] = e4m3_pack4(z);
  c[1] = e4m3_pack4(z + 4);
  return c;
}

// Rows by teams of NT lanes, V times eight columns on each.
template <int TYPE, int NT, int V>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void k_norm_forward(NormArgs p) {
  constexpr int kRows = NT < 256 ? 256 / NT : 1;
  __shared__ float lds[2][NT / 64][1];
  TeamSum<NT, 1> sum{lds};
  const int lane = threadIdx.x % NT;
  int row = blockIdx.x * kRows + threadIdx.x / NT;
  if (NT == 64) row = __builtin_amdgcn_readfirstlane(row);
  if (row >= p.rows) return;   // whole teams leave
  int seg = 0;
  if (p.seg_start) {
    seg = find_seg(p.seg_start, p.n_segs, row);
    if (seg < 0) return;
  }
  float z[V][8];
  Raw8<TYPE> rx[V], ry[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int col = (v * NT + lane) * 8;
    if (p.y) ry[v] = load8<TYPE>(p.y, (int64_t)row * p.ldy + col, p.cols - col);
    rx[v] = load8<TYPE>(p.x, (int64_t)row * p.ldx + col, p.cols - col);
  }
  if (p.y) {
#pragma unroll
    for (int v = 0; v < V; ++v) widen8<TYPE>(ry[v], z[v]);
    if (p.post != PS_NORM_NONE) {
      const float r = normalise<NT, V>(p, p.post, p.post_eps, lane, sum, z);
      if (p.y_rstd && lane == 0) p.y_rstd[row] = r;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int col = (v * NT + lane) * 8, left = p.cols - col;
      if (p.y_code) {
        u32x2_any c;
        if (p.post != PS_NORM_NONE) {
          c = pack_codes(z[v]);
        } else {
          float s;
          c = encode_block(z[v], s);
          if ((lane & 15) == 0 && left > 0)
            p.y_scale[(int64_t)row * ((p.cols + kActBlock - 1) / kActBlock) + col / kActBlock] = s;
        }
        store_codes8(p.y_code, (int64_t)row * p.cols + col, left, c);
      }
      float m[8], x[8];
      if (p.w1) {
        load_vec8(p.w1, p.vec_type, col, left, m);
#pragma unroll
        for (int j = 0; j < 8; ++j) z[v][j] *= m[j];
      }
      if (p.gate) {
        load_vec8(p.gate, p.vec_type, seg_offset(p, PS_NORM_GATE_BY_SEG, seg) + col, left, m);
#pragma unroll
        for (int j = 0; j < 8; ++j) z[v][j] *= m[j];
      }
      widen8<TYPE>(rx[v], x);
#pragma unroll
      for (int j = 0; j < 8; ++j) z[v][j] = __builtin_fmaf(p.beta, z[v][j], p.alpha * x[j]);
      store8<TYPE>(p.h, (int64_t)row * p.ldh + col, left, z[v]);
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) widen8<TYPE>(rx[v], z[v]);
  }
  const float r = normalise<NT, V>(p, p.pre, p.pre_eps, lane, sum, z);
  if (p.h_rstd && lane == 0) p.h_rstd[row] = r;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int col = (v * NT + lane) * 8, left = p.cols - col;
    if (p.h_code) store_codes8(p.h_code, (int64_t)row * p.cols + col, left, pack_codes(z[v]));
    float m[8], a[8];
    const int64_t o = seg_offset(p, PS_NORM_MOD_BY_SEG, seg) + col;
    if (p.mul) {
      load_vec8(p.mul, p.vec_type, o, left, m);
      const float one = p.flags & PS_NORM_MUL_PLUS_ONE ? 1.0f : 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) z[v][j] *= one + m[j];
    }
    if (p.add) {
      load_vec8(p.add, p.vec_type, o, left, a);
#pragma unroll
      for (int j = 0; j < 8; ++j) z[v][j] += a[j];
    }
    store8<TYPE>(p.n, (int64_t)row * p.ldn + col, left, z[v]);
  }
}

// g becomes back(g, z, r): r (g - [mean g] - z mean(g z)).
template <int NT, int V, class Sum>
__device__ __forceinline__ void back(const NormArgs& p, int kind, float r, Sum& sum, float (*g)[8], const float (*z)[8]) {
  float s[2] = {0, 0};
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      s[0] = __builtin_fmaf(g[v][j], z[v][j], s[0]);
      s[1] += g[v][j];
    }
  sum(s);
  const float gz = s[0] * p.inv_cols, m = kind == PS_NORM_LAYER ? s[1] * p.inv_cols : 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int j = 0; j < 8; ++j) g[v][j] = r * (__builtin_fmaf(-gz, z[v][j], g[v][j]) - m);
}

// A workgroup takes a strip of rows and keeps the column sums of its gradients
// in registers; where the segment changes, and at the end, they go to the
// strip's part of that segment.
template <int TYPE, int NT, int V>
__global__ __launch_bounds__(NT) void k_norm_backward(NormArgs p) {
  __shared__ float lds[2][NT / 64][2];
  TeamSum<NT, 2> sum{lds};
  const int lane = threadIdx.x;
  const int first = blockIdx.x * p.strip, last = min(p.rows - first, p.strip) + first;
  const int64_t n_part = (int64_t)p.slots * p.cols;
  const bool branch = p.dy != nullptr;
  const bool has_yh = branch && (p.post != PS_NORM_NONE || p.gate);
  float acc[3][V][8];
  int seg = -1, seg_end = first;   // the segment of the sums, and where it ends

  auto flush = [&]() {
    if (seg < 0) return;
    const int64_t o = (int64_t)(blockIdx.x + seg) * p.cols;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int col = (v * NT + lane) * 8, left = p.cols - col;
      if (p.d_add) store8<PS_TYPE_F32, false>(p.part, o + col, left, acc[0][v]);
      if (p.d_mul) store8<PS_TYPE_F32, false>(p.part + n_part, o + col, left, acc[1][v]);
      if (p.d_gate || p.d_w1) store8<PS_TYPE_F32, false>(p.part + 2 * n_part, o + col, left, acc[2][v]);
    }
  };

  for (int row = first; row < last; ++row) {
    if (row >= seg_end) {   // the first row, or the first of another segment
      flush();
      seg = 0;
      seg_end = last;
      if (p.seg_start) {
        seg = find_seg(p.seg_start, p.n_segs, row);
        // the next row to look again at: the segment's end, or the next one where there is none
        seg_end = seg < 0 ? row + 1 : min(max(p.seg_start[seg + 1], row + 1), last);
      }
#pragma unroll
      for (int i = 0; i < 3; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[i][v][j] = 0;
    }
    if (seg < 0) continue;
    float g[V][8], z[V][8];
    Raw8<TYPE> rdn[V], rdh[V];
    u32x2_any ch[V], cy[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int col = (v * NT + lane) * 8, left = p.cols - col;
      rdn[v] = load8<TYPE>(p.dn, (int64_t)row * p.lddn + col, left);
      ch[v] = load_codes8(p.h_code, (int64_t)row * p.cols + col, left);
      if (p.dh) rdh[v] = load8<TYPE>(p.dh, (int64_t)row * p.lddh + col, left);
      if (has_yh) cy[v] = load_codes8(p.y_code, (int64_t)row * p.cols + col, left);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int col = (v * NT + lane) * 8, left = p.cols - col;
      widen8<TYPE>(rdn[v], g[v]);
      codes_to_f32(ch[v], z[v]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        acc[0][v][j] += g[v][j];
        acc[1][v][j] = __builtin_fmaf(g[v][j], z[v][j], acc[1][v][j]);
      }
      if (p.mul) {
        float m[8];
        load_vec8(p.mul, p.vec_type, seg_offset(p, PS_NORM_MOD_BY_SEG, seg) + col, left, m);
        const float one = p.flags & PS_NORM_MUL_PLUS_ONE ? 1.0f : 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) g[v][j] *= one + m[j];
      }
    }
    back<NT, V>(p, p.pre, p.h_rstd[row], sum, g, z);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int col = (v * NT + lane) * 8, left = p.cols - col;
      if (p.dh) {
        float d[8];
        widen8<TYPE>(rdh[v], d);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[v][j] += d[j];
      }
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = p.alpha * g[v][j];
      store8<TYPE>(p.dx, (int64_t)row * p.lddx + col, left, o);
      if (!branch) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) g[v][j] = left > j ? p.beta * g[v][j] : 0.0f;
      if (has_yh) {
        codes_to_f32(cy[v], z[v]);
        if (p.post == PS_NORM_NONE) {
          const float s = left > 0 ? p.y_scale[(int64_t)row * ((p.cols + kActBlock - 1) / kActBlock) + col / kActBlock] : 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) z[v][j] *= s;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[2][v][j] = __builtin_fmaf(g[v][j], z[v][j], acc[2][v][j]);
      }
      float m[8];
      if (p.gate) {
        load_vec8(p.gate, p.vec_type, seg_offset(p, PS_NORM_GATE_BY_SEG, seg) + col, left, m);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[v][j] *= m[j];
      }
      if (p.w1) {
        load_vec8(p.w1, p.vec_type, col, left, m);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[v][j] *= m[j];
      }
    }
    if (!branch) continue;
    if (p.post != PS_NORM_NONE) back<NT, V>(p, p.post, p.y_rstd[row], sum, g, z);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int col = (v * NT + lane) * 8;
      store8<TYPE>(p.dy, (int64_t)row * p.lddy + col, p.cols - col, g[v]);
    }
  }
  flush();
}

// The strips' parts, added up. A workgroup joins 64 columns of one gradient (and
// one segment of it where it has one for each): 16 groups of lanes take every
// 16th strip, and their sums are added in order.
constexpr int kJoinCols = 64, kJoinGroups = 16;

struct JoinOf {
  float* out;
  int which;      // 0 sum of dn, 1 of dn xh, 2 of p yh
  bool by_seg;
  bool by_gate;   // times the gate (that of the segment), before the segments are added
  bool by_w1;     // times post_weight, at the end
};

__device__ __forceinline__ float vec1(const void* v, int type, int64_t at) {
  if (type == PS_TYPE_F32) return ((const float*)v)[at];
  if (type == PS_TYPE_BF16) return bf16_lo(((const uint16_t*)v)[at]);
  return (float)((const _Float16*)v)[at];
}

__global__ __launch_bounds__(kJoinCols * kJoinGroups) void k_norm_join(NormArgs p, JoinOf j0, JoinOf j1, JoinOf j2, JoinOf j3) {
  const JoinOf j = blockIdx.y == 0 ? j0 : blockIdx.y == 1 ? j1 : blockIdx.y == 2 ? j2 : j3;
  if (!j.by_seg && blockIdx.z) return;
  __shared__ float lds[kJoinGroups][kJoinCols];
  const int c = threadIdx.x % kJoinCols, group = threadIdx.x / kJoinCols;
  const int col = blockIdx.x * kJoinCols + c;
  const int segs = p.seg_start ? p.n_segs : 1;
  const float* part = p.part + (int64_t)j.which * p.slots * p.cols;
  float total = 0;
  if (col < p.cols) {
    for (int b = j.by_seg ? (int)blockIdx.z : 0; b < (j.by_seg ? (int)blockIdx.z + 1 : segs); ++b) {
      int lo = 0, hi = p.rows;
      if (p.seg_start) {
        lo = max(p.seg_start[b], 0);
        hi = min(p.seg_start[b + 1], p.rows);
      }
      if (hi <= lo) continue;
      float s = 0;
      for (int strip = lo / p.strip + group; strip <= (hi - 1) / p.strip; strip += kJoinGroups)
        s += part[(int64_t)(strip + b) * p.cols + col];
      if (j.by_gate) s *= vec1(p.gate, p.vec_type, seg_offset(p, PS_NORM_GATE_BY_SEG, b) + col);
      total += s;
    }
  }
  lds[group][c] = total;
  __syncthreads();
  if (group || col >= p.cols) return;
#pragma unroll
  for (int i = 1; i < kJoinGroups; ++i) total += lds[i][c];
  if (j.by_w1) total *= vec1(p.w1, p.vec_type, col);
  float* out = j.out + (j.by_seg ? (int64_t)blockIdx.z * p.cols : 0) + col;
  *out = p.accumulate ? *out + total : total;
}

template <int TYPE, int NT, int V>
ps_status forward(const NormArgs& p, hipStream_t s) {
  constexpr int kRows = NT < 256 ? 256 / NT : 1;
  hipLaunchKernelGGL((k_norm_forward<TYPE, NT, V>), dim3((p.rows + kRows - 1) / kRows), dim3(NT * kRows), 0, s, p);
  return hip_check(hipGetLastError(), "k_norm_forward launch");
}

template <int TYPE, int NT, int V>
ps_status backward(const NormArgs& p, hipStream_t s) {
  hipLaunchKernelGGL((k_norm_backward<TYPE, NT, V>), dim3((p.rows + p.strip - 1) / p.strip), dim3(NT), 0, s, p);
  return hip_check(hipGetLastError(), "k_norm_backward launch");
}

template <int TYPE>
ps_status forward(const NormArgs& p, hipStream_t s) {
  if (p.cols <= 512) return forward<TYPE, 64, 1>(p, s);
  if (p.cols <= 1024) return forward<TYPE, 64, 2>(p, s);
  if (p.cols <= 2048) return forward<TYPE, 256, 1>(p, s);
  if (p.cols <= 4096) return forward<TYPE, 256, 2>(p, s);
  if (p.cols <= 8192) return forward<TYPE, 512, 2>(p, s);
  return forward<TYPE, 1024, 2>(p, s);
}

template <int TYPE>
ps_status backward(const NormArgs& p, hipStream_t s) {
  if (p.cols <= 512) return backward<TYPE, 64, 1>(p, s);
  if (p.cols <= 1024) return backward<TYPE, 64, 2>(p, s);
  if (p.cols <= 2048) return backward<TYPE, 256, 1>(p, s);
  if (p.cols <= 4096) return backward<TYPE, 256, 2>(p, s);
  if (p.cols <= 8192) return backward<TYPE, 512, 2>(p, s);
  return backward<TYPE, 1024, 2>(p, s);
}

}  // namespace

ps_status launch_norm_forward(const NormArgs& p, int type, hipStream_t s) {
  switch (type) {
    case PS_TYPE_F32: return forward<PS_TYPE_F32>(p, s);
    case PS_TYPE_BF16: return forward<PS_TYPE_BF16>(p, s);
    default: return forward<PS_TYPE_F16>(p, s);
  }
}

ps_status launch_norm_backward(const NormArgs& p, int type, hipStream_t s) {
  if (p.rows) {
    ps_status st;
    switch (type) {
      case PS_TYPE_F32: st = backward<PS_TYPE_F32>(p, s); break;
      case PS_TYPE_BF16: st = backward<PS_TYPE_BF16>(p, s); break;
      default: st = backward<PS_TYPE_F16>(p, s); break;
    }
    if (st) return st;
  }
  JoinOf j[4] = {};
  int n = 0;
  bool by_seg = false;
  auto add = [&](float* out, int which, bool seg, bool gate, bool w1) {
    if (!out) return;
    j[n++] = {out, which, seg, gate, w1};
    by_seg |= seg;
  };
  add(p.d_add, 0, p.flags & PS_NORM_MOD_BY_SEG, false, false);
  add(p.d_mul, 1, p.flags & PS_NORM_MOD_BY_SEG, false, false);
  add(p.d_gate, 2, p.flags & PS_NORM_GATE_BY_SEG, false, p.w1 != nullptr);
  add(p.d_w1, 2, false, p.gate != nullptr, false);
  if (!n) return PS_OK;
  hipLaunchKernelGGL(k_norm_join, dim3((p.cols + kJoinCols - 1) / kJoinCols, n, by_seg ? p.n_segs : 1),
                     dim3(kJoinCols * kJoinGroups), 0, s, p, j[0], j[1], j[2], j[3]);
  return hip_check(hipGetLastError(), "k_norm_join launch");
}

}  // namespace ps
