// k_block_norm.hip - the norms after a block and before the next one, with the
// gate, the residual scale and the residual sum between them, and their
// backward pass from 8-bit normalised values.
//
// A row is held in registers by one team of lanes from its first load to its
// last store, so that means, the residual sum, both norms and the codes cost
// one pass over memory. The variance of a LayerNorm is the mean square about
// the mean (a second reduction over registers), not a difference of sums.
// Memory bounds the forward pass (16384 x 4096 bf16 with two norms 114 us, 5.9
// TB/s, the vectors in bf16; in fp32, twice as much from the L2 for each row, 125),
// memory and the barriers of a row's sums the backward one (125 us with the join
// of its column sums, 5.4 TB/s).
#include "dev_act.h"

namespace ps {
namespace {

// Sums of a team of lanes, on every lane: a wave's alone, or those of the
// workgroup's waves through shared memory. `turn` alternates between two places,
// so that one barrier a sum is enough.
constexpr int kMostWaves = 16;
struct TeamSum {
  float (*lds)[kMostWaves][2];
  int waves;
  int turn = 0;
  template <int N>
  __device__ __forceinline__ void operator()(float* v) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
    if (waves == 1) return;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) lds[turn][threadIdx.x / 64][i] = v[i];
    }
    __syncthreads();
    // each row of 16 lanes reads all waves' sums at once
    const int w = threadIdx.x & 15;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = row16_sum(w < waves ? lds[turn][w][i] : 0.0f);
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
template <int V, class Sum>
__device__ __forceinline__ float normalise(const NormArgs& p, int kind, float eps, int lane, int nt, Sum& sum, float (*z)[8]) {
  float s[1];
  if (kind == PS_NORM_LAYER) {
    s[0] = 0;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) s[0] += z[v][j];
    sum.template operator()<1>(s);
    const float mean = s[0] * p.inv_cols;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) z[v][j] = (v * nt + lane) * 8 + j < p.cols ? z[v][j] - mean : 0.0f;
  }
  s[0] = 0;
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int j = 0; j < 8; ++j) s[0] = __builtin_fmaf(z[v][j], z[v][j], s[0]);
  sum.template operator()<1>(s);
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

// A row by one team: the waves of a workgroup (V times eight columns on each
// lane, as few lanes as hold the row), or, up to 1024 columns, a wave with three
// others beside it.
template <int TYPE, int V, bool WAVE, int END>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void k_norm_forward(NormArgs p) {
  __shared__ float lds[2][kMostWaves][2];
  const int nt = WAVE ? 64 : blockDim.x, lane = WAVE ? threadIdx.x & 63 : threadIdx.x;
  TeamSum sum{lds, nt / 64};
  const int group = blockIdx.y * gridDim.x + blockIdx.x;
  const int row = WAVE ? __builtin_amdgcn_readfirstlane(group * 4 + threadIdx.x / 64) : group;
  if (row >= p.rows) return;   // whole teams leave
  int seg = 0;
  if (p.seg_start) {
    seg = find_seg(p.seg_start, p.n_segs, row);
    if (seg < 0) return;
  }
  float z[V][8];
  Raw8<TYPE> rx[V], ry[V];
  RawVec rw[V], rg[V], rm[V], ra[V];   // all loads of the row at once
  const int64_t mod = seg_offset(p, PS_NORM_MOD_BY_SEG, seg);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const Cols<END> c((v * nt + lane) * 8, p.cols);
    if (p.y) ry[v] = load8<TYPE>(scalar_pointer(row_of<TYPE>(p.y, row, p.ldy)), c);
    rx[v] = load8<TYPE>(scalar_pointer(row_of<TYPE>(p.x, row, p.ldx)), c);
    if (p.w1) rw[v] = load_vec(p.w1, p.vec_type, 0, c);
    if (p.gate) rg[v] = load_vec(p.gate, p.vec_type, seg_offset(p, PS_NORM_GATE_BY_SEG, seg), c);
    if (p.mul) rm[v] = load_vec(p.mul, p.vec_type, mod, c);
    if (p.add) ra[v] = load_vec(p.add, p.vec_type, mod, c);
  }
  if (p.y) {
#pragma unroll
    for (int v = 0; v < V; ++v) widen8<TYPE>(ry[v], Cols<END>((v * nt + lane) * 8, p.cols), z[v]);
    if (p.post != PS_NORM_NONE) {
      const float r = normalise<V>(p, p.post, p.post_eps, lane, nt, sum, z);
      if (p.y_rstd && lane == 0) p.y_rstd[row] = r;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int col = (v * nt + lane) * 8;
      const Cols<END> c8(col, p.cols);
      if (p.y_code) {
        u32x2_any c;
        if (p.post != PS_NORM_NONE) {
          c = pack_codes(z[v]);
        } else {
          float s;
          c = encode_block(z[v], s);
          if ((lane & 15) == 0 && c8.left > 0)
            p.y_scale[(int64_t)row * ((p.cols + kActBlock - 1) / kActBlock) + col / kActBlock] = s;
        }
        store_codes8(scalar_pointer(codes_of(p.y_code, row, p.cols)), col, c8, c);
      }
      float m[8], x[8];
      if (p.w1) {
        widen_vec(rw[v], p.vec_type, c8, m);
#pragma unroll
        for (int j = 0; j < 8; ++j) z[v][j] *= m[j];
      }
      if (p.gate) {
        widen_vec(rg[v], p.vec_type, c8, m);
#pragma unroll
        for (int j = 0; j < 8; ++j) z[v][j] *= m[j];
      }
      widen8<TYPE>(rx[v], c8, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) z[v][j] = __builtin_fmaf(p.beta, z[v][j], p.alpha * x[j]);
      store8<TYPE>(scalar_pointer(row_of<TYPE>(p.h, row, p.ldh)), col, c8, z[v]);
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) widen8<TYPE>(rx[v], Cols<END>((v * nt + lane) * 8, p.cols), z[v]);
  }
  const float r = normalise<V>(p, p.pre, p.pre_eps, lane, nt, sum, z);
  if (p.h_rstd && lane == 0) p.h_rstd[row] = r;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int col = (v * nt + lane) * 8;
    const Cols<END> c8(col, p.cols);
    if (p.h_code) store_codes8(scalar_pointer(codes_of(p.h_code, row, p.cols)), col, c8, pack_codes(z[v]));
    float m[8], a[8];
    if (p.mul) {
      widen_vec(rm[v], p.vec_type, c8, m);
      const float one = p.flags & PS_NORM_MUL_PLUS_ONE ? 1.0f : 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) z[v][j] *= one + m[j];
    }
    if (p.add) {
      widen_vec(ra[v], p.vec_type, c8, a);
#pragma unroll
      for (int j = 0; j < 8; ++j) z[v][j] += a[j];
    }
    store8<TYPE>(scalar_pointer(row_of<TYPE>(p.n, row, p.ldn)), col, c8, z[v]);
  }
}

// The sums that back(g, z, r) = r (g - [mean g] - z mean(g z)) needs, as the
// factors of its form fma(r, g, fma(-c, z, -d)): c = r mean(g z), d = r mean g.
template <int V, class Sum>
__device__ __forceinline__ void back_sums(const NormArgs& p, int kind, float r, Sum& sum, const float (*g)[8],
                                          const float (*z)[8], float& c, float& d) {
  float s[2] = {0, 0};
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int j = 0; j < 8; ++j) s[0] = __builtin_fmaf(g[v][j], z[v][j], s[0]);
  d = 0.0f;
  if (kind == PS_NORM_LAYER) {
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) s[1] += g[v][j];
    sum.template operator()<2>(s);
    d = r * (s[1] * p.inv_cols);
  } else {
    sum.template operator()<1>(s);
  }
  c = r * (s[0] * p.inv_cols);
}

// A value that all lanes loaded alike, in a scalar register: its vector register
// is free for the next row's.
__device__ __forceinline__ float uniform(float v) {
  return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(v)));
}

// What the backward pass finds of the branch: nothing saved, its values (a gate
// without a norm), or its normalised ones.
enum { kNoBranch = 0, kPlain = 1, kNormed = 2 };

// A workgroup takes a strip of rows, one segment's after the other's, and keeps
// the column sums of its gradients in registers until a segment's rows end; then
// they go to the strip's part of that segment. Each half of the next row is
// loaded into the registers of this one's as soon as it is used, before the sums
// whose barriers the load's latency would otherwise add to; a segment's vectors
// stay in registers, since a load behind those of the next row would wait for
// them. The widest rows (V > 1) leave no registers for either, and take their
// vectors when they are needed (4096 x 12288 with both norms 143 -> 128 us). The
// sums and two rows' values are still more than the registers hold: with four
// parts a lane 25 to 170 of them are in scratch memory (16384 columns 16-bit: 2.0
// TB/s with a branch, 4.1 without; 9001 columns 2.5 and 3.2), with three 4 to 23 with
// a branch; with one part 2 to 5 in fp32 with a branch, but for kEvery.
// Waits for a load count what was issued behind it, the fewest over all ways
// there, so a branch around a later load or store makes them waits for nearly
// everything. Rows of a multiple of 512 columns (kEvery) have no such branch:
// no lane is without columns, an absent dh reads dn's first row instead and is
// taken as zeros. 16384 x 4096 with both norms 123 -> 120 us.
// It reaches 5.6 TB/s there and 4.7 with 9216 x 5120 and a gate, where one
// workgroup of ten waves fills a compute unit (registers): the sums' barrier is
// what both wait for. Not kept: two rows loaded ahead (9216 x 5120 100 -> 101
// us), five waves to a SIMD (registers spill, 45 to 70% slower), strips of half
// the rows (5% slower).
template <int TYPE, int V, int SAVED, int END>
__global__ __launch_bounds__(V == 1 ? 1024 : 512) void k_norm_backward(NormArgs p) {
  constexpr bool kAhead = V == 1;
  __shared__ float lds[2][kMostWaves][2];
  const int nt = blockDim.x, lane = threadIdx.x;
  TeamSum sum{lds, nt / 64};
  // Without segments a strip takes every gridDim.x-th row, so that all workgroups
  // sweep the matrices from front to back together.
  const int step = p.seg_start ? 1 : gridDim.x;
  const int first = p.seg_start ? blockIdx.x * p.strip : blockIdx.x;
  const int last = p.seg_start ? min(p.rows - first, p.strip) + first : p.rows;
  const int64_t n_part = (int64_t)p.slots * p.cols;
  const int blocks = (p.cols + kActBlock - 1) / kActBlock;

  for (int row = first; row < last;) {
    int seg = 0, end = last;
    if (p.seg_start) {
      seg = find_seg(p.seg_start, p.n_segs, row);
      if (seg < 0) {
        ++row;
        continue;
      }
      end = min(max(p.seg_start[seg + 1], row + 1), last);
    }
    // m, and branch_scale * gate * post_weight (0 for columns that do not exist)
    float km[V][8], ky[V][8], acc[3][V][8];
    auto vectors = [&](bool first, bool second) __attribute__((always_inline)) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const Cols<END> c((v * nt + lane) * 8, p.cols);
        const float one = p.flags & PS_NORM_MUL_PLUS_ONE ? 1.0f : 0.0f;
        RawVec rm, rg, rw;
        if (first && p.mul) rm = load_vec(p.mul, p.vec_type, seg_offset(p, PS_NORM_MOD_BY_SEG, seg), c);
        if (second && p.gate) rg = load_vec(p.gate, p.vec_type, seg_offset(p, PS_NORM_GATE_BY_SEG, seg), c);
        if (second && p.w1) rw = load_vec(p.w1, p.vec_type, 0, c);
        float m[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (first) km[v][j] = 1.0f;
          if (second) ky[v][j] = j < c.left ? p.beta : 0.0f;
        }
        if (first && p.mul) {
          widen_vec(rm, p.vec_type, c, m);
#pragma unroll
          for (int j = 0; j < 8; ++j) km[v][j] = one + m[j];
        }
        if (second && p.gate) {
          widen_vec(rg, p.vec_type, c, m);
#pragma unroll
          for (int j = 0; j < 8; ++j) ky[v][j] *= m[j];
        }
        if (second && p.w1) {
          widen_vec(rw, p.vec_type, c, m);
#pragma unroll
          for (int j = 0; j < 8; ++j) ky[v][j] *= m[j];
        }
      }
    };
    Raw8<TYPE> dn[V], dh[V];
    u32x2_any ch[V], cy[V];
    float ys[V], h_rstd, y_rstd;
    auto load_first = [&](int r) __attribute__((always_inline)) {
      h_rstd = p.h_rstd[r];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const Cols<END> c((v * nt + lane) * 8, p.cols);
        dn[v] = load8<TYPE>(scalar_pointer(row_of<TYPE>(p.dn, r, p.lddn)), c);
        ch[v] = load_codes8(scalar_pointer(codes_of(p.h_code, r, p.cols)), c);
      }
    };
    auto load_second = [&](int r) __attribute__((always_inline)) {
      if (SAVED == kNormed) y_rstd = p.y_rstd[r];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const Cols<END> c((v * nt + lane) * 8, p.cols);
        dh[v] = load8<TYPE>(scalar_pointer(p.dh ? row_of<TYPE>(p.dh, r, p.lddh) : row_of<TYPE>(p.dn, 0, 0)), c);
        if (SAVED != kNoBranch) cy[v] = load_codes8(scalar_pointer(codes_of(p.y_code, r, p.cols)), c);
        if (SAVED == kPlain) ys[v] = p.y_scale[(int64_t)r * blocks + min((v * nt + lane) * 8, p.cols - 1) / kActBlock];
      }
    };
    if (kAhead) {
      load_first(row);
      load_second(row);
      vectors(true, true);
    }
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][v][j] = 0;

    for (; row < end; row += step) {
      if (!kAhead) {
        load_first(row);
        load_second(row);
        vectors(true, false);
      }
      const int ahead = row + step < end ? row + step : row;   // the last row is loaded twice
      float g[V][8], z[V][8], c, d;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const Cols<END> c8((v * nt + lane) * 8, p.cols);
        widen8<TYPE>(dn[v], c8, g[v]);
        codes_to_f32(ch[v], c8, z[v]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          acc[0][v][j] += g[v][j];
          acc[1][v][j] = __builtin_fmaf(g[v][j], z[v][j], acc[1][v][j]);
          g[v][j] *= km[v][j];
        }
      }
      const float r1 = uniform(h_rstd);
      if (kAhead) load_first(ahead);
      back_sums<V>(p, p.pre, r1, sum, g, z, c, d);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int col = (v * nt + lane) * 8;
        const Cols<END> c8(col, p.cols);
        float o[8];
        widen8<TYPE>(dh[v], c8, o);
        if (!p.dh) {
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          g[v][j] = __builtin_fmaf(-c, z[v][j], __builtin_fmaf(r1, g[v][j], o[j] - d));
          o[j] = p.alpha * g[v][j];
        }
        store8<TYPE>(scalar_pointer(row_of<TYPE>(p.dx, row, p.lddx)), col, c8, o);
        if (SAVED != kNoBranch) {
          codes_to_f32(cy[v], c8, z[v]);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (SAVED == kPlain) z[v][j] *= ys[v];
            acc[2][v][j] = __builtin_fmaf(g[v][j], z[v][j], acc[2][v][j]);
          }
        }
      }
      const float r2 = uniform(y_rstd);
      if (kAhead) load_second(ahead);
      if (SAVED == kNoBranch && !p.dy) continue;
      if (!kAhead) vectors(false, true);
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) g[v][j] *= ky[v][j];
      if (SAVED == kNormed) {
        back_sums<V>(p, p.post, r2, sum, g, z, c, d);
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int j = 0; j < 8; ++j) g[v][j] = __builtin_fmaf(-c, z[v][j], __builtin_fmaf(r2, g[v][j], -d));
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int col = (v * nt + lane) * 8;
        store8<TYPE>(scalar_pointer(row_of<TYPE>(p.dy, row, p.lddy)), col, Cols<END>(col, p.cols), g[v]);
      }
    }
    GLOBAL char* part = scalar_pointer(row_of<PS_TYPE_F32>(p.part, blockIdx.x + seg, p.cols));
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int col = (v * nt + lane) * 8;
      const Cols<END> c8(col, p.cols);
      if (p.d_add) store8<PS_TYPE_F32, false>(part, col, c8, acc[0][v]);
      if (p.d_mul) store8<PS_TYPE_F32, false>(part + 4 * n_part, col, c8, acc[1][v]);
      if (p.d_gate || p.d_w1) store8<PS_TYPE_F32, false>(part + 8 * n_part, col, c8, acc[2][v]);
    }
  }
}

// The strips' parts, added up. A workgroup joins 32 columns of one gradient (and
// one segment of it where it has one for each): its groups of 32 lanes take the
// strips in turn, and their sums are added in order. 32 groups where there are
// many strips to a segment, else 8.
constexpr int kJoinCols = 32;

struct JoinOf {
  float* out;
  int which;      // 0 sum of dn, 1 of dn xh, 2 of G yh
  bool by_seg;
  bool by_gate;   // times the gate (that of the segment), before the segments are added
  bool by_w1;     // times post_weight, at the end
};

__device__ __forceinline__ float vec1(const void* v, int type, int64_t at) {
  if (type == PS_TYPE_F32) return ((const float*)v)[at];
  if (type == PS_TYPE_BF16) return bf16_lo(((const uint16_t*)v)[at]);
  return (float)((const _Float16*)v)[at];
}

template <int kJoinGroups>
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
#pragma unroll 8
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
  if (j.which == 2) total *= p.beta;
  if (j.by_w1) total *= vec1(p.w1, p.vec_type, col);
  float* out = j.out + (j.by_seg ? (int64_t)blockIdx.z * p.cols : 0) + col;
  *out = p.accumulate ? *out + total : total;
}

// Waves that hold `lanes` times eight columns, v times eight a lane.
int waves_for(int lanes, int v) { return (lanes + 64 * v - 1) / (64 * v); }

template <int TYPE, int END>
ps_status forward(const NormArgs& p, hipStream_t s) {
  const int lanes = (p.cols + 7) / 8;
  const dim3 four = grid_2d((p.rows + 3) / 4);
  if (END == kShort || lanes <= 64)
    hipLaunchKernelGGL((k_norm_forward<TYPE, 1, true, END>), four, dim3(256), 0, s, p);
  else if (lanes <= 128)
    hipLaunchKernelGGL((k_norm_forward<TYPE, 2, true, END == kShort ? kPart : END>), four, dim3(256), 0, s, p);
  else if (lanes > 512 && lanes <= 1024)   // 8192 x 5120 with two norms 104 -> 93 us, 8192 x 8192 136 -> 134
    hipLaunchKernelGGL((k_norm_forward<TYPE, 1, false, END == kShort ? kPart : END>), grid_2d(p.rows),
                       dim3(waves_for(lanes, 1) * 64), 0, s, p);
  else
    hipLaunchKernelGGL((k_norm_forward<TYPE, 2, false, END == kShort ? kPart : END>), grid_2d(p.rows),
                       dim3(waves_for(lanes, 2) * 64), 0, s, p);
  return hip_check(hipGetLastError(), "k_norm_forward launch");
}

template <int TYPE>
ps_status forward(const NormArgs& p, hipStream_t s) {
  switch (end_of(p.cols)) {
    case kWhole: return forward<TYPE, kWhole>(p, s);
    case kPart: return forward<TYPE, kPart>(p, s);
    default: return forward<TYPE, kShort>(p, s);
  }
}

template <int TYPE, int SAVED, int END>
ps_status backward(const NormArgs& p, hipStream_t s) {
  constexpr int kWideEnd = END == kShort ? kPart : END;
  const int lanes = (p.cols + 7) / 8;
  const dim3 grid((p.rows + p.strip - 1) / p.strip);
  if (lanes <= 1024 && lanes % 64 == 0 && END == kWhole)
    hipLaunchKernelGGL((k_norm_backward<TYPE, 1, SAVED, kEvery>), grid, dim3(lanes), 0, s, p);
  else if (lanes <= 1024)
    hipLaunchKernelGGL((k_norm_backward<TYPE, 1, SAVED, END>), grid, dim3(waves_for(lanes, 1) * 64), 0, s, p);
  else if (lanes <= 1536)
    hipLaunchKernelGGL((k_norm_backward<TYPE, 3, SAVED, kWideEnd>), grid, dim3(waves_for(lanes, 3) * 64), 0, s, p);
  else
    hipLaunchKernelGGL((k_norm_backward<TYPE, 4, SAVED, kWideEnd>), grid, dim3(waves_for(lanes, 4) * 64), 0, s, p);
  return hip_check(hipGetLastError(), "k_norm_backward launch");
}

template <int TYPE, int SAVED>
ps_status backward(const NormArgs& p, hipStream_t s) {
  switch (end_of(p.cols)) {
    case kWhole: return backward<TYPE, SAVED, kWhole>(p, s);
    case kPart: return backward<TYPE, SAVED, kPart>(p, s);
    default: return backward<TYPE, SAVED, kShort>(p, s);
  }
}

template <int TYPE>
ps_status backward(const NormArgs& p, hipStream_t s) {
  if (!p.dy || (p.post == PS_NORM_NONE && !p.gate)) return backward<TYPE, kNoBranch>(p, s);
  return p.post == PS_NORM_NONE ? backward<TYPE, kPlain>(p, s) : backward<TYPE, kNormed>(p, s);
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
  const dim3 grid((p.cols + kJoinCols - 1) / kJoinCols, n, by_seg ? p.n_segs : 1);
  if (p.slots / (by_seg ? p.n_segs : 1) > 128)
    hipLaunchKernelGGL(k_norm_join<32>, grid, dim3(kJoinCols * 32), 0, s, p, j[0], j[1], j[2], j[3]);
  else
    hipLaunchKernelGGL(k_norm_join<8>, grid, dim3(kJoinCols * 8), 0, s, p, j[0], j[1], j[2], j[3]);
  return hip_check(hipGetLastError(), "k_norm_join launch");
}

}  // namespace ps
