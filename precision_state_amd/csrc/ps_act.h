// ps_act.h - declarations shared by the host side (ps_act.cpp) and the kernels
// (k_act.hip, k_block_norm.hip, k_wgrad.hip) of the activation checkpoints.
#pragma once

#include "ps_adamw.h"

namespace ps {

constexpr int kActBlock = PS_ACT_BLOCK;

// u / d for u < 2^31 and the d that it was made for (1 <= d < 2^31): with
// l = ceil(log2 d) and m = ceil(2^(31 + l) / d) < 2^32, u m / 2^(31 + l) is
// u / d plus an error below u / 2^(31 + l) < 1 / d, too small to reach the next
// whole number.
struct FastDiv {
  uint32_t d, m, s;
};
inline FastDiv fast_div(uint32_t d) {
  uint32_t l = 0;
  while ((1ull << l) < d) ++l;
  return {d, (uint32_t)(((1ull << (31 + l)) + d - 1) / d), 31 + l};
}

// Blocks of 128 columns of a matrix: unit u is block u % nb of row u / nb.
struct ActGrid {
  uint32_t units;
  FastDiv nb;
  int32_t cols;
};

struct GluArgs {
  const void *a, *b, *dout;
  void *out, *da, *db;
  int64_t lda, ldb, ldd, ldo;
  uint8_t *a_code, *b_code;
  float *a_scale, *b_scale;
};

ps_status launch_encode_act(const ActGrid& g, int type, const void* x, int64_t ld, uint8_t* code, float* scale, hipStream_t s);
ps_status launch_decode_act(const ActGrid& g, int type, const uint8_t* code, const float* scale, void* x, int64_t ld,
                            hipStream_t s);
ps_status launch_glu_forward(const ActGrid& g, int type, int act, const GluArgs& p, hipStream_t s);
ps_status launch_glu_backward(const ActGrid& g, int type, int act, const GluArgs& p, hipStream_t s);

// ---- block norms (k_block_norm.hip) ----
struct NormArgs {
  int32_t rows, cols, n_segs;
  const int32_t* seg_start;
  int32_t pre, post;
  uint32_t flags;
  int32_t vec_type;
  float pre_eps, post_eps, alpha, beta, inv_cols;
  const void *w1, *gate, *mul, *add;
  // forward
  const void *x, *y;
  void *h, *n;
  int64_t ldx, ldy, ldh, ldn;
  uint8_t *h_code, *y_code;
  float *h_rstd, *y_rstd, *y_scale;
  // backward (codes, rstd and scales as above, read)
  const void *dn, *dh;
  void *dx, *dy;
  int64_t lddn, lddh, lddx, lddy;
  float *d_w1, *d_gate, *d_mul, *d_add;
  float* part;              // [3][slots][cols]: sums of dn, dn * xh, G * yh over a strip's rows of a segment
  int32_t strip, slots;     // rows of a strip; strip i's part of segment b is slot i + b
  int32_t accumulate;
};
// Rows of a strip of the backward pass. At most as many strips as workgroups are
// at work at a time (16 waves a compute unit, 8 for the widest rows); of 16 rows
// at least, since a strip's sums cost as much memory traffic as one of its rows,
// but of two where that leaves less than 1024 strips, since rows take turns.
inline int32_t norm_strip_rows(int64_t rows, int64_t cols) {
  const int64_t lanes = (cols + 7) / 8, waves = (lanes + 63) / 64;
  const int64_t at_a_time = waves > 16 ? 256 : 256 * (16 / (waves > 0 ? waves : 1));
  int64_t strips = rows / 2 < 1024 ? (rows + 1) / 2 : 1024;
  if (strips < rows / 16) strips = rows / 16;
  if (strips > at_a_time) strips = at_a_time;
  return (int32_t)((rows + strips - 1) / strips);
}
ps_status launch_norm_forward(const NormArgs& p, int type, hipStream_t s);
ps_status launch_norm_backward(const NormArgs& p, int type, hipStream_t s);

// ---- weight gradients (k_wgrad.hip) ----
// How a product is cut: tiles of the result, and the tokens in splits of
// `per_split` whose partial results the join adds up (splits 1: none).
struct WgradCut {
  int32_t kind;              // index of the tile's shape
  int32_t tiles_n, tiles_k;
  int32_t splits;
  int64_t per_split;         // tokens, a multiple of the step
};
WgradCut wgrad_cut(int64_t tokens, int64_t n, int64_t k);

struct WgradArgs {
  int64_t tokens;
  int32_t n, k;
  const void* dy;
  int64_t lddy;
  const uint8_t* code;
  const float* scale;
  const float *mul, *add;
  void* dw;
  int64_t lddw;
  float* db;                 // the caller's, or NULL
  float* part;               // [splits][n][k], splits > 1
  float* db_part;            // [splits][n], splits > 1
  int32_t dy_type, dw_type, accumulate;
  WgradCut cut;
};
ps_status launch_wgrad(const WgradArgs& p, hipStream_t s);

}  // namespace ps
