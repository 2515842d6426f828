// ps_act.cpp - host side of the activation checkpoints: argument validation,
// all of it before any HIP call, and dispatch to the kernels.
#include "ps_act.h"

#include <cmath>

using namespace ps;

namespace {

constexpr int64_t kMaxRows = 0x7FFFFFFF, kMaxCols = int64_t(1) << 24, kMaxUnits = 0x7FFFFFFF;
constexpr int64_t kMaxNormRows = int64_t(1) << 30;   // a row and a step of the grid stay below 2^31
constexpr size_t up256(size_t b) { return (b + 255) / 256 * 256; }

int size_of(int32_t type) { return type == PS_TYPE_F32 ? 4 : 2; }
bool is_type(int32_t type) { return type == PS_TYPE_F32 || type == PS_TYPE_BF16 || type == PS_TYPE_F16; }
int64_t blocks_of(int64_t cols) { return (cols + kActBlock - 1) / kActBlock; }

ps_status check_shape(int64_t rows, int64_t cols) {
  if (rows < 0 || rows > kMaxRows) return fail(PS_ERR_SHAPE, "rows %lld out of range", (long long)rows);
  if (cols < 0 || cols > kMaxCols) return fail(PS_ERR_SHAPE, "cols %lld out of range", (long long)cols);
  if (rows * blocks_of(cols) > kMaxUnits) return fail(PS_ERR_SHAPE, "more than 2^31 - 1 blocks of 128 columns");
  return PS_OK;
}

// One array of a call: rows of `width` bytes, `pitch` bytes apart.
struct Span {
  const char* what;
  uintptr_t at;
  int64_t rows, width, pitch;
  bool written;
  const void* same_as;   // an array that it may be, whole
  uintptr_t end() const { return at + (uintptr_t)((rows - 1) * pitch + width); }
};

// Whether two arrays share bytes. Rows of the same pitch may lie side by side,
// as the halves of one matrix do.
bool overlap(const Span& a, const Span& b) {
  if (a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
  if (a.end() <= b.at || b.end() <= a.at) return false;
  if (a.pitch != b.pitch || a.rows == 1 || b.rows == 1) return true;
  const int64_t p = a.pitch;
  const int64_t d = b.at >= a.at ? (int64_t)((b.at - a.at) % (uintptr_t)p) : (p - (int64_t)((a.at - b.at) % (uintptr_t)p)) % p;
  return d < a.width || d + b.width > p;
}

// The arrays of a call, checked one by one and then against each other.
struct Arrays {
  static constexpr int kMost = 24;   // a norm's backward call has the most, 18
  Span v[kMost];
  int n = 0;
  ps_status status = PS_OK;

  void add(const void* p, const char* what, int64_t rows, int64_t cols, int64_t ld, int size, bool written,
           const void* same_as = nullptr) {
    if (status) return;
    if (n == kMost) {
      status = fail(PS_ERR_UNSUPPORTED, "more than %d arrays", kMost);
    } else if (!p) {
      status = fail(PS_ERR_INVALID_ARG, "%s is NULL", what);
    } else if (!is_aligned(p, (uintptr_t)size)) {
      status = fail(PS_ERR_ALIGNMENT, "%s is not %d-byte aligned", what, size);
    } else if (ld < cols || ld > (int64_t(1) << 40)) {
      status = fail(PS_ERR_SHAPE, "the rows of %s are %lld elements apart, cols is %lld", what, (long long)ld, (long long)cols);
    } else {
      v[n++] = {what, (uintptr_t)p, rows, cols * size, ld * size, written, same_as};
    }
  }
  void optional(const void* p, const char* what, int64_t rows, int64_t cols, int64_t ld, int size, bool written,
                const void* same_as = nullptr) {
    if (p) add(p, what, rows, cols, ld, size, written, same_as);
  }
  void codes(const void* p, const char* what, int64_t rows, int64_t cols, bool written) {
    add(p, what, rows, cols, cols, 1, written);
  }
  void scales(const void* p, const char* what, int64_t rows, int64_t cols, bool written) {
    add(p, what, rows, blocks_of(cols), blocks_of(cols), 4, written);
  }
  ps_status check() const {
    if (status) return status;
    for (int i = 0; i < n; ++i)
      for (int j = 0; j < i; ++j) {
        if (!v[i].written && !v[j].written) continue;
        if (!overlap(v[i], v[j])) continue;
        const Span &a = v[i], &b = v[j];
        const bool whole = a.at == b.at && a.pitch == b.pitch && a.width == b.width;
        if (whole && !(a.written && b.written) && (a.same_as == (const void*)b.at || b.same_as == (const void*)a.at)) continue;
        return fail(PS_ERR_INVALID_ARG, "%s and %s overlap", a.what, b.what);
      }
    return PS_OK;
  }
};

ActGrid grid_of(int64_t rows, int64_t cols) {
  return {(uint32_t)(rows * blocks_of(cols)), fast_div((uint32_t)blocks_of(cols)), (int32_t)cols};
}

ps_status check_codec(const void* x, int32_t type, int64_t rows, int64_t cols, int64_t ld, const uint8_t* code,
                      const float* scale, bool encode) {
  if (!is_type(type)) return fail(PS_ERR_INVALID_ARG, "unknown type %d", type);
  if (ps_status s = check_shape(rows, cols)) return s;
  if (rows == 0 || cols == 0) return PS_OK;
  Arrays a;
  a.add(x, "x", rows, cols, ld, size_of(type), !encode);
  a.codes(code, "code", rows, cols, encode);
  a.scales(scale, "scale", rows, cols, encode);
  return a.check();
}

ps_status check_glu(int64_t rows, int64_t cols, int32_t type, int32_t act) {
  if (!is_type(type)) return fail(PS_ERR_INVALID_ARG, "unknown type %d", type);
  if (act < PS_ACT_SILU || act > PS_ACT_GELU_TANH) return fail(PS_ERR_INVALID_ARG, "unknown activation %d", act);
  return check_shape(rows, cols);
}

// What a block norm's forward and backward calls have in common.
ps_status check_norm(const ps_block_norm* p) {
  if (!p) return fail(PS_ERR_INVALID_ARG, "norm is NULL");
  if (!is_type(p->type)) return fail(PS_ERR_INVALID_ARG, "unknown type %d", p->type);
  if (!is_type(p->vec_type)) return fail(PS_ERR_INVALID_ARG, "unknown vec_type %d", p->vec_type);
  if (p->pre_norm != PS_NORM_RMS && p->pre_norm != PS_NORM_LAYER)
    return fail(PS_ERR_INVALID_ARG, "pre_norm %d is not RMS or LAYER", p->pre_norm);
  if (p->post_norm < PS_NORM_NONE || p->post_norm > PS_NORM_LAYER)
    return fail(PS_ERR_INVALID_ARG, "unknown post_norm %d", p->post_norm);
  const uint32_t known = PS_NORM_GATE_BY_SEG | PS_NORM_MOD_BY_SEG | PS_NORM_MUL_PLUS_ONE;
  if (p->flags & ~known) return fail(PS_ERR_INVALID_ARG, "unknown flags 0x%x", p->flags & ~known);
  if (!is_finite(p->pre_eps) || p->pre_eps < 0 || !is_finite(p->post_eps) || p->post_eps < 0)
    return fail(PS_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (!is_finite(p->residual_scale) || !is_finite(p->branch_scale))
    return fail(PS_ERR_INVALID_ARG, "residual_scale and branch_scale must be finite");
  if (ps_status s = check_shape(p->rows, p->cols)) return s;
  if (p->rows > kMaxNormRows) return fail(PS_ERR_SHAPE, "rows %lld is more than 2^30", (long long)p->rows);
  if (p->cols > PS_NORM_MAX_COLS)
    return fail(PS_ERR_UNSUPPORTED, "cols %lld is more than %d", (long long)p->cols, PS_NORM_MAX_COLS);
  if (p->n_segs < 0 || p->n_segs > 65535) return fail(PS_ERR_SHAPE, "n_segs %d is not in 0..65535", p->n_segs);
  if ((p->n_segs > 0) != (p->seg_start != nullptr)) return fail(PS_ERR_INVALID_ARG, "n_segs and seg_start go together");
  if ((p->flags & (PS_NORM_GATE_BY_SEG | PS_NORM_MOD_BY_SEG)) && !p->n_segs)
    return fail(PS_ERR_INVALID_ARG, "vectors by segment need segments");
  if (p->post_weight && p->post_norm == PS_NORM_NONE) return fail(PS_ERR_INVALID_ARG, "post_weight needs a post_norm");
  if ((p->flags & PS_NORM_MUL_PLUS_ONE) && !p->mul) return fail(PS_ERR_INVALID_ARG, "MUL_PLUS_ONE needs mul");
  return PS_OK;
}

void add_vectors(const ps_block_norm& p, Arrays& a) {
  const int e = size_of(p.vec_type);
  const int64_t gates = p.flags & PS_NORM_GATE_BY_SEG ? p.n_segs : 1, mods = p.flags & PS_NORM_MOD_BY_SEG ? p.n_segs : 1;
  if (p.seg_start) a.add(p.seg_start, "seg_start", 1, p.n_segs + 1, p.n_segs + 1, 4, false);
  a.optional(p.post_weight, "post_weight", 1, p.cols, p.cols, e, false);
  a.optional(p.gate, "gate", gates, p.cols, p.cols, e, false);
  a.optional(p.mul, "mul", mods, p.cols, p.cols, e, false);
  a.optional(p.add, "add", mods, p.cols, p.cols, e, false);
}

NormArgs norm_args(const ps_block_norm& p) {
  NormArgs k = {};
  k.rows = (int32_t)p.rows;
  k.cols = (int32_t)p.cols;
  k.n_segs = p.n_segs;
  k.seg_start = p.seg_start;
  k.pre = p.pre_norm;
  k.post = p.post_norm;
  k.flags = p.flags;
  k.vec_type = p.vec_type;
  k.pre_eps = (float)p.pre_eps;
  k.post_eps = (float)p.post_eps;
  k.alpha = (float)p.residual_scale;
  k.beta = (float)p.branch_scale;
  k.inv_cols = p.cols ? (float)(1.0 / (double)p.cols) : 0.0f;
  k.w1 = p.post_weight;
  k.gate = p.gate;
  k.mul = p.mul;
  k.add = p.add;
  return k;
}

int64_t norm_slots(const ps_block_norm& p) {
  if (p.rows == 0 || p.cols == 0) return 0;
  const int64_t strip = norm_strip_rows(p.rows, p.cols);
  return (p.rows + strip - 1) / strip + (p.n_segs ? p.n_segs - 1 : 0);
}

size_t norm_workspace(const ps_block_norm& p) { return up256((size_t)norm_slots(p) * (size_t)p.cols * 3 * sizeof(float)); }

// The splits' partial results and column sums; a product of one split needs no workspace.
struct WgradLayout {
  size_t db_part, bytes;
};
WgradLayout wgrad_layout(const WgradCut& c, int64_t n, int64_t k) {
  if (c.splits == 1) return {0, 0};
  const size_t part = up256((size_t)c.splits * (size_t)n * (size_t)k * sizeof(float));
  return {part, part + up256((size_t)c.splits * (size_t)n * sizeof(float))};
}

ps_status check_wgrad_shape(int64_t tokens, int64_t n, int64_t k) {
  if (tokens < 0 || tokens > (int64_t(1) << 30)) return fail(PS_ERR_SHAPE, "tokens %lld out of range", (long long)tokens);
  if (n < 0 || n > kMaxCols) return fail(PS_ERR_SHAPE, "out_features %lld out of range", (long long)n);
  if (k < 0 || k > kMaxCols) return fail(PS_ERR_SHAPE, "in_features %lld out of range", (long long)k);
  if (n * k > (int64_t(1) << 36)) return fail(PS_ERR_SHAPE, "out_features * in_features is more than 2^36");
  if (tokens * blocks_of(k) > kMaxUnits) return fail(PS_ERR_SHAPE, "more than 2^31 - 1 blocks of 128 columns");
  return PS_OK;
}

}  // namespace

extern "C" {

ps_status ps_encode_act(const void* x, int32_t type, int64_t rows, int64_t cols, int64_t ld, uint8_t* code, float* scale,
                        ps_stream_t stream) {
  clear_error();
  if (ps_status s = check_codec(x, type, rows, cols, ld, code, scale, true)) return s;
  if (rows == 0 || cols == 0) return PS_OK;
  return launch_encode_act(grid_of(rows, cols), type, x, ld, code, scale, (hipStream_t)stream);
}

ps_status ps_decode_act(const uint8_t* code, const float* scale, void* x, int32_t type, int64_t rows, int64_t cols,
                        int64_t ld, ps_stream_t stream) {
  clear_error();
  if (ps_status s = check_codec(x, type, rows, cols, ld, code, scale, false)) return s;
  if (rows == 0 || cols == 0) return PS_OK;
  return launch_decode_act(grid_of(rows, cols), type, code, scale, x, ld, (hipStream_t)stream);
}

ps_status ps_glu_forward(int64_t rows, int64_t cols, int32_t type, int32_t act, const void* a, int64_t lda,
                         const void* b, int64_t ldb, void* out, int64_t ldo, uint8_t* a_code, float* a_scale,
                         uint8_t* b_code, float* b_scale, ps_stream_t stream) {
  clear_error();
  if (ps_status s = check_glu(rows, cols, type, act)) return s;
  if (rows == 0 || cols == 0) return PS_OK;
  const bool save = a_code || a_scale || b_code || b_scale;
  if (!b && (b_code || b_scale)) return fail(PS_ERR_INVALID_ARG, "b_code and b_scale need b");
  const int e = size_of(type);
  Arrays v;
  v.add(a, "a", rows, cols, lda, e, false);
  v.optional(b, "b", rows, cols, ldb, e, false);
  v.add(out, "out", rows, cols, ldo, e, true);
  if (save) {
    v.codes(a_code, "a_code", rows, cols, true);
    v.scales(a_scale, "a_scale", rows, cols, true);
    if (b) {
      v.codes(b_code, "b_code", rows, cols, true);
      v.scales(b_scale, "b_scale", rows, cols, true);
    }
  }
  if (ps_status s = v.check()) return s;
  GluArgs p = {};
  p.a = a; p.lda = lda;
  p.b = b; p.ldb = ldb;
  p.out = out; p.ldo = ldo;
  p.a_code = a_code; p.a_scale = a_scale;
  p.b_code = b_code; p.b_scale = b_scale;
  return launch_glu_forward(grid_of(rows, cols), type, act, p, (hipStream_t)stream);
}

ps_status ps_glu_backward(int64_t rows, int64_t cols, int32_t type, int32_t act, const void* dout, int64_t ldd,
                          const uint8_t* a_code, const float* a_scale, const uint8_t* b_code, const float* b_scale,
                          void* da, int64_t lda, void* db, int64_t ldb, void* out, int64_t ldo, ps_stream_t stream) {
  clear_error();
  if (ps_status s = check_glu(rows, cols, type, act)) return s;
  if (rows == 0 || cols == 0) return PS_OK;
  const bool gated = b_code || b_scale;
  if (!gated && db) return fail(PS_ERR_INVALID_ARG, "db needs b_code and b_scale");
  const int e = size_of(type);
  Arrays v;
  v.add(dout, "dout", rows, cols, ldd, e, false);
  v.codes(a_code, "a_code", rows, cols, false);
  v.scales(a_scale, "a_scale", rows, cols, false);
  v.add(da, "da", rows, cols, lda, e, true, dout);
  if (gated) {
    v.codes(b_code, "b_code", rows, cols, false);
    v.scales(b_scale, "b_scale", rows, cols, false);
    v.add(db, "db", rows, cols, ldb, e, true, dout);
  }
  v.optional(out, "out", rows, cols, ldo, e, true);
  if (ps_status s = v.check()) return s;
  GluArgs p = {};
  p.dout = dout; p.ldd = ldd;
  p.da = da; p.lda = lda;
  p.db = db; p.ldb = ldb;
  p.out = out; p.ldo = ldo;
  p.a_code = const_cast<uint8_t*>(a_code); p.a_scale = const_cast<float*>(a_scale);
  p.b_code = const_cast<uint8_t*>(b_code); p.b_scale = const_cast<float*>(b_scale);
  return launch_glu_backward(grid_of(rows, cols), type, act, p, (hipStream_t)stream);
}

ps_status ps_block_norm_forward(const ps_block_norm* norm, const ps_block_norm_fwd* io, ps_stream_t stream) {
  clear_error();
  if (ps_status s = check_norm(norm)) return s;
  if (!io) return fail(PS_ERR_INVALID_ARG, "io is NULL");
  const ps_block_norm& p = *norm;
  if (p.rows == 0 || p.cols == 0) return PS_OK;
  const int64_t rows = p.rows, cols = p.cols;
  const int e = size_of(p.type);
  const bool post = p.post_norm != PS_NORM_NONE;
  Arrays v;
  add_vectors(p, v);
  v.add(io->x, "x", rows, cols, io->ldx, e, false);
  if (io->y) {
    v.add(io->y, "y", rows, cols, io->ldy, e, false);
    v.add(io->h, "h", rows, cols, io->ldh, e, true, io->x);
  } else {
    if (io->h) return fail(PS_ERR_INVALID_ARG, "h needs y");
    if (post || p.gate) return fail(PS_ERR_INVALID_ARG, "a post_norm or gate needs y");
  }
  v.add(io->n, "n", rows, cols, io->ldn, e, true);
  if (io->h_code) v.codes(io->h_code, "h_code", rows, cols, true);
  v.optional(io->h_rstd, "h_rstd", 1, rows, rows, 4, true);
  if (io->y_code || io->y_scale || io->y_rstd) {
    if (!io->y || !(post || p.gate)) return fail(PS_ERR_INVALID_ARG, "y_code, y_scale and y_rstd need a post_norm or a gate");
    if (post ? io->y_scale != nullptr : io->y_rstd != nullptr)
      return fail(PS_ERR_INVALID_ARG, post ? "y_scale is for a call without a post_norm" : "y_rstd needs a post_norm");
    if (io->y_code) v.codes(io->y_code, "y_code", rows, cols, true);
    if (post) {
      v.optional(io->y_rstd, "y_rstd", 1, rows, rows, 4, true);
    } else {
      if (!io->y_code) return fail(PS_ERR_INVALID_ARG, "y_scale needs y_code");
      v.scales(io->y_scale, "y_scale", rows, cols, true);
    }
  }
  if (ps_status s = v.check()) return s;
  NormArgs k = norm_args(p);
  k.x = io->x; k.ldx = io->ldx;
  k.y = io->y; k.ldy = io->ldy;
  k.h = io->h; k.ldh = io->ldh;
  k.n = io->n; k.ldn = io->ldn;
  k.h_code = io->h_code; k.h_rstd = io->h_rstd;
  k.y_code = io->y_code; k.y_scale = io->y_scale; k.y_rstd = io->y_rstd;
  return launch_norm_forward(k, p.type, (hipStream_t)stream);
}

ps_status ps_block_norm_workspace_size(const ps_block_norm* norm, size_t* bytes) {
  clear_error();
  if (!bytes) return fail(PS_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = 0;
  if (ps_status s = check_norm(norm)) return s;
  *bytes = norm_workspace(*norm);
  return PS_OK;
}

ps_status ps_block_norm_backward(const ps_block_norm* norm, const ps_block_norm_bwd* io, ps_stream_t stream) {
  clear_error();
  if (ps_status s = check_norm(norm)) return s;
  if (!io) return fail(PS_ERR_INVALID_ARG, "io is NULL");
  if (io->reserved) return fail(PS_ERR_INVALID_ARG, "reserved must be 0");
  if (io->accumulate != 0 && io->accumulate != 1) return fail(PS_ERR_INVALID_ARG, "accumulate must be 0 or 1");
  const ps_block_norm& p = *norm;
  if (p.cols == 0) return PS_OK;
  const int64_t rows = p.rows, cols = p.cols;
  const int e = size_of(p.type);
  const bool post = p.post_norm != PS_NORM_NONE, branch = io->dy != nullptr;
  if (io->d_mul && !p.mul) return fail(PS_ERR_INVALID_ARG, "d_mul needs mul");
  if (io->d_add && !p.add) return fail(PS_ERR_INVALID_ARG, "d_add needs add");
  if (io->d_gate && !(p.gate && (branch || !rows))) return fail(PS_ERR_INVALID_ARG, "d_gate needs gate and dy");
  if (io->d_post_weight && !(p.post_weight && (branch || !rows)))
    return fail(PS_ERR_INVALID_ARG, "d_post_weight needs post_weight and dy");
  const int64_t gates = p.flags & PS_NORM_GATE_BY_SEG ? p.n_segs : 1, mods = p.flags & PS_NORM_MOD_BY_SEG ? p.n_segs : 1;
  Arrays v;
  add_vectors(p, v);
  if (rows) {
    v.add(io->dn, "dn", rows, cols, io->lddn, e, false);
    v.optional(io->dh, "dh", rows, cols, io->lddh, e, false);
    v.codes(io->h_code, "h_code", rows, cols, false);
    v.add(io->h_rstd, "h_rstd", 1, rows, rows, 4, false);
    const bool takes_dh = io->dx == io->dh;
    v.add(io->dx, "dx", rows, cols, io->lddx, e, true, takes_dh ? io->dh : io->dn);
    if (branch) {
      v.add(io->dy, "dy", rows, cols, io->lddy, e, true, io->dy == io->dh ? io->dh : io->dn);
      if (post || p.gate) v.codes(io->y_code, "y_code", rows, cols, false);
      if (post) v.add(io->y_rstd, "y_rstd", 1, rows, rows, 4, false);
      if (!post && p.gate) v.scales(io->y_scale, "y_scale", rows, cols, false);
    }
  }
  v.optional(io->d_post_weight, "d_post_weight", 1, cols, cols, 4, true);
  v.optional(io->d_gate, "d_gate", gates, cols, cols, 4, true);
  v.optional(io->d_mul, "d_mul", mods, cols, cols, 4, true);
  v.optional(io->d_add, "d_add", mods, cols, cols, 4, true);
  const size_t need = norm_workspace(p);
  if (need) {
    if (io->workspace_bytes < need)
      return fail(PS_ERR_WORKSPACE, "workspace has %zu bytes, %zu are needed", io->workspace_bytes, need);
    v.add(io->workspace, "workspace", 1, (int64_t)(need / 16), (int64_t)(need / 16), 16, true);
  }
  if (ps_status s = v.check()) return s;
  NormArgs k = norm_args(p);
  k.dn = io->dn; k.lddn = io->lddn;
  k.dh = io->dh; k.lddh = io->lddh;
  k.dx = io->dx; k.lddx = io->lddx;
  k.dy = io->dy; k.lddy = io->lddy;
  k.h_code = const_cast<uint8_t*>(io->h_code); k.h_rstd = const_cast<float*>(io->h_rstd);
  k.y_code = const_cast<uint8_t*>(io->y_code); k.y_scale = const_cast<float*>(io->y_scale);
  k.y_rstd = const_cast<float*>(io->y_rstd);
  k.d_w1 = io->d_post_weight; k.d_gate = io->d_gate;
  k.d_mul = io->d_mul; k.d_add = io->d_add;
  k.part = (float*)io->workspace;
  k.strip = rows ? norm_strip_rows(rows, cols) : 1;
  k.slots = (int32_t)norm_slots(p);
  k.accumulate = io->accumulate;
  return launch_norm_backward(k, p.type, (hipStream_t)stream);
}

ps_status ps_linear_wgrad_workspace_size(int64_t tokens, int64_t out_features, int64_t in_features, size_t* bytes) {
  clear_error();
  if (!bytes) return fail(PS_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = 0;
  if (ps_status s = check_wgrad_shape(tokens, out_features, in_features)) return s;
  if (out_features == 0 || in_features == 0) return PS_OK;
  *bytes = wgrad_layout(wgrad_cut(tokens, out_features, in_features), out_features, in_features).bytes;
  return PS_OK;
}

ps_status ps_linear_wgrad(const ps_linear_wgrad_args* args, ps_stream_t stream) {
  clear_error();
  if (!args) return fail(PS_ERR_INVALID_ARG, "args is NULL");
  const ps_linear_wgrad_args& a = *args;
  if (a.reserved) return fail(PS_ERR_INVALID_ARG, "reserved must be 0");
  if (a.dy_type != PS_TYPE_BF16 && a.dy_type != PS_TYPE_F16)
    return fail(a.dy_type == PS_TYPE_F32 ? PS_ERR_UNSUPPORTED : PS_ERR_INVALID_ARG, "dy_type %d is not BF16 or F16", a.dy_type);
  if (!is_type(a.dw_type)) return fail(PS_ERR_INVALID_ARG, "unknown dw_type %d", a.dw_type);
  if (a.accumulate != 0 && a.accumulate != 1) return fail(PS_ERR_INVALID_ARG, "accumulate must be 0 or 1");
  const int64_t t = a.tokens, n = a.out_features, k = a.in_features;
  if (ps_status s = check_wgrad_shape(t, n, k)) return s;
  if (n == 0 || k == 0) return PS_OK;
  Arrays v;
  if (t) {
    if (a.lddy > kMaxCols) return fail(PS_ERR_SHAPE, "lddy %lld is more than 2^24", (long long)a.lddy);
    v.add(a.dy, "dy", t, n, a.lddy, 2, false);
    v.codes(a.code, "code", t, k, false);
    if (a.scale) v.scales(a.scale, "scale", t, k, false);
  }
  v.optional(a.mul, "mul", 1, k, k, 4, false);
  v.optional(a.add, "add", 1, k, k, 4, false);
  v.add(a.dw, "dw", n, k, a.lddw, size_of(a.dw_type), true);
  v.optional(a.db, "db", 1, n, n, 4, true);
  const WgradCut cut = wgrad_cut(t, n, k);
  const WgradLayout l = wgrad_layout(cut, n, k);
  if (l.bytes) {
    if (a.workspace_bytes < l.bytes)
      return fail(PS_ERR_WORKSPACE, "workspace has %zu bytes, %zu are needed", a.workspace_bytes, l.bytes);
    v.add(a.workspace, "workspace", 1, (int64_t)(l.bytes / 16), (int64_t)(l.bytes / 16), 16, true);
  }
  if (ps_status s = v.check()) return s;
  WgradArgs p = {};
  p.tokens = t;
  p.n = (int32_t)n;
  p.k = (int32_t)k;
  p.dy = a.dy;
  p.lddy = a.lddy;
  p.code = a.code;
  p.scale = a.scale;
  p.mul = a.mul;
  p.add = a.add;
  p.dw = a.dw;
  p.lddw = a.lddw;
  p.db = a.db;
  char* ws = (char*)a.workspace;
  p.part = (float*)ws;
  p.db_part = (float*)(ws + l.db_part);
  p.dy_type = a.dy_type;
  p.dw_type = a.dw_type;
  p.accumulate = a.accumulate;
  p.cut = cut;
  return launch_wgrad(p, (hipStream_t)stream);
}

}  // extern "C"
