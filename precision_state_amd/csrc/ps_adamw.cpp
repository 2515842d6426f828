// ps_adamw.cpp - host side of the AdamW plan (ps_adamw_*): argument
// validation, the plan's layout in the caller's workspace, and dispatch.
//
// Workspace: control block | scalars of device-counted steps | counts of the
// norm's finished workgroups | their partial sums | step records by kind | their item ends | norm records | their
// chunk ends | slot of each list index in the step records. The tables are
// built once, on the host, and uploaded by ps_adamw_plan_create; afterwards
// only k_set_grads writes to them.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <vector>

#include "norm_keep.h"
#include "ps_adamw.h"

using namespace ps;

static_assert(sizeof(ps_adamw_control) == 64, "control block layout");
static_assert(sizeof(AwRec) == 80 && sizeof(AwNormRec) == 24, "record layout");

struct ps_adamw_plan {
  struct Range {   // bytes [lo, hi) of an array that the step writes
    uintptr_t lo, hi;
    int32_t tensor;
  };
  struct Grad {    // what a gradient array of list index i has to be
    int64_t n;
    int32_t type;
  };
  int device = 0;
  ps_adamw_control* ctl = nullptr;
  AwScalars* dev_sc = nullptr;
  double* partials = nullptr;
  uint32_t* counts = nullptr;   // the norm's finished workgroups; 0 between calls
  AwRec* recs = nullptr;
  AwNormRec* nrecs = nullptr;
  const uint32_t* slot = nullptr;
  AwTable table[kAwKinds] = {};
  uint32_t items[kAwKinds] = {};
  AwNormTable norm = {};
  uintptr_t ws_lo = 0, ws_hi = 0;   // the workspace's bytes
  std::vector<Range> written;       // sorted
  std::vector<Grad> grads;
  int32_t max_group = -1;
  bool lacks_residual = false;
  // the last step's scalars
  std::vector<ps_hparams> last_groups;
  int64_t last_step = 0;
  AwGroups sc = {};
  NadamProduct product[PS_ADAMW_MAX_GROUPS];
};

namespace {

constexpr size_t up256(size_t b) { return (b + 255) / 256 * 256; }
int elem_size(int32_t type) { return type == PS_TYPE_F32 ? 4 : 2; }

ps_status check(const void* p, const char* what, int i, uintptr_t align) {
  if (!p) return fail(PS_ERR_INVALID_ARG, "tensor %d: %s is NULL", i, what);
  if (!is_aligned(p, align)) return fail(PS_ERR_ALIGNMENT, "tensor %d: %s is not %d-byte aligned", i, what, (int)align);
  return PS_OK;
}

ps_status check_tensor(const ps_adamw_tensor& x, int i) {
  if (x.numel < 0 || x.numel > kMaxNumel)
    return fail(PS_ERR_SHAPE, "tensor %d: numel %lld out of range", i, (long long)x.numel);
  if (x.reserved) return fail(PS_ERR_INVALID_ARG, "tensor %d: reserved must be 0", i);
  if (x.grad_type < PS_TYPE_F32 || x.grad_type > PS_TYPE_F16)
    return fail(PS_ERR_INVALID_ARG, "tensor %d: unknown grad_type %d", i, x.grad_type);
  if (x.numel == 0) return PS_OK;
  ps_status s;
  if (x.grad && (s = check(x.grad, "grad", i, 16))) return s;
  if (!x.param) return PS_OK;
  if (x.param_type != PS_TYPE_F32 && x.param_type != PS_TYPE_BF16)
    return fail(x.param_type == PS_TYPE_F16 ? PS_ERR_UNSUPPORTED : PS_ERR_INVALID_ARG,
                "tensor %d: param_type %d is not F32 or BF16", i, x.param_type);
  if (x.state_type != PS_STATE_F32 && x.state_type != PS_STATE_E4M3)
    return fail(PS_ERR_INVALID_ARG, "tensor %d: unknown state_type %d", i, x.state_type);
  if (x.group < 0 || x.group >= PS_ADAMW_MAX_GROUPS)
    return fail(PS_ERR_INVALID_ARG, "tensor %d: group %d is not in 0..%d", i, x.group, PS_ADAMW_MAX_GROUPS - 1);
  if ((s = check(x.param, "param", i, 16)) || (s = check(x.m, "m", i, 16)) || (s = check(x.v, "v", i, 16))) return s;
  if (x.param_type == PS_TYPE_F32 && x.residual)
    return fail(PS_ERR_INVALID_ARG, "tensor %d: an F32 parameter has no residual", i);
  if (x.param_type == PS_TYPE_BF16 && x.copy)
    return fail(PS_ERR_INVALID_ARG, "tensor %d: a BF16 parameter has no copy", i);
  if (x.residual && (s = check(x.residual, "residual", i, 16))) return s;
  if (x.copy) {
    if (x.copy_type != PS_TYPE_BF16 && x.copy_type != PS_TYPE_F16)
      return fail(PS_ERR_INVALID_ARG, "tensor %d: copy_type %d is not BF16 or F16", i, x.copy_type);
    if ((s = check(x.copy, "copy", i, 16))) return s;
  }
  if (x.state_type == PS_STATE_E4M3 &&
      ((s = check(x.m_scale, "m_scale", i, 4)) || (s = check(x.v_scale, "v_scale", i, 4))))
    return s;
  return PS_OK;
}

int kind_of(const ps_adamw_tensor& x) {
  return (x.param_type == PS_TYPE_BF16 ? kAwBf16 : 0) | (x.grad_type == PS_TYPE_F32 ? kAwGrad32 : 0) |
         (x.state_type == PS_STATE_E4M3 ? kAwE4m3 : 0) | (x.copy ? kAwCopy : 0);
}

// Where the tables lie in the workspace.
struct Layout {
  size_t scalars, counts, partials, recs, ends, nrecs, nends, slot, bytes;
  int64_t n_step = 0, n_norm = 0;
  uint64_t items[kAwKinds] = {};
  uint64_t chunks = 0;
};

ps_status lay_out(const ps_adamw_tensor* t, int32_t n, Layout& l) {
  if (n < 0) return fail(PS_ERR_INVALID_ARG, "n_tensors < 0");
  if (n > 0 && !t) return fail(PS_ERR_INVALID_ARG, "tensors is NULL");
  for (int32_t i = 0; i < n; ++i) {
    if (ps_status s = check_tensor(t[i], i)) return s;
    if (t[i].numel == 0) continue;
    ++l.n_norm;
    l.chunks += (uint64_t)((t[i].numel + kNormChunk - 1) / kNormChunk);
    if (!t[i].param) continue;
    ++l.n_step;
    uint64_t& items = l.items[kind_of(t[i])];
    items += (uint64_t)((t[i].numel + kAwItemElems - 1) / kAwItemElems);
    if (items > kAwMaxItems) return fail(PS_ERR_SHAPE, "tensor list too large (more than %u work items)", kAwMaxItems);
  }
  if (l.chunks > 0x7FFFFFFFull) return fail(PS_ERR_SHAPE, "tensor list too large (more than 2^31 - 1 norm chunks)");
  size_t at = up256(sizeof(ps_adamw_control));
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += up256(bytes);
    return o;
  };
  l.scalars = take(sizeof(AwGroups));
  l.counts = take(sizeof(uint32_t) * kNormCountStride * (1 + kNormCounts));
  l.partials = take(sizeof(double) * (size_t)std::min<uint64_t>(std::max<uint64_t>(l.chunks, 1), kNormMaxWg));
  l.recs = take(sizeof(AwRec) * (size_t)l.n_step);
  l.ends = take(sizeof(uint32_t) * (size_t)l.n_step);
  l.nrecs = take(sizeof(AwNormRec) * (size_t)l.n_norm);
  l.nends = take(sizeof(uint32_t) * (size_t)l.n_norm);
  l.slot = take(2 * sizeof(uint32_t) * (size_t)n);
  l.bytes = at;
  return PS_OK;
}

// Arrays that the step writes, sorted; PS_ERR_INVALID_ARG if two overlap.
ps_status written_ranges(const ps_adamw_tensor* t, int32_t n, std::vector<ps_adamw_plan::Range>& out) {
  for (int32_t i = 0; i < n; ++i) {
    const ps_adamw_tensor& x = t[i];
    if (x.numel == 0 || !x.param) continue;
    auto add = [&](const void* p, int64_t bytes) {
      if (p) out.push_back({(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes, i});
    };
    const int64_t nb = (x.numel + kBlock - 1) / kBlock;
    const bool e8 = x.state_type == PS_STATE_E4M3;
    add(x.param, x.numel * elem_size(x.param_type));
    add(x.residual, 2 * x.numel);
    add(x.copy, 2 * x.numel);
    add(x.m, x.numel * (e8 ? 1 : 4));
    add(x.v, x.numel * (e8 ? 1 : 4));
    if (e8) {
      add(x.m_scale, 4 * nb);
      add(x.v_scale, 4 * nb);
    }
  }
  std::sort(out.begin(), out.end(), [](const auto& a, const auto& b) { return a.lo < b.lo; });
  for (size_t k = 1; k < out.size(); ++k)
    if (out[k].lo < out[k - 1].hi)
      return fail(PS_ERR_INVALID_ARG, "arrays of tensors %d and %d overlap", out[k - 1].tensor, out[k].tensor);
  return PS_OK;
}

ps_status check_grad(const ps_adamw_plan& p, const void* g, int32_t i) {
  if (!g || p.grads[i].n == 0) return PS_OK;
  if (ps_status s = check(g, "grad", i, 16)) return s;
  const uintptr_t lo = (uintptr_t)g, hi = lo + (uintptr_t)(p.grads[i].n * elem_size(p.grads[i].type));
  if (lo < p.ws_hi && p.ws_lo < hi) return fail(PS_ERR_INVALID_ARG, "tensor %d: grad overlaps the workspace", i);
  // the first written range that ends behind lo
  auto it = std::upper_bound(p.written.begin(), p.written.end(), lo, [](uintptr_t a, const auto& r) { return a < r.hi; });
  if (it != p.written.end() && it->lo < hi)
    return fail(PS_ERR_INVALID_ARG, "tensor %d: grad overlaps an array of tensor %d that the step writes", i, it->tensor);
  return PS_OK;
}

ps_status on_device(const ps_adamw_plan* p) {
  int dev = 0;
  if (ps_status s = hip_check(hipGetDevice(&dev), "hipGetDevice")) return s;
  if (dev != p->device)
    return fail(PS_ERR_INVALID_ARG, "the plan is on device %d, the current device is %d", p->device, dev);
  return PS_OK;
}

template <class F>
ps_status guarded(F f) {
  try {
    return f();
  } catch (const std::bad_alloc&) {
    return fail(PS_ERR_NO_MEMORY, "host allocation failed");
  }
}

ps_status create(const ps_adamw_tensor* t, int32_t n, void* workspace, size_t workspace_bytes, hipStream_t stream,
                 ps_adamw_plan** out) {
  Layout l;
  if (ps_status s = lay_out(t, n, l)) return s;
  ps_adamw_plan tmp;
  if (ps_status s = written_ranges(t, n, tmp.written)) return s;
  for (int32_t i = 0; i < n; ++i) tmp.grads.push_back({t[i].numel, t[i].grad_type});
  tmp.ws_lo = (uintptr_t)workspace;
  tmp.ws_hi = tmp.ws_lo + l.bytes;
  for (int32_t i = 0; i < n; ++i)
    if (ps_status s = check_grad(tmp, t[i].grad, i)) return s;
  if (!workspace || workspace_bytes < l.bytes)
    return fail(PS_ERR_WORKSPACE, "workspace is %zu bytes, %zu are needed", workspace ? workspace_bytes : (size_t)0, l.bytes);
  if (!is_aligned(workspace, 256)) return fail(PS_ERR_ALIGNMENT, "workspace is not 256-byte aligned");
  for (const auto& r : tmp.written)
    if (r.lo < tmp.ws_hi && tmp.ws_lo < r.hi)
      return fail(PS_ERR_INVALID_ARG, "the workspace overlaps an array of tensor %d", r.tensor);

  std::vector<unsigned char> image(l.bytes, 0);
  auto at = [&](size_t o) { return image.data() + o; };
  auto* ctl = (ps_adamw_control*)at(0);
  ctl->grad_mul = 1.0f;
  ctl->lr_mul = 1.0f;
  auto* recs = (AwRec*)at(l.recs);
  auto* ends = (uint32_t*)at(l.ends);
  auto* nrecs = (AwNormRec*)at(l.nrecs);
  auto* nends = (uint32_t*)at(l.nends);
  auto* slot = (uint32_t*)at(l.slot);
  char* w = (char*)workspace;
  size_t k = 0;
  for (int kind = 0; kind < kAwKinds; ++kind) {
    const size_t k0 = k;
    uint64_t items = 0;
    for (int32_t i = 0; i < n; ++i) {
      const ps_adamw_tensor& x = t[i];
      if (x.numel == 0 || !x.param || kind_of(x) != kind) continue;
      items += (uint64_t)((x.numel + kAwItemElems - 1) / kAwItemElems);
      recs[k] = AwRec{x.param, x.residual, x.copy, x.grad, x.m, x.m_scale, x.v, x.v_scale, x.numel, (uint32_t)i,
                      (uint8_t)x.group, (uint8_t)x.grad_type, (uint8_t)x.copy_type, 0};
      ends[k] = (uint32_t)items;
      slot[2 * i] = (uint32_t)(k + 1);   // 0: not a step tensor
      ++k;
      tmp.max_group = std::max(tmp.max_group, x.group);
      tmp.lacks_residual |= x.param_type == PS_TYPE_BF16 && !x.residual;
    }
    tmp.table[kind] = AwTable{(const AwRec*)(w + l.recs) + k0, (const uint32_t*)(w + l.ends) + k0, (int32_t)(k - k0)};
    tmp.items[kind] = (uint32_t)items;
  }
  uint64_t chunks = 0;
  size_t q = 0;
  for (int32_t i = 0; i < n; ++i) {
    if (t[i].numel == 0) continue;
    chunks += (uint64_t)((t[i].numel + kNormChunk - 1) / kNormChunk);
    nrecs[q] = AwNormRec{t[i].grad, t[i].numel, t[i].grad_type, 0};
    nends[q] = (uint32_t)chunks;
    slot[2 * i + 1] = (uint32_t)++q;
  }
  const uint64_t keep_from = norm_keep_from(
      tmp.grads, [](const auto& g) { return std::pair<int64_t, int64_t>(g.n, elem_size(g.type)); }, kNormChunk, kNormKeepBytes);
  tmp.norm = AwNormTable{(const AwNormRec*)(w + l.nrecs), (const uint32_t*)(w + l.nends), (int32_t)q, (uint32_t)chunks,
                         (uint32_t)keep_from, 0};
  tmp.ctl = (ps_adamw_control*)w;
  tmp.dev_sc = (AwScalars*)(w + l.scalars);
  tmp.partials = (double*)(w + l.partials);
  tmp.counts = (uint32_t*)(w + l.counts);
  tmp.recs = (AwRec*)(w + l.recs);
  tmp.nrecs = (AwNormRec*)(w + l.nrecs);
  tmp.slot = (const uint32_t*)(w + l.slot);

  if (ps_status s = hip_check(hipGetDevice(&tmp.device), "hipGetDevice")) return s;
  hipStreamCaptureStatus cap = hipStreamCaptureStatusNone;
  if (ps_status s = hip_check(hipStreamIsCapturing(stream, &cap), "hipStreamIsCapturing")) return s;
  if (cap != hipStreamCaptureStatusNone)
    return fail(PS_ERR_UNSUPPORTED, "a plan cannot be created while its stream is being captured");
  auto* plan = new ps_adamw_plan(std::move(tmp));
  ps_status s = hip_check(hipMemcpyAsync(workspace, image.data(), image.size(), hipMemcpyHostToDevice, stream),
                          "plan upload");
  const ps_status e = hip_check(hipStreamSynchronize(stream), "hipStreamSynchronize");
  if (!s) s = e;
  if (s) {
    delete plan;
    return s;
  }
  *out = plan;
  return PS_OK;
}

ps_status step(ps_adamw_plan* p, const ps_hparams* groups, int32_t n_groups, int64_t step, int32_t clipped,
               int32_t rounding, hipStream_t s) {
  if (n_groups < 1 || n_groups > PS_ADAMW_MAX_GROUPS)
    return fail(PS_ERR_INVALID_ARG, "n_groups is not in 1..%d", PS_ADAMW_MAX_GROUPS);
  if (!groups) return fail(PS_ERR_INVALID_ARG, "groups is NULL");
  if (p->max_group >= n_groups)
    return fail(PS_ERR_INVALID_ARG, "a tensor is in group %d of %d groups", p->max_group, n_groups);
  const bool same = p->last_step == step && step >= 1 && (int32_t)p->last_groups.size() == n_groups &&
                    memcmp(p->last_groups.data(), groups, sizeof(ps_hparams) * (size_t)n_groups) == 0;
  if (!same) {
    for (int32_t i = 0; i < n_groups; ++i) {
      if (ps_status st = check_hparams(&groups[i])) return st;
      if (groups[i].algo != groups[0].algo || groups[i].split_mode != groups[0].split_mode)
        return fail(PS_ERR_INVALID_ARG, "algo and split_mode must be the same in all groups");
    }
    if (step < 0) return fail(PS_ERR_INVALID_ARG, "step must be >= 0 (got %lld)", (long long)step);
    if (step == 0 && groups[0].algo != PS_ALGO_ADAM)
      return fail(PS_ERR_UNSUPPORTED, "steps counted on the device (step 0) need PS_ALGO_ADAM");
  }
  if (clipped != 0 && clipped != 1) return fail(PS_ERR_INVALID_ARG, "clipped must be 0 or 1");
  if (rounding != PS_ROUND_NEAREST && rounding != PS_ROUND_STOCHASTIC)
    return fail(PS_ERR_INVALID_ARG, "unknown rounding %d", rounding);
  if (p->lacks_residual && groups[0].split_mode != PS_SPLIT_STOCHASTIC)
    return fail(PS_ERR_INVALID_ARG, "a BF16 parameter has no residual: split_mode must be STOCHASTIC");
  if (ps_status st = on_device(p)) return st;
  if (step >= 1 && !same) {
    p->last_step = 0;
    p->last_groups.assign(groups, groups + n_groups);
    for (int32_t i = 0; i < n_groups; ++i) {
      StepScalars c;
      step_scalars_with(groups[i], step, groups[i].algo == PS_ALGO_NADAM ? nadam_product(groups[i], step, &p->product[i]) : 0.0, &c);
      p->sc.g[i] = AwScalars{c.B1, c.C1, c.B2, c.C2, c.EPS, c.A, c.RS2, c.AG, c.AM, c.CWD, c.sr_step, 0, groups[i].seed};
    }
    p->last_step = step;
  }
  // RS2 = 1 / sqrt(1 - beta2^t) is largest at t = 1; below 2^28 for every
  // double beta2 < 1 except the few next to 1.
  bool fast = true;
  for (int32_t i = 0; i < n_groups; ++i)
    fast &= groups[i].eps >= 0x1p-60 && groups[i].eps <= 0x1p58 && 1.0 - groups[i].beta2 >= 0x1p-56;
  const AwRun run{p->ctl, step == 0 ? p->dev_sc : nullptr, clipped, groups[0].algo == PS_ALGO_NADAM,
                  rounding == PS_ROUND_STOCHASTIC, fast};
  if (step == 0) {
    AwTick tick = {};
    for (int32_t i = 0; i < n_groups; ++i) {
      tick.lr[i] = groups[i].lr;
      tick.beta1[i] = groups[i].beta1;
      tick.beta2[i] = groups[i].beta2;
      tick.eps[i] = groups[i].eps;
      tick.wd[i] = groups[i].weight_decay;
      tick.seed[i] = groups[i].seed;
    }
    if (ps_status st = launch_adamw_tick(p->ctl, p->dev_sc, tick, n_groups, clipped, s)) return st;
  }
  for (int kind = 0; kind < kAwKinds; ++kind) {
    if (p->items[kind] == 0) continue;
    if (ps_status st = launch_adamw_step(kind, groups[0].split_mode, p->table[kind], p->items[kind], p->sc, run, s)) return st;
  }
  return PS_OK;
}

}  // namespace

extern "C" {

ps_status ps_adamw_workspace_size(const ps_adamw_tensor* tensors, int32_t n_tensors, size_t* bytes) {
  clear_error();
  if (!bytes) return fail(PS_ERR_INVALID_ARG, "bytes is NULL");
  Layout l;
  if (ps_status s = lay_out(tensors, n_tensors, l)) return s;
  *bytes = l.bytes;
  return PS_OK;
}

ps_status ps_adamw_plan_create(const ps_adamw_tensor* tensors, int32_t n_tensors, void* workspace,
                               size_t workspace_bytes, ps_stream_t stream, ps_adamw_plan** plan) {
  clear_error();
  if (!plan) return fail(PS_ERR_INVALID_ARG, "plan is NULL");
  *plan = nullptr;
  return guarded([&] { return create(tensors, n_tensors, workspace, workspace_bytes, (hipStream_t)stream, plan); });
}

ps_status ps_adamw_set_grads(ps_adamw_plan* plan, const void* const* grads, int32_t n_grads, ps_stream_t stream) {
  clear_error();
  if (!plan) return fail(PS_ERR_INVALID_ARG, "plan is NULL");
  if (n_grads != (int32_t)plan->grads.size())
    return fail(PS_ERR_INVALID_ARG, "n_grads is %d, the plan has %d tensors", n_grads, (int)plan->grads.size());
  if (n_grads == 0) return PS_OK;
  if (!grads) return fail(PS_ERR_INVALID_ARG, "grads is NULL");
  for (int32_t i = 0; i < n_grads; ++i)
    if (ps_status s = check_grad(*plan, grads[i], i)) return s;
  if (ps_status s = on_device(plan)) return s;
  return launch_set_grads(plan->recs, plan->nrecs, plan->slot, grads, n_grads, (hipStream_t)stream);
}

ps_status ps_adamw_grad_norm(ps_adamw_plan* plan, double max_norm, double grad_scale, ps_stream_t stream) {
  clear_error();
  if (!plan) return fail(PS_ERR_INVALID_ARG, "plan is NULL");
  if (!(max_norm > 0)) return fail(PS_ERR_INVALID_ARG, "max_norm must be > 0");
  if (!is_finite(grad_scale) || !(grad_scale > 0))
    return fail(PS_ERR_INVALID_ARG, "grad_scale must be finite and > 0");
  if (ps_status s = on_device(plan)) return s;
  return launch_grad_norm(plan->norm, plan->partials, plan->counts, plan->ctl, max_norm, grad_scale, (hipStream_t)stream);
}

ps_status ps_adamw_step(ps_adamw_plan* plan, const ps_hparams* groups, int32_t n_groups, int64_t step_no,
                        int32_t clipped, int32_t rounding, ps_stream_t stream) {
  clear_error();
  if (!plan) return fail(PS_ERR_INVALID_ARG, "plan is NULL");
  return guarded([&] { return step(plan, groups, n_groups, step_no, clipped, rounding, (hipStream_t)stream); });
}

ps_status ps_adamw_plan_destroy(ps_adamw_plan* plan) {
  clear_error();
  delete plan;
  return PS_OK;
}

ps_status ps_encode_fp8(const float* x, uint8_t* code, float* scale, int64_t n, int32_t kind, ps_stream_t stream) {
  clear_error();
  if (kind != PS_MOMENT_SIGNED && kind != PS_MOMENT_UNSIGNED) return fail(PS_ERR_INVALID_ARG, "unknown moment kind %d", kind);
  if (ps_status s = check_elementwise(n, {{x, "x"}, {code, "code"}}, {{scale, "scale"}})) return s;
  if (n == 0) return PS_OK;
  return launch_encode_fp8(x, code, scale, n, kind, (hipStream_t)stream);
}

ps_status ps_decode_fp8(const uint8_t* code, const float* scale, float* x, int64_t n, int32_t kind,
                        ps_stream_t stream) {
  clear_error();
  if (kind != PS_MOMENT_SIGNED && kind != PS_MOMENT_UNSIGNED) return fail(PS_ERR_INVALID_ARG, "unknown moment kind %d", kind);
  if (ps_status s = check_elementwise(n, {{x, "x"}, {code, "code"}}, {{scale, "scale"}})) return s;
  if (n == 0) return PS_OK;
  return launch_decode_fp8(code, scale, x, n, kind, (hipStream_t)stream);
}

}  // extern "C"
