// ps_adamw.h - declarations shared by the AdamW plan's host side
// (ps_adamw.cpp) and kernels (k_adamw.hip). Not part of the public ABI.
#pragma once

#include <initializer_list>
#include <utility>

#include "ps_internal.h"

namespace ps {

constexpr int kAwItemElems = 512;     // step work item: one 64-lane wave, 8 elements per lane, two blocks
constexpr uint32_t kAwMaxItems = 0xFFFFFFFFu / 64;   // a launch has fewer than 2^32 lanes
constexpr int kNormChunk = 8192;      // norm work item: one 256-thread workgroup, 32 elements per thread
constexpr uint32_t kNormMaxWg = 1024;      // norm workgroups (and partial sums) at most
constexpr int64_t kNormKeepBytes = 256 << 20;   // the last-level cache's size
constexpr uint32_t kNormCounts = 32;      // first-level counts of finished norm workgroups
constexpr uint32_t kNormCountStride = 64; // words from one to the next: each on a cache line of its own
constexpr int kAwGrads = 384;         // gradient pointers in one k_set_grads launch

// Kinds of step tensors: each kind of the list is one launch of its own kernel.
constexpr int kAwBf16 = 1, kAwGrad32 = 2, kAwE4m3 = 4, kAwCopy = 8, kAwKinds = 16;

struct AwRec {       // one tensor of a step
  void* w;
  uint16_t* lo;
  void* copy;
  const void* g;     // NULL: passed by
  void* m;
  float* ms;
  void* v;
  float* vs;
  int64_t n;
  uint32_t tid;      // index in the caller's list (stochastic rounding stream key)
  uint8_t group, gtype, ctype, pad;
};

struct AwTable {     // tensor i owns the work items [item_end[i-1], item_end[i])
  const AwRec* recs;
  const uint32_t* item_end;
  int32_t n;
};

struct AwNormRec {
  const void* g;     // NULL: passed by
  int64_t n;
  int32_t gtype;
  int32_t pad;
};

struct AwNormTable {
  const AwNormRec* recs;
  const uint32_t* chunk_end;
  int32_t n;
  uint32_t chunks;
  uint32_t keep_from;  // chunks from here on are read so that they stay in the last-level cache
  uint32_t pad;
};

// Scalars of one group, by value in the kernel arguments or, when the step is
// counted on the device, in the workspace.
struct AwScalars {
  float B1, C1, B2, C2, EPS, A, RS2, AG, AM, CWD;
  uint32_t sr_step, pad;
  uint64_t sr_seed;
};

struct AwGroups {
  AwScalars g[PS_ADAMW_MAX_GROUPS];
};

struct AwTick {      // hyperparameters for scalars computed on the device
  double lr[PS_ADAMW_MAX_GROUPS], beta1[PS_ADAMW_MAX_GROUPS], beta2[PS_ADAMW_MAX_GROUPS], eps[PS_ADAMW_MAX_GROUPS],
      wd[PS_ADAMW_MAX_GROUPS];
  uint64_t seed[PS_ADAMW_MAX_GROUPS];
};

// What a step's kernels take besides the table and the scalars.
struct AwRun {
  const ps_adamw_control* ctl;
  const AwScalars* dev_sc;   // non-NULL: scalars counted on the device
  int32_t clipped, nadam, round_sr;
  int32_t fast;              // EPS and RS2 of all groups are in the fast quotient's range
};

ps_status launch_adamw_step(int kind, int split, const AwTable& t, uint32_t items, const AwGroups& sc, const AwRun& run,
                            hipStream_t s);
ps_status launch_adamw_tick(ps_adamw_control* ctl, AwScalars* sc, const AwTick& hp, int n_groups, int clipped,
                            hipStream_t s);
ps_status launch_grad_norm(const AwNormTable& t, double* partials, uint32_t* counts, ps_adamw_control* ctl,
                           double max_norm, double grad_scale, hipStream_t s);
ps_status launch_set_grads(AwRec* recs, AwNormRec* nrecs, const uint32_t* slot, const void* const* grads, int32_t n,
                           hipStream_t s);
ps_status launch_encode_fp8(const float* x, uint8_t* code, float* scale, int64_t n, int kind, hipStream_t s);
ps_status launch_decode_fp8(const uint8_t* code, const float* scale, float* x, int64_t n, int kind, hipStream_t s);

// ---- host scalars (ps_scalars.cpp) ----
// P_t = mu_1 ... mu_t of NAdam, carried from one update to the next: a training
// loop multiplies once per step where the product from the start takes hundreds
// of pow() calls (the same factors in the same order, so the same double).
struct NadamProduct {
  double beta1 = 0, psi = 0;
  int64_t t = -1;
  double prod = 1.0;
};
double nadam_product(const ps_hparams& hp, int64_t t, NadamProduct* last);
void step_scalars_with(const ps_hparams& hp, int64_t t, double prod, StepScalars* o);

// ---- argument checks shared with the other entry points (ps_abi.cpp) ----
ps_status check_hparams(const ps_hparams* hp);
void clear_error();
ps_status check_elementwise(int64_t n, std::initializer_list<std::pair<const void*, const char*>> arrays,
                            std::initializer_list<std::pair<const void*, const char*>> scales);
constexpr int64_t kMaxNumel = int64_t(1) << 40;

}  // namespace ps
