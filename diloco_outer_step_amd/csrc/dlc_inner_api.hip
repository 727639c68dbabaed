// C ABI of the learners' inner step (gradient norm, AdamW): argument checks, ranges and
// kernel launches.  As in the rest of the library nothing here allocates device memory,
// keeps state between calls or waits on the stream.
#include "dlc.h"
#include "dlc_host.h"
#include "dlc_inner.h"

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstring>
#include <string>
#include <vector>

namespace {

using dlc::aligned256;
using dlc::aligned8;
using dlc::check_tensors;
using dlc::fail;
using dlc::hip_fail;
using dlc::kMaxTensorNumel;
using dlc::no_throw;
using dlc::ok;
using dlc::round256;

constexpr int64_t kNormBlocks = 2048;

// A grid's x extent times its block must stay below 2^32 threads; a range has at most
// 2^32 / 256 = 2^24 AdamW tiles of 64 threads.
constexpr int64_t kMaxLaunchBlocks = int64_t(1) << 24;

struct InnerPartition {
  std::vector<dlc::InnerGeom> launches;
  int64_t n_slots = 0;
};

struct Range {
  int64_t lo, count;
  int32_t group;
};

// Tensors of one group that follow each other in the row without padding become one
// range (of at most 2^32 - 1 elements).
std::vector<Range> join_tensors(const dlc_tensor* t, int32_t n, const int32_t* group_of) {
  std::vector<Range> ranges;
  ranges.reserve(n);
  for (int32_t i = 0; i < n; ++i) {
    const int32_t group = group_of ? group_of[i] : 0;
    if (!ranges.empty()) {
      Range& b = ranges.back();
      if (b.group == group && b.lo + b.count == t[i].loffset && b.count + t[i].numel <= kMaxTensorNumel) {
        b.count += t[i].numel;
        continue;
      }
    }
    ranges.push_back({t[i].loffset, t[i].numel, group});
  }
  return ranges;
}

// Launches of at most kMaxRanges ranges, one block for every per_block elements of a range.
InnerPartition inner_partition(const std::vector<Range>& ranges, int64_t per_block) {
  InnerPartition p;
  for (const Range& r : ranges) {
    const int64_t blocks = (r.count + per_block - 1) / per_block;
    if (p.launches.empty() || p.launches.back().n_ranges == dlc::kMaxRanges ||
        p.launches.back().n_blocks + blocks > kMaxLaunchBlocks) {
      p.launches.emplace_back();
      std::memset(&p.launches.back(), 0, sizeof(dlc::InnerGeom));
      p.launches.back().per_block = (uint32_t)per_block;
      p.launches.back().slot_base = (int32_t)p.n_slots;
    }
    dlc::InnerGeom& g = p.launches.back();
    g.r[g.n_ranges++] = {(uint32_t)(r.lo / DLC_ALIGN_ELEMS), (uint32_t)r.count,
                         (uint32_t)g.n_blocks | (uint32_t)r.group << dlc::kGroupShift};
    g.n_blocks += (int32_t)blocks;
    p.n_slots += blocks;
  }
  for (dlc::InnerGeom& g : p.launches) {
    while ((int64_t)(g.n_blocks - 1) >> g.bucket_shift >= dlc::kRangeBuckets) ++g.bucket_shift;
    const auto range_of = [&](int64_t block, int32_t from) {
      while (from + 1 < g.n_ranges && g.r[from + 1].block_first() <= block) ++from;
      return from;
    };
    int32_t at = 0;
    for (int64_t k = 0; k << g.bucket_shift < g.n_blocks; ++k) {
      const int32_t first = range_of(k << g.bucket_shift, at);
      at = range_of(std::min<int64_t>(g.n_blocks, (k + 1) << g.bucket_shift) - 1, first);
      g.bucket[k] = (uint32_t)first | (uint32_t)at << 16;
    }
  }
  return p;
}

int64_t total_elements(const std::vector<Range>& ranges) {
  int64_t n = 0;
  for (const Range& r : ranges) n += r.count;
  return n;
}

InnerPartition norm_partition(const std::vector<Range>& ranges, int32_t bytes_per_element) {
  const int64_t step = dlc::kNormStep / bytes_per_element;
  const int64_t steps = (total_elements(ranges) + step - 1) / step;
  return inner_partition(ranges, step * std::max<int64_t>(1, (steps + kNormBlocks - 1) / kNormBlocks));
}

// Few elements in few ranges: one block per learner does it all, and there is no second
// launch.  One block against two kernels, us a call from Python / us a call replayed from a
// graph (fp32, one learner; 16-bit gradients and eight learners are within 10%, but for 2^17 and
// 2^18 elements):
//   1 range    2^13: 8.7, 10.8 / 2.7, 4.1   2^16: 8.9, 11.1 / 4.5, 4.4   2^18: 11.7, 11.1 / 10.6, 4.5
//   8 ranges   2^13: 9.0, 11.1 / 4.3, 4.3   2^16: 8.9, 11.1 / 5.9, 4.4   2^18: 13.2, 11.2 / 12.3, 4.5
//   32 ranges  2^13: 11.4, 11.2 / 10.3, 4.3
// The limits are the last place where no way of calling loses more than 1.5 us.
constexpr int64_t kSmallNorm = 1 << 16, kSmallNormRanges = 8;

bool small_norm(const std::vector<Range>& ranges) {
  return (int64_t)ranges.size() <= kSmallNormRanges && total_elements(ranges) <= kSmallNorm;
}

// Calls of at most this many blocks per learner count the step in the AdamW kernel itself:
// one launch less, at the price of a ticket a block on the learner's count.  Counted by the
// blocks against by a kernel of its own, us a call from Python (fp32 gradients, 32-bit moments):
//   1 learner   16 to 128 blocks: 10.1, 12.3
//   8 learners  to 48 blocks: 10.1, 12.3   64: 10.3, 12.3   80: 11.6, 12.3   96: 13.1, 12.3   128: 16.0, 12.3
//   16 learners to 32 blocks: 7.5, 9.9   64: 10.4, 10.0 (on another machine, as the next line)
//   64 learners to 16 blocks: 7.5, 9.9   32: 9.5, 9.9   64: 25.5, 10.0
// (coded, 8 learners: 64: 11.6, 13.3   80: 13.2, 13.4   96: 14.8, 13.9).  Replayed from a graph the extra
// launch costs less: 64 blocks 3.6, 3.8 and 96 blocks 4.0, 3.8 with one learner, but with eight 16 blocks 4.5, 3.9
// and 64 blocks 9.2, 4.1.  Far above the limit tickets are out of the question: 431 us
// for a call of 9100 blocks that takes 31.
constexpr int64_t kMaxTickets = 64;

// The present learners' indices -> list (zeroed before), their number; *rc is the status.
int32_t present_learners(int32_t n_learners, const uint8_t* present, dlc::LearnerList& list, int32_t* rc) {
  *rc = DLC_OK;
  if (n_learners < 1 || n_learners > DLC_MAX_LEARNERS) {
    *rc = fail(DLC_ERR_INVALID_ARGUMENT, "n_learners must be in [1, 64]");
    return 0;
  }
  int32_t kp = 0;
  for (int32_t i = 0; i < n_learners; ++i) {
    if (present != nullptr && present[i] == 0) continue;
    list.word[kp >> 2] |= (uint32_t)i << (8 * (kp & 3));
    ++kp;
  }
  if (kp == 0) *rc = fail(DLC_ERR_NO_QUORUM, "no learner is present");
  return kp;
}

// What a call uses of one of its device arrays: for learner i, `bytes` bytes at base + i * pitch
// (addresses as numbers; an absent array has no bytes).
struct Use {
  uintptr_t base;
  uint64_t pitch, bytes;
  bool written;
};

// A row buffer's elements of `size` bytes, from the first tensor's start to the last one's end.
struct RowSpan {
  int64_t first, last;
  RowSpan(const dlc_tensor* t, int32_t n) : first(t[0].loffset), last(0) {
    for (int32_t i = 0; i < n; ++i) {
      first = std::min(first, t[i].loffset);
      last = std::max(last, t[i].loffset + t[i].numel);
    }
  }
  Use rows(const void* p, int64_t stride, int64_t size, bool written) const {
    return {reinterpret_cast<uintptr_t>(p) + uint64_t(first) * size, uint64_t(stride) * size,
            p ? uint64_t(last - first) * size : 0, written};
  }
  Use scales(const void* p, int64_t stride) const {
    const int64_t lo = first / DLC_CODE_BLOCK, hi = (last + DLC_CODE_BLOCK - 1) / DLC_CODE_BLOCK;
    return {reinterpret_cast<uintptr_t>(p) + uint64_t(lo), uint64_t(stride) / DLC_CODE_BLOCK, p ? uint64_t(hi - lo) : 0,
            true};
  }
};

Use per_learner(const void* p, bool written) {
  return {reinterpret_cast<uintptr_t>(p), sizeof(double), p ? sizeof(double) : 0, written};
}

bool apart(const Use& a, const Use& b, const dlc::LearnerList& learner, int32_t n) {
  const auto clear = [](uintptr_t x, uint64_t nx, uintptr_t y, uint64_t ny) { return x + nx <= y || y + ny <= x; };
  if (a.bytes == 0 || b.bytes == 0) return true;
  const uint64_t lo = learner[0], span = learner[n - 1] - lo;
  if (clear(a.base + lo * a.pitch, span * a.pitch + a.bytes, b.base + lo * b.pitch, span * b.pitch + b.bytes)) return true;
  for (int32_t i = 0; i < n; ++i) {  // rows of two buffers may still take turns
    for (int32_t j = 0; j < n; ++j) {
      if (!clear(a.base + learner[i] * a.pitch, a.bytes, b.base + learner[j] * b.pitch, b.bytes)) return false;
    }
  }
  return true;
}

// No array that is written may share memory with another one: blocks of a launch run in any order.
int32_t check_apart(const Use* use, int32_t n_uses, const dlc::LearnerList& learner, int32_t n) {
  for (int32_t a = 0; a < n_uses; ++a) {
    for (int32_t b = 0; b < a; ++b) {
      if ((use[a].written || use[b].written) && !apart(use[a], use[b], learner, n))
        return fail(DLC_ERR_INVALID_ARGUMENT, "the call's buffers must not overlap");
    }
  }
  return DLC_OK;
}

int32_t check_float_type(int32_t type, const char* name, bool wide) {
  if (type == DLC_BFLOAT16 || type == DLC_FLOAT16 || (wide && type == DLC_FLOAT32)) return DLC_OK;
  return fail(DLC_ERR_INVALID_ARGUMENT, std::string(name) + " is not one of the call's types");
}

int32_t element_bytes(int32_t type) { return type == DLC_FLOAT32 ? 4 : 2; }

// The moments of an AdamW call: 32-bit, or codes and scale bytes.
struct Moments {
  void* m;
  void* v;
  uint8_t* m_scales;
  uint8_t* v_scales;
  bool coded;
  uint64_t seed;
};

int32_t adamw_step(float* theta_learners, const void* grads, int32_t grad_type, const Moments& mo, int64_t* steps,
                   int64_t learner_stride, int32_t n_learners, const uint8_t* present, const dlc_tensor* tensors,
                   int32_t n_tensors, const int32_t* group_of, const dlc_adamw_group* groups, int32_t n_groups,
                   const double* grad_scale, const double* lr_scale, void* working, int32_t working_type,
                   void* hip_stream) {
  dlc::AdamWArgs a;
  std::memset(&a, 0, sizeof(a));
  int32_t rc;
  a.n_present = present_learners(n_learners, present, a.learner, &rc);
  if (rc != DLC_OK) return rc;
  if (!theta_learners || !grads || !mo.m || !mo.v || !steps || (mo.coded && (!mo.m_scales || !mo.v_scales)))
    return fail(DLC_ERR_INVALID_ARGUMENT, "theta_learners, grads, the moments and steps must not be NULL");
  const void* buffers[] = {theta_learners, grads, mo.m, mo.v, mo.m_scales, mo.v_scales, working};
  for (const void* p : buffers) {
    if (!aligned256(p)) return fail(DLC_ERR_ALIGNMENT, "device pointers must be 256-byte aligned");
  }
  if (!aligned8(steps) || !aligned8(grad_scale) || !aligned8(lr_scale))
    return fail(DLC_ERR_ALIGNMENT, "steps, grad_scale and lr_scale must be 8-byte aligned");
  rc = check_float_type(grad_type, "grad_type", true);
  if (rc == DLC_OK && working) rc = check_float_type(working_type, "working_type", false);
  if (rc == DLC_OK) rc = check_tensors(tensors, n_tensors, learner_stride, true);
  if (rc != DLC_OK) return rc;
  const RowSpan span(tensors, n_tensors);
  const int64_t moment = mo.coded ? 1 : 4;
  const Use uses[] = {span.rows(theta_learners, learner_stride, 4, true),
                      span.rows(grads, learner_stride, element_bytes(grad_type), false),
                      span.rows(mo.m, learner_stride, moment, true),
                      span.rows(mo.v, learner_stride, moment, true),
                      span.scales(mo.m_scales, learner_stride),
                      span.scales(mo.v_scales, learner_stride),
                      span.rows(working, learner_stride, 2, true),
                      per_learner(steps, true),
                      per_learner(grad_scale, false),
                      per_learner(lr_scale, false)};
  rc = check_apart(uses, (int32_t)(sizeof(uses) / sizeof(uses[0])), a.learner, a.n_present);
  if (rc != DLC_OK) return rc;
  if (!groups || n_groups < 1 || n_groups > DLC_MAX_GROUPS)
    return fail(DLC_ERR_INVALID_ARGUMENT, "groups must hold 1 to 16 groups");
  for (int32_t q = 0; q < n_groups; ++q) {
    const dlc_adamw_group& s = groups[q];
    if (!(std::isfinite(s.lr) && s.lr >= 0.0 && std::isfinite(s.weight_decay) && s.weight_decay >= 0.0))
      return fail(DLC_ERR_INVALID_ARGUMENT, "lr and weight_decay must be finite and >= 0");
    if (!(s.beta1 >= 0.0 && s.beta1 < 1.0 && s.beta2 >= 0.0 && s.beta2 < 1.0))
      return fail(DLC_ERR_INVALID_ARGUMENT, "betas must be in [0, 1)");
    // Past 2^126 the reciprocal of the update's denominator would be subnormal, which the hardware's gives as 0.
    if (!(s.eps >= FLT_MIN && s.eps <= 0x1p126))
      return fail(DLC_ERR_INVALID_ARGUMENT, "eps must be in [2^-126, 2^126]");
    a.group[q] = {s.lr, s.beta1, s.beta2, s.eps, s.weight_decay, std::log(s.beta1), std::log(s.beta2)};
  }
  if (group_of) {
    for (int32_t t = 0; t < n_tensors; ++t)
      if (group_of[t] < 0 || group_of[t] >= n_groups)
        return fail(DLC_ERR_INVALID_ARGUMENT, "tensor " + std::to_string(t) + ": no such group");
  }
  a.theta = theta_learners;
  a.grads = grads;
  a.m = mo.m;
  a.v = mo.v;
  a.m_scale = mo.m_scales;
  a.v_scale = mo.v_scales;
  a.working = working;
  a.steps = steps;
  a.grad_scale = grad_scale;
  a.lr_scale = lr_scale;
  a.stride = learner_stride;
  a.seed = mo.seed;
  const hipStream_t s = static_cast<hipStream_t>(hip_stream);
  const InnerPartition p = inner_partition(join_tensors(tensors, n_tensors, group_of),
                                           mo.coded ? dlc::kCodedTile : dlc::kAdamWTile);
  if (p.n_slots <= kMaxTickets && p.launches.size() == 1) a.tickets = (int32_t)p.n_slots;
  for (const dlc::InnerGeom& g : p.launches) {
    const hipError_t e = dlc::launch_adamw(a, grad_type, working ? working_type : dlc::kNone, mo.coded, g, s);
    if (e != hipSuccess) return hip_fail(e, "AdamW kernel launch");
  }
  if (a.tickets == 0) {
    const hipError_t e = dlc::launch_adamw_advance(a, s);
    if (e != hipSuccess) return hip_fail(e, "step count kernel launch");
  }
  return ok();
}

}  // namespace

extern "C" {

int32_t dlc_grad_norm_workspace_bytes(int32_t n_learners, const dlc_tensor* tensors, int32_t n_tensors,
                                      size_t* bytes) {
  return no_throw([&]() -> int32_t {
    if (!bytes) return fail(DLC_ERR_INVALID_ARGUMENT, "bytes is NULL");
    if (n_learners < 1 || n_learners > DLC_MAX_LEARNERS)
      return fail(DLC_ERR_INVALID_ARGUMENT, "n_learners must be in [1, 64]");
    const int32_t rc = check_tensors(tensors, n_tensors, 0, false);
    if (rc != DLC_OK) return rc;
    // blocks of 16-bit gradients have at least as many elements: no type has more slots than fp32
    const InnerPartition p = norm_partition(join_tensors(tensors, n_tensors, nullptr), 4);
    *bytes = round256((size_t)p.n_slots * n_learners * sizeof(double));
    return ok();
  });
}

int32_t dlc_grad_norm(const void* grads, int32_t grad_type, int64_t learner_stride, int32_t n_learners,
                      const uint8_t* present, const dlc_tensor* tensors, int32_t n_tensors, double unscale,
                      double max_norm, double* norm, double* grad_scale, void* workspace, size_t workspace_bytes,
                      void* hip_stream) {
  return no_throw([&]() -> int32_t {
    dlc::NormArgs a;
    std::memset(&a, 0, sizeof(a));
    int32_t rc;
    a.n_present = present_learners(n_learners, present, a.learner, &rc);
    if (rc != DLC_OK) return rc;
    if (!grads || !norm || !grad_scale)
      return fail(DLC_ERR_INVALID_ARGUMENT, "grads, norm and grad_scale must not be NULL");
    if (!aligned256(grads)) return fail(DLC_ERR_ALIGNMENT, "device pointers must be 256-byte aligned");
    if (!aligned8(norm) || !aligned8(grad_scale))
      return fail(DLC_ERR_ALIGNMENT, "norm and grad_scale must be 8-byte aligned");
    rc = check_float_type(grad_type, "grad_type", true);
    if (rc == DLC_OK) rc = check_tensors(tensors, n_tensors, learner_stride, true);
    if (rc != DLC_OK) return rc;
    if (!(std::isfinite(unscale) && unscale > 0.0))
      return fail(DLC_ERR_INVALID_ARGUMENT, "unscale must be finite and > 0");
    if (!(max_norm > 0.0)) return fail(DLC_ERR_INVALID_ARGUMENT, "max_norm must be > 0");
    const std::vector<Range> ranges = join_tensors(tensors, n_tensors, nullptr);
    const InnerPartition p = norm_partition(ranges, element_bytes(grad_type));
    const size_t need = round256((size_t)p.n_slots * a.n_present * sizeof(double));
    if (workspace == nullptr || workspace_bytes < need)
      return fail(DLC_ERR_WORKSPACE, "workspace too small: need " + std::to_string(need) + " bytes");
    if (!aligned256(workspace)) return fail(DLC_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
    const Use uses[] = {RowSpan(tensors, n_tensors).rows(grads, learner_stride, element_bytes(grad_type), false),
                        per_learner(norm, true), per_learner(grad_scale, true),
                        {reinterpret_cast<uintptr_t>(workspace), 0, need, true}};
    rc = check_apart(uses, (int32_t)(sizeof(uses) / sizeof(uses[0])), a.learner, a.n_present);
    if (rc != DLC_OK) return rc;
    a.grads = grads;
    a.stride = learner_stride;
    a.part = static_cast<double*>(workspace);
    a.norm = norm;
    a.grad_scale = grad_scale;
    a.unscale = unscale;
    a.max_norm = max_norm;
    a.n_slots = (int32_t)p.n_slots;
    const hipStream_t s = static_cast<hipStream_t>(hip_stream);
    if (small_norm(ranges)) {
      const hipError_t e = dlc::launch_norm_small(a, grad_type, p.launches[0], s);
      return e != hipSuccess ? hip_fail(e, "gradient norm kernel launch") : ok();
    }
    for (const dlc::InnerGeom& g : p.launches) {
      const hipError_t e = dlc::launch_norm_partial(a, grad_type, g, s);
      if (e != hipSuccess) return hip_fail(e, "gradient norm kernel launch");
    }
    const hipError_t e = dlc::launch_norm_final(a, s);
    if (e != hipSuccess) return hip_fail(e, "gradient norm kernel launch");
    return ok();
  });
}

int32_t dlc_adamw_step(float* theta_learners, const void* grads, int32_t grad_type, float* exp_avg,
                       float* exp_avg_sq, int64_t* steps, int64_t learner_stride, int32_t n_learners,
                       const uint8_t* present, const dlc_tensor* tensors, int32_t n_tensors, const int32_t* group_of,
                       const dlc_adamw_group* groups, int32_t n_groups, const double* grad_scale,
                       const double* lr_scale, void* working, int32_t working_type, void* hip_stream) {
  return no_throw([&]() -> int32_t {
    return adamw_step(theta_learners, grads, grad_type, {exp_avg, exp_avg_sq, nullptr, nullptr, false, 0}, steps,
                      learner_stride, n_learners, present, tensors, n_tensors, group_of, groups, n_groups, grad_scale,
                      lr_scale, working, working_type, hip_stream);
  });
}

int32_t dlc_adamw_coded_step(float* theta_learners, const void* grads, int32_t grad_type, uint8_t* m_codes,
                             uint8_t* m_scales, uint8_t* v_codes, uint8_t* v_scales, int64_t* steps,
                             int64_t learner_stride, int32_t n_learners, const uint8_t* present,
                             const dlc_tensor* tensors, int32_t n_tensors, const int32_t* group_of,
                             const dlc_adamw_group* groups, int32_t n_groups, uint64_t seed,
                             const double* grad_scale, const double* lr_scale, void* working, int32_t working_type,
                             void* hip_stream) {
  return no_throw([&]() -> int32_t {
    return adamw_step(theta_learners, grads, grad_type, {m_codes, v_codes, m_scales, v_scales, true, seed}, steps,
                      learner_stride, n_learners, present, tensors, n_tensors, group_of, groups, n_groups, grad_scale,
                      lr_scale, working, working_type, hip_stream);
  });
}

}  // extern "C"
