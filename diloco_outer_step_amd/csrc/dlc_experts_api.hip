// C ABI of the mixture-of-experts calls (the router's balance loss, merge weights from expert
// counts): argument checks, block partition and kernel launches.  As in the rest of the
// library nothing here allocates device memory, keeps state between calls or waits on the
// stream.
#include "dlc.h"
#include "dlc_experts.h"
#include "dlc_host.h"

#include <algorithm>
#include <cmath>
#include <cstring>
#include <string>

namespace {

using dlc::aligned256;
using dlc::aligned8;
using dlc::fail;
using dlc::hip_fail;
using dlc::no_throw;
using dlc::ok;
using dlc::round256;

static_assert(dlc::kMaxExperts == DLC_MAX_EXPERTS && dlc::kMaxChoices == DLC_MAX_CHOICES);
static_assert((dlc::kCountTokens - 1) * (int64_t)DLC_MAX_CHOICES * (DLC_MAX_CHOICES - 1) < (int64_t(1) << 32));

// Blocks over the logits, all learners: four for each CU, so all of them run at once and what a block
// does before and after its tokens (2 us) is done once.  1024, 1280 blocks: 32768 x 256 x 8 bf16 with the gradient
// 63.8, 65.5 us, 16384 x 128 x 8 without 17.8, 19.7 us (2048: 23.8 against 19.7 of an earlier form).
constexpr int64_t kBalanceBlocks = 1024;
constexpr int64_t kMinSteps = 2;           // of a block over the logits (1 or 2 are the same within 2%)
// Choices of a counting block: one load of 8 for each of its 512 threads (2048 and 8192 are within 1 us).
constexpr int64_t kCountChoices = 4096;
constexpr int64_t kMaxCountBlocks = 32;    // per learner, as long as a block's tokens stay below kCountTokens
// Up to so many choices every block counts all of its learner's for itself, which saves the counting kernel: four
// rounds of 8 loads a thread, which take no longer (and eagerly 3 us less).  With 20000 choices it is 26 us a
// call against 16.
constexpr int64_t kSelfCount = 8192;
// Up to so many sums (blocks times experts) one block a learner does the final ones: above it a single CU's
// loads take longer than the ticket of several blocks (16384 sums: 20.4 us a call against 18.5).
constexpr int64_t kOneFinal = 8192;
constexpr int64_t kMaxReach = int64_t(1) << 48;  // of a strided array, in elements

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Calls of so few steps run in one block per learner.  One block against the passes over the logits and the
// final sums (us a call replayed from a graph, eight learners, bf16 / eagerly, one learner):
//   64 experts    128 tokens: 6.5, 9.8 / 9.2, 12.7   512: 9.2, 9.8 / 9.3, 12.8   1024: 12.9, 11.1 / 12.6, 12.5
//   256 experts    32 tokens: 7.5, 9.7 / 9.1, 12.5    64: 10.0, 10.0 / 9.9, 12.6   128: 14.9, 10.4 / 14.4, 12.6
//   8 experts     256 tokens: 7.8, 10.0 / 9.6, 12.9  1024: 13.3, 10.5 / 13.1, 12.7
// a step being 64, 8 and 64 tokens.
constexpr int64_t kOneSteps = 8;
constexpr int64_t kOneChoices = 8192;

bool one_block(int64_t tokens, int32_t experts, int64_t top, int32_t type) {
  static_assert(kOneSteps * dlc::kBalanceOne <= dlc::kBlockTokens);
  return tokens <= kOneSteps * dlc::balance_one_tokens(type, experts) && tokens * top <= kOneChoices;
}

struct BalancePartition {
  int64_t count_blocks, count_tokens, blocks, block_tokens;
};

BalancePartition balance_partition(int64_t tokens, int32_t experts, int64_t top, int32_t type, int32_t present,
                                   bool gradient) {
  BalancePartition p;
  const int64_t step = dlc::balance_tokens(type, experts, dlc::kBalanceBlock);
  const int64_t most = std::max<int64_t>(1, kBalanceBlocks / present);
  p.block_tokens = std::max(kMinSteps * step, ceil_div(ceil_div(tokens, most), step) * step);
  p.block_tokens = std::min<int64_t>(p.block_tokens, dlc::kBlockTokens);
  p.blocks = std::max<int64_t>(1, ceil_div(tokens, p.block_tokens));
  p.count_blocks = p.blocks;
  p.count_tokens = p.block_tokens;
  if (gradient) {
    const int64_t want = tokens * top <= kSelfCount ? 1 : std::min(kMaxCountBlocks, ceil_div(tokens * top, kCountChoices));
    p.count_tokens = std::min(std::max<int64_t>(1, ceil_div(tokens, want)), dlc::kCountTokens);
    p.count_blocks = std::max<int64_t>(1, ceil_div(tokens, p.count_tokens));
  }
  return p;
}

// As many blocks as any call of at most so many tokens has, with any number of choices, with and without a gradient.
// A block's tokens are whole steps, so that fewer tokens can make more blocks: of two learners with 1024 experts, 4211
// tokens make 351 blocks of 12, 3927 make 491 of 8.  But a block has kMinSteps steps or more, and a learner no more blocks
// than its share of kBalanceBlocks unless kBlockTokens cuts them short, and likewise those that count.  These bounds do not
// fall as tokens grow, nor as experts do (a step is shorter then).
BalancePartition most_blocks(int64_t tokens, int32_t experts, int32_t type, int32_t present) {
  const int64_t step = dlc::balance_tokens(type, experts, dlc::kBalanceBlock);
  const int64_t share = std::max<int64_t>(1, kBalanceBlocks / present);
  BalancePartition p{};
  p.blocks = std::max({int64_t(1), std::min(share, ceil_div(tokens, kMinSteps * step)), ceil_div(tokens, dlc::kBlockTokens)});
  const int64_t counting = std::min(kMaxCountBlocks, ceil_div(tokens * DLC_MAX_CHOICES, kCountChoices));
  p.count_blocks = std::max({p.blocks, counting, ceil_div(tokens, dlc::kCountTokens)});
  return p;
}

size_t probs_bytes(const BalancePartition& p, int32_t experts, int32_t present) {
  return round256((size_t)present * p.blocks * experts * sizeof(double));
}

size_t counts_bytes(const BalancePartition& p, int32_t experts, int32_t present) {
  return round256((size_t)present * p.count_blocks * (experts + 2) * sizeof(uint32_t));
}

// the blocks' parts of the loss (over the logits, or of the final sums), and a ticket
int64_t loss_parts(const BalancePartition& p) { return std::max<int64_t>(p.blocks, dlc::kFinalMost); }

size_t loss_bytes(const BalancePartition& p, int32_t present) {
  return round256((size_t)present * (loss_parts(p) * sizeof(double) + sizeof(uint32_t)));
}

int32_t check_sizes(int32_t n_learners, int64_t n_tokens, int32_t n_experts) {
  if (n_learners < 1 || n_learners > DLC_MAX_LEARNERS)
    return fail(DLC_ERR_INVALID_ARGUMENT, "n_learners must be in [1, 64]");
  if (n_tokens < 0 || n_tokens > DLC_MAX_TOKENS)
    return fail(DLC_ERR_INVALID_ARGUMENT, "n_tokens must be in [0, 2^24]");
  if (n_experts < 1 || n_experts > DLC_MAX_EXPERTS)
    return fail(DLC_ERR_INVALID_ARGUMENT, "n_experts must be in [1, 1024]");
  return DLC_OK;
}

bool aligned_to(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % (uint64_t)bytes == 0; }

// A [learners][tokens][width] array of `size` bytes an element, from the first element to the
// last of learners first .. last.
struct Strided {
  const void* p;
  int64_t learner, token, width, size;
  // strides that no sum below can overflow with
  bool sound(int64_t learners, int64_t tokens) const {
    return learner >= 0 && learner <= kMaxReach / std::max<int64_t>(1, learners) && token >= 0 &&
           token <= kMaxReach / std::max<int64_t>(1, tokens);
  }
  bool rows_apart(int64_t learners, int64_t tokens) const {
    const auto nested = [&](int64_t inner, int64_t n_inner, int64_t outer, int64_t n_outer) {
      return (n_inner < 2 || inner >= width) && (n_outer < 2 || outer >= (n_inner - 1) * inner + width);
    };
    return nested(token, tokens, learner, learners) || nested(learner, learners, token, tokens);
  }
  dlc::Stretch stretch(int64_t first, int64_t last, int64_t tokens, bool written) const {
    const char* at = reinterpret_cast<const char*>(reinterpret_cast<uintptr_t>(p) + (uint64_t)(first * learner * size));
    const int64_t n = tokens == 0 ? 0 : (last - first) * learner + (tokens - 1) * token + width;
    return {at, p ? (uint64_t)(n * size) : 0, written};
  }
};

}  // namespace

extern "C" {

int32_t dlc_expert_balance_workspace_bytes(int32_t n_learners, int64_t n_tokens, int32_t n_experts, size_t* bytes) {
  return no_throw([&]() -> int32_t {
    if (!bytes) return fail(DLC_ERR_INVALID_ARGUMENT, "bytes is NULL");
    const int32_t rc = check_sizes(n_learners, n_tokens, n_experts);
    if (rc != DLC_OK) return rc;
    size_t most = 0;
    for (int32_t present = 1; present <= n_learners; ++present) {
      for (const int32_t type : {DLC_FLOAT32, DLC_BFLOAT16}) {
        const BalancePartition p = most_blocks(n_tokens, n_experts, type, present);
        most = std::max(most, probs_bytes(p, n_experts, present) + counts_bytes(p, n_experts, present) + loss_bytes(p, present));
      }
    }
    *bytes = most;
    return ok();
  });
}

int32_t dlc_expert_balance(const void* logits, int32_t logits_type, int64_t logits_learner_stride,
                           int64_t logits_token_stride, const void* choices, int32_t choices_type,
                           int64_t choices_learner_stride, int64_t choices_token_stride, const uint8_t* mask,
                           int64_t mask_learner_stride, int32_t n_learners, const uint8_t* present, int64_t n_tokens,
                           int32_t n_experts, int32_t n_choices, double coef, float* loss, int64_t* counts,
                           int64_t counts_stride, float* mean_probs, int64_t* totals, int64_t totals_stride,
                           void* grad_logits, int64_t grad_learner_stride, int64_t grad_token_stride,
                           const double* grad_scale, uint32_t flags, void* workspace, size_t workspace_bytes,
                           void* hip_stream) {
  return no_throw([&]() -> int32_t {
    int32_t rc = check_sizes(n_learners, n_tokens, n_experts);
    if (rc != DLC_OK) return rc;
    if (n_choices < 1 || n_choices > std::min(n_experts, DLC_MAX_CHOICES))
      return fail(DLC_ERR_INVALID_ARGUMENT, "n_choices must be in [1, min(n_experts, 64)]");
    if (logits_type != DLC_FLOAT32 && logits_type != DLC_BFLOAT16 && logits_type != DLC_FLOAT16)
      return fail(DLC_ERR_INVALID_ARGUMENT, "logits_type is not one of the call's types");
    if (choices_type != DLC_INT32 && choices_type != DLC_INT64)
      return fail(DLC_ERR_INVALID_ARGUMENT, "choices_type is not one of the call's types");
    if ((flags & ~DLC_ACCUMULATE) != 0) return fail(DLC_ERR_INVALID_ARGUMENT, "unknown flag");
    if (!std::isfinite(coef)) return fail(DLC_ERR_INVALID_ARGUMENT, "coef must be finite");
    if (!loss || !counts || (n_tokens > 0 && (!logits || !choices)))
      return fail(DLC_ERR_INVALID_ARGUMENT, "logits, choices, loss and counts must not be NULL");
    dlc::BalanceArgs a;
    std::memset(&a, 0, sizeof(a));
    int32_t first = -1, last = 0;
    for (int32_t i = 0; i < n_learners; ++i) {
      if (present != nullptr && present[i] == 0) continue;
      a.learner.word[a.n_present >> 2] |= (uint32_t)i << (8 * (a.n_present & 3));
      ++a.n_present;
      if (first < 0) first = i;
      last = i;
    }
    if (a.n_present == 0) return fail(DLC_ERR_NO_QUORUM, "no learner is present");
    const int64_t size = logits_type == DLC_FLOAT32 ? 4 : 2, id_size = choices_type == DLC_INT32 ? 4 : 8;
    const Strided x{logits, logits_learner_stride, logits_token_stride, n_experts, size};
    const Strided c{choices, choices_learner_stride, choices_token_stride, n_choices, id_size};
    const Strided g{grad_logits, grad_learner_stride, grad_token_stride, n_experts, size};
    const Strided k{mask, mask_learner_stride, 1, 1, 1};
    if (!x.sound(n_learners, n_tokens) || !c.sound(n_learners, n_tokens) || (mask && !k.sound(n_learners, n_tokens)) ||
        (grad_logits && !g.sound(n_learners, n_tokens)))
      return fail(DLC_ERR_INVALID_ARGUMENT, "strides must be >= 0 and stay within 2^48 elements");
    if (!aligned_to(logits, size) || !aligned_to(choices, id_size) || !aligned_to(grad_logits, size) ||
        !aligned_to(loss, 4) || !aligned_to(mean_probs, 4) || !aligned8(counts) || !aligned8(totals) ||
        !aligned8(grad_scale))
      return fail(DLC_ERR_ALIGNMENT, "device pointers must be aligned to their elements");
    if (grad_logits && !g.rows_apart(n_learners, n_tokens))
      return fail(DLC_ERR_INVALID_ARGUMENT, "rows of grad_logits overlap");
    const Strided n{counts, counts_stride, 0, n_experts, 8}, t{totals, totals_stride, 0, n_experts, 8};
    const bool several = n_learners > 1;
    if (!n.sound(n_learners, 1) || (totals && !t.sound(n_learners, 1)) || (several && counts_stride < n_experts) ||
        (several && totals && totals_stride < n_experts))
      return fail(DLC_ERR_INVALID_ARGUMENT, "rows of counts or totals overlap");
    const bool gradient = grad_logits != nullptr && n_tokens > 0;
    const bool one = one_block(n_tokens, n_experts, n_choices, logits_type);
    const BalancePartition p =
        balance_partition(n_tokens, n_experts, n_choices, logits_type, a.n_present, gradient);
    const size_t probs = probs_bytes(p, n_experts, a.n_present);
    const size_t losses = probs + counts_bytes(p, n_experts, a.n_present);
    const size_t need = one ? 0 : losses + loss_bytes(p, a.n_present);
    if (workspace == nullptr || workspace_bytes < need)
      return fail(DLC_ERR_WORKSPACE, "workspace too small: need " + std::to_string(need) + " bytes");
    if (!aligned256(workspace)) return fail(DLC_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
    const uint64_t per = (uint64_t)(last - first + 1);
    const dlc::Stretch s[] = {x.stretch(first, last, n_tokens, false),
                              c.stretch(first, last, n_tokens, false),
                              k.stretch(first, last, n_tokens, false),
                              {grad_scale ? grad_scale + first : nullptr, per * 8, false},
                              {loss + first, per * 4, true},
                              n.stretch(first, last, 1, true),
                              {mean_probs ? mean_probs + (int64_t)first * n_experts : nullptr, per * n_experts * 4, true},
                              t.stretch(first, last, 1, true),
                              g.stretch(first, last, n_tokens, true),
                              {workspace, need, true}};
    rc = dlc::check_stretches(s, (int32_t)(sizeof(s) / sizeof(s[0])));
    if (rc != DLC_OK) return rc;
    a.logits = logits;
    a.x_learner = logits_learner_stride;
    a.x_token = logits_token_stride;
    a.choices = choices;
    a.c_learner = choices_learner_stride;
    a.c_token = choices_token_stride;
    a.wide_choices = choices_type == DLC_INT64;
    a.mask = mask;
    a.mask_learner = mask_learner_stride;
    a.grad = gradient ? grad_logits : nullptr;
    a.g_learner = grad_learner_stride;
    a.g_token = grad_token_stride;
    a.grad_scale = grad_scale;
    a.accumulate = (flags & DLC_ACCUMULATE) != 0;
    a.loss = loss;
    a.counts = counts;
    a.counts_stride = counts_stride;
    a.means = mean_probs;
    a.totals = totals;
    a.totals_stride = totals_stride;
    a.part_probs = static_cast<double*>(workspace);
    a.part_counts = reinterpret_cast<uint32_t*>(static_cast<char*>(workspace) + probs);
    a.part_loss = reinterpret_cast<double*>(static_cast<char*>(workspace) + losses);
    a.tickets = reinterpret_cast<uint32_t*>(a.part_loss + (size_t)a.n_present * loss_parts(p));
    a.coef = coef;
    a.tokens = (int32_t)n_tokens;
    a.experts = n_experts;
    a.top = n_choices;
    a.top_inverse = n_choices == 1 ? 0u : (uint32_t)(((uint64_t(1) << 32) + n_choices - 1) / n_choices);
    a.count_blocks = (int32_t)p.count_blocks;
    a.count_tokens = (int32_t)p.count_tokens;
    a.blocks = (int32_t)p.blocks;
    a.loss_parts = (int32_t)loss_parts(p);
    a.final_experts = dlc::kFinalExperts;
    if (p.blocks * n_experts <= kOneFinal) {
      while (a.final_experts < std::min(n_experts, dlc::kFinalBlock)) a.final_experts *= 2;
    }
    a.block_tokens = (int32_t)p.block_tokens;
    const hipStream_t st = static_cast<hipStream_t>(hip_stream);
    hipError_t e;
    if (one) {
      e = dlc::launch_balance(a, logits_type, true, st);
    } else {
      e = gradient && p.count_blocks > 1 ? dlc::launch_balance_count(a, st) : hipSuccess;
      if (e == hipSuccess) e = dlc::launch_balance(a, logits_type, false, st);
      if (e == hipSuccess) e = dlc::launch_balance_final(a, st);
    }
    return e != hipSuccess ? hip_fail(e, "balance kernel launch") : ok();
  });
}

int32_t dlc_expert_weights(const int64_t* counts, int64_t counts_stride, int32_t n_learners, int32_t n_experts,
                           const double* weights, const double* token_weight, const int32_t* expert_of,
                           int32_t n_tensors, double* tensor_weights, void* hip_stream) {
  return no_throw([&]() -> int32_t {
    if (n_learners < 1 || n_learners > DLC_MAX_LEARNERS)
      return fail(DLC_ERR_INVALID_ARGUMENT, "n_learners must be in [1, 64]");
    if (!counts || !weights || !expert_of || !tensor_weights)
      return fail(DLC_ERR_INVALID_ARGUMENT, "counts, weights, expert_of and tensor_weights must not be NULL");
    if (n_experts < 1 || n_experts > INT16_MAX)
      return fail(DLC_ERR_INVALID_ARGUMENT, "n_experts must be in [1, 32767]");
    if (n_tensors < 1) return fail(DLC_ERR_INVALID_ARGUMENT, "n_tensors must be >= 1");
    if (!aligned8(counts) || !aligned8(tensor_weights))
      return fail(DLC_ERR_ALIGNMENT, "counts and tensor_weights must be 8-byte aligned");
    if (counts_stride > kMaxReach / n_learners || (n_learners > 1 && counts_stride < n_experts) || counts_stride < 0)
      return fail(DLC_ERR_INVALID_ARGUMENT, "rows of counts overlap");
    dlc::WeightArgs a;
    std::memset(&a, 0, sizeof(a));
    double total = 0.0;
    for (int32_t i = 0; i < n_learners; ++i) {
      if (!(weights[i] >= 0.0) || !std::isfinite(weights[i]))
        return fail(DLC_ERR_INVALID_ARGUMENT, "weights must be finite and >= 0");
      total += weights[i];
      const double w = token_weight ? token_weight[i] : 1.0;
      if (!(w >= 0.0 && w <= 0x1p900))  // the sum of 64 times 2^63 of them is finite
        return fail(DLC_ERR_INVALID_ARGUMENT, "token_weight must be in [0, 2^900]");
      a.token_weight[i] = weights[i] > 0.0 ? w : 0.0;
    }
    if (!(total > 0.0)) return fail(DLC_ERR_NO_QUORUM, "all learner weights are zero (no quorum)");
    if (!std::isfinite(total)) return fail(DLC_ERR_INVALID_ARGUMENT, "the sum of the weights is not finite");
    for (int32_t i = 0; i < n_learners; ++i) a.w_hat[i] = weights[i] / total;
    for (int32_t t = 0; t < n_tensors; ++t) {
      if (expert_of[t] < -1 || expert_of[t] >= n_experts)
        return fail(DLC_ERR_INVALID_ARGUMENT, "tensor " + std::to_string(t) + ": no such expert");
    }
    const dlc::Stretch s[] = {{counts, (uint64_t)((n_learners - 1) * counts_stride + n_experts) * 8, false},
                              {tensor_weights, (uint64_t)n_tensors * n_learners * 8, true}};
    const int32_t rc = dlc::check_stretches(s, 2);
    if (rc != DLC_OK) return rc;
    a.counts = counts;
    a.counts_stride = counts_stride;
    a.out = tensor_weights;
    a.n_learners = n_learners;
    for (int32_t t0 = 0; t0 < n_tensors; t0 += dlc::kWeightTensors) {
      a.first = t0;
      a.n_tensors = std::min(dlc::kWeightTensors, n_tensors - t0);
      for (int32_t t = 0; t < a.n_tensors; ++t) a.expert[t] = (int16_t)expert_of[t0 + t];
      const hipError_t e = dlc::launch_expert_weights(a, static_cast<hipStream_t>(hip_stream));
      if (e != hipSuccess) return hip_fail(e, "expert weights kernel launch");
    }
    return ok();
  });
}

}  // extern "C"
