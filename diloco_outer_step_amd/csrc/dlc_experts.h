// Launch descriptors of the mixture-of-experts calls (the router's balance loss, merge
// weights from expert counts), shared by the host orchestration and the gfx950 kernels.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "dlc_inner.h"

namespace dlc {

constexpr int kMaxExperts = 1024;
constexpr int kMaxChoices = 64;
// Over the logits: blocks of 256 threads with two steps' loads under way behind the one that is worked on.
// 32768 x 256 x 8 bf16, us a call: 512 threads 82, 256 80 (an early form); one step ahead 73.4, two 72.1 (a
// later one).
constexpr int kBalanceBlock = 256;
constexpr int kBalanceAhead = 2;
constexpr int kBalanceOne = 512;         // threads of the block that does a learner's whole call
constexpr int kCountBlock = 512;
constexpr int kFinalBlock = 512;
constexpr int kFinalExperts = 32;        // experts of a block of long final sums
constexpr int kFinalMost = kMaxExperts / kFinalExperts;
constexpr int kFoldTokens = 16;          // tokens a lane sums in fp32 before it goes on in fp64
constexpr int kCountWords = 1024;        // LDS words of a block's histogram copies
constexpr int kBlockTokens = 16384;      // most tokens of a block over the logits
constexpr int64_t kCountTokens = 1 << 18;  // most tokens of a counting block, see divide()

struct BalanceArgs {
  const void* logits;         // [n_learners][tokens][experts], strides in elements
  int64_t x_learner, x_token;
  const void* choices;        // [n_learners][tokens][top]
  int64_t c_learner, c_token;
  const uint8_t* mask;        // [n_learners][tokens], or NULL
  int64_t mask_learner;
  void* grad;                 // [n_learners][tokens][experts], or NULL
  int64_t g_learner, g_token;
  const double* grad_scale;   // [n_learners], or NULL
  float* loss;                // [n_learners]
  int64_t* counts;            // [n_learners][experts]
  int64_t counts_stride;
  float* means;               // [n_learners][experts], or NULL
  int64_t* totals;            // [n_learners][experts], or NULL
  int64_t totals_stride;
  uint32_t* part_counts;      // [present][count_blocks][experts + 2]: counts, kept tokens, choices in all
  double* part_probs;         // [present][blocks][experts] sums of probabilities
  double* part_loss;          // [present][loss_parts]
  uint32_t* tickets;          // [present]
  double coef;
  int32_t tokens, experts, top;
  uint32_t top_inverse;       // ceil(2^32 / top), 0 for top = 1
  int32_t count_blocks, count_tokens;  // blocks per learner that count, tokens of each
  int32_t blocks, block_tokens;        // blocks per learner over the logits, tokens of each
  int32_t final_experts;               // of a block of the final sums
  int32_t loss_parts;
  int32_t accumulate, wide_choices;
  int32_t n_present;
  LearnerList learner;
};

constexpr int kWeightTensors = 640;      // tensors per launch

struct WeightArgs {
  const int64_t* counts;
  int64_t counts_stride;
  double* out;                // [n_tensors][n_learners]
  int32_t n_learners;
  int32_t n_tensors;          // of this launch
  int64_t first;              // its first tensor
  double w_hat[64];           // normalized weights, 0 = absent
  double token_weight[64];    // 0 for absent learners
  int16_t expert[kWeightTensors];
};

static_assert(sizeof(BalanceArgs) <= 4096 && sizeof(WeightArgs) <= 4096);

// Lanes per token: the fewest that hold a row in one load of v elements each, 64 at most.
inline int balance_lanes(int experts, int v) {
  int l = 1;
  while (l < 64 && l * v < experts) l *= 2;
  return l;
}

// Tokens of a step of the one block, which has 8 or 64 lanes a token (1 where a row is narrower than a load).
inline int balance_one_tokens(int32_t type, int experts) {
  const int v = type == kF32 ? 4 : 8;
  return kBalanceOne / (experts < v ? 1 : balance_lanes(experts, v) <= 8 ? 8 : 64);
}

// Kernel launchers (dlc_experts.hip).  Each returns hipSuccess or the launch error.
hipError_t launch_balance_count(const BalanceArgs& a, hipStream_t s);
// One block per learner for the whole call, or the pass over the logits: with a gradient after
// launch_balance_count; without one it counts its own tokens' choices.
hipError_t launch_balance(const BalanceArgs& a, int32_t type, bool one, hipStream_t s);
template <int32_t kType>
hipError_t launch_balance_of(const BalanceArgs& a, bool one, hipStream_t s);  // dlc_balance_*.hip
template <>
hipError_t launch_balance_of<kF32>(const BalanceArgs& a, bool one, hipStream_t s);
template <>
hipError_t launch_balance_of<kBF16>(const BalanceArgs& a, bool one, hipStream_t s);
template <>
hipError_t launch_balance_of<kF16>(const BalanceArgs& a, bool one, hipStream_t s);
hipError_t launch_balance_final(const BalanceArgs& a, hipStream_t s);
// tokens that a block of `threads` threads takes at once
int32_t balance_tokens(int32_t type, int32_t experts, int32_t threads);
hipError_t launch_expert_weights(const WeightArgs& a, hipStream_t s);

}  // namespace dlc
