// gfx950 kernels of the mixture-of-experts calls.
//
//   k_balance_count  choices per expert, kept tokens of a block
//   k_balance_final  the blocks' sums in a fixed order -> counts, means, loss
//   k_expert_weights merge weights of every (tensor, learner) from the counts
//
// The kernels over the logits are in dlc_balance.h.
#include "dlc_balance.h"

namespace dlc {
namespace {

__global__ __launch_bounds__(kCountBlock) void k_balance_count(const BalanceArgs a) {
  __shared__ uint32_t hist[kCountWords + 1];
  const int t0 = blockIdx.x * a.count_tokens, t1 = min(a.tokens, t0 + a.count_tokens);
  count<kCountBlock>(a, a.learner[blockIdx.y], t0, t1, hist);
  uint32_t* out = a.part_counts + ((size_t)blockIdx.y * a.count_blocks + blockIdx.x) * (a.experts + 1);
  for (int k = threadIdx.x; k < a.experts; k += kCountBlock) out[k] = hist[k];
  if (threadIdx.x == 0) out[a.experts] = hist[kCountWords];
}

// A block per kFinalExperts experts of a learner: thread (s, k) sums every kFinalSlices-th
// block's expert k, then the slices in order.  One block would do, but it is a single CU's
// outstanding loads that limit it (131 KB of sums: 8 us).  The block that comes last,
// which a ticket tells it, adds the blocks' parts of the loss, in their order.
__global__ __launch_bounds__(kFinalBlock) void k_balance_final(const BalanceArgs a) {
  constexpr int kSlices = kFinalBlock / kFinalExperts;
  __shared__ double sums[kFinalBlock];
  __shared__ uint32_t counts[kFinalBlock];
  __shared__ uint32_t kept_part[kFinalBlock / 64];
  const int e = a.experts, s = threadIdx.x / kFinalExperts, c = threadIdx.x % kFinalExperts;
  const int k = blockIdx.x * kFinalExperts + c, i = a.learner[blockIdx.y];
  const bool mine = k < e;
  const uint32_t* part = a.part_counts + (size_t)blockIdx.y * a.count_blocks * (e + 1);
  const double* prob = a.part_probs + (size_t)blockIdx.y * a.blocks * e + (mine ? k : 0);
  const int64_t total = a.totals != nullptr && mine && s == 0 ? a.totals[(int64_t)i * a.totals_stride + k] : 0;
  uint32_t n = 0, count = 0;
  for (int b = threadIdx.x; b < a.count_blocks; b += kFinalBlock) n += part[(size_t)b * (e + 1) + e];
#pragma unroll 4
  for (int b = s; b < a.count_blocks; b += kSlices) count += part[(size_t)b * (e + 1) + (mine ? k : 0)];
  double v = 0.0;
#pragma unroll 8
  for (int b = s; b < a.blocks; b += kSlices) v += prob[(size_t)b * e];
  sums[threadIdx.x] = v;
  counts[threadIdx.x] = count;
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) n += __shfl_xor(n, m, 64);
  if ((threadIdx.x & 63) == 0) kept_part[threadIdx.x >> 6] = n;
  __syncthreads();
  if (threadIdx.x >= 64) return;
  uint32_t kept = 0;
#pragma unroll
  for (int w = 0; w < kFinalBlock / 64; ++w) kept += kept_part[w];
  double l = 0.0;
  if (s == 0 && mine) {
#pragma unroll
    for (int q = 1; q < kSlices; ++q) {
      v += sums[q * kFinalExperts + c];
      count += counts[q * kFinalExperts + c];
    }
    l = finish_expert(a, i, k, count, v, kept, total);
  }
  l = wave_sum(l);
  if (threadIdx.x != 0) return;
  if (gridDim.x == 1) {
    write_loss(a, i, kept, l);
    return;
  }
  double* losses = a.part_loss + (size_t)blockIdx.y * kFinalMost;
  __hip_atomic_store(&losses[blockIdx.x], l, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const uint32_t drawn = __hip_atomic_fetch_add(&a.tickets[blockIdx.y], 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
  if (drawn != gridDim.x - 1) return;
  l = 0.0;
  for (uint32_t b = 0; b < gridDim.x; ++b) l += __hip_atomic_load(&losses[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  write_loss(a, i, kept, l);
}

// ---------------------------------------------------------------------------
// k_expert_weights: a thread per tensor, learners in index order.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(64) void k_expert_weights(const WeightArgs a) {
  const int t = blockIdx.x * 64 + threadIdx.x;
  if (t >= a.n_tensors) return;
  const int e = a.expert[t];
  double* out = a.out + (a.first + t) * a.n_learners;
  const auto raw = [&](int i) {
    if (!(a.token_weight[i] > 0.0)) return 0.0;
    const int64_t c = a.counts[(int64_t)i * a.counts_stride + e];
    return c > 0 ? a.token_weight[i] * (double)c : 0.0;
  };
  double total = 0.0;
  if (e >= 0) {
    for (int i = 0; i < a.n_learners; ++i) total += raw(i);
  }
  for (int i = 0; i < a.n_learners; ++i) out[i] = total > 0.0 ? raw(i) / total : a.w_hat[i];
}


}  // namespace

hipError_t launch_balance(const BalanceArgs& a, int32_t type, bool one, hipStream_t s) {
  if (type == kF32) return launch_balance_of<kF32>(a, one, s);
  return type == kBF16 ? launch_balance_of<kBF16>(a, one, s) : launch_balance_of<kF16>(a, one, s);
}

hipError_t launch_balance_count(const BalanceArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(k_balance_count, dim3(a.count_blocks, a.n_present), dim3(kCountBlock), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_balance_final(const BalanceArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(k_balance_final, dim3((a.experts + kFinalExperts - 1) / kFinalExperts, a.n_present),
                     dim3(kFinalBlock), 0, s, a);
  return hipGetLastError();
}

int32_t balance_tokens(int32_t type, int32_t experts, int32_t threads) {
  return threads / balance_lanes(experts, type == kF32 ? 4 : 8);
}

hipError_t launch_expert_weights(const WeightArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(k_expert_weights, dim3((a.n_tensors + 63) / 64), dim3(64), 0, s, a);
  return hipGetLastError();
}

}  // namespace dlc
