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

// A launch, a load and LDS additions: 5 us whether 8 learners have 24,000 or 262,000 choices each.
__global__ __launch_bounds__(kCountBlock) void k_balance_count(const BalanceArgs a) {
  __shared__ uint32_t hist[kCountWords + 2];
  const int t0 = blockIdx.x * a.count_tokens, t1 = min(a.tokens, t0 + a.count_tokens);
  count<kCountBlock>(a, a.learner[blockIdx.y], t0, t1, hist);
  write_counts<kCountBlock>(a, a.part_counts + ((size_t)blockIdx.y * a.count_blocks + blockIdx.x) * (a.experts + 2), hist);
}

// A block per a.final_experts experts of a learner (a power of two): thread (s, c) sums every slices-th
// block's expert c, then the slices in order.  One block for all experts is limited by a single
// CU's outstanding loads (131 KB of sums: 8 us against 5), so long sums are split by
// experts.  The loss is a sum over all of them.  With a gradient the blocks over the logits knew the
// counts and left their tokens' parts of it, which the first block adds; without one the block
// that comes last, which a ticket tells it, adds the blocks' parts, in their order.
__global__ __launch_bounds__(kFinalBlock) void k_balance_final(const BalanceArgs a) {
  __shared__ double sums[kFinalBlock];
  __shared__ uint32_t counts[kFinalBlock];
  __shared__ uint32_t kept_part[kFinalBlock / 64];
  __shared__ double red[kFinalBlock / 64];
  const int e = a.experts, width = a.final_experts, slices = kFinalBlock / width;
  const int s = threadIdx.x / width, c = threadIdx.x % width;
  const int k = blockIdx.x * width + c, i = a.learner[blockIdx.y];
  const bool mine = k < e;
  const uint32_t* part = a.part_counts + (size_t)blockIdx.y * a.count_blocks * (e + 2);
  const double* prob = a.part_probs + (size_t)blockIdx.y * a.blocks * e + (mine ? k : 0);
  const int64_t total = a.totals != nullptr && mine && s == 0 ? a.totals[(int64_t)i * a.totals_stride + k] : 0;
  uint32_t n = 0, count = 0;
  for (int b = threadIdx.x; b < a.count_blocks; b += kFinalBlock) n += part[(size_t)b * (e + 2) + e];
#pragma unroll 4
  for (int b = s; b < a.count_blocks; b += slices) count += part[(size_t)b * (e + 2) + (mine ? k : 0)];
  const bool parts = a.grad != nullptr;
  double l = 0.0;
  if (parts && blockIdx.x == 0) {
    for (int b = threadIdx.x; b < a.blocks; b += kFinalBlock) l += a.part_loss[(size_t)blockIdx.y * a.loss_parts + b];
  }
  double v = 0.0;
#pragma unroll 8
  for (int b = s; b < a.blocks; b += slices) v += prob[(size_t)b * e];
  sums[threadIdx.x] = v;
  counts[threadIdx.x] = count;
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) n += __shfl_xor(n, m, 64);
  if ((threadIdx.x & 63) == 0) kept_part[threadIdx.x >> 6] = n;
  __syncthreads();
  uint32_t kept = 0;
#pragma unroll
  for (int w = 0; w < kFinalBlock / 64; ++w) kept += kept_part[w];
  if (s == 0 && mine) {
#pragma unroll 4
    for (int q = 1; q < slices; ++q) {
      v += sums[q * width + c];
      count += counts[q * width + c];
    }
    const double part = finish_expert(a, i, k, count, v, kept, total);
    if (!parts) l = part;
  }
  if (parts && blockIdx.x != 0) return;
  l = wave_sum(l);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = l;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 1; w < kFinalBlock / 64; ++w) l += red[w];
  if (parts) l = kept == 0 ? 0.0 : l / (double)kept;
  if (parts || gridDim.x == 1) {
    write_loss(a, i, kept, l);
    return;
  }
  double* losses = a.part_loss + (size_t)blockIdx.y * a.loss_parts;
  __hip_atomic_store(&losses[blockIdx.x], l, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const uint32_t drawn = __hip_atomic_fetch_add(&a.tickets[blockIdx.y], 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
  if (drawn != gridDim.x - 1) return;
  l = 0.0;
  for (uint32_t b = 0; b < gridDim.x; ++b) l += __hip_atomic_load(&losses[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  write_loss(a, i, kept, l);
}

// ---------------------------------------------------------------------------
// k_expert_weights: a thread per tensor, learners in index order (2 to 5 us: two dependent loads a learner).
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
  hipLaunchKernelGGL(k_balance_final, dim3((a.experts + a.final_experts - 1) / a.final_experts, a.n_present),
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
