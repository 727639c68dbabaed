// The balance loss's kernels over the logits, compiled once for each type of them
// (dlc_balance_*.hip).
//
//   k_balance      softmax of every token, its sum over the tokens, its gradient
//   k_balance_one  a learner's whole call in one block, for few tokens
//
// The gradient of the loss coef E sum_e f_e P_e, f the share of the choices and P the mean
// probabilities, is a softmax's: coef E / (n^2 top) p_e (c_e - sum_j p_j c_j).  It needs the
// whole counts but not P, so the choices (a fiftieth of the logits' bytes) are counted first
// and the logits are read once.  Taking c less its mean changes nothing, as sum p = 1, and
// keeps the bracket from cancelling when the experts are used evenly.
#pragma once

#include "dlc_experts.h"
#include "dlc_lanes.h"

#include <type_traits>

namespace dlc {
namespace {

__device__ __forceinline__ double wave_sum(double v) {
  return reduce<64>(v, [](double p, double q) { return p + q; });
}

// ---------------------------------------------------------------------------
// Counting
// ---------------------------------------------------------------------------
// f / top for f below kCountTokens top: the inverse is at most (top - 1) / 2^32 too large per
// unit of f, and f (top - 1) < 2^18 64^2 <= 2^32.
__device__ __forceinline__ uint32_t divide(uint32_t f, uint32_t inverse) {
  return inverse == 0 ? f : __umulhi(f, inverse);
}

// A learner's choices of tokens [t0, t1) -> hist[0 .. experts), kept tokens -> hist[kCountWords],
// choices that count for some expert -> hist[kCountWords + 1].  The words of hist hold copies of the
// histogram, so that lanes with the same choice (routers have favourites, and few experts) add to
// different words: 16 at most, which are summed at the end.
template <int kThreads, typename I>
__device__ __forceinline__ void count_choices(const BalanceArgs& a, int i, int t0, int t1, uint32_t* hist) {
  const uint32_t e = (uint32_t)a.experts;
  uint32_t copies = 1;
  while (copies < 16 && copies * e < 512) copies *= 2;  // below 1024 words in all, or E
  for (uint32_t k = threadIdx.x; k < copies * e; k += kThreads) hist[k] = 0;
  if (threadIdx.x < 2) hist[kCountWords + threadIdx.x] = 0;
  uint32_t* mine = hist + (threadIdx.x & (copies - 1)) * e;
  const I* ids = (const I*)a.choices + (int64_t)i * a.c_learner + (int64_t)t0 * a.c_token;
  const uint8_t* mask = a.mask != nullptr ? a.mask + (int64_t)i * a.mask_learner + t0 : nullptr;
  const uint32_t top = (uint32_t)a.top, n = (uint32_t)(t1 - t0) * top;
  constexpr int U = 8;
  I id[U];
  uint32_t live = 0, first = 0;  // bit u: choice u counts, is its token's first (so the token is kept)
  const auto request = [&](uint32_t f0) {
    live = first = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t f = f0 + u * kThreads;  // below 2^24 + 2^13
      const uint32_t at = f < n ? f : 0;
      const uint32_t t = divide(at, a.top_inverse), j = at - t * top;
      id[u] = ids[(int64_t)t * a.c_token + j];
      bool keep = f < n;
      if (mask != nullptr) keep = keep && mask[t] != 0;
      live |= keep ? 1u << u : 0;
      first |= keep && j == 0 ? 1u << u : 0;
    }
  };
  uint32_t kept = 0, valid = 0;
  const auto add = [&]() {
    kept += __popc(first);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if ((live >> u & 1u) != 0 && (std::make_unsigned_t<I>)id[u] < e) {
        atomicAdd(&mine[(uint32_t)id[u]], 1u);
        ++valid;
      }
    }
  };
  if (threadIdx.x < n) request(threadIdx.x);
  __syncthreads();
  for (uint32_t f0 = threadIdx.x; f0 < n; f0 += U * kThreads) {
    add();
    if (f0 + U * kThreads < n) request(f0 + U * kThreads);
  }
  // a lane per wave adds (of 64 lanes at one address the compiler makes a loop)
  const auto sum = [](uint32_t p, uint32_t q) { return p + q; };
  kept = reduce<64>(kept, sum);
  valid = reduce<64>(valid, sum);
  if (threadIdx.x % 64 < 2) atomicAdd(&hist[kCountWords + threadIdx.x % 64], threadIdx.x % 64 == 0 ? kept : valid);
  __syncthreads();
  // a thread sums the copies of its experts; only it writes hist[its experts]
  for (uint32_t k = threadIdx.x; k < e && copies > 1; k += kThreads) {
    uint32_t s = 0;
#pragma unroll 4
    for (uint32_t c = 0; c < copies; ++c) s += hist[c * e + k];
    hist[k] = s;
  }
  __syncthreads();
}

template <int kThreads>
__device__ __forceinline__ void count(const BalanceArgs& a, int i, int t0, int t1, uint32_t* hist) {
  if (a.wide_choices != 0) count_choices<kThreads, int64_t>(a, i, t0, t1, hist);
  else count_choices<kThreads, int32_t>(a, i, t0, t1, hist);
}

// ---------------------------------------------------------------------------
// The pass over the logits
// ---------------------------------------------------------------------------
enum BalanceMode { kLossOnly = 0, kGradient = 1, kAccumulate = 2 };

// A lane holds V = 16 bytes of a token's logits J times, L lanes a token, so a wave works on
// 64 / L tokens at once.  Logits lie at any address that their type allows; 16-byte loads
// need no more on gfx950.  Every lane loads and stores whole: a chunk that would pass the row's
// end is moved back to end with it, and [lo, hi) are the elements that no lane before it
// holds.  The others are computed as well and stored with the same bits, but not summed.
// Rows narrower than V are the exception (NARROW: L = J = 1, element by element).  STREAM: not to be
// kept in the caches, which is faster by 5% of the call where the gradient is written too (32768 x
// 256 x 8 bf16: 68.3 against 72.0 us) and slower by 4% where it is not.
template <typename T, int L, int J, bool NARROW, bool STREAM>
struct Chunks {
  static constexpr int V = 16 / (int)sizeof(T);
  typedef T vec __attribute__((ext_vector_type(V), aligned(sizeof(T))));
  int start[J], lo[J], hi, experts;
  __device__ __forceinline__ Chunks(int lane, int e) : hi(NARROW ? e : V), experts(e) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int at = (j * L + lane) * V;
      start[j] = NARROW ? 0 : min(at, e - V);
      lo[j] = NARROW ? 0 : min(at - start[j], V);
    }
  }
  __device__ __forceinline__ void load(const T* row, vec (&q)[J]) const {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      if constexpr (NARROW) {
#pragma unroll
        for (int c = 0; c < V; ++c) q[j][c] = row[min(c, experts - 1)];
      } else {
        q[j] = STREAM ? __builtin_nontemporal_load((const vec*)(row + start[j])) : *(const vec*)(row + start[j]);
      }
    }
  }
  __device__ __forceinline__ void store(T* row, const vec (&q)[J]) const {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      if constexpr (NARROW) {
#pragma unroll
        for (int c = 0; c < V; ++c) {
          if (c < experts) row[c] = q[j][c];
        }
      } else {
        if constexpr (STREAM) __builtin_nontemporal_store(q[j], (vec*)(row + start[j]));
        else *(vec*)(row + start[j]) = q[j];
      }
    }
  }
};

// LDS of a block over the logits.
template <typename T, int kThreads>
struct Work {
  union {
    float share[kMaxExperts];                          // (counts less their mean) times the gradient's factor
    double sums[16 / sizeof(T) * (kThreads + 8)];      // the lanes' sums of probabilities, once share has been read
  };
  double stage[kThreads];
  uint32_t bits[kBlockTokens / 32];                    // the block's kept tokens, if there is a mask
  uint32_t hist[kCountWords + 2];
  double red[kThreads / 64];
};

// Learner i's tokens [t0, t1): the gradient, and emit(k, sum of the probabilities of expert k), by one
// thread for each expert.  before() runs once the first logits are on their way; work.share is read
// after it.
//
// A step is a token for every group of L lanes.  The steps of whole blocks of tokens issue the same
// memory operations each, none of them conditional, so that a wait for one step's logits leaves
// the loads of the next kBalanceAhead steps and the stores in flight.  The tokens that are
// left over come first, while those loads are under way.
template <typename T, int L, int J, bool NARROW, int MODE, int kThreads, typename F, typename G>
__device__ __forceinline__ void pass(const BalanceArgs& a, int i, int t0, int t1, F&& before, G&& emit,
                                     Work<T, kThreads>& work) {
  using C = Chunks<T, L, J, NARROW, MODE != kLossOnly>;
  using vec = typename C::vec;
  constexpr int V = C::V;
  constexpr int kTokens = kThreads / L;
  constexpr int kAhead = J == 1 ? kBalanceAhead : 1;
  constexpr float kLog2e = 1.44269504f;
  const int slot = threadIdx.x / L;
  const int experts = a.experts;
  const C ch(threadIdx.x % L, experts);
  const bool cut = experts != L * J * V;  // some lane holds elements that are not its own
  const int whole = (t1 - t0) / kTokens, left = (t1 - t0) % kTokens;
  const T* x = (const T*)a.logits + (int64_t)i * a.x_learner;
  T* grad = MODE == kLossOnly ? nullptr : (T*)a.grad + (int64_t)i * a.g_learner;
  const bool masked = a.mask != nullptr;

  vec last[J], next[kAhead + 1][J];
  const int end = whole * kTokens + slot;
  if (left > 0) ch.load(x + (int64_t)min(t0 + end, t1 - 1) * a.x_token, last);
  const T* ahead = x + (int64_t)(t0 + slot) * a.x_token;
  const int64_t step = (int64_t)kTokens * a.x_token;
  if (whole > 0) {
#pragma unroll
    for (int k = 0; k <= kAhead; ++k) {
      ch.load(ahead, next[k]);
      ahead += k + 1 < whole ? step : 0;
    }
  }
  if (masked) {
    const uint8_t* mask = a.mask + (int64_t)i * a.mask_learner + t0;
    for (int t = threadIdx.x; t - (int)threadIdx.x < t1 - t0; t += kThreads) {  // whole waves
      const uint64_t word = __builtin_amdgcn_ballot_w64(t < t1 - t0 && mask[min(t, t1 - t0 - 1)] != 0);
      if (threadIdx.x % 64 < 2) work.bits[t / 64 * 2 + threadIdx.x % 64] = (uint32_t)(word >> (32 * (threadIdx.x % 64)));
    }
    __syncthreads();
  }
  const auto kept = [&](int t) { return !masked || (work.bits[t / 32] >> (t % 32) & 1u) != 0; };
  before();

  float own[J][V];
  if constexpr (MODE != kLossOnly) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
#pragma unroll
      for (int c = 0; c < V; ++c) own[j][c] = work.share[NARROW ? min(c, experts - 1) : ch.start[j] + c];
    }
  }
  float part[J][V] = {};
  double total[J][V] = {};
  const auto fold = [&]() {
#pragma unroll
    for (int j = 0; j < J; ++j) {
#pragma unroll
      for (int c = 0; c < V; ++c) {
        total[j][c] += (double)part[j][c];
        part[j][c] = 0.0f;
      }
    }
  };
  // One token of each group of lanes; out: its gradient (with kAccumulate, on top of the old one).
  const auto token = [&](const vec (&raw)[J], bool live, const T* row, vec (&out)[J]) {
    vec old[J];
    if constexpr (MODE == kAccumulate) ch.load(row, old);
    float v[J][V];
#pragma unroll
    for (int j = 0; j < J; ++j) {
#pragma unroll
      for (int c = 0; c < V; ++c) v[j][c] = (float)raw[j][c];
    }
    if (__builtin_amdgcn_ballot_w64(live) != ~0ull) {  // what is left out may be no number
#pragma unroll
      for (int j = 0; j < J; ++j) {
#pragma unroll
        for (int c = 0; c < V; ++c) v[j][c] = live ? v[j][c] : -__builtin_inff();
      }
    }
    float m = v[0][0];
#pragma unroll
    for (int j = 0; j < J; ++j) {
#pragma unroll
      for (int c = 0; c < V; ++c) m = fmaxf(m, v[j][c]);
    }
    m = reduce<L>(m, [](float p, float q) { return fmaxf(p, q); });
    if (m == -__builtin_inff()) m = 0.0f;  // nothing is possible: every probability is 0
    // exp(x - m) as 2^(x log2 e - m log2 e): the product m log2 e is rounded the same for the whole row, and
    // below 2^20 by too little to matter to the exponential's range
    if (__builtin_amdgcn_ballot_w64(fabsf(m) > 0x1p20f) == 0) {
      const float shift = -(m * kLog2e);
#pragma unroll
      for (int j = 0; j < J; ++j) {
#pragma unroll
        for (int c = 0; c < V; ++c) v[j][c] = __builtin_amdgcn_exp2f(__fmaf_rn(v[j][c], kLog2e, shift));
      }
    } else {
#pragma unroll
      for (int j = 0; j < J; ++j) {
#pragma unroll
        for (int c = 0; c < V; ++c) v[j][c] = __builtin_amdgcn_exp2f((v[j][c] - m) * kLog2e);
      }
    }
    float s = 0.0f, d = 0.0f;
    if (cut) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
#pragma unroll
        for (int c = 0; c < V; ++c) {
          const float e = c >= ch.lo[j] && c < ch.hi ? v[j][c] : 0.0f;
          s += e;
          if constexpr (MODE != kLossOnly) d = __fmaf_rn(e, own[j][c], d);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < J; ++j) {
#pragma unroll
        for (int c = 0; c < V; ++c) {
          s += v[j][c];
          if constexpr (MODE != kLossOnly) d = __fmaf_rn(v[j][c], own[j][c], d);
        }
      }
    }
    const auto add = [](float p, float q) { return p + q; };
    s = reduce<L>(s, add);
    if constexpr (MODE != kLossOnly) d = reduce<L>(d, add);
    const float inv = s == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(s);
    d = -(d * inv) * inv;
#pragma unroll
    for (int j = 0; j < J; ++j) {
#pragma unroll
      for (int c = 0; c < V; ++c) {
        part[j][c] = __fmaf_rn(v[j][c], inv, part[j][c]);
        if constexpr (MODE != kLossOnly) {
          v[j][c] *= __fmaf_rn(own[j][c], inv, d);
          if constexpr (MODE == kAccumulate) out[j][c] = s == 0.0f ? old[j][c] : (T)((float)old[j][c] + v[j][c]);
          else out[j][c] = (T)v[j][c];
        }
      }
    }
    // The sum is 0 where nothing is possible and where the token is left out (and nowhere else: the largest
    // logit's term is nearly 1): the gradient is 0 whatever the factor.
    if constexpr (MODE == kGradient) {
      if (__builtin_amdgcn_ballot_w64(s == 0.0f) != 0) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
#pragma unroll
          for (int c = 0; c < V; ++c) out[j][c] = s == 0.0f ? (T)0.0f : out[j][c];
        }
      }
    }
  };
  if (left > 0) {
    vec out[J];
    const bool there = t0 + end < t1;
    T* row = MODE == kLossOnly ? nullptr : grad + (int64_t)(there ? t0 + end : t0) * a.g_token;
    token(last, there && kept(there ? end : 0), row, out);
    if constexpr (MODE != kLossOnly) {
      if (there) ch.store(row, out);
    }
  }
  T* row = MODE == kLossOnly ? nullptr : grad + (int64_t)(t0 + slot) * a.g_token;
  const int64_t row_step = (int64_t)kTokens * a.g_token;
  // The first loads have long arrived; once nothing is under way at the loop's start, the waits within it count
  // the loads and stores of a round and no others.
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
  int k = 0;
  const auto go = [&](vec (&raw)[J], bool reload) {
    vec out[J];
    token(raw, kept(k * kTokens + slot), row, out);
    if (reload) {
      ch.load(ahead, raw);
      ahead += k + kAhead + 2 < whole ? step : 0;  // past the last step its loads are repeated
    }
    if constexpr (MODE != kLossOnly) {
      ch.store(row, out);
      row += row_step;
    }
    if (k % kFoldTokens == kFoldTokens - 2) fold();
    ++k;
  };
  while (k + kAhead < whole) {  // the loads of step k go to place k % (kAhead + 1): a move would wait for them
#pragma unroll
    for (int u = 0; u <= kAhead; ++u) go(next[u], true);
  }
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    if (k < whole) go(next[u], false);
  }
  fold();
  // Every lane's sums to LDS (a pitch that lets two lanes at most of each 32 meet in a bank), then for each expert
  // kSlices threads over the groups of lanes, then one over those threads.
  constexpr int kPitch = kThreads + 8, kWidth = L * V, kGroups = kThreads / L;
  constexpr int kSlices = kWidth < kThreads ? kThreads / kWidth : 1;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    __syncthreads();  // share, or the last sums, have been read
#pragma unroll
    for (int c = 0; c < V; ++c) work.sums[c * kPitch + threadIdx.x] = total[j][c];
    __syncthreads();
    for (int q = threadIdx.x % (kSlices * kWidth); q < kSlices * kWidth; q += kThreads) {
      const int slice = q / kWidth, l = q % kWidth / V, k = j * kWidth + q % kWidth;
      const int c = NARROW || k >= experts ? q % V : k - min((j * L + l) * V, experts - V);
      double s = 0.0;
#pragma unroll
      for (int g = 0; g < kGroups / kSlices; ++g) s += work.sums[c * kPitch + (slice * (kGroups / kSlices) + g) * L + l];
      if constexpr (kSlices == 1) {
        if (k < experts) emit(k, s);
      } else {
        work.stage[q] = s;
      }
    }
    if constexpr (kSlices > 1) {
      __syncthreads();
      const int k = j * kWidth + threadIdx.x;
      if ((int)threadIdx.x < kWidth && k < experts) {
        double s = 0.0;
#pragma unroll
        for (int q = 0; q < kSlices; ++q) s += work.stage[q * kWidth + threadIdx.x];
        emit(k, s);
      }
    }
  }
}

// The gradient's factor times the counts less their mean.  hist: counts, and in its last two words
// kept tokens and choices in all.
template <int kThreads>
__device__ __forceinline__ void make_share(const BalanceArgs& a, double up, const uint32_t* hist, float* share) {
  const uint32_t kept = hist[kCountWords];
  const double mean = (double)hist[kCountWords + 1] / (double)a.experts;
  const double n = kept == 0 ? 1.0 : (double)kept;
  const double f = a.coef * (double)a.experts / (n * n * (double)a.top) * up;
  for (int k = threadIdx.x; k < a.experts; k += kThreads) share[k] = (float)(f * ((double)hist[k] - mean));
  __syncthreads();
}

// Rows of part_counts summed in one column, 16 loads under way at a time.
__device__ __forceinline__ uint32_t sum_column(const uint32_t* p, int pitch, int rows) {
  uint32_t s = 0;
  int b = 0;
  for (; b + 16 <= rows; b += 16) {
    uint32_t v[16];
#pragma unroll
    for (int u = 0; u < 16; ++u) v[u] = p[(size_t)(b + u) * pitch];
#pragma unroll
    for (int u = 0; u < 16; ++u) s += v[u];
  }
#pragma unroll 4
  for (; b < rows; ++b) s += p[(size_t)b * pitch];
  return s;
}

// A row of part_counts from hist: the counts, kept tokens, choices in all.
template <int kThreads>
__device__ __forceinline__ void write_counts(const BalanceArgs& a, uint32_t* out, const uint32_t* hist) {
  for (int k = threadIdx.x; k < a.experts; k += kThreads) out[k] = hist[k];
  if (threadIdx.x < 2) out[a.experts + threadIdx.x] = hist[kCountWords + threadIdx.x];
}

// Bound by memory where there is enough of it: 32768 x 256 x 8 learners in bf16 with the gradient, 268 MB, 52 to 55 us,
// 5 TB/s (a copy of as much takes 50); 131 vector instructions for a wave's 512 logits, 62% of its time.  Small
// calls are all latency: 4096 x 64 x 4 learners (4.2 MB) 5 us, of which 2 are the counts' and 1 the final sums'.
// Added to a gradient, which is read where it is needed: the large one 403 MB, 71 to 80 us, 5 to 5.7 TB/s, the small one 7 us.
template <typename T, int L, int J, bool NARROW, int MODE>
__global__ __launch_bounds__(kBalanceBlock) void k_balance(const BalanceArgs a) {
  __shared__ Work<T, kBalanceBlock> work;
  const int i = a.learner[blockIdx.y], row = a.experts + 2;
  const int t0 = blockIdx.x * a.block_tokens, t1 = min(a.tokens, t0 + a.block_tokens);
  const double up = MODE != kLossOnly && a.grad_scale != nullptr ? a.grad_scale[i] : 1.0;
  if (blockIdx.x == 0 && threadIdx.x == 0) a.tickets[blockIdx.y] = 0;  // k_balance_final's
  const uint32_t* part = a.part_counts + (size_t)blockIdx.y * a.count_blocks * row;
  double* out = a.part_probs + ((size_t)blockIdx.y * a.blocks + blockIdx.x) * a.experts;
  double loss = 0.0;
  pass<T, L, J, NARROW, MODE, kBalanceBlock>(a, i, t0, t1, [&] {
    if (MODE == kLossOnly || a.count_blocks == 1) {
      // the gradient needs all of the learner's counts: every block counts for itself where that is little work
      if constexpr (MODE == kLossOnly) count<kBalanceBlock>(a, i, t0, t1, work.hist);
      else count<kBalanceBlock>(a, i, 0, a.tokens, work.hist);
      if (MODE == kLossOnly || blockIdx.x == 0)
        write_counts<kBalanceBlock>(a, a.part_counts + ((size_t)blockIdx.y * a.count_blocks + blockIdx.x) * row, work.hist);
    } else {
      for (int k = threadIdx.x; k < a.experts; k += kBalanceBlock) work.hist[k] = sum_column(part + k, row, a.count_blocks);
      if (threadIdx.x < 128) {  // a wave for the kept tokens, one for the choices, a lane for each block
        const int lane = threadIdx.x % 64, w = threadIdx.x / 64;
        uint32_t n = 0;
        for (int b = lane; b < a.count_blocks; b += 64) n += part[(size_t)b * row + a.experts + w];
        n = reduce<64>(n, [](uint32_t p, uint32_t q) { return p + q; });
        if (lane == 0) work.hist[kCountWords + w] = n;
      }
      __syncthreads();
    }
    if constexpr (MODE != kLossOnly) make_share<kBalanceBlock>(a, up, work.hist, work.share);
  }, [&](int k, double sum) {
    out[k] = sum;
    if constexpr (MODE != kLossOnly) loss += (double)work.hist[k] * sum;
  }, work);
  if constexpr (MODE != kLossOnly) {  // this block's tokens' part of the loss
    loss = wave_sum(loss);
    if (threadIdx.x % 64 == 0) work.red[threadIdx.x / 64] = loss;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < kBalanceBlock / 64; ++w) loss += work.red[w];
      a.part_loss[(size_t)blockIdx.y * a.loss_parts + blockIdx.x] = loss;
    }
  }
}

// What is left to do for expert k of learner i once its sums are known; returns its part of the
// loss, but for the loss's factor.
__device__ __forceinline__ double finish_expert(const BalanceArgs& a, int i, int k, uint32_t count, double sum,
                                                uint32_t kept, int64_t total) {
  const double mean = kept == 0 ? 0.0 : sum / (double)kept;
  a.counts[(int64_t)i * a.counts_stride + k] = (int64_t)count;
  if (a.totals != nullptr) a.totals[(int64_t)i * a.totals_stride + k] = total + (int64_t)count;
  if (a.means != nullptr) a.means[(int64_t)i * a.experts + k] = (float)mean;
  return (double)count * mean;
}

__device__ __forceinline__ void write_loss(const BalanceArgs& a, int i, uint32_t kept, double sum) {
  const double n = kept == 0 ? 1.0 : (double)kept;
  a.loss[i] = (float)(a.coef * (double)a.experts / (n * (double)a.top) * sum);
}

// All latency: 64 tokens of 8 experts 5 us, of which the call's launch and its loads are half.
template <typename T, int L, int J, bool NARROW, int MODE>
__global__ __launch_bounds__(kBalanceOne) void k_balance_one(const BalanceArgs a) {
  __shared__ Work<T, kBalanceOne> work;
  const int i = a.learner[blockIdx.x];
  // read early: nothing of the call's waits for memory after the logits
  const double up = MODE != kLossOnly && a.grad_scale != nullptr ? a.grad_scale[i] : 1.0;
  const int64_t* totals = a.totals != nullptr ? a.totals + (int64_t)i * a.totals_stride : nullptr;
  const int64_t total = totals != nullptr && (int)threadIdx.x < a.experts ? totals[threadIdx.x] : 0;
  double loss = 0.0;
  pass<T, L, J, NARROW, MODE, kBalanceOne>(a, i, 0, a.tokens, [&] {
    count<kBalanceOne>(a, i, 0, a.tokens, work.hist);
    if constexpr (MODE != kLossOnly) make_share<kBalanceOne>(a, up, work.hist, work.share);
  }, [&](int k, double sum) {
    const int64_t before = k == (int)threadIdx.x || totals == nullptr ? total : totals[k];
    loss += finish_expert(a, i, k, work.hist[k], sum, work.hist[kCountWords], before);
  }, work);
  loss = wave_sum(loss);
  if ((threadIdx.x & 63) == 0) work.red[threadIdx.x >> 6] = loss;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kBalanceOne / 64; ++w) loss += work.red[w];
    write_loss(a, i, work.hist[kCountWords], loss);
  }
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------
template <int N>
using Int = std::integral_constant<int, N>;

// f(lanes per token, loads per lane, whether a row is narrower than one load), lanes at least
// kLeast: a call small enough for one block is all latency, and two widths serve it.
template <int V, int kLeast, typename F>
hipError_t by_lanes(int experts, F&& f) {
  if (experts < V) return f(Int<1>(), Int<1>(), std::true_type());
  const int l = balance_lanes(experts, V);
  if constexpr (kLeast == 1) {
    switch (l) {
      case 1: return f(Int<1>(), Int<1>(), std::false_type());
      case 2: return f(Int<2>(), Int<1>(), std::false_type());
      case 4: return f(Int<4>(), Int<1>(), std::false_type());
      case 16: return f(Int<16>(), Int<1>(), std::false_type());
      case 32: return f(Int<32>(), Int<1>(), std::false_type());
      default: break;
    }
  }
  if (l <= 8) return f(Int<8>(), Int<1>(), std::false_type());
  if (experts <= 64 * V) return f(Int<64>(), Int<1>(), std::false_type());
  if constexpr (V == 4) {
    if (experts > 128 * V) return f(Int<64>(), Int<4>(), std::false_type());
  }
  return f(Int<64>(), Int<2>(), std::false_type());
}

template <typename T, int MODE>
hipError_t launch_pass(const BalanceArgs& a, bool one, hipStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  if (one) {
    return by_lanes<V, 8>(a.experts, [&](auto l, auto j, auto narrow) {
      hipLaunchKernelGGL((k_balance_one<T, decltype(l)::value, decltype(j)::value, decltype(narrow)::value, MODE>),
                         dim3(a.n_present), dim3(kBalanceOne), 0, s, a);
      return hipGetLastError();
    });
  }
  return by_lanes<V, 1>(a.experts, [&](auto l, auto j, auto narrow) {
    hipLaunchKernelGGL((k_balance<T, decltype(l)::value, decltype(j)::value, decltype(narrow)::value, MODE>),
                       dim3(a.blocks, a.n_present), dim3(kBalanceBlock), 0, s, a);
    return hipGetLastError();
  });
}

template <typename T>
hipError_t launch_typed(const BalanceArgs& a, bool one, hipStream_t s) {
  if (a.grad == nullptr) return launch_pass<T, kLossOnly>(a, one, s);
  return a.accumulate != 0 ? launch_pass<T, kAccumulate>(a, one, s) : launch_pass<T, kGradient>(a, one, s);
}

}  // namespace
}  // namespace dlc
