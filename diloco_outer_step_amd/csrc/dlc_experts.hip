// gfx950 kernels of the mixture-of-experts calls.
//
//   k_balance_count  choices per expert, kept tokens of a block
//   k_balance        softmax of every token, its sum over the tokens, its gradient
//   k_balance_final  the blocks' sums in a fixed order -> counts, means, loss
//   k_balance_one    all three in one block per learner, for few tokens
//   k_expert_weights merge weights of every (tensor, learner) from the counts
//
// The gradient of the loss coef E sum_e f_e P_e, f the share of the choices and P the mean
// probabilities, is a softmax's: coef E / (n^2 top) p_e (c_e - sum_j p_j c_j).  It needs the
// whole counts but not P, so the choices (a fiftieth of the logits' bytes) are counted first
// and the logits are read once.  Taking c less its mean changes nothing, as sum p = 1, and
// keeps the bracket from cancelling when the experts are used evenly.
#include "dlc_experts.h"

#include <type_traits>

namespace dlc {
namespace {

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
  return v;
}

// The value of a lane of the other half of each group of L lanes, both halves holding one
// value each.
template <int L>
__device__ __forceinline__ float other_half(float v) {
  const int x = __builtin_bit_cast(int, v);
  if constexpr (L == 2) return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(x, 0xB1, 0xF, 0xF, true));   // quad 1 0 3 2
  if constexpr (L == 4) return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(x, 0x4E, 0xF, 0xF, true));   // quad 2 3 0 1
  if constexpr (L == 8) return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(x, 0x141, 0xF, 0xF, true));  // half row mirrored
  if constexpr (L == 16) return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(x, 0x140, 0xF, 0xF, true)); // row mirrored
  if constexpr (L == 32) return __shfl_xor(v, 16, 64);
  if constexpr (L == 64) return __shfl_xor(v, 32, 64);
  return v;
}

template <int L, typename F>
__device__ __forceinline__ float reduce(float v, F&& f) {
  if constexpr (L >= 2) v = f(v, other_half<2>(v));
  if constexpr (L >= 4) v = f(v, other_half<4>(v));
  if constexpr (L >= 8) v = f(v, other_half<8>(v));
  if constexpr (L >= 16) v = f(v, other_half<16>(v));
  if constexpr (L >= 32) v = f(v, other_half<32>(v));
  if constexpr (L >= 64) v = f(v, other_half<64>(v));
  return v;
}

// ---------------------------------------------------------------------------
// Counting
// ---------------------------------------------------------------------------
// f / top for f below kCountTokens top: the inverse is at most (top - 1) / 2^32 too large per
// unit of f, and f (top - 1) < 2^18 64^2 <= 2^32.
__device__ __forceinline__ uint32_t divide(uint32_t f, uint32_t inverse) {
  return inverse == 0 ? f : __umulhi(f, inverse);
}

// A learner's choices of tokens [t0, t1) -> hist[0 .. experts), kept tokens -> hist[experts].
// hist holds kCountWords + 1 words: copies of the histogram, so that lanes with the same choice
// (routers have favourites, and few experts) add to different words.
template <int kThreads, typename I>
__device__ void count_choices(const BalanceArgs& a, int i, int t0, int t1, uint32_t* hist) {
  const uint32_t e = (uint32_t)a.experts;
  uint32_t copies = 1;
  while (copies < 64 && 2 * copies * e <= kCountWords) copies *= 2;
  for (uint32_t k = threadIdx.x; k < copies * e; k += kThreads) hist[k] = 0;
  if (threadIdx.x == 0) hist[kCountWords] = 0;
  __syncthreads();
  uint32_t* mine = hist + (threadIdx.x & (copies - 1)) * e;
  const I* ids = (const I*)a.choices + (int64_t)i * a.c_learner + (int64_t)t0 * a.c_token;
  const uint8_t* mask = a.mask != nullptr ? a.mask + (int64_t)i * a.mask_learner + t0 : nullptr;
  const uint32_t n = (uint32_t)(t1 - t0) * (uint32_t)a.top;
  constexpr int U = 4;
  for (uint32_t f0 = threadIdx.x; f0 < n; f0 += U * kThreads) {
    I id[U];
    bool keep[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t f = f0 + u * kThreads;  // below 2^24 + 2^12
      keep[u] = f < n;
      id[u] = 0;
      if (keep[u]) {
        const uint32_t t = divide(f, a.top_inverse);
        id[u] = ids[(int64_t)t * a.c_token + (f - t * (uint32_t)a.top)];
        if (mask != nullptr) keep[u] = mask[t] != 0;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (keep[u] && id[u] >= 0 && id[u] < (I)e) atomicAdd(&mine[(uint32_t)id[u]], 1u);
    }
  }
  if (mask != nullptr) {
    uint32_t kept = 0;
    for (int t = threadIdx.x; t < t1 - t0; t += kThreads) kept += mask[t] != 0;
    if (kept != 0) atomicAdd(&hist[kCountWords], kept);
  } else if (threadIdx.x == 0) {
    hist[kCountWords] = (uint32_t)(t1 - t0);
  }
  __syncthreads();
  // a thread sums the copies of its experts; only it writes hist[its experts]
  for (uint32_t k = threadIdx.x; k < e; k += kThreads) {
    uint32_t s = 0;
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

__global__ __launch_bounds__(kCountBlock) void k_balance_count(const BalanceArgs a) {
  __shared__ uint32_t hist[kCountWords + 1];
  const int t0 = blockIdx.x * a.count_tokens, t1 = min(a.tokens, t0 + a.count_tokens);
  count<kCountBlock>(a, a.learner[blockIdx.y], t0, t1, hist);
  uint32_t* out = a.part_counts + ((size_t)blockIdx.y * a.count_blocks + blockIdx.x) * (a.experts + 1);
  for (int k = threadIdx.x; k < a.experts; k += kCountBlock) out[k] = hist[k];
  if (threadIdx.x == 0) out[a.experts] = hist[kCountWords];
}

// ---------------------------------------------------------------------------
// The pass over the logits
// ---------------------------------------------------------------------------
// A lane holds V = 16 bytes of a token's logits J times, L lanes a token, so a wave works on
// 64 / L tokens at once.  Logits lie at any address that their type allows; 16-byte loads
// need no more on gfx950.
template <typename T, int J>
struct Chunks {
  static constexpr int V = 16 / (int)sizeof(T);
  typedef T vec __attribute__((ext_vector_type(V), aligned(sizeof(T))));
  int start[J];  // the lane's first element; the row's last V elements where its chunk would pass the end
  int lo[J];     // elements [lo, hi) of the chunk are this lane's
  int hi[J];
  __device__ __forceinline__ Chunks(int lane, int lanes, int experts) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int at = (j * lanes + lane) * V;
      start[j] = at;
      lo[j] = 0;
      hi[j] = V;
      if (at >= experts) {
        start[j] = 0;
        hi[j] = 0;
      } else if (at + V > experts) {
        start[j] = experts >= V ? experts - V : 0;
        lo[j] = at - start[j];
        hi[j] = experts >= V ? V : experts;
      }
    }
  }
  __device__ __forceinline__ void load(const T* row, int experts, vec (&q)[J]) const {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      q[j] = vec{};
      if (hi[j] == 0) continue;
      if (experts >= V) {
        q[j] = *(const vec*)(row + start[j]);
      } else {
#pragma unroll
        for (int c = 0; c < V; ++c) {
          if (c < experts) q[j][c] = row[c];
        }
      }
    }
  }
  __device__ __forceinline__ void store(T* row, const vec (&q)[J]) const {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      if (lo[j] == 0 && hi[j] == V) {
        *(vec*)(row + start[j]) = q[j];
      } else {
#pragma unroll
        for (int c = 0; c < V; ++c) {
          if (c >= lo[j] && c < hi[j]) row[start[j] + c] = q[j][c];
        }
      }
    }
  }
};

// Learner i's tokens [t0, t1): their probabilities' sums into sum[experts] (LDS), and with
// GRAD the gradient.  share: (counts less their mean) times the gradient's factor (LDS).
template <typename T, int L, int J, bool GRAD, int kThreads>
__device__ __forceinline__ void pass(const BalanceArgs& a, int i, int t0, int t1, const float* share, double* sum) {
  using C = Chunks<T, J>;
  using vec = typename C::vec;
  constexpr int V = C::V;
  constexpr int kTokens = kThreads / L;
  const int lane = threadIdx.x % L, slot = threadIdx.x / L;
  const int experts = a.experts;
  const C ch(lane, L, experts);
  const bool cut = experts != L * J * V;  // some lane holds elements that are not its own
  const T* x = (const T*)a.logits + (int64_t)i * a.x_learner;
  T* grad = GRAD ? (T*)a.grad + (int64_t)i * a.g_learner : nullptr;
  const uint8_t* mask = a.mask != nullptr ? a.mask + (int64_t)i * a.mask_learner : nullptr;
  float own[J][V];
  if constexpr (GRAD) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
#pragma unroll
      for (int c = 0; c < V; ++c) own[j][c] = c >= ch.lo[j] && c < ch.hi[j] ? share[ch.start[j] + c] : 0.0f;
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
  vec next[J];
  bool next_live = false;
  const auto request = [&](int t) {
    next_live = t < t1;
    const int at = next_live ? t : t1 - 1;
    if (mask != nullptr) next_live = next_live && mask[at] != 0;
    ch.load(x + (int64_t)at * a.x_token, experts, next);
  };
  if (t0 < t1) request(t0 + slot);
  int folded = 0;
  for (int base = t0; base < t1; base += kTokens) {
    const int t = base + slot;
    const bool live = next_live;
    float v[J][V];
#pragma unroll
    for (int j = 0; j < J; ++j) {
#pragma unroll
      for (int c = 0; c < V; ++c) v[j][c] = (float)next[j][c];
    }
    if (base + kTokens < t1) request(t + kTokens);
    if (cut || __builtin_amdgcn_ballot_w64(live) != ~0ull) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
#pragma unroll
        for (int c = 0; c < V; ++c) v[j][c] = live && c >= ch.lo[j] && c < ch.hi[j] ? v[j][c] : -__builtin_inff();
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
    float s = 0.0f, d = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
#pragma unroll
      for (int c = 0; c < V; ++c) {
        v[j][c] = __builtin_amdgcn_exp2f((v[j][c] - m) * 1.44269504f);
        s += v[j][c];
        if constexpr (GRAD) d = __fmaf_rn(v[j][c], own[j][c], d);
      }
    }
    const auto add = [](float p, float q) { return p + q; };
    s = reduce<L>(s, add);
    if constexpr (GRAD) d = reduce<L>(d, add);
    const float inv = s == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(s);
    d *= inv;
    vec out[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const float p = v[j][c] * inv;
        part[j][c] += p;
        if constexpr (GRAD) {
          const float g = p * (own[j][c] - d);
          out[j][c] = (T)g;
          v[j][c] = g;
        }
      }
    }
    if constexpr (GRAD) {
      if (t < t1 && (live || a.accumulate == 0)) {
        T* row = grad + (int64_t)t * a.g_token;
        if (a.accumulate != 0) {
          vec old[J];
          ch.load(row, experts, old);
#pragma unroll
          for (int j = 0; j < J; ++j) {
#pragma unroll
            for (int c = 0; c < V; ++c) out[j][c] = (T)((float)old[j][c] + v[j][c]);
          }
        }
        ch.store(row, out);
      }
    }
    if (++folded == kFoldTokens) {
      fold();
      folded = 0;
    }
  }
  fold();
  // over the wave's tokens, then the waves in order
#pragma unroll
  for (int j = 0; j < J; ++j) {
#pragma unroll
    for (int c = 0; c < V; ++c) {
#pragma unroll
      for (int k = L; k < 64; k *= 2) total[j][c] += __shfl_xor(total[j][c], k, 64);
    }
  }
  for (int w = 0; w < kThreads / 64; ++w) {
    if ((int)threadIdx.x / 64 == w && threadIdx.x % 64 < L) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
#pragma unroll
        for (int c = 0; c < V; ++c) {
          if (c >= ch.lo[j] && c < ch.hi[j]) {
            double* to = sum + ch.start[j] + c;
            *to = (w == 0 ? 0.0 : *to) + total[j][c];
          }
        }
      }
    }
    __syncthreads();
  }
}

// The gradient's factor times the counts less their mean.  every: experts' counts (LDS).
template <int kThreads>
__device__ __forceinline__ void make_share(const BalanceArgs& a, int i, const uint32_t* every, uint32_t kept,
                                           float* share, double* red) {
  double c = 0.0;
  for (int k = threadIdx.x; k < a.experts; k += kThreads) c += (double)every[k];
  c = wave_sum(c);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = c;
  __syncthreads();
  double mean = 0.0;
  for (int w = 0; w < kThreads / 64; ++w) mean += red[w];
  mean /= (double)a.experts;
  const double n = kept == 0 ? 1.0 : (double)kept;
  const double up = a.grad_scale != nullptr ? a.grad_scale[i] : 1.0;
  const double f = a.coef * (double)a.experts / (n * n * (double)a.top) * up;
  for (int k = threadIdx.x; k < a.experts; k += kThreads) share[k] = (float)(f * ((double)every[k] - mean));
  __syncthreads();
}

template <typename T, int L, int J, bool GRAD>
__global__ __launch_bounds__(kBalanceBlock) void k_balance(const BalanceArgs a) {
  __shared__ double sum[kMaxExperts];
  __shared__ float share[GRAD ? kMaxExperts : 1];
  __shared__ uint32_t hist[GRAD ? kMaxExperts + 1 : kCountWords + 1];
  __shared__ double red[kBalanceBlock / 64];
  const int i = a.learner[blockIdx.y];
  const int t0 = blockIdx.x * a.block_tokens, t1 = min(a.tokens, t0 + a.block_tokens);
  if constexpr (GRAD) {
    const uint32_t* part = a.part_counts + (size_t)blockIdx.y * a.count_blocks * (a.experts + 1);
    for (int k = threadIdx.x; k <= a.experts; k += kBalanceBlock) {
      uint32_t s = 0;
#pragma unroll 8
      for (int b = 0; b < a.count_blocks; ++b) s += part[(size_t)b * (a.experts + 1) + k];
      hist[k] = s;
    }
    __syncthreads();
    make_share<kBalanceBlock>(a, i, hist, hist[a.experts], share, red);
  } else {
    count<kBalanceBlock>(a, i, t0, t1, hist);
    uint32_t* out = a.part_counts + ((size_t)blockIdx.y * a.blocks + blockIdx.x) * (a.experts + 1);
    for (int k = threadIdx.x; k < a.experts; k += kBalanceBlock) out[k] = hist[k];
    if (threadIdx.x == 0) out[a.experts] = hist[kCountWords];
  }
  pass<T, L, J, GRAD, kBalanceBlock>(a, i, t0, t1, share, sum);
  double* out = a.part_probs + ((size_t)blockIdx.y * a.blocks + blockIdx.x) * a.experts;
  for (int k = threadIdx.x; k < a.experts; k += kBalanceBlock) out[k] = sum[k];
}

// A learner's results from its whole counts and probability sums, one expert a thread
// (threads past the experts hold zeros).
template <int kThreads>
__device__ __forceinline__ void finish(const BalanceArgs& a, int i, uint32_t count, double sum, uint32_t kept,
                                       double* red) {
  const int k = threadIdx.x;
  const double mean = kept == 0 ? 0.0 : sum / (double)kept;
  if (k < a.experts) {
    a.counts[(int64_t)i * a.counts_stride + k] = (int64_t)count;
    if (a.totals != nullptr) a.totals[(int64_t)i * a.totals_stride + k] += (int64_t)count;
    if (a.means != nullptr) a.means[(int64_t)i * a.experts + k] = (float)mean;
  }
  const double s = wave_sum(k < a.experts ? (double)count * mean : 0.0);
  if ((k & 63) == 0) red[k >> 6] = s;
  __syncthreads();
  if (k == 0) {
    double l = 0.0;
    for (int w = 0; w < kThreads / 64; ++w) l += red[w];
    const double n = kept == 0 ? 1.0 : (double)kept;
    a.loss[i] = (float)(a.coef * (double)a.experts / (n * (double)a.top) * l);
  }
}

// One block per learner; thread (s, k) sums every slices-th block's expert k, then the
// slices in order.
__global__ __launch_bounds__(kMaxExperts) void k_balance_final(const BalanceArgs a) {
  __shared__ double sums[kMaxExperts];
  __shared__ uint32_t counts[kMaxExperts];
  __shared__ double red[kMaxExperts / 64];
  __shared__ uint32_t kept;
  const int e = a.experts, slices = kMaxExperts / e;
  const int k = threadIdx.x % e, s = threadIdx.x / e;
  const uint32_t* part = a.part_counts + (size_t)blockIdx.x * a.count_blocks * (e + 1);
  const double* prob = a.part_probs + (size_t)blockIdx.x * a.blocks * e;
  double v = 0.0;
  uint32_t c = 0, n = 0;
  if (threadIdx.x == 0) kept = 0;
  if (s < slices) {
#pragma unroll 8
    for (int b = s; b < a.blocks; b += slices) v += prob[(size_t)b * e + k];
#pragma unroll 8
    for (int b = s; b < a.count_blocks; b += slices) c += part[(size_t)b * (e + 1) + k];
  }
  for (int b = threadIdx.x; b < a.count_blocks; b += kMaxExperts) n += part[(size_t)b * (e + 1) + e];
  sums[threadIdx.x] = v;
  counts[threadIdx.x] = c;
  __syncthreads();
  if (n != 0) atomicAdd(&kept, n);
  v = 0.0;
  c = 0;
  if ((int)threadIdx.x < e) {
    for (int q = 0; q < slices; ++q) {
      v += sums[q * e + threadIdx.x];
      c += counts[q * e + threadIdx.x];
    }
  }
  __syncthreads();
  finish<kMaxExperts>(a, a.learner[blockIdx.x], c, v, kept, red);
}

template <typename T, int L, int J, bool GRAD>
__global__ __launch_bounds__(kBalanceOne) void k_balance_one(const BalanceArgs a) {
  __shared__ double sum[kMaxExperts];
  __shared__ float share[GRAD ? kMaxExperts : 1];
  __shared__ uint32_t hist[kCountWords + 1];
  __shared__ double red[kBalanceOne / 64];
  const int i = a.learner[blockIdx.x];
  count<kBalanceOne>(a, i, 0, a.tokens, hist);
  const uint32_t kept = hist[kCountWords];
  if constexpr (GRAD) make_share<kBalanceOne>(a, i, hist, kept, share, red);
  pass<T, L, J, GRAD, kBalanceOne>(a, i, 0, a.tokens, share, sum);
  const bool mine = (int)threadIdx.x < a.experts;
  finish<kBalanceOne>(a, i, mine ? hist[threadIdx.x] : 0u, mine ? sum[threadIdx.x] : 0.0, kept, red);
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

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------
// Lanes per token: the fewest that hold a row in one 16-byte load each, 64 at most.
int lanes_of(int experts, int v) {
  int l = 1;
  while (l < 64 && l * v < experts) l *= 2;
  return l;
}

template <int N>
using Int = std::integral_constant<int, N>;

// f(lanes per token, loads per lane), lanes at least `least`: a call small enough for one block
// is all latency, and two widths serve it.
template <int V, typename F>
hipError_t by_lanes(int experts, int least, F&& f) {
  const int l = lanes_of(experts, V);
  if (least == 1) {
    switch (l) {
      case 1: return f(Int<1>(), Int<1>());
      case 2: return f(Int<2>(), Int<1>());
      case 4: return f(Int<4>(), Int<1>());
      case 16: return f(Int<16>(), Int<1>());
      case 32: return f(Int<32>(), Int<1>());
      default: break;
    }
  }
  if (l <= 8) return f(Int<8>(), Int<1>());
  if (experts <= 64 * V) return f(Int<64>(), Int<1>());
  if constexpr (V == 4) {
    if (experts > 128 * V) return f(Int<64>(), Int<4>());
  }
  return f(Int<64>(), Int<2>());
}

template <typename T, bool GRAD>
hipError_t launch_pass(const BalanceArgs& a, bool one, hipStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  if (one) {
    return by_lanes<V>(a.experts, 8, [&](auto l, auto j) {
      if constexpr (decltype(l)::value >= 8)
        hipLaunchKernelGGL((k_balance_one<T, decltype(l)::value, decltype(j)::value, GRAD>), dim3(a.n_present),
                           dim3(kBalanceOne), 0, s, a);
      return hipGetLastError();
    });
  }
  return by_lanes<V>(a.experts, 1, [&](auto l, auto j) {
    hipLaunchKernelGGL((k_balance<T, decltype(l)::value, decltype(j)::value, GRAD>), dim3(a.blocks, a.n_present),
                       dim3(kBalanceBlock), 0, s, a);
    return hipGetLastError();
  });
}

template <typename T>
hipError_t launch_typed(const BalanceArgs& a, bool one, hipStream_t s) {
  return a.grad != nullptr ? launch_pass<T, true>(a, one, s) : launch_pass<T, false>(a, one, s);
}

hipError_t launch_any(const BalanceArgs& a, int32_t type, bool one, hipStream_t s) {
  if (type == kF32) return launch_typed<float>(a, one, s);
  if (type == kBF16) return launch_typed<__bf16>(a, one, s);
  return launch_typed<_Float16>(a, one, s);
}

}  // namespace

hipError_t launch_balance_one(const BalanceArgs& a, int32_t type, hipStream_t s) {
  return launch_any(a, type, true, s);
}

hipError_t launch_balance(const BalanceArgs& a, int32_t type, hipStream_t s) {
  return launch_any(a, type, false, s);
}

hipError_t launch_balance_count(const BalanceArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(k_balance_count, dim3(a.count_blocks, a.n_present), dim3(kCountBlock), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_balance_final(const BalanceArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(k_balance_final, dim3(a.n_present), dim3(kMaxExperts), 0, s, a);
  return hipGetLastError();
}

int32_t balance_tokens(int32_t type, int32_t experts, int32_t threads) {
  return threads / lanes_of(experts, type == kF32 ? 4 : 8);
}

hipError_t launch_expert_weights(const WeightArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(k_expert_weights, dim3((a.n_tensors + 63) / 64), dim3(64), 0, s, a);
  return hipGetLastError();
}

}  // namespace dlc
