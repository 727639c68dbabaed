// gfx950 kernels of the learner's inner step: the global gradient norm with its
// clipping factor, and AdamW with 32-bit or 8-bit coded moments, over all tensors
// of all present learners.
//
//   k_norm_partial  sum of squares of a block's gradients, fp64
//   k_norm_final    the blocks' sums in a fixed order -> norm and gradient scale
//   k_norm_small    both in one block per learner, for short lists
//   k_adamw         one pass over theta, the moments and the gradients
//   k_adamw_coded   the same with coded moments
//   k_adamw_advance the learners' step counts, where k_adamw's blocks do not count them
//
// AdamW per element, with t = steps + 1, g = grad_scale * grad, eta = lr * lr_scale:
//   m     <- beta1 m + (1 - beta1) g
//   v     <- beta2 v + (1 - beta2) g^2
//   theta <- (1 - eta wd) theta - eta / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
// The moments are computed in fp64 and rounded to fp32 once; the change of theta is an
// fp32 expression of the rounded moments, subtracted from theta with one rounding.
//
// Coded moments: m is an e4m3 code and v an e5m2 code times a power of two shared by
// 64 consecutive elements (an e8m0 byte), so scaling is exact and a code's relative
// step does not depend on its block.  Codes are rounded stochastically: v moves by
// 1 - beta2 (a thousandth) of itself per step while e5m2's step is an eighth to a
// quarter of it, so rounding to nearest would never move it.  The random bits are a
// hash of (seed, t, learner, element): the same call gives the same bits, however the
// tensors are split over calls, launches and blocks.
#include "dlc_inner.h"

#include <type_traits>

namespace dlc {
namespace {

typedef float vf4 __attribute__((ext_vector_type(4)));

// Block -> (group, first element of the row, elements).  The launch geometry lives in the
// kernel arguments and is read by scalar loads; the bucket of the block number leaves few
// ranges, mostly one, to search.
struct Spot {
  int group;
  int64_t base;
  uint32_t count;
};

__device__ __forceinline__ Spot spot(const InnerGeom& g, uint32_t per_block) {
  const uint32_t b = blockIdx.x;
  const uint32_t bucket = g.bucket[b >> g.bucket_shift];
  int lo = (int)(bucket & 0xFFFFu), hi = (int)(bucket >> 16);
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (g.r[mid].block_first() <= b) lo = mid; else hi = mid - 1;
  }
  const InnerRange r = g.r[lo];
  const uint32_t first = (b - r.block_first()) * per_block;  // below count, so below 2^32
  Spot s;
  s.group = (int)r.group();
  s.base = (int64_t)r.lo64 * 64 + first;
  s.count = r.count - first < per_block ? r.count - first : per_block;
  return s;
}

// Loads of four elements at p, the first n of them the tensor's (n may be <= 0 or >= 4).
// Tensors start, and rows end, at multiples of 64 elements, so the four lie within the row
// if the first does: they are loaded whole, and what is behind the tensor is not used.
__device__ __forceinline__ void load4(const float* p, int n, float (&x)[4]) {
  vf4 q = {0.0f, 0.0f, 0.0f, 0.0f};
  if (n > 0) q = __builtin_nontemporal_load((const vf4*)p);
#pragma unroll
  for (int c = 0; c < 4; ++c) x[c] = q[c];
}

template <typename T>
__device__ __forceinline__ void store4(T* p, int n, const float (&x)[4]) {
  typedef T v4 __attribute__((ext_vector_type(4)));
  if (n >= 4) {
    v4 q;
#pragma unroll
    for (int c = 0; c < 4; ++c) q[c] = (T)x[c];
    __builtin_nontemporal_store(q, (v4*)p);
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (c < n) p[c] = (T)x[c];
    }
  }
}

// Four gradients as they lie in memory.
template <typename G>
struct Raw4 {
  typedef G v4 __attribute__((ext_vector_type(4)));
  v4 q;
  __device__ __forceinline__ void load(const G* p, int n) {
    q = v4{};
    if (n > 0) q = __builtin_nontemporal_load((const v4*)p);
  }
  __device__ __forceinline__ float value(int c) const { return (float)q[c]; }
};

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
  return v;
}

// The block's sum of v, in every thread.
template <int kThreads>
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double red[kThreads / 64];
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) s += red[w];
  return s;
}

// ---------------------------------------------------------------------------
// The gradient norm
// ---------------------------------------------------------------------------
// The thread's sum of squares over `count` elements at p that the kThreads threads share,
// 16-byte loads, U in flight.
template <int kThreads, int U, typename G>
__device__ __forceinline__ double squares(const G* p, int64_t count) {
  constexpr int V = 16 / (int)sizeof(G);
  typedef G vec __attribute__((ext_vector_type(V)));
  constexpr int64_t kStep = (int64_t)kThreads * V * U;
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  const auto add = [&](const vec& x) {
#pragma unroll
    for (int c = 0; c < V; ++c) {
      const double d = (double)(float)x[c];
      s[c & 3] = __fma_rn(d, d, s[c & 3]);
    }
  };
  int64_t at = 0;
  vec x[U];
  const auto request = [&](int64_t from) {
#pragma unroll
    for (int j = 0; j < U; ++j) x[j] = __builtin_nontemporal_load((const vec*)(p + from) + j * kThreads + threadIdx.x);
  };
  if (kStep <= count) request(0);
  for (; at + kStep <= count; at += kStep) {
    vec y[U];
#pragma unroll
    for (int j = 0; j < U; ++j) y[j] = x[j];
    if (at + 2 * kStep <= count) request(at + kStep);
#pragma unroll
    for (int j = 0; j < U; ++j) add(y[j]);
  }
  for (int64_t e = at + (int64_t)V * threadIdx.x; e < count; e += (int64_t)V * kThreads) {
    vec x = __builtin_nontemporal_load((const vec*)(p + e));  // within the row, see load4
#pragma unroll
    for (int c = 0; c < V; ++c) x[c] = c < count - e ? x[c] : (G)0.0f;
    add(x);
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

__device__ __forceinline__ void write_norm(const NormArgs& a, int i, double sum) {
  const double n = a.unscale * sqrt(sum);
  double scale = a.unscale;
  if (n > a.max_norm) scale = a.unscale * (a.max_norm / n);
  if (!__builtin_isfinite(n)) scale = 0.0;
  a.norm[i] = n;
  a.grad_scale[i] = scale;
}

template <typename G>
__global__ __launch_bounds__(kNormBlock) void k_norm_partial(const NormArgs a, const InnerGeom g) {
  const Spot sp = spot(g, g.per_block);
  const G* row = (const G*)a.grads + (int64_t)a.learner[blockIdx.y] * a.stride;
  const double s = block_sum<kNormBlock>(squares<kNormBlock, kNormLoads>(row + sp.base, sp.count));
  if (threadIdx.x == 0) a.part[(size_t)blockIdx.y * a.n_slots + g.slot_base + blockIdx.x] = s;
}

__global__ __launch_bounds__(kNormFinal) void k_norm_final(const NormArgs a) {
  const double* part = a.part + (size_t)blockIdx.x * a.n_slots;
  double s = 0.0;
  for (int b = threadIdx.x; b < a.n_slots; b += kNormFinal) s += part[b];
  s = block_sum<kNormFinal>(s);
  if (threadIdx.x == 0) write_norm(a, a.learner[blockIdx.x], s);
}

template <typename G>
__global__ __launch_bounds__(kNormFinal) void k_norm_small(const NormArgs a, const InnerGeom g) {
  const int i = a.learner[blockIdx.x];
  const G* row = (const G*)a.grads + (int64_t)i * a.stride;
  double s = 0.0;
  for (int k = 0; k < g.n_ranges; ++k) s += squares<kNormFinal, 1>(row + (int64_t)g.r[k].lo64 * 64, g.r[k].count);
  s = block_sum<kNormFinal>(s);
  if (threadIdx.x == 0) write_norm(a, i, s);
}

// ---------------------------------------------------------------------------
// AdamW
// ---------------------------------------------------------------------------
// 1 - exp(x) for x <= 0 (x = t ln(beta), so 1 - beta^t): the series of exp(y) - 1 at
// y = x / 64, then six doublings exp(2 y) - 1 = p (p + 2), which lose nothing to
// cancellation.  Below x = -40 the result is 1 in every format here.
__device__ __forceinline__ double one_minus_exp(double x) {
  const double y = fmax(x, -40.0) * 0x1p-6;
  double p = 1.0 / 39916800.0;  // 1 / 11!: the next term is below 2^-33 of the sum at y = -0.625
  p = __fma_rn(p, y, 1.0 / 3628800.0);
  p = __fma_rn(p, y, 1.0 / 362880.0);
  p = __fma_rn(p, y, 1.0 / 40320.0);
  p = __fma_rn(p, y, 1.0 / 5040.0);
  p = __fma_rn(p, y, 1.0 / 720.0);
  p = __fma_rn(p, y, 1.0 / 120.0);
  p = __fma_rn(p, y, 1.0 / 24.0);
  p = __fma_rn(p, y, 1.0 / 6.0);
  p = __fma_rn(p, y, 0.5);
  p = __fma_rn(p, y, 1.0) * y;
#pragma unroll
  for (int k = 0; k < 6; ++k) p = p * (p + 2.0);
  return -p;
}

constexpr unsigned long long kTicket = 1ull << 40;  // above any step count

// What an element's update needs besides the element: the same for a whole block.
struct Rates {
  double b1, c1, b2, c2;  // c1 = (1 - beta1) clip, c2 = (1 - beta2) clip^2
  float shrink;           // eta wd
  float size, root, eps;  // eta / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
};

// A learner's gradient scale; its step is left out unless the scale is finite and positive.
__device__ __forceinline__ double clip_of(const AdamWArgs& a, int learner) {
  return a.grad_scale != nullptr ? a.grad_scale[learner] : 1.0;
}

__device__ __forceinline__ bool takes_step(double clip) { return clip > 0.0 && __builtin_isfinite(clip); }

__device__ __forceinline__ Rates rates_of(const InnerGroup& q, double clip, double lr_scale, uint64_t t) {
  Rates r;
  const double eta = q.lr * lr_scale;
  r.b1 = q.beta1;
  r.c1 = (1.0 - q.beta1) * clip;
  r.b2 = q.beta2;
  r.c2 = (1.0 - q.beta2) * clip * clip;
  r.shrink = (float)(eta * q.weight_decay);
  // both corrections in one evaluation: beta1 in the even lanes, beta2 in the odd ones
  const int c = __float_as_int((float)one_minus_exp((double)t * (threadIdx.x & 1 ? q.log_beta2 : q.log_beta1)));
  r.size = (float)eta * __builtin_amdgcn_rcpf(__int_as_float(__builtin_amdgcn_readlane(c, 0)));
  r.root = __builtin_amdgcn_rsqf(__int_as_float(__builtin_amdgcn_readlane(c, 1)));
  r.eps = (float)q.eps;
  return r;
}

// With decimal betas the exact sums lie on fp32 rounding ties about once in a hundred
// elements (0.8 m + 0.2 g = (4 m + g) / 5), which the last bit in fp64 then decides: each
// product is rounded on its own, as any fp64 evaluation of the formula does.
__device__ __forceinline__ float new_m(double b1, double c1, double m, double grad) {
  return (float)(b1 * m + c1 * grad);
}

__device__ __forceinline__ float new_v(double b2, double c2, double v, double grad) {
  return (float)(b2 * v + c2 * grad * grad);
}

// What a block reads of its learner, before its tile: the loads overlap the search for the
// block's range.
struct Learner {
  double clip, lr_scale;
  uint64_t steps;
};

__device__ __forceinline__ Learner learner_of(const AdamWArgs& a, int i) {
  // no branches: an absent array's place is taken by steps, whose bits are not used
  const double* clip = a.grad_scale != nullptr ? a.grad_scale : (const double*)a.steps;
  const double* lr = a.lr_scale != nullptr ? a.lr_scale : (const double*)a.steps;
  const double c = clip[i], s = lr[i];
  Learner l;
  l.steps = (uint64_t)a.steps[i];
  l.clip = a.grad_scale != nullptr ? c : 1.0;
  l.lr_scale = a.lr_scale != nullptr ? s : 1.0;
  return l;
}

// The learner's step number t = steps + 1.  In calls of few blocks the blocks themselves
// count the step: each adds a ticket above the count once all of its threads have read
// it, and the one that draws the last ticket writes t over count and tickets.
__device__ __forceinline__ uint64_t next_step(const AdamWArgs& a, int i, const Learner& l) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)l.steps);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(l.steps >> 32));
  const uint64_t t = (((uint64_t)hi << 32 | lo) & (kTicket - 1)) + 1;
  if (a.tickets != 0) {
    asm volatile("" : : "s"(lo), "s"(hi) : "memory");  // the count has arrived before the barrier
    __syncthreads();
    if (threadIdx.x == 0) {
      unsigned long long* s = (unsigned long long*)&a.steps[i];
      const uint64_t drawn = __hip_atomic_fetch_add(s, kTicket, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) / kTicket;
      if (drawn == (uint64_t)a.tickets - 1) __hip_atomic_store(s, t, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  return t;
}

// theta - (eta wd theta + step).  The hardware's square root and reciprocal are within
// one unit in the last place but take no subnormal operand: with tiny_v a v below 2^-96 is
// scaled up.  m may be subnormal, so it is divided before it is scaled.
// Error, in units of 2^-24 of the step: size 5 (eta, the correction, its reciprocal 2, the
// product), root 2.5, the square root 2, the denominator's sum and eps 1, a subnormal v left
// out 1/8, the reciprocal 2, two products 2: 14.6, below 2^-20 in all; the sum with the
// decay adds half a step of its own.
__device__ __forceinline__ float new_theta(const Rates& r, float theta, float m, float v, bool tiny_v) {
  const bool tiny = tiny_v && v < 0x1p-96f;
  float s = __builtin_amdgcn_sqrtf(tiny ? v * 0x1p64f : v);
  s *= tiny ? 0x1p-32f : 1.0f;
  const float q = m * __builtin_amdgcn_rcpf(__fmaf_rn(s, r.root, r.eps));
  return theta - __fmaf_rn(r.shrink, theta, r.size * q);
}

// A subnormal v taken as 0 lowers the denominator by less than 2^-63 root: 2^-27 of itself
// at most next to an eps of 2^-36 root (4.6e-10 where root is 32; eps is 1e-8 by default).
// The rule looks at the group and the step alone, not at where in a tile an element lies, so
// the result does not depend on how tensors are joined or split.
__device__ __forceinline__ bool tiny_v_matters(const Rates& r) { return r.eps < r.root * 0x1p-36f; }

template <typename G, typename W>
__global__ __launch_bounds__(kAdamWBlock) void k_adamw(const AdamWArgs a, const InnerGeom g) {
  const int i = a.learner[blockIdx.y];
  const Learner l = learner_of(a, i);
  const Spot s = spot(g, kAdamWTile);
  const int64_t row = (int64_t)i * a.stride + s.base;
  float* theta = a.theta + row;
  float* m = (float*)a.m + row;
  float* v = (float*)a.v + row;
  const G* grad = (const G*)a.grads + row;
  const int at = threadIdx.x * 4;
  const int n = (int)s.count - at;
  const bool full = s.count == kAdamWTile;
  float th[4], mm[4], vv[4];
  Raw4<G> gr;
  const auto load = [&](int n) {
    load4(theta + at, n, th);
    load4(m + at, n, mm);
    load4(v + at, n, vv);
    gr.load(grad + at, n);
  };
  if (full) load(4);
  else load(n);
  if (!takes_step(l.clip)) return;
  const Rates r = rates_of(a.group[s.group], l.clip, l.lr_scale, next_step(a, i, l));
  const bool tiny_v = tiny_v_matters(r);
  const auto finish = [&](auto fast, int n) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      mm[c] = new_m(r.b1, r.c1, mm[c], gr.value(c));
      vv[c] = new_v(r.b2, r.c2, vv[c], gr.value(c));
      th[c] = new_theta(r, th[c], mm[c], vv[c], !decltype(fast)::value && tiny_v);
    }
    store4(theta + at, n, th);
    store4(m + at, n, mm);
    store4(v + at, n, vv);
    if constexpr (!std::is_void_v<W>) store4((W*)a.working + row + at, n, th);
  };
  if (full && !tiny_v) finish(std::true_type(), 4);
  else finish(std::false_type(), n);
}

// --- coded moments -----------------------------------------------------------
constexpr uint32_t kGolden = 0x9E3779B9u;  // first 32 bits of the golden ratio's fraction
constexpr uint32_t kRootTwo = 0x6A09E667u;  // and of the root of two's

__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x = (x ^ (x >> 16)) * kGolden;
  x = (x ^ (x >> 15)) * kRootTwo;
  return x ^ (x >> 16);
}

struct Keys {
  uint32_t k1, k2;
};

// i + 64 * (e >> 32) names the learner and the 2^32 elements that e is among.
__device__ __forceinline__ Keys keys_of(uint64_t seed, uint64_t t, int learner, uint32_t e_high) {
  Keys k;
  k.k1 = mix(mix((uint32_t)seed + (uint32_t)t) + (uint32_t)learner + 64u * e_high);
  k.k2 = mix(k.k1 + (uint32_t)(seed >> 32) + (uint32_t)t);
  return k;
}

__device__ __forceinline__ uint32_t random_bits(const Keys& k, uint32_t e) {
  uint32_t x = e + k.k1;
  x = (x ^ (x >> 16)) * kGolden + k.k2;
  x = (x ^ (x >> 15)) * kRootTwo;
  return x ^ (x >> 16);
}

// A block's scale byte puts the exponent of its largest value at 2^7 (e4m3, which ends at
// 448) or 2^14 (e5m2, 57344), so that no value reaches the format's end, rounded up or not.
constexpr int kTopM = 7, kTopV = 14;
constexpr uint32_t kNaNs = 0x7F7F7F7Fu;  // four NaNs of either format

__device__ __forceinline__ uint32_t scale_byte(uint32_t largest, int top) {
  const int b = (int)(largest >> 23) - top;
  return b > 0 ? b : 0;
}

// 2^(127 - byte): at most 2^127, at least 2^-120
__device__ __forceinline__ float inverse_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// beta * 2^(byte - 127), exact
__device__ __forceinline__ double scaled(double beta, uint32_t byte) { return ldexp(beta, (int)byte - 127); }

// The hardware's stochastic conversions add a random word below the code's last bit (from
// its top 20 bits for e4m3, 21 for e5m2) and cut; the word here is 16 random bits and a
// half.  kByte: the byte of `word` that takes the code.
template <int kByte>
__device__ __forceinline__ void code_m(uint32_t& word, float y, uint32_t bits) {
  word = __builtin_amdgcn_cvt_sr_fp8_f32(y, (int)(bits << 16 | 0x8000u), (int)word, kByte);
}

template <int kByte>
__device__ __forceinline__ void code_v(uint32_t& word, float y, uint32_t bits) {
  word = __builtin_amdgcn_cvt_sr_bf8_f32(y, (int)((bits & 0xFFFF0000u) | 0x8000u), (int)word, kByte);
}

// Four codes of a word as floats.
__device__ __forceinline__ void decode_m(uint32_t w, float (&x)[4]) {
  const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
  x[0] = a[0], x[1] = a[1], x[2] = b[0], x[3] = b[1];
}

__device__ __forceinline__ void decode_v(uint32_t w, float (&x)[4]) {
  const auto a = __builtin_amdgcn_cvt_pk_f32_bf8(w, false), b = __builtin_amdgcn_cvt_pk_f32_bf8(w, true);
  x[0] = a[0], x[1] = a[1], x[2] = b[0], x[3] = b[1];
}

__device__ __forceinline__ uint32_t load_codes(const uint8_t* p, int n) {
  return n > 0 ? __builtin_nontemporal_load((const uint32_t*)p) : 0u;
}

__device__ __forceinline__ void store_codes(uint8_t* p, int n, uint32_t w) {
  if (n >= 4) {
    __builtin_nontemporal_store(w, (uint32_t*)p);
    return;
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    if (c < n) p[c] = (uint8_t)(w >> (8 * c));
  }
}

// The largest over the 16 lanes (one row of the data-parallel primitives) that hold a
// block of 64 elements.
__device__ __forceinline__ uint32_t block_largest(uint32_t x) {
  const auto step = [&](auto ctrl) {
    const uint32_t y = (uint32_t)__builtin_amdgcn_mov_dpp((int)x, decltype(ctrl)::value, 0xF, 0xF, true);
    x = x > y ? x : y;
  };
  step(std::integral_constant<int, 0xB1>());   // lanes 1 0 3 2 of each four
  step(std::integral_constant<int, 0x4E>());   // 2 3 0 1
  step(std::integral_constant<int, 0x141>());  // each eight mirrored
  step(std::integral_constant<int, 0x140>());  // each sixteen mirrored
  return x;
}

constexpr uint32_t kInfinity = 0x7F800000u;

__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// A magnitude for the block's maximum: 0 where it is not finite.
__device__ __forceinline__ uint32_t finite_magnitude(float x) { return magnitude(x) < kInfinity ? magnitude(x) : 0u; }

__device__ __forceinline__ uint32_t max4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return max(max(a, b), max(c, d));
}

template <typename G, typename W>
__global__ __launch_bounds__(kCodedBlock) void k_adamw_coded(const AdamWArgs a, const InnerGeom g) {
  const int i = a.learner[blockIdx.y];
  const Learner l = learner_of(a, i);
  const Spot s = spot(g, kCodedTile);
  const int64_t row = (int64_t)i * a.stride + s.base;
  float* theta = a.theta + row;
  uint8_t* m = (uint8_t*)a.m + row;
  uint8_t* v = (uint8_t*)a.v + row;
  uint8_t* ms = a.m_scale + row / kCodeBlock;
  uint8_t* vs = a.v_scale + row / kCodeBlock;
  const G* grad = (const G*)a.grads + row;
  constexpr int U = kCodedQuads;
  const int at = (threadIdx.x >> 6) * (256 * U) + (threadIdx.x & 63) * 4;  // quad j at + 256 j
  const bool full = s.count == kCodedTile;
  float th[U][4];
  Raw4<G> gr[U];
  uint32_t mw[U], vw[U], mb[U], vb[U];
  const auto load = [&](auto whole) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int e = at + 256 * j;
      const int n = decltype(whole)::value ? 4 : (int)s.count - e;
      load4(theta + e, n, th[j]);
      gr[j].load(grad + e, n);
      mw[j] = load_codes(m + e, n);
      vw[j] = load_codes(v + e, n);
      mb[j] = n > 0 ? ms[e / kCodeBlock] : 0;
      vb[j] = n > 0 ? vs[e / kCodeBlock] : 0;
    }
  };
  if (full) load(std::true_type());
  else load(std::false_type());
  if (!takes_step(l.clip)) return;
  const uint64_t t = next_step(a, i, l);
  const Rates r = rates_of(a.group[s.group], l.clip, l.lr_scale, t);
  const Keys first = keys_of(a.seed, t, i, (uint32_t)(s.base >> 32));
  const bool tiny_v = tiny_v_matters(r);
  const auto finish = [&](auto fast) {
    constexpr bool kFast = decltype(fast)::value;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int e = at + 256 * j;
      const int n = kFast ? 4 : (int)s.count - e;
      const uint32_t place = (uint32_t)s.base + e;
      Keys k = first;
      if (!kFast && place < (uint32_t)s.base)  // past a multiple of 2^32
        k = keys_of(a.seed, t, i, (uint32_t)(s.base >> 32) + 1);
      const double b1 = scaled(r.b1, mb[j]), b2 = scaled(r.b2, vb[j]);
      float mm[4], vv[4];
      decode_m(mw[j], mm);
      decode_v(vw[j], vv);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        mm[c] = new_m(b1, r.c1, mm[c], gr[j].value(c));
        vv[c] = new_v(b2, r.c2, vv[c], gr[j].value(c));
        th[j][c] = new_theta(r, th[j][c], mm[c], vv[c], !kFast && tiny_v);
        if (c >= n) mm[c] = vv[c] = 0.0f;  // not the tensor's: no part of the block's maximum
      }
      // every lane of a step takes part in its block's maximum
      uint32_t mtop = block_largest(max4(magnitude(mm[0]), magnitude(mm[1]), magnitude(mm[2]), magnitude(mm[3])));
      uint32_t vtop = block_largest(max4(magnitude(vv[0]), magnitude(vv[1]), magnitude(vv[2]), magnitude(vv[3])));
      uint32_t mbad = 0, vbad = 0;
      if (__any(max(mtop, vtop) >= kInfinity)) {  // some value is not finite: it becomes NaN, the maximum is the others'
        mtop = block_largest(max4(finite_magnitude(mm[0]), finite_magnitude(mm[1]), finite_magnitude(mm[2]),
                                  finite_magnitude(mm[3])));
        vtop = block_largest(max4(finite_magnitude(vv[0]), finite_magnitude(vv[1]), finite_magnitude(vv[2]),
                                  finite_magnitude(vv[3])));
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (magnitude(mm[c]) >= kInfinity) mbad |= 0xFFu << (8 * c);
          if (magnitude(vv[c]) >= kInfinity) vbad |= 0xFFu << (8 * c);
        }
      }
      const uint32_t mbyte = scale_byte(mtop, kTopM), vbyte = scale_byte(vtop, kTopV);
      const float mi = inverse_scale(mbyte), vi = inverse_scale(vbyte);
      uint32_t mcode = 0, vcode = 0;
      const uint32_t w0 = random_bits(k, place), w1 = random_bits(k, place + 1), w2 = random_bits(k, place + 2);
      const uint32_t w3 = random_bits(k, place + 3);
      code_m<0>(mcode, mm[0] * mi, w0), code_v<0>(vcode, vv[0] * vi, w0);
      code_m<1>(mcode, mm[1] * mi, w1), code_v<1>(vcode, vv[1] * vi, w1);
      code_m<2>(mcode, mm[2] * mi, w2), code_v<2>(vcode, vv[2] * vi, w2);
      code_m<3>(mcode, mm[3] * mi, w3), code_v<3>(vcode, vv[3] * vi, w3);
      if (__any(((vcode - 0x01010101u) & ~vcode & 0x80808080u) != 0)) {  // a byte is 0: not for a positive v
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if ((vcode >> (8 * c) & 0xFFu) == 0 && vv[c] > 0.0f) vcode |= 1u << (8 * c);
        }
      }
      store4(theta + e, n, th[j]);
      store_codes(m + e, n, (mcode & ~mbad) | (kNaNs & mbad));
      store_codes(v + e, n, (vcode & ~vbad) | (kNaNs & vbad));
      if (n > 0 && e % kCodeBlock == 0) {
        ms[e / kCodeBlock] = (uint8_t)mbyte;
        vs[e / kCodeBlock] = (uint8_t)vbyte;
      }
      if constexpr (!std::is_void_v<W>) store4((W*)a.working + row + e, n, th[j]);
    }
  };
  // a block past a multiple of 2^32 elements has two sets of keys: the general path's case
  if (full && !tiny_v && (uint32_t)s.base + kCodedTile > (uint32_t)s.base) finish(std::true_type());
  else finish(std::false_type());
}

__global__ __launch_bounds__(64) void k_adamw_advance(const AdamWArgs a) {
  if ((int)threadIdx.x >= a.n_present) return;
  const int i = a.learner[threadIdx.x];
  if (takes_step(clip_of(a, i))) a.steps[i] = (a.steps[i] & (int64_t)(kTicket - 1)) + 1;
}

template <typename G, typename W>
hipError_t launch_adamw_gw(const AdamWArgs& a, bool coded, const InnerGeom& g, hipStream_t s) {
  const dim3 grid(g.n_blocks, a.n_present);
  if (coded) {
    hipLaunchKernelGGL((k_adamw_coded<G, W>), grid, dim3(kCodedBlock), 0, s, a, g);
  } else {
    hipLaunchKernelGGL((k_adamw<G, W>), grid, dim3(kAdamWBlock), kAdamWLds, s, a, g);
  }
  return hipGetLastError();
}

template <typename G>
hipError_t launch_adamw_g(const AdamWArgs& a, int32_t working_type, bool coded, const InnerGeom& g, hipStream_t s) {
  switch (working_type) {
    case kBF16: return launch_adamw_gw<G, __bf16>(a, coded, g, s);
    case kF16: return launch_adamw_gw<G, _Float16>(a, coded, g, s);
    default: return launch_adamw_gw<G, void>(a, coded, g, s);
  }
}

}  // namespace

hipError_t launch_norm_partial(const NormArgs& a, int32_t grad_type, const InnerGeom& g, hipStream_t s) {
  const dim3 grid(g.n_blocks, a.n_present), block(kNormBlock);
  switch (grad_type) {
    case kBF16: hipLaunchKernelGGL(k_norm_partial<__bf16>, grid, block, 0, s, a, g); break;
    case kF16: hipLaunchKernelGGL(k_norm_partial<_Float16>, grid, block, 0, s, a, g); break;
    default: hipLaunchKernelGGL(k_norm_partial<float>, grid, block, 0, s, a, g); break;
  }
  return hipGetLastError();
}

hipError_t launch_norm_small(const NormArgs& a, int32_t grad_type, const InnerGeom& g, hipStream_t s) {
  const dim3 grid(a.n_present), block(kNormFinal);
  switch (grad_type) {
    case kBF16: hipLaunchKernelGGL(k_norm_small<__bf16>, grid, block, 0, s, a, g); break;
    case kF16: hipLaunchKernelGGL(k_norm_small<_Float16>, grid, block, 0, s, a, g); break;
    default: hipLaunchKernelGGL(k_norm_small<float>, grid, block, 0, s, a, g); break;
  }
  return hipGetLastError();
}

hipError_t launch_norm_final(const NormArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(k_norm_final, dim3(a.n_present), dim3(kNormFinal), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_adamw(const AdamWArgs& a, int32_t grad_type, int32_t working_type, bool coded, const InnerGeom& g,
                        hipStream_t s) {
  switch (grad_type) {
    case kBF16: return launch_adamw_g<__bf16>(a, working_type, coded, g, s);
    case kF16: return launch_adamw_g<_Float16>(a, working_type, coded, g, s);
    default: return launch_adamw_g<float>(a, working_type, coded, g, s);
  }
}

hipError_t launch_adamw_advance(const AdamWArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(k_adamw_advance, dim3(1), dim3(64), 0, s, a);
  return hipGetLastError();
}

}  // namespace dlc
