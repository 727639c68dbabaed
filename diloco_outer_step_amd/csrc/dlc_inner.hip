// gfx950 kernels of the learner's inner step: the global gradient norm with its
// clipping factor, and AdamW with 32-bit or 8-bit coded moments, over all tensors
// of all present learners.
//
//   k_norm_partial  sum of squares of a block's gradients, fp64
//   k_norm_final    the blocks' sums in a fixed order -> norm and gradient scale
//   k_adamw         one pass over theta, the moments and the gradients
//   k_adamw_advance the learners' step counts
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
typedef unsigned int vu2 __attribute__((ext_vector_type(2)));

// Block -> (range, first and one past last element of the row).
struct RowSpan {
  int range;
  int64_t begin, end;
};

__device__ __forceinline__ RowSpan row_span(const InnerGeom& g) {
  const uint32_t b = blockIdx.x;
  int lo = 0, hi = g.n_ranges - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (g.r[mid].block_first <= b) lo = mid; else hi = mid - 1;
  }
  const InnerRange r = g.r[lo];
  RowSpan s;
  s.range = lo;
  const int64_t per_block = (int64_t)g.tiles_per_block * kInnerTile;
  const int64_t first = (int64_t)(b - r.block_first) * per_block;
  const int64_t last = first + per_block < (int64_t)r.count ? first + per_block : (int64_t)r.count;
  s.begin = (int64_t)r.lo64 * 64 + first;
  s.end = (int64_t)r.lo64 * 64 + last;
  return s;
}

// Four elements at p, the first n of them valid (n may be <= 0 or >= 4); others read as 0.
__device__ __forceinline__ void load4(const float* p, int64_t n, float (&x)[4]) {
  if (n >= 4) {
    const vf4 q = __builtin_nontemporal_load((const vf4*)p);
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] = q[c];
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] = c < n ? p[c] : 0.0f;
  }
}

template <typename T>
__device__ __forceinline__ void load4(const T* p, int64_t n, float (&x)[4]) {
  typedef T v4 __attribute__((ext_vector_type(4)));
  if (n >= 4) {
    const v4 q = __builtin_nontemporal_load((const v4*)p);
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] = (float)q[c];
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] = c < n ? (float)p[c] : 0.0f;
  }
}

template <typename T>
__device__ __forceinline__ void store4(T* p, int64_t n, const float (&x)[4]) {
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

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
  return v;
}

// The block's sum of v, in thread 0.
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double red[kInnerBlock / 64];
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kInnerBlock / 64; ++w) s += red[w];
  return s;
}

template <typename G>
__global__ __launch_bounds__(kInnerBlock) void k_norm_partial(const NormArgs a, const InnerGeom g) {
  const RowSpan sp = row_span(g);
  const G* row = (const G*)a.grads + (int64_t)a.learner[blockIdx.y] * a.stride;
  double s = 0.0;
  for (int64_t e = sp.begin + 4 * threadIdx.x; e < sp.end; e += 4 * kInnerBlock) {
    float x[4];
    load4(row + e, sp.end - e, x);
#pragma unroll
    for (int c = 0; c < 4; ++c) s = __fma_rn((double)x[c], (double)x[c], s);
  }
  s = block_sum(s);
  if (threadIdx.x == 0) a.part[(size_t)(g.slot_base + blockIdx.x) * a.n_present + blockIdx.y] = s;
}

__global__ __launch_bounds__(kInnerBlock) void k_norm_final(const NormArgs a) {
  double s = 0.0;
  for (int b = threadIdx.x; b < a.n_slots; b += kInnerBlock) s += a.part[(size_t)b * a.n_present + blockIdx.x];
  s = block_sum(s);
  if (threadIdx.x != 0) return;
  const int i = a.learner[blockIdx.x];
  const double n = a.unscale * sqrt(s);
  double scale = a.unscale;
  if (n > a.max_norm) scale = a.unscale * (a.max_norm / n);
  if (!__builtin_isfinite(n)) scale = 0.0;
  a.norm[i] = n;
  a.grad_scale[i] = scale;
}

// ---------------------------------------------------------------------------
// AdamW
// ---------------------------------------------------------------------------
__device__ __forceinline__ double power(double b, uint64_t t) {
  double p = 1.0;
  for (; t != 0; t >>= 1) {
    if (t & 1) p *= b;
    b *= b;
  }
  return p;
}

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
  r.size = (float)(eta / (1.0 - power(q.beta1, t)));
  r.root = (float)(1.0 / sqrt(1.0 - power(q.beta2, t)));
  r.eps = (float)q.eps;
  return r;
}

// With decimal betas the exact sums lie on fp32 rounding ties about once in a hundred
// elements (0.8 m + 0.2 g = (4 m + g) / 5), which the last bit in fp64 then decides: each
// product is rounded on its own, as any fp64 evaluation of the formula does.
__device__ __forceinline__ float new_m(double b1, double c1, double m, double grad) {
#ifdef X_FMA
  return (float)__fma_rn(b1, m, c1 * grad);
#else
  return (float)(b1 * m + c1 * grad);
#endif
}

__device__ __forceinline__ float new_v(double b2, double c2, double v, double grad) {
#ifdef X_FMA
  return (float)__fma_rn(b2, v, c2 * grad * grad);
#else
  return (float)(b2 * v + c2 * grad * grad);
#endif
}

// theta - (eta wd theta + step).  The hardware's square root and reciprocal are within
// one unit in the last place but take no subnormal operand: a tiny v is scaled up (eps,
// and with it the denominator, is a normal number).  m may be subnormal, so it is
// divided before it is scaled.
__device__ __forceinline__ float new_theta(const Rates& r, float theta, float m, float v) {
  const bool tiny = v < 0x1p-96f;
  const float s = __builtin_amdgcn_sqrtf(tiny ? v * 0x1p64f : v) * (tiny ? 0x1p-32f : 1.0f);
  const float q = m * __builtin_amdgcn_rcpf(__fmaf_rn(s, r.root, r.eps));
  return theta - __fmaf_rn(r.shrink, theta, r.size * q);
}

template <typename G, typename W>
__global__ __launch_bounds__(kInnerBlock) void k_adamw(const AdamWArgs a, const InnerGeom g) {
  const RowSpan sp = row_span(g);
  const int i = a.learner[blockIdx.y];
  const double clip = clip_of(a, i);
  if (!takes_step(clip)) return;
  const Rates r = rates_of(a.group[g.group[sp.range]], clip, a.lr_scale != nullptr ? a.lr_scale[i] : 1.0,
                           (uint64_t)a.steps[i] + 1);
  const int64_t row = (int64_t)i * a.stride;
  float* theta = a.theta + row;
  float* m = (float*)a.m + row;
  float* v = (float*)a.v + row;
  const G* grad = (const G*)a.grads + row;
  for (int64_t e = sp.begin + 4 * threadIdx.x; e < sp.end; e += 4 * kInnerBlock) {
    const int64_t n = sp.end - e;
    float th[4], gr[4], mm[4], vv[4];
    load4(theta + e, n, th);
    load4(grad + e, n, gr);
    load4(m + e, n, mm);
    load4(v + e, n, vv);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      mm[c] = new_m(r.b1, r.c1, mm[c], gr[c]);
      vv[c] = new_v(r.b2, r.c2, vv[c], gr[c]);
      th[c] = new_theta(r, th[c], mm[c], vv[c]);
    }
    store4(theta + e, n, th);
    store4(m + e, n, mm);
    store4(v + e, n, vv);
    if constexpr (!std::is_void_v<W>) store4((W*)a.working + row + e, n, th);
  }
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
constexpr float kLeastV = 0x1p-16f;  // the smallest e5m2 number

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

__device__ __forceinline__ uint32_t load_codes(const uint8_t* p, int64_t n) {
  if (n >= 4) return __builtin_nontemporal_load((const uint32_t*)p);
  uint32_t w = 0;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    if (c < n) w |= (uint32_t)p[c] << (8 * c);
  }
  return w;
}

__device__ __forceinline__ void store_codes(uint8_t* p, int64_t n, uint32_t w) {
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
__global__ __launch_bounds__(kInnerBlock) void k_adamw_coded(const AdamWArgs a, const InnerGeom g) {
  const RowSpan sp = row_span(g);
  const int i = a.learner[blockIdx.y];
  const double clip = clip_of(a, i);
  if (!takes_step(clip)) return;
  const uint64_t t = (uint64_t)a.steps[i] + 1;
  const Rates r =
      rates_of(a.group[g.group[sp.range]], clip, a.lr_scale != nullptr ? a.lr_scale[i] : 1.0, t);
  const int64_t row = (int64_t)i * a.stride;
  float* theta = a.theta + row;
  uint8_t* m = (uint8_t*)a.m + row;
  uint8_t* v = (uint8_t*)a.v + row;
  uint8_t* ms = a.m_scale + row / kCodeBlock;
  uint8_t* vs = a.v_scale + row / kCodeBlock;
  const G* grad = (const G*)a.grads + row;
  const Keys first = keys_of(a.seed, t, i, (uint32_t)(sp.begin >> 32));
  // every lane takes part in its block's maximum, so the trip count is the block's
  for (int64_t base = sp.begin; base < sp.end; base += 4 * kInnerBlock) {
    const int64_t e = base + 4 * threadIdx.x;
    const int64_t n = sp.end - e;
    const bool any = n > 0;
    float th[4], gr[4], mm[4], vv[4];
    load4(theta + e, n, th);
    load4(grad + e, n, gr);
    decode_m(load_codes(m + e, n), mm);
    decode_v(load_codes(v + e, n), vv);
    const double b1 = scaled(r.b1, any ? ms[e / kCodeBlock] : 0);
    const double b2 = scaled(r.b2, any ? vs[e / kCodeBlock] : 0);
    Keys k = first;
    if ((uint32_t)e < (uint32_t)sp.begin) k = keys_of(a.seed, t, i, (uint32_t)(e >> 32));  // past a multiple of 2^32
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      mm[c] = new_m(b1, r.c1, mm[c], gr[c]);
      vv[c] = new_v(b2, r.c2, vv[c], gr[c]);
      th[c] = new_theta(r, th[c], mm[c], vv[c]);
      if (c >= n) mm[c] = vv[c] = 0.0f;  // not the tensor's: no part of the block's maximum
    }
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
    const uint32_t mb = scale_byte(mtop, kTopM), vb = scale_byte(vtop, kTopV);
    const float mi = inverse_scale(mb), vi = inverse_scale(vb);
    float vy[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float y = vv[c] * vi;
      vy[c] = vv[c] > 0.0f && y < kLeastV ? kLeastV : y;  // a positive v is not coded as 0
    }
    uint32_t mw = 0, vw = 0;
    const uint32_t w0 = random_bits(k, (uint32_t)e), w1 = random_bits(k, (uint32_t)e + 1);
    const uint32_t w2 = random_bits(k, (uint32_t)e + 2), w3 = random_bits(k, (uint32_t)e + 3);
    code_m<0>(mw, mm[0] * mi, w0), code_v<0>(vw, vy[0], w0);
    code_m<1>(mw, mm[1] * mi, w1), code_v<1>(vw, vy[1], w1);
    code_m<2>(mw, mm[2] * mi, w2), code_v<2>(vw, vy[2], w2);
    code_m<3>(mw, mm[3] * mi, w3), code_v<3>(vw, vy[3], w3);
    store4(theta + e, n, th);
    store_codes(m + e, n, (mw & ~mbad) | (kNaNs & mbad));
    store_codes(v + e, n, (vw & ~vbad) | (kNaNs & vbad));
    if (any && e % kCodeBlock == 0) {
      ms[e / kCodeBlock] = (uint8_t)mb;
      vs[e / kCodeBlock] = (uint8_t)vb;
    }
    if constexpr (!std::is_void_v<W>) store4((W*)a.working + row + e, n, th);
  }
}

__global__ __launch_bounds__(64) void k_adamw_advance(const AdamWArgs a) {
  if ((int)threadIdx.x >= a.n_present) return;
  const int i = a.learner[threadIdx.x];
  if (takes_step(clip_of(a, i))) a.steps[i] += 1;
}

template <typename G, typename W>
hipError_t launch_adamw_gw(const AdamWArgs& a, bool coded, const InnerGeom& g, hipStream_t s) {
  const dim3 grid(g.n_blocks, a.n_present), block(kInnerBlock);
  if (coded) {
    hipLaunchKernelGGL((k_adamw_coded<G, W>), grid, block, 0, s, a, g);
  } else {
    hipLaunchKernelGGL((k_adamw<G, W>), grid, block, 0, s, a, g);
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
  const dim3 grid(g.n_blocks, a.n_present), block(kInnerBlock);
  switch (grad_type) {
    case kBF16: hipLaunchKernelGGL(k_norm_partial<__bf16>, grid, block, 0, s, a, g); break;
    case kF16: hipLaunchKernelGGL(k_norm_partial<_Float16>, grid, block, 0, s, a, g); break;
    default: hipLaunchKernelGGL(k_norm_partial<float>, grid, block, 0, s, a, g); break;
  }
  return hipGetLastError();
}

hipError_t launch_norm_final(const NormArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(k_norm_final, dim3(a.n_present), dim3(kInnerBlock), 0, s, a);
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
