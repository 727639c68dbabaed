// Reductions over the lanes of a wave without LDS.
#pragma once

#include <hip/hip_runtime.h>

namespace dlc {
namespace {

// f of v and of the other half's value, for each group of L lanes whose halves hold one value
// each.  Within rows of 16 lanes the other half is read by the instruction that uses it;
// rows are exchanged by a swap of which both results are used.
template <int L>
__device__ __forceinline__ void exchange(int x, int& y, int& z) {
  y = z = x;
  if constexpr (L == 2) y = __builtin_amdgcn_mov_dpp(x, 0xB1, 0xF, 0xF, true);    // quad 1 0 3 2
  if constexpr (L == 4) y = __builtin_amdgcn_mov_dpp(x, 0x4E, 0xF, 0xF, true);    // quad 2 3 0 1
  if constexpr (L == 8) y = __builtin_amdgcn_mov_dpp(x, 0x141, 0xF, 0xF, true);   // half row mirrored
  if constexpr (L == 16) y = __builtin_amdgcn_mov_dpp(x, 0x140, 0xF, 0xF, true);  // row mirrored
  if constexpr (L == 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    y = (int)r[0];
    z = (int)r[1];
  }
  if constexpr (L == 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    y = (int)r[0];
    z = (int)r[1];
  }
}

template <int L, typename T, typename F>
__device__ __forceinline__ T with_other_half(T v, F&& f) {
  int y[sizeof(T) / 4], z[sizeof(T) / 4], x[sizeof(T) / 4];
  __builtin_memcpy(x, &v, sizeof(T));
#pragma unroll
  for (int k = 0; k < (int)sizeof(T) / 4; ++k) exchange<L>(x[k], y[k], z[k]);
  T p, q;
  __builtin_memcpy(&p, z, sizeof(T));
  __builtin_memcpy(&q, y, sizeof(T));
  return f(p, q);
}

template <int L, typename T, typename F>
__device__ __forceinline__ T reduce(T v, F&& f) {
  if constexpr (L >= 2) v = with_other_half<2>(v, f);
  if constexpr (L >= 4) v = with_other_half<4>(v, f);
  if constexpr (L >= 8) v = with_other_half<8>(v, f);
  if constexpr (L >= 16) v = with_other_half<16>(v, f);
  if constexpr (L >= 32) v = with_other_half<32>(v, f);
  if constexpr (L >= 64) v = with_other_half<64>(v, f);
  return v;
}

}  // namespace
}  // namespace dlc
