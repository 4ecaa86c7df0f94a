// Sorted lists of 64 keys in a wave, one a lane, the largest in lane 0.
#pragma once
#include "common.hpp"

namespace {

template <int CTRL>
__device__ __forceinline__ uint64_t dpp_u64(uint64_t v) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, 0xf, 0xf, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, 0xf, 0xf, true);
  return ((uint64_t)hi << 32) | lo;
}

// The value of lane ^ M; within rows of 16 lanes by lane moves, without LDS's latency.
template <int M>
__device__ __forceinline__ uint64_t lane_xor_u64(uint64_t v) {
  if constexpr (M == 1) return dpp_u64<0xB1>(v);           // quad_perm 1 0 3 2
  else if constexpr (M == 2) return dpp_u64<0x4E>(v);      // quad_perm 2 3 0 1
  else if constexpr (M == 4) return dpp_u64<0x1B>(dpp_u64<0x141>(v));   // row_half_mirror, quad_perm 3 2 1 0
  else if constexpr (M == 8) return dpp_u64<0x128>(v);     // row_ror:8
  else return ns::shfl_xor_u64(v, M);
}

template <int M>
__device__ __forceinline__ uint64_t exchange(uint64_t x, int lane) {
  const uint64_t o = lane_xor_u64<M>(x);
  return ((lane & M) == 0) == (x > o) ? x : o;
}

// The 64 largest of two sorted lists, one key a lane: a holds one in falling
// order, b the other in rising order; the larger of each pair is a bitonic
// sequence, which six exchanges sort.
__device__ __forceinline__ uint64_t merge_lists(uint64_t a, uint64_t b, int lane) {
  uint64_t x = a > b ? a : b;
  x = exchange<32>(x, lane);
  x = exchange<16>(x, lane);
  x = exchange<8>(x, lane);
  x = exchange<4>(x, lane);
  x = exchange<2>(x, lane);
  return exchange<1>(x, lane);
}

// The value of lane ^ (2 M - 1).
template <int M>
__device__ __forceinline__ uint64_t lane_mirror_u64(uint64_t v) {
  if constexpr (M == 1) return dpp_u64<0xB1>(v);           // quad_perm 1 0 3 2
  else if constexpr (M == 2) return dpp_u64<0x1B>(v);      // quad_perm 3 2 1 0
  else if constexpr (M == 4) return dpp_u64<0x141>(v);     // row_half_mirror
  else if constexpr (M == 8) return dpp_u64<0x140>(v);     // row_mirror
  else return ns::shfl_xor_u64(v, 2 * M - 1);
}

// Two sorted runs of M lanes, side by side, to one of 2 M.
template <int M>
__device__ __forceinline__ uint64_t join_runs(uint64_t x, int lane) {
  const uint64_t o = lane_mirror_u64<M>(x);
  x = ((lane & M) == 0) == (x > o) ? x : o;
  if constexpr (M >= 32) x = exchange<16>(x, lane);
  if constexpr (M >= 16) x = exchange<8>(x, lane);
  if constexpr (M >= 8) x = exchange<4>(x, lane);
  if constexpr (M >= 4) x = exchange<2>(x, lane);
  if constexpr (M >= 2) x = exchange<1>(x, lane);
  return x;
}

// 64 keys, one a lane, in falling order.
__device__ __forceinline__ uint64_t sort_list(uint64_t x, int lane) {
  x = join_runs<1>(x, lane);
  x = join_runs<2>(x, lane);
  x = join_runs<4>(x, lane);
  x = join_runs<8>(x, lane);
  x = join_runs<16>(x, lane);
  return join_runs<32>(x, lane);
}

}  // namespace
