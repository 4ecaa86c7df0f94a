// Rows of 16- and 32-bit elements in registers, and outputs of a chosen type: what the kernels of quantised rows share.
#pragma once
#include "common.hpp"

namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));   // rows start at any element
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));


template <int ET>
__device__ __forceinline__ uint32_t load_bits(const void* x, size_t i) {
  return ET == NS_FP32 ? ((const uint32_t*)x)[i] : ((const uint16_t*)x)[i];
}

// Eight elements as they are stored: 16-bit types in one vector, float32 in two.
template <int ET>
struct Eight {
  u32x4 v[ET == NS_FP32 ? 2 : 1];

  // elements i .. i + 7 of a row, or i .. i + 3 and `step` on, zeros at or past
  // d.  `tail` is d rounded down to a vector's elements, `rest` what follows in
  // the row.  The loads stand under no condition that differs from lane to lane.
  __device__ __forceinline__ void load(const char* row, int i, int step, int tail, u32x4 rest) {
    constexpr int N = ET == NS_FP32 ? 2 : 1;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int at = i + n * step;
      u32x4 x = {0, 0, 0, 0};
      if (tail > 0) x = __builtin_nontemporal_load((const u32x4_any*)(row + (size_t)(at < tail ? at : 0) * (2 * N)));
      v[n] = at < tail ? x : (at == tail ? rest : u32x4{0, 0, 0, 0});
    }
  }
  // Elements tail .. d - 1, fewer than a vector's, and zeros.
  static __device__ __forceinline__ u32x4 rest_of(const char* row, int tail, int d) {
    u32x4 r = {0, 0, 0, 0};
    if (tail < d) {                                // uniform
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (ET == NS_FP32) {
          if (tail + c < d) r[c] = load_bits<ET>(row, tail + c);
        } else {
          if (tail + c * 2 < d) r[c] = load_bits<ET>(row, tail + c * 2);
          if (tail + c * 2 + 1 < d) r[c] |= load_bits<ET>(row, tail + c * 2 + 1) << 16;
        }
      }
    }
    return r;
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (ET == NS_FP32) return __uint_as_float(v[e >> 2][e & 3]);
    else if constexpr (ET == NS_BF16) return e & 1 ? ns::bf16_hi(v[0][e >> 1]) : ns::bf16_lo(v[0][e >> 1]);
    else return e & 1 ? ns::fp16_hi(v[0][e >> 1]) : ns::fp16_lo(v[0][e >> 1]);
  }
  // The largest magnitude as the type's own bits, which order like the values
  // with infinities and NaN on top; two at once for 16-bit types.
  __device__ __forceinline__ uint32_t top(uint32_t so_far) const {
    if constexpr (ET == NS_FP32) {
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t u = v[n][c] & 0x7FFFFFFFu;
          so_far = u > so_far ? u : so_far;
        }
      return so_far;
    } else {
      u16x2 m = __builtin_bit_cast(u16x2, so_far);
#pragma unroll
      for (int c = 0; c < 4; ++c) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v[0][c] & 0x7FFF7FFFu));
      return __builtin_bit_cast(uint32_t, m);
    }
  }
};

// Maximum over the 16 lanes of a row, in every lane.
__device__ __forceinline__ uint32_t row16_max_u32(uint32_t v) {
  uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, true);    // quad_perm 1 0 3 2
  v = o > v ? o : v;
  o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, true);             // quad_perm 2 3 0 1
  v = o > v ? o : v;
  o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, true);            // row_half_mirror
  v = o > v ? o : v;
  o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xf, 0xf, true);            // row_mirror
  return o > v ? o : v;
}

// A float32 value as it is: without this the compiler forms mixed-precision
// multiplies that round a product to fp16 at once.
__device__ __forceinline__ float as_float32(float v) {
  asm("" : "+v"(v));
  return v;
}

template <int OT>
__device__ __forceinline__ void store_out(void* out, size_t i, float v) {
  if (OT == NS_FP32) ((float*)out)[i] = v;
  else if (OT == NS_BF16) ((__bf16*)out)[i] = (__bf16)v;
  else ((_Float16*)out)[i] = (_Float16)as_float32(v);
}

template <int OT>
__device__ __forceinline__ uint32_t narrow2(float a, float b) {
  if (OT == NS_BF16) {
    const __bf16 x = (__bf16)a, y = (__bf16)b;
    return (uint32_t)__builtin_bit_cast(uint16_t, x) | (uint32_t)__builtin_bit_cast(uint16_t, y) << 16;
  }
  const _Float16 x = (_Float16)as_float32(a), y = (_Float16)as_float32(b);
  return (uint32_t)__builtin_bit_cast(uint16_t, x) | (uint32_t)__builtin_bit_cast(uint16_t, y) << 16;
}

// Eight consecutive outputs, n of them inside the row.
template <int OT>
__device__ __forceinline__ void store_eight(void* out, size_t i, const float (&v)[8], int n) {
  if (n >= 8) {
    if (OT == NS_FP32) {
      u32x4_any* d = (u32x4_any*)((float*)out + i);
      d[0] = u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
      d[1] = u32x4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])};
    } else {
      *(u32x4_any*)((uint16_t*)out + i) = u32x4{narrow2<OT>(v[0], v[1]), narrow2<OT>(v[2], v[3]),
                                                narrow2<OT>(v[4], v[5]), narrow2<OT>(v[6], v[7])};
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) store_out<OT>(out, i + e, v[e]);
  }
}

}  // namespace
