// Rows of full-vocabulary logits: 16-byte vectors of any element type, and the statistics of a softmax over their parts.
#pragma once
#include "common.hpp"

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kWide = 1024.f;          // |c max z| from which y is taken relative to the maximum itself
constexpr int kUnroll = 4;               // 16-byte vectors per lane and batch

__host__ __device__ constexpr int elem_bytes(int ET) { return ET == NS_FP32 ? 4 : 2; }
__host__ __device__ constexpr int per_vec(int ET) { return 16 / elem_bytes(ET); }

// 16 bytes at the element type's own alignment: rows of an odd vocabulary
// start anywhere, and the memory system takes such loads whole.
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));

template <int ET>
__device__ __forceinline__ float elem_of(uint32_t w, int e) {
  if (ET == NS_BF16) return e ? ns::bf16_hi(w) : ns::bf16_lo(w);
  return e ? ns::fp16_hi(w) : ns::fp16_lo(w);
}

template <int ET>
__device__ __forceinline__ void widen(u32x4 x, float (&v)[per_vec(ET)]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (ET == NS_FP32) v[i] = __uint_as_float(w[i]);
    else {
      v[2 * i] = elem_of<ET>(w[i], 0);
      v[2 * i + 1] = elem_of<ET>(w[i], 1);
    }
  }
}

template <int ET>
__device__ __forceinline__ u32x4 minus_inf() {
  const uint32_t w = ET == NS_BF16 ? 0xFF80FF80u : (ET == NS_FP16 ? 0xFC00FC00u : 0xFF800000u);
  return u32x4{w, w, w, w};
}

template <int ET>
__device__ __forceinline__ float one_elem(const void* z, size_t i) {
  if (ET == NS_FP32) return ((const float*)z)[i];
  const uint32_t w = ((const uint16_t*)z)[i];
  return elem_of<ET>(w, 0);
}

__device__ __forceinline__ float exp2_fast(float y) { return __builtin_amdgcn_exp2f(y); }

// Statistics of a part of a row: y = c (z - ref) - E.
struct Stat {
  float top, ref, E, S, W;
};

// b joined to a, both with some finite value or none (top = -inf, S = 0).
// A NaN or an infinite sum stays one.
__device__ __forceinline__ Stat join(const Stat& a, const Stat& b, float c) {
  const bool first = a.top >= b.top;
  Stat r = first ? a : b;
  const Stat o = first ? b : a;
  const float shift = c * (o.ref - r.ref) + (o.E - r.E);
  const float f = exp2_fast(shift);
  if (o.S == 0.f) return r;
  if (f > 0.f) {
    r.S += f * o.S;
    r.W += f * (o.W + o.S * shift);
  } else if (!(o.S < INFINITY)) {
    r.S = o.S;
  }
  return r;
}

// Takes a maximum into a wave's statistics, which are scaled anew where they have to be.
__device__ __forceinline__ void raise(Stat& st, float top, float c) {
  if (top > st.top) {                                      // uniform
    const bool had = st.top != -INFINITY;
    st.top = top;
    if (fabsf(top * c) < kWide) {
      const float E = rintf(top * c);
      if (!had || st.ref != 0.f || E > st.E + 4.f) {
        const float shift = had ? c * st.ref + (st.E - E) : 0.f;
        const float f = exp2_fast(shift);
        st.W = f > 0.f ? f * (st.W + st.S * shift) : 0.f;
        st.S *= f;
        st.ref = 0.f;
        st.E = E;
      }
    } else {
      const float shift = had ? c * (st.ref - top) + st.E : 0.f;
      const float f = exp2_fast(shift);
      st.W = f > 0.f ? f * (st.W + st.S * shift) : 0.f;
      st.S *= f;
      st.ref = top;
      st.E = 0.f;
    }
  }
}

// Adds a batch of a wave's vectors to its statistics; mx, lane_max and the
// result are the maxima of each vector, of the lane's and of the wave's.
template <int ET>
__device__ __forceinline__ float add_batch(const u32x4 (&x)[kUnroll], float c, Stat& st, float (&mx)[kUnroll],
                                           float& lane_max) {
  constexpr int EPV = per_vec(ET);
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    float v[EPV];
    widen<ET>(x[u], v);
    float m = v[0];
#pragma unroll
    for (int e = 1; e < EPV; ++e) m = fmaxf(m, v[e]);
    mx[u] = m;
  }
  lane_max = mx[0];
#pragma unroll
  for (int u = 1; u < kUnroll; ++u) lane_max = fmaxf(lane_max, mx[u]);
  const float top = ns::wave_max_f32(lane_max);
  raise(st, top, c);
  // A batch is summed by itself first: shorter chains of roundings.
  float S = 0.f, W = 0.f;
  const float E = st.E, ref = st.ref;
  if (ref == 0.f) {                                        // uniform
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      float v[EPV];
      widen<ET>(x[u], v);
#pragma unroll
      for (int e = 0; e < EPV; ++e) {
        const float y = fmaf(v[e], c, -E), p = exp2_fast(y);
        S += p;
        W = fmaf(p, fmaxf(y, -200.f), W);                  // 2^y is 0 for masked logits: no 0 * inf
      }
    }
  } else {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      float v[EPV];
      widen<ET>(x[u], v);
#pragma unroll
      for (int e = 0; e < EPV; ++e) {
        const float y = (v[e] - ref) * c, p = exp2_fast(y);
        S += p;
        W = fmaf(p, fmaxf(y, -200.f), W);
      }
    }
  }
  st.S += S;
  st.W += W;
  return top;
}

// Two results to a 16-bit type.  The compiler may round an fp16 product at once,
// without a float32 between: one rounding less, and nothing compares these bit
// for bit with a form that has both.
template <int ET>
__device__ __forceinline__ uint32_t narrow2(float a, float b) {
  if (ET == NS_BF16) {
    const __bf16 x = (__bf16)a, y = (__bf16)b;
    return (uint32_t)__builtin_bit_cast(uint16_t, x) | (uint32_t)__builtin_bit_cast(uint16_t, y) << 16;
  }
  const _Float16 x = (_Float16)a, y = (_Float16)b;
  return (uint32_t)__builtin_bit_cast(uint16_t, x) | (uint32_t)__builtin_bit_cast(uint16_t, y) << 16;
}

template <int ET>
__device__ __forceinline__ void put_elem(void* d, size_t i, float v) {
  if (ET == NS_FP32) ((float*)d)[i] = v;
  else ((uint16_t*)d)[i] = (uint16_t)narrow2<ET>(v, 0.f);
}

}  // namespace
