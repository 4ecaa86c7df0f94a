// Clipped policy loss with a KL term and an entropy bonus over rows of
// full-vocabulary logits, with its gradient.
//
// For row i with token a, z' = t z (t the inverse temperature) and
// logp_j = z'_j - lse(z'):
//     r = exp(logp_a - old),   s = min(r A, clip(r, 1 - e_lo, 1 + e_hi) A),
//     delta = ref - logp_a,    kl = exp(delta) - delta - 1,   H = -sum_j p_j logp_j,
//     loss_i = w (-s + beta kl - c_H H).
// The gradient of the sum of all rows' losses, times g_loss:
//     g = w (-r A [r A <= clip(r) A] + beta (1 - exp(delta))),
//     dz_j = g_loss t (g ([j = a] - p_j) + w c_H p_j (logp_j + H)).
// With y_j = log2(e) z'_j - E, S = sum 2^y_j and W = sum 2^y_j y_j the second
// line is 2^y_j (A + B y_j) off the token.  logp_a, its distances from old and
// ref and what follows from them are taken in float64, so that a ratio is as exact
// as S and products past float32's range are infinite, not NaN.
#include "common.hpp"
#include "logits.hpp"

namespace {

struct Args {
  const void* z;
  int64_t ld;
  int L, V;
  float t, c, eps;             // inverse temperature, times log2(e), and what rounding took from c, relatively
  const int32_t* tokens;       // [L]
  const float* old;            // [L]
  const float* ref;            // [L] or NULL
  const float* advantage;      // [L]
  const float* weight;         // [L] or NULL (ones)
  float eps_low, eps_high, beta, c_ent;
  float* logprob;              // [L]
  float* kl;                   // [L] or NULL
  float* entropy;              // [L] or NULL
  const float* g_loss;         // [1] or NULL (one)
  void* dz;                    // or NULL
  int64_t ld_d;
  double* row_loss;            // [L]
  int S;                       // parts of a row, a power of two
  Stat* stat;                  // [L][S], where S > 1
  struct Kept* kept;           // [L], likewise
};

// A log-probability below this is that of a probability 0 in float32 (under 2^-150, half the smallest number): no
// sampler draws such a token.  One that an older policy drew, now that unlikely, would have a ratio of 0 and a KL term
// past float32's range, which would be the whole batch's loss.  Above it a token counts as it is, however unlikely.
constexpr double kUnseen = -104.0;
constexpr double kLn2d = 0.69314718055994530942;

// What a row's gradient needs: 2^y (A + B y), and the token's element by itself, where terms past float32's range may
// cancel.
struct Slope {
  float ref, E, A, B, token;
};

// Slopes past 2^100 are taken 2^k smaller and 2^y 2^k larger, so that a slope past float32's range makes infinities of
// the elements that are past it, and zeros of masked logits.
constexpr float kLargeSlope = 0x1p100f;

// Whether a row is looked at at all.
__device__ __forceinline__ bool taken(const Args& a, size_t row, int& tok, float& w) {
  tok = a.tokens[row];
  w = a.weight ? a.weight[row] : 1.f;
  return tok >= 0 && tok < a.V && w != 0.f;
}

__device__ __forceinline__ void put_nothing(const Args& a, size_t row) {
  a.logprob[row] = 0.f;
  if (a.kl) a.kl[row] = 0.f;
  if (a.entropy) a.entropy[row] = 0.f;
  a.row_loss[row] = 0.0;
}

// e^x of a finite x as 2^n and float32's exponential of the rest, n as far as a double's exponent goes.  From e^400 on
// it stays: a product with it is past float32's range then, whatever its other factors, and still finite.
__device__ __forceinline__ double exp_of(double x) {
  const double y = x * 1.4426950408889634, n = rint(y);
  const int e = (int)fmin(fmax(n, -577.0), 577.0);
  const float rest = (float)(y - n);                       // NaN if x is; of a y past 2^52 what the product left, of no use
  return ldexp((double)exp2_fast(fabsf(rest) > 1.f ? 0.f : rest), e);
}

// A value whose distances from others are finite.
__device__ __forceinline__ double no_infinity(float v) { return fabsf(v) == INFINITY ? copysign(1e300, (double)v) : (double)v; }

// e^x - 1 and e^x - 1 - x, each by itself: neither is left of the other's digits where |x| is large.  Near 0 the second
// by its series, whose terms past the tenth are below a step of the first.  Without a branch: a row waits for this.
struct Past {
  double one, line;
};

__device__ __forceinline__ Past exp_past(double x) {
  const double e = exp_of(x) - 1.0;
  const float f = (float)x;
  float r = 1.f / 3628800;
  r = fmaf(r, f, 1.f / 362880);
  r = fmaf(r, f, 1.f / 40320);
  r = fmaf(r, f, 1.f / 5040);
  r = fmaf(r, f, 1.f / 720);
  r = fmaf(r, f, 1.f / 120);
  r = fmaf(r, f, 1.f / 24);
  r = fmaf(r, f, 1.f / 6);
  r = fmaf(r, f, 0.5f);
  const double line = (double)(r * f * f);
  const bool near = fabsf(f) <= 0.5f;
  return {near ? x + line : e, near ? line : (x > 400.0 ? e : e - x)};
}

// What a row needs beside its logits, asked for before they are read.
struct Given {
  float old, ref, advantage, w, g_loss;
  Given() = default;
  __device__ __forceinline__ Given(const Args& a, size_t row, float weight)
      : old(a.old[row]), ref(a.ref ? a.ref[row] : 0.f), advantage(a.advantage[row]), w(weight),
        g_loss(a.g_loss ? *a.g_loss : 1.f) {}
};

// The same of a row in parts, with its token (-1 of a row that is not taken) and that token's logit.  The blocks that end
// the rows and those that take the gradient run at once: they read what a row was given here, so that outputs may
// replace inputs.
struct Kept {
  Given given;
  float ztok;
  int tok;
};

// A row's outputs and slope from its statistics and its token's logit.
__device__ __forceinline__ Slope finish(const Args& a, size_t row, const Stat& s, float ztok, const Given& v, bool writes,
                                        double* row_loss = nullptr) {
  const bool bad = !(s.S < INFINITY) || s.top == INFINITY, none = s.S == 0.f;
  const float nan = __uint_as_float(0x7FC00000u);
  Slope r{s.ref, s.E, 0.f, 0.f, 0.f};
  float logp = nan, kl = 0.f, H = nan;
  double loss = 0.0;
  if (bad) {
    r.A = r.B = r.token = kl = nan;
    loss = nan;
  } else if (none) {
    logp = -INFINITY;
    H = 0.f;
  } else {
    // log2 of S by its mantissa's, in [1/sqrt 2, sqrt 2], which is near 0 where S is
    // near a power of two.  c (1 + eps) is what c stands for; the sum's large terms
    // have c z close to E.
    float c = a.c, eps = a.eps, eps_low = a.eps_low, eps_high = a.eps_high, beta = a.beta, c_ent = a.c_ent;
    // widened here, not for all of a block's rows in registers
    asm volatile("" : "+s"(c), "+s"(eps), "+s"(eps_low), "+s"(eps_high), "+s"(beta), "+s"(c_ent));
    int e;
    float m = frexpf(s.S, &e);
    if (m < 0.70710678f) m *= 2.f, --e;
    const double l0 = (double)e + (double)log2f(m), l = l0 + (double)eps * s.E;
    const double y = ((double)ztok - s.ref) * ((double)c * (1.0 + (double)eps)) - s.E;
    const double lp = kLn2d * (y - l);
    logp = (float)lp;
    H = fmaxf((float)(kLn2d * (l0 - (double)(s.W / s.S))), 0.f);
    if (lp > kUnseen) {
      // float64: a ratio of e^88 is past float32, and no advantage times that is still 0
      const double ratio = exp_of(lp - no_infinity(v.old)), adv = (double)v.advantage;
      const double lo = 1.0 - (double)eps_low, hi = 1.0 + (double)eps_high;
      const double held = ratio < lo ? lo : (ratio > hi ? hi : ratio), gain = ratio * adv, most = held * adv;
      const bool clipped = gain > most;                    // not where one of them is NaN
      double g = clipped ? 0.0 : -gain;
      loss = clipped ? -most : -gain;
      if (a.ref) {
        const Past past = exp_past(no_infinity(v.ref) - lp);
        kl = (float)past.line;
        if (beta != 0.f) {
          loss += (double)beta * past.line;
          g -= (double)beta * past.one;
        }
      }
      loss = (double)v.w * (loss - (double)c_ent * H);
      const double up = (double)v.g_loss * a.t * v.w, over = up * (double)(1.f / s.S);
      const float p = exp2_fast((float)(y - l));           // the token's
      r.token = (float)(up * (g * fmaxf(1.f - p, 0.f) + (double)(c_ent * p) * (lp + H)));
      // every y of the row and H have c as it was rounded, and so has l0
      const double A = over * ((double)c_ent * (H - kLn2d * l0) - g), B = over * c_ent * kLn2d;
      r.A = (float)A;
      r.B = (float)B;
      if (fabsf(r.A) > kLargeSlope) {
        int k;
        (void)frexp(A * (double)(1.f / kLargeSlope), &k);  // 0 of infinities
        const double b = ldexp(B, -k);
        r.E -= (float)k;
        r.A = (float)(ldexp(A, -k) - b * k);
        r.B = (float)b;
      }
    }
  }
  if (writes) {
    a.logprob[row] = logp;
    if (a.kl) a.kl[row] = kl;
    if (a.entropy) a.entropy[row] = H;
    if (!row_loss) a.row_loss[row] = loss;
  }
  if (row_loss) *row_loss = loss;
  return r;
}

// The gradient of one element.  Where ref is not 0, E is -k of a large slope, else 0.
__device__ __forceinline__ float slope_at(const Slope& s, float c, float z) {
  const float y = s.ref == 0.f ? fmaf(z, c, -s.E) : (z - s.ref) * c - s.E;
  return exp2_fast(y) * fmaf(s.B, fmaxf(y, -200.f), s.A);
}

template <int ET>
__device__ __forceinline__ u32x4 narrow(const float (&v)[per_vec(ET)]) {
  if constexpr (ET == NS_FP32) {
    return u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
  } else {
    return u32x4{narrow2<ET>(v[0], v[1]), narrow2<ET>(v[2], v[3]), narrow2<ET>(v[4], v[5]), narrow2<ET>(v[6], v[7])};
  }
}

// The gradient of a vector.  B is 0 where there is no entropy term: a usual row
// does without a third of the instructions, at a uniform branch a vector.
template <int ET>
__device__ __forceinline__ u32x4 slope_of(const Slope& s, float c, bool usual, u32x4 z) {
  float v[per_vec(ET)];
  widen<ET>(z, v);
  if (usual) {
#pragma unroll
    for (int e = 0; e < per_vec(ET); ++e) v[e] = exp2_fast(fmaf(v[e], c, -s.E)) * s.A;
  } else {
#pragma unroll
    for (int e = 0; e < per_vec(ET); ++e) v[e] = slope_at(s, c, v[e]);
  }
  return narrow<ET>(v);
}
__device__ __forceinline__ bool is_usual(const Slope& s) {
  return __builtin_amdgcn_readfirstlane((int)(s.ref == 0.f && s.B == 0.f)) != 0;
}

// Statistics of fewer elements than a vector's, one a lane.
__device__ __forceinline__ Stat stat_of_lanes(float v, float c) {
  Stat s{-INFINITY, 0.f, 0.f, 0.f, 0.f};
  const float top = ns::wave_max_f32(v);
  if (top != -INFINITY) {
    const float cm = top * c;
    s.top = top;
    s.E = fabsf(cm) < kWide ? rintf(cm) : 0.f;
    s.ref = fabsf(cm) < kWide ? 0.f : top;
  }
  const float y = s.ref == 0.f ? fmaf(v, c, -s.E) : (v - s.ref) * c;
  s.S = exp2_fast(y);
  s.W = s.S * fmaxf(y, -200.f);
  s.S = ns::wave_sum_f32(s.S);
  s.W = ns::wave_sum_f32(s.W);
  return s;
}

// A row as a buffer: its whole vectors, at any address that its elements may have.
// Vectors past the last are read as zeros and not written, without a question.
struct Row {
  __amdgpu_buffer_rsrc_t r;
  __device__ __forceinline__ Row(const void* p, size_t row, int64_t ld, int esz, int nvec)
      : r(__builtin_amdgcn_make_buffer_rsrc((char*)p + row * (size_t)ld * esz, 0, nvec * 16, 0x00027000)) {}
  __device__ __forceinline__ u32x4 get(uint32_t at) const {   // read once
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 2));
  }
  __device__ __forceinline__ void put(uint32_t at, u32x4 v) const { __builtin_amdgcn_raw_buffer_store_b128(v, r, at, 0, 2); }
};

// Adds a vector to a wave's sums.
template <int ET>
__device__ __forceinline__ void add_vector(u32x4 x, float c, Stat& st) {
  constexpr int EPV = per_vec(ET);
  float v[EPV], S = 0.f, W = 0.f;
  widen<ET>(x, v);
  if (st.ref == 0.f) {                                     // uniform
#pragma unroll
    for (int e = 0; e < EPV; ++e) {
      const float y = fmaf(v[e], c, -st.E), p = exp2_fast(y);
      S += p;
      W = fmaf(p, fmaxf(y, -200.f), W);                    // 2^y is 0 for masked logits: no 0 * inf
    }
  } else {
#pragma unroll
    for (int e = 0; e < EPV; ++e) {
      const float y = (v[e] - st.ref) * c, p = exp2_fast(y);
      S += p;
      W = fmaf(p, fmaxf(y, -200.f), W);
    }
  }
  st.S += S;
  st.W += W;
}

// The largest element of many vectors, two 16-bit elements an instruction.
// bfloat16 compares as signed integers do where some element is positive; where
// all are negative the order is reversed.  NaN is found by the sums.
template <int ET>
struct Top {
  typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
  typedef short i16x2 __attribute__((ext_vector_type(2)));
  float f = -INFINITY;
  f16x2 h = {(_Float16)-INFINITY, (_Float16)-INFINITY};
  i16x2 hi = {(short)0x8000, (short)0x8000}, lo = {0x7FFF, 0x7FFF};
  __device__ __forceinline__ void add(u32x4 x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (ET == NS_FP32) {
        f = fmaxf(f, __uint_as_float(x[i]));
      } else if constexpr (ET == NS_FP16) {
        h = __builtin_elementwise_max(h, __builtin_bit_cast(f16x2, x[i]));
      } else {
        hi = __builtin_elementwise_max(hi, __builtin_bit_cast(i16x2, x[i]));
        lo = __builtin_elementwise_min(lo, __builtin_bit_cast(i16x2, x[i]));
      }
    }
  }
  __device__ __forceinline__ float value() const {
    if constexpr (ET == NS_FP32) return f;
    if constexpr (ET == NS_FP16) return fmaxf((float)h.x, (float)h.y);
    const short a = hi.x > hi.y ? hi.x : hi.y, b = lo.x < lo.y ? lo.x : lo.y;
    return ns::bf16_lo((uint32_t)(uint16_t)(a >= 0 ? a : b));
  }
};

// A block of T threads takes a row and holds it in registers (U vectors a thread;
// what is longer is read again) between its statistics and its gradient, then
// the row gridDim.x on, whose vectors are asked for as this one's fall free: the
// memory works on both while either is computed.  Bound by memory: 4096 x 128256
// bf16 425 us, 4.9 TB/s read and written; 129 x 50257 float32, a row a block, 19 us,
// most of it the row's way in and out.
template <int ET, int T, int U>
__global__ __launch_bounds__(T) void k_policy_row(Args a) {
  constexpr int EPV = per_vec(ET), NW = T / NS_WAVE, HELD = T * U, ESZ = elem_bytes(ET);
  __shared__ Stat sh[NW];
  __shared__ Slope sh_slope;
  const int tid = threadIdx.x, lane = tid & (NS_WAVE - 1), wv = __builtin_amdgcn_readfirstlane(tid / NS_WAVE);
  const int nvec = a.V / EPV, tail = nvec * EPV + tid;
  int tok;
  float w;
  // The first row from `row` on that is taken; the others' outputs are zeros.
  const auto next_row = [&](int row) {
    for (; row < a.L; row += gridDim.x) {
      if (taken(a, (size_t)row, tok, w)) break;            // uniform
      const Row d(a.dz, (size_t)row, a.ld_d, ESZ, nvec);
      if (tid == 0) put_nothing(a, (size_t)row);
      for (int q = tid; q < nvec; q += T) d.put((uint32_t)q * 16, u32x4{0, 0, 0, 0});
      if (tail < a.V) put_elem<ET>(a.dz, (size_t)row * (size_t)a.ld_d + tail, 0.f);
    }
    return row;
  };
  int row = next_row((int)blockIdx.x);
  if (row >= a.L) return;
  // Blocks that run for long start up to 10 us apart: in step they would all ask
  // for memory at once and all compute at once (4096 x 128256 bf16 440 -> 422 us).
  if ((int)gridDim.x * 8 <= a.L)
    for (int i = (int)(blockIdx.x >> 3 & 7); i > 0; --i) __builtin_amdgcn_s_sleep(48);
  u32x4 x[U];
  {
    const Row z(a.z, (size_t)row, a.ld, ESZ, nvec);
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] = z.get((uint32_t)(u * T + tid) * 16);
  }
  while (true) {
    const size_t at = (size_t)row * (size_t)a.ld;
    const Given given(a, (size_t)row, w);
    const float ztok = one_elem<ET>(a.z, at + tok);
    float ztail = -INFINITY;
    if (tail < a.V) ztail = one_elem<ET>(a.z, at + tail);
    NS_ISSUE_FENCE();
    // each wave's vectors by themselves: their maximum, then their sums
    Top<ET> most;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if ((u + 1) * T > nvec && u * T + tid >= nvec) x[u] = minus_inf<ET>();
      most.add(x[u]);
    }
    Stat st{-INFINITY, 0.f, 0.f, 0.f, 0.f};
    raise(st, ns::wave_max_f32(most.value()), a.c);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u * T < nvec) add_vector<ET>(x[u], a.c, st);     // uniform
      asm volatile("" : "+v"(x[u]));                       // widened anew below: twice the registers otherwise
      __builtin_amdgcn_sched_barrier(0);
    }
    if (HELD < nvec) {
      const Row z(a.z, (size_t)row, a.ld, ESZ, nvec);
      constexpr int AT_ONCE = 4;
#pragma unroll 1
      for (int q = HELD; q < nvec; q += T * AT_ONCE) {
        u32x4 v[AT_ONCE];
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u) v[u] = z.get((uint32_t)(q + u * T + tid) * 16);
        Top<ET> more;
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u) {
          if (q + (u + 1) * T > nvec && q + u * T + tid >= nvec) v[u] = minus_inf<ET>();
          more.add(v[u]);
        }
        const float top = more.value();
        if (__ballot(top > st.top)) raise(st, ns::wave_max_f32(top), a.c);
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u) {
          add_vector<ET>(v[u], a.c, st);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
    st.S = ns::wave_sum_f32(st.S);
    st.W = ns::wave_sum_f32(st.W);
    if (wv == 0 && nvec * EPV < a.V) st = join(st, stat_of_lanes(ztail, a.c), a.c);
    if (NW > 1) {
      if (lane == 0) sh[wv] = st;
      __syncthreads();
    }
    Slope s;
    if (wv == 0) {
#pragma unroll
      for (int i = 1; i < NW; ++i) st = join(st, sh[i], a.c);
      s = finish(a, (size_t)row, st, ztok, given, tid == 0);
      if (NW > 1 && tid == 0) sh_slope = s;
    }
    if (NW > 1) {
      __syncthreads();
      s = sh_slope;
    }
    const int this_row = row, this_tok = tok;
    row = next_row(row + (int)gridDim.x);
    const bool more = row < a.L;
    const Row zn(a.z, (size_t)(more ? row : this_row), a.ld, ESZ, more ? nvec : 0);
    const Row d(a.dz, (size_t)this_row, a.ld_d, ESZ, nvec);
    const bool usual = is_usual(s);
    uint32_t place = (uint32_t)tid * 16;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      asm volatile("" : "+v"(place));                      // added up as it goes, not kept for every u
      if (u * T < nvec) d.put(place, slope_of<ET>(s, a.c, usual, x[u]));   // uniform
      x[u] = zn.get(place);                                // zeros behind the last row
      __builtin_amdgcn_sched_barrier(0);
      place += T * 16;
    }
    if (HELD < nvec) {
      const Row z(a.z, (size_t)this_row, a.ld, ESZ, nvec);
      for (int q = HELD + tid; q < nvec; q += T) d.put((uint32_t)q * 16, slope_of<ET>(s, a.c, usual, z.get((uint32_t)q * 16)));
    }
    const size_t to = (size_t)this_row * (size_t)a.ld_d;
    if (tail < a.V) put_elem<ET>(a.dz, to + tail, slope_at(s, a.c, ztail));
    // the thread that wrote the token's element writes it once more
    const int owner = this_tok < nvec * EPV ? this_tok / EPV % T : this_tok - nvec * EPV;
    if (tid == owner) put_elem<ET>(a.dz, to + this_tok, s.token);
    if (!more) return;
  }
}

// Many rows without a gradient: a block streams a row, two batches a wave in flight.
// Bound by memory (2048 x 151936 fp16, half left out, 59 to 64 us, 5 TB/s; 4096 x
// 128256 bf16 165, 6.4).
// Eight waves for long rows, so that blocks end early and rows that are left out
// leave no CU behind (2048 x 151936 fp16, half of them left out, 71 us with four
// waves, 64 with eight, 82 with 16), one for short ones (20000 x 2000 bf16 37 us
// with four, 67 with eight).
template <int ET, int T>
__global__ __launch_bounds__(T) void k_policy_stream(Args a) {
  constexpr int EPV = per_vec(ET), NW = T / NS_WAVE, STEP = NS_WAVE * kUnroll;
  __shared__ Stat sh[NW];
  const size_t row = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & (NS_WAVE - 1), wv = tid / NS_WAVE;
  int tok;
  float w;
  if (!taken(a, row, tok, w)) {                            // uniform
    if (tid == 0) put_nothing(a, row);
    return;
  }
  const char* zrow = (const char*)a.z + row * (size_t)a.ld * elem_bytes(ET);
  const int nvec = a.V / EPV;
  const float ztok = one_elem<ET>(zrow, tok);
  const Given given(a, row, w);
  Stat st{-INFINITY, 0.f, 0.f, 0.f, 0.f};
  const auto load = [&](int base, u32x4(&x)[kUnroll]) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int q = base + u * NS_WAVE + lane;
      x[u] = __builtin_nontemporal_load((const u32x4_any*)(zrow + (size_t)(q < nvec ? q : nvec - 1) * 16));
    }
  };
  u32x4 x0[kUnroll], x1[kUnroll];
  if (wv * STEP < nvec) load(wv * STEP, x0);
#pragma unroll 1
  for (int base = wv * STEP; base < nvec; base += NW * STEP) {
    load(base + NW * STEP, x1);
    NS_ISSUE_FENCE();
    if (base + STEP > nvec) {                              // uniform
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (base + u * NS_WAVE + lane >= nvec) x0[u] = minus_inf<ET>();
    }
    float mx[kUnroll], lane_max;
    add_batch<ET>(x0, a.c, st, mx, lane_max);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) x0[u] = x1[u];
  }
  st.S = ns::wave_sum_f32(st.S);
  st.W = ns::wave_sum_f32(st.W);
  if (wv == 0 && a.V % EPV != 0) {                         // the last elements, fewer than a vector
    const int e = nvec * EPV + lane;
    st = join(st, stat_of_lanes(e < a.V ? one_elem<ET>(zrow, e) : -INFINITY, a.c), a.c);
  }
  if (NW > 1) {
    if (lane == 0) sh[wv] = st;
    __syncthreads();
    if (wv != 0) return;
#pragma unroll
    for (int i = 1; i < NW; ++i) st = join(st, sh[i], a.c);
  }
  finish(a, row, st, ztok, given, lane == 0);
}

// Parts of rows: a wave streams part `part` of S of one row.  With S = 1 it ends
// the row, else it leaves the part's statistics.  Bound by latency (8 x 128256
// float32 4.4 us, and 4.6 for k_policy_end behind it).
constexpr int kPartWaves = 4;

template <int ET>
__global__ __launch_bounds__(kPartWaves* NS_WAVE) void k_policy_parts(Args a) {
  constexpr int EPV = per_vec(ET), STEP = NS_WAVE * kUnroll;
  const int lane = threadIdx.x & (NS_WAVE - 1);
  const int64_t item = (int64_t)blockIdx.x * kPartWaves + threadIdx.x / NS_WAVE;
  const size_t row = (size_t)(item / a.S);
  const int part = (int)(item % a.S);
  if (row >= (size_t)a.L) return;                          // wave-uniform; no block barrier below
  int tok;
  float w;
  if (!taken(a, row, tok, w)) {
    if (a.S == 1 && lane == 0) put_nothing(a, row);
    if (a.S > 1 && part == 0 && lane == 0) a.kept[row].tok = -1;
    return;
  }
  const char* zrow = (const char*)a.z + row * (size_t)a.ld * elem_bytes(ET);
  const int nvec = a.V / EPV;
  const int q0 = (int)((int64_t)nvec * part / a.S), q1 = (int)((int64_t)nvec * (part + 1) / a.S);
  Stat st{-INFINITY, 0.f, 0.f, 0.f, 0.f};
  // loads under no condition, so that a batch stays in flight behind the one that is summed
  const auto load = [&](int base, u32x4(&x)[kUnroll]) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int q = base + u * NS_WAVE + lane;
      const u32x4_any* from = (const u32x4_any*)(zrow + (size_t)(q < q1 ? q : q1 - 1) * 16);
      x[u] = a.dz ? *from : __builtin_nontemporal_load(from);   // the gradient reads them again
    }
  };
  u32x4 x0[kUnroll], x1[kUnroll];
  if (q0 < q1) load(q0, x0);
#pragma unroll 1
  for (int base = q0; base < q1; base += STEP) {
    load(base + STEP, x1);
    NS_ISSUE_FENCE();
    if (base + STEP > q1) {                                // uniform
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (base + u * NS_WAVE + lane >= q1) x0[u] = minus_inf<ET>();
    }
    float mx[kUnroll], lane_max;
    add_batch<ET>(x0, a.c, st, mx, lane_max);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) x0[u] = x1[u];
  }
  st.S = ns::wave_sum_f32(st.S);
  st.W = ns::wave_sum_f32(st.W);
  if (part + 1 == a.S && a.V % EPV != 0) {                 // the last elements, fewer than a vector
    const int e = nvec * EPV + lane;
    st = join(st, stat_of_lanes(e < a.V ? one_elem<ET>(zrow, e) : -INFINITY, a.c), a.c);
  }
  if (a.S == 1) {
    finish(a, row, st, one_elem<ET>(zrow, tok), Given(a, row, w), lane == 0);
  } else if (lane == 0) {
    a.stat[item] = st;
    if (part == 0) a.kept[row] = Kept{Given(a, row, w), one_elem<ET>(zrow, tok), tok};
  }
}

// The parts of a row joined, one in each of S lanes and the whole in all of them.
__device__ __forceinline__ Stat join_parts(const Args& a, Stat st, int lane) {
  for (int m = 1; m < a.S; m <<= 1) {
    Stat o;
    o.top = __shfl_xor(st.top, m, NS_WAVE);
    o.ref = __shfl_xor(st.ref, m, NS_WAVE);
    o.E = __shfl_xor(st.E, m, NS_WAVE);
    o.S = __shfl_xor(st.S, m, NS_WAVE);
    o.W = __shfl_xor(st.W, m, NS_WAVE);
    st = lane & m ? join(o, st, a.c) : join(st, o, a.c);   // the lower part first in both lanes
  }
  return st;
}

// The sum of a block's values, in the same order each time.
template <int T>
__device__ __forceinline__ void put_sum(double s, float* loss) {
  __shared__ double sh[T / NS_WAVE];
  const int tid = threadIdx.x;
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) s += __shfl_xor(s, m, NS_WAVE);
  if ((tid & (NS_WAVE - 1)) == 0) sh[tid / NS_WAVE] = s;
  __syncthreads();
  if (tid != 0) return;
  s = sh[0];
  for (int i = 1; i < T / NS_WAVE; ++i) s += sh[i];
  *loss = (float)s;
}

// Rows whose parts are known: the outputs of every row, S lanes each, and the loss.
constexpr int kTotalThreads = 1024;

__device__ __forceinline__ void end_rows(const Args& a, float* loss) {
  const int tid = threadIdx.x, lane = tid & (NS_WAVE - 1), part = tid & (a.S - 1);
  double total = 0.0;
  for (int row = tid / a.S; row < a.L; row += kTotalThreads / a.S) {
    const Kept kept = a.kept[row];                         // of a row that is not taken: anything but the token
    const Stat st = join_parts(a, a.stat[(size_t)row * a.S + part], lane);
    if (kept.tok >= 0) {
      double mine = 0.0;
      finish(a, row, st, kept.ztok, kept.given, part == 0, &mine);
      if (part == 0) total += mine;
    } else if (part == 0) {
      put_nothing(a, row);
    }
  }
  put_sum<kTotalThreads>(total, loss);
}

__global__ __launch_bounds__(kTotalThreads) void k_policy_end(Args a, float* loss) { end_rows(a, loss); }

// The same beside the gradient: the last block ends the rows, each of the others
// takes a part of one row and joins that row's parts for itself.  dlogits may be
// logits: a block reads its part before it writes it, and the token's logit is in
// the workspace, as all else that a row was given.
constexpr int kSlopeThreads = kTotalThreads;

template <int ET>
__global__ __launch_bounds__(kSlopeThreads) void k_policy_slope(Args a, float* loss, int chunks) {
  constexpr int EPV = per_vec(ET), U = 2;
  if (blockIdx.x + 1 == gridDim.x) {
    end_rows(a, loss);
    return;
  }
  __shared__ Slope sh;
  const size_t row = blockIdx.x / (unsigned)chunks;
  const int chunk = (int)(blockIdx.x % (unsigned)chunks);
  const int tid = threadIdx.x, lane = tid & (NS_WAVE - 1);
  const char* zrow = (const char*)a.z + row * (size_t)a.ld * elem_bytes(ET);
  char* drow = (char*)a.dz + row * (size_t)a.ld_d * elem_bytes(ET);
  const int nvec = a.V / EPV, tail = nvec * EPV + tid;
  const int q0 = chunk * kSlopeThreads * U + tid;
  const int tok = a.kept[row].tok;                         // uniform
  const bool in = tok >= 0;
  if (in && tid < NS_WAVE) {
    const Kept kept = a.kept[row];
    const Slope s = finish(a, row, join_parts(a, a.stat[row * a.S + (lane & (a.S - 1))], lane), kept.ztok, kept.given, false);
    if (tid == 0) sh = s;
  }
  u32x4 x[U];
  if (in && q0 - tid < nvec) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = q0 + u * kSlopeThreads;
      x[u] = __builtin_nontemporal_load((const u32x4_any*)(zrow + (size_t)(at < nvec ? at : 0) * 16));
    }
  }
  __syncthreads();
  Slope s{0.f, 0.f, 0.f, 0.f, 0.f};
  if (in) s = sh;
  const bool usual = is_usual(s);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int at = q0 + u * kSlopeThreads;
    if (at >= nvec) continue;
    const u32x4 y = in ? slope_of<ET>(s, a.c, usual, x[u]) : u32x4{0, 0, 0, 0};
    __builtin_nontemporal_store(y, (u32x4_any*)(drow + (size_t)at * 16));
    // the token's element once more
    if (in && at == tok / EPV) put_elem<ET>(drow, tok, s.token);
  }
  if (chunk == 0 && tail < a.V) {
    const float z = one_elem<ET>(zrow, tail);
    put_elem<ET>(drow, tail, !in ? 0.f : (tail == tok ? s.token : slope_at(s, a.c, z)));
  }
}

// The sum of the rows' losses.
__global__ __launch_bounds__(kTotalThreads) void k_policy_total(const double* __restrict__ row_loss, int L,
                                                                float* __restrict__ loss) {
  double s = 0.0;
  for (int i = threadIdx.x; i < L; i += kTotalThreads) s += row_loss[i];
  put_sum<kTotalThreads>(s, loss);
}

// Parts of a row: doubled until about 2048 waves run, each with a batch at least.
constexpr int kMaxParts = 64;
constexpr int kWavesWanted = 2048;

int parts_of(int L, int V, int dtype) {
  const int batch = NS_WAVE * kUnroll * per_vec(dtype);
  const int most = (V + batch - 1) / batch;
  int s = 1;
  while ((int64_t)s * L * 4 < kWavesWanted * 3 && s * 2 <= most && s < kMaxParts) s *= 2;
  return s;
}

// From this many rows on a block takes one and reads it once; fewer are split over
// the chip (with gradient, in parts and whole: 32 x 128256 bf16 16.8 and 25.3 us, 64 x
// 50257 float32 17.0 and 19.2, 129 x 50257 23.4 and 20.9, 256 x 128256 bf16 41.7 and
// 33.1; the loss alone, 129 x 128256 bf16, 19.1 and 17.1).
constexpr int kWholeRows = 96;

template <int ET, int T, int U>
void launch_row(const Args& a, hipStream_t stream) {
  // one block of 1024 threads a CU; smaller ones overlap each other
  const unsigned blocks = T == 1024 && a.L > 256 ? 256u : (unsigned)a.L;
  hipLaunchKernelGGL((k_policy_row<ET, T, U>), dim3(blocks), dim3(T), 0, stream, a);
}

template <int ET>
int launch_policy(Args a, float* loss, hipStream_t stream) {
  const int nvec = a.V / per_vec(ET);
  if (a.L >= kWholeRows && !a.dz) {
    const dim3 grid((unsigned)a.L);
    if (nvec <= 512) hipLaunchKernelGGL((k_policy_stream<ET, 64>), grid, dim3(64), 0, stream, a);
    else if (nvec <= 4096) hipLaunchKernelGGL((k_policy_stream<ET, 256>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((k_policy_stream<ET, 512>), grid, dim3(512), 0, stream, a);
    a.S = 1;
  } else if (a.L >= kWholeRows) {
    if (nvec <= 64 * 4) launch_row<ET, 64, 4>(a, stream);
    else if (nvec <= 256 * 4) launch_row<ET, 256, 4>(a, stream);
    else if (nvec <= 256 * 8) launch_row<ET, 256, 8>(a, stream);
    else if (nvec <= 256 * 16) launch_row<ET, 256, 16>(a, stream);
    else if (nvec <= 512 * 16) launch_row<ET, 512, 16>(a, stream);
    else launch_row<ET, 1024, 16>(a, stream);
    a.S = 1;
  } else {
    if (a.dz && a.S == 1) a.S = 2;                         // the gradient's blocks take statistics from the workspace
    const dim3 grid((unsigned)(((int64_t)a.L * a.S + kPartWaves - 1) / kPartWaves)), block(kPartWaves * NS_WAVE);
    hipLaunchKernelGGL(k_policy_parts<ET>, grid, block, 0, stream, a);
  }
  const int rc = ns_launch_status();
  if (rc != NS_OK) return rc;
  if (a.S == 1) {
    hipLaunchKernelGGL(k_policy_total, dim3(1), dim3(kTotalThreads), 0, stream, (const double*)a.row_loss, a.L, loss);
  } else if (!a.dz) {
    hipLaunchKernelGGL(k_policy_end, dim3(1), dim3(kTotalThreads), 0, stream, a, loss);
  } else {
    const int chunks = nvec > 0 ? (nvec + 2 * kSlopeThreads - 1) / (2 * kSlopeThreads) : 1;
    hipLaunchKernelGGL(k_policy_slope<ET>, dim3((unsigned)(chunks * a.L + 1)), dim3(kSlopeThreads), 0, stream, a, loss, chunks);
  }
  return ns_launch_status();
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Only as many rows as are taken in parts.
size_t kept_bytes(int L) { return align256((size_t)(L < 1 ? 1 : (L < kWholeRows ? L : kWholeRows)) * sizeof(Kept)); }

// Room for the parts of L rows or any fewer: a row has at most the parts of a
// single one (of float32, which has the smallest batches), two where there is a
// gradient, and rows in more come to less than 3/2 kWavesWanted of them together.
size_t policy_ws(int L, int V) {
  const size_t l = (size_t)(L > 0 ? L : 1), one = (size_t)parts_of(1, V, NS_FP32);
  const size_t most = l * (one < 2 ? 2 : one), few = l * 2 > kWavesWanted * 3 / 2 ? l * 2 : kWavesWanted * 3 / 2;
  return align256(l * 8) + kept_bytes(L) + align256((most < few ? most : few) * sizeof(Stat));
}

constexpr int64_t kMaxLd = (int64_t)1 << 40;

bool known_dtype(int t) { return t == NS_BF16 || t == NS_FP32 || t == NS_FP16; }
bool elem_aligned(const void* p, int dtype) { return ((uintptr_t)p) % (dtype == NS_FP32 ? 4 : 2) == 0; }
// NaN fails every comparison
bool temp_ok(float t) { return t >= NS_MIN_INV_TEMP && t <= NS_MAX_INV_TEMP; }
bool coefs_ok(float lo, float hi, float beta, float ent) {
  return lo >= 0.f && lo <= 1.f && hi >= 0.f && fabsf(beta) < INFINITY && fabsf(ent) < INFINITY;
}
bool dims_ok(int L, int V) { return L >= 0 && L <= NS_MAX_ROWS && V >= 1 && V <= NS_MAX_V; }

}  // namespace

extern "C" {

size_t nanospec_policy_loss_workspace_bytes(int32_t L, int32_t V) { return dims_ok(L, V) ? policy_ws(L, V) : 0; }

int nanospec_policy_loss(const void* logits, int64_t ld, int32_t L, int32_t V, int32_t dtype, float inv_temp,
                         const int32_t* tokens, const float* old_logprob, const float* ref_logprob,
                         const float* advantage, const float* weight, float eps_low, float eps_high, float kl_coef,
                         float ent_coef, float* loss, float* logprob, float* kl, float* entropy, const float* g_loss,
                         void* dlogits, int64_t ld_d, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!known_dtype(dtype)) return NS_EDTYPE;
  if (!dims_ok(L, V) || ld < V || ld > kMaxLd || !temp_ok(inv_temp) || !coefs_ok(eps_low, eps_high, kl_coef, ent_coef))
    return NS_EINVAL;
  if (dlogits && (ld_d < V || ld_d > kMaxLd || !elem_aligned(dlogits, dtype) || (dlogits == logits && ld_d != ld)))
    return NS_EINVAL;
  if (!loss || !ws || (((uintptr_t)ws) & 255u) || (!ref_logprob && (kl || kl_coef != 0.f))) return NS_EINVAL;
  if (L > 0 && (!logits || !tokens || !old_logprob || !advantage || !logprob || !elem_aligned(logits, dtype)))
    return NS_EINVAL;
  if (ws_bytes < policy_ws(L, V)) return NS_ECAPACITY;
  (void)hipGetLastError();
  const float c = (float)((double)inv_temp * 1.4426950408889634);
  char* base = (char*)ws;
  const int S = parts_of(L, V, dtype);
  Args a{logits, ld, L, V, inv_temp, c, (float)((double)inv_temp * 1.4426950408889634 / c - 1.0), tokens,
         old_logprob, ref_logprob, advantage, weight, eps_low, eps_high, kl_coef, ent_coef, logprob, kl, entropy,
         g_loss, dlogits, ld_d, (double*)base, S, nullptr, nullptr};
  const size_t rows = align256((size_t)(L > 0 ? L : 1) * 8);
  a.kept = (Kept*)(base + rows);
  a.stat = (Stat*)(base + rows + kept_bytes(L));
  if (L == 0) {
    hipLaunchKernelGGL(k_policy_total, dim3(1), dim3(kTotalThreads), 0, stream, (const double*)a.row_loss, 0, loss);
    return ns_launch_status();
  }
  if (dtype == NS_BF16) return launch_policy<NS_BF16>(a, loss, stream);
  if (dtype == NS_FP16) return launch_policy<NS_FP16>(a, loss, stream);
  return launch_policy<NS_FP32>(a, loss, stream);
}

}  // extern "C"
