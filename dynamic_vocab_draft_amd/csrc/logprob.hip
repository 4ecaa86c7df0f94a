// Log-probabilities of given tokens with entropy and top alternatives, and
// their gradient, over rows of full-vocabulary logits.
//
// For a row z and an inverse temperature t, with z' = t z:
//     lse = log sum_j exp(z'_j),   logp_j = z'_j - lse,   p_j = exp(logp_j),
//     H   = -sum_j p_j logp_j.
// Forward, in one pass over the row: with c = t log2(e) and an integer E near
// c max_j z_j, y_j = c z_j - E (one fused multiply-add) gives
//     S = sum 2^y_j,  W = sum 2^y_j y_j,
//     lse = ln2 (E + log2 S),  H = ln2 (log2 S - W / S),
// and E moves by whole powers of two only, so rescaling S is exact.  All of it
// is float32.
#include "common.hpp"
#include "select.hpp"

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kUnroll = 4;               // 16-byte vectors per lane and batch
constexpr int kRowWaves = 4;             // waves of a forward block
constexpr int kMaxParts = 64;            // parts of a row, at most
constexpr int kWavesWanted = 2048;       // waves that fill the chip: eight a CU
constexpr int kBuf = 256;                // candidate keys of a wave
constexpr float kWide = 1024.f;          // |c max z| from which y is taken relative to the maximum itself

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

// The smallest float above v (NaN above +infinity, which nothing reaches).
__device__ __forceinline__ float next_up(float v) {
  const uint32_t u = __float_as_uint(v);
  if (v == INFINITY) return __uint_as_float(0x7FC00000u);
  if ((u & 0x7FFFFFFFu) == 0) return __uint_as_float(1u);
  return __uint_as_float(u & 0x80000000u ? u - 1 : u + 1);
}

// Orders a wave's own LDS writes before its following reads.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

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

// ---------------------------------------------------------------------------
// The best k keys of a wave.  Elements that may still count are appended to
// an LDS buffer; when it has filled up, the k best are kept, sorted, and `lo`
// becomes the smallest value that a later element needs.  Ids rise from batch
// to batch, so a later element that only ties the k-th value loses to it.
// ---------------------------------------------------------------------------
struct Best {
  uint64_t* buf;
  int cnt, k;
  float lo;        // elements below it cannot be among the k best
  bool fresh;      // no bound yet

  __device__ __forceinline__ void compact(int lane) {
    wave_sync();
    uint64_t mine[kBuf / NS_WAVE];
    int rank[kBuf / NS_WAVE];
#pragma unroll
    for (int q = 0; q < kBuf / NS_WAVE; ++q) {
      const int i = lane + q * NS_WAVE;
      mine[q] = i < cnt ? buf[i] : 0;
      rank[q] = 0;
    }
    for (int p = 0; p < cnt; ++p) {
      const uint64_t o = buf[p];
#pragma unroll
      for (int q = 0; q < kBuf / NS_WAVE; ++q) rank[q] += o > mine[q];
    }
    wave_sync();
#pragma unroll
    for (int q = 0; q < kBuf / NS_WAVE; ++q)
      if (mine[q] != 0 && rank[q] < k) buf[rank[q]] = mine[q];
    wave_sync();
    if (cnt >= k) {
      cnt = k;
      lo = next_up(ns::key_val(buf[k - 1]));
    }
  }

  __device__ __forceinline__ void add(float v, int id, bool live, float least, int lane) {
    const bool pass = live && v >= least;
    const unsigned long long ball = __ballot(pass);
    if (!ball) return;
    if (cnt + NS_WAVE > kBuf) compact(lane);
    if (pass) buf[cnt + __popcll(ball & ((1ull << lane) - 1))] = ns::make_key(v, id);
    cnt += __popcll(ball);
  }

  // A bound before any key is held: the k-th largest of the lanes' maxima.
  __device__ __forceinline__ void start(float lane_max, int lane) {
    int gt = 0, ge = 0;
    for (int q = 0; q < NS_WAVE; ++q) {
      const float o = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(lane_max), q));
      gt += o > lane_max;
      ge += o >= lane_max;
    }
    const unsigned long long ball = __ballot(gt < k && ge >= k);
    lo = ball ? __int_as_float(__builtin_amdgcn_readlane(__float_as_int(lane_max), __ffsll(ball) - 1)) : -INFINITY;
    fresh = false;
  }
};

struct Args {
  const void* z;
  int64_t ld;
  int L, V, S, k, T;
  float t, c;                  // inverse temperature, and times log2(e)
  const int32_t* tokens;       // [L][T]
  float* logprob;              // [L][T]
  float* lse;
  float* entropy;              // or NULL
  int32_t* top_ids;            // [L][k]
  float* top_vals;
  Stat* stat;                  // [L][S]
  uint64_t* keys;              // [L][S][k]
};

// A row's outputs from its statistics.  logp = ln2 (y - log2 S) keeps the
// digits that a rounded lse would lose.
struct Row {
  float t, c, ref, E, l2, lse, H;
  bool bad, none;
  __device__ __forceinline__ Row(const Stat& s, const Args& a) : t(a.t), c(a.c) {
    bad = !(s.S < INFINITY) || s.top == INFINITY;
    none = s.S == 0.f;
    const float nan = __uint_as_float(0x7FC00000u);
    ref = s.ref;
    E = s.E;
    l2 = log2f(s.S);
    lse = bad ? nan : (none ? -INFINITY : ref * t + kLn2 * (E + l2));
    H = bad ? nan : (none ? 0.f : fmaxf(kLn2 * (l2 - s.W / s.S), 0.f));
  }
  __device__ __forceinline__ float logp(float z) const {
    if (bad) return __uint_as_float(0x7FC00000u);
    if (none || z == -INFINITY) return -INFINITY;
    const float y = ref == 0.f ? fmaf(z, c, -E) : (z - ref) * c - E;
    // far from the rest (a mask of the type's lowest value) y's last digits
    // are nothing, but c z may overflow where t z does not
    return fabsf(y) < 0x1p24f ? kLn2 * (y - l2) : z * t - lse;
  }
};

template <int ET>
__device__ __forceinline__ void put_tokens(const Args& a, const Row& r, size_t row, int i) {
  const int tok = a.tokens[row * a.T + i];
  float v = 0.f;
  if (tok >= 0 && tok < a.V) v = r.logp(one_elem<ET>(a.z, row * (size_t)a.ld + tok));
  a.logprob[row * a.T + i] = v;
}

__device__ __forceinline__ void put_top(const Args& a, const Row& r, size_t row, int i, uint64_t key) {
  const bool have = key != 0 && !r.bad;
  a.top_ids[row * a.k + i] = have ? ns::key_id(key) : -1;
  a.top_vals[row * a.k + i] = r.bad ? __uint_as_float(0x7FC00000u) : (key ? r.logp(ns::key_val(key)) : -INFINITY);
}

// One batch of a lane's vectors: statistics, then the candidates.
template <int ET, bool TOP>
__device__ __forceinline__ void take(const u32x4 (&x)[kUnroll], int q0, int q1, float c, Stat& st, Best& best,
                                     int lane) {
  constexpr int EPV = per_vec(ET);
  float mx[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    float v[EPV];
    widen<ET>(x[u], v);
    float m = v[0];
#pragma unroll
    for (int e = 1; e < EPV; ++e) m = fmaxf(m, v[e]);
    mx[u] = m;
  }
  float lane_max = mx[0];
#pragma unroll
  for (int u = 1; u < kUnroll; ++u) lane_max = fmaxf(lane_max, mx[u]);
  const float top = ns::wave_max_f32(lane_max);
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
  if (TOP) {
    if (best.fresh) best.start(lane_max, lane);
    if (top >= best.lo) {                                  // uniform
      const float least = best.lo;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (!__ballot(mx[u] >= least)) continue;
        const int q = q0 + u * NS_WAVE + lane;
        float v[EPV];
        widen<ET>(x[u], v);
#pragma unroll
        for (int e = 0; e < EPV; ++e) best.add(v[e], q * EPV + e, q < q1, least, lane);
      }
      if (best.cnt >= best.k + NS_WAVE / 2) best.compact(lane);
    }
  }
}

// Forward.  A wave owns part `part` of S of one row and streams it once with
// 16-byte loads, two register batches in turn.
template <int ET, bool TOP>
__global__ __launch_bounds__(kRowWaves* NS_WAVE) void k_logprobs(Args a) {
  constexpr int EPV = per_vec(ET), STEP = NS_WAVE * kUnroll;
  __shared__ uint64_t sh[TOP ? kRowWaves * kBuf : 1];
  const int lane = threadIdx.x & (NS_WAVE - 1), wv = threadIdx.x / NS_WAVE;
  const int64_t item = (int64_t)blockIdx.x * kRowWaves + wv;
  const size_t row = (size_t)(item / a.S);
  const int part = (int)(item % a.S);
  if (row >= (size_t)a.L) return;                          // wave-uniform; no block barrier below
  const char* zrow = (const char*)a.z + row * (size_t)a.ld * elem_bytes(ET);
  const int nvec = a.V / EPV;
  const int per = ((nvec + a.S - 1) / a.S + NS_WAVE - 1) / NS_WAVE * NS_WAVE;
  const int q0 = part * per < nvec ? part * per : nvec;
  const int q1 = part + 1 == a.S ? nvec : (q0 + per < nvec ? q0 + per : nvec);
  Stat st{-INFINITY, 0.f, 0.f, 0.f, 0.f};
  Best best{sh + (TOP ? wv * kBuf : 0), 0, a.k, -INFINITY, true};
  // Loads are never under a condition, so that the batch in flight behind them
  // can be counted: past the end they read the part's last vector again, and
  // `mask` puts -infinity in its place.
  const auto load = [&](int base, u32x4(&x)[kUnroll]) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int q = base + u * NS_WAVE + lane;
      x[u] = __builtin_nontemporal_load((const u32x4_any*)(zrow + (size_t)(q < q1 ? q : q1 - 1) * 16));
    }
  };
  const auto mask = [&](int base, u32x4(&x)[kUnroll]) {
    if (base + STEP <= q1) return;                         // uniform
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (base + u * NS_WAVE + lane >= q1) x[u] = minus_inf<ET>();
  };
  u32x4 x0[kUnroll], x1[kUnroll];
  if (q0 < q1) load(q0, x0);
  for (int base = q0; base < q1; base += 2 * STEP) {
    load(base + STEP, x1);
    NS_ISSUE_FENCE();
    mask(base, x0);
    take<ET, TOP>(x0, base, q1, a.c, st, best, lane);
    if (base + STEP >= q1) break;                          // uniform
    load(base + 2 * STEP, x0);
    NS_ISSUE_FENCE();
    mask(base + STEP, x1);
    take<ET, TOP>(x1, base + STEP, q1, a.c, st, best, lane);
  }
  if (part + 1 == a.S && a.V % EPV != 0) {                 // the last elements, fewer than a vector
    const int e = nvec * EPV + lane;
    const bool live = e < a.V;
    const float v = live ? one_elem<ET>(zrow, e) : -INFINITY;
    Stat s{-INFINITY, 0.f, 0.f, 0.f, 0.f};
    const float top = ns::wave_max_f32(v);
    if (top != -INFINITY) {
      const float cm = top * a.c;
      s.top = top;
      s.E = fabsf(cm) < kWide ? rintf(cm) : 0.f;
      s.ref = fabsf(cm) < kWide ? 0.f : top;
    }
    const float y = s.ref == 0.f ? fmaf(v, a.c, -s.E) : (v - s.ref) * a.c;
    s.S = exp2_fast(y);
    s.W = s.S * fmaxf(y, -200.f);
    st.S = ns::wave_sum_f32(st.S);
    st.W = ns::wave_sum_f32(st.W);
    s.S = ns::wave_sum_f32(s.S);
    s.W = ns::wave_sum_f32(s.W);
    st = join(st, s, a.c);
    if (TOP) {
      if (best.fresh) best.start(v, lane);
      best.add(v, e, live, best.lo, lane);
    }
  } else {
    st.S = ns::wave_sum_f32(st.S);
    st.W = ns::wave_sum_f32(st.W);
  }
  if (TOP) {
    best.compact(lane);
    wave_sync();
  }
  if (a.S == 1) {
    const Row r(st, a);
    if (lane == 0) {
      a.lse[row] = r.lse;
      if (a.entropy) a.entropy[row] = r.H;
    }
    if (lane < a.T) put_tokens<ET>(a, r, row, lane);
    if (TOP && lane < a.k) put_top(a, r, row, lane, lane < best.cnt ? best.buf[lane] : 0);
  } else {
    if (lane == 0) a.stat[item] = st;
    if (TOP && lane < a.k) a.keys[item * a.k + lane] = lane < best.cnt ? best.buf[lane] : 0;
  }
}

// Joins the S parts of a row.
template <int ET, bool TOP>
__global__ __launch_bounds__(TOP ? kSelectThreads : NS_WAVE) void k_logprobs_join(Args a) {
  const size_t row = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & (NS_WAVE - 1);
  // Every wave joins the parts for itself, in the same order.
  Stat st = lane < a.S ? a.stat[row * a.S + lane] : Stat{-INFINITY, 0.f, 0.f, 0.f, 0.f};
  for (int m = 1; m < NS_WAVE; m <<= 1) {
    Stat o;
    o.top = __shfl_xor(st.top, m, NS_WAVE);
    o.ref = __shfl_xor(st.ref, m, NS_WAVE);
    o.E = __shfl_xor(st.E, m, NS_WAVE);
    o.S = __shfl_xor(st.S, m, NS_WAVE);
    o.W = __shfl_xor(st.W, m, NS_WAVE);
    st = lane & m ? join(o, st, a.c) : join(st, o, a.c);   // the lower part first in both lanes
  }
  const Row r(st, a);
  if (tid == 0) {
    a.lse[row] = r.lse;
    if (a.entropy) a.entropy[row] = r.H;
  }
  if (tid < a.T) put_tokens<ET>(a, r, row, tid);
  if constexpr (TOP) {
    __shared__ SelectSmem sm;
    const int nk = a.S * a.k;                              // <= 64 * 64
    float val[4];
    int id[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int q = tid + u * kSelectThreads;
      const uint64_t key = q < nk ? a.keys[row * nk + q] : 0;
      val[u] = key ? ns::key_val(key) : 0.f;
      id[u] = key ? ns::key_id(key) : -1;
    }
    block_select_topk<4>(val, id, a.k, nk, sm, [&](int i, uint64_t key) { put_top(a, r, row, i, key); });
  }
}

// Parts of a row: enough waves for the chip, each with a batch at least.
int parts_of(int L, int V, int dtype) {
  const int batch = NS_WAVE * kUnroll * per_vec(dtype);
  int s = L >= kWavesWanted ? 1 : (kWavesWanted + L - 1) / (L > 0 ? L : 1);
  const int most = (V + batch - 1) / batch;
  s = s > most ? most : s;
  return s < 1 ? 1 : (s > kMaxParts ? kMaxParts : s);
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

size_t logprobs_ws(int L, int V, int k) {
  // fp32 has the smallest batches, so the most parts
  const size_t s = (size_t)parts_of(L, V, NS_FP32), l = (size_t)(L > 0 ? L : 1);
  return align256(l * s * sizeof(Stat)) + align256(l * s * (size_t)k * 8) + 256;
}

template <int ET>
void launch_logprobs(const Args& a, hipStream_t stream) {
  const dim3 grid((unsigned)(((int64_t)a.L * a.S + kRowWaves - 1) / kRowWaves)), block(kRowWaves * NS_WAVE);
  if (a.k > 0) hipLaunchKernelGGL((k_logprobs<ET, true>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((k_logprobs<ET, false>), grid, block, 0, stream, a);
  if (a.S == 1) return;
  if (a.k > 0) hipLaunchKernelGGL((k_logprobs_join<ET, true>), dim3((unsigned)a.L), dim3(kSelectThreads), 0, stream, a);
  else hipLaunchKernelGGL((k_logprobs_join<ET, false>), dim3((unsigned)a.L), dim3(NS_WAVE), 0, stream, a);
}

// ---------------------------------------------------------------------------
// Gradient.  With g_t of the tokens' log-probabilities, g_H of the entropy
// and g_l of the log-sum-exp, and G = g_l - sum_t g_t:
//     dz_j = t (p_j (G - g_H (logp_j + H)) + sum_t g_t [token_t = j]).
// With y_j = log2 p_j the first part is p_j (A + B y_j), A = t (G - g_H H),
// B = -t g_H ln2.  log2(e) lse is taken in two floats; the small one goes
// into A, B and a common factor.
// ---------------------------------------------------------------------------
struct GradArgs {
  const void* z;
  int64_t ld;
  int L, V, T;
  float t, c;
  const int32_t* tokens;
  const float* lse;
  const float* entropy;        // or NULL
  const float* g_logprob;      // [L][T]
  const float* g_entropy;      // or NULL
  const float* g_lse;          // or NULL
  void* dz;
  int64_t ld_d;
};

constexpr int kGradThreads = 256;
constexpr int kGradUnroll = 4;

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

struct Slope {
  float c, L, A, B;
  bool zero;
  // p (A + B y) of a logit
  __device__ __forceinline__ float at(float z) const {
    const float y = fmaf(z, c, -L);
    return exp2_fast(y) * fmaf(B, fmaxf(y, -200.f), A);
  }
};

// dlogits may be logits: a block reads its part of the row, and the logits of
// the tokens in it, before it writes them.
template <int ET>
__global__ __launch_bounds__(kGradThreads) void k_logprobs_grad(GradArgs a, int per, int chunks) {
  constexpr int EPV = per_vec(ET);
  __shared__ int32_t s_tok[NS_MAX_K];
  __shared__ float s_g[NS_MAX_K];
  const size_t row = blockIdx.x / (unsigned)chunks;
  const int chunk = (int)(blockIdx.x % (unsigned)chunks);
  const int tid = threadIdx.x, lane = tid & (NS_WAVE - 1);
  const char* zrow = (const char*)a.z + row * (size_t)a.ld * elem_bytes(ET);
  char* drow = (char*)a.dz + row * (size_t)a.ld_d * elem_bytes(ET);
  const int nvec = a.V / EPV;
  const int q0 = chunk * per;
  const int q1 = q0 + per < nvec ? q0 + per : nvec;
  const bool last = chunk + 1 == chunks;
  // every wave sums the tokens' gradients for itself, in the same order
  int tok = -1;
  float g = 0.f;
  if (lane < a.T) {
    tok = a.tokens[row * a.T + lane];
    g = tok >= 0 && tok < a.V ? a.g_logprob[row * a.T + lane] : 0.f;
  }
  const float sum = ns::wave_sum_f32(g);
  const float lse = a.lse[row], gH = a.g_entropy ? a.g_entropy[row] : 0.f;
  const float H = a.g_entropy ? a.entropy[row] : 0.f, gl = a.g_lse ? a.g_lse[row] : 0.f;
  Slope s;
  s.c = a.c;
  // a row without logits, or whose float32 lse no longer resolves probabilities
  s.zero = fabsf(lse) > 0x1p24f;
  s.L = lse * kLog2e;
  const float low = (float)((double)lse * 1.4426950408889634 - (double)s.L);
  const float f = exp2_fast(-low);
  s.B = -a.t * gH * kLn2 * f;
  s.A = a.t * (gl - sum - gH * H) * f - s.B * low;
  // the token of this thread, if it lies in this block's part and is its first mention
  float ztok = 0.f;
  bool mine = false;
  if (tid < NS_WAVE) {
    if (lane < a.T) {
      s_tok[lane] = tok;
      s_g[lane] = g;
    }
    const int lo = q0 * EPV, hi = last ? a.V : q1 * EPV;
    mine = lane < a.T && tok >= lo && tok < hi && tok < a.V;
    if (mine) ztok = one_elem<ET>(zrow, tok);
  }
  __syncthreads();
  if (mine) {
    float total = 0.f;
    for (int i = 0; i < a.T; ++i)
      if (s_tok[i] == tok) {
        if (i < lane) mine = false;
        total += s_g[i];
      }
    ztok = s.zero ? 0.f : s.at(ztok) + a.t * total;
  }
  for (int base = q0; base < q1; base += kGradThreads * kGradUnroll) {
    u32x4 x[kGradUnroll];
#pragma unroll
    for (int u = 0; u < kGradUnroll; ++u) {
      const int q = base + u * kGradThreads + tid;
      if (q < q1) x[u] = __builtin_nontemporal_load((const u32x4_any*)(zrow + (size_t)q * 16));
    }
    NS_ISSUE_FENCE();
#pragma unroll
    for (int u = 0; u < kGradUnroll; ++u) {
      const int q = base + u * kGradThreads + tid;
      if (q < q1) {
        float v[EPV];
        widen<ET>(x[u], v);
#pragma unroll
        for (int e = 0; e < EPV; ++e) v[e] = s.zero ? 0.f : s.at(v[e]);
        u32x4 y;
        if constexpr (ET == NS_FP32) {
          y = u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
        } else {
          y = u32x4{narrow2<ET>(v[0], v[1]), narrow2<ET>(v[2], v[3]), narrow2<ET>(v[4], v[5]), narrow2<ET>(v[6], v[7])};
        }
        __builtin_nontemporal_store(y, (u32x4_any*)(drow + (size_t)q * 16));
      }
    }
  }
  if (last) {
    const int e = nvec * EPV + tid;
    if (e < a.V) put_elem<ET>(drow, e, s.zero ? 0.f : s.at(one_elem<ET>(zrow, e)));
  }
  __syncthreads();                                         // the part is written before its tokens' elements are
  if (mine) put_elem<ET>(drow, tok, ztok);
}

template <int ET>
void launch_grad(const GradArgs& a, hipStream_t stream) {
  const int nvec = a.V / per_vec(ET);
  const int per = kGradThreads * kGradUnroll;
  const int chunks = nvec > 0 ? (nvec + per - 1) / per : 1;
  hipLaunchKernelGGL(k_logprobs_grad<ET>, dim3((unsigned)chunks * (unsigned)a.L), dim3(kGradThreads), 0,
                     stream, a, per, chunks);
}

bool known_dtype(int t) { return t == NS_BF16 || t == NS_FP32 || t == NS_FP16; }
bool elem_aligned(const void* p, int dtype) { return ((uintptr_t)p) % (dtype == NS_FP32 ? 4 : 2) == 0; }
// NaN fails both comparisons
bool temp_ok(float t) { return t >= NS_MIN_INV_TEMP && t <= NS_MAX_INV_TEMP; }
bool dims_ok(int L, int64_t ld, int V, int T) {
  return L >= 0 && L <= NS_MAX_ROWS && V >= 1 && V <= NS_MAX_V && ld >= V && T >= 0 && T <= NS_MAX_K;
}

}  // namespace

extern "C" {

size_t nanospec_token_logprobs_workspace_bytes(int32_t L, int32_t V, int32_t k) {
  if (L < 0 || L > NS_MAX_ROWS || V < 1 || V > NS_MAX_V || k < 0 || k > NS_MAX_K || k > V) return 0;
  return logprobs_ws(L, V, k);
}

int nanospec_token_logprobs(const void* logits, int64_t ld, int32_t L, int32_t V, int32_t dtype, float inv_temp,
                            const int32_t* tokens, int32_t T, int32_t k, float* logprob, float* lse, float* entropy,
                            int32_t* top_ids, float* top_logprobs, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!known_dtype(dtype)) return NS_EDTYPE;
  if (!dims_ok(L, ld, V, T) || k < 0 || k > NS_MAX_K || k > V || !temp_ok(inv_temp)) return NS_EINVAL;
  if (L == 0) return NS_OK;
  if (!logits || !lse || !ws || (T > 0 && (!tokens || !logprob)) || (k > 0 && (!top_ids || !top_logprobs)))
    return NS_EINVAL;
  if ((((uintptr_t)ws) & 255u) || !elem_aligned(logits, dtype)) return NS_EINVAL;
  if (ws_bytes < logprobs_ws(L, V, k)) return NS_ECAPACITY;
  (void)hipGetLastError();
  Args a;
  a.z = logits;
  a.ld = ld;
  a.L = L;
  a.V = V;
  a.S = parts_of(L, V, dtype);
  a.k = k;
  a.T = T;
  a.t = inv_temp;
  a.c = (float)((double)inv_temp * 1.4426950408889634);
  a.tokens = tokens;
  a.logprob = logprob;
  a.lse = lse;
  a.entropy = entropy;
  a.top_ids = top_ids;
  a.top_vals = top_logprobs;
  a.stat = (Stat*)ws;
  a.keys = (uint64_t*)((char*)ws + align256((size_t)L * a.S * sizeof(Stat)));
  if (dtype == NS_BF16) launch_logprobs<NS_BF16>(a, stream);
  else if (dtype == NS_FP16) launch_logprobs<NS_FP16>(a, stream);
  else launch_logprobs<NS_FP32>(a, stream);
  return ns_launch_status();
}

int nanospec_token_logprobs_grad(const void* logits, int64_t ld, int32_t L, int32_t V, int32_t dtype, float inv_temp,
                                 const int32_t* tokens, int32_t T, const float* lse, const float* entropy,
                                 const float* g_logprob, const float* g_entropy, const float* g_lse, void* dlogits,
                                 int64_t ld_d, hipStream_t stream) {
  if (!known_dtype(dtype)) return NS_EDTYPE;
  if (!dims_ok(L, ld, V, T) || ld_d < V || !temp_ok(inv_temp)) return NS_EINVAL;
  if (L == 0) return NS_OK;
  if (!logits || !lse || !dlogits || (T > 0 && (!tokens || !g_logprob)) || (g_entropy && !entropy)) return NS_EINVAL;
  if (!elem_aligned(logits, dtype) || !elem_aligned(dlogits, dtype)) return NS_EINVAL;
  if (dlogits == logits && ld_d != ld) return NS_EINVAL;
  (void)hipGetLastError();
  const GradArgs a{logits, ld, L, V, T, inv_temp, (float)((double)inv_temp * 1.4426950408889634), tokens, lse, entropy,
                   g_logprob, g_entropy, g_lse, dlogits, ld_d};
  if (dtype == NS_BF16) launch_grad<NS_BF16>(a, stream);
  else if (dtype == NS_FP16) launch_grad<NS_FP16>(a, stream);
  else launch_grad<NS_FP32>(a, stream);
  return ns_launch_status();
}

}  // extern "C"
