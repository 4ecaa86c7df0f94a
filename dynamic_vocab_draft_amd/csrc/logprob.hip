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
#include "lists.hpp"

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kUnroll = 4;               // 16-byte vectors per lane and batch
constexpr int kRowWaves = 4;             // waves of a forward block
constexpr int kMaxParts = 64;            // parts of a row, at most; a power of two of them
constexpr int kWavesWanted = 2048;       // waves that fill the chip: eight a CU
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

// Orders a wave's own LDS writes before its following reads.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ uint64_t lane_u64(uint64_t v, int lane) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane);
  return ((uint64_t)hi << 32) | lo;
}

// ---------------------------------------------------------------------------
// The best k keys of a wave: lane r holds the r-th (0: none yet).  The
// elements of a batch that reach the k-th value so far are collected in LDS,
// one of each lane a turn, then enter the list: one or two in turn, up to 16 by
// counting (every lane counts the keys above its own two; no candidate waits
// for the one before it), more by sorting them and merging the two lists (eight
// rows of 128256 float32 logits, k = 64, 37 -> 31 us a call, 700 of 4000 40 ->
// 30).  The turns run over a whole batch at once, not over each vector (eight
// rows, k = 8, 13.5 -> 12.4).  Ids rise from batch to batch, so a later element
// that only ties the k-th value loses to it.
// ---------------------------------------------------------------------------
struct Best {
  uint64_t* buf;       // NS_WAVE candidates
  uint64_t key;        // this lane's
  int cnt, k;
  float least;         // elements below it cannot be among the k best
  bool fresh;          // nothing seen yet

  // Enters the keys c of the lanes of `ball`, each in turn: a ballot is the rank,
  // the lanes behind it shift.
  __device__ __forceinline__ void insert(unsigned long long ball, uint64_t c, int lane) {
#pragma unroll 1
    while (ball) {                                         // uniform
      const uint64_t o = lane_u64(c, __ffsll(ball) - 1);
      ball &= ball - 1;
      const int r = __popcll(__ballot(key > o));
      // wave_shr:1, the key of the lane before
      const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)key, 0x138, 0xf, 0xf, false);
      const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(key >> 32), 0x138, 0xf, 0xf, false);
      const uint64_t before = ((uint64_t)hi << 32) | lo;
      key = lane < r ? key : (lane == r ? o : before);
    }
  }

  // Empties the collected candidates into the list.
  __device__ __forceinline__ void enter(int lane) {
    wave_sync();
    uint64_t c = lane < cnt ? buf[lane] : 0;
    if (cnt <= 2) {                                        // uniform
      insert((1ull << cnt) - 1, c, lane);
    } else if (cnt > 16) {
      key = merge_lists(key, ns::shfl_xor_u64(sort_list(c, lane), NS_WAVE - 1), lane);
    } else {
      int rk = lane, rc = 0;                               // ranks of key and c
#pragma unroll 1
      for (int p = 0; p < cnt; p += 4)                     // those past cnt are 0, above nothing
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint64_t o = lane_u64(c, p + e);
          const int above = __popcll(__ballot(key > o));   // list keys above candidate p + e
          rk += key < o;
          rc += (c < o) + (lane == p + e ? above : 0);
        }
      wave_sync();
      buf[lane] = 0;
      wave_sync();
      if (key != 0 && rk < k) buf[rk] = key;
      if (lane < cnt && rc < k) buf[rc] = c;
      wave_sync();
      key = buf[lane];
    }
    wave_sync();
    cnt = 0;
  }

  // Bit u * EPV + e: element e of a lane's vector u reaches `least`.
  template <int ET>
  __device__ __forceinline__ uint32_t reach(const u32x4 (&x)[kUnroll], const float (&mx)[kUnroll], int q, int q1) const {
    constexpr int EPV = per_vec(ET);
    uint32_t m = 0;
#pragma unroll
    for (int u = kUnroll - 1; u >= 0; --u) {
      float v[EPV];
      widen<ET>(x[u], v);
      m <<= EPV;
      if (!__ballot(mx[u] >= least)) continue;             // uniform
      uint32_t part = 0;
#pragma unroll
      for (int e = EPV - 1; e >= 0; --e) part = part + part + (v[e] >= least ? 1u : 0u);
      m |= part;
    }
    // vectors past the end are of the part's last lanes and rounds
    const int n = (q1 - q + NS_WAVE - 1) / NS_WAVE;        // vectors of this lane, q its first
    return n >= kUnroll ? m : (n <= 0 ? 0u : m & ((1u << n * EPV) - 1));
  }

  // One turn: collects the lowest marked element of each lane.
  template <int ET>
  __device__ __forceinline__ void collect(const u32x4 (&x)[kUnroll], int q, uint32_t& m, unsigned long long ball, int lane) {
    constexpr int EPV = per_vec(ET);
    const int b = (__ffs(m) - 1) & (kUnroll * EPV - 1), word = ET == NS_FP32 ? b : b >> 1;
    uint32_t w[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t lo = word & 1 ? x[u].y : x[u].x, hi = word & 1 ? x[u].w : x[u].z;
      w[u] = word & 2 ? hi : lo;
    }
    const uint32_t lo = word & 4 ? w[1] : w[0], hi = word & 4 ? w[3] : w[2], v = word & 8 ? hi : lo;
    const float f = ET == NS_FP32 ? __uint_as_float(v) : elem_of<ET>(v >> (b & 1) * 16, 0);
    if (m != 0) buf[cnt + __popcll(ball & ((1ull << lane) - 1))] = ns::make_key(f, (q + b / EPV * NS_WAVE) * EPV + b % EPV);
    cnt += __popcll(ball);
    m &= m - 1;
  }

  // Takes what reaches `least` of a batch's vectors, q the lane's first.
  // Where that is more than the buffer holds (many equal or masked logits, a
  // first batch with a large k), lanes go in order of their ids, 64 elements at
  // a time, each group raising the bound for the next: a row of equal logits
  // costs one merge.
  template <int ET>
  __device__ __forceinline__ void take_batch(const u32x4 (&x)[kUnroll], const float (&mx)[kUnroll], int q, int q1, int lane) {
    constexpr int EPV = per_vec(ET), GROUP = NS_WAVE / EPV;
    uint32_t m = reach<ET>(x, mx, q, q1);
    bool fits = true;
#pragma unroll 1
    while (true) {
      const unsigned long long ball = __ballot(m != 0);
      if (!ball) break;
      fits = cnt + __popcll(ball) <= NS_WAVE;              // uniform
      if (!fits) break;
      collect<ET>(x, q, m, ball, lane);
    }
    if (!fits) cnt = 0;
    int u = fits ? kUnroll : 0, from = 0;                  // next: the lanes from `from` on of vector u
#pragma unroll 1
    while (true) {
      if (u < kUnroll) {
        m = lane >= from ? reach<ET>(x, mx, q, q1) & (((1u << EPV) - 1) << u * EPV) : 0u;
        const int n = __builtin_amdgcn_readlane(ns::wave_incl_scan(__popc(m), lane), NS_WAVE - 1);
        const bool all = cnt + n <= NS_WAVE;
        if (all || cnt == 0) {
          if (!all && lane >= from + GROUP) m = 0;
#pragma unroll 1
          while (true) {
            const unsigned long long ball = __ballot(m != 0);
            if (!ball) break;
            collect<ET>(x, q, m, ball, lane);
          }
          from = all ? 0 : (from + GROUP) & (NS_WAVE - 1);
          u += from == 0;
          if (all) continue;
        }
      }
      if (cnt > 0) enter(lane);
      raise();
      if (u == kUnroll) break;
    }
  }

  // The bound for the next batch.
  __device__ __forceinline__ void raise() {
    const uint32_t h = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(key >> 32), k - 1);
    if (h != 0) least = next_up(ns::unord_f32(h));
  }

  // A bound before any key is held, from the lanes' maxima m: a value that at
  // least k of them reach, by bisection of the ordered bits.  It ends within a
  // hundredth of the k-th largest; the exact one would save next to nothing.
  __device__ __forceinline__ void start(float m, int lane) {
    fresh = false;
    const uint32_t o = m == m ? ns::ord_f32(m) : 0u;       // NaN: no bound
    uint32_t lo = 0, hi = 0xFFFFFFFFu;                     // k lanes reach lo, fewer than k reach hi
    {
      const uint32_t top = (uint32_t)__builtin_amdgcn_readfirstlane((int)ns::ord_f32(ns::wave_max_f32(m)));
      hi = top + 1;
      // most maxima lie within a factor of four of the largest: begin there if k do
      const uint32_t near = top > (2u << 23) ? top - (2u << 23) : 0u;
      if (__popcll(__ballot(o >= near)) >= k) lo = near;
    }
#pragma unroll 1
    for (int i = lo != 0 ? 8 : 16; i > 0; --i) {
      const uint32_t mid = lo + (hi - lo) / 2;
      if (__popcll(__ballot(o >= mid)) >= k) lo = mid;
      else hi = mid;
    }
    if (lo >= 0x00800000u) least = ns::unord_f32(lo);      // the least finite value; below it -infinity does
  }
};

struct Args {
  const void* z;
  int64_t ld;
  int L, V, S, k, T;
  float t, c, eps;             // inverse temperature, times log2(e), and what rounding took from c, relatively
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
  float t, c, eps, ref, E, l2, lse, H;
  bool bad, none;
  __device__ __forceinline__ Row(const Stat& s, const Args& a) : t(a.t), c(a.c), eps(a.eps) {
    bad = !(s.S < INFINITY) || s.top == INFINITY;
    none = s.S == 0.f;
    const float nan = __uint_as_float(0x7FC00000u);
    ref = s.ref;
    E = s.E;
    // c (1 + eps) is what c stands for.  The sum's large terms have c z close
    // to E (c (z - ref) close to 0), so all of it is 2^(eps E) times as large.
    const float l = log2f(s.S);
    l2 = l + eps * E;
    lse = bad ? nan : (none ? -INFINITY : ref * t + kLn2 * (E + l2));
    H = bad ? nan : (none ? 0.f : fmaxf(kLn2 * (l - s.W / s.S), 0.f));
  }
  __device__ __forceinline__ float logp(float z) const {
    if (bad) return __uint_as_float(0x7FC00000u);
    if (none || z == -INFINITY) return -INFINITY;
    const float y0 = ref == 0.f ? fmaf(z, c, -E) : (z - ref) * c - E;
    const float y = y0 + eps * (y0 + E);
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
    if (top >= best.least) best.take_batch<ET>(x, mx, q0 + lane, q1, lane);   // uniform
  }
}

// Forward.  A wave owns part `part` of S of one row and streams it once with
// 16-byte loads, two register batches in turn.  Bound by its bytes over many
// rows (4096 x 128256 bf16 164 us, 6.4 TB/s; with k = 4 171 to 177), by the
// latency of the selection over few (8 x 128256 float32, both launches 7.6 us;
// with k = 8 12.4).
template <int ET, bool TOP>
__global__ __launch_bounds__(kRowWaves* NS_WAVE) void k_logprobs(Args a) {
  constexpr int EPV = per_vec(ET), STEP = NS_WAVE * kUnroll;
  __shared__ uint64_t sh[TOP ? kRowWaves : 1][NS_WAVE];
  const int lane = threadIdx.x & (NS_WAVE - 1), wv = threadIdx.x / NS_WAVE;
  const int64_t item = (int64_t)blockIdx.x * kRowWaves + wv;
  const size_t row = (size_t)(item / a.S);
  const int part = (int)(item % a.S);
  if (row >= (size_t)a.L) return;                          // wave-uniform; no block barrier below
  const char* zrow = (const char*)a.z + row * (size_t)a.ld * elem_bytes(ET);
  const int nvec = a.V / EPV;
  const int q0 = (int)((int64_t)nvec * part / a.S), q1 = (int)((int64_t)nvec * (part + 1) / a.S);
  Stat st{-INFINITY, 0.f, 0.f, 0.f, 0.f};
  Best best{sh[TOP ? wv : 0], 0, 0, a.k, -INFINITY, true};
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
#pragma unroll 1
  for (int base = q0; base < q1; base += STEP) {
    load(base + STEP, x1);
    NS_ISSUE_FENCE();
    mask(base, x0);
    take<ET, TOP>(x0, base, q1, a.c, st, best, lane);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) x0[u] = x1[u];
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
      best.insert(__ballot(live && v >= best.least), ns::make_key(v, e), lane);
    }
  } else {
    st.S = ns::wave_sum_f32(st.S);
    st.W = ns::wave_sum_f32(st.W);
  }
  const uint64_t key = best.key;
  if (a.S == 1) {
    const Row r(st, a);
    if (lane == 0) {
      a.lse[row] = r.lse;
      if (a.entropy) a.entropy[row] = r.H;
    }
    if (lane < a.T) put_tokens<ET>(a, r, row, lane);
    if (TOP && lane < a.k) put_top(a, r, row, lane, key);
  } else {
    if (lane == 0) a.stat[item] = st;
    if (TOP && lane < a.k) a.keys[item * a.k + lane] = key;
  }
}

// The same for four lists of 16, one in each row of lanes: every row ends with the 16 largest of all.
__device__ __forceinline__ uint64_t merge_rows(uint64_t x, int lane) {
#pragma unroll
  for (int m = 31; m <= 47; m += 16) {                     // the neighbour row, then the next pair's, in rising order
    const uint64_t o = ns::shfl_xor_u64(x, m);
    x = x > o ? x : o;
    x = exchange<8>(x, lane);
    x = exchange<4>(x, lane);
    x = exchange<2>(x, lane);
    x = exchange<1>(x, lane);
  }
  return x;
}

constexpr int kJoinLists = 4;            // parts' lists of a wave

// Joins the S parts of a row: JW waves (one up to four parts, 16 for more)
// merge the parts' lists, four each at most, then one another's; the last wave
// joins the statistics meanwhile.
// Takes the same time whatever the keys (a bound on the k-th best, as good as
// nothing where many logits tie, is not needed).  CAP is the length of the
// lists that are merged, 0 (no alternatives), 16 or 64: with 16 a wave holds
// four of them at once.
template <int ET, int CAP, int JW>
__global__ __launch_bounds__(JW* NS_WAVE) void k_logprobs_join(Args a) {
  constexpr bool TOP = CAP != 0;
  const size_t row = blockIdx.x;
  const int lane = threadIdx.x & (NS_WAVE - 1), wv = threadIdx.x / NS_WAVE;
  const bool joins = wv == JW - 1;
  __shared__ Stat all;
  // parts, keys and tokens are asked for together
  static_assert(16 * kJoinLists == kMaxParts, "16 waves hold every part's list");
  uint64_t list[kJoinLists] = {};
  int tok = -1;
  Stat st{-INFINITY, 0.f, 0.f, 0.f, 0.f};
  if (joins && lane < a.S) st = a.stat[row * a.S + lane];
  if (joins && lane < a.T) tok = a.tokens[row * a.T + lane];
  if (CAP == 16) {
    const int p = wv * 4 + lane / 16, q = lane % 16;
    if (p < a.S && q < a.k) list[0] = a.keys[(row * a.S + p) * a.k + q];
  }
  if (CAP == 64) {
#pragma unroll
    for (int i = 0; i < kJoinLists; ++i) {
      const int p = wv + i * JW, q = i == 0 ? lane : NS_WAVE - 1 - lane;
      if (p < a.S && q < a.k) list[i] = a.keys[(row * a.S + p) * a.k + q];
    }
  }
  NS_ISSUE_FENCE();
  float ztok = 0.f;
  const bool known = tok >= 0 && tok < a.V;
  if (known) ztok = one_elem<ET>(a.z, row * (size_t)a.ld + tok);
  __shared__ uint64_t sh[TOP && JW > 1 ? JW : 1][NS_WAVE];
  uint64_t best = list[0];
  if (CAP == 16) best = merge_rows(best, lane);
  if (CAP == 64) {
#pragma unroll
    for (int i = 1; i < kJoinLists; ++i)
      if (wv + i * JW < a.S) best = merge_lists(best, list[i], lane);
  }
  if (TOP && JW > 1) {
    sh[wv][lane] = best;
    __syncthreads();
  }
  if (joins) {
    for (int m = 1; m < a.S; m <<= 1) {
      Stat o;
      o.top = __shfl_xor(st.top, m, NS_WAVE);
      o.ref = __shfl_xor(st.ref, m, NS_WAVE);
      o.E = __shfl_xor(st.E, m, NS_WAVE);
      o.S = __shfl_xor(st.S, m, NS_WAVE);
      o.W = __shfl_xor(st.W, m, NS_WAVE);
      st = lane & m ? join(o, st, a.c) : join(st, o, a.c);   // the lower part first in both lanes
    }
    st.top = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(st.top)));
    st.ref = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(st.ref)));
    st.E = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(st.E)));
    st.S = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(st.S)));
    st.W = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(st.W)));
    const Row r(st, a);
    if (TOP && JW == 1 && lane < a.k) put_top(a, r, row, lane, best);
    if (lane == 0) {
      all = st;
      a.lse[row] = r.lse;
      if (a.entropy) a.entropy[row] = r.H;
    }
    if (lane < a.T) a.logprob[row * a.T + lane] = known ? r.logp(ztok) : 0.f;
  }
  if (CAP == 16 && JW > 1) {
    if (wv < 4) best = merge_rows(sh[wv * 4 + lane / 16][lane % 16], lane);
    __syncthreads();
    if (wv < 4) sh[wv][lane] = best;
    __syncthreads();
    if (wv == 0) {
      best = merge_rows(sh[lane / 16][lane % 16], lane);
      if (lane < a.k) put_top(a, Row(all, a), row, lane, best);
    }
  }
  if (CAP == 64 && JW > 1) {
#pragma unroll
    for (int m = JW / 2; m >= 1; m >>= 1) {
      if (wv < m && wv + m < a.S) {                        // wave m .. 2 m - 1 holds something
        best = merge_lists(best, sh[wv + m][NS_WAVE - 1 - lane], lane);
        sh[wv][lane] = best;
      }
      __syncthreads();
    }
    if (wv == 0 && lane < a.k) put_top(a, Row(all, a), row, lane, best);
  }
}

// Parts of a row: doubled until about kWavesWanted waves (three quarters of
// them at least) run, each with a batch at least, from 512 rows on with two.
// 1500 rows of 128256 bf16 logits, k = 4: 76 us in two parts, 89 in one; 1000
// of 50257 33 in two, 34 in four; 1023 of 4000 9.4 in one, 11.1 in two.
int parts_of(int L, int V, int dtype) {
  const int batch = NS_WAVE * kUnroll * per_vec(dtype) * (L < 512 ? 1 : 2);
  const int most = (V + batch - 1) / batch;
  int s = 1;
  while ((int64_t)s * L * 4 < kWavesWanted * 3 && s * 2 <= most && s < kMaxParts) s *= 2;
  return s;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Room for the parts of L rows or any fewer, so that the largest call's
// workspace fits a loop's smaller ones: a row has at most the parts of a single
// one (of float32, which has the smallest batches), and rows in parts come to
// less than 3/2 kWavesWanted of them together.
size_t logprobs_ws(int L, int V, int k) {
  const size_t l = (size_t)(L > 0 ? L : 1), most = l * (size_t)parts_of(1, V, NS_FP32);
  const size_t split = most < kWavesWanted * 3 / 2 ? most : kWavesWanted * 3 / 2, n = l > split ? l : split;
  return align256(n * sizeof(Stat)) + align256(n * (size_t)k * 8) + 256;
}

template <int ET>
void launch_logprobs(const Args& a, hipStream_t stream) {
  const dim3 grid((unsigned)(((int64_t)a.L * a.S + kRowWaves - 1) / kRowWaves)), block(kRowWaves * NS_WAVE);
  if (a.k > 0) hipLaunchKernelGGL((k_logprobs<ET, true>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((k_logprobs<ET, false>), grid, block, 0, stream, a);
  if (a.S == 1) return;
  const dim3 rows((unsigned)a.L);
  const bool one = a.S <= kJoinLists;
  if (a.k == 0) hipLaunchKernelGGL((k_logprobs_join<ET, 0, 1>), rows, dim3(NS_WAVE), 0, stream, a);
  else if (a.k <= 16 && one) hipLaunchKernelGGL((k_logprobs_join<ET, 16, 1>), rows, dim3(NS_WAVE), 0, stream, a);
  else if (a.k <= 16) hipLaunchKernelGGL((k_logprobs_join<ET, 16, 16>), rows, dim3(16 * NS_WAVE), 0, stream, a);
  else if (one) hipLaunchKernelGGL((k_logprobs_join<ET, 64, 1>), rows, dim3(NS_WAVE), 0, stream, a);
  else hipLaunchKernelGGL((k_logprobs_join<ET, 64, 16>), rows, dim3(16 * NS_WAVE), 0, stream, a);
}

// ---------------------------------------------------------------------------
// Gradient.  With g_t of the tokens' log-probabilities, g_H of the entropy
// and g_l of the log-sum-exp, and G = g_l - sum_t g_t:
//     dz_j = t (p_j (G - g_H (logp_j + H)) + sum_t g_t [token_t = j]).
// With y_j = log2 p_j the first part is p_j (A + B y_j), A = t (G - g_H H),
// B = -t g_H ln2.  log2(e) lse is taken in two floats; the small one goes
// into A, B and a common factor.
//
// lse is a float32 and half a step of it passes into every p_j: 2^-15 at 1024,
// 2^-5 at 10^6 (shifted logits, a row with nothing but fp16's lowest value as a
// mask).  Beyond kNear one of the row's blocks takes the whole row, sums
// 2^(c (z_j - ref)) itself, ref = lse / t (next to lse those differences are
// exact), and takes y_j = c (z_j - ref) - log2 of the sum.  It has read the
// whole row before it writes any of it, so dlogits may be logits there too.
// Which of them rises with the row, so that all XCDs take part (4096 x 128256
// bf16, every row such a one: 623 us, 4030 with the first block of each; one
// float32 row of 128256: 48).
// ---------------------------------------------------------------------------
struct GradArgs {
  const void* z;
  int64_t ld;
  int L, V, T;
  float t, c, eps;             // as in Args
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

constexpr float kNear = 1024.f;          // |lse| up to which probabilities come from lse itself
constexpr float kFar = 0x1p24f;          // |lse| beyond which a row's gradient is 0

struct Slope {
  float c, ref, L, A, B;
  bool zero;
  // p (A + B y) of a logit
  __device__ __forceinline__ float at(float z) const {
    const float y = fmaf(z - ref, c, -L);
    return exp2_fast(y) * fmaf(B, fmaxf(y, -200.f), A);
  }
};

// Sum of 2^(c (z_j - ref)) over a row, by all threads of a block in the same
// order each time; a batch is summed by itself first.
template <int ET>
__device__ __forceinline__ float sum_of_row(const char* zrow, int V, float ref, float c, float* sh) {
  constexpr int EPV = per_vec(ET);
  const int tid = threadIdx.x, nvec = V / EPV, tail = nvec * EPV + tid;
  float S = tail < V ? exp2_fast((one_elem<ET>(zrow, tail) - ref) * c) : 0.f;
  constexpr int U = 8;
  for (int base = 0; base < nvec; base += kGradThreads * U) {
    u32x4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int q = base + u * kGradThreads + tid;
      x[u] = *(const u32x4_any*)(zrow + (size_t)(q < nvec ? q : 0) * 16);
    }
    NS_ISSUE_FENCE();
    float batch = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float v[EPV], part = 0.f;
      widen<ET>(x[u], v);
#pragma unroll
      for (int e = 0; e < EPV; ++e) part += exp2_fast((v[e] - ref) * c);
      batch += base + u * kGradThreads + tid < nvec ? part : 0.f;
    }
    S += batch;
  }
  S = ns::wave_sum_f32(S);
  if ((tid & (NS_WAVE - 1)) == 0) sh[tid / NS_WAVE] = S;
  __syncthreads();
  S = sh[0];
#pragma unroll
  for (int w = 1; w < kGradThreads / NS_WAVE; ++w) S += sh[w];
  return S;
}

// One pass, bound by its bytes (4096 x 128256 bf16 353 us, 5.95 TB/s read and
// written).  dlogits may be logits: a block reads its part of the row, and the
// logits of the tokens in it, before it writes them.
template <int ET>
__global__ __launch_bounds__(kGradThreads, 8) void k_logprobs_grad(GradArgs a, int per, int chunks) {
  constexpr int EPV = per_vec(ET);
  __shared__ int32_t s_tok[NS_MAX_K];
  __shared__ float s_g[NS_MAX_K];
  __shared__ float s_sum[kGradThreads / NS_WAVE];
  const size_t row = blockIdx.x / (unsigned)chunks;
  const int chunk = (int)(blockIdx.x % (unsigned)chunks);
  const int tid = threadIdx.x, lane = tid & (NS_WAVE - 1);
  const char* zrow = (const char*)a.z + row * (size_t)a.ld * elem_bytes(ET);
  char* drow = (char*)a.dz + row * (size_t)a.ld_d * elem_bytes(ET);
  const int nvec = a.V / EPV;
  int q0 = chunk * per;
  int q1 = q0 + per < nvec ? q0 + per : nvec;
  bool last = chunk + 1 == chunks;
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
  s.zero = fabsf(lse) > kFar;
  s.ref = 0.f;
  s.L = lse * kLog2e;
  // (c z is close to L wherever p is not small, so c's own rounding is eps L)
  float low = (float)((double)lse * 1.4426950408889634 - (double)s.L) - a.eps * s.L;
  if (fabsf(lse) > kNear && !s.zero) {                     // uniform over the row's blocks
    if (chunk != (int)(row % (unsigned)chunks)) return;
    q0 = 0;
    q1 = nvec;
    last = true;
    s.ref = lse / a.t;
    s.L = log2f(sum_of_row<ET>(zrow, a.V, s.ref, a.c, s_sum));
    low = 0.f;
  }
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
  int per = kGradThreads * kGradUnroll, chunks = nvec > 0 ? (nvec + per - 1) / per : 1;
  while (chunks > 1 && (int64_t)chunks * a.L > 1 << 22) {  // far from a launch's 2^32 threads
    per *= 2;
    chunks = (nvec + per - 1) / per;
  }
  hipLaunchKernelGGL(k_logprobs_grad<ET>, dim3((unsigned)chunks * (unsigned)a.L), dim3(kGradThreads), 0,
                     stream, a, per, chunks);
}

constexpr int64_t kMaxLd = (int64_t)1 << 40;

bool known_dtype(int t) { return t == NS_BF16 || t == NS_FP32 || t == NS_FP16; }
bool elem_aligned(const void* p, int dtype) { return ((uintptr_t)p) % (dtype == NS_FP32 ? 4 : 2) == 0; }
// NaN fails both comparisons
bool temp_ok(float t) { return t >= NS_MIN_INV_TEMP && t <= NS_MAX_INV_TEMP; }
bool dims_ok(int L, int64_t ld, int V, int T) {
  return L >= 0 && L <= NS_MAX_ROWS && V >= 1 && V <= NS_MAX_V && ld >= V && ld <= kMaxLd && T >= 0 && T <= NS_MAX_K;
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
  a.eps = (float)((double)inv_temp * 1.4426950408889634 / a.c - 1.0);
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
  if (!dims_ok(L, ld, V, T) || ld_d < V || ld_d > kMaxLd || !temp_ok(inv_temp)) return NS_EINVAL;
  if (L == 0) return NS_OK;
  if (!logits || !lse || !dlogits || (T > 0 && (!tokens || !g_logprob)) || (g_entropy && !entropy)) return NS_EINVAL;
  if (!elem_aligned(logits, dtype) || !elem_aligned(dlogits, dtype)) return NS_EINVAL;
  if (dlogits == logits && ld_d != ld) return NS_EINVAL;
  (void)hipGetLastError();
  const float c = (float)((double)inv_temp * 1.4426950408889634);
  const GradArgs a{logits, ld, L, V, T, inv_temp, c, (float)((double)inv_temp * 1.4426950408889634 / c - 1.0), tokens,
                   lse, entropy, g_logprob, g_entropy, g_lse, dlogits, ld_d};
  if (dtype == NS_BF16) launch_grad<NS_BF16>(a, stream);
  else if (dtype == NS_FP16) launch_grad<NS_FP16>(a, stream);
  else launch_grad<NS_FP32>(a, stream);
  return ns_launch_status();
}

}  // extern "C"
