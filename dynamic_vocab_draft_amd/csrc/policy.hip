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
// line is 2^y_j (A + B y_j) off the token.  What stands once a row (logp_a and
// all that follows from it) is computed in float64: a ratio is as exact as S.
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
};

constexpr double kUnseen = -104.0;       // a log-probability below this is that of a probability 0 in float32

// What a row's gradient needs: 2^y (A + B y), and G more at the token.
struct Slope {
  float ref, E, A, B, G;
};

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

// A row's outputs and slope from its statistics and its token's logit.
__device__ __forceinline__ Slope finish(const Args& a, size_t row, const Stat& s, float ztok, float w, bool writes) {
  const double kLn2d = 0.69314718055994530942;
  const bool bad = !(s.S < INFINITY) || s.top == INFINITY, none = s.S == 0.f;
  Slope r{s.ref, s.E, 0.f, 0.f, 0.f};
  double logp = 0.0, kl = 0.0, loss = 0.0;
  float H = 0.f;
  if (bad) {
    logp = kl = loss = __longlong_as_double(0x7FF8000000000000ll);
    H = r.A = r.B = r.G = (float)logp;
  } else {
    // c (1 + eps) is what c stands for; the sum's large terms have c z close to E
    const double l = none ? 0.0 : log2((double)s.S) + (double)a.eps * s.E;
    const double y = ((double)ztok - s.ref) * ((double)a.c * (1.0 + (double)a.eps)) - s.E;
    logp = none ? -INFINITY : kLn2d * (y - l);
    H = none ? 0.f : fmaxf((float)(kLn2d * (log2((double)s.S) - (double)s.W / s.S)), 0.f);
    if (logp > kUnseen) {
      const double adv = a.advantage[row], ratio = exp(logp - (double)a.old[row]);
      const double lo = 1.0 - (double)a.eps_low, hi = 1.0 + (double)a.eps_high;
      const double held = ratio < lo ? lo : (ratio > hi ? hi : ratio), gain = ratio * adv, most = held * adv;
      const bool clipped = gain > most;                    // not where one of them is NaN
      double g = clipped ? 0.0 : -gain;
      loss = clipped ? -most : -gain;
      if (a.ref) {
        const double delta = (double)a.ref[row] - logp, e = expm1(delta);
        kl = e - delta;
        if (a.beta != 0.f) {
          loss += (double)a.beta * kl;
          g -= (double)a.beta * e;
        }
      }
      loss = (double)w * (loss - (double)a.c_ent * H);
      const double up = (a.g_loss ? (double)*a.g_loss : 1.0) * (double)a.t, over = up / s.S * (double)w, ent = a.c_ent;
      r.G = (float)(up * (double)w * g);
      r.A = (float)(over * (ent * ((double)H - kLn2d * l) - g));
      r.B = (float)(over * ent * kLn2d);
    }
  }
  if (writes) {
    a.logprob[row] = (float)logp;
    if (a.kl) a.kl[row] = (float)kl;
    if (a.entropy) a.entropy[row] = H;
    a.row_loss[row] = loss;
  }
  return r;
}

// The gradient of one element.
__device__ __forceinline__ float slope_at(const Slope& s, float c, float z) {
  const float y = s.ref == 0.f ? fmaf(z, c, -s.E) : (z - s.ref) * c;
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

constexpr int kRowThreads = 512;

// A block takes a row: its statistics, its outputs, and, where there is a
// gradient, the row again.
template <int ET>
__global__ __launch_bounds__(kRowThreads) void k_policy_row(Args a) {
  constexpr int EPV = per_vec(ET), STEP = NS_WAVE * kUnroll, NW = kRowThreads / NS_WAVE;
  __shared__ Stat sh[NW];
  const size_t row = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & (NS_WAVE - 1), wv = tid / NS_WAVE;
  const char* zrow = (const char*)a.z + row * (size_t)a.ld * elem_bytes(ET);
  char* drow = (char*)a.dz + row * (size_t)a.ld_d * elem_bytes(ET);
  const int nvec = a.V / EPV, tail = nvec * EPV + tid;
  int tok;
  float w;
  if (!taken(a, row, tok, w)) {                            // uniform
    if (tid == 0) put_nothing(a, row);
    if (a.dz) {
      for (int q = tid; q < nvec; q += kRowThreads) *(u32x4_any*)(drow + (size_t)q * 16) = u32x4{0, 0, 0, 0};
      if (tail < a.V) put_elem<ET>(drow, tail, 0.f);
    }
    return;
  }
  const float ztok = one_elem<ET>(zrow, tok);
  Stat st{-INFINITY, 0.f, 0.f, 0.f, 0.f};
  for (int base = wv * STEP; base < nvec; base += NW * STEP) {
    u32x4 x[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int q = base + u * NS_WAVE + lane;
      x[u] = *(const u32x4_any*)(zrow + (size_t)(q < nvec ? q : nvec - 1) * 16);
      if (q >= nvec) x[u] = minus_inf<ET>();
    }
    float mx[kUnroll], lane_max;
    add_batch<ET>(x, a.c, st, mx, lane_max);
  }
  st.S = ns::wave_sum_f32(st.S);
  st.W = ns::wave_sum_f32(st.W);
  if (wv == 0 && nvec * EPV < a.V)
    st = join(st, stat_of_lanes(tail < a.V ? one_elem<ET>(zrow, tail) : -INFINITY, a.c), a.c);
  if (lane == 0) sh[wv] = st;
  __syncthreads();
  st = sh[0];
#pragma unroll
  for (int i = 1; i < NW; ++i) st = join(st, sh[i], a.c);
  const Slope s = finish(a, row, st, ztok, w, tid == 0);
  if (!a.dz) return;
  for (int q = tid; q < nvec; q += kRowThreads) {
    float v[EPV];
    widen<ET>(*(const u32x4_any*)(zrow + (size_t)q * 16), v);
#pragma unroll
    for (int e = 0; e < EPV; ++e) v[e] = slope_at(s, a.c, v[e]) + (q * EPV + e == tok ? s.G : 0.f);
    *(u32x4_any*)(drow + (size_t)q * 16) = narrow<ET>(v);
  }
  if (tail < a.V) put_elem<ET>(drow, tail, slope_at(s, a.c, one_elem<ET>(zrow, tail)) + (tail == tok ? s.G : 0.f));
}

// The sum of the rows' losses, in the same order each time.
constexpr int kTotalThreads = 1024;

__global__ __launch_bounds__(kTotalThreads) void k_policy_total(const double* __restrict__ row_loss, int L,
                                                                float* __restrict__ loss) {
  __shared__ double sh[kTotalThreads / NS_WAVE];
  const int tid = threadIdx.x;
  double s = 0.0;
  for (int i = tid; i < L; i += kTotalThreads) s += row_loss[i];
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) s += __shfl_xor(s, m, NS_WAVE);
  if ((tid & (NS_WAVE - 1)) == 0) sh[tid / NS_WAVE] = s;
  __syncthreads();
  if (tid != 0) return;
  s = 0.0;
  for (int i = 0; i < kTotalThreads / NS_WAVE; ++i) s += sh[i];
  *loss = (float)s;
}

template <int ET>
void launch_policy(const Args& a, hipStream_t stream) {
  hipLaunchKernelGGL(k_policy_row<ET>, dim3((unsigned)a.L), dim3(kRowThreads), 0, stream, a);
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

size_t policy_ws(int L, int V) {
  (void)V;
  return align256((size_t)(L > 0 ? L : 1) * 8);
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
  const Args a{logits, ld, L, V, inv_temp, c, (float)((double)inv_temp * 1.4426950408889634 / c - 1.0), tokens,
               old_logprob, ref_logprob, advantage, weight, eps_low, eps_high, kl_coef, ent_coef, logprob, kl, entropy,
               g_loss, dlogits, ld_d, (double*)ws};
  if (L > 0) {
    if (dtype == NS_BF16) launch_policy<NS_BF16>(a, stream);
    else if (dtype == NS_FP16) launch_policy<NS_FP16>(a, stream);
    else launch_policy<NS_FP32>(a, stream);
    const int rc = ns_launch_status();
    if (rc != NS_OK) return rc;
  }
  hipLaunchKernelGGL(k_policy_total, dim3(1), dim3(kTotalThreads), 0, stream, (const double*)a.row_loss, L, loss);
  return ns_launch_status();
}

}  // extern "C"
