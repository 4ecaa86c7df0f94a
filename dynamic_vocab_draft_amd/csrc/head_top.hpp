// The selection of the restricted heads over quantised rows: top-k over the logits that a product left in a workspace.
#pragma once
#include "common.hpp"
#include "select.hpp"

namespace {

// ---------------------------------------------------------------------------
// Top-k over the scaled logits of each hidden row
// ---------------------------------------------------------------------------
// Columns of a thread: 4 cover 4096 columns in one block; 16, for more, cover
// 16384 (64 x 15500: 11.5 us in chunks of 4096 with a join, 7.8 us in one).
constexpr int top_cols(int n_max) { return n_max <= 4 * kSelectThreads ? 4 : 16; }
constexpr int top_chunk(int n_max) { return kSelectThreads * top_cols(n_max); }

struct Top {
  const float* z;           // [B][M] rows, ld floats apart
  int64_t ld;
  const int32_t* ids;
  const int32_t* n_dev;
  int n_max, V, M, k;
  float* logits;            // [B][M][n_max] or NULL
  int32_t* out_ids;
  float* out_vals;
  uint64_t* cand;           // [B][M][chunks][k]
};

__device__ __forceinline__ void put_top(const Top& t, size_t row, int r, uint64_t key) {
  t.out_ids[row * t.k + r] = key ? ns::key_id(key) : -1;
  t.out_vals[row * t.k + r] = key ? ns::key_val(key) : -INFINITY;
}

// Block (m, c, b): the k best of chunk c of hidden row m of sequence b.
template <int U>
__global__ __launch_bounds__(kSelectThreads) void k_top_chunk(Top t) {
  constexpr int CHUNK = U * kSelectThreads;
  __shared__ SelectSmem sm;
  const int m = blockIdx.x, c = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const size_t row = (size_t)b * t.M + m;
  const int j0 = c * CHUNK;
  int n = t.n_dev ? t.n_dev[b] : t.n_max;
  // Every column is asked for before the first is looked at; the first four of
  // a thread together with the count, live or not.
  float val[U];
  int id[U];
  const auto ask = [&](int u, int end) {
    const int q = j0 + tid + u * kSelectThreads, j = q < end ? q : end - 1;
    val[u] = t.z[row * (size_t)t.ld + j];
    id[u] = t.ids ? t.ids[(size_t)b * t.n_max + j] : j;
  };
#pragma unroll
  for (int u = 0; u < 4; ++u) ask(u, t.n_max);
  NS_ISSUE_FENCE();
  n = n < 0 ? 0 : (n > t.n_max ? t.n_max : n);
  const bool final_here = n <= CHUNK;
  if (final_here && c > 0) return;
  const int lim = n - j0 < CHUNK ? n - j0 : CHUNK;       // <= 0 where nothing is live
  if (U > 4) {
    const int end = n > 0 ? n : 1;
#pragma unroll
    for (int u = 4; u < U; ++u) ask(u, end);
    NS_ISSUE_FENCE();
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int q = tid + u * kSelectThreads;
    const bool live = q < lim && id[u] >= 0 && id[u] < t.V;
    if (live && t.logits) t.logits[row * (size_t)t.n_max + j0 + q] = val[u];
    if (!live || val[u] != val[u]) {                     // NaN is never selected
      val[u] = 0.f;
      id[u] = -1;
    }
  }
  const int nlive = lim > 0 ? lim : 0;
  if (final_here)
    block_select_topk<U>(val, id, t.k, nlive, sm, [&](int r, uint64_t x) { put_top(t, row, r, x); });
  else {
    uint64_t* dst = t.cand + (row * gridDim.y + c) * (size_t)t.k;
    block_select_topk<U>(val, id, t.k, nlive, sm, [&](int r, uint64_t x) { dst[r] = x; });
  }
}

// Block (m, b): the k best of the nk = chunks * k keys of its chunks.
template <int U>
__global__ __launch_bounds__(kSelectThreads) void k_top_keys(Top t, int nk) {
  __shared__ SelectSmem sm;
  const int m = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  int n = t.n_dev ? t.n_dev[b] : t.n_max;
  if (n > t.n_max) n = t.n_max;
  if (n <= top_chunk(t.n_max)) return;
  const size_t row = (size_t)b * t.M + m;
  float val[U];
  int id[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int q = tid + u * kSelectThreads;
    const uint64_t key = q < nk ? t.cand[row * nk + q] : 0;
    val[u] = key ? ns::key_val(key) : 0.f;
    id[u] = key ? ns::key_id(key) : -1;
  }
  block_select_topk<U>(val, id, t.k, nk, sm, [&](int r, uint64_t x) { put_top(t, row, r, x); });
}

// The whole selection: one launch, or two where the columns take several chunks.
int launch_top(const Top& t, int chunks, int B, hipStream_t stream) {
  const dim3 grid((unsigned)t.M, (unsigned)chunks, (unsigned)B);
  if (top_cols(t.n_max) == 4) hipLaunchKernelGGL(k_top_chunk<4>, grid, dim3(kSelectThreads), 0, stream, t);
  else hipLaunchKernelGGL(k_top_chunk<16>, grid, dim3(kSelectThreads), 0, stream, t);
  const int rc = ns_launch_status();
  if (rc != NS_OK || chunks == 1) return rc;
  const int nk = chunks * t.k;
  const dim3 rows((unsigned)t.M, (unsigned)B), block(kSelectThreads);
  static_assert((NS_MAX_V + top_chunk(NS_MAX_V) - 1) / top_chunk(NS_MAX_V) * NS_MAX_K <= 4 * kSelectThreads,
                "k_top_keys<4> holds every chunk's keys");
  if (nk <= kSelectThreads) hipLaunchKernelGGL(k_top_keys<1>, rows, block, 0, stream, t, nk);
  else hipLaunchKernelGGL(k_top_keys<4>, rows, block, 0, stream, t, nk);
  return ns_launch_status();
}

}  // namespace
