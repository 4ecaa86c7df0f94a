// Host-side memory and undefined-behaviour checks of the 8-bit rows and the
// token log-probabilities (quant.hip, logprob.hip), built with
// AddressSanitizer and UndefinedBehaviorSanitizer on their host code by
// tests/test_sanitizers_target.py and run on a machine WITHOUT a GPU: size
// queries over edge and out-of-range arguments, argument errors, and calls
// that pass the checks with placeholder device addresses, so that the host
// planning runs for every shape class and stops at the first HIP call
// (NS_EHIP).  The addresses are never dereferenced on the host.
#include <stdint.h>
#include <stdio.h>

#include "nanospec.h"

#define CHECK(c)                                                            \
  do {                                                                      \
    if (!(c)) {                                                             \
      fprintf(stderr, "%s:%d: check failed: %s\n", __FILE__, __LINE__, #c); \
      return 1;                                                             \
    }                                                                       \
  } while (0)

namespace {

void* fake(uintptr_t i) { return (void*)(uintptr_t)(0x100000u + 0x1000u * i); }

int check_sizes() {
  const int32_t Ds[] = {INT32_MIN, -1, 0, 1, 127, 128, 129, 4096, NS_MAX_D, NS_MAX_D + 1, INT32_MAX};
  for (int32_t d : Ds) {
    const int32_t p = nanospec_quant_pitch(d);
    CHECK((d < 1 || d > NS_MAX_D) ? p == 0 : (p >= d && p < d + 128 && p % 128 == 0));
  }
  const int32_t Bs[] = {INT32_MIN, 0, 1, 8, NS_MAX_BATCH, NS_MAX_BATCH + 1, INT32_MAX};
  const int32_t Ns[] = {INT32_MIN, 0, 1, 4096, 4097, 16384, 16385, NS_MAX_V, NS_MAX_V + 1, INT32_MAX};
  const int32_t Ms[] = {-1, 0, 1, 16, 64, 65, INT32_MAX};
  const int32_t Ks[] = {-1, 0, 1, 16, 64, 65, INT32_MAX};
  for (int32_t B : Bs)
    for (int32_t n : Ns)
      for (int32_t M : Ms)
        for (int32_t k : Ks)
          for (int32_t d : Ds) {
            const bool ok = B >= 1 && B <= NS_MAX_BATCH && n >= 1 && n <= NS_MAX_V && M >= 1 && M <= NS_MAX_M &&
                            k >= 1 && k <= NS_MAX_K && d >= 1 && d <= NS_MAX_D;
            const size_t w = nanospec_quant_logits_workspace_bytes(B, n, M, k, d);
            CHECK(ok ? (w % 256 == 0 && w >= (size_t)B * M * n * 4) : w == 0);
          }
  const int32_t Ls[] = {INT32_MIN, -1, 0, 1, 60, 511, 512, 2048, NS_MAX_ROWS, NS_MAX_ROWS + 1, INT32_MAX};
  for (int32_t L : Ls)
    for (int32_t V : Ns)
      for (int32_t k : Ks) {
        const bool ok = L >= 0 && L <= NS_MAX_ROWS && V >= 1 && V <= NS_MAX_V && k >= 0 && k <= NS_MAX_K && k <= V;
        CHECK((nanospec_token_logprobs_workspace_bytes(L, V, k) > 0) == ok);
      }
  return 0;
}

int check_plans() {
  int8_t *q = (int8_t*)fake(0), *w = (int8_t*)fake(1);
  float *s = (float*)fake(2), *t = (float*)fake(3);
  int32_t* ids = (int32_t*)fake(4);
  for (int32_t dtype : {NS_BF16, NS_FP16, NS_FP32}) {
    for (int32_t R : {1, 1023, 1024, NS_MAX_ROWS})
      for (int32_t d : {1, 512, 513, 2048, 4096, 4097, 8193, NS_MAX_D})
        CHECK(nanospec_quant_rows(fake(5), d, R, d, dtype, q, s, nullptr) == NS_EHIP);
    for (int32_t M : {1, 16, 17, 33, 49, 64, 65, 128, 129, NS_MAX_ROWS})
      for (int32_t N : {1, 64, 65, 4096, 4097, 16384, 16385, NS_MAX_V})
        for (int64_t pad : {(int64_t)0, (int64_t)1 << 39})
          CHECK(nanospec_quant_matmul(q, s, M, w, t, N, NS_MAX_D, fake(6), N + pad, dtype, nullptr) == NS_EHIP);
    for (int32_t B : {1, 3, NS_MAX_BATCH})
      for (int32_t n : {1, 4096, 4097, 16384, 16385, NS_MAX_V})
        for (int32_t M : {1, 17, 33, 64})
          for (int32_t d : {8, 4096, NS_MAX_D}) {
            const size_t need = nanospec_quant_logits_workspace_bytes(B, n, M, 64, d);
            CHECK(nanospec_quant_logits_topk(w, t, ids, ids, n, B, NS_MAX_V, d, fake(6), dtype, M, 64, nullptr, ids,
                                             s, fake(7), need, nullptr) == NS_EHIP);
            CHECK(nanospec_quant_logits_topk(w, t, ids, ids, n, B, NS_MAX_V, d, fake(6), dtype, M, 64, nullptr, ids,
                                             s, fake(7), need - 1, nullptr) == NS_ECAPACITY);
          }
    for (int32_t L : {1, 8, 511, 512, 1536, 2048, NS_MAX_ROWS})
      for (int32_t V : {1, 7, 2048, 128256, NS_MAX_V})
        for (int32_t k : {0, 1, 16, 64}) {
          if (k > V) continue;
          const size_t need = nanospec_token_logprobs_workspace_bytes(L, V, k);
          CHECK(nanospec_token_logprobs(fake(5), V, L, V, dtype, 1.f, ids, 64, k, s, t, s, ids, t, fake(7), need,
                                        nullptr) == NS_EHIP);
          CHECK(nanospec_token_logprobs(fake(5), V, L, V, dtype, 1.f, ids, 64, k, s, t, s, ids, t, fake(7), 0,
                                        nullptr) == NS_ECAPACITY);
          CHECK(nanospec_token_logprobs_grad(fake(5), V, L, V, dtype, 1.f, ids, 64, s, t, s, t, t, fake(8), V,
                                             nullptr) == NS_EHIP);
        }
  }
  return 0;
}

}  // namespace

int main() {
  if (check_sizes()) return 1;
  if (check_plans()) return 1;
  printf("target host checks passed\n");
  return 0;
}
