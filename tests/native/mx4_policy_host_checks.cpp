// Host-side memory and undefined-behaviour checks of the 4-bit rows and the
// policy loss (mx4.hip, policy.hip), built with AddressSanitizer and
// UndefinedBehaviorSanitizer on their host code by
// tests/test_sanitizers_mx4_policy.py and run on a machine WITHOUT a GPU: size
// queries over edge and out-of-range arguments, argument errors, and calls
// that pass the checks with placeholder device addresses, so that the host
// planning runs for every shape class and stops at the first HIP call
// (NS_EHIP).  The addresses are never dereferenced on the host.
#include <math.h>
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
  const int32_t Ds[] = {INT32_MIN, -1, 0, 1, 255, 256, 257, 4096, NS_MAX_D, NS_MAX_D + 1, INT32_MAX};
  for (int32_t d : Ds) {
    const int32_t p = nanospec_mx4_pitch(d);
    CHECK((d < 1 || d > NS_MAX_D) ? p == 0 : (2 * p >= d && 2 * p < d + 256 && p % 128 == 0));
  }
  const int32_t Bs[] = {INT32_MIN, 0, 1, 8, NS_MAX_BATCH, NS_MAX_BATCH + 1, INT32_MAX};
  const int32_t Ns[] = {INT32_MIN, 0, 1, 4096, 4097, 16384, 16385, NS_MAX_V, NS_MAX_V + 1, INT32_MAX};
  const int32_t Ms[] = {-1, 0, 1, 16, 64, 65, INT32_MAX};
  for (int32_t B : Bs)
    for (int32_t n : Ns)
      for (int32_t M : Ms)
        for (int32_t k : Ms)
          for (int32_t d : Ds) {
            const bool ok = B >= 1 && B <= NS_MAX_BATCH && n >= 1 && n <= NS_MAX_V && M >= 1 && M <= NS_MAX_M &&
                            k >= 1 && k <= NS_MAX_K && d >= 1 && d <= NS_MAX_D;
            const size_t w = nanospec_mx4_logits_workspace_bytes(B, n, M, k, d);
            CHECK(ok ? (w % 256 == 0 && w >= (size_t)B * M * n * 4) : w == 0);
          }
  const int32_t Ls[] = {INT32_MIN, -1, 0, 1, 60, 95, 96, 512, 2048, NS_MAX_ROWS, NS_MAX_ROWS + 1, INT32_MAX};
  for (int32_t L : Ls)
    for (int32_t V : Ns) {
      const bool ok = L >= 0 && L <= NS_MAX_ROWS && V >= 1 && V <= NS_MAX_V;
      CHECK((nanospec_policy_loss_workspace_bytes(L, V) > 0) == ok);
    }
  return 0;
}

int check_plans() {
  uint8_t *q = (uint8_t*)fake(0), *w = (uint8_t*)fake(1), *s = (uint8_t*)fake(2), *t = (uint8_t*)fake(3);
  float *f = (float*)fake(4), *g = (float*)fake(5);
  int32_t* ids = (int32_t*)fake(6);
  for (int32_t dtype : {NS_BF16, NS_FP16, NS_FP32}) {
    for (int32_t R : {1, 1023, 131072, NS_MAX_ROWS})
      for (int32_t d : {1, 256, 257, 4097, NS_MAX_D}) {
        CHECK(nanospec_mx4_rows(fake(7), d, R, d, dtype, q, s, nullptr) == NS_EHIP);
        for (const int32_t* at : {(const int32_t*)nullptr, (const int32_t*)ids})
          CHECK(nanospec_mx4_gather_rows(q, s, NS_MAX_V, d, at, nullptr, R, fake(7), d, dtype, nullptr) == NS_EHIP);
      }
    for (int32_t M : {1, 16, 17, 33, 49, 64, 65, 128, 129, NS_MAX_ROWS})
      for (int32_t N : {1, 64, 65, 4096, 4097, 16384, 16385, NS_MAX_V})
        for (int64_t pad : {(int64_t)0, (int64_t)1 << 39})
          CHECK(nanospec_mx4_matmul(q, s, M, w, t, N, NS_MAX_D, fake(7), N + pad, dtype, nullptr) == NS_EHIP);
    for (int32_t B : {1, 3, NS_MAX_BATCH})
      for (int32_t n : {1, 4096, 4097, 16384, 16385, NS_MAX_V})
        for (int32_t M : {1, 17, 33, 64})
          for (int32_t d : {8, 4096, NS_MAX_D}) {
            const size_t need = nanospec_mx4_logits_workspace_bytes(B, n, M, 64, d);
            CHECK(nanospec_mx4_logits_topk(w, t, ids, ids, n, B, NS_MAX_V, d, fake(7), dtype, M, 64, nullptr, ids, f,
                                           fake(8), need, nullptr) == NS_EHIP);
            CHECK(nanospec_mx4_logits_topk(w, t, ids, ids, n, B, NS_MAX_V, d, fake(7), dtype, M, 64, nullptr, ids, f,
                                           fake(8), need - 1, nullptr) == NS_ECAPACITY);
          }
    for (int32_t L : {0, 1, 8, 95, 96, 257, 2048, NS_MAX_ROWS})
      for (int32_t V : {1, 7, 2048, 65537, 128256, NS_MAX_V})
        for (void* dz : {(void*)nullptr, fake(9)}) {
          const size_t need = nanospec_policy_loss_workspace_bytes(L, V);
          const auto call = [&](size_t bytes) {
            return nanospec_policy_loss(fake(7), V, L, V, dtype, 1.f, ids, f, g, f, g, 0.2f, INFINITY, 0.1f, 0.01f, f, f,
                                        g, g, f, dz, V, fake(8), bytes, nullptr);
          };
          CHECK(call(need) == NS_EHIP);
          CHECK(call(need - 1) == NS_ECAPACITY);
        }
  }
  return 0;
}

}  // namespace

int main() {
  if (check_sizes()) return 1;
  if (check_plans()) return 1;
  printf("4-bit and policy host checks passed\n");
  return 0;
}
