// Host threads that make their first calls at the same time, one after the
// other in the order that hurts: dsa_internal.h's allow_smem over fakes of the
// two CUDA calls it makes.  Prints "ok" and exits 0 when no thread's launch
// would find a lower limit than it asked for; tests/test_smem_limit.py
// compiles and runs it.
#include <cuda_runtime.h>

#include <cstdio>
#include <functional>

namespace fake {
int device = 0, limit[2] = {48 * 1024, 48 * 1024}, calls = 0;
std::function<void()> meanwhile;  // runs once, right behind the next change of the limit
cudaError_t get_device(int *dev) {
  *dev = device;
  return cudaSuccess;
}
template <typename Kernel>
cudaError_t set_attribute(Kernel, cudaFuncAttribute, int bytes) {
  ++calls;
  if (bytes > 227 * 1024) return cudaErrorInvalidValue;
  limit[device] = bytes;
  std::function<void()> other;
  other.swap(meanwhile);
  if (other) other();
  return cudaSuccess;
}
}  // namespace fake
#define cudaGetDevice fake::get_device
#define cudaFuncSetAttribute fake::set_attribute
#include "dsa_internal.h"

static void kernel(int) {}

static int failures = 0;
#define CHECK(cond)                                                    \
  do {                                                                 \
    if (!(cond)) {                                                     \
      std::fprintf(stderr, "line %d: %s\n", __LINE__, #cond);          \
      ++failures;                                                      \
    }                                                                  \
  } while (0)

int main() {
  constexpr int kLarge = 200 * 1024, kSmall = 100 * 1024;
  static dsa::SmemLimit done;
  // a small config's first call falls between a large one's change of the limit and its launch
  fake::meanwhile = [] {
    CHECK(dsa::allow_smem(kernel, kSmall, done) == cudaSuccess);
    CHECK(fake::limit[0] >= kSmall);
  };
  CHECK(dsa::allow_smem(kernel, kLarge, done) == cudaSuccess);
  CHECK(fake::limit[0] >= kLarge);  // the first thread launches now
  CHECK(dsa::allow_smem(kernel, kLarge, done) == cudaSuccess);
  CHECK(fake::limit[0] >= kLarge);  // and every later call
  const int calls = fake::calls;
  CHECK(dsa::allow_smem(kernel, kSmall, done) == cudaSuccess && fake::calls == calls);  // asked for once a device
  fake::device = 1;
  CHECK(dsa::allow_smem(kernel, kLarge, done) == cudaSuccess && fake::limit[1] >= kLarge);
  CHECK(dsa::allow_smem(kernel, 227 * 1024 + 16, done) != cudaSuccess);  // more than a CTA can have
  if (failures == 0) std::puts("ok");
  return failures == 0 ? 0 : 1;
}
