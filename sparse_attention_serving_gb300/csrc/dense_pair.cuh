// dense_pair.cuh -- what the kernels of dense latent attention share beyond cluster.cuh:
// waits by whole warps that end with their CTA, rings, the exponential.
#pragma once
#include "cluster.cuh"

namespace dsa {
namespace dense {

constexpr int CHUNK = 64 * 128;           // 64 rows x 64 dims in shared memory

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A bounded wait by a whole warp; false (for all lanes) once the CTA has given up.
// CLUSTER: what the other CTA's threads wrote before they arrived is read next (by
// loads: what the tensor core reads, its own CTA's copies and fences have ordered).
// One fence after the wait, not an acquire at cluster scope in every poll.  The limit
// starts over when s_abort[1] has moved: somebody is at work without waiting.
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* s_abort,
                                     uint32_t* status, uint32_t where) {
  bool ok = mbar_test(bar, parity);
  if (!ok) {
    uint64_t t0 = globaltimer_ns();
    int beat = s_abort[1];
    while (true) {
#pragma unroll 1
      for (int k = 0; k < 16 && !ok; ++k) ok = mbar_test(bar, parity);
      if (ok || *s_abort != 0) break;
      if (globaltimer_ns() - t0 > kWaitLimitNs) {
        if (s_abort[1] != beat) {
          beat = s_abort[1];
          t0 = globaltimer_ns();
          continue;
        }
        status_raise(status, DSA_ERR_DEVICE_TIMEOUT, where);
        *s_abort = 1;
        break;
      }
    }
  }
  if (CLUSTER) asm volatile("fence.acq_rel.cluster;" ::: "memory");
  return __all_sync(0xffffffffu, ok);
}

// The end of copies and products in flight, before a CTA leaves, whether it has given up or
// not; after 20 ms (they never came to be) it leaves all the same.
__device__ __forceinline__ void settle(uint64_t* bar, uint32_t parity) {
  if (mbar_test(bar, parity)) return;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_test(bar, parity) && globaltimer_ns() - t0 < 20000000ull) {
  }
}

// A ring's slot and the parity of its current use.
template <int N>
struct Ring {
  int slot = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) slot = 0, ph ^= 1;
  }
};

}  // namespace dense
}  // namespace dsa
