// waits.cuh -- bounded mbarrier waits of whole warps, with a limit that the launch gives.
#pragma once

#include "internal.h"
#include "ptx.cuh"

namespace lm {

// Makes one wait of a launch run out, for tests (null elsewhere): the first stage of CTA
// `withheld_cta` never becomes full, and waits give up after `wait_ns`.
struct WaitFault {
  int64_t withheld_cta;
  uint64_t wait_ns;
};

// Out of line, so that loops that wait carry only the first try_wait.
static __device__ __noinline__ bool mbar_wait_limited(uint32_t addr, uint32_t parity, uint64_t limit_ns,
                                                      volatile int *abort_flag, uint32_t *err_word) {
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(addr, parity)) return true;
    if ((it & 63u) == 0u) {
      if (abort_flag && *abort_flag) return false;
      const uint64_t now = global_timer_ns();
      if (t0 == 0) {
        t0 = now;
      } else if (now - t0 > limit_ns) {
        if (abort_flag) *abort_flag = 1;
        atomicOr(err_word, kErrMbarTimeout);
        return false;
      }
    }
  }
}

// Waits for the phase with the given parity, at most limit_ns.  Called by a whole warp, whose
// lanes get one answer: a lane alone may give up (the limit, or the abort flag that another
// warp has set) while the others see the phase complete, and what follows is executed by
// warps, not by lanes.  A wait that runs out sets the CTA's abort flag and the error word.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t *bar, uint32_t parity, uint64_t limit_ns,
                                               volatile int *abort_flag, uint32_t *err_word) {
  const uint32_t addr = smem_u32(bar);
  const bool ok = mbar_try_wait(addr, parity) || mbar_wait_limited(addr, parity, limit_ns, abort_flag, err_word);
  return __all_sync(0xffffffffu, ok);
}

// Waits for copies that are in flight, whatever the other warps did (no abort flag).  Returns
// false where the limit ran out: other copies of the thread's have had as long by then.
__device__ __forceinline__ bool mbar_drain(uint64_t *bar, uint32_t parity, uint64_t limit_ns, uint32_t *err_word) {
  return mbar_wait_limited(smem_u32(bar), parity, limit_ns, nullptr, err_word);
}

// Host side of a translation unit's sticky word: reads the current device's into *value (bits are
// added to it), and clears it where `clear` says so.
template <typename Word>
lm_status read_sticky(const Word &word, uint32_t *value, bool clear, cudaStream_t s) {
  void *at = nullptr;
  uint32_t v = 0;
  LM_CUDA_TRY(cudaGetSymbolAddress(&at, word));
  LM_CUDA_TRY(cudaMemcpyAsync(&v, at, sizeof(v), cudaMemcpyDeviceToHost, s));
  if (clear) LM_CUDA_TRY(cudaMemsetAsync(at, 0, sizeof(v), s));
  LM_CUDA_TRY(cudaStreamSynchronize(s));
  *value |= v;
  return LM_OK;
}

}  // namespace lm
