// Bounded waits on mbarriers, shared by the tensor-core kernels: when a limit
// runs out the kernel records FORGE_ERR_DEVICE_TIMEOUT and gives up.
#pragma once

#include "forge_internal.h"
#include "forge_ptx.cuh"

namespace forge {

struct WaitCtx {
  volatile uint32_t* abort_flag;
  int* err;
  int* site;          // where the first timeout happened (diagnostics)
  uint64_t timeout_ns;
};

// Wait sites, recorded as site*100000 + blockIdx.x*100 + index on a timeout.
enum WaitSite : int {
  kSiteProducerEmpty = 1, kSiteMmaTmemEmpty = 2, kSiteMmaFull = 3, kSiteLoaderEmpty = 4,
  kSiteEpiTmemFull = 5, kSiteEpiSlotFull = 6, kSiteEpiSlotFree = 7, kSiteDrainOperands = 8,
  kSiteDrainState = 9, kSiteDrainMma = 10, kSiteStoreSlotDone = 11, kSiteEpiExchange = 12
};

// Wait until the phase of `bar` with `parity` completes.  Gives up (returns
// false) when the CTA's abort flag is raised, if `honor_abort`, or when the
// time limit runs out, in which case it raises the abort flag and records the
// timeout in the device error word.
//
// The first test is inlined; only a wait that has to spin calls the bounded
// loop.  The MMA issuer passes through one wait per pipeline stage, and a
// call there (frame set-up, argument moves) sits between two stages' MMAs
// long enough for the tensor core to run dry: with the call the plain GEMM
// main loop ran 11 % slower.
static __device__ __forceinline__ bool wait_spin_body(uint32_t bar, uint32_t parity,
                                                      const WaitCtx& w, int site,
                                                      bool honor_abort) {
  const uint64_t t0 = globaltimer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 16; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (honor_abort && *w.abort_flag) return false;
    if (globaltimer_ns() - t0 > w.timeout_ns) {
      *w.abort_flag = 1u;
      atomicCAS(w.err, 0, kErrDeviceTimeout);
      atomicCAS(w.site, 0, site * 100000 + static_cast<int>(blockIdx.x) * 100);
      return false;
    }
  }
}
static __device__ __noinline__ bool wait_spin(uint32_t bar, uint32_t parity, const WaitCtx& w,
                                              int site, bool honor_abort) {
  return wait_spin_body(bar, parity, w, site, honor_abort);
}
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, const WaitCtx& w,
                                             int site, bool honor_abort = true) {
  if (mbar_try_wait(bar, parity)) return true;
  return wait_spin(bar, parity, w, site, honor_abort);
}

// The same with the loop inlined, for threads that hold most of their registers
// across the wait: a call would have to save them.
__device__ __forceinline__ bool wait_bounded_inline(uint32_t bar, uint32_t parity,
                                                    const WaitCtx& w, int site,
                                                    bool honor_abort = true) {
  if (mbar_try_wait(bar, parity)) return true;
  return wait_spin_body(bar, parity, w, site, honor_abort);
}

// Testing aid (forge_debug_drop_first_arrival): the first phase of `bar`, just
// initialised by this thread, waits for bytes that never come.
__device__ __forceinline__ void drop_first_arrival(int drop, uint32_t bar) {
  if (drop) mbar_expect_tx(bar, 16);
}

// The operand-stage waits of the producer and the MMA issuer.  On one CTA
// they first poll with the non-blocking test (at most kSpinTests times)
// before the bounded wait, which may suspend the thread: the hand-off of a
// stage between the two threads is then quicker, worth 3 % at BT = 512 where
// two stages have to keep the main loop fed.  On CTA pairs, whose main loop
// reads shared memory at full rate, the polling costs more than it saves.
constexpr int kSpinTests = 4096;
template <bool SPIN>
__device__ __forceinline__ bool wait_stage(uint32_t bar, uint32_t parity, const WaitCtx& w,
                                           int site) {
  if constexpr (SPIN) {
#pragma unroll 1
    for (int i = 0; i < kSpinTests; ++i)
      if (mbar_test_wait(bar, parity)) return true;
  }
  return wait_bounded(bar, parity, w, site);
}

// A bounded wait that polls with a short sleep between tests: quicker to
// notice a completed phase than a suspended wait, but issues few
// instructions while it waits.  Used by the store lanes where the host asks
// for it (GemmParams::poll_store).
__device__ __forceinline__ bool wait_poll(uint32_t bar, uint32_t parity, const WaitCtx& w,
                                          int site) {
#pragma unroll 1
  for (int i = 0; i < kSpinTests; ++i) {
    if (mbar_test_wait(bar, parity)) return true;
    __nanosleep(32);
  }
  return wait_bounded(bar, parity, w, site);
}

}  // namespace forge
