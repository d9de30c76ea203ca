// Bounded waits of the attention kernels, and the record of the first device error.
//
// The error words are per translation unit (each .cu that includes this file has
// its own set); the host reads and clears all of them.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace xs {

static __device__ int g_device_error = 0;
static __device__ DeviceErrorInfo g_error_info;
static __device__ int g_drain_failed = 0;
// %globaltimer of the record: the host reports the earliest of several kernels'.  (All words in one struct,
// one copy to read them, had the dense kernel run 0.5 to 0.9 % slower, with no more registers.)
static __device__ unsigned long long g_error_when;

// Records the first device error of the launch (later ones only find the word
// set).  Out of line: it runs at most once per launch and must not weigh on the
// register allocation of the loops that call it.
static __device__ __noinline__ void report_error(int code, int site, int d0, int d1, int d2) {
    if (atomicCAS(&g_device_error, 0, code) == 0) {
        DeviceErrorInfo r;
        r.code = code;
        r.cta = static_cast<int>(blockIdx.x);
        r.warp = static_cast<int>(threadIdx.x >> 5);
        r.lane = static_cast<int>(threadIdx.x & 31u);
        r.site = site;
        r.detail[0] = d0;
        r.detail[1] = d1;
        r.detail[2] = d2;
        g_error_info = r;
        g_error_when = globaltimer_ns();
        __threadfence();
    }
}

// Time since t0 has reached the limit.  Signed, so that a timer read that
// comes out below t0 counts as no time passed rather than as a huge one.
static __device__ __forceinline__ bool expired(uint64_t t0, uint64_t limit_ns) {
    return static_cast<long long>(globaltimer_ns() - t0) >= static_cast<long long>(limit_ns);
}

constexpr uint32_t WAIT_CHECK_EVERY = 16;   // probes between time-limit checks (a power of two)

// Bounded wait, executed by a whole warp; the result is warp-uniform.  The
// first probe is a non-blocking test; the further probes are mbarrier.try_wait
// without a time hint (the hardware's own short suspend limit: a waiting role
// resumes as soon as the phase completes, which measured 1-5 % faster per launch
// than a 200 us hint).  The abort flag and the time limit are looked at before
// the first try_wait's retry and then every WAIT_CHECK_EVERY probes: a
// %globaltimer read costs more than a probe, and a read between the phase's
// completion and the next probe delays the waiter by that much.  A limit of 0
// gives up after the first try_wait of the first wait that is not already over.  On expiry the wait records (barrier, parity, piece, block) as
// the launch's first error, unless one is recorded already.
static __device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                          uint64_t timeout_ns, int unit = -1, int blk = -1) {
    bool ok = mbar_test_wait(bar, parity);
    if (!__all_sync(0xffffffffu, ok)) {
        uint64_t t0 = 0;
        for (uint32_t n = 0; !ok; ++n) {
            ok = mbar_try_wait(bar, parity);
            if (ok || (n & (WAIT_CHECK_EVERY - 1)) != 0) continue;
            if (*abort_flag) break;
            if (n == 0) t0 = globaltimer_ns();
            if (expired(t0, timeout_ns)) {
                *abort_flag = 1;
                report_error(XS_DEVICE_TIMEOUT_CODE, static_cast<int>(bar), static_cast<int>(parity), unit, blk);
                break;
            }
        }
        ok = __all_sync(0xffffffffu, ok);
    }
    return ok;
}

// Suspend hint of the single-thread roles' probes (ns): a suspended thread is
// woken by the phase's completion, and while it sleeps it takes no issue slots
// from the softmax warps on its sub-partition (measured +1 ... +1.4 % at the long
// power-limited shapes, no change at the short ones, against hint-free probes).
constexpr uint32_t ROLE_WAIT_HINT_NS = 2000;

// The same bounded wait for a single thread (the issuing lanes of the producer
// and MMA roles), without warp votes.
static __device__ __forceinline__ bool thread_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                            uint64_t timeout_ns, int unit = -1, int blk = -1) {
    if (mbar_test_wait(bar, parity)) return true;
    uint64_t t0 = 0;
    for (uint32_t n = 0;; ++n) {
        if (mbar_try_wait_sleep(bar, parity, ROLE_WAIT_HINT_NS)) return true;
        if ((n & (WAIT_CHECK_EVERY - 1)) != 0) continue;
        if (*abort_flag) return false;
        if (n == 0) t0 = globaltimer_ns();
        if (expired(t0, timeout_ns)) {
            *abort_flag = 1;
            report_error(XS_DEVICE_TIMEOUT_CODE, static_cast<int>(bar), static_cast<int>(parity), unit, blk);
            return false;
        }
    }
}

// Wait of the abort path for an asynchronous operation already issued (a TMA
// copy, the MMAs before a commit): bounded by `limit_ns`; if it gives up, the
// operation may still be in flight when the CTA frees its tensor memory and
// exits, so that is flagged for the host (XS_ERR_DEVICE_DRAIN), beside the
// error that caused the abort.
static __device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
    if (mbar_test_wait(bar, parity)) return;
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait_sleep(bar, parity, 200000u)) {
        if (expired(t0, limit_ns)) {
            atomicOr(&g_drain_failed, 1);
            return;
        }
    }
}

// One arrival for a whole warp: every lane has finished its part (its own
// fences included) once __syncwarp returns; lane 0 then arrives.  Replaces 32
// arrivals on the same shared-memory word, which serialise.
static __device__ __forceinline__ void warp_arrive(uint32_t bar) {
    __syncwarp();
    if (lane_id() == 0) mbar_arrive(bar);
}

// Reads this translation unit's error words, and clears them if there is something to clear.
static inline cudaError_t read_and_clear_error_words(int* value, DeviceErrorInfo* info, int* drain_failed,
                                                     unsigned long long* when) {
    cudaError_t e = cudaMemcpyFromSymbol(value, g_device_error, sizeof(int));
    if (e == cudaSuccess) e = cudaMemcpyFromSymbol(drain_failed, g_drain_failed, sizeof(int));
    if (e != cudaSuccess || (*value == 0 && *drain_failed == 0)) return e;
    const int zero = 0;
    const DeviceErrorInfo none{};
    e = cudaMemcpyFromSymbol(info, g_error_info, sizeof *info);
    if (e == cudaSuccess) e = cudaMemcpyFromSymbol(when, g_error_when, sizeof *when);
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_device_error, &zero, sizeof zero);
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_drain_failed, &zero, sizeof zero);
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_error_info, &none, sizeof none);
    return e;
}

}  // namespace xs
