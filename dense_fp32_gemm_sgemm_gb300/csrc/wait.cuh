// Bounded waits on mbarriers, shared by the kernels whose roles hand work to one another.
#pragma once
#include "internal.cuh"
#include "ptx.cuh"

namespace sgemm {

constexpr unsigned long long WAIT_LIMIT_NS = 4000000000ull;

// Waits for the barrier phase of the given parity (acquire at cluster scope when
// `cluster` is set: the barrier is signalled from the peer CTA). Returns false if the
// wait ran out of time (then it raises the abort flag and the device error word) or if
// another role of this CTA already aborted.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                           int* err,
                                           unsigned long long limit_ns = WAIT_LIMIT_NS,
                                           bool cluster = false) {
    auto probe = [&]() {
        return cluster ? ptx::mbar_try_wait_cluster(bar, parity) : ptx::mbar_try_wait(bar, parity);
    };
    if (probe()) return true;
    const unsigned long long t0 = ptx::globaltimer_ns();
    while (true) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (probe()) return true;
        if (*abort_flag) return false;
        if (ptx::globaltimer_ns() - t0 > limit_ns) {
            *abort_flag = 1;
            atomicExch(err, kErrWaitTimeout);
            return false;
        }
    }
}

}  // namespace sgemm
