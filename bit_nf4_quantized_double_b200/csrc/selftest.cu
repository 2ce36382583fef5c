// Self-tests (the page has no counterpart).
//
// k_selftest_wait: the bounded waits that every pipelined kernel of this library
// uses (part of the library's failure detection). One thread arms an mbarrier
// that nothing will complete and waits on it through the same bounded wait; after
// the wait limit (1 s) the wait gives up, records QLORA_ERR_TIMEOUT in the device
// status word, and the kernel returns normally: no trap, and the context stays
// usable.
//
// k_selftest_wait_warp: the same wait made by a whole warp, whose lanes must all get the
// same answer. A second warp completes the barrier, raises the abort flag, or does both a
// different time after the wait began in every trial, the times spread over the interval
// between the wait's looks at the flag; the last trial is left to its limit (1 ms).
//
// k_selftest_rcp: the error of the reciprocal approximation that the quantiser's
// fast path relies on, over all 2^23 mantissas m in [1, 2): |r - 1/m| in units of
// r's ulp, exact in double, as a fixed-point maximum (1024 = one ulp).
#include "launch.h"
#include "tc.cuh"

namespace qnf4 {
using namespace tc;

__global__ void k_selftest_wait() {
    __shared__ __align__(8) uint64_t bar;
    __shared__ int s_abort;
    if (threadIdx.x == 0) {
        mbar_init(smem_addr(&bar), 1);
        s_abort = 0;
        fence_barrier_init();
    }
    __syncthreads();
    if (threadIdx.x == 0) (void)mbar_wait(smem_addr(&bar), 0, &s_abort);
}

constexpr int kWaitTrials = 96;
__global__ void k_selftest_wait_warp(unsigned int *out) {
    __shared__ __align__(8) uint64_t bar[kWaitTrials + 1];
    __shared__ int s_abort[kWaitTrials + 1];
    for (int i = threadIdx.x; i <= kWaitTrials; i += 64) {
        mbar_init(smem_addr(bar + i), 1);
        s_abort[i] = 0;
    }
    fence_barrier_init();
    __syncthreads();
    unsigned int split = 0, wrong = 0, gave_up = 0;
    for (int i = 0; i <= kWaitTrials; ++i) {
        const int mode = i == kWaitTrials ? -1 : i & 3;      // none; complete, abort, abort and complete, complete and abort
        volatile int *abort = s_abort + i;
        if (threadIdx.x < 32) {
            const bool ok = mbar_wait_warp(smem_addr(bar + i), 0, abort, mode < 0 ? 1000000ull : kWaitLimitNs);
            const unsigned int yes = __ballot_sync(0xffffffffu, ok);
            split += yes != 0u && yes != 0xffffffffu;
            wrong += (mode == 0 && yes != 0xffffffffu) || ((mode == 1 || mode < 0) && yes != 0u);
            gave_up += yes == 0u;
        } else if (threadIdx.x == 32 && mode >= 0) {
            const uint64_t t0 = global_timer_ns();
            while (global_timer_ns() - t0 < (uint64_t)i * 15000u) {
            }
            if (mode == 1 || mode == 2) *abort = 1;
            if (mode != 1) mbar_arrive(smem_addr(bar + i));
            if (mode == 3) *abort = 1;
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        out[0] = split;
        out[1] = wrong;
        out[2] = gave_up;
        out[3] = kWaitTrials + 1;
    }
}

__global__ void k_selftest_rcp(unsigned int *max_err) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= (1 << 23)) return;
    const float m = __uint_as_float(0x3f800000u | (unsigned)i);
    const float r = rcp_approx(m);
    int ex = 0;
    (void)frexp((double)r, &ex);                       // r = f 2^ex, f in [0.5, 1)
    const double ulp = ldexp(1.0, ex - 24);
    const double err = fabs((double)r - 1.0 / (double)m) / ulp;
    atomicMax(max_err, (unsigned int)(err * 1024.0));
}

}  // namespace qnf4

extern "C" qlora_status qlora_selftest_wait_timeout(qlora_stream_t stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    QNF4_LAUNCH("k_selftest_wait", st, qnf4::k_selftest_wait<<<1, 32, 0, st>>>());
    return cudaGetLastError() == cudaSuccess ? QLORA_OK : QLORA_ERR_CUDA;
}

extern "C" qlora_status qlora_selftest_wait_warp(unsigned int *out, qlora_stream_t stream) {
    if (!out || (reinterpret_cast<uintptr_t>(out) & 3u)) return QLORA_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    QNF4_LAUNCH("k_selftest_wait_warp", st, qnf4::k_selftest_wait_warp<<<1, 64, 0, st>>>(out));
    return cudaGetLastError() == cudaSuccess ? QLORA_OK : QLORA_ERR_CUDA;
}

extern "C" qlora_status qlora_selftest_rcp_error(unsigned int *max_err_1024, qlora_stream_t stream) {
    if (!max_err_1024) return QLORA_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cudaMemsetAsync(max_err_1024, 0, sizeof(unsigned int), st) != cudaSuccess) return QLORA_ERR_CUDA;
    QNF4_LAUNCH("k_selftest_rcp", st, qnf4::k_selftest_rcp<<<(1 << 23) / 256, 256, 0, st>>>(max_err_1024));
    return cudaGetLastError() == cudaSuccess ? QLORA_OK : QLORA_ERR_CUDA;
}
