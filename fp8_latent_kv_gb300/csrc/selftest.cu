// selftest.cu -- a diagnostic for the bounded waits every tensor-core kernel of the library uses.
//
// One CTA initialises an mbarrier that nothing ever arrives at and waits on it through the bounded waits that the kernels use
// for their TMA, MMA, softmax and cluster hand-offs: mbar_wait, and those whose limit is on the SM's clock, bar_wait (sm100.cuh),
// bar_wait_inline and bar_wait_cluster (sm100_more.cuh).
// Each gives up at its limit, sets KV8_ERR_TIMEOUT in the error word, and the kernel returns normally: no fault, no
// trap, and the context stays usable.  After each of the clock's waits another one finds the abort flag that it has set and returns at
// once.
// The tests call it to check the timeout path end to end.
#include "internal.h"
#include "sm100_more.cuh"

namespace kv8 {
namespace {

using namespace sm100;

__global__ void wait_selftest_kernel(uint64_t limit_ns, int *err_word, int *status) {
    __shared__ uint64_t bar;
    __shared__ int abort_flag, err;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        fence_barrier_init();
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        // no arrival: each gives up (2 cycles a ns: the clock is 2.07 GHz at most)
        bool done = mbar_wait(&bar, 0, nullptr, err_word, limit_ns);
        const long long cycles = 2 * (long long)limit_ns;
        auto gives_up = [&](auto wait, long long limit) {
            *(volatile int *)&abort_flag = *(volatile int *)&err = 0;
            done |= wait(limit) || *(volatile int *)&abort_flag != 1 || *(volatile int *)&err != (int)KV8_ERR_TIMEOUT;
            done |= wait(4 * cycles);  // the flag ends this one, not its limit
        };
        gives_up([&](long long limit) { return bar_wait(&bar, 0, &abort_flag, &err, limit); }, cycles);
        gives_up([&](long long limit) { return bar_wait_inline(&bar, 0, &abort_flag, &err, limit); }, cycles / 4);
        gives_up([&](long long limit) { return bar_wait_cluster(&bar, 0, &abort_flag, &err, limit); }, cycles / 4);
        if (status) *status = done ? 1 : 2;
    }
}

}  // namespace

cudaError_t launch_wait_selftest(uint64_t limit_ns, int *err_word, int *status, cudaStream_t st) {
    wait_selftest_kernel<<<1, 32, 0, st>>>(limit_ns, err_word, status);
    return cudaGetLastError();
}

}  // namespace kv8
