// selftest.cu -- a diagnostic for the bounded waits every tensor-core kernel of the library uses.
//
// One CTA initialises an mbarrier that nothing ever arrives at and waits on it through the bounded waits (sm100.cuh:
// mbar_wait, and bar_wait, whose limit is on the SM's clock) that the kernels use for their TMA, MMA and softmax hand-offs.
// Each gives up at its limit, sets KV8_ERR_TIMEOUT in the error word, and the kernel returns normally: no fault, no
// trap, and the context stays usable.  A last wait finds the abort flag that the one before it has set and returns at once.
// The tests call it to check the timeout path end to end.
#include "internal.h"
#include "sm100.cuh"

namespace kv8 {
namespace {

using namespace sm100;

__global__ void wait_selftest_kernel(uint64_t limit_ns, int *err_word, int *status) {
    __shared__ uint64_t bar;
    __shared__ int abort_flag;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        abort_flag = 0;
        fence_barrier_init();
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        // no arrival: each gives up (2 cycles a ns: the clock is 2.07 GHz at most)
        bool done = mbar_wait(&bar, 0, nullptr, err_word, limit_ns);
        const long long cycles = 2 * (long long)limit_ns;
        done |= bar_wait(&bar, 0, &abort_flag, err_word, cycles);
        done |= *(volatile int *)&abort_flag != 1;
        done |= bar_wait(&bar, 0, &abort_flag, err_word, 4 * cycles);  // the flag ends this one, not its limit
        if (status) *status = done ? 1 : 2;
    }
}

}  // namespace

cudaError_t launch_wait_selftest(uint64_t limit_ns, int *err_word, int *status, cudaStream_t st) {
    wait_selftest_kernel<<<1, 32, 0, st>>>(limit_ns, err_word, status);
    return cudaGetLastError();
}

}  // namespace kv8
