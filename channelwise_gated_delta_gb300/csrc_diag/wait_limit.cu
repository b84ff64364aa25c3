// wait_limit.cu -- test-only diagnostic (libgdr_diag.so): the bounded
// mbarrier wait the library's kernels use, run against a barrier nothing
// ever arrives on, so that a test can see a wait give up after its limit,
// set the error word and leave the kernel and the context usable -- the
// failure path of every wait in the library, exercised without a fault.
#include <cuda_runtime.h>

#include "sm100_ptx.cuh"

namespace gdr {
namespace {

using namespace sm100;

// One CTA of 32 threads: thread 0 initialises an mbarrier expecting one
// arrival, which never comes; every thread waits on its first phase with
// the given limit, and each one that gives up adds one to *gave_up.
__global__ void __launch_bounds__(32, 1)
    gdr_selftest_wait_kernel(unsigned long long limit_ns, int *gave_up) {
    __shared__ __align__(8) uint64_t bar;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        fence_mbar_init();
    }
    __syncthreads();
    if (!mbar_wait_bounded(&bar, 0, limit_ns)) atomicAdd(gave_up, 1);
}

// The wait by cycles of the kernels with many short waits, 2^24 of them, by all 32
// lanes; gave_up counts those that find the flag set.  ns: how long it took.
__global__ void __launch_bounds__(32, 1)
    gdr_selftest_cycles_kernel(int *gave_up, unsigned long long *ns) {
    __shared__ __align__(8) uint64_t bar;
    __shared__ int flag;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        fence_mbar_init();
        flag = 0;
    }
    __syncthreads();
    const uint64_t t0 = global_timer_ns();
    mbar_wait_cycles<1u << 24>(smem_u32(&bar), 0, smem_u32(&flag));
    const uint64_t t1 = global_timer_ns();
    if (*(volatile int *)&flag) atomicAdd(gave_up, 1);
    if (threadIdx.x == 0) *ns = t1 - t0;
}

}  // namespace
}  // namespace gdr

// Launches the wait by cycles.
extern "C" __attribute__((visibility("default"))) int gdr_diag_wait_cycles(
    int *gave_up, unsigned long long *ns, void *stream) {
    if (!gave_up || !ns) return -1;
    gdr::gdr_selftest_cycles_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(gave_up, ns);
    return (int)cudaGetLastError();
}

// Launches the wait on `stream` with a limit of limit_ns nanoseconds
// (1 ms .. 1 s); `gave_up` a device int the kernel adds one to per thread
// whose wait ran out.  Returns 0, -1 for bad arguments, or the cudaError_t
// of the launch.
extern "C" __attribute__((visibility("default"))) int gdr_diag_wait_limit(
    unsigned long long limit_ns, int *gave_up, void *stream) {
    if (!gave_up || limit_ns < 1000000ull || limit_ns > 1000000000ull) return -1;
    gdr::gdr_selftest_wait_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(limit_ns,
                                                                                gave_up);
    return (int)cudaGetLastError();
}
