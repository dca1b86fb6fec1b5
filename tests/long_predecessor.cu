/* A kernel that lets the next kernel of its stream start and then runs on for a
 * given number of clocks (at most 4 * 10^9), for tests of programmatic launches. */
#include <cuda_runtime.h>

__global__ void long_predecessor(long long clocks, int *out) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long t0 = clock64();
    for (long long i = 0; i < (1ll << 32) && clock64() - t0 < clocks; ++i) __nanosleep(1000);
    *out = 1;   /* what the next kernel may read only after its griddepcontrol.wait */
}

extern "C" int launch_long_predecessor(long long clocks, int *out, void *stream) {
    if (clocks > 4000000000ll) clocks = 4000000000ll;
    long_predecessor<<<1, 1, 0, static_cast<cudaStream_t>(stream)>>>(clocks, out);
    return int(cudaGetLastError());
}
