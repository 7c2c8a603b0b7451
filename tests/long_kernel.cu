// A kernel that lets the next one on its stream start at once and itself takes `us` microseconds.
#include <cuda_runtime.h>

__global__ void k_long(long long ns) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    unsigned long long t0, t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t0));
    do {
        __nanosleep(1000);
        asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    } while ((long long)(t - t0) < ns);
}

extern "C" int long_kernel(int us, void *stream) {
    if (us < 0 || us > 100000) return 1;
    k_long<<<1, 32, 0, (cudaStream_t)stream>>>(1000LL * us);
    return cudaGetLastError() != cudaSuccess;
}
