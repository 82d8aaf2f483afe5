// A kernel that lets the stream's next kernel become resident at once and then runs on for `ns`
// nanoseconds (10 s at most): what a long predecessor looks like to a programmatic dependent.
#include <cuda_runtime.h>

namespace {

__device__ unsigned long long now()
{
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

__global__ void hold(unsigned long long ns)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const unsigned long long t0 = now();
    for (int i = 0; i < 10000000 && now() - t0 < ns; ++i) __nanosleep(1000);
}

}  // namespace

extern "C" int long_predecessor(long long ns, void *stream)
{
    if (ns < 0 || ns > 10000000000ll) return (int)cudaErrorInvalidValue;
    hold<<<1, 32, 0, (cudaStream_t)stream>>>((unsigned long long)ns);
    return (int)cudaGetLastError();
}
