// srwm_sum.cu -- sums of partial results over their index, in a fixed order: the
// last step of parameter gradients, whose partials come from a few hundred CTAs.
// One CTA takes 32 columns with 32 rows in flight, so a row's reads are whole
// 128-byte lines; a column's 32 sums are joined by a warp, always in the same way.
#include <cuda_runtime.h>

#include "srwm.h"
#include "srwm_check.h"
#include "srwm_mma.cuh"
#include "srwm_sum.h"

namespace srwm {
namespace {

__global__ void __launch_bounds__(1024) sum_kernel(const SumJob job)
{
    __shared__ float s[32][33];
    griddep_wait();
    const long long width = job.n[0] + job.n[1] + job.n[2];
    const long long c = static_cast<long long>(blockIdx.x) * 32 + threadIdx.x;
    float a = 0.f;
    if (c < width) {
#pragma unroll 8
        for (long long r = threadIdx.y; r < job.rows; r += 32) a += job.part[r * width + c];
    }
    s[threadIdx.y][threadIdx.x] = a;
    __syncthreads();
    a = s[threadIdx.x][threadIdx.y];   // a warp joins one column
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    long long at = static_cast<long long>(blockIdx.x) * 32 + threadIdx.y;
    if (threadIdx.x != 0 || at >= width) return;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        if (at < job.n[k]) {
            if (job.out[k]) job.out[k][at] = job.add ? job.out[k][at] + a : a;
            return;
        }
        at -= job.n[k];
    }
}

}  // namespace

int sum_launch(const SumJob& job, cudaStream_t st)
{
    const long long width = job.n[0] + job.n[1] + job.n[2];
    return launch_behind(sum_kernel, dim3(static_cast<unsigned>((width + 31) / 32)), dim3(32, 32), 0, st, job);
}

}  // namespace srwm
