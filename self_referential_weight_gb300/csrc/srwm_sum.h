// srwm_sum.h -- host interface of the sum of partial results over their index.
#pragma once

#include <cuda_runtime.h>

namespace srwm {

// Rows of `width` = n[0] + n[1] + n[2] columns; the columns' sums over all rows go to out[0], out[1] and out[2] (NULL:
// not wanted) in an order that depends on the sizes alone.  add: to what is there.
struct SumJob {
    const float* part;
    long long rows;
    float* out[3];
    long long n[3];
    bool add;
};

// Behind the kernel that writes the partials (launch_behind in srwm_check.h).
int sum_launch(const SumJob& job, cudaStream_t st);

}  // namespace srwm
