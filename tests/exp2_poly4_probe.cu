// Test probe: evaluates the serving softmax's polynomial 2^x (csrc_serve/exp2_poly4.cuh) element-wise.
#include <cuda_runtime.h>
#include "exp2_poly4.cuh"

__global__ void exp2_poly4_kernel(const float* x, float* y, int n) {
    const int i = 2 * (blockIdx.x * blockDim.x + threadIdx.x);
    if (i + 1 < n) {
        gqa::exp2_poly4(x[i], x[i + 1], y[i], y[i + 1]);
    } else if (i < n) {
        float unused;
        gqa::exp2_poly4(x[i], 0.f, y[i], unused);
    }
}

extern "C" int exp2_poly4_eval(const float* x, float* y, int n) {
    if (n <= 0) return 0;
    const int pairs = (n + 1) / 2;
    exp2_poly4_kernel<<<(pairs + 255) / 256, 256>>>(x, y, n);
    return (int)cudaDeviceSynchronize();
}
