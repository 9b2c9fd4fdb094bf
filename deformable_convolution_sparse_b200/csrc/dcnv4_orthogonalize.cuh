// sm_100a kernels of the Newton-Schulz orthogonalisation of a stack of weight
// updates. Each matrix X (R x C) is divided by its Frobenius norm (plus eps),
// which puts its singular values in [0, 1], and then
//   A = X X^T,  X <- a X + (b A + c A A) X
// is repeated `steps` times: every singular value s goes through the odd
// polynomial a s + b s^3 + c s^5 while the singular vectors stay. The products
// are formed on the smaller side, n = min(R, C), m = max(R, C): X is taken
// transposed when R > C.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dcnv4_async.cuh"
#include "dcnv4_kernels.cuh"
#include "dcnv4_simt_gemm.cuh"

namespace dcnv4 {

struct OrthoParams {
    int B, R, C;
    int n, m;          // smaller and larger side
    int transposed;    // R > C
    int chunks;        // partial sums of squares per matrix
    float a, b, c, eps;
};

// Sum of squares of one chunk of a matrix, in fp64 (squares of fp32 values
// neither overflow nor vanish there).
template <typename T>
__global__ void __launch_bounds__(256)
ortho_sumsq_kernel(const T* __restrict__ x, double* __restrict__ part, OrthoParams p) {
    __shared__ double ws[8];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long n = static_cast<long long>(p.R) * p.C;
    const int mat = blockIdx.x / p.chunks, ch = blockIdx.x - mat * p.chunks;
    const T* xm = x + mat * n;
    double a = 0.0;
    for (long long i = static_cast<long long>(ch) * 256 + threadIdx.x; i < n; i += static_cast<long long>(p.chunks) * 256) {
        const double v = ElemTraits<T>::to_float(__ldg(xm + i));
        a += v * v;
    }
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if ((threadIdx.x & 31) == 0) ws[threadIdx.x >> 5] = a;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < 8; ++i) a += ws[i];
        part[blockIdx.x] = a;
    }
}

template <typename T>
__global__ void __launch_bounds__(256)
ortho_start_kernel(const T* __restrict__ x, const double* __restrict__ part, float* __restrict__ xn, OrthoParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long n = static_cast<long long>(p.R) * p.C;
    const int mat = blockIdx.x / p.chunks, ch = blockIdx.x - mat * p.chunks;
    double s = 0.0;
    for (int i = 0; i < p.chunks; ++i) s += part[mat * p.chunks + i];
    const float d = static_cast<float>(sqrt(s) + p.eps);
    for (long long i = static_cast<long long>(ch) * 256 + threadIdx.x; i < n; i += static_cast<long long>(p.chunks) * 256) {
        const float v = ElemTraits<T>::to_float(__ldg(x + mat * n + i)) / d;
        const int r = static_cast<int>(i / p.C), c = static_cast<int>(i - static_cast<long long>(r) * p.C);
        xn[mat * n + (p.transposed ? static_cast<long long>(c) * p.m + r : i)] = v;
    }
}

// A = X X^T
__global__ void __launch_bounds__(256)
ortho_gram_kernel(const float* __restrict__ x, float* __restrict__ g, OrthoParams p) {
    __shared__ SimtSmem sm;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int mat = blockIdx.z; mat < p.B; mat += gridDim.z) {
        const float* xm = x + static_cast<size_t>(mat) * p.n * p.m;
        float* gm = g + static_cast<size_t>(mat) * p.n * p.n;
        simt_tile(
            sm, blockIdx.x * kSimtTile, blockIdx.y * kSimtTile, p.n, p.n, 0, p.m,
            [&](int i, int k) { return xm[static_cast<size_t>(i) * p.m + k]; },
            [&](int k, int j) { return xm[static_cast<size_t>(j) * p.m + k]; },
            [&](int i, int j, float v) { gm[static_cast<size_t>(i) * p.n + j] = v; });
    }
}

// P = a I + b A + c A A
__global__ void __launch_bounds__(256)
ortho_poly_kernel(const float* __restrict__ g, float* __restrict__ q, OrthoParams p) {
    __shared__ SimtSmem sm;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int mat = blockIdx.z; mat < p.B; mat += gridDim.z) {
        const float* gm = g + static_cast<size_t>(mat) * p.n * p.n;
        float* qm = q + static_cast<size_t>(mat) * p.n * p.n;
        simt_tile(
            sm, blockIdx.x * kSimtTile, blockIdx.y * kSimtTile, p.n, p.n, 0, p.n,
            [&](int i, int k) { return gm[static_cast<size_t>(i) * p.n + k]; },
            [&](int k, int j) { return gm[static_cast<size_t>(k) * p.n + j]; },
            [&](int i, int j, float v) {
                const size_t e = static_cast<size_t>(i) * p.n + j;
                qm[e] = fmaf(p.c, v, fmaf(p.b, gm[e], i == j ? p.a : 0.f));
            });
    }
}

// X' = P X
__global__ void __launch_bounds__(256)
ortho_apply_kernel(const float* __restrict__ q, const float* __restrict__ x, float* __restrict__ xo, OrthoParams p) {
    __shared__ SimtSmem sm;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int mat = blockIdx.z; mat < p.B; mat += gridDim.z) {
        const float* qm = q + static_cast<size_t>(mat) * p.n * p.n;
        const float* xm = x + static_cast<size_t>(mat) * p.n * p.m;
        float* om = xo + static_cast<size_t>(mat) * p.n * p.m;
        simt_tile(
            sm, blockIdx.x * kSimtTile, blockIdx.y * kSimtTile, p.n, p.m, 0, p.n,
            [&](int i, int k) { return qm[static_cast<size_t>(i) * p.n + k]; },
            [&](int k, int j) { return xm[static_cast<size_t>(k) * p.m + j]; },
            [&](int i, int j, float v) { om[static_cast<size_t>(i) * p.m + j] = v; });
    }
}

template <typename T>
__global__ void __launch_bounds__(256)
ortho_finish_kernel(const float* __restrict__ xn, T* __restrict__ out, OrthoParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long n = static_cast<long long>(p.R) * p.C;
    const int mat = blockIdx.x / p.chunks, ch = blockIdx.x - mat * p.chunks;
    for (long long i = static_cast<long long>(ch) * 256 + threadIdx.x; i < n; i += static_cast<long long>(p.chunks) * 256) {
        const int r = static_cast<int>(i / p.C), c = static_cast<int>(i - static_cast<long long>(r) * p.C);
        const float v = xn[mat * n + (p.transposed ? static_cast<long long>(c) * p.m + r : i)];
        if constexpr (sizeof(T) == 4) out[mat * n + i] = v;
        else if constexpr (std::is_same<T, __half>::value) out[mat * n + i] = __float2half_rn(v);
        else out[mat * n + i] = __float2bfloat16_rn(v);
    }
}

}  // namespace dcnv4
