// sm_100a kernels of the offset/mask predictor's backward. With the projection
//   record[m, slot(o)] = bias[o] + sum_c W[o, c] y[m, c]
// and gp[m, o] = dL/drecord[m, slot(o)] (the fp32 records the aggregation's
// backward writes), the gradients are
//   dL/dy[m, c] = sum_o gp[m, o] W[o, c]
//   dL/dW[o, c] = sum_m gp[m, o] y[m, c]
//   dL/dbias[o] = sum_m gp[m, o].
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dcnv4_async.cuh"
#include "dcnv4_kernels.cuh"
#include "dcnv4_simt_gemm.cuh"

namespace dcnv4 {

struct PredBwdParams {
    int M, C, G, P, NO;
    int splits;          // ranges of pixels, each with its own partial sums of dL/dW and dL/dbias
    int split_pixels;    // pixels per range
};

// projection channel of a record slot
__host__ __device__ __forceinline__ int channel_of_slot(int s, int G, int P) {
    const int g = s / (3 * P), r = s - g * 3 * P;
    return r < 2 * P ? g * 2 * P + r : 2 * G * P + g * P + (r - 2 * P);
}

template <typename T>
__global__ void __launch_bounds__(256)
pred_grad_y_kernel(const float* __restrict__ grec, const T* __restrict__ w, float* __restrict__ gy, PredBwdParams p) {
    __shared__ SimtSmem sm;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    simt_tile(
        sm, blockIdx.x * kSimtTile, blockIdx.y * kSimtTile, p.M, p.C, 0, p.NO,
        [&](int m, int s) { return __ldg(grec + static_cast<size_t>(m) * p.NO + s); },
        [&](int s, int c) {
            return ElemTraits<T>::to_float(__ldg(w + static_cast<size_t>(channel_of_slot(s, p.G, p.P)) * p.C + c));
        },
        [&](int m, int c, float v) { gy[static_cast<size_t>(m) * p.C + c] = v; });
}

// Partial sums of one pixel range: part[split][slot][c], and pbias[split][slot].
template <typename T>
__global__ void __launch_bounds__(256)
pred_grad_w_partial_kernel(const float* __restrict__ grec, const T* __restrict__ y, float* __restrict__ part,
                           float* __restrict__ pbias, PredBwdParams p) {
    __shared__ SimtSmem sm;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int split = blockIdx.z;
    const int m0 = split * p.split_pixels, m1 = min(p.M, m0 + p.split_pixels);
    simt_tile(
        sm, blockIdx.x * kSimtTile, blockIdx.y * kSimtTile, p.NO, p.C, m0, m1,
        [&](int s, int m) { return __ldg(grec + static_cast<size_t>(m) * p.NO + s); },
        [&](int m, int c) { return ElemTraits<T>::to_float(__ldg(y + static_cast<size_t>(m) * p.C + c)); },
        [&](int s, int c, float v) { part[(static_cast<size_t>(split) * p.NO + s) * p.C + c] = v; });
    if (blockIdx.y == 0) {
        const int s = blockIdx.x * kSimtTile + threadIdx.x;
        if (threadIdx.x < kSimtTile && s < p.NO) {
            float a = 0.f;
            for (int m = m0; m < m1; ++m) a += __ldg(grec + static_cast<size_t>(m) * p.NO + s);
            pbias[static_cast<size_t>(split) * p.NO + s] = a;
        }
    }
}

// The ranges' partial sums added in order (the same order in every run), rows
// moved from record order to the projection's channel order.
__global__ void __launch_bounds__(256)
pred_grad_w_join_kernel(const float* __restrict__ part, const float* __restrict__ pbias, float* __restrict__ gw,
                        float* __restrict__ gb, PredBwdParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long n = static_cast<long long>(p.NO) * p.C;
    for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < n + p.NO;
         i += static_cast<long long>(gridDim.x) * 256) {
        float a = 0.f;
        if (i < n) {
            for (int k = 0; k < p.splits; ++k) a += __ldg(part + k * n + i);
            const int s = static_cast<int>(i / p.C), c = static_cast<int>(i - static_cast<long long>(s) * p.C);
            gw[static_cast<size_t>(channel_of_slot(s, p.G, p.P)) * p.C + c] = a;
        } else if (gb) {
            const int s = static_cast<int>(i - n);
            for (int k = 0; k < p.splits; ++k) a += __ldg(pbias + static_cast<size_t>(k) * p.NO + s);
            gb[channel_of_slot(s, p.G, p.P)] = a;
        }
    }
}

}  // namespace dcnv4
