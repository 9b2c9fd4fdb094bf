// Host side of dcnv4_predictor_backward (declared in include/dcnv4.h).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <mutex>

#include "dcnv4.h"
#include "dcnv4_internal.h"
#include "dcnv4_predictor_backward.cuh"

namespace {

#include "dcnv4_host_common.inl"

#include "dcnv4_unit_common.inl"

// Pixel ranges of the weight gradient. From the sizes alone, so that the sums'
// order (and the result's bits) are the same on every device and in every run.
void split_pixels(int M, dcnv4::PredBwdParams* p) {
    const int want = std::max(1, std::min(64, (M + 511) / 512));
    p->split_pixels = static_cast<int>((static_cast<long long>(M) + want - 1) / want);
    p->splits = M > 0 ? (M + p->split_pixels - 1) / p->split_pixels : 0;
}

long long workspace_bytes(const dcnv4::PredBwdParams& p) {
    return 4LL * p.splits * (static_cast<long long>(p.NO) * p.C + p.NO);
}

template <typename T>
int launch(const void* y, const void* w, const float* grec, float* gy, float* gw, float* gb, float* ws,
           const dcnv4::PredBwdParams& p, cudaStream_t s) {
    constexpr int t = dcnv4::kSimtTile;
    const unsigned mt = static_cast<unsigned>((static_cast<long long>(p.M) + t - 1) / t);
    const unsigned ct = static_cast<unsigned>((p.C + t - 1) / t), st = static_cast<unsigned>((p.NO + t - 1) / t);
    int rc = launch_chained(dcnv4::pred_grad_y_kernel<T>, dim3(mt, ct), 256, 0, s, grec, static_cast<const T*>(w), gy, p);
    if (rc) return rc;
    float* part = ws;
    float* pbias = ws + static_cast<size_t>(p.splits) * p.NO * p.C;
    rc = launch_chained(dcnv4::pred_grad_w_partial_kernel<T>, dim3(st, ct, static_cast<unsigned>(p.splits)), 256, 0, s,
                        grec, static_cast<const T*>(y), part, pbias, p);
    if (rc) return rc;
    const long long n = static_cast<long long>(p.NO) * p.C + p.NO;
    return launch_chained(dcnv4::pred_grad_w_join_kernel, dim3(static_cast<unsigned>(std::min<long long>((n + 255) / 256, 148 * 8))),
                          256, 0, s, static_cast<const float*>(part), static_cast<const float*>(pbias), gw, gb, p);
}

}  // namespace

extern "C" {

int dcnv4_predictor_backward_workspace(int M, int C, int G, int K, unsigned flags, int dtype, size_t* bytes) {
    long long P = 0, NO = 0;
    const int rc = check_projection(M, C, G, K, flags, dtype, &P, &NO);
    if (rc) return rc;
    if (!bytes) return DCNV4_ERR_NULL;
    dcnv4::PredBwdParams p{};
    p.M = M; p.C = C; p.G = G; p.P = static_cast<int>(P); p.NO = static_cast<int>(NO);
    split_pixels(M, &p);
    *bytes = static_cast<size_t>(workspace_bytes(p));
    return DCNV4_OK;
}

int dcnv4_predictor_backward(const void* y, const void* weight, const float* grad_offset_mask, float* grad_y,
                             float* grad_weight, float* grad_bias, void* workspace, size_t workspace_size,
                             int M, int C, int G, int K, unsigned flags, int dtype, void* stream) {
    long long P = 0, NO = 0;
    const int rc = check_projection(M, C, G, K, flags, dtype, &P, &NO);
    if (rc) return rc;
    dcnv4::PredBwdParams p{};
    p.M = M; p.C = C; p.G = G; p.P = static_cast<int>(P); p.NO = static_cast<int>(NO);
    split_pixels(M, &p);
    const int e = elem_size(dtype);
    const long long ny = static_cast<long long>(M) * C, nw = NO * C, nrec = M * NO;
    const long long need = workspace_bytes(p);
    // without pixels the weight's gradients are still written (zeros)
    if (!grad_weight || (M > 0 && (!y || !weight || !grad_offset_mask || !grad_y || !workspace))) return DCNV4_ERR_NULL;
    if (!aligned(y, e) || !aligned(weight, e) || !aligned(grad_offset_mask, 4) || !aligned(grad_y, 4) ||
        !aligned(grad_weight, 4) || !aligned(grad_bias, 4) || (M > 0 && !aligned(workspace, 16)))
        return DCNV4_ERR_ALIGN;
    if (M > 0 && workspace_size < static_cast<size_t>(need)) return DCNV4_ERR_WORKSPACE;
    const void* in[3] = {y, weight, grad_offset_mask};
    const long long in_bytes[3] = {ny * e, M > 0 ? nw * e : 0, nrec * 4};
    const void* out[4] = {grad_y, grad_weight, grad_bias, workspace};
    const long long out_bytes[4] = {ny * 4, nw * 4, grad_bias ? NO * 4 : 0, M > 0 ? need : 0};
    for (int o = 0; o < 4; ++o) {
        for (int i = 0; i < 3; ++i)
            if (overlap(out[o], out_bytes[o], in[i], in_bytes[i])) return DCNV4_ERR_ALIAS;
        for (int q = 0; q < o; ++q)
            if (overlap(out[o], out_bytes[o], out[q], out_bytes[q])) return DCNV4_ERR_ALIAS;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (M == 0) {
        if (cudaMemsetAsync(grad_weight, 0, static_cast<size_t>(nw) * 4, s) != cudaSuccess) return DCNV4_ERR_CUDA;
        if (grad_bias && cudaMemsetAsync(grad_bias, 0, static_cast<size_t>(NO) * 4, s) != cudaSuccess)
            return DCNV4_ERR_CUDA;
        return DCNV4_OK;
    }
    float* ws = static_cast<float*>(workspace);
    switch (dtype) {
        case DCNV4_F32: return launch<float>(y, weight, grad_offset_mask, grad_y, grad_weight, grad_bias, ws, p, s);
        case DCNV4_F16: return launch<__half>(y, weight, grad_offset_mask, grad_y, grad_weight, grad_bias, ws, p, s);
        default: return launch<__nv_bfloat16>(y, weight, grad_offset_mask, grad_y, grad_weight, grad_bias, ws, p, s);
    }
}

}  // extern "C"
