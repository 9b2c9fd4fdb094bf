// Host side of the microscaled 4-bit entry points: dcnv4_mx_quantize,
// dcnv4_mx_dequantize, dcnv4_predictor_mx (declared in include/dcnv4.h).
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
#include "dcnv4_mx.cuh"

namespace {

#include "dcnv4_host_common.inl"

#include "dcnv4_unit_common.inl"

// Checks shared by the quantiser and its inverse; blocks: M rows of ceil(C/32).
int check_mx(const void* x, const void* codes, const void* scales, int M, int C, int dtype, bool x_is_output,
             long long* blocks) {
    if (M < 0 || C <= 0) return DCNV4_ERR_SHAPE;
    const int e = elem_size(dtype);
    if (!e) return DCNV4_ERR_DTYPE;
    const long long nb = (static_cast<long long>(C) + 31) / 32;
    *blocks = M * nb;
    if (nb * 32 >= kLimit || *blocks * 32 >= kLimit) return DCNV4_ERR_TOO_LARGE;
    if (M == 0) return DCNV4_OK;
    if (!x || !codes || !scales) return DCNV4_ERR_NULL;
    if (!aligned(x, e) || !aligned(codes, 16)) return DCNV4_ERR_ALIGN;
    const long long xb = static_cast<long long>(M) * C * e, cb = *blocks * 16, sb = *blocks;
    if (overlap(x, xb, codes, cb) || overlap(x, xb, scales, sb)) return DCNV4_ERR_ALIAS;
    if (!x_is_output && overlap(codes, cb, scales, sb)) return DCNV4_ERR_ALIAS;
    return DCNV4_OK;
}

unsigned mx_grid(long long blocks) {
    // 64 blocks (256 threads) per CTA and round, at most 16 CTAs per SM's worth of CTAs
    return static_cast<unsigned>(std::min<long long>((blocks + 63) / 64, 148LL * 16));
}

template <typename T>
int launch_quantize(const void* x, uint8_t* codes, uint8_t* scales, int C, long long blocks, cudaStream_t s) {
    const bool vec = C % 8 == 0 && aligned(x, 16);
    auto kern = vec ? dcnv4::mx_quantize_kernel<T, true> : dcnv4::mx_quantize_kernel<T, false>;
    return launch_chained(kern, dim3(mx_grid(blocks)), 256, 0, s, static_cast<const T*>(x),
                          reinterpret_cast<uint32_t*>(codes), scales, static_cast<unsigned>(blocks),
                          dcnv4::make_fastdiv(static_cast<unsigned>((C + 31) / 32)), C);
}

template <typename T>
int launch_dequantize(const uint8_t* codes, const uint8_t* scales, void* x, int C, long long blocks, cudaStream_t s) {
    const bool vec = C % 8 == 0 && aligned(x, 16);
    auto kern = vec ? dcnv4::mx_dequantize_kernel<T, true> : dcnv4::mx_dequantize_kernel<T, false>;
    return launch_chained(kern, dim3(mx_grid(blocks)), 256, 0, s, reinterpret_cast<const uint32_t*>(codes), scales,
                          static_cast<T*>(x), static_cast<unsigned>(blocks),
                          dcnv4::make_fastdiv(static_cast<unsigned>((C + 31) / 32)), C);
}

template <typename T>
int launch_predictor_mx(const void* y, const uint8_t* wc, const uint8_t* ws, const float* bias, void* rec,
                        const dcnv4::MxProjParams& p, cudaStream_t s) {
    const bool vec = p.C % 8 == 0 && aligned(y, 16);
    auto kern = vec ? dcnv4::predictor_mx_plain_kernel<T, true> : dcnv4::predictor_mx_plain_kernel<T, false>;
    const dim3 grid(static_cast<unsigned>((static_cast<long long>(p.M) + 31) / 32), static_cast<unsigned>((p.NO + 63) / 64));
    return launch_chained(kern, grid, 256, 0, s, static_cast<const T*>(y), reinterpret_cast<const uint32_t*>(wc), ws,
                          bias, static_cast<T*>(rec), p);
}

}  // namespace

extern "C" {

int dcnv4_mx_quantize(const void* x, uint8_t* codes, uint8_t* scales, int M, int C, int dtype, void* stream) {
    long long blocks = 0;
    const int rc = check_mx(x, codes, scales, M, C, dtype, false, &blocks);
    if (rc || M == 0) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (dtype) {
        case DCNV4_F32: return launch_quantize<float>(x, codes, scales, C, blocks, s);
        case DCNV4_F16: return launch_quantize<__half>(x, codes, scales, C, blocks, s);
        default: return launch_quantize<__nv_bfloat16>(x, codes, scales, C, blocks, s);
    }
}

int dcnv4_mx_dequantize(const uint8_t* codes, const uint8_t* scales, void* x, int M, int C, int dtype, void* stream) {
    long long blocks = 0;
    const int rc = check_mx(x, codes, scales, M, C, dtype, true, &blocks);
    if (rc || M == 0) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (dtype) {
        case DCNV4_F32: return launch_dequantize<float>(codes, scales, x, C, blocks, s);
        case DCNV4_F16: return launch_dequantize<__half>(codes, scales, x, C, blocks, s);
        default: return launch_dequantize<__nv_bfloat16>(codes, scales, x, C, blocks, s);
    }
}

int dcnv4_predictor_mx(const void* y, const uint8_t* weight_codes, const uint8_t* weight_scales, const float* bias,
                       void* offset_mask, int M, int C, int G, int K, unsigned flags, int dtype, void* stream) {
    long long P = 0, NO = 0;
    const int rc = check_projection(M, C, G, K, flags, dtype, &P, &NO);
    if (rc) return rc;
    const long long nb = (static_cast<long long>(C) + 31) / 32;
    if (NO * nb * 32 >= kLimit || M * nb * 32 >= kLimit) return DCNV4_ERR_TOO_LARGE;
    if (M == 0) return DCNV4_OK;
    if (!y || !weight_codes || !weight_scales || !offset_mask) return DCNV4_ERR_NULL;
    const int e = elem_size(dtype);
    if (!aligned(y, e) || !aligned(weight_codes, 16) || !aligned(offset_mask, e) || (bias && !aligned(bias, 4)))
        return DCNV4_ERR_ALIGN;
    const long long rb = M * NO * e;
    if (overlap(offset_mask, rb, y, static_cast<long long>(M) * C * e) ||
        overlap(offset_mask, rb, weight_codes, NO * nb * 16) || overlap(offset_mask, rb, weight_scales, NO * nb) ||
        (bias && overlap(offset_mask, rb, bias, NO * 4)))
        return DCNV4_ERR_ALIAS;
    dcnv4::MxProjParams p{};
    p.M = M; p.C = C; p.G = G; p.P = static_cast<int>(P); p.NO = static_cast<int>(NO); p.nb = static_cast<int>(nb);
    p.status = dcnv4_host::device_status_word();
    if (!p.status) return DCNV4_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (dtype) {
        case DCNV4_F32: return launch_predictor_mx<float>(y, weight_codes, weight_scales, bias, offset_mask, p, s);
        case DCNV4_F16: return launch_predictor_mx<__half>(y, weight_codes, weight_scales, bias, offset_mask, p, s);
        default: return launch_predictor_mx<__nv_bfloat16>(y, weight_codes, weight_scales, bias, offset_mask, p, s);
    }
}

}  // extern "C"
