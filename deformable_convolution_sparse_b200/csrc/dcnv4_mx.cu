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

constexpr int kMxCtaThreads = 256;

// Shape of the tensor-core kernel: how many record slots a CTA owns, and its
// shared- and tensor-memory layout. False: a row does not fit.
bool plan_mx(dcnv4::MxProjParams* p, int e, bool out16, int nsm, unsigned* smem, int* ntiles, int* per_sm) {
    p->k64 = (p->nb + 1) / 2;
    p->kc = (p->nb + 3) / 4;
    p->mtiles = static_cast<int>((static_cast<long long>(p->M) + 127) / 128);
    const int no16 = (p->NO + 15) / 16 * 16;
    // as few slot tiles as fit 256 columns of tensor memory and (fp32) a staging
    // tile that leaves room for other CTAs; more of them while SMs would be idle
    // (a slot tile reads and quantises the pixels again, from L2), down to 32 slots
    const int most = e == 4 ? 112 : 240;
    int n = std::max(1, (no16 + most - 1) / most);
    const int want = static_cast<int>(std::min<long long>((no16 + 31) / 32, nsm / std::max(1, p->mtiles)));
    n = std::max(n, want);
    for (; n <= no16 / 16; ++n) {
        const int nt = ((p->NO + n - 1) / n + 15) / 16 * 16;
        p->NT = nt;
        p->groups = (nt + 127) / 128;
        p->sfa_col = static_cast<unsigned>(nt);
        p->sfb_col = p->sfa_col + 4u * p->kc;
        const unsigned cols = p->sfb_col + 4u * p->kc * p->groups;
        if (cols > 512) continue;
        p->tmem_cols = 32;
        while (p->tmem_cols < cols) p->tmem_cols <<= 1;
        *ntiles = (p->NO + nt - 1) / nt;
        // rows of the staging tile: packed when they are whole records whose stride spreads over the
        // shared-memory banks (at most 4 lanes on one), else on 16-byte boundaries an odd number of
        // 16-byte units apart
        const int row = nt * e;
        const bool whole = *ntiles == 1;
        if (whole && out16 && (p->NO * e) % 8 == 0 && (p->NO * e) % 32 != 0) {
            p->store = dcnv4::kMxStoreTile;
            p->pitch = p->NO * e;
        } else {
            const bool rows_ok = out16 && (p->NO * e) % 16 == 0 && ((p->NO - (*ntiles - 1) * nt) * e) % 16 == 0;
            p->store = rows_ok ? dcnv4::kMxStoreRows : dcnv4::kMxStoreElems;
            p->pitch = (row + 15) / 16 * 16;
            if (p->pitch % 32 == 0) p->pitch += 16;
        }
        unsigned at = static_cast<unsigned>(p->k64) * 4096u;
        auto take = [&](unsigned bytes) {
            const unsigned o = at;
            at += (bytes + 127u) / 128u * 128u;
            return o;
        };
        p->smem_sfa = take(512u * p->kc);
        p->smem_b = take(static_cast<unsigned>(p->k64) * 32u * nt);
        p->smem_sfb = take(512u * p->kc * p->groups);
        p->smem_bias = take(4u * nt);
        // the last chunk of a packed row may be written past its end, into the next row's start, by nobody:
        // columns past `width` are not written
        p->smem_stage = take(128u * p->pitch);
        p->smem_bars = take(16u);
        *smem = at + 128u;
        if (*smem <= kTileSmemLimit) {
            const unsigned sm_total = 227u * 1024u;
            *per_sm = static_cast<int>(std::min({sm_total / (*smem + 1024u), 512u / p->tmem_cols, 4u}));
            return true;
        }
    }
    return false;
}

template <typename T>
int launch_predictor_mx(const void* y, const uint8_t* wc, const uint8_t* ws, const float* bias, void* rec,
                        dcnv4::MxProjParams p, cudaStream_t s) {
    const bool vec = p.C % 8 == 0 && aligned(y, 16);
    const int nsm = sm_count();
    if (nsm <= 0) return DCNV4_ERR_CUDA;
    unsigned smem = 0;
    int ntiles = 0, per_sm = 0;
    if (plan_mx(&p, sizeof(T), aligned(rec, 16), nsm, &smem, &ntiles, &per_sm)) {
        auto kern = vec ? dcnv4::predictor_mx_kernel<T, true> : dcnv4::predictor_mx_kernel<T, false>;
        if (smem_limit_once(reinterpret_cast<const void*>(kern), static_cast<int>(kTileSmemLimit)) != cudaSuccess)
            return DCNV4_ERR_LAUNCH;
        p.walkers = std::min(p.mtiles, std::max(1, nsm * per_sm / ntiles));
        return launch_chained(kern, dim3(static_cast<unsigned>(p.walkers) * static_cast<unsigned>(ntiles)), kMxCtaThreads, smem, s,
                              static_cast<const T*>(y), reinterpret_cast<const uint4*>(wc), ws, bias,
                              static_cast<T*>(rec), p);
    }
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
    p.nbd = dcnv4::make_fastdiv(static_cast<unsigned>(nb));
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
