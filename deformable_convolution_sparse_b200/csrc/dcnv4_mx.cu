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

// 256 threads per CTA, at most 16 CTAs per SM
unsigned mx_grid(long long blocks, int lanes) {
    return static_cast<unsigned>(std::min<long long>((blocks * lanes + 255) / 256, 148LL * 16));
}

template <typename T>
int launch_quantize(const void* x, uint8_t* codes, uint8_t* scales, int C, long long blocks, cudaStream_t s) {
    const bool vec = C % 8 == 0 && aligned(x, 16);
    auto kern = vec ? dcnv4::mx_quantize_kernel<T, true> : dcnv4::mx_quantize_kernel<T, false>;
    return launch_chained(kern, dim3(mx_grid(blocks, 2)), 256, 0, s, static_cast<const T*>(x),
                          reinterpret_cast<uint2*>(codes), scales, static_cast<unsigned>(blocks),
                          dcnv4::make_fastdiv(static_cast<unsigned>((C + 31) / 32)), C);
}

template <typename T>
int launch_dequantize(const uint8_t* codes, const uint8_t* scales, void* x, int C, long long blocks, cudaStream_t s) {
    const bool vec = C % 8 == 0 && aligned(x, 16);
    auto kern = vec ? dcnv4::mx_dequantize_kernel<T, true> : dcnv4::mx_dequantize_kernel<T, false>;
    return launch_chained(kern, dim3(mx_grid(blocks, dcnv4::mx_lanes<T>())), 256, 0, s, codes, scales,
                          static_cast<T*>(x), static_cast<unsigned>(blocks),
                          dcnv4::make_fastdiv(static_cast<unsigned>((C + 31) / 32)), C);
}

// Shape of the tensor-core kernel: how many record slots a CTA owns, and its
// shared- and tensor-memory layout. False: a row does not fit.
bool plan_mx(dcnv4::MxProjParams* p, int e, bool out16, int nsm, unsigned* smem, int* ntiles, int* threads) {
    p->k64 = (p->nb + 1) / 2;
    p->kc = (p->nb + 3) / 4;
    p->mtiles = static_cast<int>((static_cast<long long>(p->M) + 127) / 128);
    const int no16 = (p->NO + 15) / 16 * 16;
    // As few slot tiles as fit (240 slots and their scales fill 256 columns of tensor memory): each slot tile reads
    // and quantises the pixels again. Measured, 129,032 pixels x 128 channels to 216 slots in one tile against two:
    // fp16 27.9 against 39.5 us, fp32 52.5 against 72.9. But more of them, down to 32 slots, while SMs would be idle:
    // 196 pixels x 256 channels to 432 slots in fp16 take 6.4 us so against 9.0, 6,000 pixels 8.6 against 9.3.
    constexpr int most = 240;
    int n = std::max(1, (no16 + most - 1) / most);
    n = std::max(n, static_cast<int>(std::min<long long>((no16 + 31) / 32, nsm / std::max(1, p->mtiles))));
    for (; n <= (p->NO + 31) / 32; ++n) {
        // several slot tiles: multiples of 32 slots, so that each starts on a whole block of the staging tile
        const int each = (p->NO + n - 1) / n, nt = n == 1 ? no16 : (each + 31) / 32 * 32;
        p->NT = nt;
        p->groups = (nt + 127) / 128;
        p->sfa_col = static_cast<unsigned>(nt);
        p->sfb_col = p->sfa_col + 4u * p->kc;
        const unsigned cols = p->sfb_col + 4u * p->kc * p->groups;
        if (cols > 512) continue;
        p->tmem_cols = 32;
        while (p->tmem_cols < cols) p->tmem_cols <<= 1;
        *ntiles = (p->NO + nt - 1) / nt;
        // the staging tile: records back to back when a CTA writes whole ones whose stride spreads over the
        // shared-memory banks (at most 4 lanes on one); else swizzled blocks for TMA where the records' rows
        // allow it; else rows an odd number of 16-byte units apart
        const int row = p->NO * e;
        unsigned stage_bytes;
        if (*ntiles == 1 && out16 && row % 32 != 0) {
            p->store = dcnv4::kMxStoreTile;
            p->pitch = row;
            stage_bytes = 128u * row;
        } else if (out16 && row % 16 == 0) {
            p->store = dcnv4::kMxStoreTma;
            p->pitch = *ntiles == 1 || nt * e % 128 == 0 ? 128 : 64;
            stage_bytes = static_cast<unsigned>((nt * e + p->pitch - 1) / p->pitch) * 128u * p->pitch;
        } else {
            p->store = dcnv4::kMxStoreElems;
            p->pitch = (nt * e + 15) / 16 * 16;
            if (p->pitch % 32 == 0) p->pitch += 16;
            stage_bytes = 128u * p->pitch;
        }
        // the staging tile first (TMA's swizzle counts from 1024-byte boundaries), the rest on 128-byte ones;
        // what has to start as zeros (A, its scales, W, its scales) lies together
        unsigned at = 0;
        auto take = [&](unsigned bytes) {
            const unsigned o = at;
            at += (bytes + 127u) / 128u * 128u;
            return o;
        };
        p->smem_stage = take(stage_bytes);
        p->smem_a = take(static_cast<unsigned>(p->k64) * 4096u);
        p->smem_sfa = take(512u * p->kc);
        p->smem_b = take(static_cast<unsigned>(p->k64) * 32u * nt);
        p->smem_sfb = take(512u * p->kc * p->groups);
        p->smem_bias = take(8u * nt);
        p->smem_bars = take(16u);
        p->smem_ring = at;
        // four CTAs of 256 threads per SM where they fit (200,704 pixels x 64 channels to 108 slots, fp16: 19.4 us
        // against 24.1 with two of 512), else CTAs of 512
        const unsigned quarter = (227u * 1024u / 4u) - 1024u - 1024u, ring = 2u * 16u * e;  // bytes per thread
        if (p->tmem_cols <= 128 && at + 256u * ring <= quarter) {
            *threads = 256;
            *smem = at + 256u * ring + 1024u;
        } else {
            *threads = 512;
            *smem = at + 512u * ring + 1024u;
        }
        if (*smem <= kTileSmemLimit) return true;
    }
    return false;
}

template <typename T, int THREADS>
int launch_mx_tc(const void* y, const uint8_t* wc, const uint8_t* ws, const float* bias, void* rec,
                 dcnv4::MxProjParams p, unsigned smem, int ntiles, int nsm, cudaStream_t s) {
    static_assert(dcnv4::MxShape<T, THREADS>::kRing == THREADS * 2u * 16u * sizeof(T), "the plan's ring");
    const bool vec = p.C % 8 == 0 && aligned(y, 16);
    CUtensorMap rmap{};
    if (p.store == dcnv4::kMxStoreTma) {
        auto encode = tensor_map_encoder();
        const cuuint64_t dims[3] = {static_cast<cuuint64_t>(p.NO), static_cast<cuuint64_t>(p.M), 1u};
        const cuuint64_t row = static_cast<cuuint64_t>(p.NO) * sizeof(T), str[2] = {row, row * static_cast<cuuint64_t>(p.M)};
        const cuuint32_t box[3] = {static_cast<cuuint32_t>(p.pitch / sizeof(T)), 128u, 1u}, es[3] = {1u, 1u, 1u};
        if (!encode || encode(&rmap, tma_dtype<T>(), 3, rec, dims, str, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              p.pitch == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                              CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return DCNV4_ERR_CUDA;
    }
    auto kern = vec ? dcnv4::predictor_mx_kernel<T, true, THREADS> : dcnv4::predictor_mx_kernel<T, false, THREADS>;
    if (smem_limit_once(reinterpret_cast<const void*>(kern), static_cast<int>(kTileSmemLimit)) != cudaSuccess)
        return DCNV4_ERR_LAUNCH;
    const int per_sm = static_cast<int>(std::min({227u * 1024u / (smem + 1024u), 512u / p.tmem_cols, 1024u / THREADS}));
    p.walkers = std::min(p.mtiles, std::max(1, nsm * std::max(1, per_sm) / ntiles));
    return launch_chained(kern, dim3(static_cast<unsigned>(p.walkers) * static_cast<unsigned>(ntiles)), THREADS, smem, s,
                          rmap, static_cast<const T*>(y), reinterpret_cast<const uint4*>(wc), ws, bias, static_cast<T*>(rec), p);
}

template <typename T>
int launch_predictor_mx(const void* y, const uint8_t* wc, const uint8_t* ws, const float* bias, void* rec,
                        dcnv4::MxProjParams p, cudaStream_t s) {
    const int nsm = sm_count();
    if (nsm <= 0) return DCNV4_ERR_CUDA;
    unsigned smem = 0;
    int ntiles = 0, threads = 0;
    if (plan_mx(&p, sizeof(T), aligned(rec, 16), nsm, &smem, &ntiles, &threads))
        return threads == 256 ? launch_mx_tc<T, 256>(y, wc, ws, bias, rec, p, smem, ntiles, nsm, s)
                              : launch_mx_tc<T, 512>(y, wc, ws, bias, rec, p, smem, ntiles, nsm, s);
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
