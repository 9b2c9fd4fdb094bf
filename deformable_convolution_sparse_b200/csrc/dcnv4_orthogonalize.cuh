// sm_100a kernels of the Newton-Schulz orthogonalisation of a stack of weight
// updates. Each matrix X (R x C) is divided by its Frobenius norm (plus eps),
// which puts its singular values in [0, 1], and then
//   A = X X^T,  X <- P X,  P = a I + b A + c A A
// is repeated `steps` times: every singular value s goes through the odd
// polynomial a s + b s^3 + c s^5 while the singular vectors stay. The products
// are formed on the smaller side, n = min(R, C), m = max(R, C): X is taken
// transposed when R > C.
//
// Precision on the tensor cores. X, A and P are kept as two fp16 planes, hi =
// fp16(v s) and lo = fp16(v s - hi), with power-of-two scales s that the
// iteration's bounds make safe (|X| <= 4, |A| <= 16, |P| <= 64, so that no
// plane exceeds 2^14): 22 bits of every entry down to about 2^-22 of the
// bound. A matrix whose norm is far below eps starts with a small X: it is kept
// lifted by 2^e (Y = 2^e X, |Y| <= 1), e going down by as many bits per step as
// the step can grow X. A product is three tensor-core products, hi hi + hi lo + lo hi (lo lo
// is below 2^-24 of it), each exact, summed in fp32. The tensor cores' fp32
// additions truncate, so a long chain of them drifts one way: the hi hi terms
// go to up to six accumulators in turn and the small cross terms to one of
// their own, and the epilogue adds these with rounding.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dcnv4_async.cuh"
#include "dcnv4_kernels.cuh"
#include "dcnv4_tcgen05.cuh"

namespace dcnv4 {

struct OrthoParams {
    int B, R, C;
    int n, m;          // smaller and larger side
    int transposed;    // R > C
    int chunks;        // partial sums of squares per matrix
    int np, mp;        // row pitches of the n x n and n x m planes, multiples of 8 elements
    float a, b, c, eps;
    int* lift;         // [B] the exponents e of the first step
    unsigned* status;
};

// scales of the planes of X, A, P
constexpr float kOrthoSX = 4096.f, kOrthoSA = 1024.f, kOrthoSP = 256.f;

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
__device__ __forceinline__ T ortho_from_float(float v) {
    if constexpr (sizeof(T) == 4) return v;
    else if constexpr (std::is_same<T, __half>::value) return __float2half_rn(v);
    else return __float2bfloat16_rn(v);
}

// v * scale as an fp16 pair
__device__ __forceinline__ void ortho_split(float v, __half& hi, __half& lo) {
    hi = __float2half_rn(v);
    lo = __float2half_rn(v - __half2float(hi));
}

// X / (norm + eps) as planes, 64 x 64 entries per CTA; with `out` (no steps)
// the quotient itself. planes: [2][B][n][mp].
template <typename T>
__global__ void __launch_bounds__(256)
ortho_start_kernel(const T* __restrict__ x, const double* __restrict__ part, __half* __restrict__ planes,
                   T* __restrict__ out, OrthoParams p) {
    __shared__ float tile[64][65];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tr = (p.R + 63) / 64, tcn = (p.C + 63) / 64;
    const int mat = static_cast<int>(blockIdx.x / (static_cast<unsigned>(tr) * tcn));
    const int t = static_cast<int>(blockIdx.x - static_cast<unsigned>(mat) * tr * tcn);
    const int r0 = (t / tcn) * 64, c0 = (t % tcn) * 64;
    double sum = 0.0;
    for (int i = 0; i < p.chunks; ++i) sum += part[static_cast<size_t>(mat) * p.chunks + i];
    const double norm = sqrt(sum), den = norm + p.eps;
    // v / den = (v 2^-k) / (den 2^-k) with den 2^-k in [1/2, 1): no overflow, whatever the norm
    int k = 0;
    const float mant = isfinite(den) ? static_cast<float>(frexp(den, &k)) : __uint_as_float(0x7fc00000u);
    // norm / den in [2^(-1-e), 2^-e)
    const int e = norm > 0.0 && isfinite(den) ? min(120, max(0, -ilogb(norm / den) - 1)) : 0;
    const int shift = out ? -k : e - k;
    if (p.lift && t == 0 && threadIdx.x == 0) p.lift[mat] = e;
    const size_t base = static_cast<size_t>(mat) * p.R * p.C;
    for (int q = threadIdx.x; q < 4096; q += 256) {
        const int r = r0 + (q >> 6), c = c0 + (q & 63);
        if (r < p.R && c < p.C) {
            const float v = scalbnf(ElemTraits<T>::to_float(__ldg(x + base + static_cast<size_t>(r) * p.C + c)), shift) / mant;
            if (out) out[base + static_cast<size_t>(r) * p.C + c] = ortho_from_float<T>(v);
            tile[q >> 6][q & 63] = v;
        }
    }
    if (out) return;
    __syncthreads();
    const size_t plane = static_cast<size_t>(p.B) * p.n * p.mp;
    __half* o = planes + static_cast<size_t>(mat) * p.n * p.mp;
    const int i0 = p.transposed ? c0 : r0, j0 = p.transposed ? r0 : c0;
    for (int q = threadIdx.x; q < 4096; q += 256) {
        const int i = q >> 6, j = q & 63;
        if (i0 + i < p.n && j0 + j < p.m) {
            __half hi, lo;
            ortho_split((p.transposed ? tile[j][i] : tile[i][j]) * kOrthoSX, hi, lo);
            const size_t at = static_cast<size_t>(i0 + i) * p.mp + j0 + j;
            o[at] = hi;
            o[plane + at] = lo;
        }
    }
}

// One product of the iteration, a 128 x 64 tile of the result per CTA.
//   kGram:  A = X X^T          (k over m; both operands K-major rows of X)
//   kPoly:  P = aI + bA + cAA  (k over n; A is symmetric: both K-major)
//   kApply: X' = P X           (k over n; X's rows run along the result's
//                               columns: an MN-major operand)
//   kLast:  kApply with the result rounded to T and written to `out`
// Warp 0 (one lane) loads 64 k at a time by TMA: 128 rows x 64 k of the left
// planes, 64 x 64 of the right ones, in a ring of kOrthoStages; warp 1 (one
// lane) issues the products; warps 2..5 read the accumulators, form the result
// and write it as planes through shared memory and TMA.
constexpr int kGram = 0, kPoly = 1, kApply = 2, kLast = 3;
constexpr int kOrthoStages = 3, kOrthoHH = 6;
constexpr unsigned kOrthoStageBytes = 2u * 16384u + 2u * 8192u;
constexpr unsigned kOrthoSmem = 1024u + kOrthoStages * kOrthoStageBytes + 2u * 16384u + 256u;

struct OrthoTile {
    int tiles_i, tiles_j;  // tiles of the result
    int kblocks;           // 64 k each
    int down, down_next;   // bits the lift has gone down before and after this step
};

template <int MODE, typename T>
__global__ void __launch_bounds__(192, 1)
ortho_product_kernel(const __grid_constant__ CUtensorMap lmap, const __grid_constant__ CUtensorMap rmap,
                     const __grid_constant__ CUtensorMap omap, T* __restrict__ out, OrthoTile g, OrthoParams p) {
    extern __shared__ unsigned char ortho_smem_raw[];
    unsigned char* sm = ortho_smem_raw + ((1024u - (smem_addr(ortho_smem_raw) & 1023u)) & 1023u);
    unsigned char* res = sm + kOrthoStages * kOrthoStageBytes;  // two 128 x 64 fp16 planes, 128-byte swizzle
    uint64_t* bars = reinterpret_cast<uint64_t*>(res + 2u * 16384u);
    uint64_t *full = bars, *empty = bars + kOrthoStages, *done = bars + 2 * kOrthoStages, *extra = done + 1;
    uint32_t* slot = reinterpret_cast<uint32_t*>(extra + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const unsigned per = static_cast<unsigned>(g.tiles_i) * g.tiles_j;
    const int mat = static_cast<int>(blockIdx.x / per);
    const unsigned t = blockIdx.x - static_cast<unsigned>(mat) * per;
    const int i0 = static_cast<int>(t / g.tiles_j) * 128, j0 = static_cast<int>(t % g.tiles_j) * 64;

    if (tid == 0) {
        for (int s = 0; s < kOrthoStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(done, 1);
        mbar_init(extra, 1);
        fence_barrier_init();
    }
    if (warp == 0) tc::alloc(slot, 512u);
    tc::fence_before();
    __syncthreads();  // every CTA holds its tensor memory before the next launch may start
    tc::fence_after();
    const uint32_t tmem = *slot;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp == 0) {
        if (lane == 0) {
            if (MODE == kPoly) {
                // A's own tile, for the b A term
                mbar_expect_tx(extra, 2u * 16384u);
                for (int pl = 0; pl < 2; ++pl)
                    tc::tma_load_3d(res + pl * 16384, &lmap, j0, i0, pl * p.B + mat, extra);
                mbar_arrive(extra);
            }
            for (int kb = 0; kb < g.kblocks; ++kb) {
                const int s = kb % kOrthoStages;
                if (kb >= kOrthoStages &&
                    !mbar_wait_bounded(&empty[s], static_cast<unsigned>(kb / kOrthoStages - 1) & 1u, kCopyWaitLimitNs)) {
                    atomicOr(p.status, kStatusCopyTimeout);
                    break;
                }
                unsigned char* st = sm + s * kOrthoStageBytes;
                mbar_expect_tx(&full[s], kOrthoStageBytes);
                for (int pl = 0; pl < 2; ++pl) {
                    tc::tma_load_3d(st + pl * 16384, &lmap, kb * 64, i0, pl * p.B + mat, &full[s]);
                    if (MODE >= kApply)
                        tc::tma_load_3d(st + 32768 + pl * 8192, &rmap, j0, kb * 64, pl * p.B + mat, &full[s]);
                    else
                        tc::tma_load_3d(st + 32768 + pl * 8192, &rmap, kb * 64, j0, pl * p.B + mat, &full[s]);
                }
                mbar_arrive(&full[s]);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr bool mn = MODE >= kApply;
            constexpr uint32_t idesc = tc::idesc_f16(tc::kFmtF16, 64, false, mn);
            bool ok = true;
            for (int kb = 0; kb < g.kblocks; ++kb) {
                const int s = kb % kOrthoStages;
                ok = mbar_wait_bounded(&full[s], static_cast<unsigned>(kb / kOrthoStages) & 1u, kCopyWaitLimitNs);
                if (!ok) break;
                tc::fence_after();
                const unsigned a = smem_addr(sm + s * kOrthoStageBytes), b = a + 32768u;
                const uint32_t hh = tmem + static_cast<uint32_t>(kb % kOrthoHH) * 64u, cross = tmem + kOrthoHH * 64u;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const unsigned bo = b + (mn ? k * 2048u : k * 32u);
                    const uint64_t ah = tc::sw128_desc(a + k * 32u), al = tc::sw128_desc(a + 16384u + k * 32u);
                    const uint64_t bh = tc::sw128_desc(bo), bl = tc::sw128_desc(bo + 8192u);
                    tc::mma_f16(hh, ah, bh, idesc, kb >= kOrthoHH || k > 0);
                    tc::mma_f16(cross, ah, bl, idesc, (kb | k) != 0);
                    tc::mma_f16(cross, al, bh, idesc, true);
                }
                tc::commit(&empty[s]);
            }
            if (ok) tc::commit(done);
            else atomicOr(p.status, kStatusCopyTimeout);
        }
    } else {
        const int quarter = warp & 3, row = quarter * 32 + lane, et = tid - 64;
        bool ok = mbar_wait_bounded(done, 0u, kCopyWaitLimitNs);
        if (MODE == kPoly) ok = ok && mbar_wait_bounded(extra, 0u, kCopyWaitLimitNs);
        if (!ok) atomicOr(p.status, kStatusCopyTimeout);
        ok = tc::bar_and(1, 128, ok);  // one decision for all four warps
        tc::fence_after();
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const int nacc = min(g.kblocks, kOrthoHH);
        if (ok) {
            const int i = i0 + row;
            const int lift = max(0, p.lift[mat] - g.down);
            // powers of two that undo the lift (A carries it twice, A A four times)
            const float ub = scalbnf(p.b, -2 * lift), uc = scalbnf(p.c, -4 * lift);
            const float ux = scalbnf(1.f, MODE == kLast ? -lift : max(0, p.lift[mat] - g.down_next) - lift);
            float* stage = reinterpret_cast<float*>(sm);  // kLast: 128 x 65 floats over the idle ring
            for (int cc = 0; cc < 4; ++cc) {
                float v[16], w[16];
                tc::ld16(lanes + kOrthoHH * 64 + cc * 16, v);
                for (int q = 0; q < nacc; ++q) {
                    tc::ld16(lanes + q * 64 + cc * 16, w);
                    tc::wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] += w[e];
                }
                // chunks 2cc, 2cc + 1 of this row in the swizzled planes
                uint4* hp = reinterpret_cast<uint4*>(res + row * 128);
                uint4* lp = reinterpret_cast<uint4*>(res + 16384 + row * 128);
                if constexpr (MODE == kLast) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) stage[row * 65 + cc * 16 + e] = v[e] * (1.f / (kOrthoSP * kOrthoSX)) * ux;
                } else {
                    float scale;  // accumulator to plane units
                    if constexpr (MODE == kGram) scale = kOrthoSA / (kOrthoSX * kOrthoSX);
                    else if constexpr (MODE == kPoly) scale = kOrthoSP / (kOrthoSA * kOrthoSA);
                    else scale = ux / kOrthoSP;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int ch = (2 * cc + h) ^ (row & 7);
                        __half hi[8], lo[8];
                        if constexpr (MODE == kPoly) {
                            *reinterpret_cast<uint4*>(hi) = hp[ch];
                            *reinterpret_cast<uint4*>(lo) = lp[ch];
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            float r = v[h * 8 + e] * scale;
                            if constexpr (MODE == kPoly) {
                                const float av = (__half2float(hi[e]) + __half2float(lo[e])) * (kOrthoSP / kOrthoSA);
                                const int j = j0 + cc * 16 + h * 8 + e;
                                r = fmaf(uc, r, fmaf(ub, av, i == j ? p.a * kOrthoSP : 0.f));
                            }
                            ortho_split(r, hi[e], lo[e]);
                        }
                        hp[ch] = *reinterpret_cast<uint4*>(hi);
                        lp[ch] = *reinterpret_cast<uint4*>(lo);
                    }
                }
            }
            if constexpr (MODE == kLast) {
                tc::bar_sync(1, 128);
                const int ni = min(128, p.n - i0), nj = min(64, p.m - j0);
                T* o = out + static_cast<size_t>(mat) * p.n * p.m;
                for (int e = et; e < 8192; e += 128) {
                    // lanes along the result's contiguous side
                    const int ii = p.transposed ? e & 127 : e >> 6, jj = p.transposed ? e >> 7 : e & 63;
                    if (ii < ni && jj < nj) {
                        const size_t at = p.transposed ? static_cast<size_t>(j0 + jj) * p.n + i0 + ii
                                                       : static_cast<size_t>(i0 + ii) * p.m + j0 + jj;
                        o[at] = ortho_from_float<T>(stage[ii * 65 + jj]);
                    }
                }
            } else {
                fence_proxy_async();
                tc::bar_sync(1, 128);
                if (et == 0) {
                    for (int pl = 0; pl < 2; ++pl) tc::tma_store_3d(&omap, j0, i0, pl * p.B + mat, res + pl * 16384);
                    tc::bulk_commit();
                    tc::bulk_wait_all();
                }
            }
        }
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 0) tc::dealloc(tmem, 512u);
}

}  // namespace dcnv4
