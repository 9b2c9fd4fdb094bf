// sm_100a kernels of the Newton-Schulz orthogonalisation of a stack of weight
// updates. Each matrix X (R x C) is divided by its Frobenius norm (plus eps),
// which puts its singular values in [0, 1], and then
//   A = X X^T,  X <- a X + Q X,  Q = b A + c A A
// is repeated `steps` times: every singular value s goes through the odd
// polynomial a s + b s^3 + c s^5 while the singular vectors stay. The products
// are formed on the smaller side, n = min(R, C), m = max(R, C): X is taken
// transposed when R > C.
//
// Precision on the tensor cores. X, A and Q are kept as two fp16 planes, hi =
// fp16(v s) and lo = fp16(v s - hi): an entry is off by at most 2^-23 of itself
// (one unit of fp32's last place; half of all entries are exact) down to 2^-16
// of the largest that the planes take, 2^14, and by 2^-39 of that below (lo is
// subnormal there). X is kept lifted, Y = 2^l X with l the largest for which
// the iteration's bounds promise |Y| <= 4 (and so |A| <= 16): l follows the
// singular values' bound down to zero as well as up, and a matrix whose norm
// is far below eps starts with as large a Y as any. Q is lifted likewise, to
// at most 64. A product is three tensor-core products, hi hi + hi lo +
// lo hi, each exact, summed in fp32 (lo lo is some 2^-24 of it, but in X X^T and
// A A it adds up along the diagonal: small matrices, whose other errors are
// least, take it as well: 1.09e-6 -> 0.86e-6 for 78 x 10). The tensor cores' fp32
// additions truncate, so a long chain of them drifts one way: the hi hi terms
// go to three accumulators in turn and the small cross terms to one of their
// own, and the epilogue adds these with rounding. The step's a X is added there
// too, and not multiplied as the diagonal of P = a I + Q: next to it every
// further addition would truncate the sum by up to a unit of its last place,
// all downwards, step after step. (12 steps of 0.9, 0.05, 0 on 129 x 257: error
// 1.8e-6 that way, 2e-7 this way; fp32 products 4e-7.)
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
    int chunks;        // partial sums of squares per matrix (one kernel per product)
    int np, mp;        // row pitches of the n x n and n x m planes, multiples of 8 elements
    float a, b, c, eps;
    int* lift;         // [B] the lifts before the first step (one kernel per product)
    unsigned* status;
};

// Powers of two before step k, from the coefficients alone: X of every matrix
// can be lifted by 2^low, and X that started lifted by 2^l by 2^(l - down);
// Q of the step by 2^up. The larger lift is taken.
struct OrthoStep {
    int low, down, up;
};
__device__ __forceinline__ int ortho_lift(const OrthoStep& s, int start) { return max(s.low, start - s.down); }

// 2^e for e <= 127; 0 below fp32's normal numbers (b, c <= 192 and what they scale is as negligible there)
__device__ __forceinline__ float ortho_pow2(int e) { return e < -126 ? 0.f : __uint_as_float(static_cast<unsigned>(e + 127) << 23); }

// scales of the planes of Y, A, Q
constexpr float kOrthoSX = 4096.f, kOrthoSA = 1024.f, kOrthoSQ = 256.f;

template <typename T>
__device__ __forceinline__ T ortho_from_float(float v) {
    if constexpr (sizeof(T) == 4) return v;
    else if constexpr (std::is_same<T, __half>::value) return __float2half_rn(v);
    else return __float2bfloat16_rn(v);
}

// v as an fp16 pair
__device__ __forceinline__ void ortho_split(float v, __half& hi, __half& lo) {
    hi = __float2half_rn(v);
    lo = __float2half_rn(v - __half2float(hi));
}

// Sum of the squares of elements first, first + stride, ... of a matrix over
// one CTA, in fp64 (squares of fp32 values neither overflow nor vanish there);
// the result is thread 0's. ws: one double per warp.
template <typename T>
__device__ __forceinline__ double ortho_sumsq(const T* __restrict__ x, long long n, long long first, long long stride,
                                              double* ws) {
    double a = 0.0;
    for (long long i = first; i < n; i += 8 * stride) {
        float v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = i + q * stride < n ? ElemTraits<T>::to_float(__ldg(x + i + q * stride)) : 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q) a = fma(static_cast<double>(v[q]), static_cast<double>(v[q]), a);
    }
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if ((threadIdx.x & 31) == 0) ws[threadIdx.x >> 5] = a;
    __syncthreads();
    if (threadIdx.x == 0)
        for (unsigned i = 1; i < blockDim.x / 32; ++i) a += ws[i];
    return a;
}

// The division by den = norm + eps and the lift, from the sum of squares:
// v / den = (v 2^-k) / (den 2^-k) with den 2^-k in [1/2, 1), so nothing
// overflows whatever the norm; norm / den 2^lift lies in [2, 4], or lift is
// as large as fp32's exponents need.
struct OrthoScale {
    float mant;
    int k, lift;
};
__device__ __forceinline__ OrthoScale ortho_scale(double sum, float eps) {
    OrthoScale s;
    const double norm = sqrt(sum), den = norm + eps;
    s.k = 0;
    s.mant = isfinite(den) ? static_cast<float>(frexp(den, &s.k)) : __uint_as_float(0x7fc00000u);
    s.lift = norm > 0.0 && isfinite(den) ? min(122, max(2, 1 - ilogb(norm / den))) : 2;
    return s;
}

// 64 x 64 entries of X / den at (r0, c0) of a matrix as planes [2][B][n][mp]
// (lifted and scaled), transposed on the way when R > C; with `out` (no steps)
// the quotient itself. All threads of the CTA; tile: 64 x 65 floats.
template <typename T>
__device__ __forceinline__ void ortho_start_tile(const T* __restrict__ x, __half* __restrict__ planes, T* __restrict__ out,
                                                 int mat, int r0, int c0, const OrthoScale& sc, float* tile,
                                                 const OrthoParams& p) {
    const size_t base = static_cast<size_t>(mat) * p.R * p.C;
    // scale, then divide: exact powers of two around one rounding
    const int shift = out ? -sc.k : sc.lift - sc.k;
    for (int q = threadIdx.x; q < 4096; q += blockDim.x) {
        const int r = r0 + (q >> 6), c = c0 + (q & 63);
        if (r < p.R && c < p.C) {
            const size_t at = base + static_cast<size_t>(r) * p.C + c;
            const float v = scalbnf(ElemTraits<T>::to_float(__ldg(x + at)), shift) / sc.mant;
            if (out) out[at] = ortho_from_float<T>(v);
            tile[(q >> 6) * 65 + (q & 63)] = v;
        }
    }
    if (out) return;
    __syncthreads();
    const size_t plane = static_cast<size_t>(p.B) * p.n * p.mp;
    __half* o = planes + static_cast<size_t>(mat) * p.n * p.mp;
    const int i0 = p.transposed ? c0 : r0, j0 = p.transposed ? r0 : c0;
    for (int q = threadIdx.x; q < 2048; q += blockDim.x) {
        const int i = q >> 5, j = (q & 31) * 2;
        if (i0 + i < p.n && j0 + j < p.m) {
            // pairs of columns (the pitch is a multiple of 8; a last odd column's partner is padding)
            __half2 hi, lo;
            const float a = p.transposed ? tile[j * 65 + i] : tile[i * 65 + j];
            const float b = j0 + j + 1 < p.m ? (p.transposed ? tile[(j + 1) * 65 + i] : tile[i * 65 + j + 1]) : 0.f;
            ortho_split(a * kOrthoSX, hi.x, lo.x);
            ortho_split(b * kOrthoSX, hi.y, lo.y);
            const size_t at = static_cast<size_t>(i0 + i) * p.mp + j0 + j;
            *reinterpret_cast<__half2*>(o + at) = hi;
            *reinterpret_cast<__half2*>(o + plane + at) = lo;
        }
    }
    __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(256)
ortho_sumsq_kernel(const T* __restrict__ x, double* __restrict__ part, OrthoParams p) {
    __shared__ double ws[8];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long n = static_cast<long long>(p.R) * p.C;
    const int mat = blockIdx.x / p.chunks, ch = blockIdx.x - mat * p.chunks;
    const double a = ortho_sumsq(x + mat * n, n, static_cast<long long>(ch) * 256 + threadIdx.x,
                                 static_cast<long long>(p.chunks) * 256, ws);
    if (threadIdx.x == 0) part[blockIdx.x] = a;
}

template <typename T>
__global__ void __launch_bounds__(256)
ortho_start_kernel(const T* __restrict__ x, const double* __restrict__ part, __half* __restrict__ planes,
                   T* __restrict__ out, OrthoParams p) {
    __shared__ float tile[64 * 65];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const unsigned tr = static_cast<unsigned>((p.R + 63) / 64), tcn = static_cast<unsigned>((p.C + 63) / 64);
    const int mat = static_cast<int>(blockIdx.x / (tr * tcn));
    const unsigned t = blockIdx.x - static_cast<unsigned>(mat) * tr * tcn;
    // at most 64 partial sums: two per lane, then a fixed tree
    const int lane = threadIdx.x & 31;
    const double* pm = part + static_cast<size_t>(mat) * p.chunks;
    double sum = (lane < p.chunks ? pm[lane] : 0.0) + (lane + 32 < p.chunks ? pm[lane + 32] : 0.0);
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const OrthoScale sc = ortho_scale(sum, p.eps);
    if (t == 0 && threadIdx.x == 0) p.lift[mat] = sc.lift;
    ortho_start_tile(x, planes, out, mat, static_cast<int>(t / tcn) * 64, static_cast<int>(t % tcn) * 64, sc, tile, p);
}

// Four accumulators at `at`, `step` columns apart (the cross terms' last), 16
// columns each, as one rounded sum.
__device__ __forceinline__ void ortho_sum4(uint32_t at, uint32_t step, float (&v)[16]) {
    float w[2][16];
    tc::ld16(at + 3 * step, v);
    tc::ld16(at + 2 * step, w[0]);
    tc::ld16(at + step, w[1]);
    tc::wait_ld();
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = (v[e] + w[0][e]) + w[1][e];
    tc::ld16(at, w[0]);
    tc::wait_ld();
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] += w[0][e];
}

// One product of the iteration, a 128 x 64 tile of the result per CTA:
//   kGram:  A = X X^T          (k over m; both operands K-major rows of X)
//   kPoly:  Q = bA + cAA   (k over n; A is symmetric: both K-major)
//   kApply: X' = aX + QX   (k over n; X's rows run along the result's
//                           columns: an MN-major operand)
//   kLast:  kApply with the result rounded to T and written to `out`
// Warp 0 (one lane) loads 64 k at a time by TMA: 128 rows x 64 k of the left
// planes, 64 x 64 of the right ones, in a ring of STAGES; warp 1 issues the
// products; warps 2..9 read the accumulators, form the result
// and write it as planes through shared memory (the idle ring) and TMA. A
// product's time is mostly latency (per tile: first load 0.8 us, products 0.3
// us per 64 k, epilogue 0.5, store 0.6; the launch about 2 us more), so the
// ring is deep, four stages, while the tiles fit the SMs once; when there are
// more tiles than SMs, two stages leave room for two CTAs per SM (256 columns
// of tensor memory each) whose latencies overlap. Whole iteration in fp32, 432
// x 256: 18 matrices (144 and 252 tiles) 119 us, all products with four stages
// 134, with two 145; 40 matrices 237 with two, 295 with four. 4 of 864 x 512
// in bf16: 154 us (147 in one run of k).
constexpr int kGram = 0, kPoly = 1, kApply = 2, kLast = 3;
constexpr int kOrthoEpi = 256, kOrthoThreads = 64 + kOrthoEpi;
// The accumulators are read out, added in registers and begun anew every this
// many 64 k, so that truncation does not grow with k: one matrix of 809 x 840
// has an error of 1.1e-6 so, 1.9e-6 without (fp32 matrix products: 2.8e-6).
constexpr int kOrthoRun = 8;
constexpr unsigned kOrthoStageBytes = 2u * 16384u + 2u * 8192u;
constexpr unsigned ortho_smem(int stages) { return 1024u + stages * kOrthoStageBytes + 128u; }

struct OrthoTiles {
    int tiles_i, tiles_j;  // tiles of the result
    int kblocks;           // 64 k each
    OrthoStep now, next;   // before and after this step
};

// RUNS: more than one run.
template <int MODE, typename T, int STAGES, bool RUNS>
__global__ void __launch_bounds__(kOrthoThreads, STAGES == 2 ? 2 : 1)
ortho_product_kernel(const __grid_constant__ CUtensorMap lmap, const __grid_constant__ CUtensorMap rmap,
                     const __grid_constant__ CUtensorMap omap, T* __restrict__ out, OrthoTiles g, OrthoParams p) {
    extern __shared__ unsigned char ortho_smem_raw[];
    unsigned char* sm = ortho_smem_raw + ((1024u - (smem_addr(ortho_smem_raw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + STAGES * kOrthoStageBytes);
    uint64_t *full = bars, *empty = bars + STAGES, *done = bars + 2 * STAGES, *drained = done + 1;
    uint64_t* drain = drained + 1;
    uint32_t* slot = reinterpret_cast<uint32_t*>(drain + 1);
    const int tid = threadIdx.x, warp = static_cast<int>(tc::uniform(threadIdx.x >> 5)), lane = tid & 31;
    const unsigned per = static_cast<unsigned>(g.tiles_i) * g.tiles_j;
    const int mat = static_cast<int>(blockIdx.x / per);
    const unsigned t = blockIdx.x - static_cast<unsigned>(mat) * per;
    const int i0 = static_cast<int>(t / g.tiles_j) * 128, j0 = static_cast<int>(t % g.tiles_j) * 64;

    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(done, 1);
        mbar_init(drained, kOrthoEpi);
        mbar_init(drain, 1);
        fence_barrier_init();
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&lmap)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&rmap)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&omap)) : "memory");
    }
    if (warp == 0) tc::alloc(slot, 256u);
    tc::fence_before();
    __syncthreads();  // every CTA holds its tensor memory before the next launch may start
    tc::fence_after();
    const uint32_t tmem = tc::uniform(*slot);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // The epilogue needs the tile's own entries of A (kPoly) or X (kApply, kLast), and finds them in the ring: the
    // order of k goes round so that the block of the left operand with this tile's columns, or the two of the right
    // one with its rows, come last.
    int k0 = 0;
    if constexpr (MODE == kPoly) k0 = (j0 / 64 + 1) % g.kblocks;
    else if constexpr (MODE >= kApply) k0 = (i0 / 64 + 2) % g.kblocks;
    bool ok = true;
    int loads = 0;  // the loading lane's steps so far

    if (warp == 0) {
        if (lane == 0) {
            for (int kb = 0; kb < g.kblocks; ++kb) {
                const int s = kb % STAGES;
                if (kb >= STAGES)
                    ok = mbar_wait_bounded(&empty[s], static_cast<unsigned>(kb / STAGES - 1) & 1u, kCopyWaitLimitNs);
                if (!ok) break;
                unsigned char* st = sm + s * kOrthoStageBytes;
                const int k = (kb + k0 < g.kblocks ? kb + k0 : kb + k0 - g.kblocks) * 64;
                mbar_expect_tx(&full[s], kOrthoStageBytes);
                for (int pl = 0; pl < 2; ++pl) {
                    tc::tma_load_3d(st + pl * 16384, &lmap, k, i0, pl * p.B + mat, &full[s]);
                    if (MODE >= kApply)
                        tc::tma_load_3d(st + 32768 + pl * 8192, &rmap, j0, k, pl * p.B + mat, &full[s]);
                    else
                        tc::tma_load_3d(st + 32768 + pl * 8192, &rmap, k, j0, pl * p.B + mat, &full[s]);
                }
                mbar_arrive(&full[s]);
                loads = kb + 1;
            }
        }
    } else if (warp == 1) {
        constexpr bool mn = MODE >= kApply;
        constexpr uint32_t idesc = tc::idesc_f16(tc::kFmtF16, 64, false, mn);
        const uint32_t lead = tc::lead_lane();
        for (int kb = 0; kb < g.kblocks; ++kb) {
            const int s = kb % STAGES;
            const int t = RUNS ? kb % kOrthoRun : kb;
            ok = tc::warp_wait(&full[s], static_cast<unsigned>(kb / STAGES) & 1u, kCopyWaitLimitNs);
            if (RUNS && t == 0 && kb > 0) ok = ok && tc::warp_wait(drained, static_cast<unsigned>(kb / kOrthoRun - 1) & 1u, kCopyWaitLimitNs);
            if (!ok) break;
            tc::fence_after();
            const unsigned base = smem_addr(sm + s * kOrthoStageBytes);
            const uint32_t a = tc::sw128(base), b = tc::sw128(base + 32768u);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t ah = a + k * 2, al = ah + 1024, bh = b + k * (mn ? 128 : 2), bl = bh + 512;
                tc::mma_f16(tmem + 192u, ah, bl, idesc, t > 0 || k > 0, lead);
                tc::mma_f16(tmem + 192u, al, bh, idesc, true, lead);
                tc::mma_f16(tmem + (k % 3) * 64u, ah, bh, idesc, t > 0 || k >= 3, lead);
            }
            if (lead) {
                tc::commit(&empty[s]);
                if (RUNS && t == kOrthoRun - 1 && kb + 1 < g.kblocks) tc::commit(done);
            }
        }
        if (ok && lead) tc::commit(done);
    } else {
        const int quarter = warp & 3, row = quarter * 32 + lane, et = tid - 64, half = (warp - 2) >> 2;
        const int lift = p.lift[mat];
        const int now = ortho_lift(g.now, lift), next = ortho_lift(g.next, lift);
        // where this thread's own row lies: hi and, a plane further on, lo (kApply and kLast: rows past the blocks of
        // 64 that there are lie past the matrix)
        const int own_kb = MODE == kPoly ? g.kblocks - 1 : max(0, g.kblocks - 2 + (row >> 6)), own_s = own_kb % STAGES;
        const unsigned char* own_row = sm + own_s * kOrthoStageBytes + (MODE == kPoly ? row * 128 : 32768 + (row & 63) * 128);
        constexpr unsigned own_plane = MODE == kPoly ? 16384u : 8192u;
        // powers of two that undo the lifts (A carries X's twice, A A four times) and give Q and the next X theirs
        // (the last ones in two factors: together they can be too small for a float)
        const int up = g.now.up, undo = MODE == kLast ? -now : next - now;
        const float ux = ortho_pow2(MODE == kLast ? undo / 2 : undo), uy = ortho_pow2(undo - undo / 2) * (1.f / kOrthoSX);
        const float uq = ortho_pow2(-up) * (1.f / kOrthoSQ);
        const float ub = p.b * ortho_pow2(up - 2 * now), uc = p.c * ortho_pow2(up - 4 * now) * (kOrthoSQ / (kOrthoSA * kOrthoSA));
        const uint32_t at = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + half * 32;
        float sum[2][16];  // the runs before the last
        unsigned r = 0;
        if constexpr (RUNS) {
#pragma unroll
            for (int cc = 0; cc < 2; ++cc)
#pragma unroll
                for (int e = 0; e < 16; ++e) sum[cc][e] = 0.f;
            for (; static_cast<int>(r + 1) * kOrthoRun < g.kblocks; ++r) {
                ok = tc::bar_and(1, kOrthoEpi, mbar_wait_bounded(done, r & 1u, kCopyWaitLimitNs));
                if (!ok) break;
                tc::fence_after();
#pragma unroll
                for (int cc = 0; cc < 2; ++cc) {
                    float v[16];
                    ortho_sum4(at + cc * 16, 64u, v);
#pragma unroll
                    for (int e = 0; e < 16; ++e) sum[cc][e] += v[e];
                }
                tc::fence_before();
                mbar_arrive(drained);
            }
        }
        // one decision for all the warps
        ok = ok && mbar_wait_bounded(done, r & 1u, kCopyWaitLimitNs);
        // (long complete: what makes the loads' bytes this thread's to read)
        if (MODE != kGram) ok = ok && mbar_wait_bounded(&full[own_s], static_cast<unsigned>(own_kb / STAGES) & 1u, kCopyWaitLimitNs);
        ok = tc::bar_and(1, kOrthoEpi, ok);
        if (ok) {
            tc::fence_after();
            float* fres = reinterpret_cast<float*>(sm);
            uint4 *hp = reinterpret_cast<uint4*>(sm + row * 128), *lp = reinterpret_cast<uint4*>(sm + 16384 + row * 128);
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) {
                float v[16];
                ortho_sum4(at + cc * 16, 64u, v);
                if constexpr (RUNS)
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] += sum[cc][e];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    __half hi[8], lo[8];
                    const int ch = (half * 4 + cc * 2 + h) ^ (row & 7);
                    if constexpr (MODE != kGram) {
                        // (kPoly: possibly the very chunk that the result takes below)
                        *reinterpret_cast<uint4*>(hi) = reinterpret_cast<const uint4*>(own_row)[ch];
                        *reinterpret_cast<uint4*>(lo) = reinterpret_cast<const uint4*>(own_row + own_plane)[ch];
                    }
                    // accumulators to plane units, with A's or X's own term added in fp32
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float r = v[h * 8 + e];
                        if constexpr (MODE == kGram) {
                            r *= kOrthoSA / (kOrthoSX * kOrthoSX);
                        } else {
                            const float own = __half2float(hi[e]) + __half2float(lo[e]);
                            if constexpr (MODE == kPoly)
                                r = fmaf(uc, r, ub * (own * (kOrthoSQ / kOrthoSA)));
                            else r = fmaf(uq, r, p.a * own) * ux;
                        }
                        if constexpr (MODE == kLast) fres[row * 64 + ((half * 32 + cc * 16 + h * 8 + e) ^ (row & 31))] = r * uy;
                        else ortho_split(r, hi[e], lo[e]);
                    }
                    if constexpr (MODE != kLast) {
                        hp[ch] = *reinterpret_cast<uint4*>(hi);
                        lp[ch] = *reinterpret_cast<uint4*>(lo);
                    }
                }
            }
            if constexpr (MODE == kLast) {
                tc::bar_sync(1, kOrthoEpi);
                const int ni = min(128, p.n - i0), nj = min(64, p.m - j0);
                T* o = out + static_cast<size_t>(mat) * p.n * p.m;
                for (int e = et; e < 8192; e += kOrthoEpi) {
                    // lanes along the result's contiguous side
                    const int ii = p.transposed ? e & 127 : e >> 6, jj = p.transposed ? e >> 7 : e & 63;
                    if (ii < ni && jj < nj) {
                        const size_t to = p.transposed ? static_cast<size_t>(j0 + jj) * p.n + i0 + ii
                                                       : static_cast<size_t>(i0 + ii) * p.m + j0 + jj;
                        o[to] = ortho_from_float<T>(fres[ii * 64 + (jj ^ (ii & 31))]);
                    }
                }
            } else {
                fence_proxy_async();
                tc::bar_sync(1, kOrthoEpi);
                if (et == 0) {
                    for (int pl = 0; pl < 2; ++pl) tc::tma_store_3d(&omap, j0, i0, pl * p.B + mat, sm + pl * 16384);
                    tc::bulk_commit();
                    tc::bulk_wait_all();
                }
            }
        }
    }
    if (!ok) atomicOr(p.status, kStatusCopyTimeout);
    tc::fence_before();
    if (!__syncthreads_and(ok)) {
        if (warp == 0 && lane == 0) tc::drain_loads<STAGES>(full, loads, STAGES);
        if (warp == 1) tc::drain_products(drain);
        __syncthreads();
    }
    tc::fence_after();
    if (warp == 0) tc::dealloc(tmem, 256u);
}

// The whole iteration of one small matrix (n <= 128, X and A together at most
// seven blocks of 64 columns) in one CTA, its planes in shared memory all the
// while. A block is 64 columns: the hi plane and the lo plane, 128 rows of 128
// bytes each, 128-byte swizzle; rows and columns past the matrix are zero. X's
// blocks serve as both operands of the Gram product (K-major) and as the right
// one of the application (MN-major), A's as both of the polynomial, which
// overwrites them with Q. One warp issues a product's instructions, then all
// warps turn the accumulators into the next operand. What bounds it is the
// chain of 3 * steps dependent products between two barriers each: for 108 x 64
// 28, 16 and 12 instructions of 49 to 58 cycles, some 2,900 cycles a step of the
// 11,000 that it takes. 4 matrices of 108 x 64 take 31 us (61 through the
// kernels above), 18 of 216 x 128 75 us (84), 300 of 108 x 64 94 us (163).
constexpr int kOrthoSmallThreads = 512, kOrthoSmallBlocks = 7;
constexpr unsigned kOrthoBlock = 2u * 16384u;
constexpr int kOrthoMaxSteps = 64;
struct OrthoSmall {
    int steps, xb, nb;       // blocks of X, of A
    int n16, m16;            // n, m rounded up to 16
    unsigned tmem_cols;
    OrthoStep step[kOrthoMaxSteps + 1];
};

// hi and lo of entry (i, j), scaled, in a row of blocks
__device__ __forceinline__ void ortho_put(unsigned char* blocks, int i, int j, float v) {
    __half hi, lo;
    ortho_split(v, hi, lo);
    unsigned char* at = blocks + (j >> 6) * kOrthoBlock + i * 128 + ((((j & 63) >> 3) ^ (i & 7)) << 4) + (j & 7) * 2;
    *reinterpret_cast<__half*>(at) = hi;
    *reinterpret_cast<__half*>(at + 16384) = lo;
}

template <typename T>
__global__ void __launch_bounds__(kOrthoSmallThreads, 1)
ortho_small_kernel(const T* __restrict__ x, T* __restrict__ out, const __grid_constant__ OrthoSmall g, OrthoParams p) {
    extern __shared__ unsigned char ortho_smem_raw[];
    __shared__ double ws[kOrthoSmallThreads / 32];
    __shared__ double total;
    __shared__ __align__(8) uint64_t done_bar;
    __shared__ uint32_t slot;
    unsigned char* xs = ortho_smem_raw + ((1024u - (smem_addr(ortho_smem_raw) & 1023u)) & 1023u);
    unsigned char* as = xs + g.xb * kOrthoBlock;
    const int tid = threadIdx.x, warp = static_cast<int>(tc::uniform(threadIdx.x >> 5)), lane = tid & 31;
    const int quarter = warp & 3, row = quarter * 32 + lane, part = warp >> 2;
    if (tid == 0) {
        mbar_init(&done_bar, 1);
        fence_barrier_init();
    }
    if (warp == 0) tc::alloc(&slot, g.tmem_cols);
    for (unsigned i = tid; i < (g.xb + g.nb) * kOrthoBlock / 16; i += kOrthoSmallThreads)
        reinterpret_cast<uint4*>(xs)[i] = make_uint4(0, 0, 0, 0);
    tc::fence_before();
    __syncthreads();  // every CTA holds its tensor memory before the next launch may start
    tc::fence_after();
    const uint32_t tmem = tc::uniform(slot), lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int mat = blockIdx.x, count = p.R * p.C;
    const T* xm = x + static_cast<size_t>(mat) * count;
    const double a = ortho_sumsq(xm, count, tid, kOrthoSmallThreads, ws);
    if (tid == 0) total = a;
    __syncthreads();
    const OrthoScale sc = ortho_scale(total, p.eps);
    for (int e = tid; e < count; e += kOrthoSmallThreads) {
        const int r = e / p.C, c = e - r * p.C;
        const float v = scalbnf(ElemTraits<T>::to_float(__ldg(xm + e)), sc.lift - sc.k) / sc.mant;
        ortho_put(xs, p.transposed ? c : r, p.transposed ? r : c, v * kOrthoSX);
    }
    fence_proxy_async();
    __syncthreads();

    unsigned phase = 0;
    bool ok = true;
    // hands the operands over to the tensor cores, lets warp 0 issue, and waits for the products
    auto product = [&](auto issue) {
        fence_proxy_async();
        tc::fence_before();
        __syncthreads();
        if (warp == 0) {
            tc::fence_after();
            const uint32_t lead = tc::lead_lane();
            issue(lead);
            if (lead) tc::commit(&done_bar);
        }
        ok = __syncthreads_and(mbar_wait_bounded(&done_bar, phase & 1u, kCopyWaitLimitNs)) != 0;
        // given up: the products in flight are waited for once more before the CTA leaves
        if (!ok) mbar_wait_bounded(&done_bar, phase & 1u, kCopyWaitLimitNs);
        ++phase;
        tc::fence_after();
    };
    // square products: n columns, four accumulators n16 columns apart; K-major operands with ksteps of 16 k
    auto square = [&](unsigned base, int ksteps, uint32_t lead) {
        const uint32_t idesc = tc::idesc_f16(tc::kFmtF16, g.n16, false, false);
        const uint32_t cross = tmem + 3 * g.n16;
        uint32_t h = tc::sw128(base), high = tmem;
#pragma unroll 1
        for (int k = 0; k < ksteps; ++k) {
            const uint32_t l = h + 1024;
            tc::mma_f16(cross, h, l, idesc, k > 0, lead);
            tc::mma_f16(cross, l, h, idesc, true, lead);
            tc::mma_f16(cross, l, l, idesc, true, lead);
            tc::mma_f16(high, h, h, idesc, k >= 3, lead);
            high = high == tmem + 2 * g.n16 ? tmem : high + g.n16;
            h += (k & 3) == 3 ? kOrthoBlock / 16 - 6 : 2;  // 16 k further, or the next block of 64
        }
    };
    const int nchunks = g.n16 / 16;
    for (int s = 0; s < g.steps && ok; ++s) {
        const int now = ortho_lift(g.step[s], sc.lift), next = ortho_lift(g.step[s + 1], sc.lift), up = g.step[s].up;
        // accumulators of order 0 past the number of k steps hold nothing: left out of the sums
        auto sums = [&](int cc, int ksteps, int step, float (&v)[16]) {
            if (ksteps >= 3) {
                ortho_sum4(lanes + cc * 16, step, v);
            } else {
                float w[16];
                tc::ld16(lanes + 3 * step + cc * 16, v);
                for (int q = 0; q < ksteps; ++q) {
                    tc::ld16(lanes + q * step + cc * 16, w);
                    tc::wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] += w[e];
                }
            }
        };
        auto chunk_of = [&](unsigned char* blocks, int cc, int h) {
            return reinterpret_cast<uint4*>(blocks + (cc >> 2) * kOrthoBlock + row * 128 + ((((cc & 3) * 2 + h) ^ (row & 7)) << 4));
        };
        auto put_chunk = [&](unsigned char* blocks, int cc, int h, const __half (&hi)[8], const __half (&lo)[8]) {
            uint4* at = chunk_of(blocks, cc, h);
            *at = *reinterpret_cast<const uint4*>(hi);
            at[1024] = *reinterpret_cast<const uint4*>(lo);
        };
        // A = X X^T
        product([&](uint32_t lead) { square(smem_addr(xs), g.m16 / 16, lead); });
        if (!ok) break;
        for (int cc = part; cc < nchunks; cc += 4) {
            float v[16];
            sums(cc, g.m16 / 16, g.n16, v);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                __half hi[8], lo[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) ortho_split(v[h * 8 + e] * (kOrthoSA / (kOrthoSX * kOrthoSX)), hi[e], lo[e]);
                put_chunk(as, cc, h, hi, lo);
            }
        }
        // Q = b A + c A A, over A
        product([&](uint32_t lead) { square(smem_addr(as), nchunks, lead); });
        if (!ok) break;
        const float ub = p.b * ortho_pow2(up - 2 * now);
        const float uc = p.c * ortho_pow2(up - 4 * now) * (kOrthoSQ / (kOrthoSA * kOrthoSA));
        for (int cc = part; cc < nchunks; cc += 4) {
            float v[16];
            sums(cc, nchunks, g.n16, v);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                __half hi[8], lo[8];
                const uint4* at = chunk_of(as, cc, h);
                *reinterpret_cast<uint4*>(hi) = *at;
                *reinterpret_cast<uint4*>(lo) = at[1024];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float av = (__half2float(hi[e]) + __half2float(lo[e])) * (kOrthoSQ / kOrthoSA);
                    ortho_split(fmaf(uc, v[h * 8 + e], ub * av), hi[e], lo[e]);
                }
                put_chunk(as, cc, h, hi, lo);
            }
        }
        // X = a X + Q X, up to 128 columns at a time, four accumulators as above `width` apart
        const bool last = s + 1 == g.steps;
        for (int j0 = 0; j0 < g.m16 && ok; j0 += 128) {
            const int width = min(128, g.m16 - j0);
            product([&](uint32_t lead) {
                const uint32_t idesc = tc::idesc_f16(tc::kFmtF16, width, false, true);
                uint32_t ah = tc::sw128(smem_addr(as)), bh = tc::sw128(smem_addr(xs) + (j0 >> 6) * kOrthoBlock, kOrthoBlock);
                const uint32_t cross = tmem + 3 * width;
                uint32_t high = tmem;
#pragma unroll 1
                for (int k = 0; k < nchunks; ++k, bh += 128) {
                    const uint32_t al = ah + 1024, bl = bh + 1024;
                    tc::mma_f16(cross, ah, bl, idesc, k > 0, lead);
                    tc::mma_f16(cross, al, bh, idesc, true, lead);
                    tc::mma_f16(high, ah, bh, idesc, k >= 3, lead);
                    high = high == tmem + 2 * width ? tmem : high + width;
                    ah += (k & 3) == 3 ? kOrthoBlock / 16 - 6 : 2;
                }
            });
            if (!ok) break;
            // (the last powers of two as two factors: together they can be too small for a float)
            const int undo = last ? -now : next - now;
            const float ux = ortho_pow2(last ? undo / 2 : undo), uq = ortho_pow2(-up) * (1.f / kOrthoSQ);
            const float uy = last ? ortho_pow2(undo - undo / 2) * (1.f / kOrthoSX) : 1.f;
            for (int cc = part; cc < width / 16; cc += 4) {
                float v[16];
                sums(cc, nchunks, width, v);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    __half hi[8], lo[8];
                    const uint4* at = chunk_of(xs, (j0 >> 4) + cc, h);
                    *reinterpret_cast<uint4*>(hi) = *at;
                    *reinterpret_cast<uint4*>(lo) = at[1024];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[h * 8 + e] = fmaf(uq, v[h * 8 + e], p.a * (__half2float(hi[e]) + __half2float(lo[e]))) * ux * uy;
                }
                if (last) {
                    // straight to `out`: a lane's 16 columns are neighbours (R <= C), or the lanes are (R > C)
                    T* o = out + static_cast<size_t>(mat) * count;
                    const int j = j0 + cc * 16;
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (row < p.n && j + e < p.m)
                            o[p.transposed ? (j + e) * p.n + row : row * p.m + j + e] = ortho_from_float<T>(v[e]);
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        __half hi[8], lo[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) ortho_split(v[h * 8 + e], hi[e], lo[e]);
                        put_chunk(xs, (j0 >> 4) + cc, h, hi, lo);
                    }
                }
            }
        }
    }
    if (!ok) atomicOr(p.status, kStatusCopyTimeout);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 0) tc::dealloc(tmem, g.tmem_cols);
}

}  // namespace dcnv4
