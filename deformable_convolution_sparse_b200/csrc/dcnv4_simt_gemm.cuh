// A plain fp32 tile product on the CUDA cores, its operands and result given
// by functors: D(i, j) = sum_k A(i, k) * B(k, j) for a 64 x 64 tile per CTA of
// 256 threads, 16 k at a time through shared memory, 4 x 4 sums per thread.
#pragma once

namespace dcnv4 {

constexpr int kSimtTile = 64, kSimtK = 16;

struct SimtSmem {
    float a[kSimtK][kSimtTile + 4];
    float b[kSimtK][kSimtTile + 4];
};

// K range [k0, k1); loads outside i < I, j < J, k < k1 give 0.
template <typename LA, typename LB, typename ST>
__device__ __forceinline__ void simt_tile(SimtSmem& sm, int i0, int j0, int I, int J, int k0, int k1, LA la, LB lb,
                                          ST st) {
    const int tid = threadIdx.x, ti = tid >> 4, tj = tid & 15;
    float acc[4][4] = {};
    for (int k = k0; k < k1; k += kSimtK) {
        for (int e = tid; e < kSimtK * kSimtTile; e += 256) {
            {
                const int i = e / kSimtK, kk = e % kSimtK;
                sm.a[kk][i] = (i0 + i < I && k + kk < k1) ? la(i0 + i, k + kk) : 0.f;
            }
            {
                const int j = e % kSimtTile, kk = e / kSimtTile;
                sm.b[kk][j] = (j0 + j < J && k + kk < k1) ? lb(k + kk, j0 + j) : 0.f;
            }
        }
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < kSimtK; ++kk) {
            float a[4], b[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                a[q] = sm.a[kk][ti * 4 + q];
                b[q] = sm.b[kk][tj * 4 + q];
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[q][r] = fmaf(a[q], b[r], acc[q][r]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (i0 + ti * 4 + q < I && j0 + tj * 4 + r < J) st(i0 + ti * 4 + q, j0 + tj * 4 + r, acc[q][r]);
}

}  // namespace dcnv4
