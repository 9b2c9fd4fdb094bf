// Host side of dcnv4_orthogonalize (declared in include/dcnv4.h).
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
#include "dcnv4_orthogonalize.cuh"

namespace {

#include "dcnv4_host_common.inl"

#include "dcnv4_unit_common.inl"

constexpr int kMaxSteps = dcnv4::kOrthoMaxSteps;

int check_stack(int B, int R, int C, int dtype) {
    if (B < 0 || R <= 0 || C <= 0) return DCNV4_ERR_SHAPE;
    if (!elem_size(dtype)) return DCNV4_ERR_DTYPE;
    // rows of the planes are padded to 8 elements; sizes are below 2^31, so the products fit 63 bits
    const long long rc = static_cast<long long>(std::min(R, C)) * ((static_cast<long long>(std::max(R, C)) + 7) / 8 * 8);
    if (rc >= kLimit || (B > 0 && rc > (kLimit - 1) / B)) return DCNV4_ERR_TOO_LARGE;
    return DCNV4_OK;
}

// The largest |a s + b s^3 + c s^5| over s in [0, r]: at r or where the
// derivative a + 3 b u + 5 c u^2 vanishes, u = s^2.
double poly_bound(double a, double b, double c, double r) {
    auto f = [&](double s) { return std::fabs(s * (a + s * s * (b + c * s * s))); };
    double best = f(r);
    const double qa = 5.0 * c, qb = 3.0 * b, qc = a, disc = qb * qb - 4.0 * qa * qc;
    if (qa == 0.0) {
        if (qb != 0.0 && -qc / qb > 0.0 && -qc / qb < r * r) best = std::max(best, f(std::sqrt(-qc / qb)));
    } else if (disc >= 0.0) {
        for (double sg : {-1.0, 1.0}) {
            const double u = (-qb + sg * std::sqrt(disc)) / (2.0 * qa);
            if (u > 0.0 && u < r * r) best = std::max(best, f(std::sqrt(u)));
        }
    }
    return best;
}

// Bounds of the iteration, and the powers of two that keep its planes in range
// (dcnv4::OrthoStep). Singular values start in [0, 1]; r bounds them before
// step k, grown the product of the steps' largest factors |a + b s^2 + c s^4|
// (what a matrix far smaller than 1 can have grown by). False: a step may lift
// a singular value above 4 or its factor above 64; or small singular values,
// whose factor is a, may fall to less than 1/16 of either bound, out of the
// range in which the planes hold them.
bool iteration_bounds(double a, double b, double c, int steps, dcnv4::OrthoStep* step) {
    // held to what ldexp and the kernels' exponents take; a matrix of 2^-700 is 0 in fp32 whatever its planes hold
    auto log2_floor = [](double v) { return v > 0.0 ? std::clamp(std::ilogb(v), -700, 700) : -700; };
    auto log2_ceil = [&](double v) { return log2_floor(v) + (v > std::ldexp(1.0, log2_floor(v)) ? 1 : 0); };
    double r = 1.0, grown = 1.0, linear = 1.0;
    for (int k = 0;; ++k) {
        step[k].low = log2_floor(4.0 / std::max(r, 1e-300));
        step[k].down = log2_ceil(grown);
        step[k].up = 0;
        if (k > 0) {
            // the change of a step is a float's factor; a lift below the largest is as safe
            step[k].low = std::min(step[k].low, step[k - 1].low + 120);
            step[k].down = std::max(step[k].down, step[k - 1].down - 120);
        }
        if (k == steps) return true;
        // extremes of the factor a + b u + c u^2 over u = s^2 in [0, r^2], and of Q's singular values, less a
        const double end = b * r * r + c * r * r * r * r, at = c != 0.0 ? -b / (2.0 * c) : 0.0;
        const double inside = at > 0.0 && at < r * r ? b * at + c * at * at : 0.0;
        const double q = std::max({std::fabs(a), std::fabs(a + end), std::fabs(a + inside)});
        const double only = std::max(std::fabs(end), std::fabs(inside));
        if (!(q <= 64.0)) return false;
        if (only > 0.0) step[k].up = std::min(120, log2_floor(64.0 / only));  // (0: Q is zero)
        r = poly_bound(a, b, c, r);
        grown *= q;
        linear *= std::fabs(a);
        if (!(r <= 4.0) || !(std::max(r, grown) <= 16.0 * linear)) return false;
    }
}

dcnv4::OrthoParams make_params(int B, int R, int C) {
    dcnv4::OrthoParams p{};
    p.B = B; p.R = R; p.C = C;
    p.n = std::min(R, C); p.m = std::max(R, C); p.transposed = R > C ? 1 : 0;
    p.np = (p.n + 7) / 8 * 8;
    p.mp = (p.m + 7) / 8 * 8;
    // one chunk per 4096 elements, at most 64
    p.chunks = static_cast<int>(std::min<long long>(64, (static_cast<long long>(R) * C + 4095) / 4096));
    return p;
}

// Workspace: the sums of squares, the lifts, then the fp16 plane pairs of X (two, in turn), A and Q.
struct Layout {
    size_t lift, x0, x1, a, p, bytes;
};
Layout layout(const dcnv4::OrthoParams& p) {
    Layout l{};
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    const size_t xb = up(static_cast<size_t>(p.B) * p.n * p.mp * 4), ab = up(static_cast<size_t>(p.B) * p.n * p.np * 4);
    l.lift = up(static_cast<size_t>(p.B) * p.chunks * 8);
    l.x0 = l.lift + up(static_cast<size_t>(p.B) * 4);
    l.x1 = l.x0 + xb;
    l.a = l.x1 + xb;
    l.p = l.a + ab;
    l.bytes = l.p + ab;
    return l;
}

// Map of a plane pair [2 * B][rows][cols] with boxes of 64 columns x `box` rows, 128-byte swizzle.
bool plane_map(CUtensorMap* map, void* base, int cols, int pitch, int rows, int planes, int box) {
    auto encode = tensor_map_encoder();
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(planes)};
    const cuuint64_t str[2] = {static_cast<cuuint64_t>(pitch) * 2, static_cast<cuuint64_t>(pitch) * rows * 2};
    const cuuint32_t bx[3] = {64u, static_cast<cuuint32_t>(box), 1u}, es[3] = {1u, 1u, 1u};
    return encode && encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, base, dims, str, bx, es,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Matrices that fit one CTA's shared memory run the whole iteration in one
// kernel, one CTA each. By the sides alone, so that a matrix's bits do not
// depend on the stack it is in. Measured, this kernel against one per product:
// 1 matrix of 8 x 8 14 us against 50, 18 of 64 x 256 60 against 68, 148 of them
// 65 against 116, 148 of 128 x 320 137 against 185; but for a few long matrices
// it loses, 18 of 64 x 320 80 against 70, of 128 x 192 89 against 75, of 128 x
// 320 128 against 81.
bool fits_one_cta(const dcnv4::OrthoParams& p) {
    if (const char* e = std::getenv("DCNV4_ORTHO_FORM"); e && std::strcmp(e, "products") == 0) return false;
    return p.n <= 128 && (p.n + 63) / 64 + (p.m + 63) / 64 <= dcnv4::kOrthoSmallBlocks;
}

template <typename T>
int launch_small(const void* x, void* out, int steps, const dcnv4::OrthoStep* step, const dcnv4::OrthoParams& p, cudaStream_t s) {
    dcnv4::OrthoSmall g{};
    g.steps = steps;
    g.xb = (p.m + 63) / 64;
    g.nb = (p.n + 63) / 64;
    g.n16 = (p.n + 15) / 16 * 16;
    g.m16 = (p.m + 15) / 16 * 16;
    const unsigned cols = static_cast<unsigned>(4 * std::max(g.n16, std::min(128, g.m16)));
    g.tmem_cols = 32;
    while (g.tmem_cols < cols) g.tmem_cols <<= 1;
    std::copy(step, step + steps + 1, g.step);
    const unsigned smem = 1024u + static_cast<unsigned>(g.xb + g.nb) * dcnv4::kOrthoBlock;
    auto kern = dcnv4::ortho_small_kernel<T>;
    constexpr unsigned most = 1024u + dcnv4::kOrthoSmallBlocks * dcnv4::kOrthoBlock;
    static_assert(most <= kTileSmemLimit, "the blocks do not fit");
    if (smem_limit_once(reinterpret_cast<const void*>(kern), static_cast<int>(most)) != cudaSuccess) return DCNV4_ERR_LAUNCH;
    return launch_chained(kern, dim3(static_cast<unsigned>(p.B)), dcnv4::kOrthoSmallThreads, smem, s,
                          static_cast<const T*>(x), static_cast<T*>(out), g, p);
}

template <int MODE, typename T>
int product(const CUtensorMap& l, const CUtensorMap& r, const CUtensorMap& o, T* out, int cols, int k,
            const dcnv4::OrthoStep* step, int nsm, const dcnv4::OrthoParams& p, cudaStream_t s) {
    dcnv4::OrthoTiles g{};
    g.tiles_i = (p.n + 127) / 128;
    g.tiles_j = (cols + 63) / 64;
    g.kblocks = (k + 63) / 64;
    g.now = step[0];
    g.next = step[1];
    const unsigned tiles = static_cast<unsigned>(p.B) * g.tiles_i * g.tiles_j;
    const bool deep = tiles <= static_cast<unsigned>(nsm);
    const bool runs = g.kblocks > dcnv4::kOrthoRun;
    auto kern = deep ? (runs ? dcnv4::ortho_product_kernel<MODE, T, 4, true> : dcnv4::ortho_product_kernel<MODE, T, 4, false>)
                     : (runs ? dcnv4::ortho_product_kernel<MODE, T, 2, true> : dcnv4::ortho_product_kernel<MODE, T, 2, false>);
    const unsigned smem = dcnv4::ortho_smem(deep ? 4 : 2);
    if (smem_limit_once(reinterpret_cast<const void*>(kern), static_cast<int>(smem)) != cudaSuccess) return DCNV4_ERR_LAUNCH;
    return launch_chained(kern, dim3(tiles), dcnv4::kOrthoThreads, smem, s, l, r, o, out, g, p);
}

template <typename T>
int launch(const void* x, void* out, unsigned char* ws, int steps, const dcnv4::OrthoStep* step, dcnv4::OrthoParams p,
           cudaStream_t s) {
    if (steps > 0 && fits_one_cta(p)) return launch_small<T>(x, out, steps, step, p, s);
    const Layout l = layout(p);
    p.lift = reinterpret_cast<int*>(ws + l.lift);
    double* part = reinterpret_cast<double*>(ws);
    __half *x0 = reinterpret_cast<__half*>(ws + l.x0), *x1 = reinterpret_cast<__half*>(ws + l.x1);
    __half *a = reinterpret_cast<__half*>(ws + l.a), *q = reinterpret_cast<__half*>(ws + l.p);
    // maps of 128-row boxes (left operands, results) and of 64-row boxes (right operands)
    CUtensorMap xm[2], xr[2], am, ar, qm;
    const int planes = 2 * p.B;
    for (int i = 0; i < 2; ++i)
        if (!plane_map(&xm[i], i ? x1 : x0, p.m, p.mp, p.n, planes, 128) ||
            !plane_map(&xr[i], i ? x1 : x0, p.m, p.mp, p.n, planes, 64))
            return DCNV4_ERR_CUDA;
    if (!plane_map(&am, a, p.n, p.np, p.n, planes, 128) || !plane_map(&ar, a, p.n, p.np, p.n, planes, 64) ||
        !plane_map(&qm, q, p.n, p.np, p.n, planes, 128))
        return DCNV4_ERR_CUDA;
    T* o = static_cast<T*>(out);
    const int nsm = sm_count();
    if (nsm <= 0) return DCNV4_ERR_CUDA;
    int rc = launch_chained(dcnv4::ortho_sumsq_kernel<T>, dim3(static_cast<unsigned>(p.B) * p.chunks), 256, 0, s,
                            static_cast<const T*>(x), part, p);
    if (rc) return rc;
    const unsigned st = static_cast<unsigned>(p.B) * ((p.R + 63) / 64) * ((p.C + 63) / 64);
    rc = launch_chained(dcnv4::ortho_start_kernel<T>, dim3(st), 256, 0, s, static_cast<const T*>(x),
                        static_cast<const double*>(part), x0, steps == 0 ? o : static_cast<T*>(nullptr), p);
    for (int k = 0, cur = 0; k < steps && !rc; ++k, cur ^= 1) {
        rc = product<dcnv4::kGram, float>(xm[cur], xr[cur], am, static_cast<float*>(nullptr), p.n, p.m, step + k, nsm, p, s);
        if (!rc) rc = product<dcnv4::kPoly, float>(am, ar, qm, static_cast<float*>(nullptr), p.n, p.n, step + k, nsm, p, s);
        if (rc) break;
        if (k + 1 < steps) rc = product<dcnv4::kApply, float>(qm, xr[cur], xm[cur ^ 1], static_cast<float*>(nullptr), p.m, p.n, step + k, nsm, p, s);
        else rc = product<dcnv4::kLast, T>(qm, xr[cur], xm[cur ^ 1], o, p.m, p.n, step + k, nsm, p, s);
    }
    return rc;
}

}  // namespace

extern "C" {

int dcnv4_orthogonalize_workspace(int B, int R, int C, int dtype, size_t* bytes) {
    const int rc = check_stack(B, R, C, dtype);
    if (rc) return rc;
    if (!bytes) return DCNV4_ERR_NULL;
    *bytes = B == 0 ? 0 : layout(make_params(B, R, C)).bytes;
    return DCNV4_OK;
}

int dcnv4_orthogonalize(const void* x, void* out, void* workspace, size_t workspace_size, int B, int R, int C,
                        int steps, float a, float b, float c, float eps, int dtype, void* stream) {
    const int rc = check_stack(B, R, C, dtype);
    if (rc) return rc;
    if (steps < 0 || steps > kMaxSteps) return DCNV4_ERR_SHAPE;
    dcnv4::OrthoStep step[kMaxSteps + 1];
    if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c) || !std::isfinite(eps) || !(eps > 0.f) ||
        !iteration_bounds(a, b, c, steps, step))
        return DCNV4_ERR_COEFFICIENTS;
    if (B == 0) return DCNV4_OK;
    if (!x || !out || !workspace) return DCNV4_ERR_NULL;
    const int e = elem_size(dtype);
    if (!aligned(x, e) || !aligned(out, e) || !aligned(workspace, 256)) return DCNV4_ERR_ALIGN;
    dcnv4::OrthoParams p = make_params(B, R, C);
    p.a = a; p.b = b; p.c = c; p.eps = eps;
    const size_t need = layout(p).bytes;
    if (workspace_size < need) return DCNV4_ERR_WORKSPACE;
    const long long nb = static_cast<long long>(B) * R * C * e;
    if (overlap(out, nb, x, nb) || overlap(workspace, static_cast<long long>(need), x, nb) ||
        overlap(workspace, static_cast<long long>(need), out, nb))
        return DCNV4_ERR_ALIAS;
    p.status = dcnv4_host::device_status_word();
    if (!p.status) return DCNV4_ERR_CUDA;
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (dtype) {
        case DCNV4_F32: return launch<float>(x, out, ws, steps, step, p, s);
        case DCNV4_F16: return launch<__half>(x, out, ws, steps, step, p, s);
        default: return launch<__nv_bfloat16>(x, out, ws, steps, step, p, s);
    }
}

}  // extern "C"
