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

constexpr int kMaxSteps = 64;

int check_stack(int B, int R, int C, int dtype) {
    if (B < 0 || R <= 0 || C <= 0) return DCNV4_ERR_SHAPE;
    if (!elem_size(dtype)) return DCNV4_ERR_DTYPE;
    // |sizes| < 2^31 each, so the first product fits 62 bits
    const long long rc = static_cast<long long>(R) * C;
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

// The iteration stays bounded: singular values start in [0, 1]; no step may
// lift one above 4, nor the factor a + b s^2 + c s^4 above 64.
bool coefficients_bounded(double a, double b, double c, int steps) {
    double r = 1.0;
    for (int k = 0; k < steps; ++k) {
        if (std::fabs(a) + std::fabs(b) * r * r + std::fabs(c) * r * r * r * r > 4096.0) return false;
        double q = std::max(std::fabs(a), std::fabs(a + b * r * r + c * r * r * r * r));
        if (c != 0.0 && -b / (2.0 * c) > 0.0 && -b / (2.0 * c) < r * r) q = std::max(q, std::fabs(a - b * b / (4.0 * c)));
        if (!(q <= 64.0)) return false;
        r = poly_bound(a, b, c, r);
        if (!(r <= 4.0)) return false;
    }
    return true;
}

dcnv4::OrthoParams make_params(int B, int R, int C) {
    dcnv4::OrthoParams p{};
    p.B = B; p.R = R; p.C = C;
    p.n = std::min(R, C); p.m = std::max(R, C); p.transposed = R > C ? 1 : 0;
    // one chunk per 4096 elements, at most 64
    p.chunks = static_cast<int>(std::min<long long>(64, (static_cast<long long>(R) * C + 4095) / 4096));
    return p;
}

struct Layout {
    size_t part, x0, x1, g, q, bytes;
};
Layout layout(const dcnv4::OrthoParams& p) {
    Layout l{};
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    const size_t xb = up(static_cast<size_t>(p.B) * p.n * p.m * 4), gb = up(static_cast<size_t>(p.B) * p.n * p.n * 4);
    l.part = 0;
    l.x0 = up(static_cast<size_t>(p.B) * p.chunks * 8);
    l.x1 = l.x0 + xb;
    l.g = l.x1 + xb;
    l.q = l.g + gb;
    l.bytes = l.q + gb;
    return l;
}

template <typename T>
int launch(const void* x, void* out, unsigned char* ws, int steps, const dcnv4::OrthoParams& p, cudaStream_t s) {
    const Layout l = layout(p);
    double* part = reinterpret_cast<double*>(ws + l.part);
    float *x0 = reinterpret_cast<float*>(ws + l.x0), *x1 = reinterpret_cast<float*>(ws + l.x1);
    float *g = reinterpret_cast<float*>(ws + l.g), *q = reinterpret_cast<float*>(ws + l.q);
    constexpr int t = dcnv4::kSimtTile;
    const unsigned nt = static_cast<unsigned>((p.n + t - 1) / t), mt = static_cast<unsigned>((p.m + t - 1) / t);
    const unsigned z = static_cast<unsigned>(std::min(p.B, 65535));
    const unsigned flat = static_cast<unsigned>(p.B) * static_cast<unsigned>(p.chunks);
    int rc = launch_chained(dcnv4::ortho_sumsq_kernel<T>, dim3(flat), 256, 0, s, static_cast<const T*>(x), part, p);
    if (rc) return rc;
    rc = launch_chained(dcnv4::ortho_start_kernel<T>, dim3(flat), 256, 0, s, static_cast<const T*>(x),
                        static_cast<const double*>(part), x0, p);
    for (int k = 0; k < steps && !rc; ++k) {
        rc = launch_chained(dcnv4::ortho_gram_kernel, dim3(nt, nt, z), 256, 0, s, static_cast<const float*>(x0), g, p);
        if (!rc) rc = launch_chained(dcnv4::ortho_poly_kernel, dim3(nt, nt, z), 256, 0, s, static_cast<const float*>(g), q, p);
        if (!rc)
            rc = launch_chained(dcnv4::ortho_apply_kernel, dim3(nt, mt, z), 256, 0, s, static_cast<const float*>(q),
                                static_cast<const float*>(x0), x1, p);
        std::swap(x0, x1);
    }
    if (rc) return rc;
    return launch_chained(dcnv4::ortho_finish_kernel<T>, dim3(flat), 256, 0, s, static_cast<const float*>(x0),
                          static_cast<T*>(out), p);
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
    if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c) || !std::isfinite(eps) || !(eps > 0.f) ||
        !coefficients_bounded(a, b, c, steps))
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
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (dtype) {
        case DCNV4_F32: return launch<float>(x, out, ws, steps, p, s);
        case DCNV4_F16: return launch<__half>(x, out, ws, steps, p, s);
        default: return launch<__nv_bfloat16>(x, out, ws, steps, p, s);
    }
}

}  // extern "C"
