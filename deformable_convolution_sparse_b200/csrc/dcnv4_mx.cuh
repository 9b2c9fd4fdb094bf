// sm_100a kernels of microscaled 4-bit floating point (the OCP Microscaling
// Formats specification v1.0, MXFP4): quantisation, its inverse, and the
// offset/mask predictor's projection with both operands in the format.
//
// A block of 32 consecutive channels v_i shares one power-of-two scale 2^e,
//   e = max(floor(log2(max_i |v_i|)) - 2, -127)
// (2 is the exponent of the largest element, 6 = 1.5 * 2^2), stored as the
// byte e + 127; element i is v_i / 2^e rounded to the nearest of
// 0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the even code, magnitudes above 6 to 6)
// with its sign, a 4-bit code (e2m1). A block that holds a NaN or an infinity
// has the scale byte 255 and element codes 0: all its values read back as NaN.
// v_i / 2^e is exact in fp32 (a multiplication by a power of two that neither
// overflows nor, where the result could round to anything but 0, underflows),
// so each element is rounded exactly once.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dcnv4_async.cuh"
#include "dcnv4_kernels.cuh"

namespace dcnv4 {

constexpr int kMxBlock = 32;       // channels that share a scale
constexpr int kMxBlockBytes = 16;  // their codes

// Eight fp32 values as e2m1 codes, value 2i in the low half of byte i.
__device__ __forceinline__ uint32_t e2m1_pack8(const float (&q)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
    return r;
}

// Bits of the largest magnitude of 8 values (NaN above infinity above numbers).
__device__ __forceinline__ uint32_t amax_bits8(const float (&v)[8]) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    return m;
}

// Scale byte of a block from the bits of its largest magnitude: the biased
// exponent less 2 (a subnormal's biased exponent reads 0 and gives 2^-127 as
// the clamp does), 255 for infinities and NaN.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
    const uint32_t ex = amax_bits >> 23;
    return ex == 255u ? 255u : (ex > 2u ? ex - 2u : 0u);
}

// 8 values of a block with scale byte s (below 255) as codes: 2^(127 - s) is a
// normal fp32 number, s being at most 252.
__device__ __forceinline__ uint32_t mx_codes8(float (&v)[8], uint32_t s) {
    if (s == 255u) return 0u;
    const float inv = __uint_as_float((254u - s) << 23);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= inv;
    return e2m1_pack8(v);
}

// 2^(s - 127) in fp32 (s = 0: the subnormal 2^-127; s = 255: NaN)
__device__ __forceinline__ float mx_scale_value(uint32_t s) {
    if (s == 255u) return __uint_as_float(0x7fc00000u);
    return __uint_as_float(s != 0u ? s << 23 : 1u << 22);
}

// magnitude of the e2m1 code c (0..7) with its sign bit (8): 0 .5 1 1.5 2 3 4 6
__device__ __forceinline__ float e2m1_value(uint32_t c) {
    const uint32_t ex = (c >> 1) & 3u, m = c & 1u;
    const float v = ex == 0u ? 0.5f * static_cast<float>(m)
                             : __uint_as_float(((ex + 126u) << 23) | (m << 22));
    return (c & 8u) ? -v : v;
}

// Channels c0 .. c0+7 of a row of C channels, zeros past the end. VEC: C is a
// multiple of 8 and the row is 16-byte aligned.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* __restrict__ row, int c0, int C, float (&v)[8]) {
    if constexpr (VEC) {
        if (c0 >= C) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0.f;
            return;
        }
        if constexpr (sizeof(T) == 4) {
            const float4 a = __ldg(reinterpret_cast<const float4*>(row + c0));
            const float4 b = __ldg(reinterpret_cast<const float4*>(row + c0 + 4));
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
            const uint4 a = __ldg(reinterpret_cast<const uint4*>(row + c0));
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = unpack2(w[i], static_cast<T*>(nullptr));
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c0 + i < C ? ElemTraits<T>::to_float(__ldg(row + c0 + i)) : 0.f;
    }
}

template <typename T>
__device__ __forceinline__ T mx_from_float(float v) {
    if constexpr (sizeof(T) == 4) return v;
    else if constexpr (std::is_same<T, __half>::value) return __float2half_rn(v);
    else return __float2bfloat16_rn(v);
}

// Quantisation: four lanes per block, 8 channels each, so that a warp reads 8
// blocks as one contiguous run with 16-byte loads and writes their codes as
// 128 contiguous bytes; the block's largest magnitude takes two shuffles.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256)
mx_quantize_kernel(const T* __restrict__ x, uint32_t* __restrict__ codes, uint8_t* __restrict__ scales,
                   unsigned blocks, FastDiv nb, int C) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int part = threadIdx.x & 3;
    const unsigned stride = gridDim.x * (blockDim.x / 4);
    // every lane of a warp makes the same number of rounds (the shuffles need all of them)
    for (unsigned b0 = blockIdx.x * (blockDim.x / 4) + ((threadIdx.x & ~31u) >> 2); b0 < blocks; b0 += stride) {
        const unsigned b = b0 + ((threadIdx.x & 31u) >> 2);
        const bool on = b < blocks;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (on) {
            const unsigned row = fdiv(b, nb);
            load8<T, VEC>(x + static_cast<size_t>(row) * C, static_cast<int>(b - row * nb.d) * kMxBlock + part * 8, C, v);
        }
        uint32_t m = amax_bits8(v);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const uint32_t s = mx_scale_byte(m);
        if (on) {
            codes[static_cast<size_t>(b) * 4 + part] = mx_codes8(v, s);
            if (part == 0) scales[b] = static_cast<uint8_t>(s);
        }
    }
}

// The inverse: four lanes per block, 8 channels each; value = element * 2^e,
// rounded once to T (exact in fp32 and, subnormals apart, in bf16).
template <typename T, bool VEC>
__global__ void __launch_bounds__(256)
mx_dequantize_kernel(const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales, T* __restrict__ x,
                     unsigned blocks, FastDiv nb, int C) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int part = threadIdx.x & 3;
    const unsigned stride = gridDim.x * (blockDim.x / 4);
    for (unsigned b = blockIdx.x * (blockDim.x / 4) + (threadIdx.x >> 2); b < blocks; b += stride) {
        const unsigned row = fdiv(b, nb);
        const int c0 = static_cast<int>(b - row * nb.d) * kMxBlock + part * 8;
        if (c0 >= C) continue;
        const uint32_t w = __ldg(codes + static_cast<size_t>(b) * 4 + part);
        const float sc = mx_scale_value(__ldg(scales + b));
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = e2m1_value((w >> (4 * i)) & 15u) * sc;
        T* o = x + static_cast<size_t>(row) * C + c0;
        if constexpr (VEC) {
            if constexpr (sizeof(T) == 4) {
                reinterpret_cast<float4*>(o)[0] = make_float4(v[0], v[1], v[2], v[3]);
                reinterpret_cast<float4*>(o)[1] = make_float4(v[4], v[5], v[6], v[7]);
            } else {
                T* t = nullptr;
                *reinterpret_cast<uint4*>(o) =
                    make_uint4(pack2(v[0], v[1], t), pack2(v[2], v[3], t), pack2(v[4], v[5], t), pack2(v[6], v[7], t));
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c0 + i < C) o[i] = mx_from_float<T>(v[i]);
        }
    }
}

// Slot of projection channel o in its record (offsets (g, comp, j) -> g*3P +
// comp*P + j, masks (g, j) -> g*3P + 2P + j) and the channel of a slot.
__host__ __device__ __forceinline__ int record_slot(int o, int G, int P) {
    if (o < 2 * G * P) return (o / (2 * P)) * 3 * P + o % (2 * P);
    const int q = o - 2 * G * P;
    return (q / P) * 3 * P + 2 * P + q % P;
}
__host__ __device__ __forceinline__ int slot_channel(int s, int G, int P) {
    const int g = s / (3 * P), r = s - g * 3 * P;
    return r < 2 * P ? g * 2 * P + r : 2 * G * P + g * P + (r - 2 * P);
}

struct MxProjParams {
    int M, C, G, P, NO;
    int nb;             // blocks per row
    unsigned* status;
};

// The projection on the CUDA cores: a tile of 32 pixels x 64 record slots per
// CTA; per block of 32 channels the pixels are quantised and the weights read
// into shared memory as fp32 values (exact), then multiplied and summed in fp32.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256)
predictor_mx_plain_kernel(const T* __restrict__ y, const uint32_t* __restrict__ wcodes,
                          const uint8_t* __restrict__ wscales, const float* __restrict__ bias, T* __restrict__ rec,
                          MxProjParams p) {
    __shared__ float ys[32][33];
    __shared__ float wsm[64][33];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x;
    const long long m0 = static_cast<long long>(blockIdx.x) * 32;
    const int s0 = blockIdx.y * 64;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const int px = tid >> 3, sl = tid & 7;  // this thread's pixel and its slots sl, sl + 8, ...
    for (int b = 0; b < p.nb; ++b) {
        if (tid < 128) {
            const int r = tid >> 2, part = tid & 3;
            float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (m0 + r < p.M)
                load8<T, VEC>(y + static_cast<size_t>(m0 + r) * p.C, b * kMxBlock + part * 8, p.C, v);
            uint32_t m = amax_bits8(v);
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const uint32_t s = mx_scale_byte(m);
            const uint32_t c = mx_codes8(v, s);
            const float sc = mx_scale_value(s);
#pragma unroll
            for (int i = 0; i < 8; ++i) ys[r][part * 8 + i] = e2m1_value((c >> (4 * i)) & 15u) * sc;
        }
        {
            const int r = tid >> 2, part = tid & 3;
            const int s = s0 + r;
            if (s < p.NO) {
                const size_t wb = static_cast<size_t>(slot_channel(s, p.G, p.P)) * p.nb + b;
                const uint32_t c = __ldg(wcodes + wb * 4 + part);
                const float sc = mx_scale_value(__ldg(wscales + wb));
#pragma unroll
                for (int i = 0; i < 8; ++i) wsm[r][part * 8 + i] = e2m1_value((c >> (4 * i)) & 15u) * sc;
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) wsm[r][part * 8 + i] = 0.f;
            }
        }
        __syncthreads();
#pragma unroll 8
        for (int k = 0; k < kMxBlock; ++k) {
            const float a = ys[px][k];
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] = fmaf(a, wsm[sl + 8 * j][k], acc[j]);
        }
        __syncthreads();
    }
    if (m0 + px < p.M) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int s = s0 + sl + 8 * j;
            if (s < p.NO)
                rec[static_cast<size_t>(m0 + px) * p.NO + s] =
                    mx_from_float<T>(acc[j] + (bias ? __ldg(bias + slot_channel(s, p.G, p.P)) : 0.f));
        }
    }
}

}  // namespace dcnv4
