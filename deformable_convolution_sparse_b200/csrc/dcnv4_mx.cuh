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
#include "dcnv4_tcgen05.cuh"

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
    int nb;             // blocks of 32 channels per row
    FastDiv nbd;        // division by nb
    // tensor-core kernel
    int mtiles;         // tiles of 128 pixels
    int walkers;        // CTAs that share the pixel tiles of one slot tile
    int NT;             // record slots per CTA (a multiple of 16)
    int k64, kc;        // steps of 64 channels (one instruction), groups of 128 (one column of scales)
    int groups;         // ceil(NT / 128)
    int pitch;          // bytes between the rows of the output staging tile
    int store;          // kMxStore*
    unsigned tmem_cols, sfa_col, sfb_col;
    unsigned smem_sfa, smem_b, smem_sfb, smem_bias, smem_stage, smem_bars;
    unsigned* status;
};

// How a tile of records leaves the staging tile: as one bulk copy (rows are
// whole records, back to back), as one bulk copy per row (16-byte multiples),
// or element by element.
constexpr int kMxStoreTile = 0, kMxStoreRows = 1, kMxStoreElems = 2;

namespace tc {
// kind::mxf4, both operands e2m1 K-major, one ue8m0 scale per 32 k, M = 128:
// B scale selector in bits 4..5, A's in 29..30 (first byte of the 16-bit pair
// of scales that a 64-k step uses: 0 or 2), e2m1 = 1 in bits 7..9 and 10..12,
// N / 8 in 17..22, ue8m0 in bit 23, M / 128 in 27..28
__host__ __device__ constexpr uint32_t idesc_mxf4(int n, uint32_t sf) {
    return (sf << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) | (1u << 27) |
           (sf << 29);
}
__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate ? 1u : 0u)
        : "memory");
}
// 32 rows of 16 bytes (row r at r * 16) into 4 tensor-memory columns, the same
// in each of the four 32-lane quarters; in order with the products issued by
// the same thread
__device__ __forceinline__ void copy_scales(uint32_t taddr, unsigned saddr) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(smem_desc(saddr, 16u, 128u, 0u))
                 : "memory");
}
}  // namespace tc

// Eight channels of one block as loaded: 16 bytes of 16-bit values, 32 of fp32.
template <typename T>
struct MxRaw {
    uint4 w[sizeof(T) == 4 ? 2 : 1];
};
template <typename T>
__device__ __forceinline__ void mx_unpack(const MxRaw<T>& r, float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
        const uint32_t w[8] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
    } else {
        const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2(w[i], static_cast<T*>(nullptr));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}

// The projection on the tensor cores. A CTA of 8 warps owns NT record slots
// and walks tiles of 128 pixels: the tile is read as it lies in
// memory (four lanes per block of 32 channels), quantised in registers and
// written to shared memory as tcgen05 operand (a block is one 16-byte row of
// an unswizzled 8 x 16-byte core matrix) with its scale bytes beside it; one
// thread moves the scales to tensor memory and issues the products (64
// channels each); then all warps read the accumulators, add the bias, round,
// and stage the records for bulk copies. The first loads of the next tile are
// issued before the wait for the products. Several CTAs share an SM (tensor
// memory: 128 or 256 columns each), so that one's loads overlap another's
// epilogue.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256, 4)
predictor_mx_kernel(const T* __restrict__ y, const uint4* __restrict__ wcodes, const uint8_t* __restrict__ wscales,
                    const float* __restrict__ bias, T* __restrict__ rec, MxProjParams p) {
    extern __shared__ unsigned char mx_smem_raw[];
    unsigned char* sm = mx_smem_raw + ((128u - (smem_addr(mx_smem_raw) & 127u)) & 127u);
    unsigned char* sfa = sm + p.smem_sfa;
    unsigned char* bsm = sm + p.smem_b;
    unsigned char* sfb = sm + p.smem_sfb;
    float* bias_s = reinterpret_cast<float*>(sm + p.smem_bias);
    unsigned char* stage = sm + p.smem_stage;
    uint64_t* done = reinterpret_cast<uint64_t*>(sm + p.smem_bars);
    uint32_t* slot = reinterpret_cast<uint32_t*>(done + 1);
    constexpr int E = sizeof(T);
    constexpr int kBatch = E == 4 ? 2 : 4;  // eight-channel pieces loaded ahead
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = static_cast<int>(blockIdx.x) % p.walkers, walkers = p.walkers;
    const int s0 = static_cast<int>(blockIdx.x) / p.walkers * p.NT, width = min(p.NT, p.NO - s0), np = (width + 15) / 16 * 16;

    if (tid == 0) {
        mbar_init(done, 1);
        fence_barrier_init();
    }
    if (warp == 0) tc::alloc(slot, p.tmem_cols);
    tc::fence_before();
    __syncthreads();  // every CTA holds its tensor memory before the next launch may start
    tc::fence_after();
    const uint32_t tmem = *slot;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int pieces = 2 * p.nb;  // per thread and tile
    MxRaw<T> ahead[kBatch];
    // piece i of this thread in a tile: block (i * 256 + tid) / 4 of the tile's 128 * nb, eighth tid % 4
    auto fetch = [&](int tile, int i, MxRaw<T>& r) {
        const unsigned b = static_cast<unsigned>(i * 64 + (tid >> 2));
        const unsigned row = fdiv(b, p.nbd);
        const int c0 = static_cast<int>(b - row * p.nb) * kMxBlock + (tid & 3) * 8;
        const long long m = static_cast<long long>(tile) * 128 + row;
        const T* src = y + m * p.C + c0;
        if constexpr (VEC) {
            const bool on = m < p.M && c0 < p.C;
#pragma unroll
            for (int q = 0; q < (E == 4 ? 2 : 1); ++q)
                r.w[q] = on ? __ldg(reinterpret_cast<const uint4*>(src) + q) : make_uint4(0, 0, 0, 0);
        } else {
            T* d = reinterpret_cast<T*>(&r);
#pragma unroll
            for (int q = 0; q < 8; ++q) d[q] = m < p.M && c0 + q < p.C ? __ldg(src + q) : mx_from_float<T>(0.f);
        }
    };
    auto fetch_batch = [&](int tile, int i0) {
#pragma unroll
        for (int q = 0; q < kBatch; ++q)
            if (i0 + q < pieces) fetch(tile, i0 + q, ahead[q]);
    };
    int tile = cta;
    if (tile < p.mtiles) fetch_batch(tile, 0);

    // the weight's rows in record order, its scales, the bias; padding is zero
    for (int i = tid; i < 2 * p.k64 * p.NT; i += 256) {
        const int j = i / p.NT, s = i - j * p.NT;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (s < width && j < p.nb)
            v = __ldg(wcodes + static_cast<size_t>(slot_channel(s0 + s, p.G, p.P)) * p.nb + j);
        *reinterpret_cast<uint4*>(bsm + static_cast<size_t>(j) * p.NT * 16 + s * 16) = v;
    }
    for (int i = tid; i < p.kc * p.groups * 128; i += 256) {
        const int s = i % (p.groups * 128), k = i / (p.groups * 128);
        uint32_t v = 0u;
        if (s < width)
            for (int q = 0; q < 4; ++q)
                if (k * 4 + q < p.nb)
                    v |= static_cast<uint32_t>(__ldg(wscales + static_cast<size_t>(slot_channel(s0 + s, p.G, p.P)) * p.nb +
                                                     k * 4 + q)) << (8 * q);
        *reinterpret_cast<uint32_t*>(sfb + (k * p.groups + (s >> 7)) * 512 + (s & 31) * 16 + ((s >> 5) & 3) * 4) = v;
    }
    for (int i = tid; i < p.kc * 128; i += 256) reinterpret_cast<uint32_t*>(sfa)[i] = 0u;
    if (p.nb & 1)
        for (int i = tid; i < 128; i += 256)
            *reinterpret_cast<uint4*>(sm + static_cast<size_t>(p.nb) * 2048 + i * 16) = make_uint4(0, 0, 0, 0);
    for (int i = tid; i < p.NT; i += 256) bias_s[i] = bias && i < width ? __ldg(bias + slot_channel(s0 + i, p.G, p.P)) : 0.f;
    __syncthreads();

    bool ok = true;
    for (int it = 0; tile < p.mtiles; tile += walkers, ++it) {
        for (int i0 = 0; i0 < pieces; i0 += kBatch) {
            if (i0 > 0) fetch_batch(tile, i0);
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                if (i0 + q >= pieces) break;
                float v[8];
                mx_unpack<T>(ahead[q], v);
                uint32_t m = amax_bits8(v);
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
                const uint32_t s = mx_scale_byte(m);
                const unsigned b = static_cast<unsigned>((i0 + q) * 64 + (tid >> 2));
                const unsigned row = fdiv(b, p.nbd), j = b - row * p.nb;
                *reinterpret_cast<uint32_t*>(sm + j * 2048u + row * 16u + (tid & 3) * 4u) = mx_codes8(v, s);
                if ((tid & 3) == 0)
                    sfa[(j >> 2) * 512u + (row & 31u) * 16u + (row >> 5) * 4u + (j & 3u)] = static_cast<unsigned char>(s);
            }
        }
        fence_proxy_async();
        // the bulk copies that read the staging tile have done so
        if (warp == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        tc::fence_before();
        __syncthreads();
        if (tid == 0) {
            tc::fence_after();
            if (it == 0)
                for (int i = 0; i < p.kc * p.groups; ++i) tc::copy_scales(tmem + p.sfb_col + i * 4, smem_addr(sfb + i * 512));
            for (int i = 0; i < p.kc; ++i) tc::copy_scales(tmem + p.sfa_col + i * 4, smem_addr(sfa + i * 512));
            for (int k = 0; k < p.k64; ++k)
                tc::mma_mxf4(tmem, tc::smem_desc(smem_addr(sm) + k * 4096u, 2048u, 128u, 0u),
                             tc::smem_desc(smem_addr(bsm) + k * 32u * p.NT, 16u * p.NT, 128u, 0u),
                             tc::idesc_mxf4(np, (k & 1) * 2u), tmem + p.sfa_col + (k >> 1) * 4,
                             tmem + p.sfb_col + (k >> 1) * 4 * p.groups, k > 0);
            tc::commit(done);
        }
        if (tile + walkers < p.mtiles) fetch_batch(tile + walkers, 0);
        ok = __syncthreads_and(mbar_wait_bounded(done, static_cast<unsigned>(it) & 1u, kCopyWaitLimitNs)) != 0;
        if (!ok) break;
        tc::fence_after();

        // accumulator row = pixel: lane 32 * (warp % 4) + lane; 16-column chunks shared by two warps
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        unsigned char* orow = stage + static_cast<size_t>(row) * p.pitch;
        for (int c0 = (warp >> 2) * 16; c0 < np; c0 += 32) {
            float v[16];
            tc::ld16(lanes + c0, v);
            tc::wait_ld();
#pragma unroll
            for (int q = 0; q < 16; q += 4) {
                const float4 b4 = *reinterpret_cast<const float4*>(bias_s + c0 + q);
                v[q] += b4.x; v[q + 1] += b4.y; v[q + 2] += b4.z; v[q + 3] += b4.w;
            }
            if (p.store != kMxStoreElems && c0 + 16 <= width) {
                // rows start on 8-byte boundaries at least, on 16-byte ones unless they are packed
                uint32_t w[16 * E / 4];
                if constexpr (E == 4) {
#pragma unroll
                    for (int q = 0; q < 16; ++q) w[q] = __float_as_uint(v[q]);
                } else {
#pragma unroll
                    for (int q = 0; q < 8; ++q) w[q] = pack2(v[2 * q], v[2 * q + 1], static_cast<T*>(nullptr));
                }
                if (p.pitch & 15) {
#pragma unroll
                    for (int q = 0; q < 4 * E; q += 2)
                        *reinterpret_cast<uint2*>(orow + c0 * E + q * 4) = make_uint2(w[q], w[q + 1]);
                } else {
#pragma unroll
                    for (int q = 0; q < 4 * E; q += 4)
                        *reinterpret_cast<uint4*>(orow + c0 * E + q * 4) = make_uint4(w[q], w[q + 1], w[q + 2], w[q + 3]);
                }
            } else {
#pragma unroll
                for (int q = 0; q < 16; ++q)
                    if (c0 + q < width) reinterpret_cast<T*>(orow)[c0 + q] = mx_from_float<T>(v[q]);
            }
        }
        fence_proxy_async();
        tc::fence_before();
        __syncthreads();
        const int rows = static_cast<int>(min(128LL, p.M - static_cast<long long>(tile) * 128));
        T* dst = rec + static_cast<size_t>(tile) * 128 * p.NO + s0;
        const unsigned row_bytes = static_cast<unsigned>(width) * E;
        if (p.store == kMxStoreTile && (rows * row_bytes) % 16u == 0u) {
            if (tid == 0)
                asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
                             "r"(smem_addr(stage)), "r"(rows * row_bytes)
                             : "memory");
        } else if (p.store == kMxStoreRows) {
            if (warp == 0)
                for (int r = lane; r < rows; r += 32)
                    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                                     dst + static_cast<size_t>(r) * p.NO),
                                 "r"(smem_addr(stage + static_cast<size_t>(r) * p.pitch)), "r"(row_bytes)
                                 : "memory");
        } else {
            for (int r = warp; r < rows; r += 8)
                for (int c = lane; c < width; c += 32)
                    dst[static_cast<size_t>(r) * p.NO + c] =
                        reinterpret_cast<const T*>(stage + static_cast<size_t>(r) * p.pitch)[c];
        }
        if (warp == 0) tc::bulk_commit();
    }
    if (!ok && tid == 0) atomicOr(p.status, kStatusCopyTimeout);
    if (warp == 0) tc::bulk_wait_all();
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 0) tc::dealloc(tmem, p.tmem_cols);
}

// The projection on the CUDA cores, for rows too long for the kernel above to
// hold (about 2,900 channels): a tile of 32 pixels x 64 record slots per
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
