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
#include "dcnv4_records.cuh"
#include "dcnv4_tcgen05.cuh"

namespace dcnv4 {

constexpr int kMxBlock = 32;  // channels that share a scale (16 bytes of codes)

// Eight fp32 values as e2m1 codes, value 2i in the low half of byte i.
__device__ __forceinline__ uint32_t e2m1_pack8(const float* q) {
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

// Scale byte of a block from the bits of its largest magnitude: the biased
// exponent less 2 (a subnormal's biased exponent reads 0 and gives 2^-127 as
// the clamp does), 255 for infinities and NaN.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
    const uint32_t ex = amax_bits >> 23;
    return ex == 255u ? 255u : (ex > 2u ? ex - 2u : 0u);
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

// Eight e2m1 codes as fp32 values (exact by way of fp16).
__device__ __forceinline__ void e2m1_unpack8(uint32_t codes, float (&v)[8]) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float2 f = unpack2(h[q], static_cast<__half*>(nullptr));
        v[2 * q] = f.x;
        v[2 * q + 1] = f.y;
    }
}

// Sixteen channels (half a block) as they lie in memory: 32 bytes of 16-bit
// values, 64 of fp32.
template <typename T>
struct MxRaw {
    static constexpr int kVecs = sizeof(T);
    uint4 w[kVecs];
};

// Channels c0 .. c0+15 of a row of C channels, zeros past the end. VEC: C is a
// multiple of 8 and the row is 16-byte aligned.
template <typename T, bool VEC>
__device__ __forceinline__ void mx_load(const T* __restrict__ row, int c0, int C, MxRaw<T>& r) {
    constexpr int per = 16 / sizeof(T);
    if constexpr (VEC) {
#pragma unroll
        for (int q = 0; q < MxRaw<T>::kVecs; ++q)
            r.w[q] = c0 + q * per < C ? __ldg(reinterpret_cast<const uint4*>(row + c0) + q) : make_uint4(0, 0, 0, 0);
    } else {
        uint32_t w[4 * MxRaw<T>::kVecs];
#pragma unroll
        for (int q = 0; q < 16; q += 4 / sizeof(T)) {
            uint32_t v = 0u;
#pragma unroll
            for (int k = 0; k < 4 / static_cast<int>(sizeof(T)); ++k)
                if (c0 + q + k < C) {
                    if constexpr (sizeof(T) == 4) v = __float_as_uint(__ldg(row + c0 + q));
                    else v |= static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(row) + c0 + q + k)) << (16 * k);
                }
            w[q * sizeof(T) / 4] = v;
        }
#pragma unroll
        for (int q = 0; q < MxRaw<T>::kVecs; ++q) r.w[q] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    }
}

// Quantises a block whose halves two neighbouring lanes hold: its scale byte,
// and the codes of this lane's half. Bit patterns without their sign order as
// the magnitudes do (NaN above infinity above numbers), so the largest one
// takes integer maxima, two 16-bit values at a time. KEEP_ZERO: the codes of a
// block of NaN (scale byte 255) are 0 (else they are arbitrary).
template <bool KEEP_ZERO, typename T>
__device__ __forceinline__ uint32_t mx_half_block(const MxRaw<T>& r, uint2& codes) {
    constexpr int NW = 4 * MxRaw<T>::kVecs;
    const uint32_t* w = reinterpret_cast<const uint32_t*>(r.w);
    uint32_t bits;
    if constexpr (sizeof(T) == 4) {
        uint32_t m = 0u;
#pragma unroll
        for (int q = 0; q < NW; ++q) m = max(m, w[q] & 0x7fffffffu);
        bits = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    } else {
        uint32_t m = 0u;
#pragma unroll
        for (int q = 0; q < NW; ++q) m = __vmaxu2(m, w[q] & 0x7fff7fffu);
        m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m & 0xffffu, m >> 16);
        if constexpr (std::is_same<T, __half>::value) bits = __float_as_uint(__half2float(__ushort_as_half(static_cast<uint16_t>(m))));
        else bits = m << 16;
    }
    const uint32_t s = mx_scale_byte(bits);
    // 2^(127 - s) is a normal fp32 number, s being at most 252 or 255
    const float inv = __uint_as_float((254u - s) << 23);
    float v[16];
#pragma unroll
    for (int q = 0; q < NW; ++q) {
        if constexpr (sizeof(T) == 4) {
            v[q] = __uint_as_float(w[q]) * inv;
        } else {
            const float2 f = unpack2(w[q], static_cast<T*>(nullptr));
            v[2 * q] = f.x * inv;
            v[2 * q + 1] = f.y * inv;
        }
    }
    codes = make_uint2(e2m1_pack8(v), e2m1_pack8(v + 8));
    if (KEEP_ZERO && s == 255u) codes = make_uint2(0u, 0u);
    return s;
}

template <typename T>
__device__ __forceinline__ T mx_from_float(float v) {
    if constexpr (sizeof(T) == 4) return v;
    else if constexpr (std::is_same<T, __half>::value) return __float2half_rn(v);
    else return __float2bfloat16_rn(v);
}

// Quantisation: two lanes per block, so that a warp reads 16 blocks as one
// contiguous run with 16-byte loads and writes their codes as 256 contiguous
// bytes. Memory-bound: 200,704 x 64 bf16 values (32.5 MB) in 6.3 us, fp32 (58
// MB) in 10.0, in loops over more than the L2 holds; several blocks' loads per
// lane ahead of the arithmetic measured 6.8 and 10.4.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256)
mx_quantize_kernel(const T* __restrict__ x, uint2* __restrict__ codes, uint8_t* __restrict__ scales,
                   unsigned blocks, FastDiv nb, int C) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int half = threadIdx.x & 1;
    const unsigned stride = gridDim.x * (blockDim.x / 2);
    // every lane of a warp makes the same number of rounds (the shuffles need all of them)
    for (unsigned b0 = blockIdx.x * (blockDim.x / 2) + ((threadIdx.x & ~31u) >> 1); b0 < blocks; b0 += stride) {
        const unsigned b = b0 + ((threadIdx.x & 31u) >> 1);
        const unsigned row = fdiv(min(b, blocks - 1u), nb);
        MxRaw<T> r;
        // past the last block: the last one again, not written
        mx_load<T, VEC>(x + static_cast<size_t>(row) * C, static_cast<int>(min(b, blocks - 1u) - row * nb.d) * kMxBlock + half * 16, C, r);
        uint2 c;
        const uint32_t s = mx_half_block<true>(r, c);
        if (b < blocks) {
            codes[static_cast<size_t>(b) * 2 + half] = c;
            if (half == 0) scales[b] = static_cast<uint8_t>(s);
        }
    }
}

// The inverse: a lane writes 16 bytes, four lanes per block of 16-bit values and
// eight of fp32; value = element * 2^e, rounded once to T (exact in fp32 and,
// subnormals apart, in bf16). The sizes above come back in 7.8 (bf16) and 13.3
// us (fp32: 4.4 TB/s, mostly writes); elements taken apart by arithmetic instead
// of conversions made bf16 11.2.
template <typename T>
constexpr int mx_lanes() {
    return 2 * sizeof(T);
}
template <typename T, bool VEC>
__global__ void __launch_bounds__(256)
mx_dequantize_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, T* __restrict__ x,
                     unsigned blocks, FastDiv nb, int C) {
    constexpr int L = mx_lanes<T>(), N = kMxBlock / L;  // lanes per block, channels per lane
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int part = threadIdx.x % L;
    const unsigned stride = gridDim.x * (blockDim.x / L);
    for (unsigned b = blockIdx.x * (blockDim.x / L) + threadIdx.x / L; b < blocks; b += stride) {
        const unsigned row = fdiv(b, nb);
        const int c0 = static_cast<int>(b - row * nb.d) * kMxBlock + part * N;
        if (c0 >= C) continue;
        // fp32: two lanes share a word
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(codes) + static_cast<size_t>(b) * 4 + part / (8 / N));
        const float sc = mx_scale_value(__ldg(scales + b));
        float v[8];
        e2m1_unpack8(w, v);
        if (N == 4 && (part & 1))
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = v[i + 4];
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] *= sc;
        T* o = x + static_cast<size_t>(row) * C + c0;
        if constexpr (VEC) {
            if constexpr (sizeof(T) == 4) {
                *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
            } else {
                T* t = nullptr;
                *reinterpret_cast<uint4*>(o) =
                    make_uint4(pack2(v[0], v[1], t), pack2(v[2], v[3], t), pack2(v[4], v[5], t), pack2(v[6], v[7], t));
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (c0 + i < C) o[i] = mx_from_float<T>(v[i]);
        }
    }
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
    int pitch;          // bytes between the rows of the staging tile (kMxStoreTma: of a block, 128 or 64)
    int store;          // kMxStore*
    unsigned tmem_cols, sfa_col, sfb_col;
    unsigned smem_a, smem_sfa, smem_b, smem_sfb, smem_bias, smem_stage, smem_ring, smem_bars;
    unsigned* status;
};

// How a tile of records leaves the staging tile: as one bulk copy (rows are
// whole records, back to back as in memory), by TMA (blocks of 128 or 64 bytes
// of columns x 128 rows, swizzled), or element by element.
constexpr int kMxStoreTile = 0, kMxStoreTma = 1, kMxStoreElems = 2;

namespace tc {
// kind::mxf4, both operands e2m1 K-major, one ue8m0 scale per 32 k, M = 128:
// B scale selector in bits 4..5, A's in 29..30 (first byte of the 16-bit pair
// of scales that a 64-k step uses: 0 or 2), e2m1 = 1 in bits 7..9 and 10..12,
// N / 8 in 17..22, ue8m0 in bit 23, M / 128 in 27..28
__host__ __device__ constexpr uint32_t idesc_mxf4(int n, uint32_t sf) {
    return (sf << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) | (1u << 27) |
           (sf << 29);
}
// (called by a whole warp, as mma_f16)
__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         bool accumulate, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "setp.ne.b32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate ? 1u : 0u), "r"(lead)
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

// The projection on the tensor cores. A CTA owns NT record slots and walks
// tiles of 128 pixels: the tile is read as it lies in memory (two lanes per
// block of 32 channels) through a ring of kAhead pieces per thread that runs
// ahead across tiles with asynchronous copies, quantised in registers and
// written to shared memory as tcgen05 operand (a block is one 16-byte row of
// an unswizzled 8 x 16-byte core matrix) with its scale bytes beside it; one
// thread moves the scales to tensor memory and issues the products (64
// channels each); then all warps read the accumulators, add the bias, round,
// and stage the records for bulk copies. Two CTAs of 512 threads share an SM,
// or four of 256 where 128 columns of tensor memory and a quarter of the
// shared memory do, so that one's loads overlap another's epilogue.
//
// Memory bounds the formula (pixels in, records out); what bounds the kernel is
// the chain of phases per tile (quantise, products, epilogue: some 8,000 cycles
// with four CTAs to an SM, whose schedulers issue 57 % of the time) and 3,000
// cycles of set-up per CTA. Measured on B200: 200,704 pixels x 64 fp16 channels
// to 108 slots 20.7 us (69 MB: 3.3 TB/s), 129,032 x 128 bf16 to 216 slots 28.2
// us (3.1 TB/s), 26,047 x 320 fp32 to 192 slots 24 us, 196 x 256 to 432 6.4 us.
template <typename T, int THREADS>
struct MxShape {
    static constexpr int kPiece = 16 * sizeof(T);  // sixteen channels
    static constexpr int kAhead = 2;
    static constexpr unsigned kRing = kAhead * THREADS * kPiece;
};

template <typename T, bool VEC, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
predictor_mx_kernel(const __grid_constant__ CUtensorMap rmap, const T* __restrict__ y, const uint4* __restrict__ wcodes,
                    const uint8_t* __restrict__ wscales, const float* __restrict__ bias, T* __restrict__ rec,
                    MxProjParams p) {
    using S = MxShape<T, THREADS>;
    extern __shared__ unsigned char mx_smem_raw[];
    unsigned char* sm = mx_smem_raw + ((1024u - (smem_addr(mx_smem_raw) & 1023u)) & 1023u);
    unsigned char* asm_ = sm + p.smem_a;
    unsigned char* sfa = sm + p.smem_sfa;
    unsigned char* bsm = sm + p.smem_b;
    unsigned char* sfb = sm + p.smem_sfb;
    float* bias_s = reinterpret_cast<float*>(sm + p.smem_bias);
    int* channel = reinterpret_cast<int*>(bias_s + p.NT);  // projection channel of each slot
    unsigned char* stage = sm + p.smem_stage;
    unsigned char* ring = sm + p.smem_ring;
    uint64_t* done = reinterpret_cast<uint64_t*>(sm + p.smem_bars);
    uint32_t* slot = reinterpret_cast<uint32_t*>(done + 1);
    constexpr int E = sizeof(T);
    const int tid = threadIdx.x, warp = static_cast<int>(tc::uniform(threadIdx.x >> 5)), lane = tid & 31;
    const int cta = static_cast<int>(blockIdx.x) % p.walkers, walkers = p.walkers;
    const int s0 = static_cast<int>(blockIdx.x) / p.walkers * p.NT, width = min(p.NT, p.NO - s0), np = (width + 15) / 16 * 16;

    if (tid == 0) {
        mbar_init(done, 1);
        fence_barrier_init();
    }
    if (warp == 0) tc::alloc(slot, p.tmem_cols);
    // what is not written below is padding: zero weights, zero scales, zero pixels
    for (unsigned i = tid; i < (p.smem_bias - p.smem_a) / 16; i += THREADS) reinterpret_cast<uint4*>(asm_)[i] = make_uint4(0, 0, 0, 0);
    for (int i = tid; i < width; i += THREADS) channel[i] = slot_channel(s0 + i, p.G, p.P);
    tc::fence_before();
    __syncthreads();  // every CTA holds its tensor memory before the next launch may start
    tc::fence_after();
    const uint32_t tmem = tc::uniform(*slot);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // Pieces: the half blocks of a tile (two per block, 128 * nb blocks) go round the threads; (row, j) of this
    // thread's current one, and the step to its next. With an odd nb the last round of 512 threads is half empty
    // (whole warps).
    const unsigned step_row = fdiv(THREADS / 2, p.nbd), step_j = THREADS / 2 - step_row * p.nb;
    const unsigned first = static_cast<unsigned>(tid >> 1), first_row = fdiv(first, p.nbd), first_j = first - first_row * p.nb;
    const int half = tid & 1;
    auto advance = [&](unsigned& row, unsigned& j) {
        row += step_row;
        j += step_j;
        if (j >= static_cast<unsigned>(p.nb)) {
            j -= p.nb;
            ++row;
        }
    };
    // the ring: slots of this thread alone, so a wait for its own copies is all it takes
    int ahead_tile = first_row < 128u ? cta : p.mtiles;  // (one block per row leaves half of 512 threads without any)
    unsigned ahead_row = first_row, ahead_j = first_j, ahead_slot = 0;
    const unsigned my_ring = smem_addr(ring) + tid * 16u;
    auto fetch = [&]() {
        if constexpr (VEC) {
            if (ahead_tile < p.mtiles) {
                const unsigned c0 = ahead_j * kMxBlock + half * 16;
                if (static_cast<int>(ahead_row) < p.M - ahead_tile * 128) {
                    const T* src = y + static_cast<size_t>(ahead_tile) * 128 * p.C + (ahead_row * p.C + c0);
                    const unsigned dst = my_ring + ahead_slot;
#pragma unroll
                    for (int q = 0; q < MxRaw<T>::kVecs; ++q)
                        if (static_cast<int>(c0) + q * (16 / E) < p.C)
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + q * (S::kAhead * THREADS * 16)),
                                         "l"(src + q * (16 / E))
                                         : "memory");
                }
                ahead_slot = ahead_slot == (S::kAhead - 1) * THREADS * 16u ? 0u : ahead_slot + THREADS * 16u;
                advance(ahead_row, ahead_j);
                if (ahead_row >= 128u) {
                    ahead_row = first_row;
                    ahead_j = first_j;
                    ahead_tile += walkers;
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    };
    for (int n = 0; n < S::kAhead; ++n) fetch();

    // the weight's rows in record order with their scales, four blocks in flight per thread, and the bias
    {
        const int items = width * p.nb;
        for (int i0 = tid; i0 < items; i0 += 4 * THREADS) {
            uint4 v[4];
            uint8_t sc[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int i = i0 + q * THREADS;
                if (i < items) {
                    const int s = static_cast<int>(fdiv(static_cast<unsigned>(i), p.nbd)), j = i - s * p.nb;
                    const size_t at = static_cast<size_t>(channel[s]) * p.nb + j;
                    v[q] = __ldg(wcodes + at);
                    sc[q] = __ldg(wscales + at);
                }
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int i = i0 + q * THREADS;
                if (i < items) {
                    const int s = static_cast<int>(fdiv(static_cast<unsigned>(i), p.nbd)), j = i - s * p.nb;
                    *reinterpret_cast<uint4*>(bsm + static_cast<size_t>(j) * p.NT * 16 + s * 16) = v[q];
                    sfb[((j >> 2) * p.groups + (s >> 7)) * 512 + (s & 31) * 16 + ((s >> 5) & 3) * 4 + (j & 3)] = sc[q];
                }
            }
        }
        for (int i = tid; i < p.NT; i += THREADS) bias_s[i] = bias && i < width ? __ldg(bias + channel[i]) : 0.f;
    }
    __syncthreads();

    bool ok = true;
    unsigned at_slot = 0;
    for (int tile = cta, it = 0; tile < p.mtiles; tile += walkers, ++it) {
        const int rows = static_cast<int>(min(128LL, p.M - static_cast<long long>(tile) * 128));
        for (unsigned row = first_row, j = first_j; row < 128u; advance(row, j)) {
            const int c0 = static_cast<int>(j) * kMxBlock + half * 16;
            MxRaw<T> r;
            if constexpr (VEC) {
                asm volatile("cp.async.wait_group %0;" ::"n"(S::kAhead - 1) : "memory");
                const unsigned char* at = ring + at_slot + tid * 16;
                at_slot = at_slot == (S::kAhead - 1) * THREADS * 16u ? 0u : at_slot + THREADS * 16u;
#pragma unroll
                for (int q = 0; q < MxRaw<T>::kVecs; ++q)
                    r.w[q] = static_cast<int>(row) < rows && c0 + q * (16 / E) < p.C
                                 ? *reinterpret_cast<const uint4*>(at + q * (S::kAhead * THREADS * 16)) : make_uint4(0, 0, 0, 0);
            } else {
                mx_load<T, false>(y + (static_cast<long long>(tile) * 128 + min(static_cast<int>(row), rows - 1)) * p.C, c0, p.C, r);
            }
            uint2 codes;
            const uint32_t s = mx_half_block<false>(r, codes);
            fetch();  // into the slot just read (the shuffle used what it held)
            *reinterpret_cast<uint2*>(asm_ + j * 2048u + row * 16u + half * 8u) = codes;
            if (half == 0)
                sfa[(j >> 2) * 512u + (row & 31u) * 16u + (row >> 5) * 4u + (j & 3u)] = static_cast<unsigned char>(s);
        }
        fence_proxy_async();
        // the bulk copies that read the staging tile have done so
        if (warp == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        tc::fence_before();
        __syncthreads();
        if (warp == 0) {
            tc::fence_after();
            const uint32_t lead = tc::lead_lane();
            if (lead) {
                if (it == 0)
                    for (int i = 0; i < p.kc * p.groups; ++i) tc::copy_scales(tmem + p.sfb_col + i * 4, smem_addr(sfb + i * 512));
                for (int i = 0; i < p.kc; ++i) tc::copy_scales(tmem + p.sfa_col + i * 4, smem_addr(sfa + i * 512));
            }
            __syncwarp();
            const uint64_t a = tc::smem_desc(smem_addr(asm_), 2048u, 128u, 0u), b = tc::smem_desc(smem_addr(bsm), 16u * p.NT, 128u, 0u);
            for (int k = 0; k < p.k64; ++k)
                tc::mma_mxf4(tmem, a + k * 256u, b + static_cast<unsigned>(k) * 2u * p.NT, tc::idesc_mxf4(np, (k & 1) * 2u),
                             tmem + p.sfa_col + (k >> 1) * 4, tmem + p.sfb_col + (k >> 1) * 4 * p.groups, k > 0, lead);
            if (lead) tc::commit(done);
        }
        // one warp polls; the others wait at the barrier, where they take no issue slots
        ok = __syncthreads_and(warp != 0 || mbar_wait_bounded(done, static_cast<unsigned>(it) & 1u, kCopyWaitLimitNs)) != 0;
        if (!ok) {
            // given up: the copies and products in flight are waited for, again with a limit, before the CTA leaves
            asm volatile("cp.async.wait_all;" ::: "memory");
            if (warp == 0) mbar_wait_bounded(done, static_cast<unsigned>(it) & 1u, kCopyWaitLimitNs);
            break;
        }
        tc::fence_after();

        // accumulator row = pixel: lane 32 * (warp % 4) + lane; 16-column chunks shared out among a quarter's warps
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        unsigned char* orow = stage + static_cast<size_t>(row) * p.pitch;
        // kMxStoreTma: 16-byte chunk k of a row of a 128-byte block lies at k ^ (row mod 8), of a 64-byte one at
        // k ^ (row / 2 mod 4), as the map's swizzle has it
        const unsigned twist = p.pitch == 128 ? row & 7 : (row >> 1) & 3, cpb = static_cast<unsigned>(p.pitch) >> 4;
        for (int c0 = (warp >> 2) * 16; c0 < np; c0 += THREADS / 8) {
            float v[16];
            tc::ld16(lanes + c0, v);
            tc::wait_ld();
#pragma unroll
            for (int q = 0; q < 16; q += 4) {
                const float4 b4 = *reinterpret_cast<const float4*>(bias_s + c0 + q);
                v[q] += b4.x; v[q + 1] += b4.y; v[q + 2] += b4.z; v[q + 3] += b4.w;
            }
            uint32_t w[4 * E];
            if constexpr (E == 4) {
#pragma unroll
                for (int q = 0; q < 16; ++q) w[q] = __float_as_uint(v[q]);
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q) w[q] = pack2(v[2 * q], v[2 * q + 1], static_cast<T*>(nullptr));
            }
            if (p.store == kMxStoreTma) {
#pragma unroll
                for (int q = 0; q < E; ++q) {
                    const unsigned k = static_cast<unsigned>(c0) * E / 16u + q;
                    const unsigned block = cpb == 8 ? k >> 3 : k >> 2, kk = k & (cpb - 1);
                    *reinterpret_cast<uint4*>(stage + block * 128u * p.pitch + row * p.pitch + ((kk ^ twist) << 4)) =
                        make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
                }
            } else if ((p.pitch & 7) == 0 && c0 + 16 <= width) {
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
        T* dst = rec + static_cast<size_t>(tile) * 128 * p.NO + s0;
        const unsigned row_bytes = static_cast<unsigned>(width) * E;
        if (p.store == kMxStoreTile && (rows * row_bytes) % 16u == 0u) {
            if (tid == 0)
                asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
                             "r"(smem_addr(stage)), "r"(rows * row_bytes)
                             : "memory");
        } else if (p.store == kMxStoreTma) {
            if (tid == 0)
                for (unsigned q = 0; q * p.pitch < row_bytes; ++q)
                    tc::tma_store_3d(&rmap, s0 + static_cast<int>(q * p.pitch / E), tile * 128, 0, stage + q * 128u * p.pitch);
        } else {
            for (int r = warp; r < rows; r += THREADS / 32)
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
        if (tid < 64) {
            const int r = tid >> 1, half = tid & 1;
            MxRaw<T> raw;
            mx_load<T, VEC>(y + static_cast<size_t>(min(m0 + r, p.M - 1LL)) * p.C, b * kMxBlock + half * 16, p.C, raw);
            uint2 c;
            const float sc = mx_scale_value(mx_half_block<true>(raw, c));
#pragma unroll
            for (int i = 0; i < 16; ++i) ys[r][half * 16 + i] = e2m1_value(((i < 8 ? c.x : c.y) >> (4 * (i & 7))) & 15u) * sc;
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
