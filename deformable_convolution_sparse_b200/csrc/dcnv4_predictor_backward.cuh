// sm_100a kernels of the offset/mask predictor's backward. With the projection
//   record[m, slot(o)] = bias[o] + sum_c W[o, c] y[m, c]
// and g[m, s] = dL/drecord[m, s] (the fp32 records the aggregation's backward
// writes), the gradients are, over record slots s,
//   dL/dy[m, c] = sum_s g[m, s] W[s, c]
//   dL/dW[s, c] = sum_m g[m, s] y[m, c]
//   dL/dbias[s] = sum_m g[m, s]
// and the rows of the last two are moved to the projection's channel order.
//
// Precision on the tensor cores. An fp32 value is the exact sum of three bf16
// values, h = bf16(v), m = bf16(v - h), l = v - h - m (24 bits in three times
// 8; below 2^-110 l falls under bf16's smallest number, and the sum is off by at
// most 2^-134); fp16 takes two and bf16 one. A product of two
// such sums keeps the pairs whose orders add to at most 2 (the others are
// below 2^-26 of it): 3 tensor-core products for bf16 operands, 5 for fp16, 6
// for fp32, each exact, summed in fp32. The tensor cores' additions truncate,
// so a long chain of them drifts one way: the pairs of order 0 go to up to
// three accumulators in turn, the small others to one of their own, and these
// are added with rounding when they are read; the weight's gradient is read
// out every kFlushTiles tiles of pixels.
//
// Memory bounds the formulas. 16-bit y with at most 64 channels and 128 slots
// takes one kernel that reads g once; else g is read by two (dL/dW's sums beside
// dL/dy's need more tensor memory than there is, the planes of y and W more
// shared memory). What bounds the kernels: DRAM latency against the 64 to 96 KB
// of raw tiles a CTA can keep in flight beside its operand planes (such a ring
// alone, without any work, reads g at 3.0 to 3.5 TB/s), and for three planes of
// y the products themselves. Measured on B200, everything together: 200,704
// pixels x 64 channels x 108 slots in bf16 41 us (71 by the two kernels), in
// fp16 59 (87), 129,032 x 128 x 216 slots in bf16 93, 26,047 x 320 fp32 x 192
// slots 100, 196 x 256 fp16 x 432 slots 21, all replayed from a graph. Rows that
// TMA cannot take, 200,704 x 64 in bf16 with 27 slots 71, with 54 83, with 81 93.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dcnv4_async.cuh"
#include "dcnv4_kernels.cuh"
#include "dcnv4_records.cuh"
#include "dcnv4_tcgen05.cuh"

namespace dcnv4 {

struct PredBwdParams {
    int M, C, G, P, NO;
    int tiles;           // tiles of 128 pixels
    int chunks;          // chunks of 64 record slots
    int slices;          // slices of the input channels: CT each (grad_y), 128 each (grad_weight)
    int wrows, wpitch;   // rows and pitch of a plane of W in record order (multiples of 64)
    int groups;          // groups of 128 slots (grad_weight)
    int walkers;         // CTAs that share the pixel tiles of a (slice, group), each with partial sums of its own
    int direct;          // one walker: its sums are the gradients, in the projection's row order
    int tma_out;         // grad_y by TMA
    int raws;            // grad_weight: raw tiles (0: direct reads)
    unsigned ystep;      // grad_weight: bytes between y's planes, 16 KB per block of 64 channels of a slice
    unsigned* status;
};

constexpr int kFlushTiles = 16;
// the wait for a run of kFlushTiles tiles: every copy of it has its own limit, one after the other at worst
constexpr uint64_t kFlushWaitLimitNs = 2 * kCopyWaitLimitNs;

template <typename T>
constexpr int split_planes() {
    return sizeof(T) == 4 ? 3 : std::is_same<T, __half>::value ? 2 : 1;
}

// Row of slot s's sums in a walker's part, or in the gradient itself.
__device__ __forceinline__ size_t sum_row(const PredBwdParams& p, int walker, int s) {
    return p.direct ? static_cast<size_t>(slot_channel(s, p.G, p.P)) : static_cast<size_t>(walker) * p.NO + s;
}

// Two fp32 values as bf16 pairs of falling order (a in the low half).
template <int PLANES>
__device__ __forceinline__ void split_pair(float a, float b, uint32_t (&w)[PLANES]) {
#pragma unroll
    for (int q = 0; q < PLANES; ++q) {
        w[q] = pack2(a, b, static_cast<__nv_bfloat16*>(nullptr));
        if (q + 1 < PLANES) {
            a -= __uint_as_float(w[q] << 16);
            b -= __uint_as_float(w[q] & 0xffff0000u);
        }
    }
}

// eight 16-bit values as fp32
template <typename T>
__device__ __forceinline__ void unpack8(const uint4& w, T* t, float (&v)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 f = unpack2(u[k], t);
        v[2 * k] = f.x;
        v[2 * k + 1] = f.y;
    }
}

// Eight values as 16-byte chunks of PLANES swizzled tiles `step` bytes apart:
// row r, chunk ch of 128-byte rows.
template <int PLANES>
__device__ __forceinline__ void store_split8(unsigned char* tile, unsigned step, int r, int ch, const float (&v)[8]) {
    uint32_t w[4][PLANES];
#pragma unroll
    for (int q = 0; q < 4; ++q) split_pair<PLANES>(v[2 * q], v[2 * q + 1], w[q]);
    unsigned char* at = tile + r * 128 + ((ch ^ (r & 7)) << 4);
#pragma unroll
    for (int q = 0; q < PLANES; ++q)
        *reinterpret_cast<uint4*>(at + q * step) = make_uint4(w[0][q], w[1][q], w[2][q], w[3][q]);
}

// W's planes in record order, zero padded: planes [PLANES][wrows][wpitch].
template <typename T>
__global__ void __launch_bounds__(256)
pred_split_weight_kernel(const T* __restrict__ w, __nv_bfloat16* __restrict__ planes, PredBwdParams p) {
    constexpr int PL = split_planes<T>();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long n = static_cast<long long>(p.wrows) * p.wpitch / 2;
    for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < n;
         i += static_cast<long long>(gridDim.x) * 256) {
        const int s = static_cast<int>(2 * i / p.wpitch), c = static_cast<int>(2 * i - static_cast<long long>(s) * p.wpitch);
        float a = 0.f, b = 0.f;
        if (s < p.NO) {
            const T* row = w + static_cast<size_t>(slot_channel(s, p.G, p.P)) * p.C;
            if (c < p.C) a = ElemTraits<T>::to_float(__ldg(row + c));
            if (c + 1 < p.C) b = ElemTraits<T>::to_float(__ldg(row + c + 1));
        }
        uint32_t q[PL];
        split_pair<PL>(a, b, q);
#pragma unroll
        for (int k = 0; k < PL; ++k) reinterpret_cast<uint32_t*>(planes)[k * n + i] = q[k];
    }
}

// Columns of a row-major matrix (record slots of g, channels of y) are turned
// into operand planes 64 at a time, 128 pixels each. Two groups of kGroup
// threads take the chunks in turn, so that one's waits fall into the other's
// work, in pieces of eight columns: only the groups of eight columns below the
// last 16 valid ones are touched (a chunk's other columns are never read, or
// only into sums that nobody reads). A thread has at most four pieces, of the
// same columns and rows `rows` apart. By TMA the values come through a ring of
// raw tiles (blocks of 128 bytes of columns x 128 rows, 128-byte swizzle, zeros
// past the matrix): reads through L1 would have no room there, since the
// operand tiles take most of an SM's memory, and so few of them in flight that
// DRAM idles (measured: 31 % of its rate). A raw tile is given back as soon as
// its values are in registers, so that the ring is nearly always in flight;
// landed() is what makes sure of that, since an arrival after the reads in
// program order can overtake those still on their way (the next tile then
// showed up in them). Matrices whose rows TMA cannot take are read directly.
constexpr int kConv = 512, kGroup = 256, kPieces = 4;
constexpr unsigned kRaw = 32768u;  // 128 rows x 64 fp32
struct ChunkWalk {
    int ng, row, grp, rows;  // groups of eight columns; this thread's first row, its columns, rows per round
    __device__ __forceinline__ ChunkWalk(int columns, int tid) {
        const int t = tid % kGroup;
        ng = min(8, (columns + 15) / 16 * 2);
        rows = kGroup / ng;
        row = t / ng;
        grp = t - row * ng;
        if (row >= rows) row = 128;  // the threads left over
    }
};
template <typename T>
struct Piece {
    float v[kPieces][8];
    // from a raw tile: column c of row r is in block c / (128 / sizeof(T)), 16-byte chunk k at k ^ (r mod 8)
    __device__ __forceinline__ void from_raw(const unsigned char* raw, const ChunkWalk& walk) {
#pragma unroll
        for (int q = 0; q < kPieces; ++q) {
            const int row = walk.row + q * walk.rows;
            if (row >= 128) {
#pragma unroll
                for (int k = 0; k < 8; ++k) v[q][k] = 0.f;
                continue;
            }
            if constexpr (sizeof(T) == 4) {
                // groups 0..3 and 4..7 of a row lie in two blocks at the same banks: the latter read their second
                // half first
                const unsigned char* at = raw + (walk.grp >> 2) * 16384 + row * 128;
                const int late = walk.grp >> 2;
                const float4 a = *reinterpret_cast<const float4*>(at + ((((walk.grp & 3) * 2 + late) ^ (row & 7)) << 4));
                const float4 b = *reinterpret_cast<const float4*>(at + ((((walk.grp & 3) * 2 + 1 - late) ^ (row & 7)) << 4));
                v[q][0] = late ? b.x : a.x; v[q][1] = late ? b.y : a.y; v[q][2] = late ? b.z : a.z; v[q][3] = late ? b.w : a.w;
                v[q][4] = late ? a.x : b.x; v[q][5] = late ? a.y : b.y; v[q][6] = late ? a.z : b.z; v[q][7] = late ? a.w : b.w;
            } else {
                const uint4 w = *reinterpret_cast<const uint4*>(raw + row * 128 + ((walk.grp ^ (row & 7)) << 4));
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 f = unpack2(u[k], static_cast<T*>(nullptr));
                    v[q][2 * k] = f.x;
                    v[q][2 * k + 1] = f.y;
                }
            }
        }
    }
    // All lanes of the warp: returns once every lane's values have arrived. The vote needs them all, and
    // instructions issue in order; the branch it decides does nothing of use.
    __device__ __forceinline__ void landed() const {
        uint32_t u = 0u;
#pragma unroll
        for (int q = 0; q < kPieces; ++q)
#pragma unroll
            for (int k = 0; k < 8; ++k) u |= __float_as_uint(v[q][k]);
        if (__any_sync(0xffffffffu, u == 0x80000001u)) __nanosleep(1);
    }
    // from memory: rows m0.. of M, columns c0.. of C
    __device__ __forceinline__ void from_global(const T* __restrict__ x, const ChunkWalk& walk, long long m0, int M, int c0, int C) {
#pragma unroll
        for (int q = 0; q < kPieces; ++q) {
            const int row = walk.row + q * walk.rows;
            const T* src = x + (m0 + row) * C + c0 + walk.grp * 8;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[q][k] = row < 128 && m0 + row < M && c0 + walk.grp * 8 + k < C ? ElemTraits<T>::to_float(__ldg(src + k)) : 0.f;
        }
    }
    template <int PLANES>
    __device__ __forceinline__ void store(unsigned char* tile, unsigned step, const ChunkWalk& walk) const {
#pragma unroll
        for (int q = 0; q < kPieces; ++q) {
            const int row = walk.row + q * walk.rows;
            if (row < 128) store_split8<PLANES>(tile, step, row, walk.grp, v[q]);
        }
    }
};
// A converting thread's sums of g for the bias, eight slots: fp32 over runs of
// at most kBiasRun tiles, fp64 from there on, so that the error does not grow
// with the number of pixels (9,000,001 equal values in one fp32 sum per thread:
// 4e-6 of the sum). The fp64 sums are kept in memory (volatile: registers are
// what these threads have least of) and touched once a run. Even unused they
// cost 0.4 to 2.5 us, so calls whose CTAs have one run at most (303,104 pixels
// in the one-pass kernel) take builds without them (not LONG); fp64 in the sums
// over the threads and in the join too cost 3 to 6 us.
constexpr int kBiasRun = 16;
template <bool LONG>
struct BiasSums {
    static constexpr int kRun = LONG ? kBiasRun : 1 << 29;  // tiles
    float run[8] = {};
    volatile double total[LONG ? 8 : 1];
    __device__ __forceinline__ void add(const float (&v)[kPieces][8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e)  // rows past the tile hold zeros
            run[e] += (v[0][e] + v[1][e]) + (v[2][e] + v[3][e]);
    }
    __device__ __forceinline__ void flush(bool first) {
        if constexpr (LONG) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                total[e] = first ? static_cast<double>(run[e]) : total[e] + static_cast<double>(run[e]);
                run[e] = 0.f;
            }
        }
    }
    __device__ __forceinline__ void finish() {
        if constexpr (LONG) {
#pragma unroll
            for (int e = 0; e < 8; ++e) run[e] = static_cast<float>(total[e] + static_cast<double>(run[e]));
        }
    }
};
// the operand tiles this warp's threads wrote, handed over (one arrival per warp)
__device__ __forceinline__ void hand_over(uint64_t* bar, int lane) {
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

// grad_y: tiles of 128 pixels x CT channels. Warps 0..15 write the planes of g
// as the left operand (K-major), 64 slots at a time; warp 16 loads g's raw
// tiles and the same slots' rows of W's planes by TMA, these as the right
// operand (their rows run along the channels: MN-major); warp 17 issues the
// products; warps 18..21 read the accumulators (two sets, in turn) and write
// the tile through shared memory and TMA, 32 channels at a time.
template <int CT, int WP>
struct GradYShape {
    static constexpr int kStages = 2;
    static constexpr int kHigh = CT == 64 ? 3 : 1;  // accumulators of order 0
    static constexpr unsigned kWBytes = WP * (CT / 64) * 8192u;
    static constexpr unsigned kStage = 3u * 16384u + kWBytes;
    static constexpr unsigned kOut = 16384u;
    // raw tiles: as many as fit, up to three (each takes about 2 us to come from a busy DRAM)
    static constexpr int kRaws = kStages * kStage + kOut + 3 * kRaw <= 224u * 1024u   ? 3
                                 : kStages * kStage + kOut + 2 * kRaw <= 224u * 1024u ? 2
                                                                                      : 1;
    static constexpr unsigned kSmem = 1024u + kStages * kStage + kOut + kRaws * kRaw + 256u;
    static constexpr unsigned kAcc = (kHigh + 1) * CT;  // columns of one set
};
constexpr int kGradYThreads = kConv + 64 + 128;

template <int CT, int WP, bool RAW>
__global__ void __launch_bounds__(kGradYThreads, 1)
pred_grad_y_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap gmap,
                   const __grid_constant__ CUtensorMap omap, const float* __restrict__ grec, float* __restrict__ gy,
                   PredBwdParams p) {
    using S = GradYShape<CT, WP>;
    extern __shared__ unsigned char pb_smem_raw[];
    unsigned char* sm = pb_smem_raw + ((1024u - (smem_addr(pb_smem_raw) & 1023u)) & 1023u);
    unsigned char* outs = sm + S::kStages * S::kStage;
    unsigned char* raws = outs + S::kOut;
    uint64_t* bars = reinterpret_cast<uint64_t*>(raws + S::kRaws * kRaw);
    uint64_t *full_g = bars, *full_w = bars + 2, *empty = bars + 4, *acc_full = bars + 6, *acc_empty = bars + 8,
             *raw_full = bars + 10, *raw_empty = bars + 14;  // of step it: the (it mod 4)-th
    uint32_t* slot = reinterpret_cast<uint32_t*>(bars + 18);
    uint64_t* drain = bars + 19;
    const int tid = threadIdx.x, warp = static_cast<int>(tc::uniform(threadIdx.x >> 5)), lane = tid & 31;

    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&full_g[s], kGroup / 32);
            mbar_init(&full_w[s], 1);
            mbar_init(&empty[s], 1);
            mbar_init(&acc_full[s], 1);
            mbar_init(&acc_empty[s], 128);
        }
        for (int s = 0; s < 4; ++s) {
            mbar_init(&raw_full[s], 1);
            mbar_init(&raw_empty[s], kGroup / 32);
        }
        mbar_init(drain, 1);
        fence_barrier_init();
    }
    if (warp == 16) tc::alloc(slot, 512u);
    tc::fence_before();
    __syncthreads();  // every CTA holds its tensor memory before the next launch may start
    tc::fence_after();
    const uint32_t tmem = tc::uniform(*slot);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // items: (tile, slice), slices of a tile side by side
    const long long items = static_cast<long long>(p.tiles) * p.slices;
    const long long mine = blockIdx.x < items ? (items - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;
    const long long steps = mine * p.chunks;
    bool ok = true;
    long long raw_n = 0, w_n = 0;  // the loading lane's steps so far

    if (warp < 16) {
        const ChunkWalk whole(64, tid), tail(p.NO - (p.chunks - 1) * 64, tid);
        Piece<float> piece;
        const int s = warp >> 3;  // this group's operand stage, and the parity of its steps
        int chunk = s;
        long long n = 0;          // the item
        for (long long it = s; it < steps && ok; it += 2, chunk += 2) {
            while (chunk >= p.chunks) {
                chunk -= p.chunks;
                ++n;
            }
            const ChunkWalk& walk = chunk + 1 < p.chunks ? whole : tail;
            if constexpr (RAW) {
                ok = tc::warp_wait(&raw_full[it & 3], static_cast<unsigned>(it >> 2) & 1u, kCopyWaitLimitNs);
                if (!ok) break;
                piece.from_raw(raws + (it % S::kRaws) * kRaw, walk);
                piece.landed();
                if (lane == 0) mbar_arrive(&raw_empty[it & 3]);
            } else {
                const long long item = blockIdx.x + n * gridDim.x;
                piece.from_global(grec, walk, item / p.slices * 128, p.M, chunk * 64, p.NO);
            }
            if (it >= 2) ok = tc::warp_wait(&empty[s], static_cast<unsigned>((it >> 1) - 1) & 1u, kCopyWaitLimitNs);
            if (!ok) break;
            piece.template store<3>(sm + s * S::kStage, 16384u, walk);
            hand_over(&full_g[s], lane);
        }
    } else if (warp == 16) {
        if (lane == 0) {
            // raw tiles run ahead of the operand stages by as many as the ring holds
            auto where = [&](long long it, int& m0, int& c0, int& s0) {
                const long long item = blockIdx.x + (it / p.chunks) * gridDim.x;
                m0 = static_cast<int>(item / p.slices) * 128;
                c0 = static_cast<int>(item % p.slices) * CT;
                s0 = static_cast<int>(it % p.chunks) * 64;
            };
            auto load_raw = [&](long long it) {
                if (!RAW || it >= steps) return;
                // the tile's place is free once step it - kRaws has given it back. A group waits for every fourth
                // step's barrier after its own use of it four steps before, whatever the ring's length.
                const int r = static_cast<int>(it % S::kRaws), f = static_cast<int>(it & 3);
                const long long before = it - S::kRaws;
                if (before >= 0)
                    ok = mbar_wait_bounded(&raw_empty[before & 3], static_cast<unsigned>(before >> 2) & 1u, kCopyWaitLimitNs);
                if (!ok) return;
                int m0, c0, s0;
                where(it, m0, c0, s0);
                const int halves = s0 + 32 < p.NO ? 2 : 1;
                mbar_expect_tx(&raw_full[f], halves * 16384u);
                for (int h = 0; h < halves; ++h) tc::tma_load_3d(raws + r * kRaw + h * 16384, &gmap, s0 + h * 32, m0, 0, &raw_full[f]);
                mbar_arrive(&raw_full[f]);
                raw_n = it + 1;
            };
            for (int k = 0; k < S::kRaws; ++k) load_raw(k);
            for (long long it = 0; it < steps && ok; ++it) {
                const int s = static_cast<int>(it & 1);
                if (it >= 2) ok = mbar_wait_bounded(&empty[s], static_cast<unsigned>((it >> 1) - 1) & 1u, kCopyWaitLimitNs);
                if (!ok) break;
                int m0, c0, s0;
                where(it, m0, c0, s0);
                unsigned char* w = sm + s * S::kStage + 3 * 16384;
                mbar_expect_tx(&full_w[s], S::kWBytes);
                for (int pl = 0; pl < WP; ++pl)
                    for (int b = 0; b < CT / 64; ++b)
                        tc::tma_load_3d(w + (pl * (CT / 64) + b) * 8192, &wmap, c0 + b * 64, s0, pl, &full_w[s]);
                mbar_arrive(&full_w[s]);
                w_n = it + 1;
                load_raw(it + S::kRaws);
            }
        }
    } else if (warp == 17) {
        constexpr uint32_t idesc = tc::idesc_f16(tc::kFmtBf16, CT, false, true);
        const uint32_t lead = tc::lead_lane();
        int chunk = 0, b = 0;
        long long n = 0;  // the item
        for (long long it = 0; it < steps && ok; ++it) {
            const int s = static_cast<int>(it & 1);
            if (chunk == 0 && n >= 2)
                ok = tc::warp_wait(&acc_empty[b], static_cast<unsigned>((n >> 1) - 1) & 1u, kCopyWaitLimitNs);
            ok = ok && tc::warp_wait(&full_g[s], static_cast<unsigned>(it >> 1) & 1u, kCopyWaitLimitNs) &&
                 tc::warp_wait(&full_w[s], static_cast<unsigned>(it >> 1) & 1u, kCopyWaitLimitNs);
            if (!ok) break;
            tc::fence_after();
            const uint32_t acc = tmem + b * S::kAcc, low = acc + S::kHigh * CT;
            const unsigned base = smem_addr(sm + s * S::kStage);
            const uint32_t a = tc::sw128(base), w = tc::sw128(base + 3u * 16384u, 8192u);
            const int ksteps = (min(64, p.NO - chunk * 64) + 15) / 16;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (k >= ksteps) break;
#pragma unroll
                for (int i = 0; i < 3; ++i)
#pragma unroll
                    for (int j = 0; j < WP; ++j) {
                        if (i + j > 2) continue;
                        const uint32_t ad = a + i * 1024 + k * 2, bd = w + j * (CT / 64) * 512 + k * 128;
                        const bool first_low = k == 0 && i == (WP > 1 ? 0 : 1) && j == (WP > 1 ? 1 : 0);
                        if (i + j == 0) tc::mma_f16(acc + (k % S::kHigh) * CT, ad, bd, idesc, chunk > 0 || k >= S::kHigh, lead);
                        else tc::mma_f16(low, ad, bd, idesc, chunk > 0 || !first_low, lead);
                    }
            }
            if (lead) {
                tc::commit(&empty[s]);
                if (chunk == p.chunks - 1) tc::commit(&acc_full[b]);
            }
            if (++chunk == p.chunks) {
                chunk = 0;
                b ^= 1;
                ++n;
            }
        }
    } else {
        const int quarter = warp & 3, row = quarter * 32 + lane, et = tid - (kConv + 64);
        const int high = min(S::kHigh, (p.NO + 15) / 16);
        for (long long n = 0; n < mine; ++n) {
            const long long item = blockIdx.x + n * gridDim.x;
            const long long m0 = item / p.slices * 128;
            const int c0 = static_cast<int>(item % p.slices) * CT, b = static_cast<int>(n & 1);
            ok = tc::bar_and(1, 128, mbar_wait_bounded(&acc_full[b], static_cast<unsigned>(n >> 1) & 1u, kCopyWaitLimitNs));
            if (!ok) break;
            tc::fence_after();
            const uint32_t acc = tmem + b * S::kAcc + (static_cast<uint32_t>(quarter * 32) << 16);
            for (int h = 0; h < CT / 32; ++h) {
                const int ch = c0 + h * 32;
                if (ch >= p.C) break;
                // the store that read the staging tile has done so
                if (et == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                tc::bar_sync(1, 128);
                for (int cc = 0; cc < 2; ++cc) {
                    float v[16], w[16];
                    tc::ld16(acc + S::kHigh * CT + h * 32 + cc * 16, v);
                    for (int q = 0; q < high; ++q) {
                        tc::ld16(acc + q * CT + h * 32 + cc * 16, w);
                        tc::wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] += w[e];
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        *reinterpret_cast<float4*>(outs + row * 128 + (((cc * 4 + q) ^ (row & 7)) << 4)) =
                            make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                }
                if (p.tma_out) fence_proxy_async();
                tc::bar_sync(1, 128);
                if (p.tma_out) {
                    if (et == 0) {
                        tc::tma_store_3d(&omap, ch, static_cast<int>(m0), 0, outs);
                        tc::bulk_commit();
                    }
                } else {
                    const int rows = static_cast<int>(min(128LL, p.M - m0));
                    if (ch + lane < p.C)
                        for (int r = quarter; r < rows; r += 4)
                            gy[(m0 + r) * p.C + ch + lane] = *reinterpret_cast<const float*>(
                                outs + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
                }
            }
            tc::fence_before();
            mbar_arrive(&acc_empty[b]);
        }
        if (et == 0) tc::bulk_wait_all();
    }
    if (!ok) atomicOr(p.status, kStatusCopyTimeout);
    tc::fence_before();
    if (!__syncthreads_and(ok)) {
        if (warp == 16 && lane == 0) {
            tc::drain_loads<4>(raw_full, raw_n, S::kRaws);
            tc::drain_loads<2>(full_w, w_n, 2);
        }
        if (warp == 17) tc::drain_products(drain);
        __syncthreads();
    }
    tc::fence_after();
    if (warp == 16) tc::dealloc(tmem, 512u);
}

// grad_weight and grad_bias, partial sums: 128 channels x 128 slots per CTA,
// the pixels of every walkers-th tile. Warps 0..15 write the planes of y (the
// left operand) and, 64 slots at a time, of g (the right one), both with rows
// that run along channels or slots: MN-major; the same threads sum g for the
// bias. y in bf16 is its own plane and comes straight by TMA. Of warps 16..19,
// one issues the products and a lane of another the TMA loads; every kFlushTiles
// tiles all four read the accumulators out to part [walkers][NO][C] (one walker:
// to the gradient), lanes along the channels. A slice of at most 64 channels reads its one block of 64
// for both halves of the M = 128 products.
template <typename T, bool RAW>
struct GradWShape {
    static constexpr int YP = split_planes<T>();
    static constexpr bool kDirectY = RAW && YP == 1;  // y's plane by TMA
    static constexpr int kYStages = YP == 1 ? 2 : 1;
    static constexpr unsigned kG = 3u * 16384u;
    static constexpr unsigned fixed(unsigned ystep) { return kYStages * YP * ystep + 2u * kG; }
    // as many raw tiles as fit, up to three
    static constexpr int raws(unsigned ystep) {
        return !RAW ? 0 : fixed(ystep) + 3 * kRaw <= 224u * 1024u ? 3 : fixed(ystep) + 2 * kRaw <= 224u * 1024u ? 2 : 1;
    }
    static constexpr unsigned smem(unsigned ystep) { return 1024u + fixed(ystep) + raws(ystep) * kRaw + 256u; }
};
constexpr int kGradWThreads = kConv + 128;

template <typename T, bool RAW, bool LONG>
__global__ void __launch_bounds__(kGradWThreads, 1)
pred_grad_w_kernel(const __grid_constant__ CUtensorMap gmap, const __grid_constant__ CUtensorMap ymap,
                   const float* __restrict__ grec, const T* __restrict__ y, float* __restrict__ part,
                   float* __restrict__ pbias, PredBwdParams p) {
    using S = GradWShape<T, RAW>;
    constexpr int YP = S::YP;
    extern __shared__ unsigned char pb_smem_raw[];
    unsigned char* sm = pb_smem_raw + ((1024u - (smem_addr(pb_smem_raw) & 1023u)) & 1023u);
    const unsigned ystage = YP * p.ystep;
    unsigned char* gsm = sm + S::kYStages * ystage;
    unsigned char* raws = gsm + 2 * S::kG;
    uint64_t* bars = reinterpret_cast<uint64_t*>(raws + p.raws * kRaw);
    uint64_t *full_y = bars, *empty_y = bars + 2, *full_g = bars + 4, *empty_g = bars + 6, *acc_full = bars + 8,
             *raw_full = bars + 9, *raw_empty = bars + 13;  // of raw tile k: the (k mod 4)-th
    uint32_t* slot = reinterpret_cast<uint32_t*>(bars + 17);
    uint64_t* drain = bars + 18;
    const int tid = threadIdx.x, warp = static_cast<int>(tc::uniform(threadIdx.x >> 5)), lane = tid & 31;

    // CTA -> walker, (slice, group); the slices and groups of one walker side by side
    const int per = p.slices * p.groups;
    const int walker = static_cast<int>(blockIdx.x) / per, which = static_cast<int>(blockIdx.x) % per;
    const int c0 = which % p.slices * 128, g0 = which / p.slices * 128;
    const int nch = (min(128, p.NO - g0) + 63) / 64;    // chunks of this group
    const bool wide = p.C - c0 > 64;
    const int ny = wide ? 2 : 1;                        // blocks of 64 channels of this slice
    const int mine = walker < p.tiles ? (p.tiles - walker + p.walkers - 1) / p.walkers : 0;
    auto pixel = [&](int i) { return (static_cast<long long>(walker) + static_cast<long long>(i) * p.walkers) * 128; };

    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&full_y[s], S::kDirectY ? 1 : kGroup / 32 * ny);
            mbar_init(&empty_y[s], 1);
            mbar_init(&full_g[s], kGroup / 32);
            mbar_init(&empty_g[s], 1);
        }
        for (int s = 0; s < 4; ++s) {
            mbar_init(&raw_full[s], 1);
            mbar_init(&raw_empty[s], kGroup / 32);
        }
        mbar_init(acc_full, 1);
        mbar_init(drain, 1);
        fence_barrier_init();
    }
    if (warp == 16) tc::alloc(slot, 512u);
    tc::fence_before();
    __syncthreads();  // every CTA holds its tensor memory before the next launch may start
    tc::fence_after();
    const uint32_t tmem = tc::uniform(*slot);
    // No wait for the launch before, which is grad_y's: this kernel reads nothing of it, and it starts once all of
    // that one's CTAs have let it, after their own wait, so that everything before them is complete. It does wait at
    // its end, so that whatever waits for this kernel has grad_y as well.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    bool ok = true;
    int raw_n = 0, y_n = 0;  // the loading lane's raw tiles and tiles of y so far

    if (warp < 16) {
        const bool sums = c0 == 0 && pbias != nullptr;
        using Sums = BiasSums<LONG>;
        Sums bs[2];                       // of each chunk
        const ChunkWalk walk0(p.NO - g0, tid), walk1(nch == 2 ? p.NO - g0 - 64 : 64, tid);
        const ChunkWalk ywalk0(p.C - c0, tid), ywalk1(wide ? p.C - c0 - 64 : 64, tid);
        const int group = warp >> 3;
        // chunks (of y, then of g, tile by tile) so far, and their place in the ring; this group takes those of its
        // parity
        int k = 0;
        unsigned char* place = raws;
        auto next = [&] {
            ++k;
            place = place == raws + (p.raws - 1) * kRaw ? raws : place + kRaw;
        };
        auto take = [&](auto& piece, const ChunkWalk& walk) {
            ok = tc::warp_wait(&raw_full[k & 3], static_cast<unsigned>(k >> 2) & 1u, kCopyWaitLimitNs);
            if (!ok) return;
            piece.from_raw(place, walk);
            piece.landed();
            if (lane == 0) mbar_arrive(&raw_empty[k & 3]);
        };
        for (int begin = 0; begin < mine && ok; begin += Sums::kRun) {
            for (int i = begin, end = min(mine, begin + Sums::kRun); i < end && ok; ++i) {
                // With one stage of y, both groups wait for its release once a tile, before their first store. A group
                // that writes y (or a stage of g) in every other tile only would otherwise miss a phase of the barrier
                // and take the one before for the one it needs.
                bool freed = i == 0;
                auto y_freed = [&] {
                    if constexpr (!S::kDirectY && S::kYStages == 1) {
                        if (!freed) ok = ok && tc::warp_wait(&empty_y[0], static_cast<unsigned>(i - 1) & 1u, kCopyWaitLimitNs);
                        freed = true;
                    }
                };
                if constexpr (!S::kDirectY) {
                    const int ys = i % S::kYStages, yn = i / S::kYStages;
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        if (b >= ny || !ok) break;
                        if ((k & 1) == group) {
                            const ChunkWalk& walk = b ? ywalk1 : ywalk0;
                            Piece<T> piece;
                            if constexpr (RAW) take(piece, walk);
                            else piece.from_global(y, walk, pixel(i), p.M, c0 + b * 64, p.C);
                            y_freed();
                            if (S::kYStages > 1 && yn > 0)
                                ok = ok && tc::warp_wait(&empty_y[ys], static_cast<unsigned>(yn - 1) & 1u, kCopyWaitLimitNs);
                            if (!ok) break;
                            piece.template store<YP>(sm + ys * ystage + b * 16384, p.ystep, walk);
                            hand_over(&full_y[ys], lane);
                        }
                        next();
                    }
                }
#pragma unroll
                for (int ch = 0; ch < 2; ++ch) {
                    if (ch >= nch || !ok) break;
                    if ((k & 1) == group) {
                        const ChunkWalk& walk = ch ? walk1 : walk0;
                        const int n = i * nch + ch, s = n & 1;
                        Piece<float> piece;
                        if constexpr (RAW) take(piece, walk);
                        else piece.from_global(grec, walk, pixel(i), p.M, g0 + ch * 64, p.NO);
                        y_freed();
                        if (n >= 2) ok = ok && tc::warp_wait(&empty_g[s], static_cast<unsigned>((n >> 1) - 1) & 1u, kCopyWaitLimitNs);
                        if (!ok) break;
                        piece.template store<3>(gsm + s * S::kG, 16384u, walk);
                        hand_over(&full_g[s], lane);
                        if (sums) bs[ch].add(piece.v);
                    }
                    next();
                }
            }
            if (sums && begin + Sums::kRun < mine) {
                bs[0].flush(begin == 0);
                bs[1].flush(begin == 0);
            }
        }
        if (sums) {
            // once the last products have read the operand tiles (a commit covers all those before it), the
            // threads' sums are added there, a slot's in the order of its rows' pieces
            const int last = mine * nch;
            if (ok && last > 0) {
                const int s = (last - 1) & 1;
                ok = tc::warp_wait(&empty_g[s], static_cast<unsigned>((last - 1) >> 1) & 1u, kCopyWaitLimitNs);
            }
            float* red = reinterpret_cast<float*>(gsm);  // [thread][8], one chunk at a time
#pragma unroll
            for (int ch = 0; ch < 2; ++ch) {
                if (ch >= nch) break;
                const int ng = ch ? walk1.ng : walk0.ng, rows = ch ? walk1.rows : walk0.rows;
                tc::bar_sync(2, kConv);
                if (ok) {
                    if (mine > Sums::kRun) bs[ch].finish();
#pragma unroll
                    for (int k = 0; k < 8; ++k) red[tid * 8 + k] = bs[ch].run[k];
                }
                tc::bar_sync(2, kConv);
                // eight threads per slot, every eighth of the slot's threads of both groups each, then the eight
                const int s = tid >> 3, part8 = tid & 7;
                float v = 0.f;
                if (s < ng * 8)
                    for (int r = part8; r < rows; r += 8) {
                        const float* at = red + (r * ng + (s >> 3)) * 8 + (s & 7);
                        v += at[0] + at[kGroup * 8];
                    }
                v += __shfl_xor_sync(0xffffffffu, v, 1);
                v += __shfl_xor_sync(0xffffffffu, v, 2);
                v += __shfl_xor_sync(0xffffffffu, v, 4);
                if (ok && part8 == 0 && s < ng * 8 && g0 + ch * 64 + s < p.NO)
                    pbias[sum_row(p, walker, g0 + ch * 64 + s)] = v;
            }
        }
    } else {
        // Up to kFlushTiles tiles: warp 16 issues the products, a lane of warp 17 the loads; then
        // all four warps read the sums out.
        constexpr uint32_t idesc = tc::idesc_f16(tc::kFmtBf16, 64, true, true);
        const unsigned second = wide ? 16384u : 0u;
        const int quarter = warp & 3, row = quarter * 32 + lane, c = c0 + row;
        const bool on = c < p.C && (wide || row < 64);
        int r = 0;
        auto load_raw = [&](const CUtensorMap* map, int col, int step, int blocks, long long m0) {
            const int f = raw_n & 3, before = raw_n - p.raws;
            if (before >= 0)
                ok = mbar_wait_bounded(&raw_empty[before & 3], static_cast<unsigned>(before >> 2) & 1u, kCopyWaitLimitNs);
            if (!ok) return;
            mbar_expect_tx(&raw_full[f], blocks * 16384u);
            for (int b = 0; b < blocks; ++b)
                tc::tma_load_3d(raws + r * kRaw + b * 16384, map, col + b * step, static_cast<int>(m0), 0, &raw_full[f]);
            mbar_arrive(&raw_full[f]);
            ++raw_n;
            r = r + 1 == p.raws ? 0 : r + 1;
        };
        for (int f = 0; f * kFlushTiles < mine; ++f) {
            const int begin = f * kFlushTiles, end = min(mine, begin + kFlushTiles);
            if (RAW && warp == 17 && lane == 0) {
                for (int i = begin; i < end && ok; ++i) {
                    const long long m0 = pixel(i);
                    if constexpr (S::kDirectY) {
                        const int ys = i % S::kYStages, yn = i / S::kYStages;
                        if (yn > 0) ok = mbar_wait_bounded(&empty_y[ys], static_cast<unsigned>(yn - 1) & 1u, kCopyWaitLimitNs);
                        if (!ok) break;
                        mbar_expect_tx(&full_y[ys], ny * 16384u);
                        for (int b = 0; b < ny; ++b)
                            tc::tma_load_3d(sm + ys * ystage + b * 16384, &ymap, c0 + b * 64, static_cast<int>(m0), 0, &full_y[ys]);
                        mbar_arrive(&full_y[ys]);
                        y_n = i + 1;
                    } else {
                        for (int b = 0; b < ny && ok; ++b) {
                            const int col = c0 + b * 64;
                            load_raw(&ymap, col, 32, sizeof(T) == 4 && col + 32 < p.C ? 2 : 1, m0);
                        }
                    }
                    for (int ch = 0; ch < nch && ok; ++ch) {
                        const int col = g0 + ch * 64;
                        load_raw(&gmap, col, 32, col + 32 < p.NO ? 2 : 1, m0);
                    }
                }
            }
            if (warp == 16) {
                tc::fence_after();
                const uint32_t lead = tc::lead_lane();
                for (int i = begin; i < end && ok; ++i) {
                    const int ys = i % S::kYStages, t = i - begin;
                    ok = tc::warp_wait(&full_y[ys], static_cast<unsigned>(i / S::kYStages) & 1u, kCopyWaitLimitNs);
                    for (int ch = 0; ch < nch && ok; ++ch) {
                        const int n = i * nch + ch, s = n & 1;
                        ok = tc::warp_wait(&full_g[s], static_cast<unsigned>(n >> 1) & 1u, kCopyWaitLimitNs);
                        if (!ok) break;
                        tc::fence_after();
                        const uint32_t a = tc::sw128(smem_addr(sm + ys * ystage), second), b = tc::sw128(smem_addr(gsm + s * S::kG));
                        const uint32_t acc = tmem + ch * 64;
                        uint32_t high = acc;
#pragma unroll 1
                        for (int k = 0; k < 8; ++k) {
#pragma unroll
                            for (int gi = 0; gi < 3; ++gi)
#pragma unroll
                                for (int j = 0; j < YP; ++j) {
                                    if (gi + j > 2) continue;
                                    const uint32_t ad = a + j * (p.ystep / 16) + k * 128, bd = b + gi * 1024 + k * 128;
                                    const bool first_low = gi == (YP > 1 ? 0 : 1) && j == (YP > 1 ? 1 : 0);
                                    if (gi + j == 0) tc::mma_f16(high, ad, bd, idesc, t > 0 || k >= 3, lead);
                                    else tc::mma_f16(acc + 384, ad, bd, idesc, t > 0 || k > 0 || !first_low, lead);
                                }
                            high = high == acc + 256 ? acc : high + 128;
                        }
                        if (lead) tc::commit(&empty_g[s]);
                    }
                    if (ok && lead) tc::commit(&empty_y[ys]);
                }
                if (ok && lead) tc::commit(acc_full);
            }
            __syncwarp();
            ok = tc::bar_and(1, 128, ok && mbar_wait_bounded(acc_full, static_cast<unsigned>(f) & 1u, kFlushWaitLimitNs));
            if (!ok) break;
            tc::fence_after();
            const uint32_t acc = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
            for (int q = 0; q < nch * 4; ++q) {
                float v[16], w[16];
                tc::ld16(acc + 384 + q * 16, v);
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    tc::ld16(acc + k * 128 + q * 16, w);
                    tc::wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] += w[e];
                }
                const int s = g0 + q * 16;
                // rows in the gradient's order take divisions: one per lane, handed round
                const int mapped = p.direct ? slot_channel(min(s + (lane & 15), p.NO - 1), p.G, p.P) : 0;
                const size_t first = static_cast<size_t>(walker) * p.NO + s;
                size_t at[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int m = __shfl_sync(0xffffffffu, mapped, e);
                    at[e] = (p.direct ? static_cast<size_t>(m) : first + e) * p.C + c;
                }
                auto entry = [&](int e) -> float& { return part[at[e]]; };
                if (f > 0) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) w[e] = on && s + e < p.NO ? entry(e) : 0.f;
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] += w[e];
                }
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (on && s + e < p.NO) entry(e) = v[e];
            }
            tc::fence_before();
            tc::bar_sync(1, 128);
        }
    }
    if (!ok) atomicOr(p.status, kStatusCopyTimeout);
    tc::fence_before();
    if (!__syncthreads_and(ok)) {
        if (warp == 17 && lane == 0) {
            tc::drain_loads<4>(raw_full, raw_n, p.raws);
            tc::drain_loads<2>(full_y, y_n, 2);
        }
        if (warp == 16) tc::drain_products(drain);
        __syncthreads();
    }
    tc::fence_after();
    if (warp == 16) tc::dealloc(tmem, 512u);
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// All of it in one pass over g, for 16-bit y with at most 64 channels and 128
// slots: the planes of a tile of g serve both as grad_y's left operand (K-major,
// 64 slots at a time) and as the transposed grad_weight's (MN-major: 128 slots
// x 64 channels of sums), so that both sets of sums, three accumulators and the
// small terms' each, fill the tensor memory exactly. W's planes are laid out
// once per CTA. Warps 0..15 write the planes of g and sum it for the bias; a
// lane of warp 16 loads; warp 17 issues; warps 18..21 read grad_y's sums after
// every tile and grad_weight's every kFlushTiles. bf16 y is its own plane and
// comes by TMA; fp16's two planes of y and W leave no room for raw tiles of y
// nor for staging grad_y, so y comes through registers, a tile ahead, and
// grad_y leaves from them (65 slots or more: both groups of converters then
// have a chunk of every tile, and see every phase of y's one stage).
template <typename T>
struct GradBothShape {
    static constexpr int PL = split_planes<T>(), kRaws = 2, kYStages = PL == 1 ? 2 : 1;
    static constexpr unsigned kG = 3u * 16384u, kY = PL * 16384u, kW = PL * 16384u, kOut = PL == 1 ? 16384u : 0u;
    static constexpr unsigned kSmem = 1024u + 2 * kG + kYStages * kY + kW + kOut + kRaws * kRaw + 256u;
};

template <typename T, bool LONG>
__global__ void __launch_bounds__(kGradYThreads, 1)
pred_grad_both_kernel(const __grid_constant__ CUtensorMap gmap, const __grid_constant__ CUtensorMap ymap,
                      const __grid_constant__ CUtensorMap omap, const T* __restrict__ y, const T* __restrict__ w,
                      float* __restrict__ gy, float* __restrict__ part, float* __restrict__ pbias, PredBwdParams p) {
    using S = GradBothShape<T>;
    constexpr int PL = S::PL;
    extern __shared__ unsigned char pb_smem_raw[];
    unsigned char* gsm = pb_smem_raw + ((1024u - (smem_addr(pb_smem_raw) & 1023u)) & 1023u);
    unsigned char* ysm = gsm + 2 * S::kG;
    unsigned char* wsm = ysm + S::kYStages * S::kY;
    unsigned char* outs = wsm + S::kW;
    unsigned char* raws = outs + S::kOut;
    uint64_t* bars = reinterpret_cast<uint64_t*>(raws + S::kRaws * kRaw);
    uint64_t *full_g = bars, *empty_g = bars + 2, *full_y = bars + 4, *empty_y = bars + 6, *raw_full = bars + 8,
             *raw_empty = bars + 12, *full_w = bars + 16, *acc_full = bars + 17, *acc_empty = bars + 18,
             *sum_full = bars + 19, *sum_empty = bars + 20;  // raw tiles: step n's the (n mod 4)-th
    uint32_t* slot = reinterpret_cast<uint32_t*>(bars + 21);
    uint64_t* drain = bars + 22;
    const int tid = threadIdx.x, warp = static_cast<int>(tc::uniform(threadIdx.x >> 5)), lane = tid & 31;
    const int walker = static_cast<int>(blockIdx.x), nch = (p.NO + 63) / 64;
    const int mine = (p.tiles - walker + p.walkers - 1) / p.walkers, steps = mine * nch;
    auto pixel = [&](int i) { return (walker + i * p.walkers) * 128; };

    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&full_g[s], kGroup / 32);
            mbar_init(&empty_g[s], 1);
            mbar_init(&full_y[s], PL == 1 ? 1 : kConv / 32);
            mbar_init(&empty_y[s], 1);
        }
        for (int s = 0; s < 4; ++s) {
            mbar_init(&raw_full[s], 1);
            mbar_init(&raw_empty[s], kGroup / 32);
        }
        mbar_init(full_w, kConv / 32);
        mbar_init(acc_full, 1);
        mbar_init(acc_empty, 128);
        mbar_init(sum_full, 1);
        mbar_init(sum_empty, 128);
        mbar_init(drain, 1);
        fence_barrier_init();
    }
    if (warp == 16) tc::alloc(slot, 512u);
    tc::fence_before();
    __syncthreads();  // every CTA holds its tensor memory before the next launch may start
    tc::fence_after();
    const uint32_t tmem = tc::uniform(*slot);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    bool ok = true;
    int raw_n = 0, y_n = 0;  // the loading lane's raw tiles and tiles of y so far

    if (warp < 16) {
        // W's rows in record order, zeros past its end: row = slot, 16-byte chunk j at j ^ (row mod 8)
        for (int q = tid; q < nch * 512; q += kConv) {
            const int r = q >> 3, j = q & 7;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < p.NO && j * 8 < p.C)
                v = __ldg(reinterpret_cast<const uint4*>(w + static_cast<size_t>(slot_channel(r, p.G, p.P)) * p.C + j * 8));
            if constexpr (PL == 1) {
                *reinterpret_cast<uint4*>(wsm + r * 128 + ((j ^ (r & 7)) << 4)) = v;
            } else {
                float f[8];
                unpack8(v, static_cast<T*>(nullptr), f);
                store_split8<PL>(wsm, 16384u, r, j, f);
            }
        }
        hand_over(full_w, lane);
        // this group takes the chunks of its parity: with two a tile always the same one
        const int s = warp >> 3;
        const bool last = nch == 1 || s == 1;
        const ChunkWalk walk(last ? p.NO - (nch - 1) * 64 : 64, tid);
        using Sums = BiasSums<LONG>;
        Sums bs;
        // fp16 (always two chunks): y comes through registers, a tile ahead; this thread's pixel and 16 channels
        const int yrow = s * 64 + (tid % kGroup >> 2), yc = (tid & 3) * 16;
        uint4 yv[2];
        auto load_y = [&](int i) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int m = i < mine ? pixel(i) + yrow : p.M, c = yc + q * 8;
                yv[q] = m < p.M && c < p.C ? __ldg(reinterpret_cast<const uint4*>(y + static_cast<size_t>(m) * p.C + c))
                                           : make_uint4(0, 0, 0, 0);
            }
        };
        if constexpr (PL > 1) load_y(0);
        for (int begin = s; begin < steps && ok; begin += 2 * Sums::kRun) {
            for (int n = begin, end = min(steps, begin + 2 * Sums::kRun); n < end; n += 2) {
                ok = tc::warp_wait(&raw_full[n & 3], static_cast<unsigned>(n >> 2) & 1u, kCopyWaitLimitNs);
                if (!ok) break;
                Piece<float> piece;
                piece.from_raw(raws + s * kRaw, walk);
                piece.landed();
                if (lane == 0) mbar_arrive(&raw_empty[n & 3]);
                if (n >= 2) ok = tc::warp_wait(&empty_g[s], static_cast<unsigned>((n >> 1) - 1) & 1u, kCopyWaitLimitNs);
                if (!ok) break;
                piece.template store<3>(gsm + s * S::kG, 16384u, walk);
                hand_over(&full_g[s], lane);
                if constexpr (PL > 1) {
                    const int i = n >> 1;
                    if (i > 0) ok = tc::warp_wait(&empty_y[0], static_cast<unsigned>(i - 1) & 1u, kCopyWaitLimitNs);
                    if (!ok) break;
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        float f[8];
                        unpack8(yv[q], static_cast<T*>(nullptr), f);
                        store_split8<PL>(ysm, 16384u, yrow, (yc >> 3) + q, f);
                    }
                    hand_over(full_y, lane);
                    load_y(i + 1);
                }
                bs.add(piece.v);
            }
            if (begin + 2 * Sums::kRun < steps) bs.flush(begin == s);
        }
        if (pbias != nullptr) {
            // once the last products have read the operand tiles (a commit covers all those before it), the
            // threads' sums are added there, a slot's in the order of its rows' pieces
            const int end = (steps - 1) & 1;
            if (ok) ok = tc::warp_wait(&empty_g[end], static_cast<unsigned>((steps - 1) >> 1) & 1u, kCopyWaitLimitNs);
            float* red = reinterpret_cast<float*>(gsm);  // [thread][8]
            tc::bar_sync(2, kConv);
            if (ok) {
                if (s + 2 * Sums::kRun < steps) bs.finish();
#pragma unroll
                for (int k = 0; k < 8; ++k) red[tid * 8 + k] = bs.run[k];
            }
            tc::bar_sync(2, kConv);
            const int t = tid >> 3, part8 = tid & 7;
            for (int ch = 0; ch < nch; ++ch) {
                // eight threads per slot, every eighth of the slot's threads each, then the eight
                const ChunkWalk of(ch + 1 < nch ? 64 : p.NO - ch * 64, tid);
                const float* from = red + ch * kGroup * 8;
                float v = 0.f;
                if (t < of.ng * 8)
                    for (int r = part8; r < of.rows; r += 8) {
                        const float* at = from + (r * of.ng + (t >> 3)) * 8 + (t & 7);
                        v += nch == 1 ? at[0] + at[kGroup * 8] : at[0];
                    }
                v += __shfl_xor_sync(0xffffffffu, v, 1);
                v += __shfl_xor_sync(0xffffffffu, v, 2);
                v += __shfl_xor_sync(0xffffffffu, v, 4);
                if (ok && part8 == 0 && t < of.ng * 8 && ch * 64 + t < p.NO)
                    pbias[sum_row(p, walker, ch * 64 + t)] = v;
            }
        }
    } else if (warp == 16) {
        if (lane == 0) {
            for (int i = 0; i < mine && ok; ++i) {
                for (int ch = 0; ch < nch && ok; ++ch) {
                    const int n = i * nch + ch, f = n & 3, halves = ch * 64 + 32 < p.NO ? 2 : 1;
                    if (n >= S::kRaws)
                        ok = mbar_wait_bounded(&raw_empty[(n - S::kRaws) & 3], static_cast<unsigned>((n - S::kRaws) >> 2) & 1u,
                                               kCopyWaitLimitNs);
                    if (!ok) break;
                    mbar_expect_tx(&raw_full[f], halves * 16384u);
                    for (int h = 0; h < halves; ++h)
                        tc::tma_load_3d(raws + (n & 1) * kRaw + h * 16384, &gmap, ch * 64 + h * 32, pixel(i), 0, &raw_full[f]);
                    mbar_arrive(&raw_full[f]);
                    raw_n = n + 1;
                }
                if constexpr (PL > 1) continue;
                const int ys = i & 1;
                if (ok && i >= 2) ok = mbar_wait_bounded(&empty_y[ys], static_cast<unsigned>((i >> 1) - 1) & 1u, kCopyWaitLimitNs);
                if (!ok) break;
                mbar_expect_tx(&full_y[ys], S::kY);
                tc::tma_load_3d(ysm + ys * S::kY, &ymap, 0, pixel(i), 0, &full_y[ys]);
                mbar_arrive(&full_y[ys]);
                y_n = i + 1;
            }
        }
    } else if (warp == 17) {
        constexpr uint32_t iy = tc::idesc_f16(tc::kFmtBf16, 64, false, true), iw = tc::idesc_f16(tc::kFmtBf16, 64, true, true);
        const uint32_t lead = tc::lead_lane(), sums = tmem + 256u;
        ok = tc::warp_wait(full_w, 0u, kCopyWaitLimitNs);
        for (int i = 0; i < mine && ok; ++i) {
            const int ys = i % S::kYStages, t = i % kFlushTiles;
            // grad_y, as the chunks come
            if (i > 0) ok = tc::warp_wait(acc_empty, static_cast<unsigned>(i - 1) & 1u, kCopyWaitLimitNs);
            for (int ch = 0; ch < nch && ok; ++ch) {
                const int n = i * nch + ch, s = n & 1;
                ok = tc::warp_wait(&full_g[s], static_cast<unsigned>(n >> 1) & 1u, kCopyWaitLimitNs);
                if (!ok) break;
                tc::fence_after();
                const uint32_t a = tc::sw128(smem_addr(gsm + s * S::kG)), b = tc::sw128(smem_addr(wsm + ch * 8192));
                const int ksteps = (min(64, p.NO - ch * 64) + 15) / 16;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (k >= ksteps) break;
                    tc::mma_f16(tmem + (k % 3) * 64u, a + k * 2, b + k * 128, iy, ch > 0 || k >= 3, lead);
#pragma unroll
                    for (int q = 1; q < (PL == 1 ? 3 : 5); ++q) {  // (g's plane, W's): 1 0, 2 0, 0 1, 1 1
                        const int gi = q < 3 ? q : q - 3, wi = q < 3 ? 0 : 1;
                        tc::mma_f16(tmem + 192u, a + gi * 1024 + k * 2, b + wi * 1024 + k * 128, iy, ch > 0 || k > 0 || q > 1, lead);
                    }
                }
            }
            if (!ok) break;
            if (lead) tc::commit(acc_full);
            // grad_weight, both chunks (a single one stands in for the second, whose sums nobody reads)
            if (t == 0 && i > 0) ok = tc::warp_wait(sum_empty, static_cast<unsigned>(i / kFlushTiles - 1) & 1u, kCopyWaitLimitNs);
            ok = ok && tc::warp_wait(&full_y[ys], static_cast<unsigned>(i / S::kYStages) & 1u, kCopyWaitLimitNs);
            if (!ok) break;
            tc::fence_after();
            const int s0 = (i * nch) & 1;
            const uint32_t a = tc::sw128(smem_addr(gsm + s0 * S::kG), nch == 2 ? S::kG : 0u), b = tc::sw128(smem_addr(ysm + ys * S::kY));
            uint32_t high = sums;
#pragma unroll 1
            for (int k = 0; k < 8; ++k) {
                tc::mma_f16(high, a + k * 128, b + k * 128, iw, t > 0 || k >= 3, lead);
#pragma unroll
                for (int q = 1; q < (PL == 1 ? 3 : 5); ++q) {
                    const int gi = q < 3 ? q : q - 3, yi = q < 3 ? 0 : 1;
                    tc::mma_f16(sums + 192u, a + gi * 1024 + k * 128, b + yi * 1024 + k * 128, iw, t > 0 || k > 0 || q > 1, lead);
                }
                high = high == sums + 128 ? sums : high + 64;
            }
            if (lead) {
                for (int ch = 0; ch < nch; ++ch) tc::commit(&empty_g[(s0 + ch) & 1]);
                tc::commit(&empty_y[ys]);
                if (t == kFlushTiles - 1 || i == mine - 1) tc::commit(sum_full);
            }
        }
    } else {
        const int quarter = warp & 3, row = quarter * 32 + lane, et = tid - (kConv + 64);
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const int high = min(3, (min(64, p.NO) + 15) / 16);
        // three accumulators (as many of them as hold anything) and the small terms', 16 columns
        auto add4 = [&](uint32_t at, int count, float (&v)[16]) {
            float x[16];
            tc::ld16(at + 192u, v);
            for (int q = 0; q < count; ++q) {
                tc::ld16(at + q * 64u, x);
                tc::wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] += x[e];
            }
        };
        for (int i = 0; i < mine; ++i) {
            ok = tc::bar_and(1, 128, mbar_wait_bounded(acc_full, static_cast<unsigned>(i) & 1u, kCopyWaitLimitNs));
            if (!ok) break;
            tc::fence_after();
            if constexpr (PL > 1) {
                // no room for a staging tile: each lane writes its pixel's row
                const int m = pixel(i) + row;
                for (int c = 0; c < 64 && c < p.C; c += 16) {
                    float v[16];
                    add4(lanes + c, high, v);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (m < p.M && c + q * 4 < p.C)
                            *reinterpret_cast<float4*>(gy + static_cast<size_t>(m) * p.C + c + q * 4) =
                                make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                }
            } else {
                for (int h = 0; h < 2 && h * 32 < p.C; ++h) {
                    // the store that read the staging tile has done so
                    if (et == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                    tc::bar_sync(1, 128);
                    for (int cc = 0; cc < 2; ++cc) {
                        float v[16];
                        add4(lanes + h * 32 + cc * 16, high, v);
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            *reinterpret_cast<float4*>(outs + row * 128 + (((cc * 4 + q) ^ (row & 7)) << 4)) =
                                make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                    }
                    fence_proxy_async();
                    tc::bar_sync(1, 128);
                    if (et == 0) {
                        tc::tma_store_3d(&omap, h * 32, pixel(i), 0, outs);
                        tc::bulk_commit();
                    }
                }
            }
            tc::fence_before();
            mbar_arrive(acc_empty);
            if (i % kFlushTiles != kFlushTiles - 1 && i != mine - 1) continue;
            const int f = i / kFlushTiles;
            ok = tc::bar_and(1, 128, mbar_wait_bounded(sum_full, static_cast<unsigned>(f) & 1u, kFlushWaitLimitNs));
            if (!ok) break;
            tc::fence_after();
            float* o = part + (row < p.NO ? sum_row(p, walker, row) : 0u) * p.C;  // accumulator row = slot
            for (int q = 0; q < 4; ++q) {
                float v[16];
                add4(lanes + 256u + q * 16, 3, v);
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                    if (row < p.NO && q * 16 + e < p.C) {
                        float4* at = reinterpret_cast<float4*>(o + q * 16 + e);
                        float4 r = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                        if (f > 0) {
                            const float4 b = *at;
                            r = make_float4(r.x + b.x, r.y + b.y, r.z + b.z, r.w + b.w);
                        }
                        *at = r;
                    }
            }
            tc::fence_before();
            mbar_arrive(sum_empty);
        }
        if (et == 0) tc::bulk_wait_all();
    }
    if (!ok) atomicOr(p.status, kStatusCopyTimeout);
    tc::fence_before();
    if (!__syncthreads_and(ok)) {
        if (warp == 16 && lane == 0) {
            tc::drain_loads<4>(raw_full, raw_n, S::kRaws);
            tc::drain_loads<2>(full_y, y_n, 2);
        }
        if (warp == 17) tc::drain_products(drain);
        __syncthreads();
    }
    tc::fence_after();
    if (warp == 16) tc::dealloc(tmem, 512u);
}

// The walkers' partial sums added in a fixed order (sixteen strided runs of
// walkers, then the sixteen), rows moved from record order to the projection's
// channel order: 32 entries per CTA.
__global__ void __launch_bounds__(512)
pred_grad_w_join_kernel(const float* __restrict__ part, const float* __restrict__ pbias, float* __restrict__ gw,
                        float* __restrict__ gb, PredBwdParams p) {
    __shared__ float red[16][32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long n = static_cast<long long>(p.NO) * p.C, total = n + (gb ? p.NO : 0);
    const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
    for (long long i0 = static_cast<long long>(blockIdx.x) * 32; i0 < total; i0 += static_cast<long long>(gridDim.x) * 32) {
        const long long i = i0 + lane;
        float a = 0.f;
        if (i < total) {
            const float* src = i < n ? part + i : pbias + (i - n);
            const long long step = i < n ? n : p.NO;
#pragma unroll 8
            for (int k = run; k < p.walkers; k += 16) a += __ldg(src + k * step);
        }
        red[run][lane] = a;
        __syncthreads();
        if (run == 0 && i < total) {
            for (int k = 1; k < 16; ++k) a += red[k][lane];
            if (i < n) {
                const int s = static_cast<int>(i / p.C), c = static_cast<int>(i - static_cast<long long>(s) * p.C);
                gw[static_cast<size_t>(slot_channel(s, p.G, p.P)) * p.C + c] = a;
            } else {
                gb[slot_channel(static_cast<int>(i - n), p.G, p.P)] = a;
            }
        }
        __syncthreads();
    }
}

}  // namespace dcnv4
