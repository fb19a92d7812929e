// xent.cu -- softmax cross entropy over a vocabulary, straight from the hidden states: the logits
// l = H W^T exist only as accumulators in tensor memory and, in the backward pass, as one piece of
// the vocabulary's worth of bf16 gradients.
//   lse_n = log sum_v exp l_nv,  loss_n = lse_n - l_{n,t_n}
//   E_nv = (exp(l_nv - lse_n) - [v = t_n]) c_n,  dH = E W,  dW = E^T H
// Rows whose target is ignore_index are gathered away first (k_xent_rows): they cost no products, and
// whatever they hold, NaN included, meets no product.  The number of rows left stays on the device; the
// product kernels read it and skip what lies past it.
//
// One product kernel (k_product) in four roles, which differ in their operands' major axes and in
// what is done with the accumulators:
//   kStats  H W^T   -> per row and 128 columns the maximum and the sum of exponentials, and l_{n,t_n}
//   kGrad   H W^T   -> E (bf16), one piece of the vocabulary
//   kHidden E W     -> dH, summed in fp32 over the pieces
//   kWeight E^T H   -> dW of the piece, finished
// E is the one rounding to fewer bits before an output: its entries meet bf16 operands in the tensor
// cores, which want both operands of one type.  The gradients are then 2.0e-3 (2-norm) from 64 bits, where
// their own rounding to bf16 alone leaves 1.65e-3.
//
// Many rows: the tensor cores bound it, and their power limit once a sequence lasts.  4096 rows x 2048 x 32768
// words take 0.29 ms forward and 0.88 ms backward in bursts of 30 calls (a product 0.27-0.30 ms or 1.8-2.0
// PFLOP/s), 0.32 and 0.99 ms over two seconds; 8192 x 4096 x 131072 4.5 and 13.7 ms in bursts of four, 5.0 and
// 15.3 over two seconds.  Few rows: the weight's bytes.  16 x 4096 x 131072 (1.07 GB) takes 177 us forward
// (6.1 TB/s) and 563 us backward, where it is read twice and written once.
// Rows left out save the products of three roles in proportion; dH's tiles and the split of its K are laid out
// for all rows.  4096 x 2048 x 32768 with nine rows in ten ignored: 59 us forward, 268 backward; the 410 rows
// given alone: 55 and 171.
#include <algorithm>
#include <cstdio>

#include "internal.h"
#include "launch.cuh"
#include "tensor.cuh"

namespace lmo {
namespace {

constexpr int kTileN = 256;       // accumulator columns
constexpr int kTileK = 64;        // one 128-byte swizzle row of bf16
// kStats: blocks of K to an accumulator, 1024 products (see k_product).  2048 x 4096 x 32768: 299 us and a relative
// error of lse of 5.4e-7 (2-norm, hidden states that lean towards their targets' rows); 512 products 308 us and
// 2.6e-7, all 4096 298 us and 2.2e-6; elementary fp32 operations 4.0e-7.  Between 0.9 and 2.3 times as far off as
// those (300 x 1290 x 5000: 6.4e-7 against 2.8e-7); 512 products would stay within 1.25 times, for 2-8 % of the
// forward call and 0-1 % of both.
constexpr int kChunk = 16;
constexpr int kProductThreads = 384;   // warp 0 copies, warp 1 multiplies, warp 2 holds tensor memory, warps 4-11 finish
// Stages of 48 KiB (one CTA: 128 rows of A, 256 of B) or 32 KiB (a pair: 128 and 128 each).
__host__ __device__ constexpr int product_stages(int cta) { return cta == 1 ? 4 : 6; }
constexpr int kFinishBytes = 8 * 32 * 128;      // 32 rows of 128 bytes for each finishing warp (Stage)
constexpr uint32_t kTmemColumns = 512; // two accumulators of 256 columns
constexpr float kLog2e = 1.4426950408889634f;

enum { kStats = 0, kGrad = 1, kHidden = 2, kWeight = 3 };

// First words of the workspace.
struct XentHead {
    int32_t rows;      // rows with a target
    float grad_scale;  // backward: the largest |grad_loss|; E is in units of it (see k_xent_rows)
};

struct ProductArgs {
    const XentHead* head;
    int32_t m_tiles, n_tiles;   // tiles of the whole problem (rows: at most)
    int32_t k_blocks;           // K in blocks of 64 (kWeight: at most; the rows decide)
    int32_t splits;             // parts of K, each with its own output (kHidden)
    int32_t b_off;              // where the piece starts in B's map: first row (kStats, kGrad) or K row (kHidden)
    int32_t v_off;              // where it starts in the vocabulary
    int32_t vocab, dim;
    int64_t rows_pad;           // rows of the per-row arrays
    const int32_t* target;      // per gathered row
    const float* lse;           // kGrad
    const float* scale;         // kGrad
    float2* part;               // kStats: [tile][rows_pad]
    float* target_logit;        // kStats
    uint16_t* e;                // kGrad: [rows_pad][lde]
    int64_t lde;
    float* acc;                 // kHidden: [splits][rows_pad][ldacc]
    int64_t ldacc;
    int32_t first, last;        // kHidden: the first piece (nothing to add to), the last (dH itself; not if K is split)
    uint16_t* dh;               // kHidden
    int64_t lddh;
    int32_t dh_aligned;         // bytes that every row of dH starts on a multiple of: 16, 8, 4 or 2
    const int32_t* row_of;      // kHidden: gathered row -> row of dH
    uint16_t* dw;               // kWeight: dW, row b_off + m
    int64_t lddw;
    int32_t dw_aligned;         // kWeight: the same of dW
    uint64_t wait_ns;           // a wait's limit
    int32_t stall;              // tests of that limit: what the first cluster withholds (Stall), or 0
};
// One copying thread's blocks after the second (of the pair's first or second CTA), or the accumulators.
enum Stall { kStallCopy = 1, kStallPeer = 2, kStallFree = 3 };

// e^x for the softmax: the argument is a difference taken before the change of base.  (Subtracting base log2 e
// from x log2 e in one multiply-add saves an instruction, but rounds base log2 e: an error of the exponent
// that grows with the logits and overflows it past 2^40.)
__device__ __forceinline__ float exp_of(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * kLog2e));
    return y;
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// 16 bf16 values (8 words) to 32 bytes: a whole sector in one store.
__device__ __forceinline__ void store_32b(uint16_t* p, const uint32_t* r) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
                 "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// A finishing warp's corner of shared memory: a lane holds a row of the tile, but memory wants whole lines, so 32
// rows of 128 bytes are turned round in it -- each lane puts its row, then eight lanes take 16 bytes
// each of one row, four rows at a time.  The 16-byte pieces of row i lie at their number XOR i mod 8:
// neither side meets a bank twice.  dW of 16 rows x 4096 x 131072, all of it writing (1.07 GB), takes 235 us
// so; 32 bytes a lane written straight to memory keep L2 busy with single sectors: 283 us.
struct Stage {
    char* base;
    __device__ __forceinline__ void put(int lane, const uint32_t* w) const {   // 32 words
#pragma unroll
        for (int q = 0; q < 8; ++q)
            *reinterpret_cast<uint4*>(base + lane * 128 + ((q ^ (lane & 7)) << 4)) =
                make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    }
    __device__ __forceinline__ uint4 get(int row, int q) const {
        return *reinterpret_cast<const uint4*>(base + row * 128 + ((q ^ (row & 7)) << 4));
    }
    __device__ __forceinline__ uint32_t word(int row, int i) const {   // 32 bits
        return *reinterpret_cast<const uint32_t*>(base + row * 128 + (((i >> 2) ^ (row & 7)) << 4) + 4 * (i & 3));
    }
    __device__ __forceinline__ uint16_t half(int row, int i) const {   // 16 bits
        return *reinterpret_cast<const uint16_t*>(base + row * 128 + (((i >> 3) ^ (row & 7)) << 4) + 2 * (i & 7));
    }
};

// Loads one K block of an operand: `rows` rows of M or N from `mn`, 64 of K from `k`.
template <bool kMn, int kRows, int kCta>
__device__ __forceinline__ void load_operand(uint32_t dst, const CUtensorMap* map, int mn, int k, uint32_t bar) {
    if (!kMn) {
        tma_load<kCta>(dst, map, k, mn, bar);
    } else {
#pragma unroll
        for (int i = 0; i < kRows / 64; ++i) tma_load<kCta>(dst + i * 8192, map, mn + 64 * i, k, bar);
    }
}

// D = A B over tiles of 128 kCta x 256, one CTA (or a pair on one tile, kCta = 2) per SM, persistent.
// Roles by warp: TMA into a ring of stages; tcgen05.mma from them into one of two accumulators;
// eight warps -- a warp per 32 rows and half of the columns -- take the other accumulator out.
// The tensor cores cut the accumulator's low bits at each addition, always towards zero: over a
// long K that is a drift (products of one sign, K = 4096: lse 1.2e-5 low, 1.8e-6 as it is), which the loss
// would show.  kStats therefore starts a new accumulator every kChunk blocks of K and adds them up
// in registers, rounded to nearest; the other accumulator hides the extra reading of tensor memory.
// Every wait is bounded (mbar_wait); one that runs out raises gave_up in all CTAs of the cluster and each role
// stops at its next wait.  A tile is finished only behind its own products' completion (nothing else
// arrives on the done barriers); the finishing warps write NaN for what they did not get.  When every
// role has stopped, copies and products in flight are waited for, bounded too, and the kernel returns
// with tensor memory freed.
template <int kMode, int kCta>
__global__ void __launch_bounds__(kProductThreads, 1) k_product(const __grid_constant__ CUtensorMap map_a,
                                                                const __grid_constant__ CUtensorMap map_b,
                                                                const ProductArgs p) {
    constexpr bool kAMn = kMode == kWeight, kBMn = kMode == kHidden || kMode == kWeight;
    constexpr int kStages = product_stages(kCta);
    constexpr int kRowsB = kTileN / kCta;
    constexpr uint32_t kBytesA = 128 * kTileK * 2, kBytesB = kRowsB * kTileK * 2, kStage = kBytesA + kBytesB;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bars[2 * kStages + 5];
    __shared__ uint32_t tmem_base;
    __shared__ int gave_up;
    __shared__ int copied;   // blocks of K that this CTA's copying thread has issued, when it has stopped
    const uint32_t tiles = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * kStages, done0 = empty0 + 8 * kStages, free0 = done0 + 16;
    const uint32_t drained = free0 + 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = kCta == 2 ? cluster_rank() : 0u;
    if (threadIdx.x == 0) {
        gave_up = 0;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full0 + 8 * i, 1);
            mbar_init(empty0 + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(done0 + 8 * i, 1);
            mbar_init(free0 + 8 * i, 8 * kCta);
        }
        mbar_init(drained, 1);
        mbar_init_fence();
        tma_prefetch_map(&map_a);
        tma_prefetch_map(&map_b);
    }
    if (warp == 2) tmem_alloc<kCta>(smem_u32(&tmem_base), kTmemColumns);
    tc_fence_before();
    __syncthreads();
    if (kCta == 2) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    auto wait = [&](uint32_t bar, uint32_t parity) { return mbar_wait<kCta>(bar, parity, &gave_up, p.wait_ns); };
    pdl_sync();

    const int rows = p.head->rows;
    const int m_tiles = kMode == kWeight ? p.m_tiles : (rows + 128 * kCta - 1) / (128 * kCta);
    const int k_blocks = kMode == kWeight ? (rows + kTileK - 1) / kTileK : p.k_blocks;
    const int per_split = (k_blocks + p.splits - 1) / p.splits;
    const int units = m_tiles * p.n_tiles * p.splits;
    const int first_unit = (int)blockIdx.x / kCta, stride = (int)gridDim.x / kCta;
    // unit -> split, then tiles in strips of 8 columns, rows of tiles within a strip: the units in
    // flight at one time share their rows of A and columns of B in L2
    auto unit_tile = [&](int u, int& m, int& n, int& k0, int& k1, int& split) {
        split = 0;
        if (p.splits > 1) {
            const int per = m_tiles * p.n_tiles;
            split = u / per;
            u -= split * per;
        }
        const int strip = u / (m_tiles * 8), in = u - strip * m_tiles * 8;
        const int width = min(8, p.n_tiles - strip * 8);
        m = width == 8 ? in >> 3 : in / width;
        n = strip * 8 + in - m * width;
        k0 = min(k_blocks, split * per_split);
        k1 = min(k_blocks, k0 + per_split);
    };
    // blocks of K that share an accumulator
    auto chunk_end = [&](int k, int k1) { return kMode == kStats ? min(k1, k + kChunk) : k1; };

    if (warp < 4) {
        if (kMode == kStats) regs_down<40>();
        if (warp == 0 && elect_lane()) {
            const int stop = first_unit == 0 && p.stall == kStallCopy + (int)rank ? 2 : 0x7FFFFFFF;
            int stage = 0;
            uint32_t phase = 0;
            int issued = 0;
            bool ok = true;
            for (int u = first_unit; ok && u < units; u += stride) {
                int m, n, k0, k1, split;
                unit_tile(u, m, n, k0, k1, split);
                const int am = (m * kCta + (int)rank) * 128, bn = n * kTileN + (int)rank * kRowsB;
                for (int kb = k0; kb < k1; ++kb) {
                    ok = issued != stop && wait(empty0 + 8 * stage, phase ^ 1u);
                    if (!ok) break;
                    const uint32_t bar = kCta == 2 ? cluster_addr(full0 + 8 * stage, 0) : full0 + 8 * stage;
                    if (rank == 0) mbar_expect_tx(full0 + 8 * stage, kStage * kCta);
                    const uint32_t a = tiles + stage * kStage, b = a + kBytesA;
                    load_operand<kAMn, 128, kCta>(a, &map_a, am, kb * kTileK, bar);
                    if (kMode == kHidden)
                        load_operand<kBMn, kRowsB, kCta>(b, &map_b, bn, p.b_off + kb * kTileK, bar);
                    else
                        load_operand<kBMn, kRowsB, kCta>(b, &map_b, bn + (kMode == kWeight ? 0 : p.b_off), kb * kTileK, bar);
                    ++issued;
                    if (++stage == kStages) stage = 0, phase ^= 1u;
                }
            }
            // the last stages come back before the CTA ends: nothing arrives on its barriers after that
            for (int i = max(0, issued - kStages); ok && i < issued; ++i)
                ok = wait(empty0 + 8 * (i % kStages), i / kStages & 1);
            copied = issued;
        } else if (warp == 1 && rank == 0 && elect_lane()) {
            constexpr uint32_t idesc = mma_desc(128 * kCta, kTileN, kAMn, kBMn);
            constexpr uint32_t step_a = kAMn ? 2048u : 32u, step_b = kBMn ? 2048u : 32u;
            int stage = 0, buf = 0;
            uint32_t phase = 0, buf_phase = 0;
            bool ok = true;
            for (int u = first_unit; ok && u < units; u += stride) {
                int m, n, k0, k1, split;
                unit_tile(u, m, n, k0, k1, split);
                int k = k0;
                do {
                    const int end = chunk_end(k, k1);
                    ok = wait(free0 + 8 * buf, buf_phase ^ 1u);
                    if (!ok) break;
                    tc_fence_after();
                    for (int kb = k; kb < end; ++kb) {
                        ok = wait(full0 + 8 * stage, phase);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t a = tiles + stage * kStage, b = a + kBytesA;
#pragma unroll
                        for (int j = 0; j < kTileK / 16; ++j)
                            mma_bf16<kCta>(tmem + buf * kTileN, operand_desc(a + j * step_a, 8192, 1024),
                                           operand_desc(b + j * step_b, 8192, 1024), idesc, kb > k || j > 0);
                        mma_commit<kCta>(empty0 + 8 * stage);
                        if (++stage == kStages) stage = 0, phase ^= 1u;
                    }
                    if (!ok) break;
                    mma_commit<kCta>(done0 + 8 * buf);
                    if (++buf == 2) buf = 0, buf_phase ^= 1u;
                    k = end;
                } while (k < k1);
            }
        }
        __syncwarp();
    } else {
        if (kMode == kStats) regs_up<232>();
        const int w = warp & 3, half = (warp >> 2) - 1;   // tensor memory lanes are dealt to warps by warp % 4
        const uint32_t lanes = (uint32_t)(32 * w) << 16;
        const Stage stage{reinterpret_cast<char*>(smem_raw) + (tiles - smem_u32(smem_raw)) + kStages * kStage + (warp - 4) * 32 * 128};
        int buf = 0;
        uint32_t buf_phase = 0;
        bool ok = true;
        auto wait_done = [&]() {
            if (ok) ok = wait(done0 + 8 * buf, buf_phase);
            ok = __all_sync(0xFFFFFFFFu, ok);
            tc_fence_after();
        };
        // Hands the accumulator back.  The arrival waits for the thread's stores to be seen (by the pair, in L2,
        // if there is one), so it comes before a tile's last stores, not behind them (16 x 4096 x 131072:
        // backward 664 us behind them, 573 before).
        auto release = [&]() {
            tc_fence_before();
            __syncwarp();
            if (lane == 0 && ok && !(p.stall == kStallFree && blockIdx.x < kCta)) {
                if (kCta == 2) mbar_arrive_cluster(cluster_addr(free0 + 8 * buf, 0));
                else mbar_arrive(free0 + 8 * buf);
            }
            if (++buf == 2) buf = 0, buf_phase ^= 1u;
        };
        constexpr float kNan = __builtin_nanf("");
        for (int u = first_unit; u < units; u += stride) {
            int m, n, k0, k1, split;
            unit_tile(u, m, n, k0, k1, split);
            const int row = (m * kCta + (int)rank) * 128 + 32 * w + lane;   // this thread's row of the tile
            const int c0 = n * kTileN + half * 128;                         // and its first of 128 columns
            if (kMode == kStats) {
                float x[128];
                int k = k0;
                do {
                    wait_done();
#pragma unroll
                    for (int c = 0; c < 128; c += 32) {
                        uint32_t r[32];
                        tmem_load32(tmem + buf * kTileN + lanes + half * 128 + c, r);
                        tmem_wait(r);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            x[c + j] = k == k0 ? __uint_as_float(r[j]) : x[c + j] + __uint_as_float(r[j]);
                    }
                    release();
                    k = chunk_end(k, k1);
                } while (k < k1);
                const int left = p.vocab - (p.v_off + c0);
                const int t = row < rows ? p.target[row] - (p.v_off + c0) : -1;
                float top = -INFINITY, sum = 0.0f;
#pragma unroll
                for (int j = 0; j < 128; ++j) {
                    if (j >= left) x[j] = -INFINITY;
                    top = fmaxf(top, x[j]);
                }
                const float base = top == -INFINITY ? 0.0f : top;
                if (t >= 0 && t < 128) {
                    float l = 0.0f;
#pragma unroll
                    for (int j = 0; j < 128; ++j) l = t == j ? x[j] : l;
                    p.target_logit[row] = l;
                }
#pragma unroll
                for (int j = 0; j < 128; ++j) sum += exp_of(x[j] - base);
                if (row < rows) p.part[(int64_t)((p.v_off + c0) / 128) * p.rows_pad + row] = make_float2(top, ok ? sum : kNan);
                __syncwarp();
                continue;
            }
            wait_done();
            const uint32_t acc = tmem + buf * kTileN + lanes + half * 128;
            const bool none = k0 == k1;                                     // no products: the tile is zero
            if (kMode == kGrad) {
                const bool live = row < rows;
                const int t = live ? p.target[row] - p.v_off - c0 : -1;     // the target's column of this half
                const float g = live ? (ok ? p.scale[row] : kNan) : 0.0f;
                const float base = live ? p.lse[row] : 0.0f;
                uint16_t* const out = p.e + row * p.lde + c0;
#pragma unroll 1
                for (int c = 0; c < 128; c += 32) {
                    uint32_t r[32];
                    tmem_load32(acc + c, r);
                    tmem_wait(r);
                    const int left = p.vocab - (p.v_off + c0 + c);
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        float x = exp_of(__uint_as_float(r[j]) - base);
                        if (t == c + j) x -= 1.0f;
                        // rows past the last and columns past the vocabulary are zero, whatever was multiplied
                        r[j] = __float_as_uint(live && j < left ? x * g : 0.0f);
                    }
#pragma unroll
                    for (int j = 0; j < 32; j += 2) r[j / 2] = bf16_pair(__uint_as_float(r[j]), __uint_as_float(r[j + 1]));
                    if (c == 96) release();   // before the last stores: see release
                    store_32b(out + c, r);
                    store_32b(out + c + 16, r + 8);
                }
                continue;
            }
            const float g = p.head->grad_scale;
            if (kMode == kHidden) {
                // fp32, in the order of the pieces: one launch per piece, one lane per element
                const int64_t to_row = row < rows && p.last ? p.row_of[row] : -1;   // of dH
                const int first_row = row - lane, q = lane & 7;
                float* const part = p.acc + ((int64_t)split * p.rows_pad + first_row) * p.ldacc + c0 + 4 * q;
#pragma unroll 1
                for (int c = 0; c < 128; c += 32) {
                    if (c0 + c >= p.dim) break;
                    uint32_t r[32];
                    tmem_load32(acc + c, r);
                    tmem_wait(r);
                    if (none || !ok) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) r[j] = ok ? 0u : 0x7FC00000u;
                    }
                    stage.put(lane, r);
                    __syncwarp();
#pragma unroll 4
                    for (int i = lane >> 3; i < 32; i += 4) {
                        const int64_t to = __shfl_sync(0xFFFFFFFFu, to_row, i);
                        if (first_row + i >= rows) continue;
                        const uint4 v = stage.get(i, q);
                        float4 x = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
                        float4* const sum = reinterpret_cast<float4*>(part + i * p.ldacc + c);
                        if (!p.first) {
                            const float4 y = *sum;
                            x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
                        }
                        if (!p.last) {
                            *sum = x;
                            continue;
                        }
                        uint16_t* const o = p.dh + to * p.lddh + c0 + c + 4 * q;
                        const uint2 y = make_uint2(bf16_pair(x.x * g, x.y * g), bf16_pair(x.z * g, x.w * g));
                        const int left = p.dim - (c0 + c + 4 * q);
                        if (p.dh_aligned >= 8 && left >= 4) {
                            *reinterpret_cast<uint2*>(o) = y;
                        } else {
                            const uint16_t h[4] = {(uint16_t)y.x, (uint16_t)(y.x >> 16), (uint16_t)y.y, (uint16_t)(y.y >> 16)};
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (j < left) o[j] = h[j];
                        }
                    }
                    __syncwarp();
                }
                release();
                continue;
            }
            const int first_v = p.v_off + row - lane;   // of the warp's 32 rows of dW
            uint16_t* const out = p.dw + first_v * p.lddw + c0;
            const int have = min(32, p.vocab - first_v);
            auto take = [&](int c, uint32_t* o) {       // 64 columns
#pragma unroll
                for (int h = 0; h < 64; h += 32) {
                    uint32_t r[32];
                    tmem_load32(acc + c + h, r);
                    tmem_wait(r);
#pragma unroll
                    for (int j = 0; j < 32; j += 2)
                        o[(h + j) / 2] = bf16_pair(__uint_as_float(r[j]) * g, __uint_as_float(r[j + 1]) * g);
                }
                if (none || !ok) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = ok ? 0u : 0x7FC07FC0u;
                }
            };
            auto write = [&](int c, const uint32_t* o) {
                const int left = p.dim - (c0 + c);
                if (left <= 0) return;
                stage.put(lane, o);
                __syncwarp();
                if (p.dw_aligned == 16 && left >= 64) {
#pragma unroll
                    for (int i = lane >> 3; i < 32; i += 4)
                        if (i < have) *reinterpret_cast<uint4*>(out + i * p.lddw + c + 8 * (lane & 7)) = stage.get(i, lane & 7);
                } else if (p.dw_aligned >= 4) {        // a row at a time, two elements a lane
                    const int l = 2 * lane;
#pragma unroll 4
                    for (int i = 0; i < have; ++i) {
                        const uint32_t x = stage.word(i, lane);
                        uint16_t* const at = out + i * p.lddw + c + l;
                        if (l + 1 < left) *reinterpret_cast<uint32_t*>(at) = x;
                        else if (l < left) *at = (uint16_t)x;
                    }
                } else {
#pragma unroll 4
                    for (int i = 0; i < have; ++i) {
                        uint16_t* const at = out + i * p.lddw + c + lane;
                        if (lane < left) at[0] = stage.half(i, lane);
                        if (lane + 32 < left) at[32] = stage.half(i, lane + 32);
                    }
                }
                __syncwarp();
            };
#pragma unroll 1
            for (int c = 0; c < 128; c += 64) {
                uint32_t o[32];
                take(c, o);
                if (c == 64) release();   // before the last stores: see release
                write(c, o);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (kCta == 2) cluster_sync();
    // every role of the cluster has stopped: the flag is the same for all of its threads
    if (*static_cast<volatile int*>(&gave_up)) {
        const bool leader = kCta == 1 || cluster_rank() == 0u;   // read again: a register less over the loops above
        if (warp == 0 && elect_lane() && leader) {
            // Both CTAs' copies are counted on the first one's barriers; their threads may have stopped at different blocks.
            const int mine = copied, other = kCta == 2 ? load_cluster(cluster_addr(smem_u32(&copied), 1)) : mine;
            const int most = max(mine, other);
            for (int i = max(0, most - kStages); i < most; ++i) {   // blocks before these have been multiplied
                const uint32_t bar = full0 + 8 * (i % kStages);
                if (i >= mine) mbar_expect_tx(bar, kStage);            // the other's half alone
                else if (i >= other) mbar_complete_tx(bar, kStage);    // the other's half will not come
                mbar_drain(bar, i / kStages & 1);
            }
        } else if (warp == 1 && elect_lane()) {   // the thread that multiplied, and in the other CTA the one that would
            if (leader) mma_commit<kCta>(drained);
            mbar_drain(drained, 0);
        }
        __syncthreads();
        if (kCta == 2) cluster_sync();
    }
    tc_fence_after();
    if (warp == 2) tmem_free<kCta>(tmem, kTmemColumns);
}

// ---- rows -------------------------------------------------------------------------------------
// Eight consecutive elements from any address of 16-bit elements, in the widest loads it allows.
__device__ __forceinline__ uint4 load8_any(const uint16_t* p) {
    if (aligned16(p)) return *reinterpret_cast<const uint4*>(p);
    if ((reinterpret_cast<uintptr_t>(p) & 3u) == 0u) {
        const uint32_t* q = reinterpret_cast<const uint32_t*>(p);
        return make_uint4(q[0], q[1], q[2], q[3]);
    }
    const uint32_t* q = reinterpret_cast<const uint32_t*>(p + 1);
    const uint32_t a = p[0], b = q[0], c = q[1], d = q[2], e = p[7];
    return make_uint4(a | (b << 16), __funnelshift_l(b, c, 16), __funnelshift_l(c, d, 16), (d >> 16) | (e << 16));
}
// Elements i..i+7 of a row of `dim`, zero past its end.
__device__ __forceinline__ uint4 load_row8(const uint16_t* row, int i, int dim) {
    if (i + 8 <= dim) return load8_any(row + i);
    uint32_t h[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = i + j < dim ? row[i + j] : 0u;
    return make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16));
}

struct RowArgs {
    const int64_t* target;
    int64_t rows, ignore;
    int32_t vocab, dim;
    const uint16_t* hidden;
    int64_t ldh;
    bool vec;               // every row of hidden is whole 16-byte vectors
    int64_t per_cta;        // rows to a CTA
    XentHead* head;
    uint16_t* hc;           // gathered rows, ldhc elements apart
    int64_t ldhc;
    int32_t* row_of;        // gathered row -> row
    int32_t* pos_of;        // backward: row -> gathered row, or -1
    int32_t* target_of;     // per gathered row; -1 for a target outside the vocabulary
    float* loss;            // forward: outputs, zeroed for rows without a target
    float* lse;
    const float* lse_in;    // backward
    const float* grad;
    float* lse_of;
    float* scale_of;
    uint16_t* dh;           // backward: zeroed for rows left out (NULL: not written)
    int64_t lddh;
};

// Gathers the rows that count, in their order: tables per gathered row, and the rows themselves side by
// side.  Each CTA takes a run of rows and first counts, over all targets, how many rows before it
// count (every CTA reads every target: 8 or 12 bytes a row out of L2, less than a launch between a
// scan and a copy would take until the rows are hundreds of thousands).  16 rows of 2048: 4-5 us;
// 4096: 14 us for 34 MB.
// Backward: rows whose grad_loss is zero are left out too.  E is formed in units of the largest
// |grad_loss|, which the gradients are multiplied with in fp32 at the end: with equal grad_loss
// (a mean) E's largest entries are then near -1, where bf16 is at its finest, whatever the mean's
// divisor rounds to.
__global__ void __launch_bounds__(kThreads) k_xent_rows(const RowArgs a) {
    __shared__ int before_s, total_s;
    __shared__ uint32_t top_s;
    __shared__ int warp_count[kThreads / 32 + 1];
    __shared__ int list_src[kThreads], list_pos[kThreads];
    pdl_sync();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) before_s = total_s = 0, top_s = 0u;
    __syncthreads();
    const int64_t start = (int64_t)blockIdx.x * a.per_cta, end = min(a.rows, start + a.per_cta);
    int before = 0, total = 0;
    uint32_t top = 0u;   // of the finite ones: a NaN or an infinity stays in its row
#pragma unroll 4
    for (int64_t n = threadIdx.x; n < a.rows; n += kThreads) {
        bool counts = a.target[n] != a.ignore;
        if (a.grad) {
            const uint32_t b = __float_as_uint(a.grad[n]) & 0x7FFFFFFFu;
            counts = counts && b != 0u;
            if (counts && b < 0x7F800000u) top = max(top, b);
        }
        total += counts;
        before += counts && n < start;
    }
    before = __reduce_add_sync(0xFFFFFFFFu, before);
    total = __reduce_add_sync(0xFFFFFFFFu, total);
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if (lane == 0) {
        atomicAdd(&before_s, before);
        atomicAdd(&total_s, total);
        atomicMax(&top_s, top);
    }
    __syncthreads();
    total = total_s;
    const float unit = top_s != 0u ? __uint_as_float(top_s) : 1.0f;
    int base = before_s;
    const int vecs = (int)(a.ldhc / 8);
    for (int64_t n0 = start; n0 < end; n0 += kThreads) {
        const int64_t n = n0 + threadIdx.x;
        const int64_t t = n < end ? a.target[n] : a.ignore;
        const float g = a.grad && n < end ? a.grad[n] : 1.0f;
        const bool counts = t != a.ignore && g != 0.0f;
        const unsigned votes = __ballot_sync(0xFFFFFFFFu, counts);
        if (lane == 0) warp_count[warp] = __popc(votes);
        __syncthreads();
        int pos = 0, here = 0;
        for (int i = 0; i < kThreads / 32; ++i) {
            pos += i < warp ? warp_count[i] : 0;
            here += warp_count[i];
        }
        pos += __popc(votes & ((1u << lane) - 1u));
        if (counts) {
            const bool in = t >= 0 && t < a.vocab;
            const int to = base + pos;
            list_src[pos] = (int)(n - n0);
            list_pos[pos] = to;
            a.row_of[to] = (int32_t)n;
            a.target_of[to] = in ? (int32_t)t : -1;
            if (a.grad) {
                a.pos_of[n] = to;
                a.lse_of[to] = a.lse_in[n];
                a.scale_of[to] = in ? g / unit : __int_as_float(0x7FC00000);
            }
        } else if (n < end) {
            if (a.grad) a.pos_of[n] = -1;
            else a.loss[n] = a.lse[n] = 0.0f;
        }
        __syncthreads();
        if (a.vec) {
            const int all = here * vecs;   // at most 256 rows of vectors
#pragma unroll 4
            for (int i = threadIdx.x; i < all; i += kThreads) {
                const int k = i / vecs, c = (i - k * vecs) * 8;
                *reinterpret_cast<uint4*>(a.hc + (int64_t)list_pos[k] * a.ldhc + c) =
                    *reinterpret_cast<const uint4*>(a.hidden + (n0 + list_src[k]) * a.ldh + c);
            }
        } else {
            for (int64_t i = threadIdx.x; i < (int64_t)here * vecs; i += kThreads) {
                const int k = (int)(i / vecs), c = (int)(i - (int64_t)k * vecs) * 8;
                *reinterpret_cast<uint4*>(a.hc + (int64_t)list_pos[k] * a.ldhc + c) =
                    load_row8(a.hidden + (n0 + list_src[k]) * a.ldh, c, a.dim);
            }
        }
        if (a.dh && here < (int)min((int64_t)kThreads, end - n0)) {
            for (int64_t m = n0; m < min(end, n0 + kThreads); ++m) {
                const bool out = a.target[m] == a.ignore || a.grad[m] == 0.0f;
                if (out)
                    for (int c = threadIdx.x; c < a.dim; c += kThreads) a.dh[m * a.lddh + c] = 0;
            }
        }
        base += here;
        __syncthreads();
    }
    // backward: the rows' last block of K is filled up with zeros (E is zero there, which NaN would not heed)
    if (a.grad) {
        const int fill = (total + kTileK - 1) / kTileK * kTileK;
        for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < (int64_t)(fill - total) * vecs;
             i += (int64_t)gridDim.x * kThreads)
            *reinterpret_cast<uint4*>(a.hc + (int64_t)total * a.ldhc + 8 * i) = make_uint4(0, 0, 0, 0);
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        a.head->rows = total;
        a.head->grad_scale = unit;
    }
}

// Rows of the weight that TMA cannot address (16-byte steps) copied side by side.  The first piece is copied
// beside the gathering of the rows, which has nothing to do with it; later ones wait for the
// products that read the piece before.  50021 x 1290: 38 us, 6.8 TB/s read and written.  (Pieces of 24 to
// 96 MiB, which would stay in L2, cost more in launches than they save: forward with 1024 rows 144-161
// against 139 us.)
__global__ void __launch_bounds__(kThreads) k_xent_pack(const uint16_t* __restrict__ src, int64_t lds, uint16_t* __restrict__ dst,
                                                        int64_t ldd, int64_t rows, int dim, bool first) {
    if (!first) pdl_sync();
    const int vecs = (int)(ldd / 8);
    const int64_t n = rows * vecs, step = (int64_t)gridDim.x * kThreads;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += step) {
        const int64_t row = i / vecs;
        *reinterpret_cast<uint4*>(dst + 8 * i) = load_row8(src + row * lds, (int)(i - row * vecs) * 8, dim);
    }
    if (first) pdl_sync();
}

// Joins a row's (maximum, sum) pairs of all 128-word tiles, kRows rows a CTA: a thread its share of the tiles, then
// the lanes of a warp, then the warps, in a fixed order.  Latency bounds it: one row a CTA while
// there are few (256 tiles: 16 rows 5.0 us against 6.0 with eight, 304 rows 5.8 against 6.2, 1024 rows
// 8.5 against 6.2).
template <int kRows>
__global__ void __launch_bounds__(kThreads) k_xent_loss(const XentHead* head, const float2* __restrict__ part, int tiles,
                                                        int64_t rows_pad, const float* __restrict__ target_logit,
                                                        const int32_t* __restrict__ target, const int32_t* __restrict__ row_of,
                                                        float* __restrict__ loss, float* __restrict__ lse) {
    constexpr int kLanes = kThreads / kRows;
    __shared__ float2 red[kThreads / 32][kRows];
    pdl_sync();
    const int tx = threadIdx.x % kRows, ty = threadIdx.x / kRows;
    const int rows = head->rows;
    auto join = [](float2 a, float2 b) {
        const float m = fmaxf(a.x, b.x);
        if (m == -INFINITY) return make_float2(m, a.y + b.y);
        return make_float2(m, a.y * expf(a.x - m) + b.y * expf(b.x - m));
    };
    for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < rows; r0 += (int64_t)gridDim.x * kRows) {
        const int64_t c = r0 + tx;
        float2 s = make_float2(-INFINITY, 0.0f);
        if (c < rows) {
            for (int k = ty; k < tiles; k += 4 * kLanes) {   // four loads at a time
                float2 q[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    q[i] = k + kLanes * i < tiles ? part[(k + kLanes * i) * rows_pad + c] : make_float2(-INFINITY, 0.0f);
#pragma unroll
                for (int i = 0; i < 4; ++i) s = join(s, q[i]);
            }
        }
#pragma unroll
        for (int o = kRows; o < 32; o <<= 1)
            s = join(s, make_float2(__shfl_xor_sync(0xFFFFFFFFu, s.x, o), __shfl_xor_sync(0xFFFFFFFFu, s.y, o)));
        if ((threadIdx.x & 31) < kRows) red[threadIdx.x >> 5][tx] = s;
        __syncthreads();
        if (threadIdx.x < kRows && c < rows) {
            for (int k = 1; k < kThreads / 32; ++k) s = join(s, red[k][tx]);
            const float l = s.x + logf(s.y);
            const int64_t n = row_of[c];
            lse[n] = l;
            loss[n] = target[c] < 0 ? __int_as_float(0x7FC00000) : l - target_logit[c];
        }
        __syncthreads();
    }
}

// dH rows from the fp32 parts of a split K; zero for rows left out.  A CTA takes 128 columns of a row, 32 lanes
// four each, its eight warps every eighth part; then the warps' sums in order (16 rows x 4096, nine
// parts: 4.2 us; 1024 x 2048, two parts: 20 us).
__global__ void __launch_bounds__(kThreads) k_xent_hidden(const XentHead* head, const int32_t* __restrict__ pos_of,
                                                          const float* __restrict__ acc, int splits, int64_t rows_pad,
                                                          int64_t ldacc, uint16_t* __restrict__ dh, int64_t lddh, int dim,
                                                          bool vec) {
    __shared__ float4 red[kThreads / 32][32];
    pdl_sync();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t n = blockIdx.x, c = pos_of[n];
    const int i = blockIdx.y * 128 + 4 * lane;
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (c >= 0 && i < dim) {
#pragma unroll 8
        for (int s = warp; s < splits; s += kThreads / 32) {
            const float4 y = *reinterpret_cast<const float4*>(acc + ((int64_t)s * rows_pad + c) * ldacc + i);
            x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
        }
    }
    red[warp][lane] = x;
    __syncthreads();
    if (warp != 0 || i >= dim) return;
    for (int k = 1; k < kThreads / 32; ++k) {
        const float4 y = red[k][lane];
        x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
    }
    const float g = head->grad_scale;
    uint16_t* const o = dh + n * lddh + i;
    const uint32_t lo = bf16_pair(x.x * g, x.y * g), hi = bf16_pair(x.z * g, x.w * g);
    if (vec && i + 4 <= dim) {
        *reinterpret_cast<uint2*>(o) = make_uint2(lo, hi);
    } else {
        const uint16_t h[4] = {(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi, (uint16_t)(hi >> 16)};
        for (int j = 0; j < 4 && i + j < dim; ++j) o[j] = h[j];
    }
}

// ---- host -------------------------------------------------------------------------------------
int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

int row_alignment(const void* p, int64_t ld) {
    for (int a : {16, 8, 4})
        if (is_aligned(p, a) && ld % (a / 2) == 0) return a;
    return 2;
}

// Sizes and workspace layout of a call.
struct XentPlan {
    int64_t rows, dim, vocab;
    bool pack_w;                // the weight's rows cannot be addressed by TMA: copied piece by piece
    int cta;                    // CTAs on a tile
    int64_t rows_pad, ldh, piece, ldacc;   // ldh: of the gathered rows and a copied weight
    int splits;
    size_t row_of, pos_of, target_of, lse_of, scale_of, target_logit, hc, wc, part, e, acc, bytes;
};

// How much of the vocabulary's gradient exists at a time (bytes of E, of a copied piece of the weight).  Each
// piece costs three launches with their ramps; backward with 64, 128, 256, 512 MiB: 4096 x 2048 x 32768 894, 871,
// 870, 870 us in bursts, 8192 x 4096 x 131072 16.9, 16.0, 15.4, 15.1 ms under the power limit.
constexpr int64_t kPieceBytes = 256ll << 20;
constexpr int64_t kPieceMin = 8192;

XentPlan plan_xent(int64_t rows, int64_t dim, int64_t vocab, const void* weight, int64_t ldw, bool backward) {
    XentPlan p{};
    p.rows = rows;
    p.dim = dim;
    p.vocab = vocab;
    p.pack_w = !is_aligned(weight, 16) || ldw % 8 != 0;
    // a pair needs 256 rows to be full, and halves what each CTA reads of the weight: backward of 64 rows x 2048 x
    // 32768 with single CTAs 122 us, pairs 125; 128 x 4096 x 131072 690, 720; 192 rows 142, 132; 512 rows 199, 173
    p.cta = rows > 128 ? 2 : 1;
    p.rows_pad = up(std::max<int64_t>(rows, 1), 128 * p.cta);
    p.ldh = up(dim, 8);
    int64_t piece = up(vocab, kTileN);
    if (backward) piece = std::min(piece, std::max(kPieceMin, kPieceBytes / (2 * p.rows_pad) / kTileN * kTileN));
    if (p.pack_w) piece = std::min(piece, std::max(kPieceMin, kPieceBytes / (2 * p.ldh) / kTileN * kTileN));
    p.piece = piece;
    p.ldacc = up(dim, 32);
    // few rows leave dH few tiles: K (the piece) is split until the tiles fill the GPU (152 SMs; not asked of the
    // device, because the workspace call answers without one), 512 columns at least
    // (backward of 16 x 4096 x 131072 675 us, 1184 unsplit; 200 x 1024 x 32768 82, 196; 1024 x 2048 x 32768 253, 302)
    const int64_t tiles = p.rows_pad / (128 * p.cta) * ((dim + kTileN - 1) / kTileN);
    p.splits = (int)std::max<int64_t>(1, std::min<int64_t>({152 / p.cta / tiles, p.piece / 512, 64}));
    size_t at = 256;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at = (at + bytes + 255) & ~(size_t)255;
        return o;
    };
    p.row_of = take(4 * p.rows_pad);
    p.pos_of = take(4 * p.rows_pad);
    p.target_of = take(4 * p.rows_pad);
    p.hc = take(2 * p.rows_pad * p.ldh);
    if (p.pack_w) p.wc = take(2 * p.piece * p.ldh);
    if (backward) {
        p.lse_of = take(4 * p.rows_pad);
        p.scale_of = take(4 * p.rows_pad);
        p.e = take(2 * p.rows_pad * p.piece);
        p.acc = take(4 * p.splits * p.rows_pad * p.ldacc);
    } else {
        p.target_logit = take(4 * p.rows_pad);
        p.part = take(8 * (up(vocab, kTileN) / 128) * p.rows_pad);
    }
    p.bytes = at;
    return p;
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static EncodeFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult st;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &st) != cudaSuccess ||
            st != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

// Map of a [rows][cols] bf16 matrix (row stride ld elements) for boxes of box_rows rows of 64 elements.
int make_map(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
    EncodeFn fn = encode_fn();
    if (!fn) return set_error(OPTIM_ECUDA, "cuTensorMapEncodeTiled is not available");
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, one[2] = {1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, one,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return set_error(OPTIM_ECUDA, "tensor map of a %lld x %lld matrix: error %d", (long long)rows, (long long)cols, (int)r);
    return OPTIM_OK;
}

// LMOPT_FAULT_INJECT=stall_<stats|grad|hidden|weight>_<copy|peer|free>: what that product's first cluster
// withholds, so that its waits run out (tests).
int injected_stall(int mode) {
    static const char* const roles[] = {"stats", "grad", "hidden", "weight"};
    static const char* const what[] = {"copy", "peer", "free"};
    char name[32];
    for (int i = 0; i < 3; ++i) {
        std::snprintf(name, sizeof name, "stall_%s_%s", roles[mode], what[i]);
        if (fault_injected(name)) return kStallCopy + i;
    }
    return 0;
}

template <int kMode, int kCta>
int launch_product_t(const CUtensorMap& a, const CUtensorMap& b, ProductArgs p, cudaStream_t s) {
    constexpr int kSmem = 1024 + product_stages(kCta) * (128 + kTileN / kCta) * kTileK * 2 + kFinishBytes;
    auto kernel = k_product<kMode, kCta>;
    static std::atomic<uint64_t> allowed{0};
    const int rc = allow_smem(kernel, kSmem, allowed);
    if (rc) return rc;
    p.stall = faults_injected() ? injected_stall(kMode) : 0;
    p.wait_ns = p.stall ? kWaitNs / 40 : kWaitNs;
    const int64_t units = (int64_t)p.m_tiles * p.n_tiles * p.splits;
    const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(units, sm_count() / kCta)) * kCta;
    return check_cuda(launch_after(kernel, grid, kProductThreads, kSmem, kCta, s, a, b, p), "product launch");
}

template <int kMode>
int launch_product(const XentPlan& pl, const CUtensorMap& a, const CUtensorMap& b, const ProductArgs& p, cudaStream_t s) {
    return pl.cta == 2 ? launch_product_t<kMode, 2>(a, b, p, s) : launch_product_t<kMode, 1>(a, b, p, s);
}

}  // namespace

size_t xent_workspace_bytes(int64_t rows, int64_t dim, int64_t vocab, const void* weight, int64_t ldw, bool backward) {
    return plan_xent(rows, dim, vocab, weight, ldw, backward).bytes;
}

int launch_xent(const XentCall& c, cudaStream_t s) {
    const XentPlan pl = plan_xent(c.rows, c.dim, c.vocab, c.weight, c.ldw, c.backward);
    char* const ws = static_cast<char*>(c.workspace);
    XentHead* const head = reinterpret_cast<XentHead*>(ws);
    int32_t* const row_of = reinterpret_cast<int32_t*>(ws + pl.row_of);
    int32_t* const pos_of = reinterpret_cast<int32_t*>(ws + pl.pos_of);
    int32_t* const target_of = reinterpret_cast<int32_t*>(ws + pl.target_of);
    uint16_t* const hc = reinterpret_cast<uint16_t*>(ws + pl.hc);
    RowArgs ra{};
    ra.target = c.target;
    ra.rows = c.rows;
    ra.ignore = c.ignore_index;
    ra.vocab = (int32_t)c.vocab;
    ra.dim = (int32_t)c.dim;
    ra.hidden = static_cast<const uint16_t*>(c.hidden);
    ra.ldh = c.ldh;
    ra.vec = is_aligned(c.hidden, 16) && c.ldh % 8 == 0 && c.dim % 8 == 0 && c.dim < (1 << 22);
    ra.head = head;
    ra.hc = hc;
    ra.ldhc = pl.ldh;
    ra.row_of = row_of;
    ra.target_of = target_of;
    if (c.backward) {
        ra.pos_of = pos_of;
        ra.lse_in = c.lse;
        ra.grad = c.grad_loss;
        ra.lse_of = reinterpret_cast<float*>(ws + pl.lse_of);
        ra.scale_of = reinterpret_cast<float*>(ws + pl.scale_of);
        if (pl.splits == 1) ra.dh = static_cast<uint16_t*>(c.d_hidden);   // else k_xent_hidden writes every row
        ra.lddh = c.lddh;
    } else {
        ra.loss = c.loss;
        ra.lse = c.lse;
    }
    // a row to a CTA while there are few (64 rows: 4.3 us against 5.8 with four), two CTAs on an SM at most
    ra.per_cta = std::max<int64_t>(1, (c.rows + 2 * sm_count() - 1) / (2 * sm_count()));
    int rc = check_cuda(launch_after(k_xent_rows, std::max<int64_t>(1, (c.rows + ra.per_cta - 1) / ra.per_cta), kThreads, 0, 1, s,
                                     ra), "row gathering launch");

    ProductArgs p{};
    p.head = head;
    p.vocab = (int32_t)c.vocab;
    p.dim = (int32_t)c.dim;
    p.rows_pad = pl.rows_pad;
    p.target = target_of;
    p.lse = ra.lse_of;
    p.scale = ra.scale_of;
    p.part = reinterpret_cast<float2*>(ws + pl.part);
    p.target_logit = reinterpret_cast<float*>(ws + pl.target_logit);
    p.e = reinterpret_cast<uint16_t*>(ws + pl.e);
    p.lde = pl.piece;
    p.acc = reinterpret_cast<float*>(ws + pl.acc);
    p.ldacc = pl.ldacc;
    p.row_of = row_of;
    p.dh = static_cast<uint16_t*>(c.d_hidden);
    p.lddh = c.lddh;
    p.dh_aligned = row_alignment(c.d_hidden, c.lddh);
    p.dw = static_cast<uint16_t*>(c.d_weight);
    p.lddw = c.lddw;
    p.dw_aligned = row_alignment(c.d_weight, c.lddw);
    const int row_tiles = (int)(pl.rows_pad / (128 * pl.cta)), dim_tiles = (int)((c.dim + kTileN - 1) / kTileN);
    const int dim_blocks = (int)((c.dim + kTileK - 1) / kTileK);
    const int box_b = kTileN / pl.cta;
    CUtensorMap h_k{}, h_mn{}, e_k{}, e_mn{}, w_k{}, w_mn{};
    if (!rc) rc = make_map(&h_k, hc, pl.rows_pad, c.dim, pl.ldh, 128);
    if (!rc && c.backward) {
        rc = make_map(&h_mn, hc, pl.rows_pad, c.dim, pl.ldh, 64);
        if (!rc) rc = make_map(&e_k, p.e, pl.rows_pad, pl.piece, pl.piece, 128);
        if (!rc) rc = make_map(&e_mn, p.e, pl.rows_pad, pl.piece, pl.piece, 64);
    }
    for (int64_t v0 = 0; !rc && v0 < c.vocab; v0 += pl.piece) {
        const int64_t width = std::min(pl.piece, c.vocab - v0);
        const uint16_t* w = static_cast<const uint16_t*>(c.weight);
        if (pl.pack_w) {   // the piece's rows, side by side; the maps then start at the piece
            uint16_t* const wc = reinterpret_cast<uint16_t*>(ws + pl.wc);
            rc = check_cuda(launch_after(k_xent_pack, std::min<int64_t>(width, (int64_t)sm_count() * 8), kThreads, 0, 1, s,
                                         w + v0 * c.ldw, c.ldw, wc, pl.ldh, width, (int)c.dim, v0 == 0), "weight copy launch");
            w = wc;
        }
        if (!rc && (pl.pack_w || v0 == 0)) {
            const int64_t map_rows = pl.pack_w ? width : c.vocab, ld = pl.pack_w ? pl.ldh : c.ldw;
            rc = make_map(&w_k, w, map_rows, c.dim, ld, box_b);
            if (!rc && c.backward) rc = make_map(&w_mn, w, map_rows, c.dim, ld, 64);
        }
        if (rc) break;
        ProductArgs q = p;
        q.splits = 1;
        q.b_off = pl.pack_w ? 0 : (int32_t)v0;
        q.v_off = (int32_t)v0;
        q.m_tiles = row_tiles;
        q.n_tiles = (int)((width + kTileN - 1) / kTileN);
        q.k_blocks = dim_blocks;
        if (!c.backward) {
            rc = launch_product<kStats>(pl, h_k, w_k, q, s);
            continue;
        }
        rc = launch_product<kGrad>(pl, h_k, w_k, q, s);
        if (!rc && c.d_hidden) {
            ProductArgs h = q;
            h.n_tiles = dim_tiles;
            h.k_blocks = (int)((width + kTileK - 1) / kTileK);
            h.splits = pl.splits;
            h.first = v0 == 0;
            h.last = pl.splits == 1 && v0 + width == c.vocab;
            rc = launch_product<kHidden>(pl, e_k, w_mn, h, s);
        }
        if (!rc && c.d_weight) {
            ProductArgs d = q;
            d.m_tiles = (int)((width + 128 * pl.cta - 1) / (128 * pl.cta));
            d.n_tiles = dim_tiles;
            rc = launch_product<kWeight>(pl, e_mn, h_mn, d, s);
        }
    }
    if (rc) return rc;
    if (!c.backward) {
        const bool few = c.rows <= 2 * sm_count();
        return check_cuda(launch_after(few ? k_xent_loss<1> : k_xent_loss<8>,
                                       few ? c.rows : std::min<int64_t>((c.rows + 7) / 8, (int64_t)sm_count() * 8), kThreads, 0, 1, s,
                                       head, p.part, (int)((c.vocab + 127) / 128), pl.rows_pad, p.target_logit, target_of,
                                       row_of, c.loss, c.lse), "loss launch");
    }
    if (!c.d_hidden || c.rows == 0 || pl.splits == 1) return OPTIM_OK;
    const bool vec = is_aligned(c.d_hidden, 8) && c.lddh % 4 == 0;
    return check_cuda(launch_after(k_xent_hidden, dim3((unsigned)c.rows, (unsigned)((c.dim + 127) / 128)), kThreads, 0, 1, s, head,
                                   pos_of, p.acc, pl.splits, pl.rows_pad, pl.ldacc, p.dh, c.lddh, (int)c.dim, vec),
                      "hidden gradient launch");
}

}  // namespace lmo

using namespace lmo;

static int check_matrix(const void* p, int64_t ld, int64_t rows, int64_t cols, const char* name) {
    if (rows == 0) return OPTIM_OK;
    if (!p) return set_error(OPTIM_EINVAL, "%s is NULL", name);
    if (rows > 1 && ld < cols) return set_error(OPTIM_EINVAL, "%s: row stride %lld below %lld", name, (long long)ld, (long long)cols);
    if (!is_aligned(p, 2)) return set_error(OPTIM_EALIGN, "%s not 2-byte aligned", name);
    return OPTIM_OK;
}
static int check_array(const void* p, size_t align, const char* name) {
    if (!p) return set_error(OPTIM_EINVAL, "%s is NULL", name);
    if (!is_aligned(p, align)) return set_error(OPTIM_EALIGN, "%s not %zu-byte aligned", name, align);
    return OPTIM_OK;
}

// Tile and row numbers are 32-bit in the kernels.
static int check_sizes(int64_t rows, int64_t dim, int64_t vocab) {
    if (rows < 0 || dim < 1 || vocab < 1) return set_error(OPTIM_EINVAL, "need rows >= 0, dim >= 1 and vocab >= 1");
    const int64_t most = (int64_t)1 << 28, tiles = (int64_t)1 << 30;
    if (rows > most || dim > most || vocab > most || (rows / 128 + 2) * (vocab / 128 + 2) > tiles ||
        (vocab / 128 + 2) * (dim / 128 + 2) > tiles || (rows / 128 + 2) * (dim / 128 + 2) * 64 > tiles)
        return set_error(OPTIM_EINVAL, "%lld rows, dim %lld, vocab %lld: too large", (long long)rows, (long long)dim, (long long)vocab);
    return OPTIM_OK;
}

static int check_xent(XentCall& c) {
    int rc = check_sizes(c.rows, c.dim, c.vocab);
    if (!rc) rc = check_matrix(c.hidden, c.ldh, c.rows, c.dim, "hidden");
    if (!rc) rc = check_matrix(c.weight, c.ldw, c.vocab, c.dim, "weight");
    if (!rc && c.rows > 0) rc = check_array(c.target, 8, "target");
    if (!rc && c.rows > 0) rc = check_array(c.lse, 4, "lse");
    if (rc) return rc;
    if (c.vocab == 1) c.ldw = std::max(c.ldw, c.dim);   // the stride of a single row is anything
    const size_t need = xent_workspace_bytes(c.rows, c.dim, c.vocab, c.weight, c.ldw, c.backward);
    rc = check_array(c.workspace, 256, "workspace");
    if (!rc && c.workspace_bytes < need)
        rc = set_error(OPTIM_EINVAL, "workspace of %zu bytes, %zu needed", c.workspace_bytes, need);
    return rc;
}

extern "C" {

int loss_xent_workspace(int64_t rows, int64_t dim, int64_t vocab, const void* weight, int64_t ldw, int32_t backward,
                        size_t* bytes) {
    if (!bytes) return set_error(OPTIM_EINVAL, "bytes is NULL");
    const int rc = check_sizes(rows, dim, vocab);
    if (rc) return rc;
    *bytes = xent_workspace_bytes(rows, dim, vocab, weight, vocab == 1 ? std::max(ldw, dim) : ldw, backward != 0);
    return OPTIM_OK;
}

int loss_xent_forward(const void* hidden, int64_t ldh, const void* weight, int64_t ldw, const int64_t* target, int64_t rows,
                      int64_t dim, int64_t vocab, int64_t ignore_index, float* loss, float* lse, void* workspace,
                      size_t workspace_bytes, void* stream) {
    XentCall c{};
    c.hidden = hidden, c.ldh = ldh, c.weight = weight, c.ldw = ldw, c.target = target;
    c.rows = rows, c.dim = dim, c.vocab = vocab, c.ignore_index = ignore_index;
    c.loss = loss, c.lse = lse, c.workspace = workspace, c.workspace_bytes = workspace_bytes;
    int rc = check_xent(c);
    if (!rc && rows > 0) rc = check_array(loss, 4, "loss");
    if (rc || rows == 0) return rc;
    return launch_xent(c, static_cast<cudaStream_t>(stream));
}

int loss_xent_backward(const void* hidden, int64_t ldh, const void* weight, int64_t ldw, const int64_t* target,
                       const float* lse, const float* grad_loss, int64_t rows, int64_t dim, int64_t vocab,
                       int64_t ignore_index, void* d_hidden, int64_t lddh, void* d_weight, int64_t lddw, void* workspace,
                       size_t workspace_bytes, void* stream) {
    XentCall c{};
    c.hidden = hidden, c.ldh = ldh, c.weight = weight, c.ldw = ldw, c.target = target;
    c.rows = rows, c.dim = dim, c.vocab = vocab, c.ignore_index = ignore_index;
    c.lse = const_cast<float*>(lse), c.grad_loss = grad_loss, c.backward = true;
    c.d_hidden = d_hidden, c.lddh = lddh, c.d_weight = d_weight, c.lddw = lddw;
    c.workspace = workspace, c.workspace_bytes = workspace_bytes;
    int rc = check_xent(c);
    if (!rc && rows > 0) rc = check_array(grad_loss, 4, "grad_loss");
    if (!rc && d_hidden) rc = check_matrix(d_hidden, lddh, rows, dim, "d_hidden");
    if (!rc && d_weight) rc = check_matrix(d_weight, lddw, vocab, dim, "d_weight");
    if (rc || (!d_hidden && !d_weight)) return rc;
    return launch_xent(c, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
