// attn_backward.cu -- the gradients of causal attention over packed sequences with grouped heads.
//   p_ij = exp(s_ij - lse_i),  delta_i = dO_i o_i,  dS_ij = p_ij (dO_i v_j - delta_i)
//   dq_i = scale sum_j dS_ij k_j,  dk_j = scale sum_i dS_ij q_i,  dv_j = sum_i p_ij dO_i   (i: of all heads that share j)
// Scores are formed again.  Two product kernels, one for dq (a tile of queries, the keys stream by) and one for dk and
// dv (a tile of keys, the queries of the group's heads stream by): every sum has one owner and one order, at the
// price of forming p and dS twice (7 products, not 5); adding dq up from the tiles of keys would need atomics, whose order changes
// results, or a buffer of fp32.
//
// Both are one kernel in two roles.  A CTA holds two operands of 128 rows (Q and dO, in tensor memory, or K and V, in shared memory) and
// streams pairs of blocks of 64 rows of the other two.  X = A0 B0' and Y = A1 B1' go into one of two pairs of accumulators (64 columns
// each), eight warps turn them into p and dS, in bf16, in place (the tensor cores want both operands of one type), and those are the A
// operands, from tensor memory, of the sums' products (with B0 and B1 read along their rows).  For keys X and Y are the transposed
// scores: nothing is ever transposed through shared memory.  Blocks of 64 so that two pairs and the two sums fit in the 512
// columns; while the warps work on one pair the tensor cores fill the other.
//
// What bf16 costs.  dq, dk and dv are rounded once at their end (1.65e-3 in the 2-norm), p and dS once before (as much again): within 2.4e-3 of 64
// bits.  For heads up to 80 dq takes dS in two bf16 parts (a product more): 1.7e-3.
// The rounding of out does not count: delta formed from out as it was rounded is off by some 2^-9 |dO||o|, and every dS of the row by p_ij times that.  In dq this
// makes sum_j p_ij k_j times it, which is as large as a key where a row's weights lie on few keys, or where the keys have a mean, while dq itself may be small
// (on 512 tokens it was 5e-3 of dq with sharp weights, 2e-1 with keys and values whose mean is four times their spread).  So dq's kernel sums its dS,
// which the true delta would make 0: the keys' kernel takes delta without that excess, and dq is rid of the excess times sum_j p_ij k_j, which
// is formed beside it (a product more).  Where dS is in one part, the excess is that of the rounded values: then dq, like the formula's, does not
// change when a vector is added to all keys.  16384 tokens, 16 / 4 heads of 64, 80, 96, 128: dq 1042, 1173, 1126, 1268 us; without the product
// and with dS in two parts 975, 1040, 1095, 1190.
//
// Many rows: the tensor cores bound it, and their power.  16384 tokens, 16 / 4 heads of 128: dq 1.27 ms, dk and dv 1.33 ms, together 8 products of
// 0.55e12 operations at 1.69 PFLOP/s (a library product in a burst: 1.93).  128 x 64 scores from shared memory take 48 cycles for 16 elements of
// the head where 32 would do (128 bytes a cycle); operands in tensor memory free dq's of it.  A lone CTA takes 7 us from its start to its end, of
// which two blocks are 1.3: texts of 1 to 2035 tokens (11287 rows, 12 / 3 heads of 80) take 194 us, of which the products are 41.
// What the warps' part cost before: tests of masked places in every block (one set of instructions in two), operands read row by row
// from memory (a line a lane, 3 us a tile), a wait that reads the timer (half of the waits last less).
#include <type_traits>

#include "attn.cuh"

namespace lmo {
namespace {

constexpr int kTile = 128, kStep = 64;           // rows of a CTA's tile and of a streamed block
constexpr int kAttnThreads = 384;                // warp 0 copies, warp 1 multiplies, warp 2 holds tensor memory; 4-11: p and dS
constexpr uint32_t kTileBytes = kTile * 256, kStepBytes = kStep * 256;
constexpr int kStages = 4;                       // of a pair of streamed blocks
constexpr int kFewBlocks = 12;
// Tiles of the CTA's own rows in shared memory: Q, dO and out (which go into tensor memory, or into delta), or K and V.
__host__ __device__ constexpr int own_tiles(int role) { return role == 0 ? 3 : 2; }
__host__ __device__ constexpr size_t smem_of(int role) {
    return own_tiles(role) * kTileBytes + kStages * (2 * kStepBytes + (role == 0 ? 0 : kStep * 8)) + 1024;
}

// The rows' -lse (times log2 e) and -delta, by blocks of 64 rows of a sequence: 64 of one, 64 of the other.  Blocks are numbered as tiles
// of 64 (find_tile), `slots` a head; rows behind a sequence's end have -inf (p is 0) and 0.
struct RowBlock {
    float lse[kStep], delta[kStep];
};

__device__ __forceinline__ float dot8(const uint4& a, const uint4& b) {
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s = fmaf(__uint_as_float(x[i] << 16), __uint_as_float(y[i] << 16), s);
        s = fmaf(__uint_as_float(x[i] & 0xFFFF0000u), __uint_as_float(y[i] & 0xFFFF0000u), s);
    }
    return s;
}

enum { kQueries = 0, kKeys = 1 };

// Columns of tensor memory (512).  X and Y: two blocks' scores each.  Keys: dk, dv.  Queries: the sums of dS K and of p K, and the tile's
// operands Q and dO.  Heads over 80 have no room for a second X, which is then formed when the warps have read the one before, nor for what dS's
// rounding left; over 96 none for dO, which is read from shared memory (48 cycles for 16 elements of a block instead of 32).  A head's 16 elements
// take 8 columns as an operand, 16 as a sum.  (Heads of 96 with a second X and dO in shared memory: 16384 tokens, dq 1361 us.)
template <int kRole, int kSteps>
struct Columns {
    static constexpr bool kWide = kRole == kQueries && kSteps > 5, kBoth = kRole == kQueries && kSteps <= 6;     // kBoth: Q and dO are here
    static constexpr uint32_t kX = 0, kNextX = kWide ? 0 : 64, kY = kWide ? 64 : 128, kNextY = 64;
    static constexpr uint32_t kSum = kWide ? 192 : 256, kDv = 384, kMean = kSum + (kSteps * 16 + 31) / 32 * 32;   // sums start at multiples of 32
    static constexpr uint32_t kQ = kMean + kSteps * 16, kDo = kQ + kSteps * 8;
    static_assert(kRole == kKeys || kQ + (kBoth ? 2 : 1) * kSteps * 8 <= 512, "tensor memory");
};

struct BackwardArgs {
    Sequences seq;
    int64_t slots, row_slots;           // tiles of 128, blocks of 64
    int32_t heads, kv_heads, group, dim;
    int32_t splits;                     // kKeys: CTAs (a cluster) that share a tile's blocks
    float scale;
    RowBlock* rows;
    const float* lse;                   // kQueries
    HeadRows out0, out1;                // dq; or dk, dv
    const uint16_t* d_out;              // kKeys: for what is taken out of masked blocks
    int64_t lddo, hsdo;
    uint64_t wait_ns;
    int32_t stall;                      // tests of the waits' limit: what the first sequence's first tile of head 0 withholds (Stall), or 0
};
enum Stall { kStallCopy = 1, kStallSoftmax = 2 };

// What was cleared of d_out in the masked blocks of a tile of keys (its own rows and the sequence's last block), for the sums of one key.
template <int N>
__device__ __forceinline__ void add_cleared(const BackwardArgs& p, const Tile& tile, int kv, int64_t row, int c, float (&z)[N]) {
    const int64_t own = min(tile.first + kTile, tile.end);
    const int64_t last = tile.first + (tile.end - tile.first) / kStep * kStep;   // first row of a block that is not whole
    for (int g = 0; g < p.group; ++g) {
        const uint16_t* const d_out = p.d_out + (int64_t)(kv * p.group + g) * p.hsdo;
        add_non_finite(z, d_out, p.lddo, row, own, c, p.dim);
        add_non_finite(z, d_out, p.lddo, max(own, last), tile.end, c, p.dim);
    }
}
__device__ __forceinline__ void store8(uint16_t* to, float a, float b, float c, float d, float e, float f, float g, float h) {
    *reinterpret_cast<uint4*>(to) = make_uint4(pack_bf16(a, b), pack_bf16(c, d), pack_bf16(e, f), pack_bf16(g, h));
}
// A CTA's sums for its cluster, over the operands that it is done with: four elements of 128 rows next to each other.
__device__ __forceinline__ float4* part_at(char* base, int which, int c, int row) {
    return reinterpret_cast<float4*>(base + which * (kTile * 512)) + (c / 4) * kTile + row;
}

// maps: the tile's operands (a0, a1), the streamed ones (b0, b1): Q, dO, K, V for queries (and out), K, V, Q, dO for keys
template <int kRole, int kSteps>
__global__ void __launch_bounds__(kAttnThreads, 1) k_attn_backward(const __grid_constant__ CUtensorMap map_a0, const __grid_constant__ CUtensorMap map_a1,
                                                                   const __grid_constant__ CUtensorMap map_b0, const __grid_constant__ CUtensorMap map_b1,
                                                                   const __grid_constant__ CUtensorMap map_out, const BackwardArgs p) {
    extern __shared__ uint8_t smem_raw[];
    using At = Columns<kRole, kSteps>;
    __shared__ uint64_t bars[1 + 2 * kStages + 4 + 6];
    __shared__ uint32_t tmem_base;
    __shared__ int gave_up, found, copied;
    __shared__ float tile_delta[kRole == kQueries ? kTile : 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // before anything of the stream is needed
    const uint32_t a_full = smem_u32(bars), full = a_full + 8, empty = full + 8 * kStages, x_done = empty + 8 * kStages, ready = x_done + 16,
                   sums_done = ready + 16, drained = sums_done + 8, halves_ready = drained + 8, delta_ready = halves_ready + 8, tile_full = delta_ready + 8,
                   x_free = tile_full + 8;
    if (threadIdx.x == 0) {
        gave_up = found = copied = 0;
        mbar_init(a_full, 8);
        mbar_init(tile_full, 1);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(x_done + 8 * i, 1);
            mbar_init(ready + 8 * i, 8);
        }
        mbar_init(sums_done, 1);
        mbar_init(drained, 1);
        mbar_init(halves_ready, 8);
        mbar_init(delta_ready, 4);
        mbar_init(x_free, 8);
        mbar_init_fence();
        tma_prefetch_map(&map_a0);
        tma_prefetch_map(&map_a1);
        if (kRole == kQueries) tma_prefetch_map(&map_out);
        tma_prefetch_map(&map_b0);
        tma_prefetch_map(&map_b1);
    }
    if (warp == 2) tmem_alloc<1>(smem_u32(&tmem_base), 512);
    tc_fence_before();
    pdl_sync();
    const int heads = kRole == kQueries ? p.heads : p.kv_heads;
    const int rank = kRole == kKeys && p.splits > 1 ? (int)cluster_rank() : 0;
    const unsigned unit = kRole == kKeys ? blockIdx.x / (unsigned)p.splits : blockIdx.x;
    const int head = (int)(unit % (unsigned)heads);
    // the tiles with the most work first: the last queries, the first keys
    const int64_t slot = unit / (unsigned)heads;
    const Tile tile = find_tile<kTile>(p.seq, kRole == kQueries ? p.slots - 1 - slot : slot);
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    auto leave = [&]() {
        if (warp == 2) tmem_free<1>(tmem, 512);
    };
    if (tile.first >= tile.end) return leave();
    if (tile.segment == 0 || tile.segment == p.seq.n + 1) {   // rows of no sequence
        const int rows = (int)min((int64_t)kTile, tile.end - tile.first), vecs = p.dim / 8;
        for (int i = threadIdx.x; rank == 0 && i < rows * vecs; i += kAttnThreads) {
            const int64_t row = tile.first + i / vecs;
            const int c = i % vecs * 8;
            if (p.out0.p) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out0.p) + head * p.out0.head + row * p.out0.row + c) = make_uint4(0, 0, 0, 0);
            if (kRole == kKeys)
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out1.p) + head * p.out1.head + row * p.out1.row + c) = make_uint4(0, 0, 0, 0);
        }
        return leave();
    }

    // Streamed blocks: for queries those of the keys up to the tile's last row, for keys those of the queries from the tile's first row
    // on, head by head.
    const int64_t stream_first = kRole == kQueries ? tile.start : tile.first;
    const int64_t stream_end = kRole == kQueries ? min(tile.first + kTile, tile.end) : tile.end;
    const int per_head = (int)((stream_end - stream_first + kStep - 1) / kStep);
    const int all_blocks = per_head * (kRole == kQueries ? 1 : p.group);
    // CTAs of the cluster that take part: each has a start and an end of its own that cost as much as several blocks
    const int splits = kRole == kKeys ? min(p.splits, max(1, all_blocks / kFewBlocks)) : 1;
    if (rank >= splits) return leave();
    const int first_block = (int)((int64_t)all_blocks * rank / splits), blocks = (int)((int64_t)all_blocks * (rank + 1) / splits) - first_block;

    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    char* const base_ptr = reinterpret_cast<char*>(smem_raw) + (base - smem_u32(smem_raw));
    const uint32_t stages = base + own_tiles(kRole) * kTileBytes;      // stage: B0, B1
    const uint32_t row_stages = stages + kStages * 2 * kStepBytes;       // kKeys: RowBlock each
    auto wait = [&](uint32_t bar, uint32_t parity) { return mbar_wait<1>(bar, parity, &gave_up, p.wait_ns); };

    const int stall = head == 0 && rank == 0 && tile.segment == 1 && tile.first == tile.start ? p.stall : 0;

    if (warp < 4) {
        regs_down<88>();
        if (warp == 0 && elect_lane()) {
            const int stop = stall == kStallCopy ? 0 : 0x7FFFFFFF;
            const uint32_t boxes = p.dim > 64 ? 2 : 1;
            mbar_expect_tx(tile_full, own_tiles(kRole) * boxes * kTile * 128);
            load_rows<kTile>(base, &map_a0, p.dim, head, tile.first, tile_full);
            load_rows<kTile>(base + kTileBytes, &map_a1, p.dim, head, tile.first, tile_full);
            if (kRole == kQueries) load_rows<kTile>(base + 2 * kTileBytes, &map_out, p.dim, head, tile.first, tile_full);
            int issued = 0, in = first_block % per_head;
            int of = kRole == kQueries ? head / p.group : head * p.group + first_block / per_head;     // head of the streamed operands
            const int64_t row_slot = kRole == kKeys ? (tile.start / kStep + tile.segment) + (tile.first - tile.start) / kStep : 0;
            bool ok = true;
            uint32_t stage = 0, phase = 0;
            for (int i = 0; ok && i < blocks; ++i) {
                ok = issued != stop && wait(empty + 8 * stage, phase ^ 1u);
                if (!ok) break;
                const uint32_t bar = full + 8 * stage, b = stages + stage * 2 * kStepBytes;
                mbar_expect_tx(bar, 2 * boxes * kStep * 128 + (kRole == kKeys ? (uint32_t)sizeof(RowBlock) : 0u));
                const int64_t row = stream_first + (int64_t)in * kStep;
                load_rows<kStep>(b, &map_b0, p.dim, of, row, bar);
                load_rows<kStep>(b + kStepBytes, &map_b1, p.dim, of, row, bar);
                if (kRole == kKeys)
                    bulk_load(row_stages + stage * (uint32_t)sizeof(RowBlock), p.rows + of * p.row_slots + row_slot + in, sizeof(RowBlock), bar);
                ++issued;
                if (++stage == kStages) stage = 0, phase ^= 1u;
                if (++in == per_head) in = 0, ++of;
            }
            // the last stages come back before the CTA ends: nothing arrives on its barriers after that
            for (int i = max(0, blocks - kStages); ok && i < blocks; ++i) ok = wait(empty + 8 * (i % kStages), i / kStages & 1);
            copied = issued;
        } else if (warp == 1 && elect_lane()) {
            constexpr uint32_t desc_x = mma_desc(128, kStep, false, false), desc_sum = mma_desc(128, kSteps * 16, false, true);
            constexpr uint32_t up = desc_upper(1024);
            const uint32_t a_lo = desc_lower(base, 8192), b_lo = desc_lower(stages, kStep * 128);
            bool ok = wait(tile_full, 0) && (kRole == kKeys || wait(a_full, 0));
            tc_fence_after();
            uint32_t next = 0, parity = 0, stage = 0;       // of the block whose scores, and whose sums, come next
            auto scores = [&](int i) {
                ok = wait(full + 8 * next, parity);
                if (!ok) return;
                tc_fence_after();
                const uint32_t b0 = b_lo + next * (2 * kStepBytes >> 4), b1 = b0 + (kStepBytes >> 4);
                const uint32_t x = tmem + At::kX + (i & 1) * At::kNextX, y = tmem + At::kY + (i & 1) * At::kNextY;
                auto of_head = [](int j, int rows) { return (uint32_t)((j >> 2) * (rows * 8) + (j & 3) * 2); };   // 16 elements of a head
                if (kRole == kKeys) {
#pragma unroll
                    for (int j = 0; j < kSteps; ++j) mma_ss(x, a_lo + of_head(j, kTile), b0 + of_head(j, kStep), up, desc_x, j == 0);
                }
#pragma unroll
                for (int j = 0; j < kSteps; ++j) {
                    if (At::kBoth) mma_ts(y, tmem + At::kDo + j * 8, b1 + of_head(j, kStep), up, desc_x, j == 0);
                    else mma_ss(y, a_lo + (kTileBytes >> 4) + of_head(j, kTile), b1 + of_head(j, kStep), up, desc_x, j == 0);
                }
                if (kRole == kQueries) {
                    if (At::kWide && i > 0) {
                        ok = wait(x_free, (i - 1) & 1);
                        if (!ok) return;
                        tc_fence_after();
                    }
#pragma unroll
                    for (int j = 0; j < kSteps; ++j) mma_ts(x, tmem + At::kQ + j * 8, b0 + of_head(j, kStep), up, desc_x, j == 0);
                }
                mma_commit<1>(x_done + 8 * (i & 1));
                if (++next == kStages) next = 0, parity ^= 1u;
            };
            if (ok && blocks) scores(0);
            for (int i = 0; ok && i < blocks; ++i) {
                if (i + 1 < blocks) scores(i + 1);      // over p and dS of block i - 1, behind the products that read them
                if (ok) ok = wait(ready + 8 * (i & 1), i / 2 & 1);
                if (!ok) break;
                tc_fence_after();
                const uint32_t b = b_lo + stage * (2 * kStepBytes >> 4);
                const uint32_t x = tmem + At::kX + (i & 1) * At::kNextX, y = tmem + At::kY + (i & 1) * At::kNextY;
                auto add = [&](uint32_t sum, uint32_t a, uint32_t rows, bool first) {     // a's weights times 64 rows
#pragma unroll
                    for (int j = 0; j < kStep / 16; ++j) mma_ts(sum, a + (j >> 1) * 32 + (j & 1) * 8, rows + j * 128, up, desc_sum, first && j == 0);
                };
                if (kRole == kKeys) add(tmem + At::kDv, x, b + (kStepBytes >> 4), i == 0);                   // dv += p' dO
                add(tmem + At::kSum, y, b, i == 0);                                                         // dq += dS K, dk += dS' Q
                if (kRole == kQueries) {
                    if (!At::kWide) add(tmem + At::kSum, y + 16, b, false);                                  // what dS's rounding left
                    add(tmem + At::kMean, At::kWide ? y + 16 : x, b, i == 0);                               // p K
                }
                mma_commit<1>(empty + 8 * stage);
                if (++stage == kStages) stage = 0;
            }
            if (ok) mma_commit<1>(sums_done);
        }
        __syncwarp();
    } else {
        regs_up<208>();
        const int t = (warp >> 2) - 1;                                         // columns 32 t .. 32 t + 31 of every block
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const int in = 32 * (warp & 3) + lane;                                 // this thread's row of the tile
        const int64_t row = tile.first + in;
        const float c = p.scale * kLog2e;
        const F2 c2 = f2(c, c);
        float my_lse = 0.0f, my_delta = 0.0f;
        bool ok = true;
        if (kRole == kQueries) {
            // Q (four warps) and dO (the others, where it has room) into tensor memory, two elements a column; delta from out as it was rounded.
            // (Rows come in by copies: a lane's own row read from memory takes a line of every lane for each 16 bytes, 3 us a tile.)
            ok = wait(tile_full, 0);
            const char* const mine = base_ptr + t * kTileBytes + in * 128;
            float s[4] = {};
#pragma unroll
            for (int h = 0; h < (kSteps + 3) / 4; ++h) {
                uint32_t r[32];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int at = h * kTile * 128 + (k ^ (in & 7)) * 16;      // of the eighth elements from 64 h + 8 k on
                    const uint4 v = *reinterpret_cast<const uint4*>(mine + at);
                    r[4 * k] = v.x, r[4 * k + 1] = v.y, r[4 * k + 2] = v.z, r[4 * k + 3] = v.w;
                    if (t == 1) s[k & 3] += dot8(*reinterpret_cast<const uint4*>(mine + kTileBytes + at), v);
                }
                const uint32_t to = tmem + lanes + (t ? At::kDo : At::kQ) + 32 * h;
                if (t == 0 || At::kBoth) {
                    if (h == 0 || kSteps == 8) tmem_store32(to, r);
                    else if (kSteps == 6) tmem_store16(to, reinterpret_cast<const uint32_t(&)[16]>(r));
                    else tmem_store8(to, reinterpret_cast<const uint32_t(&)[8]>(r));
                }
            }
            my_delta = -((s[0] + s[1]) + (s[2] + s[3]));
            tmem_store_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(a_full);
            my_lse = row < tile.end ? p.lse[head * p.seq.rows + row] * -kLog2e : -INFINITY;
            if (t == 1) {
                tile_delta[in] = my_delta;
                __syncwarp();
                if (lane == 0) mbar_arrive(delta_ready);
            } else {
                ok = wait(delta_ready, 0) && ok;
                my_delta = tile_delta[in];
            }
        }
        F2 excess[2] = {f2(0.0f, 0.0f), f2(0.0f, 0.0f)};                       // sum of dS
        F2 rounded[2] = {f2(0.0f, 0.0f), f2(0.0f, 0.0f)};                      // kWide: of dS as it is multiplied
        const F2 minus1 = f2(-1.0f, -1.0f), my_lse2 = f2(my_lse, my_lse), my_delta2 = f2(my_delta, my_delta);
        int at = first_block % per_head;                                       // the block's place in its head
        ok = __all_sync(0xFFFFFFFFu, ok);
        uint32_t stage = 0, phase = 0;
        for (int i = 0; ok && i < blocks; ++i, stage = stage == kStages - 1 ? 0 : stage + 1, phase ^= stage == 0 ? 1u : 0u) {
            const int64_t first = stream_first + (int64_t)at * kStep;          // the block's first row
            if (++at == per_head) at = 0;
            // keys behind a row of the tile, queries before one, or rows behind the sequence: in the block, and among the warp's own
            const bool partly = kRole == kQueries ? first + kStep > tile.first : first < tile.first + kTile || first + kStep > tile.end;
            const int64_t top = tile.first + 32 * (warp & 3), left = first + 32 * t;
            const bool masked = kRole == kQueries ? left + 31 > top : left < top + 31 || left + 32 > tile.end;
            ok = wait(x_done + 8 * (i & 1), i / 2 & 1);
            // what the copies brought is read here too
            if (ok && (kRole == kKeys || partly)) ok = wait(full + 8 * stage, phase);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            tc_fence_after();
            const uint32_t x_at = tmem + lanes + At::kX + (i & 1) * At::kNextX + 32 * t, y_at = tmem + lanes + At::kY + (i & 1) * At::kNextY + 32 * t;
            uint32_t x[32], y[32];
            tmem_load32(x_at, x);
            tmem_load32(y_at, y);
            tmem_wait(x);
            tmem_wait(y);
            if (At::kWide) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(x_free);
            }
            const RowBlock* const rb = reinterpret_cast<const RowBlock*>(base_ptr + (row_stages - base)) + stage;
            uint32_t pw[16], dw[16], left_w[16];      // p, dS, and (queries, not kWide) what the rounding of dS left
            // the columns that the row sees: from .. to - 1 (tests of them only where some are masked: they cost as much as the rest)
            const int from = kRole == kQueries ? 0 : (int)max(row - first, (int64_t)0) - 32 * t;
            const int to = (int)min((kRole == kQueries ? row + 1 : tile.end) - first, (int64_t)kStep) - 32 * t;
            // a row that sees one key: p is 1 and dS 0 (or NaN), whatever the two products' roundings say
            const bool only = kRole == kQueries && row == tile.start;
            const int one = (int)max(tile.start - first, (int64_t)-1) - 32 * t;
            auto weights = [&](auto some) {
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                    F2 l[2] = {my_lse2, my_lse2}, d[2] = {my_delta2, my_delta2};
                    if (kRole == kKeys) {
                        const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(&rb->lse[32 * t + k]), b = *reinterpret_cast<const ulonglong2*>(&rb->delta[32 * t + k]);
                        l[0].x = a.x, l[1].x = a.y, d[0].x = b.x, d[1].x = b.y;
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int e = k + 2 * h;
                        float a, b, u, w;
                        split2(fma2(f2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), c2, l[h]), a, b);
                        a = exp2_approx(a), b = exp2_approx(b);
                        split2(mul2(f2(a, b), add2(f2(__uint_as_float(y[e]), __uint_as_float(y[e + 1])), d[h])), u, w);
                        if constexpr (decltype(some)::value) {                 // 0 whatever was multiplied
                            if (e < from || e >= to) a = u = 0.0f;
                            if (e + 1 < from || e + 1 >= to) b = w = 0.0f;
                            if (kRole == kQueries ? only : e == one) u *= 0.0f;
                            if (kRole == kQueries ? only : e + 1 == one) w *= 0.0f;
                        }
                        dw[e / 2] = pack_bf16(u, w);
                        pw[e / 2] = pack_bf16(a, b);
                        if (kRole == kQueries) {
                            const F2 as = f2(__uint_as_float(dw[e / 2] << 16), __uint_as_float(dw[e / 2] & 0xFFFF0000u));
                            excess[h] = add2(excess[h], f2(u, w));
                            if (At::kWide) {
                                rounded[h] = add2(rounded[h], as);
                            } else {
                                split2(fma2(as, minus1, f2(u, w)), a, b);
                                left_w[e / 2] = pack_bf16(a, b);
                            }
                        }
                    }
                }
            };
            if (masked) weights(std::true_type{});
            else weights(std::false_type{});
            tmem_store16(At::kWide ? y_at + 16 : x_at, pw);
            tmem_store16(y_at, dw);
            if (kRole == kQueries && !At::kWide) tmem_store16(y_at + 16, left_w);
            tmem_store_wait();
            if (partly && in < kStep) {      // rows of masked places are not multiplied, not even by 0
                char* const b = base_ptr + (stages - base) + stage * 2 * kStepBytes;
                if (t == 0) clear_non_finite<kStep>(b, p.dim, in);
                else if (kRole == kKeys && clear_non_finite<kStep>(b + kStepBytes, p.dim, in)) found = 1;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0 && stall != kStallSoftmax) mbar_arrive(ready + 8 * (i & 1));
        }
        ok = ok && wait(sums_done, 0) && *static_cast<volatile int*>(&gave_up) == 0;     // whoever gave up
        ok = __all_sync(0xFFFFFFFFu, ok);
        tc_fence_after();
        float off = 0.0f;
        if (kRole == kQueries) {
            // sum_j p_ij dP_ij is delta_i, and sum_j dS_ij = 0 with it: what is left of the sum is how far off the rounding of out made
            // delta.  The keys' gradients take the better one; dq is rid of off sum_j p_ij k_j.
            float a, b;
            split2(add2(excess[0], excess[1]), a, b);
            float* const halves = reinterpret_cast<float*>(base_ptr);          // over Q, which is done with
            halves[kTile * t + in] = a + b;
            if (At::kWide) {
                split2(add2(rounded[0], rounded[1]), a, b);
                halves[kTile * (2 + t) + in] = a + b;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(halves_ready);
            ok = wait(halves_ready, 0) && ok;
            off = halves[in] + halves[kTile + in];
            if (t == 0) {
                // tiles of 128 start at a block of 64
                RowBlock& to = p.rows[head * p.row_slots + (tile.start / kStep + tile.segment) + (tile.first - tile.start) / kStep + in / kStep];
                if (tile.first + in / kStep * kStep < tile.end) {
                    to.lse[in % kStep] = my_lse;
                    to.delta[in % kStep] = row >= tile.end ? 0.0f : ok ? my_delta - off : __builtin_nanf("");
                }
            }
            if (At::kWide) off = halves[2 * kTile + in] + halves[3 * kTile + in];
            ok = __all_sync(0xFFFFFFFFu, ok);
        }
        // the first four warps take half of dq or dk out, the others the other half or dv
        const bool live = row < tile.end;
        const int which = kRole == kKeys ? t : 0;
        const HeadRows& o = which ? p.out1 : p.out0;
        uint16_t* const to = static_cast<uint16_t*>(o.p) + head * o.head + row * o.row;
        const bool sectors = (reinterpret_cast<uintptr_t>(to) & 31u) == 0;
        const float f = !ok ? __builtin_nanf("") : which ? 1.0f : p.scale;
        const uint32_t sum_at = tmem + lanes + (which ? At::kDv : At::kSum);
#pragma unroll 1
        for (int q = kRole == kQueries ? 32 * t : 0; q < p.dim; q += kRole == kQueries ? 64 : 32) {
            uint32_t r[32], mean[32];
            tmem_load32(sum_at + q, r);
            if (kRole == kQueries) tmem_load32(tmem + lanes + At::kMean + q, mean);
            tmem_wait(r);
            if (kRole == kQueries) tmem_wait(mean);
            float z[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) {
                z[k] = __uint_as_float(r[k]);
                if (kRole == kQueries) z[k] = fmaf(-off, __uint_as_float(mean[k]), z[k]);
                z[k] = blocks ? z[k] * f : 0.0f;
            }
            if (splits > 1) {
#pragma unroll
                for (int k = 0; k < 32; k += 4)
                    *part_at(base_ptr, which, q + k, in) = make_float4(z[k], z[k + 1], z[k + 2], z[k + 3]);
            } else if (live && o.p) {
                if (which && *static_cast<volatile int*>(&found)) add_cleared(p, tile, head, row, q, z);
                store16(to + q, z, p.dim - q, sectors);
                store16(to + q + 16, z + 16, p.dim - q - 16, sectors);
            }
            __syncwarp();
        }
    }
    if (kRole == kKeys && splits > 1) {
        // the cluster's sums, in the order of its CTAs; each finishes its share of the tile's rows
        __syncwarp();
        cluster_sync();
        const int low = kTile * rank / splits, share = kTile * (rank + 1) / splits - low, vecs = p.dim / 8;
        bool had = false, late = false;
        for (int r = 0; r < splits; ++r) {
            had |= load_cluster(cluster_addr(smem_u32(&found), r)) != 0;
            late |= load_cluster(cluster_addr(smem_u32(&gave_up), r)) != 0;
        }
        for (int i = threadIdx.x; i < 2 * vecs * share; i += kAttnThreads) {
            const int in = low + i % share, which = i / share % 2, c = i / share / 2 * 8;
            float z[8] = {};
            for (int r = 0; r < splits; ++r) {
                const uint32_t from = cluster_addr(smem_u32(part_at(base_ptr, which, c, in)), r);
                const float4 a = load_cluster_f4(from), b = load_cluster_f4(from + kTile * 16);
                z[0] += a.x, z[1] += a.y, z[2] += a.z, z[3] += a.w, z[4] += b.x, z[5] += b.y, z[6] += b.z, z[7] += b.w;
            }
            const int64_t row = tile.first + in;
            if (row >= tile.end) continue;
            if (late) z[0] = z[1] = z[2] = z[3] = z[4] = z[5] = z[6] = z[7] = __builtin_nanf("");
            if (which && had) add_cleared(p, tile, head, row, c, z);
            const HeadRows& o = which ? p.out1 : p.out0;
            store8(static_cast<uint16_t*>(o.p) + head * o.head + row * o.row + c, z[0], z[1], z[2], z[3], z[4], z[5], z[6], z[7]);
        }
        __syncwarp();
        cluster_sync();
    }
    tc_fence_before();
    __syncthreads();
    // every role has stopped; after a wait that ran out, what is in flight is waited for, bounded too
    if (*static_cast<volatile int*>(&gave_up)) {
        if (warp == 1 && elect_lane()) {
            mma_commit<1>(drained);
            mbar_drain(drained, 0);
        }
        if (warp == 0 && elect_lane()) {
            const int n = copied;
            mbar_drain(tile_full, 0);
            for (int i = max(0, n - kStages); i < n; ++i) mbar_drain(full + 8 * (i % kStages), i / kStages & 1);
        }
        __syncthreads();
    }
    tc_fence_after();
    if (warp == 2) tmem_free<1>(tmem, 512);
}

int injected_stall(int role) {
    const char* const names[2][2] = {{"stall_attention_dq_copy", "stall_attention_dq_softmax"}, {"stall_attention_dkv_copy", "stall_attention_dkv_softmax"}};
    return fault_injected(names[role][0]) ? kStallCopy : fault_injected(names[role][1]) ? kStallSoftmax : 0;
}

// CTAs that may share a tile of keys: more while all of them find place at one time.  (A cluster waits for as many free SMs as it
// has CTAs, those of little use among them: 8192 tokens in 16 sequences, 4 / 2 heads of 64, 164 units, 21 us with one CTA,
// 34 with two, 50 with eight; 1024 tokens, 16 / 2 heads of 128, 22 units, 175 us with one, 41 with four.)
int key_splits(const AttnCall& c) {
    const int64_t units = tile_slots(c.seq, kTile) * c.kv_heads, most = (c.seq.rows + kStep - 1) / kStep * (c.heads / c.kv_heads);
    int splits = 1;
    while (splits < 8 && 2 * units * splits <= sm_count() && most >= 2 * splits * kFewBlocks) splits *= 2;
    return splits;
}

template <int kRole, int kSteps>
int launch_role(const AttnCall& c, const HeadRows (&operands)[4], cudaStream_t s) {
    const bool queries = kRole == kQueries;
    CUtensorMap map[5] = {};
    for (int i = 0; i < (queries ? 5 : 4); ++i) {
        const HeadRows& t = i < 4 ? operands[i] : c.out;
        const bool own = i < 2 || i == 4;
        const int rc = make_head_map(&map[i], t.p, c.seq.rows, own == queries ? c.heads : c.kv_heads, c.dim, t.row, t.head, own ? kTile : kStep);
        if (rc) return rc;
    }
    static std::atomic<uint64_t> allowed{0};
    const int rc = allow_smem(k_attn_backward<kRole, kSteps>, (int)smem_of(kRole), allowed);
    if (rc) return rc;
    BackwardArgs a{};
    a.seq = c.seq;
    a.slots = tile_slots(c.seq, kTile), a.row_slots = tile_slots(c.seq, kStep);
    a.heads = (int)c.heads, a.kv_heads = (int)c.kv_heads, a.group = (int)(c.heads / c.kv_heads), a.dim = (int)c.dim;
    a.splits = queries ? 1 : key_splits(c);
    a.scale = c.scale;
    a.rows = static_cast<RowBlock*>(c.workspace);
    a.lse = c.lse;
    a.out0 = queries ? c.dq : c.dk, a.out1 = c.dv;
    a.d_out = static_cast<const uint16_t*>(c.d_out.p), a.lddo = c.d_out.row, a.hsdo = c.d_out.head;
    a.stall = faults_injected() ? injected_stall(kRole) : 0;
    a.wait_ns = a.stall ? kWaitNs / 40 : kWaitNs;
    return check_cuda(launch_after(k_attn_backward<kRole, kSteps>, (unsigned)(a.slots * (queries ? c.heads : c.kv_heads) * a.splits), kAttnThreads, smem_of(kRole), a.splits, s,
                                   map[0], map[1], map[2], map[3], map[4], a),
                      "attention backward launch");
}

}  // namespace

size_t attn_workspace_bytes(const AttnCall& c) { return (size_t)tile_slots(c.seq, kStep) * c.heads * sizeof(RowBlock); }

int launch_attn_backward(const AttnCall& c, cudaStream_t s) {
    const HeadRows keys[4] = {c.k, c.v, c.q, c.d_out}, queries[4] = {c.q, c.d_out, c.k, c.v};
    int rc = with_steps(c.dim, [&](auto steps) { return launch_role<kQueries, decltype(steps)::value>(c, queries, s); });   // delta too
    if (!rc && c.dk.p) rc = with_steps(c.dim, [&](auto steps) { return launch_role<kKeys, decltype(steps)::value>(c, keys, s); });
    return rc;
}

}  // namespace lmo
