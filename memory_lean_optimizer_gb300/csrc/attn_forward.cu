// attn_forward.cu -- causal attention over packed sequences, grouped heads, forward.
//   s_ij = scale q_i k_j (j <= i, of i's sequence),  lse_i = log sum_j exp s_ij,  o_i = sum_j exp(s_ij - lse_i) v_j
// One pass over the keys with a running reference m and sum (Milakov and Gimelshein, Online normalizer calculation for softmax, 2018): p_ij = 2^(s_ij
// log2 e - m), o and the sum are in units of 2^m.
//
// A CTA takes 256 rows of one head as two tiles of 128, which share the keys' and values' blocks of 128 rows
// in shared memory.  Scores and outputs are accumulators in tensor memory (2 x 128 and 2 x 128 columns, all 512); a
// thread of a tile's four softmax warps holds one row's 128 scores, so that maxima and sums need no other
// thread.  P goes back, in bf16, into the first half of its scores' columns (heads of up to 64: into columns of its own)
// and is the A operand of P V from there.
// The tensor cores work in the order P0 V, Q0 K', P1 V, Q1 K' (K' the next block; heads of up to 64: Q0 K', Q1 K', P0 V, P1 V): while they
// serve one tile, the other's softmax runs.  P in bf16: the tensor cores want both operands of one type; the sum is of the fp32 values.
//
// m follows the running maximum only when that has grown by 8 (p then stays below 2^8, far from any limit of fp32 or
// bf16): the outputs in tensor memory are rescaled a few times a row, not once a block.
//
// Heads of 128: the tensor cores bound it, and their power.  16384 tokens, 16 / 4 heads of 128: 0.65 ms (1.69 PFLOP/s; a library product in a
// burst 1.93); 32768: 2.69 ms (1.63).
// Heads of up to 64 have room for P beside its scores, so that the next scores are there when a softmax ends (kApart).  16384 tokens in one sequence
// 540 us (P over its scores: 557), in sequences of 1024 81 us (97), of 256 64 us (67).  What bounds them is the softmax: two warps share a
// scheduler, and the pair of tiles takes 2500 cycles a block of keys where its arithmetic alone takes 1450 (1024 of them exponentials, a quarter of
// a warp a cycle), with its waits and arrivals 1700 to 1950, and the products 1024.  A warp of its own for each tile's products gained nothing (561).
// Short sequences: a tile's chain of steps (the tile looked up 0.7 us, copies and scores 1.3, softmax 1.5, product 0.4, output 0.9).  64
// sequences of 512, 8 heads of 128: 89 us.  CTAs that take over units that have not started, so that one's end lies beside the next one's
// beginning, gained nothing there and lost 3 % of the long ones.
#include "attn.cuh"

namespace lmo {
namespace {

constexpr int kTile = 128;                       // rows of a tile, keys of a block
constexpr int kAttnThreads = 384;                   // warp 0 copies, warp 1 multiplies, warp 2 holds tensor memory; 4-7 and 8-11: a tile each
constexpr uint32_t kTileBytes = kTile * 256;     // 128 elements of bf16 to a row
constexpr int kStages = 2;
constexpr size_t kSmem = (2 + 2 * kStages) * kTileBytes + 1024;
constexpr float kSlack = 8.0f;

struct ForwardArgs {
    Sequences seq;
    int64_t slots;
    int32_t heads, group, dim;     // group: query heads to a key head
    float scale;
    uint16_t* out;
    int64_t ldo, hso;
    float* lse;                    // [heads][rows]
    const uint16_t* v;
    int64_t ldv, hsv;
    uint64_t wait_ns;
    int32_t stall;                 // tests of the waits' limit: what the first sequence's first tile of head 0 withholds (Stall), or 0
};
enum Stall { kStallCopy = 1, kStallSoftmax = 2 };

template <int kSteps>
__global__ void __launch_bounds__(kAttnThreads, 1) k_attn_forward(const __grid_constant__ CUtensorMap map_q,
                                                               const __grid_constant__ CUtensorMap map_k,
                                                               const __grid_constant__ CUtensorMap map_v, const ForwardArgs p) {
    extern __shared__ uint8_t smem_raw[];
    constexpr bool kApart = kSteps <= 4;           // P beside its scores: 2 x 128 columns of scores, 2 x 64 of P, 2 x 64 of outputs
    constexpr uint32_t kP = kApart ? 256 : 0, kO = kApart ? 384 : 256, kTileP = kApart ? 64 : 128, kTileO = kApart ? 64 : 128;
    __shared__ uint64_t bars[2 + 4 * kStages + 8 + 1];
    __shared__ uint32_t tmem_base;
    __shared__ int gave_up, found[2], copied[2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // before anything of the stream is needed
    const uint32_t q_full = smem_u32(bars), k_full = q_full + 16, k_empty = k_full + 8 * kStages, v_full = k_empty + 8 * kStages,
                   v_empty = v_full + 8 * kStages, s_done = v_empty + 8 * kStages, p_ready = s_done + 16, o_done = p_ready + 16,
                   s_free = o_done + 16, drained = s_free + 16;
    if (threadIdx.x == 0) {
        gave_up = 0;
        found[0] = found[1] = copied[0] = copied[1] = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full + 8 * i, 1);
            mbar_init(s_done + 8 * i, 1);
            mbar_init(p_ready + 8 * i, 4);
            mbar_init(o_done + 8 * i, 1);
            mbar_init(s_free + 8 * i, 4);
        }
        for (int i = 0; i < kStages; ++i) {
            mbar_init(k_full + 8 * i, 1);
            mbar_init(k_empty + 8 * i, 1);
            mbar_init(v_full + 8 * i, 1);
            mbar_init(v_empty + 8 * i, 1);
        }
        mbar_init(drained, 1);
        mbar_init_fence();
        tma_prefetch_map(&map_q);
        tma_prefetch_map(&map_k);
        tma_prefetch_map(&map_v);
    }
    if (warp == 2) tmem_alloc<1>(smem_u32(&tmem_base), 512);
    tc_fence_before();
    pdl_sync();
    const int head = (int)(blockIdx.x % (unsigned)p.heads);
    // later tiles see more keys: they come first
    const Tile tile = find_tile<2 * kTile>(p.seq, p.slots - 1 - blockIdx.x / (unsigned)p.heads);   // a barrier of the CTA too
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    if (tile.first >= tile.end) {
        if (warp == 2) tmem_free<1>(tmem, 512);
        return;
    }
    uint16_t* const out = p.out + head * p.hso;
    float* const lse = p.lse + (int64_t)head * p.seq.rows;
    if (tile.segment == 0 || tile.segment == p.seq.n + 1) {   // rows of no sequence
        const int rows = (int)min((int64_t)(2 * kTile), tile.end - tile.first), vecs = p.dim / 8;
        for (int i = threadIdx.x; i < rows * vecs; i += kAttnThreads)
            *reinterpret_cast<uint4*>(out + (tile.first + i / vecs) * p.ldo + i % vecs * 8) = make_uint4(0, 0, 0, 0);
        for (int i = threadIdx.x; i < rows; i += kAttnThreads) lse[tile.first + i] = 0.0f;
        if (warp == 2) tmem_free<1>(tmem, 512);
        return;
    }

    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    char* const base_ptr = reinterpret_cast<char*>(smem_raw) + (base - smem_u32(smem_raw));
    const uint32_t q_tile = base, k_tile = base + 2 * kTileBytes, v_tile = k_tile + kStages * kTileBytes;
    auto wait = [&](uint32_t bar, uint32_t parity) { return mbar_wait<1>(bar, parity, &gave_up, p.wait_ns); };

    const int left = (int)min(tile.end - tile.first, (int64_t)(2 * kTile));     // rows of the two tiles
    const int before = (int)((tile.first - tile.start) / kTile);                // blocks of keys before the first tile's own
    const int n0 = before + 1, n1 = left > kTile ? before + 2 : 0;              // blocks that the tiles see
    const int blocks = max(n0, n1);

    const int stall = head == 0 && tile.segment == 1 && tile.first == tile.start ? p.stall : 0;

    if (warp < 4) {
        regs_down<72>();
        if (warp == 0 && elect_lane()) {
            const int stop = stall == kStallCopy ? 0 : 0x7FFFFFFF;
            const int kv = head / p.group;
            const uint32_t boxes = p.dim > 64 ? 2 : 1;
            for (int t = 0; t < (n1 ? 2 : 1); ++t) {
                mbar_expect_tx(q_full + 8 * t, boxes * kTile * 128);
                load_rows<kTile>(q_tile + t * kTileBytes, &map_q, p.dim, head, tile.first + t * kTile, q_full + 8 * t);
            }
            int copied_k = 0, copied_v = 0;
            bool ok = true;
            for (int j = 0; ok && j < blocks; ++j) {
                const int stage = j % kStages;
                const uint32_t phase = j / kStages & 1;
                ok = copied_v != stop && wait(k_empty + 8 * stage, phase ^ 1u);
                if (!ok) break;
                mbar_expect_tx(k_full + 8 * stage, boxes * kTile * 128);
                load_rows<kTile>(k_tile + stage * kTileBytes, &map_k, p.dim, kv, tile.start + (int64_t)j * kTile, k_full + 8 * stage);
                ++copied_k;
                ok = wait(v_empty + 8 * stage, phase ^ 1u);
                if (!ok) break;
                mbar_expect_tx(v_full + 8 * stage, boxes * kTile * 128);
                load_rows<kTile>(v_tile + stage * kTileBytes, &map_v, p.dim, kv, tile.start + (int64_t)j * kTile, v_full + 8 * stage);
                ++copied_v;
            }
            // the last stages come back before the CTA ends: nothing arrives on its barriers after that
            for (int j = max(0, blocks - kStages); ok && j < blocks; ++j)
                ok = wait(k_empty + 8 * (j % kStages), j / kStages & 1) && wait(v_empty + 8 * (j % kStages), j / kStages & 1);
            copied[0] = copied_k, copied[1] = copied_v;
        } else if (warp == 1 && elect_lane()) {
            constexpr uint32_t desc_s = mma_desc(128, kTile, false, false), desc_o = mma_desc(128, kSteps * 16, false, true);
            bool ok = true;
            constexpr uint32_t up = desc_upper(1024);
            const uint32_t q_lo = desc_lower(q_tile, 8192), k_lo = desc_lower(k_tile, 8192), v_lo = desc_lower(v_tile, kTile * 128);
            auto scores = [&](int t, int j) {                                   // S_t = Q_t K_j'
                const uint32_t a = q_lo + t * (kTileBytes >> 4), b = k_lo + j % kStages * (kTileBytes >> 4);
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    const uint32_t off = (i >> 2) * (kTile * 8) + (i & 3) * 2;
                    mma_ss(tmem + t * 128, a + off, b + off, up, desc_s, i == 0);
                }
                mma_commit<1>(s_done + 8 * t);
            };
            ok = wait(k_full, 0);
            for (int t = 0; ok && t < (n1 ? 2 : 1); ++t) {
                ok = wait(q_full + 8 * t, 0);
                if (!ok) break;
                tc_fence_after();
                scores(t, 0);
            }
            if (ok) mma_commit<1>(k_empty);
            for (int j = 0; ok && j < blocks; ++j) {
                const int stage = j % kStages, next = (j + 1) % kStages;
                ok = wait(v_full + 8 * stage, j / kStages & 1);
                if (ok && j + 1 < blocks) ok = wait(k_full + 8 * next, (j + 1) / kStages & 1);
                if (kApart && j + 1 < blocks) {
                    for (int t = 0; ok && t < 2; ++t) {
                        if (j + 1 >= (t ? n1 : n0)) continue;
                        ok = wait(s_free + 8 * t, j & 1);
                        if (!ok) break;
                        tc_fence_after();
                        scores(t, j + 1);
                    }
                    if (!ok) break;
                    mma_commit<1>(k_empty + 8 * next);
                }
                for (int t = 0; ok && t < 2; ++t) {
                    const int n = t ? n1 : n0;
                    if (j >= n) continue;
                    ok = wait(p_ready + 8 * t, j & 1);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int i = 0; i < kTile / 16; ++i)
                        mma_ts(tmem + kO + t * kTileO, tmem + kP + t * kTileP + i * 8, v_lo + stage * (kTileBytes >> 4) + i * 128, up, desc_o, i == 0 && j == 0);
                    mma_commit<1>(o_done + 8 * t);
                    if (!kApart && j + 1 < n) scores(t, j + 1);      // into the columns of P, behind the product that reads it
                }
                if (!ok) break;
                mma_commit<1>(v_empty + 8 * stage);
                if (!kApart && j + 1 < blocks) mma_commit<1>(k_empty + 8 * next);
            }
        }
        __syncwarp();
    } else {
        regs_up<216>();
        const int t = (warp >> 2) - 1, n = t ? n1 : n0;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t s_at = tmem + lanes + t * 128, p_at = tmem + lanes + kP + t * kTileP, o_at = tmem + lanes + kO + t * kTileO;
        const int in = 32 * (warp & 3) + lane;                                  // this thread's row of the tile
        const float c = p.scale * kLog2e;
        const F2 c2 = f2(c, c);
        float m = -INFINITY, sum = 0.0f;
        bool ok = true;
        for (int j = 0; j < n; ++j) {
            ok = wait(s_done + 8 * t, j & 1);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            tc_fence_after();
            uint32_t x[4][32];
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_load32(s_at + 32 * q, x[q]);
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_wait(x[q]);
            if (kApart) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_free + 8 * t);
            }
            if (j == n - 1) {      // the tile's own block: keys behind the row
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (q < (warp & 3)) continue;
                    const int seen = q == (warp & 3) ? lane : -1;
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (k > seen) x[q][k] = 0xFF800000u;
                }
            }
            float top[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                top[q] = __uint_as_float(x[q][0]);
#pragma unroll
                for (int k = 1; k < 32; ++k) top[q] = fmaxf(top[q], __uint_as_float(x[q][k]));
            }
            const float now = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * c;
            const bool grow = now > m + kSlack;
            if (kApart && j > 0) {      // the product that reads the last P
                ok = wait(o_done + 8 * t, (j - 1) & 1);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                tc_fence_after();
            }
            if (j == 0) {
                m = now;
            } else if (__any_sync(0xFFFFFFFFu, grow)) {
                const float f = grow ? exp2_approx(m - now) : 1.0f;
                if (grow) m = now;
                sum *= f;
                if (!kApart) {
                    ok = wait(o_done + 8 * t, (j - 1) & 1);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    tc_fence_after();
                }
#pragma unroll 1
                for (int q = 0; q < p.dim; q += 32) {
                    uint32_t o[32];
                    tmem_load32(o_at + q, o);
                    tmem_wait(o);
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                    tmem_store32(o_at + q, o);
                }
            }
            const float ref = m == -INFINITY ? 0.0f : m;      // all scores so far -inf: weights of 0
            const F2 ref2 = f2(-ref, -ref);
            F2 part[4] = {f2(0.0f, 0.0f), f2(0.0f, 0.0f), f2(0.0f, 0.0f), f2(0.0f, 0.0f)};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t w[32];
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        float a, b;
                        split2(fma2(f2(__uint_as_float(x[2 * h + q][k]), __uint_as_float(x[2 * h + q][k + 1])), c2, ref2), a, b);
                        a = exp2_approx(a), b = exp2_approx(b);
                        part[k / 2 & 3] = add2(part[k / 2 & 3], f2(a, b));
                        w[16 * q + k / 2] = pack_bf16(a, b);
                    }
                tmem_store32(p_at + 32 * h, w);
            }
            tmem_store_wait();
            float a, b;
            split2(add2(add2(part[0], part[1]), add2(part[2], part[3])), a, b);
            sum += a + b;
            if (j == n - 1) {      // values of masked keys are not multiplied, not even by 0
                ok = wait(v_full + 8 * (j % kStages), j / kStages & 1);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                if (clear_non_finite<kTile>(base_ptr + (v_tile - base) + j % kStages * kTileBytes, p.dim, in)) found[t] = 1;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0 && stall != kStallSoftmax) mbar_arrive(p_ready + 8 * t);
        }
        if (n) {
            ok = ok && wait(o_done + 8 * t, (n - 1) & 1) && *static_cast<volatile int*>(&gave_up) == 0;     // whoever gave up
            ok = __all_sync(0xFFFFFFFFu, ok);
            tc_fence_after();
            const int64_t row = tile.first + t * kTile + in;
            const bool live = row < tile.end;
            uint16_t* const to = out + row * p.ldo;
            const bool sectors = (reinterpret_cast<uintptr_t>(to) & 31u) == 0;
            const float inv = ok ? 1.0f / sum : __builtin_nanf("");
            if (live) lse[row] = ok ? (m + log2f(sum)) * kLn2 : __builtin_nanf("");
            // blocks whose values were cleared: the first tile's own (seen by both), the second's own
            const bool had0 = *static_cast<volatile int*>(&found[0]) != 0, had1 = t && *static_cast<volatile int*>(&found[1]) != 0;
#pragma unroll
            for (int h = 0; h < (kSteps + 3) / 4; ++h) {
                uint32_t o[2][32];
                tmem_load32(o_at + 64 * h, o[0]);
                tmem_load32(o_at + 64 * h + 32, o[1]);
                tmem_wait(o[0]);
                tmem_wait(o[1]);
                if (live) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int q = 64 * h + 32 * i;
                        float y[32];
#pragma unroll
                        for (int k = 0; k < 32; ++k) y[k] = __uint_as_float(o[i][k]) * inv;
                        if (had0 || had1) {
                            const uint16_t* const v = p.v + (int64_t)(head / p.group) * p.hsv;
                            if (had0) add_non_finite(y, v, p.ldv, tile.first, min(tile.first + kTile, row + 1), q, p.dim);
                            if (had1) add_non_finite(y, v, p.ldv, tile.first + kTile, row + 1, q, p.dim);
                        }
                        store16(to + q, y, p.dim - q, sectors);
                        store16(to + q + 16, y + 16, p.dim - q - 16, sectors);
                    }
                }
                __syncwarp();
            }
        }
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
            const int copied_k = copied[0], copied_v = copied[1];
            for (int t = 0; t < (n1 ? 2 : 1); ++t) mbar_drain(q_full + 8 * t, 0);
            for (int j = max(0, copied_k - kStages); j < copied_k; ++j) mbar_drain(k_full + 8 * (j % kStages), j / kStages & 1);
            for (int j = max(0, copied_v - kStages); j < copied_v; ++j) mbar_drain(v_full + 8 * (j % kStages), j / kStages & 1);
        }
        __syncthreads();
    }
    tc_fence_after();
    if (warp == 2) tmem_free<1>(tmem, 512);
}

int injected_stall() { return fault_injected("stall_attention_copy") ? kStallCopy : fault_injected("stall_attention_softmax") ? kStallSoftmax : 0; }

}  // namespace

template <int kSteps>
static int launch_steps(const AttnCall& c, cudaStream_t s) {
    CUtensorMap q, k, v;
    int rc = make_head_map(&q, c.q.p, c.seq.rows, c.heads, c.dim, c.q.row, c.q.head, kTile);
    if (!rc) rc = make_head_map(&k, c.k.p, c.seq.rows, c.kv_heads, c.dim, c.k.row, c.k.head, kTile);
    if (!rc) rc = make_head_map(&v, c.v.p, c.seq.rows, c.kv_heads, c.dim, c.v.row, c.v.head, kTile);
    static std::atomic<uint64_t> allowed{0};
    if (!rc) rc = allow_smem(k_attn_forward<kSteps>, (int)kSmem, allowed);
    if (rc) return rc;
    ForwardArgs a{};
    a.seq = c.seq;
    a.slots = tile_slots(c.seq, 2 * kTile);
    a.heads = (int)c.heads, a.group = (int)(c.heads / c.kv_heads), a.dim = (int)c.dim;
    a.scale = c.scale;
    a.out = static_cast<uint16_t*>(c.out.p), a.ldo = c.out.row, a.hso = c.out.head;
    a.lse = c.lse;
    a.v = static_cast<const uint16_t*>(c.v.p), a.ldv = c.v.row, a.hsv = c.v.head;
    a.stall = faults_injected() ? injected_stall() : 0;
    a.wait_ns = a.stall ? kWaitNs / 40 : kWaitNs;
    return check_cuda(launch_after(k_attn_forward<kSteps>, (unsigned)(a.slots * c.heads), kAttnThreads, kSmem, 1, s, q, k, v, a), "attention launch");
}

int launch_attn_forward(const AttnCall& c, cudaStream_t s) {
    return with_steps(c.dim, [&](auto steps) { return launch_steps<decltype(steps)::value>(c, s); });
}

}  // namespace lmo
