// attn.cuh -- what the attention kernels share: where the packed sequences' tiles are, and their operands.
#pragma once

#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "launch.cuh"
#include "packed.cuh"
#include "tensor.cuh"
#include "tensor_map.h"

namespace lmo {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// The sequences of a call: rows cu[i] .. cu[i + 1] - 1 of its buffers, or (cu NULL) `n` of rows / n each.
struct Sequences {
    const int32_t* cu;
    int32_t n;
    int64_t rows;
    // Borders of n + 2 segments: the rows before the first sequence, the sequences, the rows behind the last.
    // Whatever cu holds, they lie within the buffers.
    __device__ __forceinline__ int64_t border(int i) const {
        if (i == 0) return 0;
        if (i == n + 2) return rows;
        if (!cu) return (int64_t)(i - 1) * (rows / n);
        return min(max((int64_t)__ldg(cu + i - 1), (int64_t)0), rows);
    }
};
// bf16 [rows][heads][dim], strides in elements.
struct HeadRows {
    void* p;
    int64_t row, head;
};
struct AttnCall {
    HeadRows q, k, v, out, d_out, dq, dk, dv;
    float* lse;
    Sequences seq;
    int64_t heads, kv_heads, dim;
    float scale;
    void* workspace;      // backward
};
// Calls f with the products' steps of 16 along a head, a constant of the kernels: tests of their number between the products cost more
// than products.  What lies past the head's end is zero.  Four, five, six and eight: 16384 tokens, 16 / 4 heads of 80, forward and
// backward, take 586 and 2167 us in five steps, 637 and 2391 in eight; heads of 96, 618 and 2269 in six, 674 and 2470 in eight.
template <class F>
int with_steps(int64_t dim, F f) {
    if (dim <= 64) return f(std::integral_constant<int, 4>());
    if (dim <= 80) return f(std::integral_constant<int, 5>());
    if (dim <= 96) return f(std::integral_constant<int, 6>());
    return f(std::integral_constant<int, 8>());
}
int launch_attn_forward(const AttnCall& c, cudaStream_t s);
int launch_attn_backward(const AttnCall& c, cudaStream_t s);
size_t attn_workspace_bytes(const AttnCall& c);

// Tiles of kRows rows start at each segment's start.  A segment's tiles are numbered from border / kRows + its
// number on: that leaves room for all of them and needs no pass over the segments before it.
inline int64_t tile_slots(const Sequences& s, int rows) { return s.rows / rows + s.n + 2; }

struct Tile {
    int segment;          // 0 and n + 1: no sequence, rows to be set to zero
    int64_t start, end;   // the segment's rows
    int64_t first;        // the tile's first row; no tile if it is `end` or behind it
};
// The tile of a slot.  All threads of the CTA call it, once; each probes one border a round (one round for as many
// segments as threads).
template <int kRows>
__device__ __forceinline__ Tile find_tile(const Sequences& s, int64_t slot) {
    __shared__ int64_t border[2];
    int lo = 0, count = s.n + 2;                      // segments lo .. lo + count - 1
    for (;;) {
        const int step = (count + (int)blockDim.x - 1) / (int)blockDim.x;
        const int i = (int)threadIdx.x * step;
        int64_t at = 0, next = 0;
        if (i < count) {
            at = s.border(lo + i);
            if (step == 1) next = s.border(lo + i + 1);
        }
        const int below = max(__syncthreads_count(i < count && at / kRows + (lo + i) <= slot), 1) - 1;
        if (step == 1 && (int)threadIdx.x == below) border[0] = at, border[1] = next;
        lo += below * step;
        count = min(step, count - below * step);
        if (step == 1) break;
    }
    __syncthreads();
    Tile t;
    t.segment = lo;
    t.start = border[0];
    t.end = max(border[1], t.start);
    t.first = t.start + (slot - (t.start / kRows + lo)) * kRows;
    if (t.first < t.start) t.first = t.end;           // borders that fall
    return t;
}

// One of q, k, v, d_out as a map of boxes of one head's rows, 64 elements wide (what lies past the head reads as zero).
inline int make_head_map(CUtensorMap* map, const void* base, int64_t rows, int64_t heads, int64_t dim, int64_t ld, int64_t hs, int box_rows) {
    EncodeFn fn = encode_fn();
    if (!fn) return set_error(OPTIM_ECUDA, "cuTensorMapEncodeTiled is not available");
    // a dimension of one element has no stride of its own
    if (heads == 1) hs = dim;
    if (rows == 1) ld = heads * dim;
    const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)hs * 2, (cuuint64_t)ld * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)box_rows};
    const CUresult r = encode_bf16_map(fn, map, 3, base, dims, strides, box);
    if (r != CUDA_SUCCESS)
        return set_error(OPTIM_ECUDA, "tensor map of %lld x %lld heads of %lld: error %d", (long long)rows, (long long)heads, (long long)dim, (int)r);
    return OPTIM_OK;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Sixteen elements of a row: a whole sector in one store where the row allows it.
__device__ __forceinline__ void store16(uint16_t* to, const float* x, int left, bool sectors) {
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = pack_bf16(x[2 * k], x[2 * k + 1]);
    if (sectors && left >= 16) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]),
                     "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        if (left > 0) *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
        if (left > 8) *reinterpret_cast<uint4*>(to + 8) = make_uint4(w[4], w[5], w[6], w[7]);
    }
}
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A tile's rows in shared memory: boxes of 64 elements (128 bytes) of kRows rows, one after the other.
// One box or two of a head's rows.
template <int kRows>
__device__ __forceinline__ void load_rows(uint32_t dst, const CUtensorMap* map, int dim, int head, int64_t row, uint32_t bar) {
    tma_load_3d(dst, map, 0, head, (int)row, bar);
    if (dim > 64) tma_load_3d(dst + kRows * 128, map, 64, head, (int)row, bar);
}

// Zeroes the infinities and NaN of a tile in shared memory, thread `i` in row i, for a product with weights of which
// some are masked: 0 times those is NaN.  True if there was any (then the thread's stores are made visible to the tensor cores).
// Rows lie 128 bytes apart, so the threads of a warp start at different banks.  (Eight loads at a time: one by one, each with its test, a
// row of 128 elements took 1900 cycles, more than the softmax that it ends.)
__device__ __forceinline__ uint32_t non_finite(uint32_t w) {      // an exponent of ones and the bit below it make a carry into the sign's place
    return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
}
template <int kRows>
__device__ __forceinline__ bool clear_non_finite(char* tile, int dim, int i) {
    bool any = false;
    for (int box = 0; box < (dim > 64 ? 2 : 1); ++box) {
        char* const row = tile + box * kRows * 128 + i * 128;
        uint4 v[8];
        uint32_t bad = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = *reinterpret_cast<const uint4*>(row + ((q + i) & 7) * 16);
#pragma unroll
        for (int q = 0; q < 8; ++q) bad |= non_finite(v[q].x) | non_finite(v[q].y) | non_finite(v[q].z) | non_finite(v[q].w);
        if (bad) {
            any = true;
            auto finite = [](uint32_t w) { return w & ~((non_finite(w) >> 15) * 0xFFFFu); };
#pragma unroll 1
            for (int q = 0; q < 8; ++q) {
                uint4* const at = reinterpret_cast<uint4*>(row + q * 16);
                const uint4 x = *at;
                *at = make_uint4(finite(x.x), finite(x.y), finite(x.z), finite(x.w));
            }
        }
    }
    if (any) smem_to_async();
    return any;
}

// What clear_non_finite took out of rows a..b-1 (elements c .. c + N - 1 of a head), added to sums whose weights are positive.
template <int N>
__device__ __forceinline__ void add_non_finite(float (&x)[N], const uint16_t* base, int64_t ld, int64_t a, int64_t b, int c, int dim) {
    for (int64_t r = a; r < b; ++r)
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (c + k < dim) {
                const uint32_t h = base[r * ld + c + k];
                if ((h & 0x7F80u) == 0x7F80u) x[k] += bf16_to_f32(h);
            }
}

}  // namespace lmo
