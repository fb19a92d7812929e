// rope.cu -- rotary positions: pairs of a head's elements turned by an angle that grows with the position.
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t) factor,  t = position * frequency of the pair
// The inverse (backward pass) turns by -t.  Angles are exact whatever the position: a pair's frequency
// comes as turns per position in 64-bit fixed point, so that the low 64 bits of the integer product
// position * turns are the angle's fraction of a turn, off by position * 2^-65 turns at most; sine and
// cosine are taken of what lies past the nearest quarter turn.  (In fp32 an angle of 10^5 radians is off by
// up to 4e-3.)
//
// Memory bounds it: every element is read once and written once, queries and keys in one launch, and the
// sines of a position are worked out once for all of its heads.  16384 tokens, 32 / 8 heads of 128, bf16: 57 us in halves (5.9 TB/s), 63
// interleaved (5.3); 5003 tokens, 12 / 3 heads of 80, fp32, half of each turned: 7.8 us (6.2).
#include <cuda_bf16.h>

#include <algorithm>

#include "internal.h"
#include "launch.cuh"

namespace lmo {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxTokens = 8;

struct RopeTensor {
    const void* x;
    void* y;
    int64_t ldx, ldy;      // elements from one token to the next
    int64_t hsx, hsy;      // and from one head to the next
    int32_t heads;
};
struct RopeArgs {
    RopeTensor t[2];
    const int64_t* positions;
    const uint64_t* turns;
    int64_t rows;
    int32_t dim, rotary, tokens;   // tokens to a CTA
    uint32_t per_head;             // 2^32 / units of a head, rounded up, where that finds the head of every unit; or 0
    float factor;
    bool inverse;
};

template <int kBytes>
struct Word;
template <>
struct Word<2> { using type = uint16_t; };
template <>
struct Word<4> { using type = uint32_t; };
template <>
struct Word<8> { using type = uint2; };
template <>
struct Word<16> { using type = uint4; };

__device__ __forceinline__ float value(uint16_t x) { return bf16_to_f32(x); }
__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ void put(uint16_t& to, float x) { to = __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
__device__ __forceinline__ void put(float& to, float x) { to = x; }

// V elements moved as one word.
template <class T, int V>
union Piece {
    typename Word<V * sizeof(T)>::type w;
    T e[V];
    __device__ __forceinline__ Piece() {}
};
template <class T, int V>
__device__ __forceinline__ Piece<T, V> load(const T* p) {
    Piece<T, V> r;
    r.w = *reinterpret_cast<const decltype(r.w)*>(p);
    return r;
}
template <class T, int V>
__device__ __forceinline__ void store(T* p, const Piece<T, V>& r) {
    *reinterpret_cast<decltype(r.w)*>(p) = r.w;
}

// A head is cut into units: first those that turn (two pieces of V elements half the rotated part
// apart, or one piece of V / 2 neighbouring pairs), then pieces that are copied.
template <class T, int V, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) k_rope(const RopeArgs p) {
    extern __shared__ float2 table[];      // [tokens][rotary / 2]: cosine and sine, times the factor
    pdl_sync();
    const int half = p.rotary / 2;
    const int64_t first = (int64_t)blockIdx.x * p.tokens;
    const int n = (int)min((int64_t)p.tokens, p.rows - first);
    for (int i = threadIdx.x; i < n * half; i += kRopeThreads) {
        const int token = i / half, j = i - token * half;
        const uint64_t turn = (uint64_t)p.positions[first + token] * p.turns[j];
        const uint64_t quarter = (turn + (1ull << 61)) >> 62;               // the nearest quarter turn
        const int64_t rest = (int64_t)(turn - (quarter << 62));             // within an eighth of a turn of it
        float s, c;
        sincospif((float)rest * 0x1p-63f, &s, &c);                          // half turns
        if (quarter & 1) {
            const float was = c;
            c = -s;
            s = was;
        }
        if (quarter & 2) c = -c, s = -s;
        if (p.inverse) s = -s;
        table[i] = make_float2(c * p.factor, s * p.factor);
    }
    __syncthreads();
    constexpr int kStep = !kInterleaved ? V : V > 1 ? V / 2 : 1;      // pairs to a unit
    const int turning = half / kStep, units = turning + (p.dim - p.rotary) / V;
    const int all = (p.t[0].heads + p.t[1].heads) * units;
    constexpr bool kSingles = kInterleaved && V == 1;                 // pairs that are not aligned to pairs
    struct Unit {
        const T* x;
        T* y;
        int pair;              // its first pair of the table, or -1: copied
        bool live;
        Piece<T, V> a, b;
    };
    // two units at a time, so that one's loads do not wait for the other's stores (50003 tokens, 12 / 3 heads of 80, fp32: 156 -> 78 us)
    int token = 0, rest = (int)threadIdx.x;                           // unit `rest` of that token
    for (;;) {
        Unit unit[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            Unit& w = unit[j];
            while (rest >= all) rest -= all, ++token;
            w.live = token < n;
            int head = p.per_head ? (int)__umulhi((uint32_t)rest, p.per_head) : rest / units;
            const int u = rest - head * units;
            const bool second = head >= p.t[0].heads;
            const RopeTensor& t = second ? p.t[1] : p.t[0];
            if (second) head -= p.t[0].heads;
            const int c = u >= turning ? p.rotary + (u - turning) * V : kSingles ? 2 * u : u * V;
            w.x = static_cast<const T*>(t.x) + (first + token) * t.ldx + head * t.hsx + c;
            w.y = static_cast<T*>(t.y) + (first + token) * t.ldy + head * t.hsy + c;
            w.pair = u >= turning ? -1 : token * half + u * kStep;
            if (w.live) {
                w.a = load<T, V>(w.x);
                if (w.pair >= 0 && (kSingles || !kInterleaved)) w.b = load<T, V>(w.x + (kSingles ? 1 : half));
            }
            rest += kRopeThreads;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            Unit& w = unit[j];
            if (!w.live) return;
            if (w.pair >= 0) {
                const float2* const cs = table + w.pair;
                if (kInterleaved && !kSingles) {
#pragma unroll
                    for (int k = 0; k + 1 < V; k += 2) {
                        const float2 r = cs[k / 2];
                        const float f = value(w.a.e[k]), g = value(w.a.e[k + 1]);
                        put(w.a.e[k], fmaf(f, r.x, -(g * r.y)));
                        put(w.a.e[k + 1], fmaf(g, r.x, f * r.y));
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < V; ++k) {
                        const float2 r = cs[k];
                        const float f = value(w.a.e[k]), g = value(w.b.e[k]);
                        put(w.a.e[k], fmaf(f, r.x, -(g * r.y)));
                        put(w.b.e[k], fmaf(g, r.x, f * r.y));
                    }
                    store<T, V>(w.y + (kSingles ? 1 : half), w.b);
                }
            }
            store<T, V>(w.y, w.a);
        }
    }
}

template <class T, int V, bool kInterleaved>
int rope_v(RopeArgs& a, cudaStream_t s) {
    a.tokens = (int)std::min<int64_t>(kMaxTokens, std::max<int64_t>(1, a.rows / ((int64_t)sm_count() * 8)));
    const uint64_t units = a.rotary / 2 / (!kInterleaved ? V : V > 1 ? V / 2 : 1) + (a.dim - a.rotary) / V;
    // x ceil(2^32 / u) / 2^32 has the quotient x / u as its whole part while x u < 2^32
    a.per_head = units > 1 && (uint64_t)(a.t[0].heads + a.t[1].heads) * units * units < (1ull << 32) ? (uint32_t)(((1ull << 32) + units - 1) / units) : 0;
    const int64_t grid = (a.rows + a.tokens - 1) / a.tokens;
    const size_t smem = (size_t)a.tokens * (a.rotary / 2) * sizeof(float2);
    return check_cuda(launch_after(k_rope<T, V, kInterleaved>, (unsigned)grid, kRopeThreads, smem, 1, s, a), "rotary launch");
}

// The widest unit that the sizes, strides and addresses allow.
template <class T>
int rope_t(RopeArgs& a, bool interleaved, cudaStream_t s) {
    uint64_t all = (uint64_t)a.dim | (uint64_t)a.rotary | (uint64_t)(interleaved ? 0 : a.rotary / 2);
    uint64_t bytes = 0;
    for (const RopeTensor& t : a.t) {
        if (!t.heads) continue;
        if (a.rows > 1) all |= (uint64_t)t.ldx | (uint64_t)t.ldy;
        if (t.heads > 1) all |= (uint64_t)t.hsx | (uint64_t)t.hsy;
        bytes |= reinterpret_cast<uintptr_t>(t.x) | reinterpret_cast<uintptr_t>(t.y);
    }
    int v = 16 / (int)sizeof(T);
    while (v > 1 && (all % v || bytes % (v * sizeof(T)))) v /= 2;
    if (interleaved) {
        if constexpr (sizeof(T) == 2)
            if (v == 8) return rope_v<T, 8, true>(a, s);
        if (v == 4) return rope_v<T, 4, true>(a, s);
        if (v == 2) return rope_v<T, 2, true>(a, s);
        return rope_v<T, 1, true>(a, s);
    }
    if constexpr (sizeof(T) == 2)
        if (v == 8) return rope_v<T, 8, false>(a, s);
    if (v == 4) return rope_v<T, 4, false>(a, s);
    if (v == 2) return rope_v<T, 2, false>(a, s);
    return rope_v<T, 1, false>(a, s);
}

}  // namespace
}  // namespace lmo

using namespace lmo;

static int check_rope_tensor(const char* name, const void* x, int64_t ldx, int64_t hsx, const void* y, int64_t ldy, int64_t hsy,
                             int64_t rows, int64_t heads, int64_t dim, size_t elem) {
    if (!x || !y) return set_error(OPTIM_EINVAL, "%s or its output is NULL", name);
    if (!is_aligned(x, elem) || !is_aligned(y, elem)) return set_error(OPTIM_EALIGN, "%s or its output not aligned to its elements", name);
    // the input may repeat rows or heads; places of the output must not meet
    if (ldx < 0 || hsx < 0 || (heads > 1 && hsy < dim) || (rows > 1 && ldy < (heads - 1) * hsy + dim && hsy < (rows - 1) * ldy + dim))
        return set_error(OPTIM_EINVAL, "%s: strides of %lld and %lld (output %lld and %lld) elements for heads of %lld", name,
                         (long long)ldx, (long long)hsx, (long long)ldy, (long long)hsy, (long long)dim);
    return OPTIM_OK;
}

extern "C" int rope_apply(const void* q, int64_t q_row, int64_t q_head, void* q_out, int64_t qo_row, int64_t qo_head, int64_t q_heads,
                          const void* k, int64_t k_row, int64_t k_head, void* k_out, int64_t ko_row, int64_t ko_head, int64_t k_heads,
                          const int64_t* positions, const uint64_t* turns, int64_t rows, int64_t dim, int64_t rotary, float factor,
                          int32_t interleaved, int32_t inverse, int32_t type, void* stream) {
    if (type != OPTIM_BF16 && type != OPTIM_F32) return set_error(OPTIM_EINVAL, "type must be OPTIM_BF16 or OPTIM_F32");
    if (rows < 0 || rows >= ((int64_t)1 << 31)) return set_error(OPTIM_EINVAL, "rows must lie in [0, 2^31)");
    if (dim < 1 || dim > 1024) return set_error(OPTIM_EINVAL, "a head must have 1 to 1024 elements");
    if (rotary < 0 || rotary > dim || rotary % 2) return set_error(OPTIM_EINVAL, "rotary must be even and at most dim");
    if (q_heads < 0 || k_heads < 0 || q_heads + k_heads > 65536) return set_error(OPTIM_EINVAL, "at most 65536 heads");
    if (!(factor >= -FLT_MAX && factor <= FLT_MAX)) return set_error(OPTIM_EINVAL, "factor is not finite");
    if (rows == 0 || q_heads + k_heads == 0) return OPTIM_OK;
    const size_t elem = type == OPTIM_BF16 ? 2 : 4;
    int rc = OPTIM_OK;
    if (q_heads) rc = check_rope_tensor("q", q, q_row, q_head, q_out, qo_row, qo_head, rows, q_heads, dim, elem);
    if (!rc && k_heads) rc = check_rope_tensor("k", k, k_row, k_head, k_out, ko_row, ko_head, rows, k_heads, dim, elem);
    if (rc) return rc;
    if (rotary && (!positions || !turns)) return set_error(OPTIM_EINVAL, "positions or turns is NULL");
    if (!is_aligned(positions, 8) || !is_aligned(turns, 8)) return set_error(OPTIM_EALIGN, "positions or turns not 8-byte aligned");
    RopeArgs a{{{q, q_out, q_row, qo_row, q_head, qo_head, (int32_t)q_heads}, {k, k_out, k_row, ko_row, k_head, ko_head, (int32_t)k_heads}},
               positions, turns, rows, (int32_t)dim, (int32_t)rotary, 0, 0, factor, inverse != 0};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return type == OPTIM_BF16 ? rope_t<uint16_t>(a, interleaved != 0, s) : rope_t<float>(a, interleaved != 0, s);
}
