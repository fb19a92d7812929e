// adamw.cu -- AdamW over the tensors of a group, states in fp32 or in 8 bits (OPTIM_KIND_ADAMW,
// OPTIM_KIND_ADAMW_U8).  One launch and one pass per element:
//   g' = s g;  m = b1 m + (1-b1) g';  v = b2 v + (1-b2) (g' g')
//   w = w - (lr wd) w;  w = w - (k1 m) / (sqrt(v) k2 + eps),  k1 = lr / (1-b1^t), k2 = 1 / sqrt(1-b2^t)
// every product, sum, root and quotient rounded once to fp32 (no multiply-add is fused here: the
// same sequence of elementary operations anywhere gives the same bits).
//
// 8-bit storage: the companded codec of the u16 states with 8-bit codes, and a scale for each block
// of 256 elements in place of one for each tensor, so that the scale is known to the warp that
// holds the block and no pass over the gradient comes first.  Per block q_m = sqrt(max |m|) / 127
// and q_v = max(v)^(1/4) / 255 (largest finite values), r = 1 / q^2;
//   code_m = 128 + sgn(m) rint(sqrt(|m| r_m)),  m = t |t|, t = (code_m - 128) q_m
//   code_v = rint(sqrt(sqrt(v) r_v)),           v = (z z)(z z), z = code_v q_v
// A positive v keeps a code of at least 1: decoded to zero, it would leave a kept m divided by eps
// alone in a later step whose gradient is zero.
//
// 278M elements, 8 bits with Kahan residuals: 690-730 us for 3.9 GB (5.4-5.7 TB/s), bound by instruction issue (67
// an element: the update's root and quotient, four code roots, their checks); a kernel that moves the same
// bytes and computes nothing takes 552 us.  120M elements with fp32 states: 467 us, at the copy rate.
// Without residuals 835 us (rounding to bf16 costs more than the residual's bytes), with stochastic
// rounding 853 us.  Blocks with an exact zero in a moment leave the fast path: one in every block 1.71 ms,
// nine elements in ten of all-zero blocks 1.55 ms.
#include "internal.h"
#include "launch.cuh"
#include "packed.cuh"

namespace lmo {
namespace {

constexpr int kBlk = OPTIM_U8_BLOCK;   // 256: one warp, 8 elements per lane
static_assert(kBlk == 256, "a block is one warp's 32 x 8 elements");

struct AdamWPrm {
    float b1, omb1, b2, omb2, eps, lr_wd, k1, k2;
    const float* grad_scale;   // device scalar s, or NULL: 1
    int64_t step;
    int32_t plain_range;       // k1, k2 and eps lie where the branch-free quotient holds (see Range)
    PhiloxKey key;
};

__device__ __forceinline__ void adamw_elem(const AdamWPrm& k, float gs, float& w, float g, float& m, float& v) {
    g = __fmul_rn(g, gs);
    m = __fadd_rn(__fmul_rn(k.b1, m), __fmul_rn(k.omb1, g));
    v = __fadd_rn(__fmul_rn(k.b2, v), __fmul_rn(k.omb2, __fmul_rn(g, g)));
    w = __fsub_rn(w, __fmul_rn(k.lr_wd, w));
    const float den = __fadd_rn(__fmul_rn(sqrt_rn_z(v), k.k2), k.eps);
    w = __fsub_rn(w, div_rn_z(__fmul_rn(k.k1, m), den));
}

// Stores the updated weight (Kahan split, stochastic rounding or RNE); returns the bf16 word.
template <bool kSR>
__device__ __forceinline__ uint32_t store_bits(float w1, bool has_res, uint32_t rnd, uint32_t& lo) {
    const uint32_t b = __float_as_uint(w1);
    lo = b & 0xFFFFu;
    if (has_res) return b >> 16;
    return kSR ? sr_bf16(w1, rnd) : rne_bf16(w1);
}

__device__ __forceinline__ int64_t u8_scale_offset(int64_t n) { return (n + 15) & ~(int64_t)15; }

// Byte k of a word in the mantissa of 2^23, and as a float, minus `bias` (2^23 plus the code's zero point).
template <int kB>
__device__ __forceinline__ float byte_in_2p23(uint32_t word) {
    return __uint_as_float(__byte_perm(word, 0x4B000000u, 0x7440 | kB));
}
template <int kB>
__device__ __forceinline__ float byte_to_f32(uint32_t word, float bias) {
    return __fsub_rn(byte_in_2p23<kB>(word), bias);
}
__device__ __forceinline__ float dec8_m(float c, float q) {
    const float t = __fmul_rn(c, q);
    return __fmul_rn(t, fabsf(t));
}
__device__ __forceinline__ float dec8_v(float c, float q) {
    const float z = __fmul_rn(c, q), z2 = __fmul_rn(z, z);
    return __fmul_rn(z2, z2);
}
// 8 codes (two words) decoded with a block's constant.
template <bool kSigned>
__device__ __forceinline__ void dec8(const uint2& c, float q, float (&x)[8]) {
    constexpr float bias = kSigned ? 8388736.0f : 8388608.0f;
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float f[4] = {byte_to_f32<0>(w[h], bias), byte_to_f32<1>(w[h], bias), byte_to_f32<2>(w[h], bias),
                            byte_to_f32<3>(w[h], bias)};
#pragma unroll
        for (int j = 0; j < 4; ++j) x[4 * h + j] = kSigned ? dec8_m(f[j], q) : dec8_v(f[j], q);
    }
}
// Encoders: the code is in the low byte of the returned word (rint by adding 1.5 * 2^23, plus 128
// for the first moment's zero point).
__device__ __forceinline__ uint32_t enc8_m(float m, float r) {
    const float y = fminf(sqrt_rn_z(__fmul_rn(fabsf(m), r)), 127.0f);
    return __float_as_uint(__fadd_rn(12583040.0f, copysignf(y, m)));
}
// sv = sqrt(v), shared with the update's denominator (zero for v = 0 alone).
__device__ __forceinline__ uint32_t enc8_v(float sv, float r) {
    const float y = fminf(sqrt_rn_z(__fmul_rn(sv, r)), 255.0f);
    return __float_as_uint(__fadd_rn(12582912.0f, sv == 0.0f ? 0.0f : fmaxf(y, 1.0f)));
}
__device__ __forceinline__ uint32_t pack_byte0(const uint32_t* b) {
    return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
}
__device__ __forceinline__ float code_factor(float q) {
    return q > 0.0f ? fminf(__fdiv_rn(1.0f, __fmul_rn(q, q)), FLT_MAX) : 0.0f;
}

// Largest finite magnitude of a block (8 values per lane).
__device__ __forceinline__ float block_top(const float (&x)[8]) {
    uint32_t top = 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7FFFFFFFu);
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if (top >= 0x7F800000u) {   // warp-uniform: an infinity or a NaN is among them
        top = 0u;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t b = __float_as_uint(x[e]) & 0x7FFFFFFFu;
            top = max(top, b < 0x7F800000u ? b : 0u);
        }
        top = __reduce_max_sync(0xFFFFFFFFu, top);
    }
    return __uint_as_float(top);
}

// 8 consecutive 16-bit words at element i of which `cnt` exist (vec: 16-byte aligned, all 8 do).
__device__ __forceinline__ uint4 load8h(const uint16_t* __restrict__ p, int64_t i, int cnt, bool vec) {
    if (vec) return ld_stream(reinterpret_cast<const uint4*>(p + i));
    uint32_t h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = e < cnt ? p[i + e] : 0u;
    return make_uint4(pack_lo16(h[0], h[1]), pack_lo16(h[2], h[3]), pack_lo16(h[4], h[5]), pack_lo16(h[6], h[7]));
}
__device__ __forceinline__ void store8h(uint16_t* __restrict__ p, int64_t i, int cnt, bool vec, const uint4& x) {
    if (vec) return st_stream(reinterpret_cast<uint4*>(p + i), x);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < cnt) p[i + e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
}
__device__ __forceinline__ uint2 load8b(const uint8_t* __restrict__ p, int64_t i, int cnt, bool vec) {
    if (vec) return __ldcs(reinterpret_cast<const uint2*>(p + i));
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < cnt) w[e >> 2] |= (uint32_t)p[i + e] << (8 * (e & 3));
    return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store8b(uint8_t* __restrict__ p, int64_t i, int cnt, bool vec, const uint2& x) {
    if (vec) return __stcs(reinterpret_cast<uint2*>(p + i), x);
    const uint32_t w[2] = {x.x, x.y};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < cnt) p[i + e] = (uint8_t)(w[e >> 2] >> (8 * (e & 3)));
}
__device__ __forceinline__ void load8f(const float* __restrict__ p, int64_t i, int cnt, bool vec, float (&x)[8]) {
    if (vec) {
        *reinterpret_cast<float4*>(x) = ld_stream(reinterpret_cast<const float4*>(p + i));
        *reinterpret_cast<float4*>(x + 4) = ld_stream(reinterpret_cast<const float4*>(p + i + 4));
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = e < cnt ? p[i + e] : 0.0f;
}
__device__ __forceinline__ void store8f(float* __restrict__ p, int64_t i, int cnt, bool vec, const float (&x)[8]) {
    if (vec) {
        st_stream(reinterpret_cast<float4*>(p + i), *reinterpret_cast<const float4*>(x));
        st_stream(reinterpret_cast<float4*>(p + i + 4), *reinterpret_cast<const float4*>(x + 4));
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < cnt) p[i + e] = x[e];
}

// What a warp needs to know about its CTA's tensor.
struct Tensor {
    uint16_t* w;
    uint16_t* res;
    const uint16_t* g;
    void* m;
    void* v;
    uint32_t index;
    bool has_res, u8;
};

// One block of 256 elements from b0, any alignment, any length: lane l holds elements b0 + 8l .. + 7.
// Elements past `end` load as zero weight, gradient and state and are not stored (they cannot raise
// a block's maximum).  8-bit states: qmv holds the block's constants, old in, new out.  Returns the largest
// exponent field stored.
template <bool kSR, bool kU8>
__device__ __forceinline__ uint32_t adamw_block(const AdamWPrm& k, const Tensor& t, float gs, int64_t b0, int64_t end, bool aligned,
                                             float2& qmv) {
    const int lane = threadIdx.x & 31;
    const int64_t i = b0 + 8 * lane;
    const int cnt = (int)max((int64_t)0, min((int64_t)8, end - i));
    const bool vec = aligned && cnt == 8;
    uint4 W = load8h(t.w, i, cnt, vec), G = load8h(t.g, i, cnt, vec);
    uint4 R = t.has_res ? load8h(t.res, i, cnt, vec) : make_uint4(0, 0, 0, 0);
    uint8_t* const mc = static_cast<uint8_t*>(t.m);
    uint8_t* const vc = static_cast<uint8_t*>(t.v);
    const bool u8 = kU8 && t.u8;
    float m[8], v[8];
    if (u8) {
        dec8<true>(load8b(mc, i, cnt, vec), qmv.x, m);
        dec8<false>(load8b(vc, i, cnt, vec), qmv.y, v);
    } else {
        load8f(static_cast<const float*>(t.m), i, cnt, vec, m);
        load8f(static_cast<const float*>(t.v), i, cnt, vec, v);
    }
    uint32_t rnd[4] = {0u, 0u, 0u, 0u};
    if (kSR && !t.has_res) sr_block8(k.key, (uint64_t)k.step, t.index, i, rnd);
    uint32_t* w32 = reinterpret_cast<uint32_t*>(&W);
    uint32_t* r32 = reinterpret_cast<uint32_t*>(&R);
    const uint32_t g32[4] = {G.x, G.y, G.z, G.w};
    uint32_t nf = 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int q = e >> 1, sh = 16 * (e & 1);
        float w = __uint_as_float(__byte_perm(r32[q], w32[q], e & 1 ? 0x7632 : 0x5410));
        // past the end the codes' zero point is not zero: keep those lanes' states at zero
        if (kU8 && e >= cnt) m[e] = v[e] = 0.0f;
        adamw_elem(k, gs, w, bf16_to_f32((g32[q] >> sh) & 0xFFFFu), m[e], v[e]);
        uint32_t lo;
        const uint32_t hi = store_bits<kSR>(w, t.has_res, (rnd[q] >> sh) & 0xFFFFu, lo);
        w32[q] = (w32[q] & ~(0xFFFFu << sh)) | (hi << sh);
        r32[q] = (r32[q] & ~(0xFFFFu << sh)) | (lo << sh);
        if (e < cnt) nf = max(nf, hi & 0x7FFFu);
    }
    store8h(t.w, i, cnt, vec, W);
    if (t.has_res) store8h(t.res, i, cnt, vec, R);
    if (u8) {
        const float qm = __fmul_rn(__fsqrt_rn(block_top(m)), 1.0f / 127.0f);
        const float qv = __fmul_rn(__fsqrt_rn(__fsqrt_rn(block_top(v))), 1.0f / 255.0f);
        const float rm = code_factor(qm), rv = code_factor(qv);
        uint32_t cm[8], cv[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            cm[e] = enc8_m(m[e], rm);
            cv[e] = enc8_v(sqrt_rn_z(v[e]), rv);
        }
        store8b(mc, i, cnt, vec, make_uint2(pack_byte0(cm), pack_byte0(cm + 4)));
        store8b(vc, i, cnt, vec, make_uint2(pack_byte0(cv), pack_byte0(cv + 4)));
        qmv = make_float2(qm, qv);
    } else {
        store8f(static_cast<float*>(t.m), i, cnt, vec, m);
        store8f(static_cast<float*>(t.v), i, cnt, vec, v);
    }
    return nf;
}

// a - b as b times -1 plus a: the product is exact, so the one rounding is the difference's.  Sums are
// written as differences from a negated operand, with a product only as b: a packed sum of products
// was seen to come out as one multiply-add in spite of .rn (a sixth of a million random cases of
// b1 m + omb1 g; none of them in this form).
__device__ __forceinline__ F2 sub2(F2 a, F2 b) {
    F2 r;
    const F2 minus = f2(-1.0f, -1.0f);
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.x) : "l"(b.x), "l"(minus.x), "l"(a.x));
    return r;
}
__device__ __forceinline__ float sqrt_approx(float x) {
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rsqrt_approx(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Root and quotient rounded to nearest without a branch, two at a time, by the multiply-add sequences of
// Markstein ("IA-64 and Elementary Functions", 2000): an approximate 1/sqrt(x) or 1/b refined once,
// then the exact remainder x - g^2 or a - b q added back.  Compared with __fsqrt_rn over every
// significand and both parities of the exponent, with the correctly rounded reciprocal over every
// significand, and with __fdiv_rn on 2e10 random pairs and the 1.7e7 pairs whose quotient is
// closest to the middle of two numbers: no difference.  The intermediate results must not leave the
// normal range, which Range states; CUDA's own have no such limit, but a branch each, and
// sixteen branches in a lane's block of eight keep its elements from overlapping.
struct Range {   // of v and |m|, given plain_range: 2^-30 <= k1 <= 2^20, 1 <= k2 <= 2^13, eps <= 1
    static constexpr float v_min = 0x1p-96f, v_max = 0x1p40f, m_min = 0x1p-60f, m_max = 0x1p20f;
};
// -sqrt(x) from nx = -x.
__device__ __forceinline__ F2 neg_sqrt2(F2 nx) {
    float a, b;
    split2(nx, a, b);
    const F2 y = f2(rsqrt_approx(-a), rsqrt_approx(-b)), half = f2(0.5f, 0.5f);
    F2 ng = mul2(nx, y), h = mul2(y, half);
    const F2 e = fma2(ng, h, half);
    ng = fma2(ng, e, ng);
    h = fma2(h, e, h);
    return fma2(fma2(ng, ng, nx), h, ng);
}
// (-a, sqrt(-b)): the first moment's constant takes one root, the second's two.
__device__ __forceinline__ F2 neg_sqrt2_second(float a, float b) {
    float drop, second;
    split2(neg_sqrt2(f2(b, b)), drop, second);
    return f2(-a, -second);
}
// a / b from nb = -b.
__device__ __forceinline__ F2 div2(F2 a, F2 nb) {
    float x, y;
    split2(nb, x, y);
    F2 r = f2(rcp_approx(-x), rcp_approx(-y));
    r = fma2(fma2(nb, r, f2(1.0f, 1.0f)), r, r);
    const F2 q = mul2(a, r);
    return fma2(fma2(nb, q, a), r, q);
}

// What one lane holds of a block between its loads and its arithmetic.
struct Raw {
    uint4 w, r, g;
    uint2 m, v;
};
// A ring of blocks for each warp in shared memory, kAhead of them on their way at a time without a register: a lane
// copies (cp.async) what it will read itself, so that waiting for its own copies is all the order there is.
constexpr int kRing = 3, kAhead = kRing - 1;
constexpr int kStageBytes = 8 * kBlk;   // w, residual, g: 512 bytes each; codes: 256 each
constexpr int kRingBytes = kThreads / 32 * kRing * kStageBytes;
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void fetch_block(uint32_t stage, const Tensor& t, int64_t b0) {
    const int lane = threadIdx.x & 31;
    const int64_t i = b0 + 8 * lane;
    copy16(stage + 16 * lane, t.w + i);
    copy16(stage + 512 + 16 * lane, t.g + i);
    if (t.has_res) copy16(stage + 1024 + 16 * lane, t.res + i);
    copy8(stage + 1536 + 8 * lane, static_cast<const uint8_t*>(t.m) + i);
    copy8(stage + 1792 + 8 * lane, static_cast<const uint8_t*>(t.v) + i);
}
__device__ __forceinline__ void read_block(Raw& x, const char* stage, const Tensor& t) {
    const int lane = threadIdx.x & 31;
    x.w = *reinterpret_cast<const uint4*>(stage + 16 * lane);
    x.g = *reinterpret_cast<const uint4*>(stage + 512 + 16 * lane);
    x.r = t.has_res ? *reinterpret_cast<const uint4*>(stage + 1024 + 16 * lane) : make_uint4(0, 0, 0, 0);
    x.m = *reinterpret_cast<const uint2*>(stage + 1536 + 8 * lane);
    x.v = *reinterpret_cast<const uint2*>(stage + 1792 + 8 * lane);
}

// A whole aligned block with 8-bit states: the results of adamw_block, two elements to an instruction
// where one exists.  The step moves 14 bytes an element, which leaves some 75 instructions an
// element (152 SMs at 1.9 GHz, 6.8 TB/s) before it is bound by their issue and not by memory, so three things are cut:
//  - the update's root and quotient have no branch (above).
//  - the codes' roots.  A code is the nearest integer to a root; an approximate root (relative error
//    2^-23 by the instruction's specification, 2^-24 the exact one's rounding: 4.6e-5 at 255) gives
//    the same integer unless it lies within 5e-5 of the middle between two, and only a lane that
//    has such a one (1 in 600) forms its eight codes from the exact roots.
//  - the block's constants.  Those of m and of v are the halves of one pair.
// A block with a moment outside Range (an exact zero, an infinity or a NaN among them) or a weight that comes
// out infinite or NaN is left to adamw_block as a whole: false, and nothing of it is stored.
template <bool kSR>
__device__ __forceinline__ bool adamw_block_fast(const AdamWPrm& k, const Tensor& t, float gs, int64_t b0, const Raw& x, float2& qmv) {
    const int lane = threadIdx.x & 31;
    const int64_t i = b0 + 8 * lane;
    const uint32_t wr[4] = {x.w.x, x.w.y, x.w.z, x.w.w}, rr[4] = {x.r.x, x.r.y, x.r.z, x.r.w};
    const uint32_t gr[4] = {x.g.x, x.g.y, x.g.z, x.g.w}, mr[2] = {x.m.x, x.m.y}, vr[2] = {x.v.x, x.v.y};
    const F2 qm2 = f2(qmv.x, qmv.x), qv2 = f2(qmv.y, qmv.y), gs2 = f2(gs, gs);
    const F2 b1 = f2(k.b1, k.b1), n_omb1 = f2(-k.omb1, -k.omb1), n_b2 = f2(-k.b2, -k.b2), omb2 = f2(k.omb2, k.omb2);
    const F2 wd = f2(k.lr_wd, k.lr_wd), k1 = f2(k.k1, k.k1), n_k2 = f2(-k.k2, -k.k2), n_eps = f2(-k.eps, -k.eps);
    uint32_t rnd[4] = {0u, 0u, 0u, 0u};
    if (kSR && !t.has_res) sr_block8(k.key, (uint64_t)k.step, t.index, i, rnd);
    float m[8], nsv[8];          // the new first moments, and minus the roots of the second
    float top_m = 0.0f, top_v = 0.0f, low_m = FLT_MAX, low_v = FLT_MAX, spill = 0.0f;
    F2 bad = f2(0.0f, 0.0f);     // 0 times the weights
    uint32_t wo[4], ro[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        // the pair's codes: byte 2 (q mod 2) and the next of word q / 2
        const uint32_t mw = mr[q >> 1], vw = vr[q >> 1];
        const F2 cm = q & 1 ? f2(byte_in_2p23<2>(mw), byte_in_2p23<3>(mw)) : f2(byte_in_2p23<0>(mw), byte_in_2p23<1>(mw));
        const F2 cv = q & 1 ? f2(byte_in_2p23<2>(vw), byte_in_2p23<3>(vw)) : f2(byte_in_2p23<0>(vw), byte_in_2p23<1>(vw));
        const F2 tm = mul2(sub2(cm, f2(8388736.0f, 8388736.0f)), qm2), tv = mul2(sub2(cv, f2(8388608.0f, 8388608.0f)), qv2);
        const F2 tv2 = mul2(tv, tv);
        float ta, tb, ma, mb, na, nb;
        split2(tm, ta, tb);
        split2(mul2(tm, tm), ma, mb);
        const F2 m0 = f2(copysignf(ma, ta), copysignf(mb, tb)), v0 = mul2(tv2, tv2);   // t |t|, (z z)(z z)
        const F2 g = mul2(f2(__uint_as_float(gr[q] << 16), __uint_as_float(gr[q] & 0xFFFF0000u)), gs2);
        const F2 m1 = sub2(mul2(b1, m0), mul2(n_omb1, g));
        const F2 nv = sub2(mul2(n_b2, v0), mul2(omb2, mul2(g, g)));                    // -v
        const F2 root = neg_sqrt2(nv);
        const F2 upd = div2(mul2(k1, m1), sub2(n_eps, mul2(root, n_k2)));
        F2 w = f2(__uint_as_float(__byte_perm(rr[q], wr[q], 0x5410)), __uint_as_float(__byte_perm(rr[q], wr[q], 0x7632)));
        w = sub2(sub2(w, mul2(wd, w)), upd);
        split2(m1, m[2 * q], m[2 * q + 1]);
        split2(root, nsv[2 * q], nsv[2 * q + 1]);
        split2(nv, na, nb);
        top_m = fmaxf(top_m, fmaxf(fabsf(m[2 * q]), fabsf(m[2 * q + 1])));
        low_m = fminf(low_m, fminf(fabsf(m[2 * q]), fabsf(m[2 * q + 1])));
        top_v = fmaxf(top_v, fmaxf(-na, -nb));
        low_v = fminf(low_v, fminf(-na, -nb));
        float wa, wb;
        split2(w, wa, wb);
        bad = fma2(w, f2(0.0f, 0.0f), bad);
        if (t.has_res) {
            wo[q] = pack_hi16(__float_as_uint(wa), __float_as_uint(wb));
            ro[q] = pack_lo16(__float_as_uint(wa), __float_as_uint(wb));
        } else {
            uint32_t lo;
            wo[q] = pack_lo16(store_bits<kSR>(wa, false, rnd[q] & 0xFFFFu, lo), store_bits<kSR>(wb, false, rnd[q] >> 16, lo));
            ro[q] = 0u;
            // rounding to bf16 can carry a finite weight to infinity
            if ((wo[q] & 0x7F80u) == 0x7F80u || (wo[q] & 0x7F800000u) == 0x7F800000u) spill = 1.0f;
        }
    }
    // minima and maxima pass over a NaN, but it reaches the weight
    float bad_a, bad_b;
    split2(bad, bad_a, bad_b);
    const bool plain = k.plain_range && low_v >= Range::v_min && top_v <= Range::v_max && low_m >= Range::m_min &&
                       top_m <= Range::m_max && bad_a + bad_b == 0.0f && spill == 0.0f;
    if (!__all_sync(0xFFFFFFFFu, plain)) return false;
    st_stream(reinterpret_cast<uint4*>(t.w + i), make_uint4(wo[0], wo[1], wo[2], wo[3]));
    if (t.has_res) st_stream(reinterpret_cast<uint4*>(t.res + i), make_uint4(ro[0], ro[1], ro[2], ro[3]));

    top_m = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top_m)));
    top_v = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top_v)));
    // the constants of both moments side by side, by the same branch-free root and quotient (their range holds)
    float root_m, root_v, rm, rv;
    split2(neg_sqrt2(f2(-top_m, -top_v)), root_m, root_v);
    const F2 q0 = mul2(neg_sqrt2_second(root_m, root_v), f2(1.0f / 127.0f, 1.0f / 255.0f));
    split2(div2(f2(1.0f, 1.0f), mul2(mul2(q0, q0), f2(-1.0f, -1.0f))), rm, rv);
    uint32_t cm[8], cv[8];
    float off = 0.0f;
    const F2 zero_m = f2(12583040.0f, 12583040.0f), zero_v = f2(12582912.0f, 12582912.0f);   // 1.5 * 2^23 (+ 128)
    const F2 n_zero_m = f2(-12583040.0f, -12583040.0f), n_zero_v = f2(-12582912.0f, -12582912.0f);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        float xa, xb, ya, yb;
        split2(mul2(f2(m[e], m[e + 1]), f2(rm, rm)), xa, xb);
        const F2 y = f2(copysignf(sqrt_approx(fabsf(xa)), xa), copysignf(sqrt_approx(fabsf(xb)), xb));
        F2 c = sub2(y, n_zero_m);
        split2(c, xa, xb);
        cm[e] = __float_as_uint(xa);
        cm[e + 1] = __float_as_uint(xb);
        split2(sub2(y, sub2(c, zero_m)), ya, yb);
        off = fmaxf(off, fmaxf(fabsf(ya), fabsf(yb)));
        split2(mul2(f2(nsv[e], nsv[e + 1]), f2(rv, rv)), xa, xb);
        const F2 z = f2(fmaxf(sqrt_approx(fabsf(xa)), 1.0f), fmaxf(sqrt_approx(fabsf(xb)), 1.0f));   // v > 0 here
        c = sub2(z, n_zero_v);
        split2(c, xa, xb);
        cv[e] = __float_as_uint(xa);
        cv[e + 1] = __float_as_uint(xb);
        split2(sub2(z, sub2(c, zero_v)), ya, yb);
        off = fmaxf(off, fmaxf(fabsf(ya), fabsf(yb)));
    }
    if (off > 0.49995f) {
#pragma unroll 1
        for (int e = 0; e < 8; ++e) {   // rotated through the first place: no indexed registers
            const float me = m[0], se = -nsv[0];
#pragma unroll
            for (int j = 0; j < 7; ++j) m[j] = m[j + 1], nsv[j] = nsv[j + 1], cm[j] = cm[j + 1], cv[j] = cv[j + 1];
            cm[7] = enc8_m(me, rm);
            cv[7] = enc8_v(se, rv);
        }
    }
    __stcs(reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.m) + i), make_uint2(pack_byte0(cm), pack_byte0(cm + 4)));
    __stcs(reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.v) + i), make_uint2(pack_byte0(cv), pack_byte0(cv + 4)));
    split2(q0, qmv.x, qmv.y);
    return true;
}

// Each warp takes a run of blocks of its CTA's chunk.  With 8-bit states lane j holds the constants of the run's
// j-th block from before the first to after the last -- one load and one store of neighbours (read
// and written block by block, 4 bytes in a sector that other warps write too, they cost more than
// all the other traffic: 1494 against 595 us at 278M parameters) -- and the whole aligned
// blocks go through adamw_block_fast, the next two on their way while one is computed.
template <bool kSR, bool kU8>
__global__ void __launch_bounds__(kThreads, 3) k_adamw_step(NadamLaunch L, AdamWPrm k) {
    extern __shared__ __align__(16) char ring[];   // kU8: kRingBytes
    __shared__ int counted;
    pdl_sync();
    if (threadIdx.x == 0) counted = 0;
    __syncthreads();
    const Chunk c = L.chunks[blockIdx.x];
    const TensorRec rec = L.tensors[c.tensor];
    Tensor t;
    t.w = rec.w;
    t.res = rec.res;
    t.g = L.grads[c.tensor];
    t.m = rec.m;
    t.v = rec.v;
    t.index = c.tensor;
    t.has_res = (rec.flags & kFlagRes) != 0;
    t.u8 = kU8 && (rec.flags & kFlagSmall) == 0;
    const int64_t start = (int64_t)c.index * L.chunk, end = min(rec.numel, start + L.chunk);
    const float gs = k.grad_scale ? __ldg(k.grad_scale) : 1.0f;
    const bool aligned = aligned16(t.w) && (!t.has_res || aligned16(t.res)) && aligned16(t.g) && aligned16(t.m) &&
                         aligned16(t.v);
    const int lane = threadIdx.x & 31;
    const int run = (int)(L.chunk / kThreads * 32 / kBlk);           // blocks to a warp: 1 to 16
    const int64_t first = start + (int64_t)(threadIdx.x >> 5) * run * kBlk;
    const int blocks = (int)max((int64_t)0, min((int64_t)run, (end - first + kBlk - 1) / kBlk));
    float* const mq = reinterpret_cast<float*>(static_cast<uint8_t*>(t.m) + u8_scale_offset(rec.numel)) + first / kBlk + lane;
    float* const vq = reinterpret_cast<float*>(static_cast<uint8_t*>(t.v) + u8_scale_offset(rec.numel)) + first / kBlk + lane;
    float2 q = make_float2(0.0f, 0.0f);
    if (kU8 && t.u8 && lane < blocks) q = make_float2(*mq, *vq);
    uint32_t done = 0u;   // bit j: block j is finished
    if (kU8 && t.u8 && aligned) {
        const int whole = (int)((min(end, first + (int64_t)blocks * kBlk) - first) / kBlk);
        char* const stages = ring + (threadIdx.x >> 5) * kRing * kStageBytes;
        const uint32_t stages0 = (uint32_t)__cvta_generic_to_shared(stages);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (j < whole) fetch_block(stages0 + j * kStageBytes, t, first + (int64_t)j * kBlk);
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
        int at = 0;
        for (int j = 0; j < whole; ++j) {
            const int to = at + kAhead < kRing ? at + kAhead : at + kAhead - kRing;
            if (j + kAhead < whole) fetch_block(stages0 + to * kStageBytes, t, first + (int64_t)(j + kAhead) * kBlk);
            asm volatile("cp.async.commit_group;" ::: "memory");
            asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
            Raw x;
            read_block(x, stages + at * kStageBytes, t);
            if (++at == kRing) at = 0;
            float2 qj = make_float2(__shfl_sync(0xFFFFFFFFu, q.x, j), __shfl_sync(0xFFFFFFFFu, q.y, j));
            if (adamw_block_fast<kSR>(k, t, gs, first + (int64_t)j * kBlk, x, qj)) done |= 1u << j;
            if (lane == j) q = qj;
        }
    }
    uint32_t nf = 0u;
    for (int j = 0; j < blocks; ++j) {
        if (done >> j & 1u) continue;
        float2 qj = make_float2(__shfl_sync(0xFFFFFFFFu, q.x, j), __shfl_sync(0xFFFFFFFFu, q.y, j));
        nf = max(nf, adamw_block<kSR, kU8>(k, t, gs, first + (int64_t)j * kBlk, end, aligned, qj));
        if (lane == j) q = qj;
    }
    if (kU8 && t.u8 && lane < blocks) {
        *mq = q.x;
        *vq = q.y;
    }
    // once per chunk, without a barrier that would hold the CTA's warps for its slowest
    if (nf >= 0x7F80u && atomicExch(&counted, 1) == 0) atomicAdd(L.nonfinite, 1ull);
}

// Moments of every tensor as fp32 values, into flat buffers (tensor i at 64 * slot64 elements).
template <bool kU8>
__global__ void __launch_bounds__(kThreads) k_adamw_unpack(NadamLaunch L, float* __restrict__ fm, float* __restrict__ fv) {
    pdl_sync();
    const Chunk c = L.chunks[blockIdx.x];
    const TensorRec t = L.tensors[c.tensor];
    const bool u8 = kU8 && (t.flags & kFlagSmall) == 0;
    const int64_t n = t.numel;
    int64_t start = (int64_t)c.index * L.chunk;
    const int64_t end = min(n, start + L.chunk);
    float* const om = fm + 64 * (int64_t)t.slot64;
    float* const ov = fv + 64 * (int64_t)t.slot64;
    const bool in16 = aligned16(t.m) && aligned16(t.v), out16 = aligned16(fm) && aligned16(fv);
    const uint8_t* mc = static_cast<const uint8_t*>(t.m);
    const uint8_t* vc = static_cast<const uint8_t*>(t.v);
    const float* mq = u8 ? reinterpret_cast<const float*>(mc + u8_scale_offset(n)) : nullptr;
    const float* vq = u8 ? reinterpret_cast<const float*>(vc + u8_scale_offset(n)) : nullptr;
    // four elements a lane: a word of codes in, one 16-byte store of each moment, neighbours side by side
    if (u8 && in16 && out16) {
        const int64_t whole = start + (end - start) / 4 * 4;
#pragma unroll 4
        for (int64_t i = start + 4 * (int64_t)threadIdx.x; i < whole; i += 4 * kThreads) {
            float m[8], v[8];
            dec8<true>(make_uint2(__ldcs(reinterpret_cast<const uint32_t*>(mc + i)), 0u), mq[i / kBlk], m);
            dec8<false>(make_uint2(__ldcs(reinterpret_cast<const uint32_t*>(vc + i)), 0u), vq[i / kBlk], v);
            st_stream(reinterpret_cast<float4*>(om + i), make_float4(m[0], m[1], m[2], m[3]));
            st_stream(reinterpret_cast<float4*>(ov + i), make_float4(v[0], v[1], v[2], v[3]));
        }
        start = whole;
    }
    for (int64_t i = start + threadIdx.x; i < end; i += kThreads) {
        float m[8], v[8];
        if (u8) {
            dec8<true>(make_uint2(mc[i], 0u), mq[i / kBlk], m);
            dec8<false>(make_uint2(vc[i], 0u), vq[i / kBlk], v);
        } else {
            m[0] = __ldcs(static_cast<const float*>(t.m) + i);
            v[0] = __ldcs(static_cast<const float*>(t.v) + i);
        }
        om[i] = m[0];
        ov[i] = v[0];
    }
}

}  // namespace

int launch_adamw_step(const NadamLaunch& L, const AdamWScalars& s, bool u8, cudaStream_t stream) {
    if (L.n_chunks_total == 0) return OPTIM_OK;
    const bool plain_range = s.k1 >= 0x1p-30f && s.k1 <= 0x1p20f && s.k2 >= 1.0f && s.k2 <= 0x1p13f && s.eps <= 1.0f;
    const AdamWPrm k{s.b1, s.omb1, s.b2, s.omb2, s.eps, s.lr_wd, s.k1, s.k2, s.grad_scale, s.step, plain_range,
                     philox_key(s.seed)};
    // started while the stream's last kernel drains: a step and the unpacking after it are short for small groups
    auto kernel = u8 ? (s.sr ? k_adamw_step<true, true> : k_adamw_step<false, true>)
                     : (s.sr ? k_adamw_step<true, false> : k_adamw_step<false, false>);
    const int smem = u8 ? kRingBytes : 0;
    if (u8) {
        static std::atomic<uint64_t> allowed[2];
        const int rc = allow_smem(kernel, smem, allowed[s.sr ? 1 : 0]);
        if (rc) return rc;
    }
    return check_cuda(launch_after(kernel, L.n_chunks_total, kThreads, smem, 1, stream, L, k), "adamw step launch");
}

int launch_adamw_unpack(const NadamLaunch& L, bool u8, float* m, float* v, cudaStream_t stream) {
    if (L.n_chunks_total == 0) return OPTIM_OK;
    return check_cuda(launch_after(u8 ? k_adamw_unpack<true> : k_adamw_unpack<false>, L.n_chunks_total, kThreads, 0, 1, stream,
                                   L, m, v), "adamw unpack launch");
}

}  // namespace lmo
