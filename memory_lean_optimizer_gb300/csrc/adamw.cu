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
#include "internal.h"

namespace lmo {
namespace {

constexpr int kBlk = OPTIM_U8_BLOCK;   // 256: one warp, 8 elements per lane
static_assert(kBlk == 256, "a block is one warp's 32 x 8 elements");

struct AdamWPrm {
    float b1, omb1, b2, omb2, eps, lr_wd, k1, k2;
    const float* grad_scale;   // device scalar s, or NULL: 1
    int64_t step;
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

// Byte k of a word as a float, minus `bias` (2^23 plus the code's zero point).
template <int kB>
__device__ __forceinline__ float byte_to_f32(uint32_t word, float bias) {
    return __fsub_rn(__uint_as_float(__byte_perm(word, 0x4B000000u, 0x7440 | kB)), bias);
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
__device__ __forceinline__ uint32_t enc8_v(float v, float r) {
    const float y = fminf(sqrt_rn_z(__fmul_rn(sqrt_rn_z(v), r)), 255.0f);
    return __float_as_uint(__fadd_rn(12582912.0f, v == 0.0f ? 0.0f : fmaxf(y, 1.0f)));
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

// Each warp takes blocks of 256 elements of its CTA's chunk; a lane holds 8 consecutive ones.
// Elements past the tensor's end load as zero weight, gradient and state and are not stored (they
// cannot raise a block's maximum).
template <bool kSR, bool kU8>
__global__ void __launch_bounds__(kThreads) k_adamw_step(NadamLaunch L, AdamWPrm k) {
    __shared__ uint32_t red[32];
    const Chunk c = L.chunks[blockIdx.x];
    const TensorRec t = L.tensors[c.tensor];
    const uint16_t* __restrict__ g = L.grads[c.tensor];
    const bool has_res = (t.flags & kFlagRes) != 0;
    const bool u8 = kU8 && (t.flags & kFlagSmall) == 0;
    const int64_t n = t.numel;
    const int64_t start = (int64_t)c.index * L.chunk;
    const int64_t end = min(n, start + L.chunk);
    const float gs = k.grad_scale ? __ldg(k.grad_scale) : 1.0f;
    const bool aligned = aligned16(t.w) && (!has_res || aligned16(t.res)) && aligned16(g) && aligned16(t.m) &&
                         aligned16(t.v);
    uint8_t* const mc = static_cast<uint8_t*>(t.m);
    uint8_t* const vc = static_cast<uint8_t*>(t.v);
    float* const mq = u8 ? reinterpret_cast<float*>(mc + u8_scale_offset(n)) : nullptr;
    float* const vq = u8 ? reinterpret_cast<float*>(vc + u8_scale_offset(n)) : nullptr;
    uint32_t nf = 0u;
    const int lane = threadIdx.x & 31;
    for (int64_t b0 = start + (threadIdx.x >> 5) * kBlk; b0 < end; b0 += (kThreads / 32) * kBlk) {
        const int64_t i = b0 + 8 * lane;
        const int cnt = (int)max((int64_t)0, min((int64_t)8, end - i));
        const bool vec = aligned && cnt == 8;
        uint4 W = load8h(t.w, i, cnt, vec), G = load8h(g, i, cnt, vec);
        uint4 R = has_res ? load8h(t.res, i, cnt, vec) : make_uint4(0, 0, 0, 0);
        float m[8], v[8];
        if (u8) {
            dec8<true>(load8b(mc, i, cnt, vec), mq[b0 / kBlk], m);
            dec8<false>(load8b(vc, i, cnt, vec), vq[b0 / kBlk], v);
        } else {
            load8f(static_cast<const float*>(t.m), i, cnt, vec, m);
            load8f(static_cast<const float*>(t.v), i, cnt, vec, v);
        }
        uint32_t rnd[4] = {0u, 0u, 0u, 0u};
        if (kSR && !has_res) sr_block8(k.key, (uint64_t)k.step, c.tensor, i, rnd);
        uint32_t* w32 = reinterpret_cast<uint32_t*>(&W);
        uint32_t* r32 = reinterpret_cast<uint32_t*>(&R);
        const uint32_t g32[4] = {G.x, G.y, G.z, G.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int q = e >> 1, sh = 16 * (e & 1);
            const uint32_t hw = (w32[q] >> sh) & 0xFFFFu, lw = (r32[q] >> sh) & 0xFFFFu;
            float w = __uint_as_float((hw << 16) | lw);
            // past the end the codes' zero point is not zero: keep those lanes' states at zero
            if (kU8 && e >= cnt) m[e] = v[e] = 0.0f;
            adamw_elem(k, gs, w, bf16_to_f32((g32[q] >> sh) & 0xFFFFu), m[e], v[e]);
            uint32_t lo;
            const uint32_t hi = store_bits<kSR>(w, has_res, (rnd[q] >> sh) & 0xFFFFu, lo);
            w32[q] = (w32[q] & ~(0xFFFFu << sh)) | (hi << sh);
            r32[q] = (r32[q] & ~(0xFFFFu << sh)) | (lo << sh);
            if (e < cnt) nf = max(nf, hi & 0x7FFFu);
        }
        store8h(t.w, i, cnt, vec, W);
        if (has_res) store8h(t.res, i, cnt, vec, R);
        if (u8) {
            const float qm = __fmul_rn(__fsqrt_rn(block_top(m)), 1.0f / 127.0f);
            const float qv = __fmul_rn(__fsqrt_rn(__fsqrt_rn(block_top(v))), 1.0f / 255.0f);
            const float rm = code_factor(qm), rv = code_factor(qv);
            uint32_t cm[8], cv[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                cm[e] = enc8_m(m[e], rm);
                cv[e] = enc8_v(v[e], rv);
            }
            store8b(mc, i, cnt, vec, make_uint2(pack_byte0(cm), pack_byte0(cm + 4)));
            store8b(vc, i, cnt, vec, make_uint2(pack_byte0(cv), pack_byte0(cv + 4)));
            if (lane == 0) {
                mq[b0 / kBlk] = qm;
                vq[b0 / kBlk] = qv;
            }
        } else {
            store8f(static_cast<float*>(t.m), i, cnt, vec, m);
            store8f(static_cast<float*>(t.v), i, cnt, vec, v);
        }
    }
    uint32_t r[1] = {nf >= 0x7F80u ? 1u : 0u};
    block_max_u32<1>(r, red);
    if (threadIdx.x == 0 && r[0]) atomicAdd(L.nonfinite, 1ull);
}

// Moments of every tensor as fp32 values, into flat buffers (tensor i at 64 * slot64 elements).
template <bool kU8>
__global__ void __launch_bounds__(kThreads) k_adamw_unpack(NadamLaunch L, float* __restrict__ fm, float* __restrict__ fv) {
    const Chunk c = L.chunks[blockIdx.x];
    const TensorRec t = L.tensors[c.tensor];
    const bool u8 = kU8 && (t.flags & kFlagSmall) == 0;
    const int64_t n = t.numel;
    const int64_t start = (int64_t)c.index * L.chunk;
    const int64_t end = min(n, start + L.chunk);
    float* const om = fm + 64 * (int64_t)t.slot64;
    float* const ov = fv + 64 * (int64_t)t.slot64;
    const bool in16 = aligned16(t.m) && aligned16(t.v), out16 = aligned16(fm) && aligned16(fv);
    const uint8_t* mc = static_cast<const uint8_t*>(t.m);
    const uint8_t* vc = static_cast<const uint8_t*>(t.v);
    const float* mq = u8 ? reinterpret_cast<const float*>(mc + u8_scale_offset(n)) : nullptr;
    const float* vq = u8 ? reinterpret_cast<const float*>(vc + u8_scale_offset(n)) : nullptr;
    for (int64_t i = start + 8 * (int64_t)threadIdx.x; i < end; i += 8 * kThreads) {
        const int cnt = (int)min((int64_t)8, end - i);
        float m[8], v[8];
        if (u8) {
            dec8<true>(load8b(mc, i, cnt, in16 && cnt == 8), mq[i / kBlk], m);
            dec8<false>(load8b(vc, i, cnt, in16 && cnt == 8), vq[i / kBlk], v);
        } else {
            load8f(static_cast<const float*>(t.m), i, cnt, in16 && cnt == 8, m);
            load8f(static_cast<const float*>(t.v), i, cnt, in16 && cnt == 8, v);
        }
        store8f(om, i, cnt, out16 && cnt == 8, m);
        store8f(ov, i, cnt, out16 && cnt == 8, v);
    }
}

}  // namespace

int launch_adamw_step(const NadamLaunch& L, const AdamWScalars& s, bool u8, cudaStream_t stream) {
    if (L.n_chunks_total == 0) return OPTIM_OK;
    const AdamWPrm k{s.b1, s.omb1, s.b2, s.omb2, s.eps, s.lr_wd, s.k1, s.k2, s.grad_scale, s.step, philox_key(s.seed)};
    const unsigned grid = (unsigned)L.n_chunks_total;
    if (u8) {
        if (s.sr) k_adamw_step<true, true><<<grid, kThreads, 0, stream>>>(L, k);
        else k_adamw_step<false, true><<<grid, kThreads, 0, stream>>>(L, k);
    } else {
        if (s.sr) k_adamw_step<true, false><<<grid, kThreads, 0, stream>>>(L, k);
        else k_adamw_step<false, false><<<grid, kThreads, 0, stream>>>(L, k);
    }
    return check_cuda(cudaGetLastError(), "adamw step launch");
}

int launch_adamw_unpack(const NadamLaunch& L, bool u8, float* m, float* v, cudaStream_t stream) {
    if (L.n_chunks_total == 0) return OPTIM_OK;
    const unsigned grid = (unsigned)L.n_chunks_total;
    if (u8) k_adamw_unpack<true><<<grid, kThreads, 0, stream>>>(L, m, v);
    else k_adamw_unpack<false><<<grid, kThreads, 0, stream>>>(L, m, v);
    return check_cuda(cudaGetLastError(), "adamw unpack launch");
}

}  // namespace lmo
