// act.cu -- activation checkpoints in 8 bits, and the gated activation whose backward pass reads them.
//
// A row is cut into blocks of 32 elements; a block keeps one exponent byte E and 32 codes c from -127 to 127:
// x = c 2^(E - 133).  E is the smallest with which no element of the block rounds past 127 (E = 127 + the
// exponent of the largest magnitude, one more if that rounds to 128), so an element is off by half a
// step at most, and the largest is 63.75 steps at least: 1 / 127.5 of it (0.784 %).  (Below 2^-126 the step stays 2^-133; from 127.5 2^121 on it
// cannot grow, and the largest take the code 127, off by less than a step.)  Steps are powers of two: codes are exact roundings (to
// nearest even) whatever arithmetic forms them, and c 2^(E - 133) is exact in bf16 and fp32.  A block that holds
// an infinity or a NaN has E = 255 and comes back as NaN.
//
// The gated activation h = g s(g) u, s(g) = 1 / (1 + e^-g), keeps its two inputs in this form alone; its
// backward pass reads the codes and, with dh, gives
//   dg = dh u s(g) (1 + g (1 - s(g))),  du = dh g s(g),  and h again (for the next product's weight gradient).
//
// Memory bounds all four kernels: one reading, one writing, 16 elements to a thread (two threads a block).  16384 x 8192 bf16: packed in 69 us
// (5.9 TB/s), read back in 67 (6.1), the gated activation 178 us (6.1; CTAs of 256 threads: 187), its gradients 195 us (6.9, the last writes
// still in L2; with 64 registers a thread instead of the 48 that let ten CTAs on an SM: 205).  fp32: packed in 95 us, read back in 133 (5.1), the gated
// activation 266 us (7.1, again with writes still in L2), its gradients 427 (5.7).
#include <cuda_bf16.h>

#include <algorithm>

#include "internal.h"
#include "launch.cuh"
#include "packed.cuh"

namespace lmo {
namespace {

constexpr int kActThreads = 128;
constexpr int kBlock = 32, kPer = 16;      // elements that share an exponent; elements to a thread
constexpr uint32_t kNoExponent = 255;      // of a block with an infinity or a NaN

// A thread's sixteen elements, at `off` of a matrix, the first `n` of them there (the rest zero).  kVec: 16-byte aligned.
__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(w[i] << 16), f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
}
__device__ __forceinline__ float value(uint16_t x) { return bf16_to_f32(x); }
__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ void put(uint16_t* to, float x) { *to = __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
__device__ __forceinline__ void put(float* to, float x) { *to = x; }
__device__ __forceinline__ void load16_wide(const uint16_t* p, float (&f)[kPer]) {
    unpack8(reinterpret_cast<const uint4*>(p)[0], f);
    unpack8(reinterpret_cast<const uint4*>(p)[1], f + 8);
}
__device__ __forceinline__ void load16_wide(const float* p, float (&f)[kPer]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 a = reinterpret_cast<const float4*>(p)[i];
        f[4 * i] = a.x, f[4 * i + 1] = a.y, f[4 * i + 2] = a.z, f[4 * i + 3] = a.w;
    }
}
__device__ __forceinline__ void store16_wide(uint16_t* p, const float (&f)[kPer]) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}
__device__ __forceinline__ void store16_wide(float* p, const float (&f)[kPer]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) reinterpret_cast<float4*>(p)[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
}

// Rows off 16 bytes: sixteen single elements a thread would be 32 places far apart for every access of a warp.  Instead half a warp
// takes a thread's sixteen elements, next to each other, and they are turned round in 2 KiB of shared memory of the warp's own (fp32;
// 16-byte pieces of thread t at their number XOR t / 2 mod 4, so that neither side meets a bank twice).
// 5003 x 2047 fp32: packed in 10.3 us (single elements: 21), read back in 9.9 (44), the gated activation 36 (64), its gradients 52 (133).
struct Turn {
    float* smem;     // 512 floats of the warp
    int lane;
    __device__ __forceinline__ float* piece(int thread, int q) const { return smem + 16 * thread + 4 * (q ^ (thread >> 1 & 3)); }
    template <class T>
    __device__ __forceinline__ void load(const T* base, int64_t off, int n, float (&f)[kPer]) const {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int of = 2 * k + (lane >> 4), e = lane & 15;
            const int64_t at = __shfl_sync(0xFFFFFFFFu, off, of);
            const int have = __shfl_sync(0xFFFFFFFFu, n, of);
            piece(of, e >> 2)[e & 3] = e < have ? value(base[at + e]) : 0.0f;
        }
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float4 a = *reinterpret_cast<const float4*>(piece(lane, q));
            f[4 * q] = a.x, f[4 * q + 1] = a.y, f[4 * q + 2] = a.z, f[4 * q + 3] = a.w;
        }
        __syncwarp();
    }
    template <class T>
    __device__ __forceinline__ void store(T* base, int64_t off, int n, const float (&f)[kPer]) const {
#pragma unroll
        for (int q = 0; q < 4; ++q) *reinterpret_cast<float4*>(piece(lane, q)) = make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int of = 2 * k + (lane >> 4), e = lane & 15;
            const int64_t at = __shfl_sync(0xFFFFFFFFu, off, of);
            const int have = __shfl_sync(0xFFFFFFFFu, n, of);
            if (e < have) put(base + at + e, piece(of, e >> 2)[e & 3]);
        }
        __syncwarp();
    }
};
// All threads of a warp call these together.
template <bool kVec, class T>
__device__ __forceinline__ void load16(const Turn& turn, const T* base, int64_t off, int n, float (&f)[kPer]) {
    if (!kVec) {
        turn.load(base, off, n, f);
    } else if (n == kPer) {
        load16_wide(base + off, f);
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) f[i] = i < n ? value(base[off + i]) : 0.0f;
    }
}
template <bool kVec, class T>
__device__ __forceinline__ void store16(const Turn& turn, T* base, int64_t off, int n, const float (&f)[kPer]) {
    if (!kVec) {
        turn.store(base, off, n, f);
    } else if (n == kPer) {
        store16_wide(base + off, f);
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (i < n) put(base + off + i, f[i]);
    }
}
template <bool kVec>
__device__ __forceinline__ Turn turn_of() {
    __shared__ float4 smem[kVec ? 1 : kActThreads * kPer / 4];
    return {reinterpret_cast<float*>(smem) + (kVec ? 0 : threadIdx.x / 32 * 512), (int)(threadIdx.x & 31)};
}

// Codes of this thread's half of a block and the block's exponent.  Both threads of a block call it together.
__device__ __forceinline__ uint32_t encode(const float (&f)[kPer], uint4& codes) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) top = max(top, __float_as_uint(f[i]) & 0x7FFFFFFFu);   // bits of magnitudes order like them
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    if (top >= 0x7F800000u) {
        codes = make_uint4(0, 0, 0, 0);
        return kNoExponent;
    }
    uint32_t e = top >> 23;
    // rounds to 128: a mantissa of 1.9921875 or more; below 2^-126 there is no hidden one
    e += (top & 0x7FFFFFu) >= (e ? 0x7F0000u : 0x7F8000u);
    e = min(e, 254u);                       // magnitudes from 127.5 2^121 on keep the last step, code 127
    // x 2^(133 - e): in two factors, for the first alone may not exist
    const int k = 133 - (int)e, k1 = min(k, 127);
    const float s1 = __uint_as_float((uint32_t)(k1 + 127) << 23), s2 = __uint_as_float((uint32_t)(k - k1 + 127) << 23);
    // 1.5 2^23 + c holds c in its low byte: one rounding, to nearest even
    constexpr float kMagic = 12582912.0f;
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(fminf(fmaf(f[4 * q + i] * s1, s2, kMagic), kMagic + 127.0f));
        w[q] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    }
    if (e == 254u) {                        // the other end: -128 does not exist
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = __vmaxs4(w[q], 0x81818181u);
    }
    codes = make_uint4(w[0], w[1], w[2], w[3]);
    return e;
}

// The values of sixteen codes.
__device__ __forceinline__ void decode(const uint4& codes, uint32_t e, float (&f)[kPer]) {
    // 2^(e - 133); below 2^-126 a subnormal
    const float step = __uint_as_float(e == kNoExponent ? 0x7FFFFFFFu : e >= 7 ? (e - 6) << 23 : 1u << (e + 16));
    const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
    const F2 bias = f2(-8388736.0f, -8388736.0f), step2 = f2(step, step);    // 2^23 + 128
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint32_t b = w[q] ^ 0x80808080u;
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const F2 v = f2(__uint_as_float(__byte_perm(b, 0x4B000000u, 0x7440 + i)),
                            __uint_as_float(__byte_perm(b, 0x4B000000u, 0x7441 + i)));
            split2(mul2(add2(v, bias), step2), f[4 * q + i], f[4 * q + i + 1]);
        }
    }
}

// 1 / (1 + e^-g).  For bf16 outputs the hardware's approximate exponential and reciprocal (2^-22 of the value)
// lie far below the output's rounding; fp32 outputs take the full functions.  Gates below -87.3 give 0 in bf16 (s lies
// below fp32's normal values and the reciprocal flushes it), in fp32 those below -88.7 (1 + e^-g overflows).
template <class T>
__device__ __forceinline__ float sigmoid(float g) {
    if (sizeof(T) == 4) return __frcp_rn(1.0f + expf(-g));
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}

struct ActArgs {
    const void* in;          // x, gate and up, or dh
    int64_t ld_in;
    int8_t* codes;
    int64_t ldc;             // bytes from one row of codes to the next, a multiple of 32
    uint8_t* exponents;
    int64_t lde;
    void* out;               // x, h, or the gradients of gate and up
    int64_t ld_out;
    void* h;                 // backward: h again, or NULL
    int64_t ldh;
    uint32_t rows, per_row;  // threads to a row: 16 elements each, two a block
    int32_t cols;
};

// Where a thread's sixteen elements are; past the last row (both threads of a block alike) there are none.
struct Place {
    int64_t row;
    int col, n;              // first column, how many are there
    bool live;
    __device__ __forceinline__ Place(const ActArgs& p) {
        const uint64_t i = (uint64_t)blockIdx.x * kActThreads + threadIdx.x;
        const uint32_t r = i < 0xFFFFFFFFull ? (uint32_t)i / p.per_row : (uint32_t)(i / p.per_row);
        col = (int)(i - (uint64_t)r * p.per_row) * kPer;
        live = r < p.rows;
        row = live ? r : 0;
        n = live ? min(max(p.cols - col, 0), kPer) : 0;
    }
};
__device__ __forceinline__ uint4* code_at(const ActArgs& p, int64_t row, int col) {
    return reinterpret_cast<uint4*>(p.codes + row * p.ldc + col);
}

template <class T, bool kVec>
__global__ void __launch_bounds__(kActThreads) k_act_pack(const ActArgs p) {
    const Turn turn = turn_of<kVec>();
    pdl_sync();
    const Place at(p);
    float f[kPer];
    load16<kVec>(turn, static_cast<const T*>(p.in), at.row * p.ld_in + at.col, at.n, f);
    uint4 c;
    const uint32_t e = encode(f, c);
    if (!at.live) return;
    *code_at(p, at.row, at.col) = c;
    if (at.col % kBlock == 0) p.exponents[at.row * p.lde + at.col / kBlock] = (uint8_t)e;
}

template <class T, bool kVec>
__global__ void __launch_bounds__(kActThreads) k_act_unpack(const ActArgs p) {
    const Turn turn = turn_of<kVec>();
    pdl_sync();
    const Place at(p);
    if (kVec && !at.live) return;
    float f[kPer];
    decode(*code_at(p, at.row, at.live ? at.col : 0), p.exponents[at.row * p.lde + (at.live ? at.col / kBlock : 0)], f);
    store16<kVec>(turn, static_cast<T*>(p.out), at.row * p.ld_out + at.col, at.n, f);
}

// Rows 2r and 2r + 1 of the codes are the gate and the up part of row r.
template <class T, bool kVec>
__global__ void __launch_bounds__(kActThreads) k_swiglu_forward(const ActArgs p) {
    const Turn turn = turn_of<kVec>();
    pdl_sync();
    const Place at(p);
    float g[kPer], u[kPer];
    const int64_t from = at.row * p.ld_in + at.col;
    load16<kVec>(turn, static_cast<const T*>(p.in), from, at.n, g);
    load16<kVec>(turn, static_cast<const T*>(p.in), from + p.cols, at.n, u);
    if (p.codes) {
        uint4 cg, cu;
        const uint32_t eg = encode(g, cg), eu = encode(u, cu);
        if (at.live) {
            *code_at(p, 2 * at.row, at.col) = cg;
            *code_at(p, 2 * at.row + 1, at.col) = cu;
            if (at.col % kBlock == 0) {
                uint8_t* const e = p.exponents + 2 * at.row * p.lde + at.col / kBlock;
                e[0] = (uint8_t)eg;
                e[p.lde] = (uint8_t)eu;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) g[i] = g[i] * sigmoid<T>(g[i]) * u[i];
    store16<kVec>(turn, static_cast<T*>(p.out), at.row * p.ld_out + at.col, at.n, g);
}

template <class T, bool kVec>
__global__ void __launch_bounds__(kActThreads, sizeof(T) == 2 && kVec ? 10 : 1) k_swiglu_backward(const ActArgs p) {
    const Turn turn = turn_of<kVec>();
    pdl_sync();
    const Place at(p);
    if (kVec && !at.live) return;
    float g[kPer], u[kPer], d[kPer];
    const int col = at.live ? at.col : 0;
    const uint4 cg = *code_at(p, 2 * at.row, col), cu = *code_at(p, 2 * at.row + 1, col);
    const uint8_t* const e = p.exponents + 2 * at.row * p.lde + col / kBlock;
    const uint32_t eg = e[0], eu = e[p.lde];
    load16<kVec>(turn, static_cast<const T*>(p.in), at.row * p.ld_in + at.col, at.n, d);
    decode(cg, eg, g);
    decode(cu, eu, u);
    float h[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const float s = sigmoid<T>(g[i]), a = g[i] * s, b = d[i] * u[i];
        h[i] = a * u[i];
        g[i] = b * fmaf(a, 1.0f - s, s);
        u[i] = d[i] * a;
    }
    const int64_t to = at.row * p.ld_out + at.col;
    store16<kVec>(turn, static_cast<T*>(p.out), to, at.n, g);
    store16<kVec>(turn, static_cast<T*>(p.out), to + p.cols, at.n, u);
    if (p.h) store16<kVec>(turn, static_cast<T*>(p.h), at.row * p.ldh + at.col, at.n, h);
}

bool vectors(const void* p, int64_t ld, size_t elem) { return is_aligned(p, 16) && (size_t)ld * elem % 16 == 0; }

template <class F>
int launch_act(F kernel, const ActArgs& a, const char* what, cudaStream_t s) {
    const uint64_t threads = (uint64_t)a.rows * a.per_row;
    return check_cuda(launch_after(kernel, (unsigned)((threads + kActThreads - 1) / kActThreads), kActThreads, 0, 1, s, a), what);
}

int check_act(int64_t rows, int64_t cols, int32_t type) {
    if (type != OPTIM_BF16 && type != OPTIM_F32) return set_error(OPTIM_EINVAL, "type must be OPTIM_BF16 or OPTIM_F32");
    if (rows < 0 || cols < 1 || rows >= ((int64_t)1 << 31) || cols >= ((int64_t)1 << 30))
        return set_error(OPTIM_EINVAL, "need 0 <= rows < 2^31 and 1 <= cols < 2^30");
    if (rows > ((int64_t)1 << 37) / ((cols + kBlock - 1) / kBlock)) return set_error(OPTIM_EINVAL, "rows x cols too large");
    return OPTIM_OK;
}
int check_matrix(const void* p, int64_t ld, int64_t rows, int64_t cols, int32_t type, const char* name) {
    if (!p) return set_error(OPTIM_EINVAL, "%s is NULL", name);
    if (ld < cols && rows > 1) return set_error(OPTIM_EINVAL, "%s: row stride %lld below its %lld columns", name, (long long)ld, (long long)cols);
    if (!is_aligned(p, type == OPTIM_BF16 ? 2 : 4)) return set_error(OPTIM_EALIGN, "%s not aligned to its elements", name);
    return OPTIM_OK;
}
int check_codes(const int8_t* codes, int64_t ldc, const uint8_t* exponents, int64_t lde, int64_t cols) {
    const int64_t blocks = (cols + kBlock - 1) / kBlock;
    if (!codes || !exponents) return set_error(OPTIM_EINVAL, "codes or exponents is NULL");
    if (ldc < blocks * kBlock || ldc % kBlock) return set_error(OPTIM_EINVAL, "ldc must be a multiple of 32, %lld at least", (long long)blocks * kBlock);
    if (lde < blocks) return set_error(OPTIM_EINVAL, "lde below the row's %lld blocks", (long long)blocks);
    if (!is_aligned(codes, 16)) return set_error(OPTIM_EALIGN, "codes not 16-byte aligned");
    return OPTIM_OK;
}
uint32_t per_row_of(int64_t cols) { return (uint32_t)((cols + kBlock - 1) / kBlock * (kBlock / kPer)); }

}  // namespace
}  // namespace lmo

using namespace lmo;

extern "C" {

int act_pack_i8(const void* x, int64_t ldx, int8_t* codes, int64_t ldc, uint8_t* exponents, int64_t lde, int64_t rows, int64_t cols,
                int32_t type, void* stream) {
    int rc = check_act(rows, cols, type);
    if (rc || rows == 0) return rc;
    rc = check_matrix(x, ldx, rows, cols, type, "x");
    if (!rc) rc = check_codes(codes, ldc, exponents, lde, cols);
    if (rc) return rc;
    const ActArgs a{x, ldx, codes, ldc, exponents, lde, nullptr, 0, nullptr, 0, (uint32_t)rows, per_row_of(cols), (int32_t)cols};
    const bool vec = vectors(x, ldx, type == OPTIM_BF16 ? 2 : 4);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const char* what = "activation pack launch";
    if (type == OPTIM_BF16) return vec ? launch_act(k_act_pack<uint16_t, true>, a, what, s) : launch_act(k_act_pack<uint16_t, false>, a, what, s);
    return vec ? launch_act(k_act_pack<float, true>, a, what, s) : launch_act(k_act_pack<float, false>, a, what, s);
}

int act_unpack_i8(const int8_t* codes, int64_t ldc, const uint8_t* exponents, int64_t lde, void* x, int64_t ldx, int64_t rows,
                  int64_t cols, int32_t type, void* stream) {
    int rc = check_act(rows, cols, type);
    if (rc || rows == 0) return rc;
    rc = check_matrix(x, ldx, rows, cols, type, "x");
    if (!rc) rc = check_codes(codes, ldc, exponents, lde, cols);
    if (rc) return rc;
    const ActArgs a{nullptr, 0, const_cast<int8_t*>(codes), ldc, const_cast<uint8_t*>(exponents), lde, x, ldx, nullptr, 0,
                    (uint32_t)rows, per_row_of(cols), (int32_t)cols};
    const bool vec = vectors(x, ldx, type == OPTIM_BF16 ? 2 : 4);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const char* what = "activation unpack launch";
    if (type == OPTIM_BF16) return vec ? launch_act(k_act_unpack<uint16_t, true>, a, what, s) : launch_act(k_act_unpack<uint16_t, false>, a, what, s);
    return vec ? launch_act(k_act_unpack<float, true>, a, what, s) : launch_act(k_act_unpack<float, false>, a, what, s);
}

int act_swiglu_forward(const void* gate_up, int64_t ldg, void* h, int64_t ldh, int8_t* codes, int64_t ldc, uint8_t* exponents,
                       int64_t lde, int64_t rows, int64_t cols, int32_t type, void* stream) {
    int rc = check_act(rows, cols, type);
    if (rc || rows == 0) return rc;
    rc = check_matrix(gate_up, ldg, rows, 2 * cols, type, "gate_up");
    if (!rc) rc = check_matrix(h, ldh, rows, cols, type, "h");
    if (!rc && (codes || exponents)) rc = check_codes(codes, ldc, exponents, lde, cols);
    if (rc) return rc;
    const ActArgs a{gate_up, ldg, codes, ldc, exponents, lde, h, ldh, nullptr, 0, (uint32_t)rows, per_row_of(cols), (int32_t)cols};
    const size_t elem = type == OPTIM_BF16 ? 2 : 4;
    const bool vec = vectors(gate_up, ldg, elem) && vectors(h, ldh, elem) && (size_t)cols * elem % 16 == 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const char* what = "gated activation launch";
    if (type == OPTIM_BF16) return vec ? launch_act(k_swiglu_forward<uint16_t, true>, a, what, s) : launch_act(k_swiglu_forward<uint16_t, false>, a, what, s);
    return vec ? launch_act(k_swiglu_forward<float, true>, a, what, s) : launch_act(k_swiglu_forward<float, false>, a, what, s);
}

int act_swiglu_backward(const void* dh, int64_t lddh, const int8_t* codes, int64_t ldc, const uint8_t* exponents, int64_t lde,
                        void* d_gate_up, int64_t ldg, void* h, int64_t ldh, int64_t rows, int64_t cols, int32_t type, void* stream) {
    int rc = check_act(rows, cols, type);
    if (rc || rows == 0) return rc;
    rc = check_matrix(dh, lddh, rows, cols, type, "dh");
    if (!rc) rc = check_codes(codes, ldc, exponents, lde, cols);
    if (!rc) rc = check_matrix(d_gate_up, ldg, rows, 2 * cols, type, "d_gate_up");
    if (!rc && h) rc = check_matrix(h, ldh, rows, cols, type, "h");
    if (rc) return rc;
    const ActArgs a{dh, lddh, const_cast<int8_t*>(codes), ldc, const_cast<uint8_t*>(exponents), lde, d_gate_up, ldg, h, ldh,
                    (uint32_t)rows, per_row_of(cols), (int32_t)cols};
    const size_t elem = type == OPTIM_BF16 ? 2 : 4;
    const bool vec = vectors(dh, lddh, elem) && vectors(d_gate_up, ldg, elem) && (!h || vectors(h, ldh, elem)) && (size_t)cols * elem % 16 == 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const char* what = "gated activation backward launch";
    if (type == OPTIM_BF16) return vec ? launch_act(k_swiglu_backward<uint16_t, true>, a, what, s) : launch_act(k_swiglu_backward<uint16_t, false>, a, what, s);
    return vec ? launch_act(k_swiglu_backward<float, true>, a, what, s) : launch_act(k_swiglu_backward<float, false>, a, what, s);
}

}  // extern "C"
