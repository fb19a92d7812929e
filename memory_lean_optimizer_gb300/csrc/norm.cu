// norm.cu -- layer norm over the rows of a matrix, forward and backward.
//   mu = mean x, r = 1 / sqrt(mean (x - mu)^2 + eps), y = (x - mu) r w + b
//   xh = (x - mu) r, a = dy w, dx = r (a - mean a - xh mean(a xh)), dw = sum_rows dy xh, db = sum_rows dy
// Values are fp32 from load to store, whatever the types; the variance is taken around the mean
// (a second sum over the row), not as a difference of squares.  Sums run in a fixed order, so two
// runs agree bit for bit.
//
// 16384 x 4096 bf16: forward 60 us (4.5 TB/s of the bytes that it must move), backward 83 us (4.9 TB/s).
// Neither waits for memory alone: instructions issue in 60-70 % of the cycles (23 an element over both), and
// the registers that hold the rows leave few warps to cover the reductions' chains of shuffles.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "internal.h"
#include "launch.cuh"
#include "packed.cuh"

namespace lmo {
namespace {

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }
__device__ __forceinline__ void store1(uint16_t* p, float x) { *p = (uint16_t)rne_bf16(x); }

// V consecutive elements, as they are stored (V * sizeof(T) bytes, one access) and as fp32.
template <class T, int V>
struct Vec;
template <>
struct Vec<float, 1> {
    float r;
    __device__ __forceinline__ void load(const float* p) { r = *p; }
    __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = r; }
    static __device__ __forceinline__ void store(float* p, const float (&f)[1]) { *p = f[0]; }
};
template <>
struct Vec<uint16_t, 1> {
    uint16_t r;
    __device__ __forceinline__ void load(const uint16_t* p) { r = *p; }
    __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = bf16_to_f32(r); }
    static __device__ __forceinline__ void store(uint16_t* p, const float (&f)[1]) { *p = (uint16_t)rne_bf16(f[0]); }
};
template <>
struct Vec<float, 4> {
    float4 r;
    __device__ __forceinline__ void load(const float* p) { r = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void get(float (&f)[4]) const { f[0] = r.x, f[1] = r.y, f[2] = r.z, f[3] = r.w; }
    static __device__ __forceinline__ void store(float* p, const float (&f)[4]) {
        *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    }
};
template <>
struct Vec<uint16_t, 4> {
    uint2 r;
    __device__ __forceinline__ void load(const uint16_t* p) { r = *reinterpret_cast<const uint2*>(p); }
    __device__ __forceinline__ void get(float (&f)[4]) const {
        f[0] = __uint_as_float(r.x << 16), f[1] = __uint_as_float(r.x & 0xFFFF0000u);
        f[2] = __uint_as_float(r.y << 16), f[3] = __uint_as_float(r.y & 0xFFFF0000u);
    }
};
template <>
struct Vec<uint16_t, 8> {
    uint4 r;
    __device__ __forceinline__ void load(const uint16_t* p) { r = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ void store(uint16_t* p, const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // two values per instruction, to nearest even
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Vec<float, 8> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = *reinterpret_cast<const float4*>(p);
        b = *reinterpret_cast<const float4*>(p + 4);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
};

// Sums of N values over the blockDim.x threads that share a row, in every one of them, in a fixed order.
// One warp: by shuffles alone.  More: each warp leaves its sums in shared memory and, after one
// barrier, every thread adds them all; `turn` alternates between two areas, so the next call's writes
// cannot meet this call's reads (a third call is a barrier away).
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*smem)[2][32], int& turn) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = warp_sum_f32(v[i]);
    if (blockDim.x == 32) return;
    const int nw = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) smem[turn][i][threadIdx.x >> 5] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float s = 0.0f;
        for (int k = 0; k < nw; k += 4) {   // the areas are zero past the last warp
            const float4 q = *reinterpret_cast<const float4*>(&smem[turn][i][k]);
            s += (q.x + q.y) + (q.z + q.w);
        }
        v[i] = s;
    }
    turn ^= 1;
}
__device__ __forceinline__ void clear_sums(float (*smem)[2][32]) {
    if (threadIdx.y == 0)
        for (int i = threadIdx.x; i < 128; i += blockDim.x) (&smem[0][0][0])[i] = 0.0f;
    __syncthreads();
}

__device__ __forceinline__ float total(F2 p) {
    float a, b;
    split2(p, a, b);
    return a + b;
}

// What a thread holds of a row is K slices of kWide values.  Rows that can be read in 16-byte vectors (kWide = V
// values next to each other, element (k * blockDim.x + threadIdx.x) * V on), or not (V = 1): single
// elements (2k * kT + threadIdx.x) and kT further, kT threads to a row, two to a slice so that the
// packed instructions serve them as well; the second of the last slice may lie past the row's end.
template <class T, int V, int kT>
struct Slice {
    static constexpr int kWide = V > 1 ? V : 2, n = kWide / 2;
    static __device__ __forceinline__ int column(int k) {
        return V > 1 ? (k * (int)blockDim.x + (int)threadIdx.x) * V : 2 * k * kT + (int)threadIdx.x;
    }
    Vec<T, V> raw[V > 1 ? 1 : 2];
    // c: column(k), below dim
    __device__ __forceinline__ void load(const T* row, int c, int dim) {
        raw[0].load(row + c);
        if (V == 1) {
            raw[V > 1 ? 0 : 1] = Vec<T, V>{};
            if (c + kT < dim) raw[V > 1 ? 0 : 1].load(row + c + kT);
        }
    }
    __device__ __forceinline__ void get(F2 (&p)[n]) const {
        float f[V], g[V];
        raw[0].get(f);
        raw[V > 1 ? 0 : 1].get(g);
#pragma unroll
        for (int i = 0; i < n; ++i) p[i] = V > 1 ? f2(f[2 * i % V], f[(2 * i + 1) % V]) : f2(f[0], g[0]);
    }
    static __device__ __forceinline__ void store(T* row, int c, int dim, const F2 (&p)[n]) {
        float f[V], g[V];
#pragma unroll
        for (int i = 0; i < n; ++i) {
            if (V > 1) split2(p[i], f[2 * i % V], f[(2 * i + 1) % V]);
            else split2(p[i], f[0], g[0]);
        }
        Vec<T, V>::store(row + c, f);
        if (V == 1 && c + kT < dim) Vec<T, V>::store(row + c + kT, g);
    }
};

// Rows on their way: a thread copies (cp.async) its own slices of the rows it will take next into its own places
// of shared memory, kRowsAhead rows before it reads them, so that the copies cost no registers -- loads
// into registers a row ahead were moved down to their use by the compiler -- and waiting for its
// own copies is all the order there is.  Single bf16 elements are too small for these copies (4
// bytes): kAsync false, and the row is loaded where it is used.
constexpr int kPlaces = 3, kRowsAhead = kPlaces - 1;
template <class T, int V, int K, int kT>
struct Coming {
    static constexpr bool kAsync = V > 1 || sizeof(T) == 4;
    static constexpr int kUnit = V > 1 ? 16 : 4, kPer = V > 1 ? K : 2 * K;   // bytes of a copy, copies to a row and thread
    using S = Slice<T, V, kT>;
    char* mine;
    int threads;
    __device__ __forceinline__ Coming(char* smem) {
        threads = (int)(blockDim.x * blockDim.y);
        mine = smem + (threadIdx.y * blockDim.x + threadIdx.x) * kUnit;
    }
    __device__ __forceinline__ char* at(int place, int i) const {
        return mine + (place * kPer + i) * threads * kUnit;
    }
    static __device__ __forceinline__ void copy(char* dst, const T* src) {
        const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst);
        if (V > 1) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(src) : "memory");
        else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(src) : "memory");
    }
    __device__ __forceinline__ void fetch(int place, const T* row, int dim) const {
        if constexpr (kAsync) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = S::column(k);
                if (V > 1) {
                    if (c < dim) copy(at(place, k), row + c);
                } else {
                    if (c < dim) copy(at(place, 2 * k), row + c);
                    if (c + kT < dim) copy(at(place, 2 * k + 1), row + c + kT);
                }
            }
        }
    }
    static __device__ __forceinline__ void close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    static __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kRowsAhead) : "memory"); }
    // Slice k, whose first column c is below dim (row: where it is in memory, for kAsync false).
    __device__ __forceinline__ S read(int place, int k, const T* row, int c, int dim) const {
        S x;
        if (!kAsync) {
            x.load(row, c, dim);
        } else if (V > 1) {
            x.raw[0].load(reinterpret_cast<const T*>(at(place, k)));
        } else {
            x.raw[0].load(reinterpret_cast<const T*>(at(place, 2 * k)));
            x.raw[V > 1 ? 0 : 1] = Vec<T, V>{};
            if (c + kT < dim) x.raw[V > 1 ? 0 : 1].load(reinterpret_cast<const T*>(at(place, 2 * k + 1)));
        }
        return x;
    }
    static size_t bytes(int threads) { return kAsync ? (size_t)kPlaces * kPer * threads * kUnit : 0; }
};

// Forward, the row in registers: blockDim.x threads hold a row, blockDim.y rows at a time.  x is read once, y
// written once.
template <class TX, class TW, int V, int K, int kT, int kMaxThreads, int kMinCtas>
__global__ void __launch_bounds__(kMaxThreads, kMinCtas) k_norm_forward(const TX* x, int64_t ldx, const TW* __restrict__ w,
                                                                        const TW* __restrict__ b, TX* y, int64_t ldy,
                                                                        float* __restrict__ mean, float* __restrict__ rstd,
                                                                        int64_t rows, int dim, float eps) {
    using S = Slice<TX, V, kT>;
    extern __shared__ __align__(16) char coming_smem[];
    __shared__ __align__(16) float red[2][2][32];
    pdl_sync();
    clear_sums(red);
    const Coming<TX, V, K, kT> coming(coming_smem);
    const float inv = 1.0f / (float)dim;
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    int turn = 0, place = 0;
    int64_t r = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
#pragma unroll
    for (int i = 0; i < kRowsAhead; ++i) {
        if (r + i * step < rows) coming.fetch(i, x + (r + i * step) * ldx, dim);
        coming.close();
    }
    for (; r < rows; r += step) {
        const int into = place == 0 ? kRowsAhead : place - 1;
        if (r + kRowsAhead * step < rows) coming.fetch(into, x + (r + kRowsAhead * step) * ldx, dim);
        coming.close();
        coming.wait();
        F2 f[K][S::n];
        F2 acc = f2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = S::column(k);
            if (c < dim) {
                coming.read(place, k, x + r * ldx, c, dim).get(f[k]);
#pragma unroll
                for (int i = 0; i < S::n; ++i) acc = add2(acc, f[k][i]);
            }
        }
        if (++place == kPlaces) place = 0;
        float s[1] = {total(acc)};
        row_sums(s, red, turn);
        const float mu = s[0] * inv;
        const F2 n_mu = f2(-mu, -mu);
        acc = f2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = S::column(k);
            if (c < dim) {
#pragma unroll
                for (int i = 0; i < S::n; ++i) {
                    f[k][i] = add2(f[k][i], V > 1 || c + kT < dim ? n_mu : f2(-mu, 0.0f));   // past the end: stays 0
                    acc = fma2(f[k][i], f[k][i], acc);
                }
            }
        }
        s[0] = total(acc);
        row_sums(s, red, turn);
        const float rs = 1.0f / sqrtf(fmaf(s[0], inv, eps));
        const F2 rs2 = f2(rs, rs);
        TX* const py = y + r * ldy;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = S::column(k);
            if (c < dim) {
                Slice<TW, V, kT> raw_w, raw_b;
                F2 wv[S::n], bv[S::n];
                raw_w.load(w, c, dim);
                raw_w.get(wv);
                if (b) {
                    raw_b.load(b, c, dim);
                    raw_b.get(bv);
                }
#pragma unroll
                for (int i = 0; i < S::n; ++i) f[k][i] = fma2(mul2(f[k][i], rs2), wv[i], b ? bv[i] : f2(0.0f, 0.0f));
                S::store(py, c, dim, f[k]);
            }
        }
        if (threadIdx.x == 0) {
            if (mean) mean[r] = mu;
            if (rstd) rstd[r] = rs;
        }
    }
}

// Backward with everything in one pass: x and dy are read once, dx written once, and each thread
// keeps the sums of dy xh and dy of its own columns over all of its CTA's rows, so that the weight's
// gradient costs no second reading -- one fp32 row of each per CTA at the end (partial[CTA][2][dim],
// joined by k_norm_join in CTA order).  kAhead: the next row is on its way while this one is reduced
// (where the registers allow it).
template <class TX, class TW, int V, int K, int kT, int kMaxThreads, bool kAhead>
__global__ void __launch_bounds__(kMaxThreads, 1) k_norm_backward(const TX* dy, int64_t lddy, const TX* x, int64_t ldx,
                                                                  const TW* __restrict__ w, const float* __restrict__ mean,
                                                                  const float* __restrict__ rstd, TX* dx, int64_t lddx,
                                                                  float* __restrict__ partial, int64_t rows, int dim) {
    using S = Slice<TX, V, kT>;
    __shared__ __align__(16) float red[2][2][32];
    extern __shared__ float cols[];   // [2][dim], only when blockDim.y > 1
    pdl_sync();
    clear_sums(red);
    const float inv = 1.0f / (float)dim;
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    int turn = 0;
    F2 aw[K][S::n], ab[K][S::n], wv[K][S::n];
    S rx[K], rg[K];
    int64_t r = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const TX* px = x + r * ldx;
    const TX* pg = dy + r * lddy;
    float mu = 0.0f, rs = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = S::column(k);
#pragma unroll
        for (int i = 0; i < S::n; ++i) aw[k][i] = ab[k][i] = wv[k][i] = f2(0.0f, 0.0f);
        if (c < dim) {
            Slice<TW, V, kT> raw_w;
            raw_w.load(w, c, dim);
            raw_w.get(wv[k]);
            if (kAhead && r < rows) {
                rx[k].load(px, c, dim);
                rg[k].load(pg, c, dim);
            }
        }
    }
    if (kAhead && r < rows) mu = mean[r], rs = rstd[r];
    for (; r < rows; r += step) {
        if (!kAhead) {
            mu = mean[r], rs = rstd[r];
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = S::column(k);
                if (c < dim) {
                    rx[k].load(px, c, dim);
                    rg[k].load(pg, c, dim);
                }
            }
        }
        px += step * ldx;
        pg += step * lddy;
        S nx[K], ng[K];
        float nmu = 0.0f, nrs = 0.0f;
        if (kAhead && r + step < rows) {
            nmu = mean[r + step], nrs = rstd[r + step];
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = S::column(k);
                if (c < dim) {
                    nx[k].load(px, c, dim);
                    ng[k].load(pg, c, dim);
                }
            }
        }
        const F2 n_mu = f2(-mu, -mu), rs2 = f2(rs, rs);
        F2 sa = f2(0.0f, 0.0f), sx = sa;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (S::column(k) < dim) {
                F2 vx[S::n], vg[S::n];   // past the end dy is 0 and adds nothing
                rx[k].get(vx);
                rg[k].get(vg);
#pragma unroll
                for (int i = 0; i < S::n; ++i) {
                    const F2 xh = mul2(add2(vx[i], n_mu), rs2), a = mul2(vg[i], wv[k][i]);
                    aw[k][i] = fma2(vg[i], xh, aw[k][i]);
                    ab[k][i] = add2(ab[k][i], vg[i]);
                    sa = add2(sa, a);
                    sx = fma2(a, xh, sx);
                }
            }
        }
        if (dx) {   // uniform: the barrier inside is reached by all threads or none
            float s[2] = {total(sa), total(sx)};
            row_sums(s, red, turn);
            const F2 m1 = f2(-s[0] * inv, -s[0] * inv), m2 = f2(-s[1] * inv, -s[1] * inv);
            TX* const pd = dx + r * lddx;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = S::column(k);
                if (c < dim) {
                    F2 vx[S::n], vg[S::n];
                    rx[k].get(vx);
                    rg[k].get(vg);
#pragma unroll
                    for (int i = 0; i < S::n; ++i) {
                        const F2 xh = mul2(add2(vx[i], n_mu), rs2), a = mul2(vg[i], wv[k][i]);
                        vg[i] = mul2(add2(fma2(xh, m2, a), m1), rs2);
                    }
                    S::store(pd, c, dim, vg);
                }
            }
        }
        if (kAhead) {
            mu = nmu, rs = nrs;
#pragma unroll
            for (int k = 0; k < K; ++k) rx[k] = nx[k], rg[k] = ng[k];
        }
    }
    if (!partial) return;
    float* const out = partial + (int64_t)blockIdx.x * 2 * dim;
    for (int turn_y = 0; turn_y < (int)blockDim.y; ++turn_y) {   // rows of warps add up in their order
        if ((int)threadIdx.y == turn_y) {
            const bool last = turn_y + 1 == (int)blockDim.y;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = S::column(k);
#pragma unroll
                for (int i = 0; i < S::n; ++i) {
                    float w2[2], b2[2];
                    split2(aw[k][i], w2[0], w2[1]);
                    split2(ab[k][i], b2[0], b2[1]);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int at = V > 1 ? c + 2 * i + e : c + e * kT;
                        if (at < dim) {
                            (last ? out : cols)[at] = turn_y ? cols[at] + w2[e] : w2[e];
                            (last ? out : cols)[dim + at] = turn_y ? cols[dim + at] + b2[e] : b2[e];
                        }
                    }
                }
            }
        }
        if (blockDim.y > 1) __syncthreads();
    }
}

// Sum of the partial rows: column j of [2][dim] over `slices`, sixteen threads each a slice in sixteen, then
// their sums in order.
template <class TW>
__global__ void __launch_bounds__(512) k_norm_join(const float* __restrict__ partial, int slices, TW* __restrict__ dw,
                                                        TW* __restrict__ db, int64_t dim) {
    __shared__ float red[16][33];
    pdl_sync();
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t j = (int64_t)blockIdx.x * 32 + tx;
    float s = 0.0f;
    if (j < 2 * dim)
#pragma unroll 8
        for (int k = ty; k < slices; k += 16) s += partial[(int64_t)k * 2 * dim + j];
    red[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && j < 2 * dim) {
        s = red[0][tx];
        for (int k = 1; k < 16; ++k) s += red[k][tx];
        TW* const out = j < dim ? dw : db;
        if (out) store1(out + (j < dim ? j : j - dim), s);
    }
}

// ---- rows too long for the registers of one CTA: each pass reads them again -------------------
// Sum over the block, in every thread.
__device__ __forceinline__ float block_sum(float x, float* smem /* 33 */) {
    x = warp_sum_f32(x);
    if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = x;
    __syncthreads();
    if (threadIdx.x < 32) {
        float s = threadIdx.x < (blockDim.x >> 5) ? smem[threadIdx.x] : 0.0f;
        s = warp_sum_f32(s);
        if (threadIdx.x == 0) smem[32] = s;
    }
    __syncthreads();
    x = smem[32];
    __syncthreads();
    return x;
}

template <class TX, class TW>
__global__ void __launch_bounds__(kThreads) k_norm_forward_long(const TX* x, int64_t ldx, const TW* __restrict__ w,
                                                           const TW* __restrict__ b, TX* y, int64_t ldy,
                                                           float* __restrict__ mean, float* __restrict__ rstd,
                                                           int64_t rows, int64_t dim, float eps) {
    __shared__ float red[33];
    const float inv = 1.0f / (float)dim;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const TX* px = x + r * ldx;
        TX* py = y + r * ldy;
        float s = 0.0f;
        for (int64_t i = threadIdx.x; i < dim; i += kThreads) s += load1(px + i);
        const float mu = block_sum(s, red) * inv;
        s = 0.0f;
        for (int64_t i = threadIdx.x; i < dim; i += kThreads) {
            const float d = load1(px + i) - mu;
            s = fmaf(d, d, s);
        }
        const float rs = 1.0f / sqrtf(fmaf(block_sum(s, red), inv, eps));
        for (int64_t i = threadIdx.x; i < dim; i += kThreads)
            store1(py + i, fmaf((load1(px + i) - mu) * rs, load1(w + i), b ? load1(b + i) : 0.0f));
        if (threadIdx.x == 0) {
            if (mean) mean[r] = mu;
            if (rstd) rstd[r] = rs;
        }
    }
}

template <class TX, class TW>
__global__ void __launch_bounds__(kThreads) k_norm_dx_long(const TX* dy, int64_t lddy, const TX* __restrict__ x,
                                                      int64_t ldx, const TW* __restrict__ w, const float* __restrict__ mean,
                                                      const float* __restrict__ rstd, TX* dx, int64_t lddx,
                                                      int64_t rows, int64_t dim) {
    __shared__ float red[33];
    const float inv = 1.0f / (float)dim;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const float mu = mean[r], rs = rstd[r];
        const TX* px = x + r * ldx;
        const TX* pdy = dy + r * lddy;
        float s1 = 0.0f, s2 = 0.0f;
        for (int64_t i = threadIdx.x; i < dim; i += kThreads) {
            const float a = load1(pdy + i) * load1(w + i);
            s1 += a;
            s2 = fmaf(a, (load1(px + i) - mu) * rs, s2);
        }
        const float m1 = block_sum(s1, red) * inv, m2 = block_sum(s2, red) * inv;
        for (int64_t i = threadIdx.x; i < dim; i += kThreads) {
            const float a = load1(pdy + i) * load1(w + i), xh = (load1(px + i) - mu) * rs;
            store1(dx + r * lddx + i, rs * (a - m1 - xh * m2));
        }
    }
}

// Column sums of dy xh and dy over one slice of the rows: partial[slice][0 or 1][dim].
template <class TX>
__global__ void __launch_bounds__(kThreads) k_norm_dw_long(const TX* __restrict__ dy, int64_t lddy, const TX* __restrict__ x,
                                                      int64_t ldx, const float* __restrict__ mean,
                                                      const float* __restrict__ rstd, float* __restrict__ partial,
                                                      int64_t rows, int64_t dim) {
    __shared__ float red[2][8][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + tx;
    float sw = 0.0f, sb = 0.0f;
    if (c < dim) {
        for (int64_t r = (int64_t)blockIdx.y * 8 + ty; r < rows; r += (int64_t)gridDim.y * 8) {
            const float g = load1(dy + r * lddy + c);
            sw = fmaf(g, (load1(x + r * ldx + c) - mean[r]) * rstd[r], sw);
            sb += g;
        }
    }
    red[0][ty][tx] = sw;
    red[1][ty][tx] = sb;
    __syncthreads();
    if (ty < 2 && c < dim) {
        float s = 0.0f;
        for (int k = 0; k < 8; ++k) s += red[ty][k][tx];
        partial[((int64_t)blockIdx.y * 2 + ty) * dim + c] = s;
    }
}

constexpr int kMostSmem = 96 * 1024;   // 512 threads with 32 bf16 or 16 fp32 values each

// Partial rows of the weight's gradient at most: 4 CTAs on each of 152 SMs (fixed, because the workspace call answers
// without a device).
constexpr int kMaxSlices = 608;

unsigned row_grid(int64_t rows) { return (unsigned)std::min<int64_t>(rows, (int64_t)sm_count() * 8); }

bool rows_aligned(const void* p, int64_t ld, size_t elem) { return is_aligned(p, 16) && (size_t)ld * elem % 16 == 0; }

// How a row is laid over threads: K slices a thread (Slice), tx threads a row, ty rows a CTA.
struct RowShape {
    int V = 0, K = 0, tx = 0, ty = 1;   // K = 0: too long
};
// Two 16-byte vectors a thread up to 512 threads, then four.  One vector shares what a thread does for a row besides
// its values (the trees, the addresses, the root) among too few of them, and with four the
// registers leave too few threads on an SM: 16384 x 4096 bf16, forward / backward, one 78 / 109,
// two 64 / 86, four 73 / 115 us; 8192 x 4096 fp32, two 63 / 80, four 68 / 124 us.  A row inside one
// warp, where it fits, needs no barrier.
RowShape row_shape(int64_t dim, int vec, bool aligned) {
    if (aligned && dim % vec == 0) {
        const int64_t units = dim / vec;
        if (units <= 128) return {vec, 4, 32, 4};
        for (int k : {2, 4})
            if (units <= 512 * k) return {vec, k, (int)((units + 32 * k - 1) / (32 * k) * 32), 1};
        return {};
    }
    for (int t : {32, 64, 128, 256, 512})
        if (dim <= 16 * t) return {1, 8, t, t == 32 ? 4 : 1};
    return {};
}

// CTAs of one kernel that fit on the GPU at once, `wanted` at most.  `last` (one per kernel) remembers the answer for
// the last shape, threads << 48 | smem << 16 | CTAs an SM: the query costs as much as a launch.
template <class F>
int64_t resident(F kernel, int threads, size_t smem, int64_t wanted, std::atomic<uint64_t>& last) {
    if (wanted <= sm_count()) return wanted;
    const uint64_t shape = (uint64_t)threads << 48 | (uint64_t)smem << 16;
    uint64_t known = last.load(std::memory_order_relaxed);
    if ((known & ~(uint64_t)0xFFFF) != shape || (known & 0xFFFF) == 0) {
        int per_sm = 0;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem) != cudaSuccess || per_sm < 1) per_sm = 1;
        known = shape | (uint64_t)per_sm;
        last.store(known, std::memory_order_relaxed);
    }
    return std::min<int64_t>(wanted, (int64_t)(known & 0xFFFF) * sm_count());
}

template <class TX, class TW, int V, int K, int kT, int kMax, int kMin>
int forward_rows(const NormForward& a, const RowShape& sh, cudaStream_t s) {
    auto kernel = k_norm_forward<TX, TW, V, K, kT, kMax, kMin>;
    const size_t smem = Coming<TX, V, K, kT>::bytes(sh.tx * sh.ty);
    static std::atomic<uint64_t> last{0}, allowed{0};
    const int rc = allow_smem(kernel, kMostSmem, allowed);
    if (rc) return rc;
    const int64_t grid = resident(kernel, sh.tx * sh.ty, smem, (a.rows + sh.ty - 1) / sh.ty, last);
    return check_cuda(launch_after(kernel, grid, dim3(sh.tx, sh.ty), smem, 1, s, static_cast<const TX*>(a.x), a.ldx,
                                   static_cast<const TW*>(a.weight), static_cast<const TW*>(a.bias), static_cast<TX*>(a.y),
                                   a.ldy, a.mean, a.rstd, a.rows, (int)a.dim, a.eps), "layer norm launch");
}

template <class TX, class TW>
int forward_t(const NormForward& a, cudaStream_t s) {
    constexpr int kVec = 16 / sizeof(TX);
    const bool aligned = rows_aligned(a.x, a.ldx, sizeof(TX)) && rows_aligned(a.y, a.ldy, sizeof(TX)) &&
                         is_aligned(a.weight, 16) && is_aligned(a.bias, 16);
    const RowShape sh = row_shape(a.dim, kVec, aligned);
    if (sh.V > 1 && sh.tx == 32) return forward_rows<TX, TW, kVec, 4, 0, 128, 4>(a, sh, s);
    if (sh.V > 1 && sh.K == 2) return forward_rows<TX, TW, kVec, 2, 0, 512, 2>(a, sh, s);
    if (sh.V > 1 && sh.K == 4) return forward_rows<TX, TW, kVec, 4, 0, 512, 1>(a, sh, s);
    if (sh.V == 1 && sh.tx == 32) return forward_rows<TX, TW, 1, 8, 32, 128, 4>(a, sh, s);
    if (sh.V == 1 && sh.tx == 64) return forward_rows<TX, TW, 1, 8, 64, 64, 8>(a, sh, s);
    if (sh.V == 1 && sh.tx == 128) return forward_rows<TX, TW, 1, 8, 128, 128, 5>(a, sh, s);
    if (sh.V == 1 && sh.tx == 256) return forward_rows<TX, TW, 1, 8, 256, 256, 2>(a, sh, s);
    if (sh.V == 1 && sh.tx == 512) return forward_rows<TX, TW, 1, 8, 512, 512, 1>(a, sh, s);
    k_norm_forward_long<TX, TW><<<row_grid(a.rows), kThreads, 0, s>>>(
        static_cast<const TX*>(a.x), a.ldx, static_cast<const TW*>(a.weight), static_cast<const TW*>(a.bias),
        static_cast<TX*>(a.y), a.ldy, a.mean, a.rstd, a.rows, a.dim, a.eps);
    return check_cuda(cudaGetLastError(), "layer norm launch");
}

template <class TW>
int join_slices(const NormBackward& a, int slices, cudaStream_t s) {
    return check_cuda(launch_after(k_norm_join<TW>, (2 * a.dim + 31) / 32, 512, 0, 1, s, a.partial, slices,
                                   static_cast<TW*>(a.dweight), static_cast<TW*>(a.dbias), a.dim),
                      "layer norm weight gradient launch");
}

template <class TX, class TW, int V, int K, int kT, int kMax, bool kAhead>
int backward_rows(const NormBackward& a, const RowShape& sh, cudaStream_t s) {
    auto kernel = k_norm_backward<TX, TW, V, K, kT, kMax, kAhead>;
    const bool sums = a.dweight || a.dbias;
    const size_t smem = sh.ty > 1 ? 2 * sizeof(float) * (size_t)a.dim : 0;
    static std::atomic<uint64_t> last{0};
    const int64_t wanted = std::min<int64_t>((a.rows + sh.ty - 1) / sh.ty, kMaxSlices);
    const int64_t grid = std::max<int64_t>(1, resident(kernel, sh.tx * sh.ty, smem, wanted, last));
    const int rc = check_cuda(launch_after(kernel, grid, dim3(sh.tx, sh.ty), smem, 1, s, static_cast<const TX*>(a.dy), a.lddy,
                                           static_cast<const TX*>(a.x), a.ldx, static_cast<const TW*>(a.weight), a.mean, a.rstd,
                                           static_cast<TX*>(a.dx), a.lddx, sums ? a.partial : nullptr, a.rows, (int)a.dim),
                              "layer norm backward launch");
    return rc || !sums ? rc : join_slices<TW>(a, (int)grid, s);
}

template <class TX, class TW>
int backward_t(const NormBackward& a, cudaStream_t s) {
    constexpr int kVec = 16 / sizeof(TX);
    const bool aligned = rows_aligned(a.x, a.ldx, sizeof(TX)) && rows_aligned(a.dy, a.lddy, sizeof(TX)) &&
                         (!a.dx || rows_aligned(a.dx, a.lddx, sizeof(TX))) && is_aligned(a.weight, 16);
    const RowShape sh = row_shape(a.dim, kVec, aligned);
    if (sh.V > 1 && sh.tx == 32) return backward_rows<TX, TW, kVec, 4, 0, 128, true>(a, sh, s);
    if (sh.V > 1 && sh.K == 2) return backward_rows<TX, TW, kVec, 2, 0, 512, true>(a, sh, s);
    if (sh.V > 1 && sh.K == 4) return backward_rows<TX, TW, kVec, 4, 0, 512, false>(a, sh, s);
    if (sh.V == 1 && sh.tx == 32) return backward_rows<TX, TW, 1, 8, 32, 128, true>(a, sh, s);
    if (sh.V == 1 && sh.tx == 64) return backward_rows<TX, TW, 1, 8, 64, 64, true>(a, sh, s);
    if (sh.V == 1 && sh.tx == 128) return backward_rows<TX, TW, 1, 8, 128, 128, true>(a, sh, s);
    if (sh.V == 1 && sh.tx == 256) return backward_rows<TX, TW, 1, 8, 256, 256, true>(a, sh, s);
    if (sh.V == 1 && sh.tx == 512) return backward_rows<TX, TW, 1, 8, 512, 512, false>(a, sh, s);
    const TX* dy = static_cast<const TX*>(a.dy);
    const TX* x = static_cast<const TX*>(a.x);
    if (a.dweight || a.dbias) {   // before dx, which may lie over dy
        const int slices = (int)std::max<int64_t>(1, std::min<int64_t>((a.rows + 63) / 64, 256));
        k_norm_dw_long<TX><<<dim3((unsigned)((a.dim + 31) / 32), (unsigned)slices), kThreads, 0, s>>>(
            dy, a.lddy, x, a.ldx, a.mean, a.rstd, a.partial, a.rows, a.dim);
        const int rc = join_slices<TW>(a, slices, s);
        if (rc) return rc;
    }
    if (!a.dx || a.rows == 0) return OPTIM_OK;
    k_norm_dx_long<TX, TW><<<row_grid(a.rows), kThreads, 0, s>>>(dy, a.lddy, x, a.ldx, static_cast<const TW*>(a.weight),
                                                                a.mean, a.rstd, static_cast<TX*>(a.dx), a.lddx, a.rows,
                                                                a.dim);
    return check_cuda(cudaGetLastError(), "layer norm backward launch");
}

}  // namespace

size_t norm_partial_bytes(int64_t rows, int64_t dim) { return (size_t)std::min<int64_t>(std::max<int64_t>(rows, 1), kMaxSlices) * 2 * (size_t)dim * sizeof(float); }

int launch_norm_forward(const NormForward& a, cudaStream_t s) {
    if (a.rows == 0) return OPTIM_OK;
    if (a.x_bf16) return a.w_bf16 ? forward_t<uint16_t, uint16_t>(a, s) : forward_t<uint16_t, float>(a, s);
    return a.w_bf16 ? forward_t<float, uint16_t>(a, s) : forward_t<float, float>(a, s);
}

int launch_norm_backward(const NormBackward& a, cudaStream_t s) {
    if (a.x_bf16) return a.w_bf16 ? backward_t<uint16_t, uint16_t>(a, s) : backward_t<uint16_t, float>(a, s);
    return a.w_bf16 ? backward_t<float, uint16_t>(a, s) : backward_t<float, float>(a, s);
}

}  // namespace lmo

using namespace lmo;

static int check_norm(int64_t rows, int64_t dim, int32_t x_type, int32_t w_type) {
    if (rows < 0 || dim < 1) return set_error(OPTIM_EINVAL, "need rows >= 0 and dim >= 1");
    if (dim >= ((int64_t)1 << 31) || rows >= ((int64_t)1 << 31))
        return set_error(OPTIM_EINVAL, "rows and dim must be below 2^31");
    if ((x_type != OPTIM_BF16 && x_type != OPTIM_F32) || (w_type != OPTIM_BF16 && w_type != OPTIM_F32))
        return set_error(OPTIM_EINVAL, "types must be OPTIM_BF16 or OPTIM_F32");
    return OPTIM_OK;
}

static int check_rows(const void* p, int64_t ld, int64_t rows, int64_t dim, int32_t type, const char* name) {
    if (rows == 0) return OPTIM_OK;
    if (!p) return set_error(OPTIM_EINVAL, "%s is NULL", name);
    if (ld < dim && rows > 1) return set_error(OPTIM_EINVAL, "%s: row stride %lld below dim %lld", name, (long long)ld, (long long)dim);
    if (!is_aligned(p, type == OPTIM_BF16 ? 2 : 4)) return set_error(OPTIM_EALIGN, "%s not aligned to its elements", name);
    return OPTIM_OK;
}

extern "C" {

int norm_layer_forward(const void* x, int64_t ldx, const void* weight, const void* bias, void* y, int64_t ldy, float* mean,
                       float* rstd, int64_t rows, int64_t dim, float eps, int32_t x_type, int32_t w_type, void* stream) {
    int rc = check_norm(rows, dim, x_type, w_type);
    if (!rc && !(eps >= 0.0f && eps <= FLT_MAX)) rc = set_error(OPTIM_EINVAL, "eps is negative or not finite");
    if (!rc) rc = check_rows(x, ldx, rows, dim, x_type, "x");
    if (!rc) rc = check_rows(weight, dim, 1, dim, w_type, "weight");
    if (!rc && bias) rc = check_rows(bias, dim, 1, dim, w_type, "bias");
    if (!rc) rc = check_rows(y, ldy, rows, dim, x_type, "y");
    if (!rc && mean) rc = check_rows(mean, 1, rows, 1, OPTIM_F32, "mean");
    if (!rc && rstd) rc = check_rows(rstd, 1, rows, 1, OPTIM_F32, "rstd");
    if (rc) return rc;
    return launch_norm_forward({x, ldx, weight, bias, y, ldy, mean, rstd, rows, dim, eps, x_type == OPTIM_BF16,
                                w_type == OPTIM_BF16}, static_cast<cudaStream_t>(stream));
}

int norm_layer_workspace(int64_t rows, int64_t dim, size_t* bytes) {
    int rc = check_norm(rows, dim, OPTIM_BF16, OPTIM_BF16);
    if (!rc && !bytes) rc = set_error(OPTIM_EINVAL, "bytes is NULL");
    if (!rc) *bytes = norm_partial_bytes(rows, dim);
    return rc;
}

int norm_layer_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* weight, const float* mean,
                        const float* rstd, void* dx, int64_t lddx, void* dweight, void* dbias, int64_t rows, int64_t dim,
                        int32_t x_type, int32_t w_type, void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_norm(rows, dim, x_type, w_type);
    if (!rc) rc = check_rows(dy, lddy, rows, dim, x_type, "dy");
    if (!rc) rc = check_rows(x, ldx, rows, dim, x_type, "x");
    if (!rc) rc = check_rows(weight, dim, 1, dim, w_type, "weight");
    if (!rc) rc = check_rows(mean, 1, rows, 1, OPTIM_F32, "mean");
    if (!rc) rc = check_rows(rstd, 1, rows, 1, OPTIM_F32, "rstd");
    if (!rc && dx) rc = check_rows(dx, lddx, rows, dim, x_type, "dx");
    if (!rc && dweight) rc = check_rows(dweight, dim, 1, dim, w_type, "dweight");
    if (!rc && dbias) rc = check_rows(dbias, dim, 1, dim, w_type, "dbias");
    if (!rc && (dweight || dbias)) {
        const size_t need = norm_partial_bytes(rows, dim);
        rc = check_rows(workspace, 1, 1, 1, OPTIM_F32, "workspace");
        if (!rc && !is_aligned(workspace, 16)) rc = set_error(OPTIM_EALIGN, "workspace not 16-byte aligned");
        if (!rc && workspace_bytes < need)
            rc = set_error(OPTIM_EINVAL, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
    }
    if (rc) return rc;
    return launch_norm_backward({dy, lddy, x, ldx, weight, mean, rstd, dx, lddx, dweight, dbias,
                                 static_cast<float*>(workspace), rows, dim, x_type == OPTIM_BF16, w_type == OPTIM_BF16},
                                static_cast<cudaStream_t>(stream));
}

}  // extern "C"
