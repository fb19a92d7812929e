// norm.cu -- layer norm over the rows of a matrix, forward and backward.
//   mu = mean x, r = 1 / sqrt(mean (x - mu)^2 + eps), y = (x - mu) r w + b
//   xh = (x - mu) r, a = dy w, dx = r (a - mean a - xh mean(a xh)), dw = sum_rows dy xh, db = sum_rows dy
// Values are fp32 from load to store, whatever the types; the variance is taken around the mean
// (a second sum over the row), not as a difference of squares.  Sums run in a fixed order, so two
// runs agree bit for bit.
#include <cuda_bf16.h>

#include <algorithm>

#include "internal.h"

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

// Sums of N values over the blockDim.x threads that share a row, in every one of them.  One warp: by
// shuffles alone.  More: each warp leaves its sums in shared memory and, after one barrier, every
// warp adds them all in the same order; `turn` alternates between two areas, so the next call's
// writes cannot meet this call's reads (a third call is a barrier away).
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*smem)[2][32], int& turn) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = warp_sum_f32(v[i]);
    if (blockDim.x == 32) return;
    const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) smem[turn][i][threadIdx.x >> 5] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = warp_sum_f32(lane < nw ? smem[turn][i][lane] : 0.0f);
    turn ^= 1;
}

// Forward, the row in registers: blockDim.x threads hold a row as K vectors of V elements each (element
// (k * blockDim.x + threadIdx.x) * V of it), blockDim.y rows at a time.  x is read once, y written
// once; the next row is on its way while this one is reduced.
template <class TX, class TW, int V, int K>
__global__ void __launch_bounds__(1024) k_norm_forward(const TX* x, int64_t ldx, const TW* __restrict__ w,
                                                       const TW* __restrict__ b, TX* y, int64_t ldy,
                                                       float* __restrict__ mean, float* __restrict__ rstd, int64_t rows,
                                                       int dim, float eps) {
    __shared__ float red[2][2][32];
    const float inv = 1.0f / (float)dim;
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    int turn = 0;
    int64_t r = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    Vec<TX, V> raw[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * (int)blockDim.x + (int)threadIdx.x) * V;
        if (r < rows && c < dim) raw[k].load(x + r * ldx + c);
    }
    for (; r < rows; r += step) {
        float f[K][V];
        float s[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * (int)blockDim.x + (int)threadIdx.x) * V;
            if (c < dim) {
                raw[k].get(f[k]);
#pragma unroll
                for (int e = 0; e < V; ++e) s[0] += f[k][e];
                if (r + step < rows) raw[k].load(x + (r + step) * ldx + c);
            }
        }
        row_sum(s, red, turn);
        const float mu = s[0] * inv;
        s[0] = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * (int)blockDim.x + (int)threadIdx.x) * V;
            if (c < dim) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    f[k][e] -= mu;
                    s[0] = fmaf(f[k][e], f[k][e], s[0]);
                }
            }
        }
        row_sum(s, red, turn);
        const float rs = 1.0f / sqrtf(fmaf(s[0], inv, eps));
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * (int)blockDim.x + (int)threadIdx.x) * V;
            if (c < dim) {
                Vec<TW, V> wv, bv;
                float wf[V], bf[V];
                wv.load(w + c);
                wv.get(wf);
#pragma unroll
                for (int e = 0; e < V; ++e) bf[e] = 0.0f;
                if (b) {
                    bv.load(b + c);
                    bv.get(bf);
                }
#pragma unroll
                for (int e = 0; e < V; ++e) f[k][e] = fmaf(f[k][e] * rs, wf[e], bf[e]);
                Vec<TX, V>::store(y + r * ldy + c, f[k]);
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
// joined by k_norm_join in CTA order).
template <class TX, class TW, int V, int K, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads) k_norm_backward(const TX* dy, int64_t lddy, const TX* x, int64_t ldx,
                                                               const TW* __restrict__ w, const float* __restrict__ mean,
                                                               const float* __restrict__ rstd, TX* dx, int64_t lddx,
                                                               float* __restrict__ partial, int64_t rows, int dim) {
    __shared__ float red[2][2][32];
    extern __shared__ float cols[];   // [2][dim], only when blockDim.y > 1
    constexpr bool kPre = K * V <= 16;   // the next row on its way: more would not fit in registers
    const float inv = 1.0f / (float)dim;
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    int turn = 0;
    float aw[K][V], ab[K][V], wf[K][V];
    Vec<TX, V> rx[K], rg[K];
    int64_t r = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    float mu = 0.0f, rs = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * (int)blockDim.x + (int)threadIdx.x) * V;
#pragma unroll
        for (int e = 0; e < V; ++e) aw[k][e] = ab[k][e] = 0.0f;
        if (c < dim) {
            Vec<TW, V> wv;
            wv.load(w + c);
            wv.get(wf[k]);
            if (kPre && r < rows) {
                rx[k].load(x + r * ldx + c);
                rg[k].load(dy + r * lddy + c);
            }
        }
    }
    if (kPre && r < rows) {
        mu = mean[r];
        rs = rstd[r];
    }
    for (; r < rows; r += step) {
        if (!kPre) {
            mu = mean[r];
            rs = rstd[r];
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = (k * (int)blockDim.x + (int)threadIdx.x) * V;
                if (c < dim) {
                    rx[k].load(x + r * ldx + c);
                    rg[k].load(dy + r * lddy + c);
                }
            }
        }
        Vec<TX, V> nx[K], ng[K];
        float nmu = 0.0f, nrs = 0.0f;
        if (kPre && r + step < rows) {
            nmu = mean[r + step];
            nrs = rstd[r + step];
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = (k * (int)blockDim.x + (int)threadIdx.x) * V;
                if (c < dim) {
                    nx[k].load(x + (r + step) * ldx + c);
                    ng[k].load(dy + (r + step) * lddy + c);
                }
            }
        }
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * (int)blockDim.x + (int)threadIdx.x) * V;
            if (c < dim) {
                float fx[V], fg[V];
                rx[k].get(fx);
                rg[k].get(fg);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float xh = (fx[e] - mu) * rs, a = fg[e] * wf[k][e];
                    aw[k][e] = fmaf(fg[e], xh, aw[k][e]);
                    ab[k][e] += fg[e];
                    s[0] += a;
                    s[1] = fmaf(a, xh, s[1]);
                }
            }
        }
        if (dx) {   // uniform: the barrier inside is reached by all threads or none
            row_sum(s, red, turn);
            const float m1 = s[0] * inv, m2 = s[1] * inv;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = (k * (int)blockDim.x + (int)threadIdx.x) * V;
                if (c < dim) {
                    float fx[V], fg[V];
                    rx[k].get(fx);
                    rg[k].get(fg);
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        fg[e] = rs * (fmaf(-((fx[e] - mu) * rs), m2, fg[e] * wf[k][e]) - m1);
                    Vec<TX, V>::store(dx + r * lddx + c, fg);
                }
            }
        }
        if (kPre) {
            mu = nmu;
            rs = nrs;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                rx[k] = nx[k];
                rg[k] = ng[k];
            }
        }
    }
    if (!partial) return;
    float* const out = partial + (int64_t)blockIdx.x * 2 * dim;
    for (int turn_y = 0; turn_y < (int)blockDim.y; ++turn_y) {   // rows of warps add up in their order
        if ((int)threadIdx.y == turn_y) {
            const bool last = turn_y + 1 == (int)blockDim.y;
#pragma unroll
            for (int k = 0; k < K; ++k) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const int c = (k * (int)blockDim.x + (int)threadIdx.x) * V + e;
                    if (c < dim) {
                        const float pw = turn_y ? cols[c] + aw[k][e] : aw[k][e];
                        const float pb = turn_y ? cols[dim + c] + ab[k][e] : ab[k][e];
                        (last ? out : cols)[c] = pw;
                        (last ? out : cols)[dim + c] = pb;
                    }
                }
            }
        }
        if (blockDim.y > 1) __syncthreads();
    }
}

// Sum of the partial rows: column j of [2][dim] over `slices`, eight threads each a slice in eight, then their
// sums in order.
template <class TW>
__global__ void __launch_bounds__(kThreads) k_norm_join(const float* __restrict__ partial, int slices, TW* __restrict__ dw,
                                                        TW* __restrict__ db, int64_t dim) {
    __shared__ float red[8][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t j = (int64_t)blockIdx.x * 32 + tx;
    float s = 0.0f;
    if (j < 2 * dim)
        for (int k = ty; k < slices; k += 8) s += partial[(int64_t)k * 2 * dim + j];
    red[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && j < 2 * dim) {
        s = red[0][tx];
        for (int k = 1; k < 8; ++k) s += red[k][tx];
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

// Partial rows of the weight's gradient at most: 4 CTAs on each of 152 SMs.
constexpr int kMaxSlices = 608;

unsigned row_grid(int64_t rows) { return (unsigned)std::min<int64_t>(rows, (int64_t)sm_count() * 8); }

bool rows_aligned(const void* p, int64_t ld, size_t elem) { return is_aligned(p, 16) && (size_t)ld * elem % 16 == 0; }

// How a row is laid over threads: V elements a vector, K vectors a thread, tx threads, ty rows a CTA.
struct RowShape {
    int V = 0, K = 0, tx = 0, ty = 1;   // K = 0: too long
};
// Few threads with several vectors each keep a row inside one warp where it fits (no barrier);
// above that two vectors each -- enough loads in flight, and room in the registers for the next
// row -- up to `max_threads`, then four.  Rows that cannot be read in 16-byte vectors (odd width,
// stride or start) take single elements, eight or sixteen a thread.
RowShape row_shape(int64_t dim, int vec, bool aligned, int max_threads) {
    RowShape s;
    s.V = aligned && dim % vec == 0 ? vec : 1;
    const int64_t units = dim / s.V;
    const int k_warp = s.V > 1 ? 4 : 8, k_few = s.V > 1 ? 2 : 8, k_many = s.V > 1 ? 4 : 16;
    if (units <= 32 * k_warp) {
        s.K = k_warp;
        s.tx = 32;
        s.ty = 4;
        return s;
    }
    for (int k : {k_few, k_many}) {
        const int64_t t = (units + k - 1) / k;
        if (t <= max_threads) {
            s.K = k;
            s.tx = (int)((t + 31) / 32 * 32);
            return s;
        }
    }
    return s;
}

// CTAs of one kernel that fit on the GPU at once.
template <class F>
int64_t resident(F kernel, int threads, size_t smem) {
    int per_sm = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem) != cudaSuccess || per_sm < 1) per_sm = 1;
    return (int64_t)per_sm * sm_count();
}

template <class TX, class TW, int V, int K>
int forward_rows(const NormForward& a, const RowShape& sh, cudaStream_t s) {
    auto kernel = k_norm_forward<TX, TW, V, K>;
    const int64_t grid = std::min((a.rows + sh.ty - 1) / sh.ty, resident(kernel, sh.tx * sh.ty, 0));
    kernel<<<(unsigned)grid, dim3(sh.tx, sh.ty), 0, s>>>(
        static_cast<const TX*>(a.x), a.ldx, static_cast<const TW*>(a.weight), static_cast<const TW*>(a.bias),
        static_cast<TX*>(a.y), a.ldy, a.mean, a.rstd, a.rows, (int)a.dim, a.eps);
    return check_cuda(cudaGetLastError(), "layer norm launch");
}

template <class TX, class TW>
int forward_t(const NormForward& a, cudaStream_t s) {
    constexpr int kVec = 16 / sizeof(TX);
    const bool aligned = rows_aligned(a.x, a.ldx, sizeof(TX)) && rows_aligned(a.y, a.ldy, sizeof(TX)) &&
                         is_aligned(a.weight, 16) && is_aligned(a.bias, 16);
    const RowShape sh = row_shape(a.dim, kVec, aligned, 1024);
    if (sh.V > 1 && sh.K == 2) return forward_rows<TX, TW, kVec, 2>(a, sh, s);
    if (sh.V > 1 && sh.K == 4) return forward_rows<TX, TW, kVec, 4>(a, sh, s);
    if (sh.V == 1 && sh.K == 8) return forward_rows<TX, TW, 1, 8>(a, sh, s);
    if (sh.V == 1 && sh.K == 16) return forward_rows<TX, TW, 1, 16>(a, sh, s);
    k_norm_forward_long<TX, TW><<<row_grid(a.rows), kThreads, 0, s>>>(
        static_cast<const TX*>(a.x), a.ldx, static_cast<const TW*>(a.weight), static_cast<const TW*>(a.bias),
        static_cast<TX*>(a.y), a.ldy, a.mean, a.rstd, a.rows, a.dim, a.eps);
    return check_cuda(cudaGetLastError(), "layer norm launch");
}

template <class TW>
int join_slices(const NormBackward& a, int slices, cudaStream_t s) {
    k_norm_join<TW><<<(unsigned)((2 * a.dim + 31) / 32), kThreads, 0, s>>>(a.partial, slices, static_cast<TW*>(a.dweight),
                                                                          static_cast<TW*>(a.dbias), a.dim);
    return check_cuda(cudaGetLastError(), "layer norm weight gradient launch");
}

template <class TX, class TW, int V, int K>
int backward_rows(const NormBackward& a, const RowShape& sh, cudaStream_t s) {
    auto kernel = k_norm_backward<TX, TW, V, K, 512>;
    const bool sums = a.dweight || a.dbias;
    const size_t smem = sh.ty > 1 ? 2 * sizeof(float) * (size_t)a.dim : 0;
    const int64_t grid = std::max<int64_t>(1, std::min({(a.rows + sh.ty - 1) / sh.ty, (int64_t)kMaxSlices,
                                                        resident(kernel, sh.tx * sh.ty, smem)}));
    kernel<<<(unsigned)grid, dim3(sh.tx, sh.ty), smem, s>>>(
        static_cast<const TX*>(a.dy), a.lddy, static_cast<const TX*>(a.x), a.ldx, static_cast<const TW*>(a.weight), a.mean,
        a.rstd, static_cast<TX*>(a.dx), a.lddx, sums ? a.partial : nullptr, a.rows, (int)a.dim);
    const int rc = check_cuda(cudaGetLastError(), "layer norm backward launch");
    return rc || !sums ? rc : join_slices<TW>(a, (int)grid, s);
}

template <class TX, class TW>
int backward_t(const NormBackward& a, cudaStream_t s) {
    constexpr int kVec = 16 / sizeof(TX);
    const bool aligned = rows_aligned(a.x, a.ldx, sizeof(TX)) && rows_aligned(a.dy, a.lddy, sizeof(TX)) &&
                         (!a.dx || rows_aligned(a.dx, a.lddx, sizeof(TX))) && is_aligned(a.weight, 16);
    const RowShape sh = row_shape(a.dim, kVec, aligned, 512);
    if (sh.V > 1 && sh.K == 2) return backward_rows<TX, TW, kVec, 2>(a, sh, s);
    if (sh.V > 1 && sh.K == 4) return backward_rows<TX, TW, kVec, 4>(a, sh, s);
    if (sh.V == 1 && sh.K == 8) return backward_rows<TX, TW, 1, 8>(a, sh, s);
    if (sh.V == 1 && sh.K == 16) return backward_rows<TX, TW, 1, 16>(a, sh, s);
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
