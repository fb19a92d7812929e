// norm.cu -- layer norm over the rows of a matrix, forward and backward.
//   mu = mean x, r = 1 / sqrt(mean (x - mu)^2 + eps), y = (x - mu) r w + b
//   xh = (x - mu) r, a = dy w, dx = r (a - mean a - xh mean(a xh)), dw = sum_rows dy xh, db = sum_rows dy
// Values are fp32 from load to store, whatever the types; the variance is taken around the mean
// (a second sum over the row), not as a difference of squares.  Sums run in a fixed order, so two
// runs agree bit for bit.
#include <algorithm>

#include "internal.h"

namespace lmo {
namespace {

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }
__device__ __forceinline__ void store1(uint16_t* p, float x) { *p = (uint16_t)rne_bf16(x); }

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
__global__ void __launch_bounds__(kThreads) k_norm_forward(const TX* x, int64_t ldx, const TW* __restrict__ w,
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
__global__ void __launch_bounds__(kThreads) k_norm_dx(const TX* dy, int64_t lddy, const TX* __restrict__ x,
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
__global__ void __launch_bounds__(kThreads) k_norm_dw(const TX* __restrict__ dy, int64_t lddy, const TX* __restrict__ x,
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

template <class TW>
__global__ void __launch_bounds__(kThreads) k_norm_join(const float* __restrict__ partial, int slices, TW* __restrict__ dw,
                                                        TW* __restrict__ db, int64_t dim) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (c >= dim) return;
    float sw = 0.0f, sb = 0.0f;
    for (int k = 0; k < slices; ++k) {
        sw += partial[(int64_t)k * 2 * dim + c];
        sb += partial[((int64_t)k * 2 + 1) * dim + c];
    }
    if (dw) store1(dw + c, sw);
    if (db) store1(db + c, sb);
}

int norm_slices(int64_t rows) { return (int)std::max<int64_t>(1, std::min<int64_t>((rows + 63) / 64, 256)); }

unsigned row_grid(int64_t rows) { return (unsigned)std::min<int64_t>(rows, (int64_t)sm_count() * 8); }

template <class TX, class TW>
int forward_t(const NormForward& a, cudaStream_t s) {
    k_norm_forward<TX, TW><<<row_grid(a.rows), kThreads, 0, s>>>(
        static_cast<const TX*>(a.x), a.ldx, static_cast<const TW*>(a.weight), static_cast<const TW*>(a.bias),
        static_cast<TX*>(a.y), a.ldy, a.mean, a.rstd, a.rows, a.dim, a.eps);
    return check_cuda(cudaGetLastError(), "layer norm launch");
}

template <class TX, class TW>
int backward_t(const NormBackward& a, cudaStream_t s) {
    const TX* dy = static_cast<const TX*>(a.dy);
    const TX* x = static_cast<const TX*>(a.x);
    if (a.dweight || a.dbias) {   // before dx, which may lie over dy
        const int slices = norm_slices(a.rows);
        k_norm_dw<TX><<<dim3((unsigned)((a.dim + 31) / 32), (unsigned)slices), kThreads, 0, s>>>(
            dy, a.lddy, x, a.ldx, a.mean, a.rstd, a.partial, a.rows, a.dim);
        k_norm_join<TW><<<(unsigned)((a.dim + kThreads - 1) / kThreads), kThreads, 0, s>>>(
            a.partial, slices, static_cast<TW*>(a.dweight), static_cast<TW*>(a.dbias), a.dim);
        const int rc = check_cuda(cudaGetLastError(), "layer norm weight gradient launch");
        if (rc) return rc;
    }
    if (!a.dx || a.rows == 0) return OPTIM_OK;
    k_norm_dx<TX, TW><<<row_grid(a.rows), kThreads, 0, s>>>(dy, a.lddy, x, a.ldx, static_cast<const TW*>(a.weight),
                                                           a.mean, a.rstd, static_cast<TX*>(a.dx), a.lddx, a.rows, a.dim);
    return check_cuda(cudaGetLastError(), "layer norm backward launch");
}

}  // namespace

size_t norm_partial_bytes(int64_t rows, int64_t dim) { return (size_t)norm_slices(rows) * 2 * (size_t)dim * sizeof(float); }

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
