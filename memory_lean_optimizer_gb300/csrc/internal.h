// internal.h -- host-side declarations shared by the library's translation units.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <vector>

#include "common.cuh"

namespace lmo {

// True when the environment variable LMOPT_FAULT_INJECT equals `what` (host-side fault
// injection for the error-path tests: h2d, d2h, alloc, timeout, stall_*).
bool fault_injected(const char* what);
// True when it is set at all.
bool faults_injected();
// Records the thread-local error message and returns `code`.
int set_error(int code, const char* fmt, ...);
// OPTIM_OK if e == cudaSuccess, else records "<what>: <cuda message>" and returns OPTIM_ECUDA.
int check_cuda(cudaError_t e, const char* what);
// Streaming-multiprocessor count of the current device (cached per device).
int sm_count();
// Grid for a grid-stride elementwise kernel over `units` work units of kThreads each.
unsigned grid_for(int64_t units);

// Lets a kernel use `bytes` of dynamic shared memory on the current device, once for each device (`done`: a bit
// each, one word per kernel).
template <class F>
int allow_smem(F kernel, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    int rc = check_cuda(cudaGetDevice(&dev), "cudaGetDevice");
    if (rc) return rc;
    const uint64_t bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_relaxed) & bit) return OPTIM_OK;
    rc = check_cuda(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes), "kernel shared memory");
    if (!rc) done.fetch_or(bit, std::memory_order_relaxed);
    return rc;
}

inline bool is_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// ---- launchers (each returns OPTIM_OK or OPTIM_ECUDA after checking the launch) ----
int launch_kahan_split(const float* src, uint16_t* hi, uint16_t* lo, int64_t n, cudaStream_t s);
int launch_kahan_merge(const uint16_t* hi, const uint16_t* lo, float* dst, int64_t n, cudaStream_t s);
int launch_state_pack(const float* src, uint16_t* codes, float* scale, int64_t n, int is_signed,
                      cudaStream_t s);
int launch_state_unpack(const uint16_t* codes, const float* scale, float* dst, int64_t n,
                        int is_signed, cudaStream_t s);

// Per-step scalars of the NAdam/Adam kernel (host-computed: double, then one rounding).
struct NadamScalars {
    float lr, b1, omb1, b2, omb2, eps, lr_wd, c_m, c_g, k2;
    int32_t decoupled;
    int32_t parity;
    int32_t sr;        // stochastic rounding for tensors without a residual
    uint64_t seed;
    uint64_t step;
};

struct NadamLaunch {
    const TensorRec* tensors;
    const uint16_t* const* grads;
    ScaleRec* scales;
    const Chunk* chunks;
    unsigned long long* nonfinite;
    int32_t n_chunks_large;   // chunks of u16-state tensors come first
    int32_t n_chunks_total;
    int32_t f24;              // moments stored as f24 planes instead of u16 codes
    uint8_t* zero_chunk;      // per u16 chunk: the gradient pre-pass saw an exact zero (K2 then
                              // takes the zero-guarded arithmetic for that chunk)
    int64_t chunk;            // elements per chunk (a power of two, kChunkMin..kChunkU16)
};
// K1 (gradient maxima; nothing for f24 moments), then K2 (the update; `mid`, if not null, is
// recorded on the stream before it).  A step is both, in this order, on one stream.
int launch_nadam_prepass(const NadamLaunch& L, const NadamScalars& k, cudaStream_t s);
int launch_nadam_update(const NadamLaunch& L, const NadamScalars& k, cudaStream_t s, cudaEvent_t mid);
// The pre-pass and the update in one cooperative launch (one CTA per chunk), for groups whose
// chunks all fit on the GPU at once: nadam_fused_capacity() chunks at most (0: not available).
// bar: the group's barrier counter; target: its value once every CTA of this launch has arrived.
int nadam_fused_capacity(bool sr);
int launch_nadam_fused(const NadamLaunch& L, const NadamScalars& k, cudaStream_t s, unsigned* bar, unsigned target);
// Per tensor {G (this step), A_m, A_v (previous step)} to / from 3 consecutive floats.
int launch_scales_gather(const ScaleRec* sc, float* buf, int n, int parity, cudaStream_t s);
int launch_scales_scatter(ScaleRec* sc, const float* buf, int n, int parity, cudaStream_t s);

// Per-step scalars of the Adan kernel.
struct AdanScalars {
    float lr, b1, omb1, b2, omb2, b3, omb3, eps, inv_decay;
    int32_t sr;
    int64_t step;
    uint64_t seed;
};
int launch_adan_step(const NadamLaunch& L, const AdanScalars& k, cudaStream_t s);

// Per-step scalars of the AdamW kernel (grad_scale: a device scalar, or NULL for 1).
struct AdamWScalars {
    float b1, omb1, b2, omb2, eps, lr_wd, k1, k2;
    const float* grad_scale;
    int32_t sr;
    int64_t step;
    uint64_t seed;
};
// u8: tensors above kSmall elements keep 8-bit states (OPTIM_KIND_ADAMW_U8).
int launch_adamw_step(const NadamLaunch& L, const AdamWScalars& k, bool u8, cudaStream_t s);
// Every tensor's moments as fp32, into flat buffers laid out by TensorRec::slot64.
int launch_adamw_unpack(const NadamLaunch& L, bool u8, float* m, float* v, cudaStream_t s);

// Layer norm over rows of dim elements (row strides ld*, in elements; types by the two flags).
struct NormForward {
    const void* x;
    int64_t ldx;
    const void* weight;
    const void* bias;      // or NULL
    void* y;
    int64_t ldy;
    float* mean;           // or NULL
    float* rstd;           // or NULL
    int64_t rows, dim;
    float eps;
    bool x_bf16, w_bf16;   // else fp32
};
struct NormBackward {
    const void* dy;
    int64_t lddy;
    const void* x;
    int64_t ldx;
    const void* weight;
    const float* mean;
    const float* rstd;
    void* dx;              // or NULL
    int64_t lddx;
    void* dweight;         // or NULL
    void* dbias;           // or NULL
    float* partial;        // norm_partial_bytes
    int64_t rows, dim;
    bool x_bf16, w_bf16;
};
size_t norm_partial_bytes(int64_t rows, int64_t dim);
int launch_norm_forward(const NormForward& a, cudaStream_t s);
int launch_norm_backward(const NormBackward& a, cudaStream_t s);

// Softmax cross entropy of hidden [rows][dim] against weight [vocab][dim] (bf16, row strides ld*).
struct XentCall {
    const void* hidden;
    int64_t ldh;
    const void* weight;
    int64_t ldw;
    const int64_t* target;
    int64_t rows, dim, vocab, ignore_index;
    float* loss;              // forward: output
    float* lse;               // forward: output; backward: input
    const float* grad_loss;   // backward: factor of each row's loss
    bool backward;
    void* d_hidden;           // backward, or NULL
    int64_t lddh;
    void* d_weight;           // backward, or NULL
    int64_t lddw;
    void* workspace;
    size_t workspace_bytes;
};
size_t xent_workspace_bytes(int64_t rows, int64_t dim, int64_t vocab, const void* weight, int64_t ldw, bool backward);
int launch_xent(const XentCall& c, cudaStream_t s);

}  // namespace lmo
