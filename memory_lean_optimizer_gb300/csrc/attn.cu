// attn.cu -- the attention calls: what they accept.
#include "attn.cuh"

using namespace lmo;

namespace {

int check_attn(const AttnCall& c) {
    if (c.seq.rows < 0 || c.seq.rows >= ((int64_t)1 << 31) - 512) return set_error(OPTIM_EINVAL, "rows must lie in [0, 2^31 - 512)");
    if (c.seq.n < 0 || c.seq.n > (1 << 30)) return set_error(OPTIM_EINVAL, "need 0 to 2^30 sequences");
    if (!c.seq.cu && (c.seq.n < 1 || c.seq.rows % c.seq.n)) return set_error(OPTIM_EINVAL, "%lld rows are not %d sequences of one length", (long long)c.seq.rows, c.seq.n);
    if (!is_aligned(c.seq.cu, 4)) return set_error(OPTIM_EALIGN, "cu_seqlens not 4-byte aligned");
    if (c.dim < 8 || c.dim > 128 || c.dim % 8) return set_error(OPTIM_EINVAL, "heads must have 8 to 128 elements, a multiple of 8, not %lld", (long long)c.dim);
    if (c.heads < 1 || c.kv_heads < 1 || c.heads > 65536 || c.heads % c.kv_heads)
        return set_error(OPTIM_EINVAL, "%lld query heads cannot share %lld key heads", (long long)c.heads, (long long)c.kv_heads);
    if (!(c.scale > 0.0f && c.scale * kLog2e <= FLT_MAX))      // scores are taken in powers of two
        return set_error(OPTIM_EINVAL, "scale must be positive and finite, times log2(e) too");
    if (tile_slots(c.seq, 64) > (((int64_t)1 << 31) - 1) / c.heads) return set_error(OPTIM_EINVAL, "too many rows, sequences and heads");
    return OPTIM_OK;
}

int check_heads(const HeadRows& t, int64_t rows, int64_t heads, int64_t dim, const char* name) {
    if (!t.p) return set_error(OPTIM_EINVAL, "%s is NULL", name);
    if ((heads > 1 && t.head < dim) || (rows > 1 && t.row < dim) || t.row >= ((int64_t)1 << 38) || t.head >= ((int64_t)1 << 38))
        return set_error(OPTIM_EINVAL, "%s: strides of %lld and %lld elements for heads of %lld", name, (long long)t.row, (long long)t.head, (long long)dim);
    if (!is_aligned(t.p, 16) || (heads > 1 && t.head % 8) || (rows > 1 && t.row % 8))
        return set_error(OPTIM_EALIGN, "%s: heads must start on 16 bytes", name);
    return OPTIM_OK;
}

// Places of an output must not meet.
int check_out(const HeadRows& t, int64_t rows, int64_t heads, int64_t dim, const char* name) {
    const int rc = check_heads(t, rows, heads, dim, name);
    if (rc) return rc;
    if (heads > 1 && rows > 1 && t.row < (heads - 1) * t.head + dim && t.head < (rows - 1) * t.row + dim)
        return set_error(OPTIM_EINVAL, "%s: rows and heads overlap", name);
    return OPTIM_OK;
}

}  // namespace

extern "C" {

int attn_forward(const void* q, int64_t q_row, int64_t q_head, const void* k, int64_t k_row, int64_t k_head, const void* v, int64_t v_row,
                 int64_t v_head, void* out, int64_t out_row, int64_t out_head, float* lse, const int32_t* cu_seqlens, int64_t sequences,
                 int64_t rows, int64_t heads, int64_t kv_heads, int64_t dim, float scale, void* stream) {
    if (sequences < 0 || sequences > (1 << 30)) return set_error(OPTIM_EINVAL, "need 0 to 2^30 sequences");
    AttnCall c{};
    c.q = {const_cast<void*>(q), q_row, q_head}, c.k = {const_cast<void*>(k), k_row, k_head}, c.v = {const_cast<void*>(v), v_row, v_head};
    c.out = {out, out_row, out_head};
    c.lse = lse;
    c.seq = {cu_seqlens, (int32_t)sequences, rows};
    c.heads = heads, c.kv_heads = kv_heads, c.dim = dim, c.scale = scale;
    int rc = check_attn(c);
    if (rc || rows == 0) return rc;
    rc = check_heads(c.q, rows, heads, dim, "q");
    if (!rc) rc = check_heads(c.k, rows, kv_heads, dim, "k");
    if (!rc) rc = check_heads(c.v, rows, kv_heads, dim, "v");
    if (!rc) rc = check_out(c.out, rows, heads, dim, "out");
    if (!rc && !lse) rc = set_error(OPTIM_EINVAL, "lse is NULL");
    if (!rc && !is_aligned(lse, 4)) rc = set_error(OPTIM_EALIGN, "lse not 4-byte aligned");
    return rc ? rc : launch_attn_forward(c, static_cast<cudaStream_t>(stream));
}

int attn_workspace(const int32_t* cu_seqlens, int64_t sequences, int64_t rows, int64_t heads, int64_t kv_heads, int64_t dim, size_t* bytes) {
    if (sequences < 0 || sequences > (1 << 30)) return set_error(OPTIM_EINVAL, "need 0 to 2^30 sequences");
    AttnCall c{};
    c.seq = {cu_seqlens, (int32_t)sequences, rows};
    c.heads = heads, c.kv_heads = kv_heads, c.dim = dim, c.scale = 1.0f;
    const int rc = check_attn(c);
    if (rc) return rc;
    if (!bytes) return set_error(OPTIM_EINVAL, "bytes is NULL");
    *bytes = attn_workspace_bytes(c);
    return OPTIM_OK;
}

int attn_backward(const void* d_out, int64_t do_row, int64_t do_head, const void* q, int64_t q_row, int64_t q_head, const void* k,
                  int64_t k_row, int64_t k_head, const void* v, int64_t v_row, int64_t v_head, const void* out, int64_t out_row,
                  int64_t out_head, const float* lse, void* dq, int64_t dq_row, int64_t dq_head, void* dk, int64_t dk_row, int64_t dk_head,
                  void* dv, int64_t dv_row, int64_t dv_head, const int32_t* cu_seqlens, int64_t sequences, int64_t rows, int64_t heads,
                  int64_t kv_heads, int64_t dim, float scale, void* workspace, size_t workspace_bytes, void* stream) {
    if (sequences < 0 || sequences > (1 << 30)) return set_error(OPTIM_EINVAL, "need 0 to 2^30 sequences");
    AttnCall c{};
    c.q = {const_cast<void*>(q), q_row, q_head}, c.k = {const_cast<void*>(k), k_row, k_head}, c.v = {const_cast<void*>(v), v_row, v_head};
    c.out = {const_cast<void*>(out), out_row, out_head}, c.d_out = {const_cast<void*>(d_out), do_row, do_head};
    c.dq = {dq, dq_row, dq_head}, c.dk = {dk, dk_row, dk_head}, c.dv = {dv, dv_row, dv_head};
    c.lse = const_cast<float*>(lse);
    c.seq = {cu_seqlens, (int32_t)sequences, rows};
    c.heads = heads, c.kv_heads = kv_heads, c.dim = dim, c.scale = scale;
    c.workspace = workspace;
    int rc = check_attn(c);
    if (!rc && !dk != !dv) rc = set_error(OPTIM_EINVAL, "dk and dv go together");
    if (rc || rows == 0 || (!dq && !dk)) return rc;
    rc = check_heads(c.d_out, rows, heads, dim, "d_out");
    if (!rc) rc = check_heads(c.q, rows, heads, dim, "q");
    if (!rc) rc = check_heads(c.k, rows, kv_heads, dim, "k");
    if (!rc) rc = check_heads(c.v, rows, kv_heads, dim, "v");
    if (!rc) rc = check_heads(c.out, rows, heads, dim, "out");
    if (!rc && !lse) rc = set_error(OPTIM_EINVAL, "lse is NULL");
    if (!rc && !is_aligned(lse, 4)) rc = set_error(OPTIM_EALIGN, "lse not 4-byte aligned");
    if (!rc && dq) rc = check_out(c.dq, rows, heads, dim, "dq");
    if (!rc && dk) rc = check_out(c.dk, rows, kv_heads, dim, "dk");
    if (!rc && dv) rc = check_out(c.dv, rows, kv_heads, dim, "dv");
    const size_t need = attn_workspace_bytes(c);
    if (!rc && !workspace) rc = set_error(OPTIM_EINVAL, "workspace is NULL");
    if (!rc && !is_aligned(workspace, 256)) rc = set_error(OPTIM_EALIGN, "workspace not 256-byte aligned");
    if (!rc && workspace_bytes < need) rc = set_error(OPTIM_EINVAL, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
    return rc ? rc : launch_attn_backward(c, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
