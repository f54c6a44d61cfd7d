// Host side of the C ABI of the gated linear recurrence, the 8-bit activation
// checkpoints and the RMS norm: argument validation and dispatch to the HIP
// launchers.  Every check here runs before any HIP call, so invalid arguments
// never reach the device.
#include <math.h>
#include <stdint.h>

#include "kda.h"
#include "kda_ops_launch.h"

namespace {

bool valid_dtype(int32_t t) { return t == KDA_F32 || t == KDA_BF16; }
uintptr_t dsize(int32_t t) { return t == KDA_F32 ? 4 : 2; }
bool aligned_to(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
// A required pointer with its element alignment; an optional one.
bool req(const void *p, uintptr_t a) { return p && aligned_to(p, a); }
bool opt(const void *p, uintptr_t a) { return aligned_to(p, a); }

// Row lengths above this are refused: kernels hold a position in a row, and a few
// lanes' width behind its end, in 32 bits.
constexpr int32_t kMaxRow = 1 << 30;

// a * b stays well inside int64 for device indexing.
bool product_fits(int64_t a, int64_t b) {
    const int64_t lim = (int64_t)1 << 50;
    return a <= lim && b <= lim && (b == 0 || a <= lim / b);
}

kda_status_t finish(int rc) { return rc != 0 ? KDA_ERR_HIP : KDA_OK; }
char *fresh_error(size_t *len) {
    char *e = kda::hip_error_text(len);
    e[0] = '\0';
    return e;
}

bool glr_sizes_ok(int32_t B, int32_t T, int32_t D, int64_t N) {
    if (B <= 0 || T < 0 || D <= 0 || N < 0) return false;
    return product_fits((int64_t)B * T, D) && product_fits(N, D);
}

kda::GlrArgs glr_sizes(int32_t B, int32_t T, int32_t D, int32_t num_seqs, bool varlen, int32_t io_dtype) {
    kda::GlrArgs a = {};
    // the address is not read: it says that the batch is packed
    a.cu_seqlens = varlen ? reinterpret_cast<const int32_t *>(uintptr_t(16)) : nullptr;
    a.num_seqs = varlen ? num_seqs : B;
    a.seq_len = T;
    a.tokens = (int64_t)B * T;
    a.D = D;
    a.io_bf16 = io_dtype == KDA_BF16;
    return a;
}

// Shared by the forward and the backward: `backward` says which pointers apply.
kda_status_t glr_impl(bool backward, const void *x, const void *log_alpha, const void *h_in, const float *h_scales,
                      bool act8, const float *h0, const int32_t *cu_seqlens, int32_t num_seqs, const float *d_hT,
                      void *out, void *dlog_alpha, float *state_out, int32_t B, int32_t T, int32_t D,
                      int32_t io_dtype, int32_t gate_dtype, void *workspace, size_t workspace_bytes, void *stream) {
    if (!valid_dtype(io_dtype) || !valid_dtype(gate_dtype)) return KDA_ERR_UNSUPPORTED;
    if (cu_seqlens) {
        if (B != 1 || num_seqs <= 0 || !aligned_to(cu_seqlens, 4)) return KDA_ERR_INVALID_ARGUMENT;
    } else if (num_seqs != 0 && num_seqs != B) {
        return KDA_ERR_INVALID_ARGUMENT;
    }
    if (!glr_sizes_ok(B, T, D, cu_seqlens ? num_seqs : B)) return KDA_ERR_INVALID_ARGUMENT;
    if (D > kMaxRow) return KDA_ERR_UNSUPPORTED;
    const bool have_tokens = T > 0;
    const uintptr_t ios = dsize(io_dtype), gs = dsize(gate_dtype);
    if (have_tokens) {
        if (!req(x, ios) || !req(log_alpha, gs) || !req(out, ios)) return KDA_ERR_INVALID_ARGUMENT;
        if (backward && (!req(h_in, act8 ? 1 : ios) || !req(dlog_alpha, gs))) return KDA_ERR_INVALID_ARGUMENT;
        if (act8 && !req(h_scales, 4)) return KDA_ERR_INVALID_ARGUMENT;
    }
    if (!opt(h0, 4) || !opt(d_hT, 4) || !opt(state_out, 4)) return KDA_ERR_INVALID_ARGUMENT;
    kda::GlrArgs a = glr_sizes(B, T, D, num_seqs, cu_seqlens != nullptr, io_dtype);
    a.gate_bf16 = gate_dtype == KDA_BF16;
    a.backward = backward;
    if (!kda::glr_grids_fit(a)) return KDA_ERR_UNSUPPORTED;
    const size_t need = kda::glr_workspace_bytes(a);
    if (need > 0 && (workspace_bytes < need || !workspace)) return KDA_ERR_WORKSPACE;
    if (workspace && !aligned_to(workspace, 16)) return KDA_ERR_INVALID_ARGUMENT;
    if (!have_tokens && !state_out) return KDA_OK;
    a.x = x; a.log_alpha = log_alpha; a.h_in = h_in; a.h_scales = act8 ? h_scales : nullptr;
    a.h0 = h0; a.d_hT = d_hT; a.cu_seqlens = cu_seqlens;
    a.out = out; a.dlog_alpha = dlog_alpha; a.state_out = state_out;
    a.workspace = workspace; a.workspace_bytes = workspace_bytes;
    size_t len;
    char *err = fresh_error(&len);
    return finish(kda::launch_glr(a, stream, err, len));
}

kda_status_t act8_impl(bool pack, const void *x, void *out, const int8_t *codes, const float *scales, int64_t rows,
                       int32_t cols, int32_t io_dtype, void *stream) {
    if (!valid_dtype(io_dtype)) return KDA_ERR_UNSUPPORTED;
    if (rows < 0 || cols <= 0 || !product_fits(rows, cols)) return KDA_ERR_INVALID_ARGUMENT;
    if (cols > kMaxRow) return KDA_ERR_UNSUPPORTED;
    if (rows == 0) return KDA_OK;
    if (!req(pack ? x : out, dsize(io_dtype)) || !codes || !req(scales, 4)) return KDA_ERR_INVALID_ARGUMENT;
    kda::Act8Args a = {};
    a.x = x; a.out = out;
    a.codes = const_cast<int8_t *>(codes); a.scales = const_cast<float *>(scales);
    a.rows = rows; a.cols = cols; a.io_bf16 = io_dtype == KDA_BF16;
    if (!kda::act8_grids_fit(a)) return KDA_ERR_UNSUPPORTED;
    size_t len;
    char *err = fresh_error(&len);
    return finish(pack ? kda::launch_act8_pack(a, stream, err, len) : kda::launch_act8_unpack(a, stream, err, len));
}

kda_status_t norm_fwd_impl(const void *x, const void *residual, const void *weight, void *y, int8_t *codes,
                           float *scales, bool act8, void *r, float *rstd, int64_t rows, int32_t cols, float eps,
                           int32_t io_dtype, int32_t w_dtype, void *stream) {
    if (!valid_dtype(io_dtype) || !valid_dtype(w_dtype)) return KDA_ERR_UNSUPPORTED;
    if (rows < 0 || cols <= 0 || !product_fits(rows, cols)) return KDA_ERR_INVALID_ARGUMENT;
    if (cols > kMaxRow) return KDA_ERR_UNSUPPORTED;
    if (!isfinite(eps) || eps <= 0.f) return KDA_ERR_INVALID_ARGUMENT;
    const uintptr_t ios = dsize(io_dtype);
    if (!opt(weight, dsize(w_dtype)) || !opt(rstd, 4)) return KDA_ERR_INVALID_ARGUMENT;
    if (rows == 0) return KDA_OK;
    if (!req(x, ios) || !opt(residual, ios) || (residual && !req(r, ios))) return KDA_ERR_INVALID_ARGUMENT;
    if (act8 ? (!codes || !req(scales, 4)) : !req(y, ios)) return KDA_ERR_INVALID_ARGUMENT;
    kda::NormArgs a = {};
    a.x = x; a.residual = residual; a.weight = weight;
    a.y = act8 ? nullptr : y; a.codes = act8 ? codes : nullptr; a.scales = act8 ? scales : nullptr;
    a.r = residual ? r : nullptr; a.rstd = rstd;
    a.rows = rows; a.cols = cols; a.eps = eps;
    a.io_bf16 = io_dtype == KDA_BF16; a.w_bf16 = w_dtype == KDA_BF16;
    if (!kda::norm_grids_fit(a)) return KDA_ERR_UNSUPPORTED;
    size_t len;
    char *err = fresh_error(&len);
    return finish(kda::launch_norm_fwd(a, stream, err, len));
}

kda_status_t norm_bwd_impl(const void *r, const int8_t *codes, const float *scales, bool act8, const void *weight,
                           const float *rstd, const void *grad_y, const void *grad_r, void *grad_x, void *grad_w,
                           int64_t rows, int32_t cols, int32_t io_dtype, int32_t w_dtype, void *workspace,
                           size_t workspace_bytes, void *stream) {
    if (!valid_dtype(io_dtype) || !valid_dtype(w_dtype)) return KDA_ERR_UNSUPPORTED;
    if (rows < 0 || cols <= 0 || !product_fits(rows, cols)) return KDA_ERR_INVALID_ARGUMENT;
    if (cols > kMaxRow) return KDA_ERR_UNSUPPORTED;
    const uintptr_t ios = dsize(io_dtype), ws = dsize(w_dtype);
    if (!opt(weight, ws) || !opt(grad_w, ws)) return KDA_ERR_INVALID_ARGUMENT;
    if (rows > 0) {
        if (act8 ? (!codes || !req(scales, 4)) : !req(r, ios)) return KDA_ERR_INVALID_ARGUMENT;
        if (!req(rstd, 4) || !req(grad_y, ios) || !opt(grad_r, ios) || !req(grad_x, ios))
            return KDA_ERR_INVALID_ARGUMENT;
    } else if (!grad_w) {
        return KDA_OK;
    }
    kda::NormArgs a = {};
    a.x = act8 ? nullptr : r; a.weight = weight;
    a.codes = act8 ? const_cast<int8_t *>(codes) : nullptr; a.scales = act8 ? const_cast<float *>(scales) : nullptr;
    a.rstd = const_cast<float *>(rstd);
    a.grad_y = grad_y; a.grad_r = grad_r; a.grad_x = grad_x; a.grad_w = grad_w;
    a.rows = rows; a.cols = cols;
    a.io_bf16 = io_dtype == KDA_BF16; a.w_bf16 = w_dtype == KDA_BF16;
    if (!kda::norm_grids_fit(a)) return KDA_ERR_UNSUPPORTED;
    if (grad_w && rows > 0) {
        const size_t need = kda::norm_bwd_workspace_bytes(rows, cols);
        if (need > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    }
    if (workspace && !aligned_to(workspace, 16)) return KDA_ERR_INVALID_ARGUMENT;
    a.workspace = workspace; a.workspace_bytes = workspace_bytes;
    size_t len;
    char *err = fresh_error(&len);
    return finish(kda::launch_norm_bwd(a, stream, err, len));
}

// Workspace of the chunkwise backward from 8-bit checkpoints: the backward's
// own, then q, k and v read back in io_dtype.
struct ChunkAct8Layout {
    size_t base, q, k, v, total;
};
size_t up256(size_t x) { return (x + 255) / 256 * 256; }
bool chunk_act8_layout(int32_t B, int32_t T, int32_t H, int32_t d_k, int32_t d_v, int32_t num_seqs, int32_t io_dtype,
                       ChunkAct8Layout &L) {
    // 0 for sizes that the backward refuses (and only for those)
    L.base = kda_chunk_bwd_workspace_size(B, T, H, d_k, d_v, num_seqs, io_dtype);
    if (B <= 0 || T < 0 || H <= 0 || (L.base == 0 && T > 0)) return false;
    const size_t rows = (size_t)B * T * H, e = io_dtype == KDA_F32 ? 4 : 2;
    L.q = up256(L.base);
    L.k = L.q + up256(rows * d_k * e);
    L.v = L.k + up256(rows * d_k * e);
    L.total = L.v + up256(rows * d_v * e);
    return true;
}

kda_status_t chunk_bwd_act8_impl(const int8_t *qc, const float *qs, const int8_t *kc, const float *ks,
                                 const int8_t *vc, const float *vs, const void *log_alpha, const void *beta,
                                 const float *h0, const int32_t *cu_seqlens, int32_t num_seqs, const void *grad_o,
                                 const float *grad_hT, void *grad_q, void *grad_k, void *grad_v, void *grad_log_alpha,
                                 void *grad_beta, float *grad_h0, int32_t B, int32_t T, int32_t H, int32_t d_k,
                                 int32_t d_v, int32_t io_dtype, int32_t gate_dtype, void *workspace,
                                 size_t workspace_bytes, void *stream, bool gdn) {
    const auto bwd = [&](const void *q, const void *k, const void *v, size_t bytes) {
        return (gdn ? kda_gdn_chunk_bwd : kda_chunk_bwd)(q, k, v, log_alpha, beta, h0, cu_seqlens, num_seqs, grad_o,
                                                         grad_hT, grad_q, grad_k, grad_v, grad_log_alpha, grad_beta,
                                                         grad_h0, B, T, H, d_k, d_v, io_dtype, gate_dtype, workspace,
                                                         bytes, stream);
    };
    ChunkAct8Layout L = {};
    const bool sized = valid_dtype(io_dtype) &&
                       chunk_act8_layout(B, T, H, d_k, d_v, cu_seqlens ? num_seqs : 0, io_dtype, L);
    const bool have_tokens = sized && T > 0;
    // every check of the backward comes first, on a call that ends at its
    // workspace check and enqueues nothing
    void *const here = workspace ? workspace : reinterpret_cast<void *>(uintptr_t(256));
    const kda_status_t checked = bwd(here, here, here, 0);
    if (checked != KDA_ERR_WORKSPACE) return checked;
    if (!sized) return KDA_ERR_INVALID_ARGUMENT;
    if (have_tokens && (!qc || !kc || !vc || !req(qs, 4) || !req(ks, 4) || !req(vs, 4)))
        return KDA_ERR_INVALID_ARGUMENT;
    if (!workspace || workspace_bytes < L.total) return KDA_ERR_WORKSPACE;
    if (!aligned_to(workspace, 16)) return KDA_ERR_INVALID_ARGUMENT;
    uint8_t *const ws = static_cast<uint8_t *>(workspace);
    if (have_tokens) {
        const int64_t rows = (int64_t)B * T * H;
        const struct { const int8_t *c; const float *s; size_t at; int32_t d; } part[3] = {
            {qc, qs, L.q, d_k}, {kc, ks, L.k, d_k}, {vc, vs, L.v, d_v}};
        for (const auto &p : part) {
            const kda_status_t rc = kda_act8_unpack(p.c, p.s, ws + p.at, rows, p.d, io_dtype, stream);
            if (rc != KDA_OK) return rc;
        }
    }
    return bwd(ws + L.q, ws + L.k, ws + L.v, L.base);
}

}  // namespace

extern "C" {

size_t kda_glr_workspace_size(int32_t B, int32_t T, int32_t D, int32_t num_seqs, int32_t io_dtype) {
    if (!valid_dtype(io_dtype) || num_seqs < 0 || (num_seqs > 0 && B != 1)) return 0;
    if (!glr_sizes_ok(B, T, D, num_seqs > 0 ? num_seqs : B) || D > kMaxRow) return 0;
    return kda::glr_workspace_bytes(glr_sizes(B, T, D, num_seqs, num_seqs > 0, io_dtype));
}

kda_status_t kda_glr_fwd(const void *x, const void *log_alpha, const float *h0, const int32_t *cu_seqlens,
                         int32_t num_seqs, void *h, float *h_T, int32_t B, int32_t T, int32_t D, int32_t io_dtype,
                         int32_t gate_dtype, void *workspace, size_t workspace_bytes, void *stream) {
    return glr_impl(false, x, log_alpha, nullptr, nullptr, false, h0, cu_seqlens, num_seqs, nullptr, h, nullptr, h_T,
                    B, T, D, io_dtype, gate_dtype, workspace, workspace_bytes, stream);
}

kda_status_t kda_glr_bwd(const void *log_alpha, const void *h, const float *h0, const int32_t *cu_seqlens,
                         int32_t num_seqs, const void *grad_h, const float *grad_hT, void *grad_x,
                         void *grad_log_alpha, float *grad_h0, int32_t B, int32_t T, int32_t D, int32_t io_dtype,
                         int32_t gate_dtype, void *workspace, size_t workspace_bytes, void *stream) {
    return glr_impl(true, grad_h, log_alpha, h, nullptr, false, h0, cu_seqlens, num_seqs, grad_hT, grad_x,
                    grad_log_alpha, grad_h0, B, T, D, io_dtype, gate_dtype, workspace, workspace_bytes, stream);
}

kda_status_t kda_glr_bwd_act8(const void *log_alpha, const int8_t *h_codes, const float *h_scales, const float *h0,
                              const int32_t *cu_seqlens, int32_t num_seqs, const void *grad_h, const float *grad_hT,
                              void *grad_x, void *grad_log_alpha, float *grad_h0, int32_t B, int32_t T, int32_t D,
                              int32_t io_dtype, int32_t gate_dtype, void *workspace, size_t workspace_bytes,
                              void *stream) {
    return glr_impl(true, grad_h, log_alpha, h_codes, h_scales, true, h0, cu_seqlens, num_seqs, grad_hT, grad_x,
                    grad_log_alpha, grad_h0, B, T, D, io_dtype, gate_dtype, workspace, workspace_bytes, stream);
}

kda_status_t kda_glr_step(const void *x, const void *log_alpha, float *S, void *h, int32_t B, int32_t D,
                          int32_t io_dtype, int32_t gate_dtype, void *stream) {
    if (!valid_dtype(io_dtype) || !valid_dtype(gate_dtype)) return KDA_ERR_UNSUPPORTED;
    if (B <= 0 || D <= 0) return KDA_ERR_INVALID_ARGUMENT;
    if (!req(x, dsize(io_dtype)) || !req(log_alpha, dsize(gate_dtype)) || !req(S, 4) || !req(h, dsize(io_dtype)))
        return KDA_ERR_INVALID_ARGUMENT;
    kda::GlrStepArgs a = {};
    a.x = x; a.log_alpha = log_alpha; a.S = S; a.h = h;
    a.n = (int64_t)B * D;
    a.io_bf16 = io_dtype == KDA_BF16; a.gate_bf16 = gate_dtype == KDA_BF16;
    if (!kda::glr_step_grids_fit(a)) return KDA_ERR_UNSUPPORTED;
    size_t len;
    char *err = fresh_error(&len);
    return finish(kda::launch_glr_step(a, stream, err, len));
}

kda_status_t kda_act8_pack(const void *x, int8_t *codes, float *scales, int64_t rows, int32_t cols, int32_t io_dtype,
                           void *stream) {
    return act8_impl(true, x, nullptr, codes, scales, rows, cols, io_dtype, stream);
}

kda_status_t kda_act8_unpack(const int8_t *codes, const float *scales, void *x, int64_t rows, int32_t cols,
                             int32_t io_dtype, void *stream) {
    return act8_impl(false, nullptr, x, codes, scales, rows, cols, io_dtype, stream);
}

size_t kda_chunk_bwd_act8_workspace_size(int32_t B, int32_t T, int32_t H, int32_t d_k, int32_t d_v,
                                         int32_t num_seqs, int32_t io_dtype) {
    ChunkAct8Layout L = {};
    if (!valid_dtype(io_dtype)) return 0;
    return chunk_act8_layout(B, T, H, d_k, d_v, num_seqs, io_dtype, L) ? L.total : 0;
}

kda_status_t kda_chunk_bwd_act8(const int8_t *q_codes, const float *q_scales, const int8_t *k_codes,
                                const float *k_scales, const int8_t *v_codes, const float *v_scales,
                                const void *log_alpha, const void *beta, const float *h0, const int32_t *cu_seqlens,
                                int32_t num_seqs, const void *grad_o, const float *grad_hT, void *grad_q,
                                void *grad_k, void *grad_v, void *grad_log_alpha, void *grad_beta, float *grad_h0,
                                int32_t B, int32_t T, int32_t H, int32_t d_k, int32_t d_v, int32_t io_dtype,
                                int32_t gate_dtype, void *workspace, size_t workspace_bytes, void *stream) {
    return chunk_bwd_act8_impl(q_codes, q_scales, k_codes, k_scales, v_codes, v_scales, log_alpha, beta, h0,
                               cu_seqlens, num_seqs, grad_o, grad_hT, grad_q, grad_k, grad_v, grad_log_alpha,
                               grad_beta, grad_h0, B, T, H, d_k, d_v, io_dtype, gate_dtype, workspace,
                               workspace_bytes, stream, false);
}

kda_status_t kda_gdn_chunk_bwd_act8(const int8_t *q_codes, const float *q_scales, const int8_t *k_codes,
                                    const float *k_scales, const int8_t *v_codes, const float *v_scales,
                                    const void *log_alpha, const void *beta, const float *h0,
                                    const int32_t *cu_seqlens, int32_t num_seqs, const void *grad_o,
                                    const float *grad_hT, void *grad_q, void *grad_k, void *grad_v,
                                    void *grad_log_alpha, void *grad_beta, float *grad_h0, int32_t B, int32_t T,
                                    int32_t H, int32_t d_k, int32_t d_v, int32_t io_dtype, int32_t gate_dtype,
                                    void *workspace, size_t workspace_bytes, void *stream) {
    return chunk_bwd_act8_impl(q_codes, q_scales, k_codes, k_scales, v_codes, v_scales, log_alpha, beta, h0,
                               cu_seqlens, num_seqs, grad_o, grad_hT, grad_q, grad_k, grad_v, grad_log_alpha,
                               grad_beta, grad_h0, B, T, H, d_k, d_v, io_dtype, gate_dtype, workspace,
                               workspace_bytes, stream, true);
}

kda_status_t kda_rmsnorm_fwd(const void *x, const void *residual, const void *weight, void *y, void *r, float *rstd,
                             int64_t rows, int32_t cols, float eps, int32_t io_dtype, int32_t w_dtype, void *stream) {
    return norm_fwd_impl(x, residual, weight, y, nullptr, nullptr, false, r, rstd, rows, cols, eps, io_dtype, w_dtype,
                         stream);
}

kda_status_t kda_rmsnorm_fwd_act8(const void *x, const void *residual, const void *weight, int8_t *codes,
                                  float *scales, void *r, float *rstd, int64_t rows, int32_t cols, float eps,
                                  int32_t io_dtype, int32_t w_dtype, void *stream) {
    return norm_fwd_impl(x, residual, weight, nullptr, codes, scales, true, r, rstd, rows, cols, eps, io_dtype,
                         w_dtype, stream);
}

size_t kda_rmsnorm_bwd_workspace_size(int64_t rows, int32_t cols) {
    if (rows < 0 || cols <= 0 || cols > kMaxRow || !product_fits(rows, cols)) return 0;
    return kda::norm_bwd_workspace_bytes(rows, cols);
}

kda_status_t kda_rmsnorm_bwd(const void *r, const void *weight, const float *rstd, const void *grad_y,
                             const void *grad_r, void *grad_x, void *grad_weight, int64_t rows, int32_t cols,
                             int32_t io_dtype, int32_t w_dtype, void *workspace, size_t workspace_bytes,
                             void *stream) {
    return norm_bwd_impl(r, nullptr, nullptr, false, weight, rstd, grad_y, grad_r, grad_x, grad_weight, rows, cols,
                         io_dtype, w_dtype, workspace, workspace_bytes, stream);
}

kda_status_t kda_rmsnorm_bwd_act8(const int8_t *r_codes, const float *r_scales, const void *weight, const float *rstd,
                                  const void *grad_y, const void *grad_r, void *grad_x, void *grad_weight,
                                  int64_t rows, int32_t cols, int32_t io_dtype, int32_t w_dtype, void *workspace,
                                  size_t workspace_bytes, void *stream) {
    return norm_bwd_impl(nullptr, r_codes, r_scales, true, weight, rstd, grad_y, grad_r, grad_x, grad_weight, rows,
                         cols, io_dtype, w_dtype, workspace, workspace_bytes, stream);
}

}  // extern "C"
