// Internal interface between the host-side C ABI of the gated linear recurrence,
// the 8-bit activation checkpoints and the RMS norm (kda_ops_api.cpp) and their
// HIP launchers (kda_glr.hip, kda_act8.hip, kda_norm.hip).  Not part of the
// public ABI.
#pragma once
#include <stddef.h>
#include <stdint.h>

namespace kda {

constexpr int32_t kAct8Block = 128;   // values that share a scale
inline int64_t act8_blocks(int64_t cols) { return (cols + kAct8Block - 1) / kAct8Block; }

struct GlrArgs {
    const void *x;              // forward: x; backward: grad_h
    const void *log_alpha;
    const void *h_in;           // backward: h, or its codes (h_scales given)
    const float *h_scales;      // [tokens, ceil(D / 128)], or nullptr
    const float *h0;            // [N, D], or nullptr (zeros)
    const float *d_hT;          // backward: gradient of h_T, or nullptr (zeros)
    const int32_t *cu_seqlens;  // device, or nullptr (equal-length batch)
    void *out;                  // forward: h; backward: grad_x
    void *dlog_alpha;           // backward
    float *state_out;           // forward: h_T; backward: grad_h0; or nullptr
    int64_t num_seqs, seq_len, tokens;   // N, T, B * T
    int32_t D;
    int32_t io_bf16, gate_bf16;
    int32_t backward;
    void *workspace;
    size_t workspace_bytes;
};

size_t glr_workspace_bytes(const GlrArgs &a);   // pointers are not read
bool glr_grids_fit(const GlrArgs &a);
int launch_glr(const GlrArgs &a, void *stream, char *err, size_t err_len);

struct GlrStepArgs {
    const void *x, *log_alpha;
    float *S;
    void *h;
    int64_t n;                  // B * D
    int32_t io_bf16, gate_bf16;
};
bool glr_step_grids_fit(const GlrStepArgs &a);
int launch_glr_step(const GlrStepArgs &a, void *stream, char *err, size_t err_len);

struct Act8Args {
    const void *x;              // pack: values (io dtype); unpack: unused
    void *out;                  // unpack: values (io dtype)
    int8_t *codes;
    float *scales;
    int64_t rows;
    int32_t cols;
    int32_t io_bf16;
};
bool act8_grids_fit(const Act8Args &a);
int launch_act8_pack(const Act8Args &a, void *stream, char *err, size_t err_len);
int launch_act8_unpack(const Act8Args &a, void *stream, char *err, size_t err_len);

struct NormArgs {
    const void *x;              // forward: x; backward: r, or nullptr with codes
    const void *residual;       // forward, or nullptr
    const void *weight;         // or nullptr (ones)
    void *y;                    // forward: y, or nullptr with codes
    void *r;                    // forward: x + residual
    int8_t *codes;              // forward: y's codes (out); backward: r's codes (in)
    float *scales;
    float *rstd;                // forward: out or nullptr; backward: in
    const void *grad_y, *grad_r;
    void *grad_x, *grad_w;      // grad_w or nullptr
    int64_t rows;
    int32_t cols;
    float eps;
    int32_t io_bf16, w_bf16;
    void *workspace;
    size_t workspace_bytes;
};
bool norm_grids_fit(const NormArgs &a);
size_t norm_bwd_workspace_bytes(int64_t rows, int32_t cols);
int launch_norm_fwd(const NormArgs &a, void *stream, char *err, size_t err_len);
int launch_norm_bwd(const NormArgs &a, void *stream, char *err, size_t err_len);

// The calling thread's text of the last HIP error (kda_last_hip_error).
char *hip_error_text(size_t *len);

}  // namespace kda
