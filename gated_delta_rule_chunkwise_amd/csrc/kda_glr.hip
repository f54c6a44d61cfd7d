// Gated linear recurrence: kda_glr_fwd, kda_glr_bwd, kda_glr_bwd_act8, kda_glr_step.
#include <stdio.h>

#include "kda_act8.h"
#include "kda_launch.h"
#include "kda_ops_launch.h"

namespace kda {
namespace {

constexpr int kThreads = 256;

// One thread per (sequence, channel), the tokens in order.
template <typename IO, typename GT>
__global__ __launch_bounds__(kThreads) void glr_fwd_kernel(const IO *__restrict__ x, const GT *__restrict__ la,
                                                           const float *h0, const int32_t *__restrict__ cu,
                                                           int64_t N, int64_t T, int32_t D, IO *__restrict__ h,
                                                           float *h_T) {
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= N * D) return;
    const int64_t n = i / D, c = i % D;
    const int64_t b = cu ? cu[n] : n * T, e = cu ? cu[n + 1] : (n + 1) * T;
    float s = h0 ? h0[i] : 0.f;
    for (int64_t t = b; t < e; ++t) {
        const float a = __expf(to_f32(la[t * D + c]));
        s = (a == 0.f ? 0.f : a * s) + to_f32(x[t * D + c]);
        h[t * D + c] = from_f32<IO>(s);
    }
    if (h_T) h_T[i] = s;
}

template <typename IO, typename GT, bool ACT8>
__global__ __launch_bounds__(kThreads) void glr_bwd_kernel(const IO *__restrict__ gh, const GT *__restrict__ la,
                                                           const void *__restrict__ h, const float *__restrict__ hs,
                                                           const float *__restrict__ h0, const float *g_hT,
                                                           const int32_t *__restrict__ cu, int64_t N, int64_t T,
                                                           int32_t D, IO *__restrict__ dx, GT *__restrict__ dla,
                                                           float *dh0) {
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= N * D) return;
    const int64_t n = i / D, c = i % D, nb = (D + kAct8Block - 1) / kAct8Block;
    const int64_t b = cu ? cu[n] : n * T, e = cu ? cu[n + 1] : (n + 1) * T;
    float s = g_hT ? g_hT[i] : 0.f;
    for (int64_t t = e - 1; t >= b; --t) {
        const float a = __expf(to_f32(la[t * D + c]));
        const float g = to_f32(gh[t * D + c]) + s;
        s = a == 0.f ? 0.f : a * g;
        float prev;
        if (t == b) prev = h0 ? h0[i] : 0.f;
        else if constexpr (ACT8)
            prev = act8_value(((const int8_t *)h)[(t - 1) * D + c], hs[(t - 1) * nb + c / kAct8Block]);
        else prev = to_f32(((const IO *)h)[(t - 1) * D + c]);
        dx[t * D + c] = from_f32<IO>(g);
        dla[t * D + c] = from_f32<GT>(a == 0.f ? 0.f : prev * s);
    }
    if (dh0) dh0[i] = s;
}

template <typename IO, typename GT>
__global__ __launch_bounds__(kThreads) void glr_step_kernel(const IO *__restrict__ x, const GT *__restrict__ la,
                                                            float *__restrict__ S, IO *__restrict__ h, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= n) return;
    const float a = __expf(to_f32(la[i]));
    const float s = (a == 0.f ? 0.f : a * S[i]) + to_f32(x[i]);
    S[i] = s;
    h[i] = from_f32<IO>(s);
}

int64_t blocks(int64_t n) { return (n + kThreads - 1) / kThreads; }

template <typename IO, typename GT> hipError_t launch_t(const GlrArgs &a, hipStream_t st) {
    const dim3 grid((unsigned)blocks(a.num_seqs * a.D));
    if (!a.backward)
        hipLaunchKernelGGL((glr_fwd_kernel<IO, GT>), grid, dim3(kThreads), 0, st, (const IO *)a.x,
                           (const GT *)a.log_alpha, a.h0, a.cu_seqlens, a.num_seqs, a.seq_len, a.D, (IO *)a.out,
                           a.state_out);
    else if (a.h_scales)
        hipLaunchKernelGGL((glr_bwd_kernel<IO, GT, true>), grid, dim3(kThreads), 0, st, (const IO *)a.x,
                           (const GT *)a.log_alpha, a.h_in, a.h_scales, a.h0, a.d_hT, a.cu_seqlens, a.num_seqs,
                           a.seq_len, a.D, (IO *)a.out, (GT *)a.dlog_alpha, a.state_out);
    else
        hipLaunchKernelGGL((glr_bwd_kernel<IO, GT, false>), grid, dim3(kThreads), 0, st, (const IO *)a.x,
                           (const GT *)a.log_alpha, a.h_in, a.h_scales, a.h0, a.d_hT, a.cu_seqlens, a.num_seqs,
                           a.seq_len, a.D, (IO *)a.out, (GT *)a.dlog_alpha, a.state_out);
    return hipGetLastError();
}

template <typename IO, typename GT> hipError_t step_t(const GlrStepArgs &a, hipStream_t st) {
    hipLaunchKernelGGL((glr_step_kernel<IO, GT>), dim3((unsigned)blocks(a.n)), dim3(kThreads), 0, st,
                       (const IO *)a.x, (const GT *)a.log_alpha, a.S, (IO *)a.h, a.n);
    return hipGetLastError();
}

int status(hipError_t e, char *err, size_t err_len) {
    if (e == hipSuccess) return 0;
    snprintf(err, err_len, "%s", hipGetErrorString(e));
    return -1;
}

}  // namespace

size_t glr_workspace_bytes(const GlrArgs &) { return 0; }
bool glr_grids_fit(const GlrArgs &a) { return grid_fits(blocks(a.num_seqs * a.D), kThreads); }
bool glr_step_grids_fit(const GlrStepArgs &a) { return grid_fits(blocks(a.n), kThreads); }

int launch_glr(const GlrArgs &a, void *stream, char *err, size_t err_len) {
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    hipError_t e;
    if (a.io_bf16) e = a.gate_bf16 ? launch_t<bf16_t, bf16_t>(a, st) : launch_t<bf16_t, float>(a, st);
    else e = a.gate_bf16 ? launch_t<float, bf16_t>(a, st) : launch_t<float, float>(a, st);
    return status(e, err, err_len);
}

int launch_glr_step(const GlrStepArgs &a, void *stream, char *err, size_t err_len) {
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    hipError_t e;
    if (a.io_bf16) e = a.gate_bf16 ? step_t<bf16_t, bf16_t>(a, st) : step_t<bf16_t, float>(a, st);
    else e = a.gate_bf16 ? step_t<float, bf16_t>(a, st) : step_t<float, float>(a, st);
    return status(e, err, err_len);
}

}  // namespace kda
