// RMS norm with the residual's addition: kda_rmsnorm_fwd, kda_rmsnorm_bwd and
// their 8-bit forms.
#include <stdio.h>

#include "kda_act8.h"
#include "kda_launch.h"
#include "kda_ops_launch.h"

namespace kda {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float block_sum(float x, float *sh) {
    x = wave_sum(x);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = x;
    __syncthreads();
    return (sh[0] + sh[1]) + (sh[2] + sh[3]);
}

template <typename WT> __device__ __forceinline__ float weight_at(const WT *w, int c) { return w ? to_f32(w[c]) : 1.f; }

// One workgroup per row, its columns in turn; the sum is read back from r.
template <typename IO, typename WT, bool ACT8>
__global__ __launch_bounds__(kThreads) void norm_fwd_kernel(const IO *x, const IO *res, const WT *__restrict__ w,
                                                            IO *__restrict__ y, IO *r, int8_t *__restrict__ codes,
                                                            float *__restrict__ scales, float *__restrict__ rstd,
                                                            int32_t cols, float eps) {
    __shared__ float sh[4];
    const int64_t row = blockIdx.x, at = row * cols;
    float ss = 0.f;
    for (int c = threadIdx.x; c < cols; c += kThreads) {
        float v = to_f32(x[at + c]);
        if (res) {
            const IO rv = from_f32<IO>(v + to_f32(res[at + c]));
            r[at + c] = rv;
            v = to_f32(rv);
        }
        ss += v * v;
    }
    const float rs = 1.f / sqrtf(block_sum(ss, sh) / (float)cols + eps);
    if (rstd && threadIdx.x == 0) rstd[row] = rs;
    const IO *src = res ? r : x;    // a thread reads back its own columns
    if constexpr (!ACT8) {
        for (int c = threadIdx.x; c < cols; c += kThreads)
            y[at + c] = from_f32<IO>(to_f32(src[at + c]) * rs * weight_at(w, c));
    } else {
        __syncthreads();
        const int lane = threadIdx.x & 63, nb = (cols + kAct8Block - 1) / kAct8Block;
        for (int b = threadIdx.x >> 6; b < nb; b += kThreads / 64) {
            const int c0 = b * kAct8Block + lane, c1 = c0 + 64;
            const float v0 = c0 < cols ? to_f32(src[at + c0]) * rs * weight_at(w, c0) : 0.f;
            const float v1 = c1 < cols ? to_f32(src[at + c1]) * rs * weight_at(w, c1) : 0.f;
            uint32_t m = max(abs_bits(v0), abs_bits(v1));
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o));
            const float s = act8_scale(m), inv = 1.f / s;
            const bool bad = m >= kInfBits;
            if (c0 < cols) codes[at + c0] = bad ? 0 : (int8_t)act8_code(v0, s, inv);
            if (c1 < cols) codes[at + c1] = bad ? 0 : (int8_t)act8_code(v1, s, inv);
            if (lane == 0) scales[row * nb + b] = s;
        }
    }
}

template <typename IO, bool ACT8>
__device__ __forceinline__ float saved_at(const IO *r, const int8_t *codes, const float *scales, int64_t row, int c,
                                          int cols, int nb) {
    if constexpr (ACT8) return act8_value(codes[row * cols + c], scales[row * nb + c / kAct8Block]);
    else return to_f32(r[row * cols + c]);
}

template <typename IO, typename WT, bool ACT8>
__global__ __launch_bounds__(kThreads) void norm_bwd_kernel(const IO *__restrict__ r, const int8_t *__restrict__ codes,
                                                            const float *__restrict__ scales,
                                                            const WT *__restrict__ w, const float *__restrict__ rstd,
                                                            const IO *gy, const IO *gr, IO *gx, int32_t cols) {
    __shared__ float sh[4];
    const int64_t row = blockIdx.x, at = row * cols;
    const int nb = (cols + kAct8Block - 1) / kAct8Block;
    float m = 0.f;
    for (int c = threadIdx.x; c < cols; c += kThreads)
        m += saved_at<IO, ACT8>(r, codes, scales, row, c, cols, nb) * weight_at(w, c) * to_f32(gy[at + c]);
    const float rs = rstd[row], k = block_sum(m, sh) / (float)cols * rs * rs;
    for (int c = threadIdx.x; c < cols; c += kThreads) {
        float d = rs * (weight_at(w, c) * to_f32(gy[at + c]) -
                        saved_at<IO, ACT8>(r, codes, scales, row, c, cols, nb) * k);
        if (gr) d += to_f32(gr[at + c]);
        gx[at + c] = from_f32<IO>(d);
    }
}

template <typename IO, typename WT, bool ACT8>
__global__ __launch_bounds__(kThreads) void norm_gw_kernel(const IO *__restrict__ r, const int8_t *__restrict__ codes,
                                                           const float *__restrict__ scales,
                                                           const float *__restrict__ rstd, const IO *__restrict__ gy,
                                                           WT *__restrict__ gw, int64_t rows, int32_t cols) {
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= cols) return;
    const int nb = (cols + kAct8Block - 1) / kAct8Block;
    float s = 0.f;
    for (int64_t row = 0; row < rows; ++row)
        s += to_f32(gy[row * cols + c]) * saved_at<IO, ACT8>(r, codes, scales, row, c, cols, nb) * rstd[row];
    gw[c] = from_f32<WT>(s);
}

int status(hipError_t e, char *err, size_t err_len) {
    if (e == hipSuccess) return 0;
    snprintf(err, err_len, "%s", hipGetErrorString(e));
    return -1;
}

template <typename IO, typename WT, bool ACT8> hipError_t fwd_t(const NormArgs &a, hipStream_t st) {
    hipLaunchKernelGGL((norm_fwd_kernel<IO, WT, ACT8>), dim3((unsigned)a.rows), dim3(kThreads), 0, st,
                       (const IO *)a.x, (const IO *)a.residual, (const WT *)a.weight, (IO *)a.y, (IO *)a.r, a.codes,
                       a.scales, a.rstd, a.cols, a.eps);
    return hipGetLastError();
}
template <typename IO, typename WT, bool ACT8> hipError_t bwd_t(const NormArgs &a, hipStream_t st) {
    // the weight's gradient first: grad_x may be written over grad_y
    if (a.grad_w)
        hipLaunchKernelGGL((norm_gw_kernel<IO, WT, ACT8>), dim3((unsigned)((a.cols + kThreads - 1) / kThreads)),
                           dim3(kThreads), 0, st, (const IO *)a.x, a.codes, a.scales, a.rstd, (const IO *)a.grad_y,
                           (WT *)a.grad_w, a.rows, a.cols);
    if (a.rows > 0)
        hipLaunchKernelGGL((norm_bwd_kernel<IO, WT, ACT8>), dim3((unsigned)a.rows), dim3(kThreads), 0, st,
                           (const IO *)a.x, a.codes, a.scales, (const WT *)a.weight, a.rstd, (const IO *)a.grad_y,
                           (const IO *)a.grad_r, (IO *)a.grad_x, a.cols);
    return hipGetLastError();
}

}  // namespace

bool norm_grids_fit(const NormArgs &a) { return grid_fits(a.rows, kThreads); }
size_t norm_bwd_workspace_bytes(int64_t, int32_t) { return 0; }

int launch_norm_fwd(const NormArgs &a, void *stream, char *err, size_t err_len) {
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    hipError_t e;
    if (a.codes)
        e = a.io_bf16 ? (a.w_bf16 ? fwd_t<bf16_t, bf16_t, true>(a, st) : fwd_t<bf16_t, float, true>(a, st))
                      : (a.w_bf16 ? fwd_t<float, bf16_t, true>(a, st) : fwd_t<float, float, true>(a, st));
    else
        e = a.io_bf16 ? (a.w_bf16 ? fwd_t<bf16_t, bf16_t, false>(a, st) : fwd_t<bf16_t, float, false>(a, st))
                      : (a.w_bf16 ? fwd_t<float, bf16_t, false>(a, st) : fwd_t<float, float, false>(a, st));
    return status(e, err, err_len);
}

int launch_norm_bwd(const NormArgs &a, void *stream, char *err, size_t err_len) {
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    hipError_t e;
    if (a.codes)
        e = a.io_bf16 ? (a.w_bf16 ? bwd_t<bf16_t, bf16_t, true>(a, st) : bwd_t<bf16_t, float, true>(a, st))
                      : (a.w_bf16 ? bwd_t<float, bf16_t, true>(a, st) : bwd_t<float, float, true>(a, st));
    else
        e = a.io_bf16 ? (a.w_bf16 ? bwd_t<bf16_t, bf16_t, false>(a, st) : bwd_t<bf16_t, float, false>(a, st))
                      : (a.w_bf16 ? bwd_t<float, bf16_t, false>(a, st) : bwd_t<float, float, false>(a, st));
    return status(e, err, err_len);
}

}  // namespace kda
