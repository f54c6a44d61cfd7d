// 8-bit activation checkpoints: kda_act8_pack and kda_act8_unpack.
#include <stdio.h>

#include "kda_act8.h"
#include "kda_launch.h"
#include "kda_ops_launch.h"

namespace kda {
namespace {

constexpr int kThreads = 256;

// One wave per block of 128 values, two per lane.
template <typename IO>
__global__ __launch_bounds__(kThreads) void pack_kernel(const IO *__restrict__ x, int8_t *__restrict__ codes,
                                                        float *__restrict__ scales, int64_t rows, int32_t cols,
                                                        int32_t nb) {
    const int lane = threadIdx.x & 63;
    const int64_t b = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
    if (b >= rows * nb) return;
    const int64_t row = b / nb;
    const int c0 = (int)(b % nb) * kAct8Block + lane, c1 = c0 + 64;
    const IO *xr = x + row * cols;
    const float v0 = c0 < cols ? to_f32(xr[c0]) : 0.f, v1 = c1 < cols ? to_f32(xr[c1]) : 0.f;
    uint32_t m = max(abs_bits(v0), abs_bits(v1));
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o));
    const float s = act8_scale(m), inv = 1.f / s;
    const bool bad = m >= kInfBits;
    if (c0 < cols) codes[row * cols + c0] = bad ? 0 : (int8_t)act8_code(v0, s, inv);
    if (c1 < cols) codes[row * cols + c1] = bad ? 0 : (int8_t)act8_code(v1, s, inv);
    if (lane == 0) scales[b] = s;
}

template <typename IO>
__global__ __launch_bounds__(kThreads) void unpack_kernel(const int8_t *__restrict__ codes,
                                                          const float *__restrict__ scales, IO *__restrict__ x,
                                                          int64_t rows, int32_t cols, int32_t nb) {
    const int lane = threadIdx.x & 63;
    const int64_t b = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
    if (b >= rows * nb) return;
    const int64_t row = b / nb;
    const int c0 = (int)(b % nb) * kAct8Block + lane, c1 = c0 + 64;
    const float s = scales[b];
    if (c0 < cols) x[row * cols + c0] = from_f32<IO>(act8_value(codes[row * cols + c0], s));
    if (c1 < cols) x[row * cols + c1] = from_f32<IO>(act8_value(codes[row * cols + c1], s));
}

int64_t block_grid(const Act8Args &a) {
    return (a.rows * act8_blocks(a.cols) + kThreads / 64 - 1) / (kThreads / 64);
}

int status(hipError_t e, char *err, size_t err_len) {
    if (e == hipSuccess) return 0;
    snprintf(err, err_len, "%s", hipGetErrorString(e));
    return -1;
}

template <typename IO> hipError_t pack_t(const Act8Args &a, hipStream_t st) {
    hipLaunchKernelGGL((pack_kernel<IO>), dim3((unsigned)block_grid(a)), dim3(kThreads), 0, st, (const IO *)a.x,
                       a.codes, a.scales, a.rows, a.cols, (int32_t)act8_blocks(a.cols));
    return hipGetLastError();
}
template <typename IO> hipError_t unpack_t(const Act8Args &a, hipStream_t st) {
    hipLaunchKernelGGL((unpack_kernel<IO>), dim3((unsigned)block_grid(a)), dim3(kThreads), 0, st, a.codes, a.scales,
                       (IO *)a.out, a.rows, a.cols, (int32_t)act8_blocks(a.cols));
    return hipGetLastError();
}

}  // namespace

bool act8_grids_fit(const Act8Args &a) { return grid_fits(block_grid(a), kThreads); }

int launch_act8_pack(const Act8Args &a, void *stream, char *err, size_t err_len) {
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    return status(a.io_bf16 ? pack_t<bf16_t>(a, st) : pack_t<float>(a, st), err, err_len);
}
int launch_act8_unpack(const Act8Args &a, void *stream, char *err, size_t err_len) {
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    return status(a.io_bf16 ? unpack_t<bf16_t>(a, st) : unpack_t<float>(a, st), err, err_len);
}

}  // namespace kda
