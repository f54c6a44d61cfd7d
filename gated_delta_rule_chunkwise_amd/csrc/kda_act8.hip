// 8-bit activation checkpoints: kda_act8_pack and kda_act8_unpack.
//
// Both are one pass over the data, bound by HBM: bf16 3 + 4/128 bytes a value.  A
// lane takes eight consecutive values (16 bytes of bf16, and 8 of codes, a load), 16
// lanes a block of 128, or 8 lanes one of 64 (activations of 64 channels a head,
// which would leave half of the lanes idle otherwise).  The block's largest
// magnitude goes round its lanes by data-parallel moves, without LDS.  A lane has
// the loads of kBlocks blocks in flight.  65536 x 4096 bf16 there and back: 274 us
// (5.95 TB/s) with two blocks a lane, 284 with one, 280 with four, 358 with eight.
#include <stdio.h>

#include "kda_act8.h"
#include "kda_launch.h"
#include "kda_ops_launch.h"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kBlocks = 2;

// Where a lane's piece of block b is: the row's blocks are WIDTH long but for the
// last.  WHOLE: rows are whole blocks, so blocks are simply consecutive.
template <int WIDTH, bool WHOLE> struct Piece {
    int64_t at;   // of the lane's eight values
    int n;        // of them inside the row
    __device__ __forceinline__ Piece(int64_t b, int lane, int32_t cols, int32_t nb) {
        if constexpr (WHOLE) {
            at = b * WIDTH + lane * 8;
            n = 8;
        } else {
            const int64_t row = (uint64_t)b >> 32 ? b / nb : (int64_t)((uint32_t)b / (uint32_t)nb);
            const int c = (int)(b - row * nb) * WIDTH + lane * 8;
            at = row * cols + c;
            n = max(0, min(8, cols - c));
        }
    }
};

template <typename IO, int WIDTH, bool WHOLE>
__global__ __launch_bounds__(kThreads) void pack_kernel(const IO *__restrict__ x, int8_t *__restrict__ codes,
                                                        float *__restrict__ scales, int64_t blocks, int32_t cols,
                                                        int32_t nb) {
    constexpr int LANES = WIDTH / 8, PER = kThreads / LANES;
    const int lane = threadIdx.x % LANES;
    const int64_t first = (int64_t)blockIdx.x * PER * kBlocks + threadIdx.x / LANES;
    Eight<IO> v[kBlocks];
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) {
        const int64_t b = first + k * PER;
        if (b >= blocks) continue;
        const Piece<WIDTH, WHOLE> p(b, lane, cols, nb);
        if (p.n == 8) {
            v[k].load(x + p.at);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[k].set(e, e < p.n ? to_f32(x[p.at + e]) : 0.f);
        }
    }
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) {
        const int64_t b = first + k * PER;
        if (b >= blocks) continue;   // all lanes of a block alike
        float f[8];
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            f[e] = v[k].get(e);
            m = max(m, abs_bits(f[e]));
        }
        const float s = act8_scale(lanes_max<LANES>(m));
        const Codes8 c = act8_codes(f, s);
        const Piece<WIDTH, WHOLE> p(b, lane, cols, nb);
        if (p.n == 8) {
            c.store(codes + p.at);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < p.n) codes[p.at + e] = c.get(e);
        }
        if (lane == 0) scales[b] = s;
    }
}

template <typename IO, int WIDTH, bool WHOLE>
__global__ __launch_bounds__(kThreads) void unpack_kernel(const int8_t *__restrict__ codes,
                                                          const float *__restrict__ scales, IO *__restrict__ x,
                                                          int64_t blocks, int32_t cols, int32_t nb) {
    constexpr int LANES = WIDTH / 8, PER = kThreads / LANES;
    const int lane = threadIdx.x % LANES;
    const int64_t first = (int64_t)blockIdx.x * PER * kBlocks + threadIdx.x / LANES;
    Codes8 c[kBlocks];
    float s[kBlocks];
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) {
        const int64_t b = first + k * PER;
        if (b >= blocks) continue;
        const Piece<WIDTH, WHOLE> p(b, lane, cols, nb);
        s[k] = scales[b];
        if (p.n == 8) {
            c[k].load(codes + p.at);
        } else {
            c[k].w[0] = c[k].w[1] = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < p.n) c[k].w[e / 4] |= (uint32_t)(uint8_t)codes[p.at + e] << (8 * (e % 4));
        }
    }
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) {
        const int64_t b = first + k * PER;
        if (b >= blocks) continue;
        const Piece<WIDTH, WHOLE> p(b, lane, cols, nb);
        Eight<IO> v;
#pragma unroll
        for (int e = 0; e < 8; ++e) v.set(e, act8_value(c[k].get(e), s[k]));
        if (p.n == 8) {
            v.store(x + p.at);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < p.n) x[p.at + e] = from_f32<IO>(v.get(e));
        }
    }
}

// Rows of up to 64 values are blocks of their own of that width.
bool narrow(const Act8Args &a) { return a.cols <= 64; }
int64_t grid_of(const Act8Args &a) {
    const int64_t per = kThreads / (narrow(a) ? 8 : 16) * kBlocks;
    return (a.rows * act8_blocks(a.cols) + per - 1) / per;
}

int status(hipError_t e, char *err, size_t err_len) {
    if (e == hipSuccess) return 0;
    snprintf(err, err_len, "%s", hipGetErrorString(e));
    return -1;
}

template <typename IO, int WIDTH, bool WHOLE> void launch_w(const Act8Args &a, bool pack, hipStream_t st) {
    const dim3 grid((unsigned)grid_of(a));
    const int32_t nb = (int32_t)act8_blocks(a.cols);
    if (pack)
        hipLaunchKernelGGL((pack_kernel<IO, WIDTH, WHOLE>), grid, dim3(kThreads), 0, st, (const IO *)a.x, a.codes,
                           a.scales, a.rows * nb, a.cols, nb);
    else
        hipLaunchKernelGGL((unpack_kernel<IO, WIDTH, WHOLE>), grid, dim3(kThreads), 0, st, a.codes, a.scales,
                           (IO *)a.out, a.rows * nb, a.cols, nb);
}
template <typename IO> hipError_t launch_t(const Act8Args &a, bool pack, hipStream_t st) {
    if (narrow(a)) a.cols == 64 ? launch_w<IO, 64, true>(a, pack, st) : launch_w<IO, 64, false>(a, pack, st);
    else a.cols % 128 == 0 ? launch_w<IO, 128, true>(a, pack, st) : launch_w<IO, 128, false>(a, pack, st);
    return hipGetLastError();
}

}  // namespace

bool act8_grids_fit(const Act8Args &a) { return grid_fits(grid_of(a), kThreads); }

int launch_act8_pack(const Act8Args &a, void *stream, char *err, size_t err_len) {
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    return status(a.io_bf16 ? launch_t<bf16_t>(a, true, st) : launch_t<float>(a, true, st), err, err_len);
}
int launch_act8_unpack(const Act8Args &a, void *stream, char *err, size_t err_len) {
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    return status(a.io_bf16 ? launch_t<bf16_t>(a, false, st) : launch_t<float>(a, false, st), err, err_len);
}

}  // namespace kda
