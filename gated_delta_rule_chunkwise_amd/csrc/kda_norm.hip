// RMS norm with the residual's addition: kda_rmsnorm_fwd, kda_rmsnorm_bwd and
// their 8-bit forms.
//
// Bound by HBM: each input is read once, each output written once.  A row is held
// in the registers of LANES lanes as NP pieces of eight values each (piece p of the
// row in lane p % LANES), so that the second use of the row, after its mean is
// known, reads nothing: 8 lanes for rows of up to 64 values, 16 up to 128 (a row of
// 16 lanes: sums by data-parallel moves), a wave up to 1024, a workgroup up to
// 16384.  Which it is goes by the row's length alone, so a row's result does not
// depend on how many rows there are.  Longer rows are read twice.  A workgroup
// takes one group of rows and ends: 65536 x 4096 bf16 with residual and 8-bit output
// in 427 us (6.3 TB/s), against 520 with persistent workgroups that walk the rows.
//
// The weight's gradient sums over rows: each workgroup adds up its rows in
// registers and writes one partial row; a second launch adds the partial rows, in a
// fixed order.
#include <stdio.h>

#include <algorithm>

#include "kda_act8.h"
#include "kda_launch.h"
#include "kda_ops_launch.h"

namespace kda {
namespace {

constexpr int kThreads = 256;
// Workgroups of a backward, and partial rows: 65536 x 2048 bf16 194 us, against 203
// with 1024 (more to join) and 317 with 256 (one a CU).
constexpr int kMaxPartials = 512;
constexpr int kLongest = 16384;        // longest row that is held in registers

// The sum of x over a row's lanes, in each of them (LANES = kThreads: the
// workgroup; sh has a slot of its own for each of two rows in turn).
template <int LANES> __device__ __forceinline__ float row_sum(float x, float (*sh)[4], int turn) {
    if constexpr (LANES <= 16) {
        x += dpp_mov<0xB1>(x);
        x += dpp_mov<0x4E>(x);
        x += dpp_mov<0x141>(x);
        if constexpr (LANES == 16) x += dpp_mov<0x140>(x);
        return x;
    } else if constexpr (LANES == 64) {
        return wave_sum(x);
    } else {
        x = wave_sum(x);
        if ((threadIdx.x & 63) == 0) sh[turn][threadIdx.x >> 6] = x;
        __syncthreads();
        return (sh[turn][0] + sh[turn][1]) + (sh[turn][2] + sh[turn][3]);
    }
}

// n of eight values; the others are 0.
template <typename X> __device__ __forceinline__ void load_piece(Eight<X> &v, const X *p, int n) {
    if (n == 8) {
        v.load(p);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v.set(e, e < n ? to_f32(p[e]) : 0.f);
    }
}
template <typename X> __device__ __forceinline__ void store_piece(const Eight<X> &v, X *p, int n) {
    if (n == 8) {
        v.store(p);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) p[e] = from_f32<X>(v.get(e));
    }
}
template <typename WT> __device__ __forceinline__ void load_weight(Eight<WT> &v, const WT *w, int c, int n) {
    if (!w) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v.set(e, 1.f);
    } else if (n == 8) {
        v.load_kept(w + c);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v.set(e, e < n ? to_f32(w[c + e]) : 0.f);
    }
}

template <typename IO, typename WT, int LANES, int NP, bool ACT8>
__global__ __launch_bounds__(kThreads) void norm_fwd_kernel(const IO *x, const IO *res, const WT *__restrict__ w,
                                                            IO *__restrict__ y, IO *r, int8_t *__restrict__ codes,
                                                            float *__restrict__ scales, float *__restrict__ rstd,
                                                            int64_t rows, int32_t cols, float eps) {
    constexpr int PER = kThreads / LANES, kBlockLanes = LANES < 16 ? LANES : 16;
    __shared__ float sh[2][4];
    const int lane = threadIdx.x % LANES, nb = (cols + kAct8Block - 1) / kAct8Block;
    Eight<WT> wv[NP];
    int n[NP];
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        const int c = (lane + k * LANES) * 8;
        n[k] = max(0, min(8, cols - c));
        load_weight(wv[k], w, c, n[k]);
    }
    const int64_t row = (int64_t)blockIdx.x * PER + threadIdx.x / LANES;
    if (row < rows) {
        const int64_t at = row * cols + lane * 8;
        Eight<IO> v[NP];
#pragma unroll
        for (int k = 0; k < NP; ++k) load_piece(v[k], x + at + k * LANES * 8, n[k]);
        if (res) {
            Eight<IO> u[NP];
#pragma unroll
            for (int k = 0; k < NP; ++k) load_piece(u[k], res + at + k * LANES * 8, n[k]);
#pragma unroll
            for (int k = 0; k < NP; ++k) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[k].set(e, v[k].get(e) + u[k].get(e));   // rounded to the stream's type
                store_piece(v[k], r + at + k * LANES * 8, n[k]);
            }
        }
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < NP; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(v[k].get(e), v[k].get(e), ss);
        const float rs = 1.f / sqrtf(row_sum<LANES>(ss, sh, 0) / (float)cols + eps);
        if (rstd && lane == 0) rstd[row] = rs;
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = v[k].get(e) * rs * wv[k].get(e);
            const int64_t to = at + k * LANES * 8;
            if constexpr (!ACT8) {
                Eight<IO> o;
#pragma unroll
                for (int e = 0; e < 8; ++e) o.set(e, f[e]);
                store_piece(o, y + to, n[k]);
            } else {
                // sixteen neighbouring lanes hold one block of 128
                uint32_t m = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) m = max(m, e < n[k] ? abs_bits(f[e]) : 0u);
                const float s = act8_scale(lanes_max<kBlockLanes>(m));
                const Codes8 c = act8_codes(f, s);
                if (n[k] == 8) {
                    c.store(codes + to);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (e < n[k]) codes[to + e] = c.get(e);
                }
                if (lane % 16 == 0 && n[k] > 0) scales[row * nb + (lane + k * LANES) / 16] = s;
            }
        }
    }
}

// What the forward kept of a row: r, or its codes and scales.
template <typename IO, bool ACT8> struct Saved;
template <typename IO> struct Saved<IO, false> {
    Eight<IO> v;
    __device__ __forceinline__ void load(const void *p, const float *, int64_t at, int64_t, int n) {
        load_piece(v, static_cast<const IO *>(p) + at, n);
    }
    __device__ __forceinline__ float get(int e) const { return v.get(e); }
};
template <typename IO> struct Saved<IO, true> {
    Codes8 c;
    float s;
    __device__ __forceinline__ void load(const void *p, const float *scales, int64_t at, int64_t block, int n) {
        const int8_t *q = static_cast<const int8_t *>(p) + at;
        s = n > 0 ? scales[block] : 0.f;
        if (n == 8) {
            c.load(q);
        } else {
            c.w[0] = c.w[1] = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) c.w[e / 4] |= (uint32_t)(uint8_t)q[e] << (8 * (e % 4));
        }
    }
    __device__ __forceinline__ float get(int e) const { return act8_value(c.get(e), s); }
};

template <typename IO, typename WT, int LANES, int NP, bool ACT8>
__global__ __launch_bounds__(kThreads) void norm_bwd_kernel(const void *__restrict__ saved,
                                                            const float *__restrict__ scales,
                                                            const WT *__restrict__ w, const float *__restrict__ rstd,
                                                            const IO *gy, const IO *gr, IO *gx,
                                                            float *__restrict__ partial, int64_t rows, int32_t cols) {
    constexpr int PER = kThreads / LANES;
    __shared__ float sh[2][4];
    const int lane = threadIdx.x % LANES, nb = (cols + kAct8Block - 1) / kAct8Block;
    Eight<WT> wv[NP];
    int n[NP];
    float dw[NP][8];
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        const int c = (lane + k * LANES) * 8;
        n[k] = max(0, min(8, cols - c));
        load_weight(wv[k], w, c, n[k]);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[k][e] = 0.f;
    }
    int turn = 0;
    for (int64_t row = (int64_t)blockIdx.x * PER + threadIdx.x / LANES; row < rows;
         row += (int64_t)gridDim.x * PER, turn ^= 1) {
        const int64_t at = row * cols + lane * 8;
        Saved<IO, ACT8> v[NP];
        Eight<IO> g[NP], q[NP];
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            v[k].load(saved, scales, at + k * LANES * 8, row * nb + (lane + k * LANES) / 16, n[k]);
            load_piece(g[k], gy + at + k * LANES * 8, n[k]);
            if (gr) load_piece(q[k], gr + at + k * LANES * 8, n[k]);
        }
        const float rs = rstd[row];
        float m = 0.f;
#pragma unroll
        for (int k = 0; k < NP; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float t = v[k].get(e) * g[k].get(e);   // also the weight's gradient, but for rstd
                m = fmaf(t, wv[k].get(e), m);
                dw[k][e] = fmaf(t, rs, dw[k][e]);
            }
        const float f = row_sum<LANES>(m, sh, turn) / (float)cols * rs * rs;
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            Eight<IO> o;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float d = rs * (wv[k].get(e) * g[k].get(e) - v[k].get(e) * f);
                if (gr) d += q[k].get(e);
                o.set(e, d);
            }
            store_piece(o, gx + at + k * LANES * 8, n[k]);
        }
    }
    if (!partial) return;
    // one partial row a workgroup: the rows that it held side by side are joined here
    if constexpr (PER > 1) {
        __shared__ float all[PER][LANES * NP * 8 + 4];
#pragma unroll
        for (int k = 0; k < NP; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) all[threadIdx.x / LANES][(lane + k * LANES) * 8 + e] = dw[k][e];
        __syncthreads();
        for (int c = threadIdx.x; c < cols; c += kThreads) {
            float s = 0.f;
#pragma unroll
            for (int u = 0; u < PER; ++u) s += all[u][c];
            partial[(int64_t)blockIdx.x * cols + c] = s;
        }
    } else {
#pragma unroll
        for (int k = 0; k < NP; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n[k]) partial[(int64_t)blockIdx.x * cols + (lane + k * LANES) * 8 + e] = dw[k][e];
    }
}

// The sum of the partial rows: 32 columns a workgroup, 8 threads deep in columns
// and 32 in rows, each with sixteen rows' loads in flight (it is the latency of these
// that it takes: 512 partial rows of 128 columns in 11 us one at a time).
__global__ __launch_bounds__(kThreads) void norm_join_kernel(const float *__restrict__ partial, int32_t partials,
                                                             int32_t cols, void *gw, int32_t w_bf16) {
    __shared__ float sh[32][33];
    const int cg = threadIdx.x % 8, rg = threadIdx.x / 8, c0 = blockIdx.x * 32 + cg * 4;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    for (int row = rg; row < partials; row += 32 * 16) {
        float v[16][4];
#pragma unroll
        for (int k = 0; k < 16; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool there = row + 32 * k < partials && c0 + e < cols;
                v[k][e] = there ? partial[(int64_t)(row + 32 * k) * cols + c0 + e] : 0.f;
            }
#pragma unroll
        for (int k = 0; k < 16; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] += v[k][e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) sh[rg][cg * 4 + e] = s[e];
    __syncthreads();
    if (threadIdx.x < 32) {
        const int c = blockIdx.x * 32 + threadIdx.x;
        float t = 0.f;
#pragma unroll
        for (int u = 0; u < 32; ++u) t += sh[u][threadIdx.x];
        if (c < cols) {
            if (w_bf16) static_cast<bf16_t *>(gw)[c] = from_f32<bf16_t>(t);
            else static_cast<float *>(gw)[c] = t;
        }
    }
}

// ---- rows that do not fit the registers: read twice ------------------------------
template <typename WT> __device__ __forceinline__ float weight_at(const WT *w, int c) { return w ? to_f32(w[c]) : 1.f; }

template <typename IO, typename WT, bool ACT8>
__global__ __launch_bounds__(kThreads) void norm_fwd_long_kernel(const IO *x, const IO *res, const WT *__restrict__ w,
                                                                 IO *__restrict__ y, IO *r,
                                                                 int8_t *__restrict__ codes,
                                                                 float *__restrict__ scales,
                                                                 float *__restrict__ rstd, int32_t cols, float eps) {
    __shared__ float sh[2][4];
    const int64_t row = blockIdx.x, at = row * cols;
    float ss = 0.f;
    for (int c = threadIdx.x * 8; c < cols; c += kThreads * 8) {
        const int n = min(8, cols - c);
        Eight<IO> v, u;
        load_piece(v, x + at + c, n);
        if (res) {
            load_piece(u, res + at + c, n);
#pragma unroll
            for (int e = 0; e < 8; ++e) v.set(e, v.get(e) + u.get(e));
            store_piece(v, r + at + c, n);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(v.get(e), v.get(e), ss);
    }
    const float rs = 1.f / sqrtf(row_sum<kThreads>(ss, sh, 0) / (float)cols + eps);
    if (rstd && threadIdx.x == 0) rstd[row] = rs;
    const IO *src = res ? r : x;    // a thread reads back its own pieces
    const int lane = threadIdx.x, nb = (cols + kAct8Block - 1) / kAct8Block;
    for (int c = lane * 8, k = 0; k * kThreads * 8 < cols; c += kThreads * 8, ++k) {
        const int n = max(0, min(8, cols - c));
        Eight<IO> v;
        load_piece(v, src + at + c, n);
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = e < n ? v.get(e) * rs * weight_at(w, c + e) : 0.f;
        if constexpr (!ACT8) {
            Eight<IO> o;
#pragma unroll
            for (int e = 0; e < 8; ++e) o.set(e, f[e]);
            store_piece(o, y + at + c, n);
        } else {
            uint32_t m = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) m = max(m, abs_bits(f[e]));
            const float s = act8_scale(lanes_max<16>(m));
            const Codes8 q = act8_codes(f, s);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) codes[at + c + e] = q.get(e);
            if (lane % 16 == 0 && n > 0) scales[row * nb + c / kAct8Block] = s;
        }
    }
}

template <typename IO, typename WT, bool ACT8>
__global__ __launch_bounds__(kThreads) void norm_bwd_long_kernel(const void *__restrict__ saved,
                                                                 const float *__restrict__ scales,
                                                                 const WT *__restrict__ w,
                                                                 const float *__restrict__ rstd, const IO *gy,
                                                                 const IO *gr, IO *gx, int32_t cols) {
    __shared__ float sh[2][4];
    const int64_t row = blockIdx.x, at = row * cols;
    const int nb = (cols + kAct8Block - 1) / kAct8Block;
    float m = 0.f;
    for (int c = threadIdx.x * 8; c < cols; c += kThreads * 8) {
        const int n = min(8, cols - c);
        Saved<IO, ACT8> v;
        Eight<IO> g;
        v.load(saved, scales, at + c, row * nb + c / kAct8Block, n);
        load_piece(g, gy + at + c, n);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) m = fmaf(v.get(e) * g.get(e), weight_at(w, c + e), m);
    }
    const float rs = rstd[row], f = row_sum<kThreads>(m, sh, 0) / (float)cols * rs * rs;
    for (int c = threadIdx.x * 8; c < cols; c += kThreads * 8) {
        const int n = min(8, cols - c);
        Saved<IO, ACT8> v;
        Eight<IO> g, q, o;
        v.load(saved, scales, at + c, row * nb + c / kAct8Block, n);
        load_piece(g, gy + at + c, n);
        if (gr) load_piece(q, gr + at + c, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float d = e < n ? rs * (weight_at(w, c + e) * g.get(e) - v.get(e) * f) : 0.f;
            if (gr) d += q.get(e);
            o.set(e, d);
        }
        store_piece(o, gx + at + c, n);
    }
}

// Partial rows of the weight's gradient for long rows: a workgroup takes 2048
// columns of every gridDim.y-th row.
template <typename IO, bool ACT8>
__global__ __launch_bounds__(kThreads) void norm_partial_kernel(const void *__restrict__ saved,
                                                                const float *__restrict__ scales,
                                                                const float *__restrict__ rstd,
                                                                const IO *__restrict__ gy,
                                                                float *__restrict__ partial, int64_t rows,
                                                                int32_t cols) {
    const int c = (blockIdx.x * kThreads + threadIdx.x) * 8, n = min(8, cols - c);
    const int nb = (cols + kAct8Block - 1) / kAct8Block;
    if (n <= 0) return;
    float dw[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
        Saved<IO, ACT8> v;
        Eight<IO> g;
        v.load(saved, scales, row * cols + c, row * nb + c / kAct8Block, n);
        load_piece(g, gy + row * cols + c, n);
        const float rs = rstd[row];
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[e] = fmaf(v.get(e) * g.get(e), rs, dw[e]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < n) partial[(int64_t)blockIdx.y * cols + c + e] = dw[e];
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int row_lanes(int32_t cols) { return cols <= 64 ? 8 : cols <= 128 ? 16 : cols <= 1024 ? 64 : kThreads; }
// Partial rows, and in the register form workgroups, of a backward: rows enough for
// each to pay for its partial row.
int64_t partial_rows(int64_t rows, int32_t cols) {
    if (cols > kLongest) return std::min<int64_t>(std::max<int64_t>(ceil_div(rows, 64), 1), 64);
    return std::min<int64_t>(ceil_div(rows, kThreads / row_lanes(cols)), kMaxPartials);
}

int status(hipError_t e, char *err, size_t err_len) {
    if (e == hipSuccess) return 0;
    snprintf(err, err_len, "%s", hipGetErrorString(e));
    return -1;
}

template <typename IO, typename WT, int LANES, int NP, bool ACT8> void fwd_n(const NormArgs &a, hipStream_t st) {
    const int64_t groups = ceil_div(a.rows, kThreads / LANES);
    hipLaunchKernelGGL((norm_fwd_kernel<IO, WT, LANES, NP, ACT8>), dim3((unsigned)groups), dim3(kThreads), 0, st,
                       (const IO *)a.x, (const IO *)a.residual, (const WT *)a.weight, (IO *)a.y, (IO *)a.r, a.codes,
                       a.scales, a.rstd, a.rows, a.cols, a.eps);
}
template <typename IO, typename WT, int LANES, int NP, bool ACT8> void bwd_n(const NormArgs &a, hipStream_t st) {
    hipLaunchKernelGGL((norm_bwd_kernel<IO, WT, LANES, NP, ACT8>), dim3((unsigned)partial_rows(a.rows, a.cols)),
                       dim3(kThreads), 0, st, ACT8 ? (const void *)a.codes : a.x, a.scales, (const WT *)a.weight,
                       a.rstd, (const IO *)a.grad_y, (const IO *)a.grad_r, (IO *)a.grad_x,
                       a.grad_w ? (float *)a.workspace : nullptr, a.rows, a.cols);
}

// The register form for a.cols: f.template operator()<LANES, NP>().
template <typename F> void with_layout(int32_t cols, F f) {
    using std::integral_constant;
#define KDA_LAYOUT(L, N) f(integral_constant<int, L>(), integral_constant<int, N>())
    if (cols <= 64) KDA_LAYOUT(8, 1);
    else if (cols <= 128) KDA_LAYOUT(16, 1);
    else if (cols <= 512) KDA_LAYOUT(64, 1);
    else if (cols <= 1024) KDA_LAYOUT(64, 2);
    else if (cols <= 2048) KDA_LAYOUT(256, 1);
    else if (cols <= 4096) KDA_LAYOUT(256, 2);
    else if (cols <= 8192) KDA_LAYOUT(256, 4);
    else KDA_LAYOUT(256, 8);
#undef KDA_LAYOUT
}

template <typename IO, typename WT, bool ACT8> hipError_t fwd_t(const NormArgs &a, hipStream_t st) {
    if (a.cols > kLongest)
        hipLaunchKernelGGL((norm_fwd_long_kernel<IO, WT, ACT8>), dim3((unsigned)a.rows), dim3(kThreads), 0, st,
                           (const IO *)a.x, (const IO *)a.residual, (const WT *)a.weight, (IO *)a.y, (IO *)a.r,
                           a.codes, a.scales, a.rstd, a.cols, a.eps);
    else
        with_layout(a.cols, [&](auto lanes, auto np) {
            fwd_n<IO, WT, decltype(lanes)::value, decltype(np)::value, ACT8>(a, st);
        });
    return hipGetLastError();
}

template <typename IO, typename WT, bool ACT8> hipError_t bwd_t(const NormArgs &a, hipStream_t st) {
    const int32_t partials = a.rows > 0 ? (int32_t)partial_rows(a.rows, a.cols) : 0;
    float *partial = static_cast<float *>(a.workspace);
    if (a.rows > 0 && a.cols > kLongest) {
        const void *saved = ACT8 ? (const void *)a.codes : a.x;
        if (a.grad_w)   // first: grad_x may be written over grad_y
            hipLaunchKernelGGL((norm_partial_kernel<IO, ACT8>),
                               dim3((unsigned)ceil_div(a.cols, kThreads * 8), (unsigned)partials), dim3(kThreads), 0,
                               st, saved, a.scales, a.rstd, (const IO *)a.grad_y, partial, a.rows, a.cols);
        hipLaunchKernelGGL((norm_bwd_long_kernel<IO, WT, ACT8>), dim3((unsigned)a.rows), dim3(kThreads), 0, st, saved,
                           a.scales, (const WT *)a.weight, a.rstd, (const IO *)a.grad_y, (const IO *)a.grad_r,
                           (IO *)a.grad_x, a.cols);
    } else if (a.rows > 0) {
        with_layout(a.cols, [&](auto lanes, auto np) {
            bwd_n<IO, WT, decltype(lanes)::value, decltype(np)::value, ACT8>(a, st);
        });
    }
    if (a.grad_w)
        hipLaunchKernelGGL(norm_join_kernel, dim3((unsigned)ceil_div(a.cols, 32)), dim3(kThreads), 0, st, partial,
                           partials, a.cols, a.grad_w, a.w_bf16);
    return hipGetLastError();
}

template <bool ACT8> hipError_t fwd_a(const NormArgs &a, hipStream_t st) {
    if (a.io_bf16) return a.w_bf16 ? fwd_t<bf16_t, bf16_t, ACT8>(a, st) : fwd_t<bf16_t, float, ACT8>(a, st);
    return a.w_bf16 ? fwd_t<float, bf16_t, ACT8>(a, st) : fwd_t<float, float, ACT8>(a, st);
}
template <bool ACT8> hipError_t bwd_a(const NormArgs &a, hipStream_t st) {
    if (a.io_bf16) return a.w_bf16 ? bwd_t<bf16_t, bf16_t, ACT8>(a, st) : bwd_t<bf16_t, float, ACT8>(a, st);
    return a.w_bf16 ? bwd_t<float, bf16_t, ACT8>(a, st) : bwd_t<float, float, ACT8>(a, st);
}

}  // namespace

bool norm_grids_fit(const NormArgs &a) {
    const int64_t per = a.cols > kLongest ? 1 : kThreads / row_lanes(a.cols);
    return grid_fits(ceil_div(a.rows, per), kThreads) && grid_fits(ceil_div(a.cols, 32), kThreads);
}
size_t norm_bwd_workspace_bytes(int64_t rows, int32_t cols) {
    return rows > 0 ? (size_t)partial_rows(rows, cols) * cols * sizeof(float) : 0;
}

int launch_norm_fwd(const NormArgs &a, void *stream, char *err, size_t err_len) {
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    return status(a.codes ? fwd_a<true>(a, st) : fwd_a<false>(a, st), err, err_len);
}

int launch_norm_bwd(const NormArgs &a, void *stream, char *err, size_t err_len) {
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    return status(a.codes ? bwd_a<true>(a, st) : bwd_a<false>(a, st), err, err_len);
}

}  // namespace kda
