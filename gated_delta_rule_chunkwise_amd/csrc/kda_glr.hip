// Gated linear recurrence: kda_glr_fwd, kda_glr_bwd, kda_glr_bwd_act8, kda_glr_step.
//
// One token is an affine map of a channel's state: forward s -> alpha s + x,
// backward (from the last token to the first) c -> alpha (grad_h + c).  Maps
// compose: (A2, B2) after (A1, B1) is (A2 A1, A2 B1 + B2).  All calls are bound by
// HBM, so every input is read once and kept in registers until the state in front
// of it is known:
//
//   - the tokens of the whole batch are one flat axis, cut into time tiles; a tile
//     of a channel block is one workgroup, a span of kR tokens of it one "row" of
//     lanes (a wave, or a part of one where D is small).  A sequence's first token
//     is a map with A = 0 (B takes h0), so sequences need no tiles of their own and
//     a batch of short ones fills its tiles like a long one;
//   - each row composes its span; the rows' maps meet in LDS, the tile's map goes to
//     the workspace;
//   - tiles come in groups of kG.  The last tile of a group publishes, in place of
//     its map, the state behind it (a map with A = 0), so a tile's incoming state is
//     the composition of at most kG published maps, in a fixed order whatever the
//     timing: the results are the same bits on every call;
//   - with that state the rows run their spans once more, from registers, and write.
//
// A published map is one 64-bit word with its own validity (all ones: not there
// yet), read and written by relaxed agent-scope atomics: no fence, no flag.  Tiles
// are handed out by a ticket in order of time, so a tile only ever waits for tiles
// that are already running: the wait ends.
#include <stdio.h>

#include <algorithm>
#include <type_traits>

#include "kda_act8.h"
#include "kda_launch.h"
#include "kda_ops_launch.h"

namespace kda {
namespace {

constexpr int kW = 8;              // waves of a workgroup
constexpr int kNT = 64 * kW;       // its threads
constexpr int kG = 16;             // tiles of a group
constexpr int kMinLanes = 8;       // channel lanes of a row at least
constexpr int kTicketPitch = 32;   // a cache line of its own for each
constexpr uint64_t kAbsent = ~(uint64_t)0;
// A wait that could only be broken by a fault elsewhere still ends (after seconds),
// with a NaN state.
constexpr int kMaxPolls = 1 << 24;

enum Mode : int { kFwd = 0, kBwd = 1, kBwd8 = 2 };

constexpr int R = 32;              // tokens of a row's span

// VEC consecutive values of X as loaded, and as fp32.
template <typename X, int VEC> struct Raw;
template <typename X> struct Raw<X, 1> { typedef X type; };
template <> struct Raw<float, 2> { typedef float type __attribute__((ext_vector_type(2))); };
template <> struct Raw<bf16_t, 2> { typedef bf16x2_t type; };
template <> struct Raw<int8_t, 2> { typedef int8_t type __attribute__((ext_vector_type(2))); };

template <int VEC, typename RAW> __device__ __forceinline__ float raw_at(const RAW &r, int e) {
    if constexpr (VEC == 1) return (float)r;
    else return (float)r[e];
}
template <typename X, int VEC> __device__ __forceinline__ typename Raw<X, VEC>::type load_raw(const X *p) {
    return __builtin_nontemporal_load(reinterpret_cast<const typename Raw<X, VEC>::type *>(p));
}
template <typename X, int VEC> __device__ __forceinline__ void store_vec(X *p, const float (&v)[VEC]) {
    typename Raw<X, VEC>::type r;
    if constexpr (VEC == 1) {
        r = from_f32<X>(v[0]);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) r[e] = from_f32<X>(v[e]);
    }
    __builtin_nontemporal_store(r, reinterpret_cast<typename Raw<X, VEC>::type *>(p));
}
template <int VEC> __device__ __forceinline__ void load_f32(const float *p, float (&v)[VEC]) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = p[e];
}

// a s, where a = 0 drops s whatever it is (a reset).
__device__ __forceinline__ float decayed(float a, float s) { return a == 0.f ? 0.f : a * s; }

struct GlrParams {
    const void *x, *la, *h;
    const float *hs, *h0, *g_hT;
    const int32_t *cu;
    void *out, *dla;
    float *state_out;
    int64_t N, T, tokens;
    int32_t D, chan_tiles, lane_log;   // lanes of a row: 1 << lane_log
    int64_t time_tiles;
    uint64_t *words;                   // [time_tiles, D] published maps
    uint32_t *tickets;                 // one for each channel tile, kTicketPitch apart
};

// The sequences of the flat token axis.
struct Seqs {
    const int32_t *cu;
    int64_t N, T;
    __device__ __forceinline__ int64_t begin(int64_t n) const { return cu ? cu[n] : n * T; }
    __device__ __forceinline__ int64_t end(int64_t n) const { return cu ? cu[n + 1] : (n + 1) * T; }
    // The (non-empty) sequence of token t.
    __device__ __forceinline__ int64_t find(int64_t t) const {
        if (!cu) return t / T;
        int64_t lo = 0, hi = N - 1;   // largest n with cu[n] <= t
        while (lo < hi) {
            const int64_t mid = (lo + hi + 1) >> 1;
            if (cu[mid] <= t) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    }
};

template <typename IO, typename GT, int MODE, int VEC> struct Row {
    typedef typename std::conditional<MODE == kBwd8, int8_t, IO>::type HT;
    typename Raw<IO, VEC>::type x[R];
    typename Raw<GT, VEC>::type la[R];
    typename Raw<HT, VEC>::type h[R];        // backward: h of the token before
    float start[VEC];                        // forward: h0 of the last sequence that starts here
    int start_at;
};

// ---- the span of one row, all of it inside one sequence ------------------------
template <typename IO, typename GT, int MODE, int VEC>
__device__ __forceinline__ void compose_inside(const Row<IO, GT, MODE, VEC> &row, float (&L)[VEC], float (&B)[VEC]) {
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int i = MODE == kFwd ? k : R - 1 - k;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float l = raw_at<VEC>(row.la[i], e), a = __expf(l), x = raw_at<VEC>(row.x[i], e);
            L[e] += l;
            B[e] = MODE == kFwd ? decayed(a, B[e]) + x : decayed(a, x + B[e]);
        }
    }
}

template <typename IO, typename GT, int MODE, int VEC>
__device__ __forceinline__ void finish_inside(const GlrParams &p, const Row<IO, GT, MODE, VEC> &row, const float *hs,
                                              int64_t t0, int c0, float (&s)[VEC]) {
    IO *out = static_cast<IO *>(p.out);
    GT *dla = static_cast<GT *>(p.dla);
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int i = MODE == kFwd ? k : R - 1 - k;
        const int64_t at = (t0 + i) * p.D + c0;
        float o[VEC], d[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float a = __expf(raw_at<VEC>(row.la[i], e)), x = raw_at<VEC>(row.x[i], e);
            if constexpr (MODE == kFwd) {
                s[e] = decayed(a, s[e]) + x;
                o[e] = s[e];
            } else {
                o[e] = x + s[e];
                s[e] = decayed(a, o[e]);
                float h = raw_at<VEC>(row.h[i], e);
                if constexpr (MODE == kBwd8) h *= hs[i];
                d[e] = a == 0.f ? 0.f : h * s[e];
            }
        }
        store_vec<IO, VEC>(out + at, o);
        if constexpr (MODE != kFwd) store_vec<GT, VEC>(dla + at, d);
    }
}

// ---- a span with sequence borders in it, or at the batch's end ------------------
// A sequence that starts in one row and ends in another has its h0 read here, in
// the first pass, and kept: its h_T, which may be the same memory, is written by
// another workgroup as soon as this one has published.
template <typename IO, typename GT, int MODE, int VEC>
__device__ __forceinline__ void compose_border(const GlrParams &p, const Seqs &q, Row<IO, GT, MODE, VEC> &row,
                                               int64_t t0, int nv, int c0, float (&L)[VEC], float (&B)[VEC]) {
    row.start_at = -1;
    if (nv <= 0) return;
    int64_t n = q.find(MODE == kFwd ? t0 : t0 + nv - 1), b = q.begin(n), e_ = q.end(n);
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int i = MODE == kFwd ? k : R - 1 - k;
        const int64_t t = t0 + i;
        if (i >= nv) continue;
        if (MODE == kFwd ? t == b : t + 1 == e_) {
            const float *src = MODE == kFwd ? p.h0 : p.g_hT;
#pragma unroll
            for (int e = 0; e < VEC; ++e) L[e] = -__builtin_inff(), B[e] = 0.f;
            if (src) load_f32<VEC>(src + n * p.D + c0, B);
            if constexpr (MODE == kFwd) {
                row.start_at = i;
#pragma unroll
                for (int e = 0; e < VEC; ++e) row.start[e] = B[e];
            }
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float l = raw_at<VEC>(row.la[i], e), a = __expf(l), x = raw_at<VEC>(row.x[i], e);
            L[e] += l;
            B[e] = MODE == kFwd ? decayed(a, B[e]) + x : decayed(a, x + B[e]);
        }
        if constexpr (MODE == kFwd) {
            if (t + 1 == e_ && i + 1 < nv) {
                do { ++n; e_ = q.end(n); } while (e_ <= t + 1);
                b = t + 1;
            }
        } else {
            if (t == b && i > 0) {
                do { --n; b = q.begin(n); } while (b >= t);
                e_ = t;
            }
        }
    }
}

template <typename IO, typename GT, int MODE, int VEC>
__device__ __forceinline__ void finish_border(const GlrParams &p, const Seqs &q, const Row<IO, GT, MODE, VEC> &row,
                                              const float *hs, int64_t t0, int nv, int c0, float (&s)[VEC]) {
    if (nv <= 0) return;
    IO *out = static_cast<IO *>(p.out);
    GT *dla = static_cast<GT *>(p.dla);
    int64_t n = q.find(MODE == kFwd ? t0 : t0 + nv - 1), b = q.begin(n), e_ = q.end(n);
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int i = MODE == kFwd ? k : R - 1 - k;
        const int64_t t = t0 + i;
        if (i >= nv) continue;
        if (MODE == kFwd ? t == b : t + 1 == e_) {
            const float *src = MODE == kFwd ? p.h0 : p.g_hT;
#pragma unroll
            for (int e = 0; e < VEC; ++e) s[e] = 0.f;
            if (MODE == kFwd && i == row.start_at) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) s[e] = row.start[e];
            } else if (src) {
                load_f32<VEC>(src + n * p.D + c0, s);
            }
        }
        const int64_t at = t * p.D + c0;
        float o[VEC], d[VEC], h[VEC];
        if constexpr (MODE != kFwd) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                h[e] = raw_at<VEC>(row.h[i], e);
                if constexpr (MODE == kBwd8) h[e] *= hs[i];
            }
            if (t == b) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) h[e] = 0.f;
                if (p.h0) load_f32<VEC>(p.h0 + n * p.D + c0, h);
            }
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float a = __expf(raw_at<VEC>(row.la[i], e)), x = raw_at<VEC>(row.x[i], e);
            if constexpr (MODE == kFwd) {
                s[e] = decayed(a, s[e]) + x;
                o[e] = s[e];
            } else {
                o[e] = x + s[e];
                s[e] = decayed(a, o[e]);
                d[e] = a == 0.f ? 0.f : h[e] * s[e];
            }
        }
        store_vec<IO, VEC>(out + at, o);
        if constexpr (MODE != kFwd) store_vec<GT, VEC>(dla + at, d);
        if (MODE == kFwd ? t + 1 == e_ : t == b) {
            if (p.state_out) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) p.state_out[n * p.D + c0 + e] = s[e];
            }
            if constexpr (MODE == kFwd) {
                if (i + 1 < nv) {
                    do { ++n; e_ = q.end(n); } while (e_ <= t + 1);
                    b = t + 1;
                }
            } else {
                if (i > 0) {
                    do { --n; b = q.begin(n); } while (b >= t);
                    e_ = t;
                }
            }
        }
    }
}

template <int MODE, int VEC> struct alignas(16) GlrShared {
    float A[kNT * VEC], B[kNT * VEC];               // the rows' maps
    float pA[kG][64 * VEC], pB[kG][64 * VEC];       // the published maps in front of the tile
    float hs[MODE == kBwd8 ? kNT / kMinLanes * R : 1];   // scales of the rows' saved h
    uint32_t tile;
};

template <typename IO, typename GT, int MODE, int VEC>
__global__ __launch_bounds__(kNT) void glr_kernel(const GlrParams p) {
    typedef typename Row<IO, GT, MODE, VEC>::HT HT;
    __shared__ GlrShared<MODE, VEC> sm;
    const int tid = threadIdx.x;
    const int ct = (int)(blockIdx.x % p.chan_tiles);
    int64_t tt = 0;                                    // in the order of the scan
    if (p.time_tiles > 1) {
        if (tid == 0)
            sm.tile = __hip_atomic_fetch_add(p.tickets + ct * kTicketPitch, 1u, __ATOMIC_RELAXED,
                                             __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        tt = sm.tile;
    }
    const int lanes = 1 << p.lane_log, rows = kNT >> p.lane_log;
    const int cl = tid & (lanes - 1), v = tid >> p.lane_log;   // lane of a row, row in the order of the scan
    const int c0 = (ct * lanes + cl) * VEC;
    const bool chan = c0 < p.D;
    const Seqs q = {p.cu, p.N, p.T};
    int64_t valid = p.tokens;                          // rows behind the last sequence are not touched
    if (p.cu) valid = min(valid, (int64_t)p.cu[p.N]);
    const int64_t span = MODE == kFwd ? tt * rows + v : (p.time_tiles - 1 - tt) * rows + (rows - 1 - v);
    const int64_t t0 = span * R;
    const int nv = chan ? (int)max((int64_t)0, min((int64_t)R, valid - t0)) : 0;

    Row<IO, GT, MODE, VEC> row;
    {
        const IO *x = static_cast<const IO *>(p.x) + t0 * p.D + c0;
        const GT *la = static_cast<const GT *>(p.la) + t0 * p.D + c0;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (i < nv) {
                row.la[i] = load_raw<GT, VEC>(la + (int64_t)i * p.D);
                row.x[i] = load_raw<IO, VEC>(x + (int64_t)i * p.D);
            }
        }
    }
    if (p.state_out) {   // empty sequences pass their state on
        for (int64_t n = tt; n < p.N; n += p.time_tiles) {
            if (v == 0 && chan && q.begin(n) == q.end(n)) {
                const float *src = MODE == kFwd ? p.h0 : p.g_hT;
#pragma unroll
                for (int e = 0; e < VEC; ++e) p.state_out[n * p.D + c0 + e] = src ? src[n * p.D + c0 + e] : 0.f;
            }
        }
    }
    bool inside = nv == R || !chan;
    if (nv == R) {
        const int64_t n = q.find(t0);
        inside = q.begin(n) < t0 && q.end(n) > t0 + R;
    }
    const bool plain = __all(inside) && __any(chan);

    float L[VEC], A[VEC], B[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) L[e] = 0.f, B[e] = 0.f;
    if (plain) {
        if (chan) compose_inside<IO, GT, MODE, VEC>(row, L, B);
    } else {
        compose_border<IO, GT, MODE, VEC>(p, q, row, t0, nv, c0, L, B);
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        A[e] = __expf(L[e]);
        sm.A[tid * VEC + e] = A[e];
        sm.B[tid * VEC + e] = B[e];
    }
    if constexpr (MODE != kFwd) {
        const HT *h = static_cast<const HT *>(p.h) + (t0 - 1) * p.D + c0;
        const int nb = (p.D + kAct8Block - 1) / kAct8Block;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (i < nv && t0 + i > 0) {
                row.h[i] = load_raw<HT, VEC>(h + (int64_t)i * p.D);
            }
        }
        if constexpr (MODE == kBwd8) {   // a tile's channels lie in one block of 128
            const int64_t tile0 = (p.time_tiles - 1 - tt) * rows * R;
            for (int i = tid; i < rows * R; i += kNT) {
                const int64_t t = tile0 + i;
                if (t > 0 && t < valid) sm.hs[i] = p.hs[(t - 1) * nb + ct * lanes * VEC / kAct8Block];
            }
        }
    }
    __syncthreads();

    float s[VEC];   // the state in front of this tile
#pragma unroll
    for (int e = 0; e < VEC; ++e) s[e] = 0.f;
    if (p.time_tiles > 1) {
        const int pos = (int)(tt % kG);
        const int64_t first = tt - pos > 0 ? tt - pos - 1 : 0;   // the state behind the last group, or the first map
        const int cnt = (int)(tt - first);
        if (v == rows - 1) {
            // the tile's map: the rows in front of this one, then this one
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                float a = 1.f, b = 0.f;
                for (int u = 0; u < rows; ++u) {
                    const int k = (u * lanes + cl) * VEC + e;
                    b = decayed(sm.A[k], b) + sm.B[k];
                    a *= sm.A[k];
                }
                A[e] = a;
                B[e] = b;
            }
        }
        const auto publish = [&](int e, float a, float b) {
            uint32_t ab = __builtin_bit_cast(uint32_t, a);
            if (ab == 0xffffffffu) ab = 0x7fc00000u;
            __hip_atomic_store(p.words + tt * p.D + c0 + e, (uint64_t)__builtin_bit_cast(uint32_t, b) << 32 | ab,
                               __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        };
        if (v == rows - 1 && chan && pos != kG - 1) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) publish(e, A[e], B[e]);
        }
        for (int j = v; j < cnt; j += rows) {
            const uint64_t *w = p.words + (first + j) * p.D + c0;
            uint64_t got[VEC];
            int polls = 0;
            bool there = !chan;
            while (!there && polls < kMaxPolls) {
                there = true;
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    got[e] = __hip_atomic_load(w + e, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
                for (int e = 0; e < VEC; ++e) there = there && (uint32_t)got[e] != 0xffffffffu;
                if (!there) __builtin_amdgcn_s_sleep(1);
                ++polls;
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float nan = __builtin_nanf("");
                sm.pA[j][cl * VEC + e] = there && chan ? __builtin_bit_cast(float, (uint32_t)got[e]) : nan;
                sm.pB[j][cl * VEC + e] = there && chan ? __builtin_bit_cast(float, (uint32_t)(got[e] >> 32)) : nan;
            }
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            for (int j = 0; j < cnt; ++j) s[e] = decayed(sm.pA[j][cl * VEC + e], s[e]) + sm.pB[j][cl * VEC + e];
        if (v == rows - 1 && chan && pos == kG - 1) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) publish(e, 0.f, decayed(A[e], s[e]) + B[e]);
        }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        for (int u = 0; u < v; ++u) {
            const int k = (u * lanes + cl) * VEC + e;
            s[e] = decayed(sm.A[k], s[e]) + sm.B[k];
        }
    }
    const float *hs = sm.hs + (MODE == kBwd8 ? (rows - 1 - v) * R : 0);
    if (plain) {
        if (chan) finish_inside<IO, GT, MODE, VEC>(p, row, hs, t0, c0, s);
    } else {
        finish_border<IO, GT, MODE, VEC>(p, q, row, hs, t0, nv, c0, s);
    }
}

// The workspace of a call: the tickets 0, every word absent.
__global__ __launch_bounds__(256) void glr_clear_kernel(uint32_t *tickets, int64_t nt, uint64_t *words, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    for (int64_t k = i; k < nt; k += (int64_t)gridDim.x * 256) tickets[k] = 0;
    for (int64_t k = i; k < n; k += (int64_t)gridDim.x * 256) words[k] = kAbsent;
}

constexpr int kThreads = 256;
template <typename IO, typename GT>
__global__ __launch_bounds__(kThreads) void glr_step_kernel(const IO *__restrict__ x, const GT *__restrict__ la,
                                                            float *__restrict__ S, IO *__restrict__ h, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= n) return;
    const float s = decayed(__expf(to_f32(la[i])), S[i]) + to_f32(x[i]);
    S[i] = s;
    h[i] = from_f32<IO>(s);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct GlrPlan {
    int vec, lane_log;
    int64_t chan_tiles, time_tiles;
};
// Two channels a lane in bf16 where the addresses allow it, one otherwise: a wave's
// load is 256 bytes of a token (128 in the odd bf16 case).  A row of lanes covers
// the channels up to a wave's width; with fewer channels a wave takes several rows.
GlrPlan glr_plan(const GlrArgs &a, int vec) {
    GlrPlan g = {};
    g.vec = vec;
    const int64_t need = ceil_div(a.D, vec);
    g.lane_log = 3;
    while (g.lane_log < 6 && (1 << g.lane_log) < need) ++g.lane_log;
    g.chan_tiles = ceil_div(need, (int64_t)1 << g.lane_log);
    const int64_t tile = (int64_t)(kNT >> g.lane_log) * R;
    g.time_tiles = a.tokens > tile ? ceil_div(a.tokens, tile) : 1;
    return g;
}
static_assert(kMinLanes == 8, "the plan's smallest row");

bool glr_aligned(const GlrArgs &a) {
    const auto ok = [](const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; };
    const uintptr_t gt = a.gate_bf16 ? 4 : 8;
    return a.D % 2 == 0 && ok(a.x, 4) && ok(a.out, 4) && ok(a.log_alpha, gt) && ok(a.dlog_alpha, gt) &&
           ok(a.h_in, a.h_scales ? 2 : 4);
}

template <typename IO, typename GT, int MODE> hipError_t launch_m(const GlrArgs &a, hipStream_t st) {
    const GlrPlan g = glr_plan(a, a.io_bf16 && glr_aligned(a) ? 2 : 1);
    GlrParams p = {a.x, a.log_alpha, a.h_in, a.h_scales, a.h0, a.d_hT, a.cu_seqlens, a.out, a.dlog_alpha, a.state_out,
                   a.num_seqs, a.seq_len, a.tokens, a.D, (int32_t)g.chan_tiles, g.lane_log, g.time_tiles, nullptr,
                   nullptr};
    if (g.time_tiles > 1) {
        const int64_t nt = g.chan_tiles * kTicketPitch, n = g.time_tiles * a.D;
        p.tickets = static_cast<uint32_t *>(a.workspace);
        p.words = reinterpret_cast<uint64_t *>(p.tickets + nt);
        hipLaunchKernelGGL(glr_clear_kernel, dim3((unsigned)std::min(ceil_div(n, 256), (int64_t)2048)), dim3(256), 0, st,
                           p.tickets, nt, p.words, n);
    }
    const dim3 grid((unsigned)(g.time_tiles * g.chan_tiles));
    if constexpr (sizeof(IO) == 2) {
        if (g.vec == 2) {
            hipLaunchKernelGGL((glr_kernel<IO, GT, MODE, 2>), grid, dim3(kNT), 0, st, p);
            return hipGetLastError();
        }
    }
    hipLaunchKernelGGL((glr_kernel<IO, GT, MODE, 1>), grid, dim3(kNT), 0, st, p);
    return hipGetLastError();
}

template <typename IO, typename GT> hipError_t launch_t(const GlrArgs &a, hipStream_t st) {
    if (!a.backward) return launch_m<IO, GT, kFwd>(a, st);
    return a.h_scales ? launch_m<IO, GT, kBwd8>(a, st) : launch_m<IO, GT, kBwd>(a, st);
}

template <typename IO, typename GT> hipError_t step_t(const GlrStepArgs &a, hipStream_t st) {
    hipLaunchKernelGGL((glr_step_kernel<IO, GT>), dim3((unsigned)ceil_div(a.n, kThreads)), dim3(kThreads), 0, st,
                       (const IO *)a.x, (const GT *)a.log_alpha, a.S, (IO *)a.h, a.n);
    return hipGetLastError();
}

int status(hipError_t e, char *err, size_t err_len) {
    if (e == hipSuccess) return 0;
    snprintf(err, err_len, "%s", hipGetErrorString(e));
    return -1;
}

}  // namespace

// For the widest time axis of either layout (the addresses are not known here).
size_t glr_workspace_bytes(const GlrArgs &a) {
    size_t need = 0;
    for (int vec : {1, 2}) {
        const GlrPlan g = glr_plan(a, vec);
        if (g.time_tiles > 1)
            need = std::max(need, (size_t)g.chan_tiles * kTicketPitch * sizeof(uint32_t) +
                                      (size_t)g.time_tiles * a.D * sizeof(uint64_t));
    }
    return need;
}
bool glr_grids_fit(const GlrArgs &a) {
    for (int vec : {1, 2}) {
        const GlrPlan g = glr_plan(a, vec);
        if (g.time_tiles > kMaxWorkItems / kNT / g.chan_tiles || !grid_fits(g.time_tiles * g.chan_tiles, kNT))
            return false;
    }
    return true;
}
bool glr_step_grids_fit(const GlrStepArgs &a) { return grid_fits(ceil_div(a.n, kThreads), kThreads); }

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
