// Gated linear recurrence: kda_glr_fwd, kda_glr_bwd, kda_glr_bwd_act8, kda_glr_step.
//
// One token is an affine map of a channel's state: forward s -> alpha s + x,
// backward (from the last token to the first) c -> alpha (grad_h + c).  Maps
// compose: (A2, B2) after (A1, B1) is (A2 A1, A2 B1 + B2).  All calls are bound by
// HBM, so every input is read once and kept in registers until the state in front
// of it is known:
//
//   - the tokens of the whole batch are one flat axis, cut into time tiles; a tile
//     of a channel block is one workgroup, a span of some tokens of it one "row" of
//     up to 64 lanes.  A sequence's first token is a map with A = 0 (B takes h0), so
//     sequences need no tiles of their own and a batch of short ones fills its tiles
//     like a long one;
//   - each row composes its span; the rows' maps meet in LDS, the tile's map goes to
//     the workspace;
//   - tiles come in groups.  The last tile of a group publishes, in place of its
//     map, the state behind it (a map with A = 0), so a tile's incoming state is the
//     composition of at most a group of published maps, in a fixed order whatever
//     the timing: the results are the same bits on every call;
//   - with that state the rows run their spans once more, from registers, and write.
//
// A published map is one 64-bit word with its own validity (all ones: not there
// yet), read and written by relaxed agent-scope atomics: no fence, no flag.  Tiles
// are handed out by a ticket in order of time, one for each channel tile, so a tile
// only ever waits for tiles that are already running: the wait ends.
//
// Measured (copies on this card: 6.2 TB/s): bf16 forward of 65536 x 4096 in 314 us
// (5.1 TB/s), backward of 65536 x 2048 in 250 us (5.4 TB/s), from 8-bit h over a
// packed batch of 139,000 tokens x 2048 in 557 us (4.6 TB/s), 2% of each for factors
// that tell a reset from one that is out of range; without the waits for
// other tiles the first is 8% shorter, the rest of the way is the pieces of 512 bytes
// of a token that a wave takes.  Smaller tiles (64 tokens) and one workgroup a CU
// (256 tokens) took 20% and 10% longer.  Rows of an odd number of channels share
// lines at both ends of each piece: 387 fp32 channels run at 3.4 TB/s, 384 at 4.2.
// With few channels the chain of states counts: 139,000 tokens x 256 in 99 us, 68
// groups in turn.
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
constexpr int kXcds = 8;           // chiplets, each with an L2 of its own
constexpr int kMaxGroup = 16;      // tiles of a group at most
constexpr int kMinSpan = 8;        // shortest span of the wide form
constexpr int kStaged = 1024;      // borders that are kept in LDS
constexpr int kMinLanes = 8;       // channel lanes of a row at least
constexpr int kMaxScales = 2048;   // tokens x blocks of a tile
constexpr int kTicketPitch = 32;   // a cache line of its own for each
constexpr uint64_t kAbsent = ~(uint64_t)0;
// A wait that could only be broken by a fault elsewhere still ends (after seconds),
// with a NaN state.
constexpr int kMaxPolls = 1 << 24;

enum Mode : int { kFwd = 0, kBwd = 1, kBwd8 = 2 };

// Tokens of a row's span.  What a lane keeps of a token (8 bytes of x, its gates,
// in the backward 8 more of h) times these is about 64 registers forward and 72
// backward: two workgroups share a CU.
template <typename IO, typename GT, int MODE, int VEC> constexpr int span_tokens() {
    if (VEC == 1) return 32;
    const int bytes = 8 + VEC * (int)sizeof(GT) + (MODE == 0 ? 0 : 8);
    return bytes <= 16 ? 16 : bytes <= 24 ? (MODE == 0 ? 10 : 12) : 8;
}

// VEC consecutive values of X as loaded, and as fp32.
template <typename X, int VEC> struct Raw;
template <typename X> struct Raw<X, 1> { typedef X type; };
template <> struct Raw<float, 2> { typedef float type __attribute__((ext_vector_type(2))); };
template <> struct Raw<bf16_t, 4> { typedef bf16x4_t type; };
// Codes stay the whole number that was loaded until they are used: bytes taken
// apart at once would wait for the load.
template <> struct Raw<int8_t, 4> { typedef uint32_t type; };
template <> struct Raw<int8_t, 2> { typedef uint16_t type; };
template <> struct Raw<bf16_t, 2> { typedef bf16x2_t type; };
template <> struct Raw<float, 4> { typedef f32x4_t type; };

template <int VEC, typename RAW> __device__ __forceinline__ float raw_at(const RAW &r, int e) {
    if constexpr (std::is_same<RAW, uint32_t>::value || std::is_same<RAW, uint16_t>::value)
        return (float)(int8_t)(r >> (8 * e));
    else if constexpr (VEC == 1) return (float)r;
    else return (float)r[e];
}
// Rows of an odd number of channels put a lane's values at any element's address:
// the hardware loads and stores them there.
template <typename X, int VEC, bool KEEP> __device__ __forceinline__ typename Raw<X, VEC>::type load_raw(const X *p) {
    typedef typename Raw<X, VEC>::type at __attribute__((aligned(sizeof(X))));
    if constexpr (KEEP) return *reinterpret_cast<const at *>(p);
    else return __builtin_nontemporal_load(reinterpret_cast<const at *>(p));
}
template <typename X, int VEC> __device__ __forceinline__ void store_vec(X *p, const float (&v)[VEC]) {
    typename Raw<X, VEC>::type r;
    if constexpr (VEC == 1) {
        r = from_f32<X>(v[0]);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) r[e] = from_f32<X>(v[e]);
    }
    typedef typename Raw<X, VEC>::type at __attribute__((aligned(sizeof(X))));
    __builtin_nontemporal_store(r, reinterpret_cast<at *>(p));
}
template <int VEC> __device__ __forceinline__ void load_f32(const float *p, float (&v)[VEC]) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = p[e];
}

// a s, where a = 0 drops s whatever it is (a reset).
__device__ __forceinline__ float decayed(float a, float s) { return a == 0.f ? 0.f : a * s; }
// The factor of a span or a tile is 0 only where one of its tokens is a reset;
// otherwise it ends at the smallest positive number, whose product with a state is as
// good as 0, but for an infinity or a NaN, which stay what they are.  Factors are not
// negative: their bits are in their order.
__device__ __forceinline__ uint32_t bits_of(float a) { return __builtin_bit_cast(uint32_t, a); }
__device__ __forceinline__ float not_below(float a, uint32_t least) {
    return __builtin_bit_cast(float, max(bits_of(a), least));
}

struct GlrParams {
    const void *x, *la, *h;
    const float *hs, *h0, *g_hT;
    const int32_t *cu;
    void *out, *dla;
    float *state_out;
    int64_t N, T, tokens;
    int32_t D, chan_tiles, lanes;      // lanes of a row
    int64_t time_tiles;
    uint64_t *words;                   // published maps: [time tile][channel tile][e][lane]
    int32_t over;                      // h_T is written over h0
    int32_t keep;                      // tokens share cache lines: inputs stay in the L2
    int32_t group;                     // tiles of a group
    uint32_t *tickets;                 // one for each channel tile, kTicketPitch apart
};

// The sequences of the flat token axis.
struct Seqs {
    const int32_t *cu, *lds;   // the borders, or nullptr; their copy in LDS, where they are staged
    bool staged;
    int64_t N, T;
    __device__ __forceinline__ int64_t border(int64_t n) const { return staged ? lds[n] : cu[n]; }
    __device__ __forceinline__ int64_t begin(int64_t n) const { return cu ? border(n) : n * T; }
    __device__ __forceinline__ int64_t end(int64_t n) const { return cu ? border(n + 1) : (n + 1) * T; }
    // The (non-empty) sequence of token t.
    __device__ __forceinline__ int64_t find(int64_t t) const {
        if (!cu) return t / T;
        int64_t lo = 0, hi = N - 1;   // largest n with cu[n] <= t
        while (lo < hi) {
            const int64_t mid = (lo + hi + 1) >> 1;
            if (border(mid) <= t) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    }
};

// From sequence n to that of token t, which is n's or (in the order of the scan) a
// later one: past the empty ones.
template <int MODE> __device__ __forceinline__ int64_t step_to(const Seqs &q, int64_t n, int64_t t) {
    if constexpr (MODE == kFwd) while (q.end(n) <= t) ++n;
    else while (q.begin(n) > t) --n;
    return n;
}

template <typename IO, typename GT, int MODE, int VEC> struct Row {
    static constexpr int R = span_tokens<IO, GT, MODE, VEC>();
    typedef typename std::conditional<MODE == kBwd8, int8_t, IO>::type HT;
    typename Raw<IO, VEC>::type x[R];
    typename Raw<GT, VEC>::type la[R];
    typename Raw<HT, VEC>::type h[R];        // backward: h of the token before
    float start[VEC];                        // forward: h0 of the last sequence that starts here
    int start_at;

    template <bool KEEP> __device__ __forceinline__ void load_inputs(const GlrParams &p, int64_t t0, int nv, int c0) {
        const IO *xp = static_cast<const IO *>(p.x) + t0 * p.D + c0;
        const GT *gp = static_cast<const GT *>(p.la) + t0 * p.D + c0;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (i < nv) {
                la[i] = load_raw<GT, VEC, KEEP>(gp + (int64_t)i * p.D);
                x[i] = load_raw<IO, VEC, KEEP>(xp + (int64_t)i * p.D);
            }
        }
    }
    template <bool KEEP> __device__ __forceinline__ void load_saved(const GlrParams &p, int64_t t0, int nv, int c0) {
        const HT *hp = static_cast<const HT *>(p.h) + (t0 - 1) * p.D + c0;
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (i < nv && t0 + i > 0) h[i] = load_raw<HT, VEC, KEEP>(hp + (int64_t)i * p.D);
    }
};

// ---- the span of one row, all of it inside one sequence ------------------------
template <typename IO, typename GT, int MODE, int VEC>
__device__ __forceinline__ void compose_inside(const Row<IO, GT, MODE, VEC> &row, float (&L)[VEC], float (&B)[VEC]) {
    constexpr int R = span_tokens<IO, GT, MODE, VEC>();
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
                                              int64_t t0, int c0, int skip, float (&s)[VEC]) {
    constexpr int R = span_tokens<IO, GT, MODE, VEC>();
    IO *out = static_cast<IO *>(p.out) + t0 * p.D + c0;
    GT *dla = static_cast<GT *>(p.dla) + t0 * p.D + c0;
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int i = MODE == kFwd ? k : R - 1 - k;
        const int64_t to = (int64_t)i * p.D;   // the same for all lanes
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
        if (skip) {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (e >= skip) out[to + e] = from_f32<IO>(o[e]);
        } else {
            store_vec<IO, VEC>(out + to, o);
        }
        if constexpr (MODE != kFwd) store_vec<GT, VEC>(dla + to, d);
    }
}

// ---- a span with sequence borders in it, or at the batch's end ------------------
// Which of a row's tokens are the first and the last of their sequences (a bit
// each), and the sequences of its first and last token.
struct Borders {
    uint32_t first, last;
    int32_t n_first, n_last;
    __device__ __forceinline__ Borders(const Seqs &q, int64_t t0, int nv) : first(0), last(0), n_first(0), n_last(0) {
        if (nv <= 0) return;
        int64_t n = q.find(t0), e = q.end(n);
        n_first = (int32_t)n;
        if (q.begin(n) == t0) first = 1;
        while (e < t0 + nv) {
            const int k = (int)(e - t0);
            last |= 1u << (k - 1);
            first |= 1u << k;
            do e = q.end(++n);
            while (e <= t0 + k);
        }
        if (e == t0 + nv) last |= 1u << (nv - 1);
        n_last = (int32_t)n;
    }
};

// A sequence that starts in one row and ends in another has its h0 read here, in
// the first pass, and kept: its h_T, which may be the same memory, is written by
// another workgroup as soon as this one has published.
template <typename IO, typename GT, int MODE, int VEC>
__device__ __forceinline__ void compose_border(const GlrParams &p, const Seqs &q, const Borders &at,
                                               Row<IO, GT, MODE, VEC> &row, int64_t t0, int nv, int c0,
                                               float (&L)[VEC], float (&B)[VEC]) {
    constexpr int R = span_tokens<IO, GT, MODE, VEC>();
    const uint32_t starts = MODE == kFwd ? at.first : at.last;
    int64_t n = MODE == kFwd ? at.n_first : at.n_last;
    row.start_at = -1;
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int i = MODE == kFwd ? k : R - 1 - k;
        if (i >= nv) continue;
        if (starts >> i & 1) {
            const float *src = MODE == kFwd ? p.h0 : p.g_hT;
            n = step_to<MODE>(q, n, t0 + i);
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
    }
}

template <typename IO, typename GT, int MODE, int VEC>
__device__ __forceinline__ void finish_border(const GlrParams &p, const Seqs &q, const Borders &at,
                                              const Row<IO, GT, MODE, VEC> &row, const float *hs, int64_t t0, int nv,
                                              int c0, int skip, float (&s)[VEC]) {
    constexpr int R = span_tokens<IO, GT, MODE, VEC>();
    const uint32_t starts = MODE == kFwd ? at.first : at.last, ends = MODE == kFwd ? at.last : at.first;
    int64_t n = MODE == kFwd ? at.n_first : at.n_last;
    IO *out = static_cast<IO *>(p.out) + t0 * p.D + c0;
    GT *dla = static_cast<GT *>(p.dla) + t0 * p.D + c0;
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int i = MODE == kFwd ? k : R - 1 - k;
        if (i >= nv) continue;
        if (starts >> i & 1) {
            const float *src = MODE == kFwd ? p.h0 : p.g_hT;
            n = step_to<MODE>(q, n, t0 + i);
#pragma unroll
            for (int e = 0; e < VEC; ++e) s[e] = 0.f;
            if (MODE == kFwd && i == row.start_at) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) s[e] = row.start[e];
            } else if (src) {
                load_f32<VEC>(src + n * p.D + c0, s);
            }
        }
        const int64_t to = (int64_t)i * p.D;
        float o[VEC], d[VEC], h[VEC];
        if constexpr (MODE != kFwd) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                h[e] = raw_at<VEC>(row.h[i], e);
                if constexpr (MODE == kBwd8) h[e] *= hs[i];
            }
            if (ends >> i & 1) {
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
        if (skip) {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (e >= skip) out[to + e] = from_f32<IO>(o[e]);
        } else {
            store_vec<IO, VEC>(out + to, o);
        }
        if constexpr (MODE != kFwd) store_vec<GT, VEC>(dla + to, d);
        if ((ends >> i & 1) && p.state_out) {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (e >= skip) p.state_out[n * p.D + c0 + e] = s[e];
        }
    }
}

// A map s -> a s + b of a lane's channels.
template <int VEC> struct alignas(VEC * 8) Map {
    float a[VEC], b[VEC];
    __device__ __forceinline__ void then(const Map &m) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            b[e] = decayed(m.a[e], b[e]) + m.b[e];
            a[e] = not_below(a[e] * m.a[e], min(min(bits_of(a[e]), bits_of(m.a[e])), 1u));
        }
    }
    // then m[0], m[stride], .., n of them: loads in batches, so that their latency
    // is paid once for each four
    __device__ __forceinline__ void then_all(const Map *m, int stride, int n) {
        for (int j = 0; j < n; j += 4) {
            Map w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = m[min(j + k, n - 1) * stride];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (j + k < n) then(w[k]);
        }
    }
};

template <int MODE, int VEC> struct alignas(32) GlrShared {
    Map<VEC> row[kNT];                              // the rows' maps
    Map<VEC> pre[kMaxGroup][64];                    // the maps of the group's tiles in front of this one
    float state[64 * VEC];                          // the state behind the last group
    float hs[MODE == kBwd8 ? kMaxScales : 1];       // scales of the tile's saved h
    int32_t cu[kStaged];
    uint32_t tile;
};

template <typename IO, typename GT, int MODE, int VEC>
__global__ __launch_bounds__(kNT, 4) void glr_kernel(const GlrParams p) {
    constexpr int R = span_tokens<IO, GT, MODE, VEC>();
    __shared__ GlrShared<MODE, VEC> sm;
    // Workgroups go to the 8 XCDs in turn: the channel tiles of a time tile follow one
    // another on the same XCD, whose L2 joins what they have of shared lines.
    const int tid = threadIdx.x;
    const int ct = (int)(p.time_tiles > 1 ? blockIdx.x / kXcds % p.chan_tiles : blockIdx.x);
    const bool staged = p.cu && p.N < kStaged;
    int64_t valid = p.tokens;                          // rows behind the last sequence are not touched
    if (p.cu) valid = min(valid, (int64_t)p.cu[p.N]);
    if (staged)
        for (int i = tid; i <= (int)p.N; i += kNT) sm.cu[i] = p.cu[i];
    if (p.time_tiles > 1 && tid == 0)
        sm.tile = __hip_atomic_fetch_add(p.tickets + ct * kTicketPitch, 1u, __ATOMIC_RELAXED,
                                         __HIP_MEMORY_SCOPE_AGENT);
    if (p.time_tiles > 1 || staged) __syncthreads();
    const int64_t tt = p.time_tiles > 1 ? sm.tile : 0;   // in the order of the scan
    if (tt >= p.time_tiles) return;                      // of a grid rounded up to whole XCDs
    const int lanes = p.lanes, rows = kNT / lanes;
    const int v = tid / lanes, cl = tid - v * lanes;     // row in the order of the scan, lane of it
    // where VEC does not divide D, the last lane's channels overlap its neighbour's:
    // both compute and write the same values
    const int cv = (ct * lanes + cl) * VEC, c0 = min(cv, p.D - VEC);
    const bool chan = cv < p.D && v < rows, last = v == rows - 1;
    // With h_T over h0 the neighbour's h_T may be there before the last lane reads
    // h0: what that lane has for the shared channels is not written then.
    const int skip = MODE == kFwd && p.over ? cv - c0 : 0;
    const Seqs q = {p.cu, sm.cu, staged, p.N, p.T};
    const int64_t span = MODE == kFwd ? tt * rows + v : (p.time_tiles - 1 - tt) * rows + (rows - 1 - v);
    const int64_t t0 = span * R;
    const int nv = chan ? (int)max((int64_t)0, min((int64_t)R, valid - t0)) : 0;

    // scales of the saved h: [block of the tile][token of the tile]
    const int b0 = ct * lanes * VEC / kAct8Block, nt = rows * R;
    float hsv[kMaxScales / kNT];
    if constexpr (MODE == kBwd8) {
        const int nb = (p.D + kAct8Block - 1) / kAct8Block;
        const int blocks = (min((ct + 1) * lanes * VEC, p.D) - 1) / kAct8Block - b0 + 1;
        const int64_t tile0 = (p.time_tiles - 1 - tt) * nt;
#pragma unroll
        for (int k = 0; k < kMaxScales / kNT; ++k) {
            const int i = tid + k * kNT, b = i / nt;
            const int64_t t = tile0 + i - b * nt;
            hsv[k] = b < blocks && t > 0 && t < valid ? p.hs[(t - 1) * nb + b0 + b] : 0.f;
        }
    }
    Row<IO, GT, MODE, VEC> row;
    if (p.keep) row.template load_inputs<true>(p, t0, nv, c0);
    else row.template load_inputs<false>(p, t0, nv, c0);
    const Borders at(q, t0, nv);
    const bool plain = __all(!chan || (nv == R && !at.first && !at.last)) && __any(chan);
    if (p.state_out) {   // empty sequences pass their state on
        for (int64_t n = tt; n < p.N; n += p.time_tiles) {
            if (v == 0 && chan && q.begin(n) == q.end(n)) {
                const float *src = MODE == kFwd ? p.h0 : p.g_hT;
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    p.state_out[n * p.D + c0 + e] = src ? src[n * p.D + c0 + e] : 0.f;
            }
        }
    }

    float L[VEC];   // the logarithm of the span's factor
    Map<VEC> own;
#pragma unroll
    for (int e = 0; e < VEC; ++e) L[e] = 0.f, own.b[e] = 0.f;
    if (!plain) compose_border<IO, GT, MODE, VEC>(p, q, at, row, t0, nv, c0, L, own.b);
    else if (chan) compose_inside<IO, GT, MODE, VEC>(row, L, own.b);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        own.a[e] = __expf(L[e]);
        // out of range, and not by a border or a gate of -inf: seldom, so that only
        // then the gates are asked whether one of them is a reset
        if (own.a[e] == 0.f && L[e] > -__builtin_inff()) {
            float least = 0.f;
#pragma unroll
            for (int i = 0; i < R; ++i)
                if (i < nv) least = fminf(least, raw_at<VEC>(row.la[i], e));
            own.a[e] = not_below(0.f, __expf(least) == 0.f ? 0 : 1);
        }
    }
    sm.row[tid] = own;
    if constexpr (MODE == kBwd8) {
#pragma unroll
        for (int k = 0; k < kMaxScales / kNT; ++k) sm.hs[tid + k * kNT] = hsv[k];
    }
    if constexpr (MODE != kFwd) {
        if (p.keep) row.template load_saved<true>(p, t0, nv, c0);
        else row.template load_saved<false>(p, t0, nv, c0);
    }
    __syncthreads();

    Map<VEC> s;   // its b: the state in front of this row
#pragma unroll
    for (int e = 0; e < VEC; ++e) s.a[e] = 1.f, s.b[e] = 0.f;
    if (p.time_tiles > 1) {
        const int pos = (int)(tt % p.group);         // tiles of the group in front of this one
        const bool anchored = tt >= p.group, closes = pos == p.group - 1;
        // a wave's words of one e are consecutive: whole lines to and from memory
        const int64_t pitch = (int64_t)p.chan_tiles * lanes * VEC;
        uint64_t *const words = p.words + (int64_t)ct * lanes * VEC + cl;
        const auto publish = [&](const Map<VEC> &m) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                uint32_t ab = __builtin_bit_cast(uint32_t, m.a[e]);
                if (ab == 0xffffffffu) ab = 0x7fc00000u;
                __hip_atomic_store(words + tt * pitch + e * lanes,
                                   (uint64_t)__builtin_bit_cast(uint32_t, m.b[e]) << 32 | ab, __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
            }
        };
        const auto await = [&](int64_t tile) {
            const uint64_t *w = words + tile * pitch;
            uint64_t got[VEC];
            bool there = false;
            for (int polls = 0; !there && polls < kMaxPolls; ++polls) {
                if (polls) __builtin_amdgcn_s_sleep(1);
                there = true;
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    got[e] = __hip_atomic_load(w + e * lanes, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
                for (int e = 0; e < VEC; ++e) there = there && (uint32_t)got[e] != 0xffffffffu;
            }
            Map<VEC> m;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                m.a[e] = there ? __builtin_bit_cast(float, (uint32_t)got[e]) : __builtin_nanf("");
                m.b[e] = there ? __builtin_bit_cast(float, (uint32_t)(got[e] >> 32)) : __builtin_nanf("");
            }
            return m;
        };
        Map<VEC> tile = s;   // the tile's map
        if (last && chan) {
            tile.then_all(sm.row + cl, lanes, rows);
            if (!closes) publish(tile);
        }
        if (chan)
            for (int j = v; j < pos; j += rows) sm.pre[j][cl] = await(tt - pos + j);
        if (pos) {
            __syncthreads();
            if (chan) s.then_all(&sm.pre[0][cl], 64, pos);
        }
        // The state behind the last group comes last, and what follows from it is
        // short: this is the chain that a long sequence waits for.
        if (last && chan) {
            Map<VEC> in = s;
#pragma unroll
            for (int e = 0; e < VEC; ++e) in.b[e] = 0.f;
            if (anchored) in = await(tt - pos - 1);
            if (closes) {
                Map<VEC> out = in;
                out.then(s);
                out.then(tile);
#pragma unroll
                for (int e = 0; e < VEC; ++e) out.a[e] = 0.f;
                publish(out);
            }
            if (anchored)
#pragma unroll
                for (int e = 0; e < VEC; ++e) sm.state[cl * VEC + e] = in.b[e];
        }
        if (anchored) {
            __syncthreads();
            if (chan) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) s.b[e] += decayed(s.a[e], sm.state[cl * VEC + e]);
            }
        }
    }
    if (chan) s.then_all(sm.row + cl, lanes, v);
    const float *hs = sm.hs;
    if constexpr (MODE == kBwd8) hs += (c0 / kAct8Block - b0) * nt + (rows - 1 - v) * R;
    if (plain) {
        if (chan) finish_inside<IO, GT, MODE, VEC>(p, row, hs, t0, c0, skip, s.b);
    } else {
        // Kept in the forward (20,000 sequences of 1 to 12 tokens: 337 against 359 us
        // for finding them again); in the backward, whose registers they would
        // overflow, found again (65536 x 2048: 244 against 250 us).
        if constexpr (MODE == kFwd)
            finish_border<IO, GT, MODE, VEC>(p, q, at, row, hs, t0, nv, c0, skip, s.b);
        else
            finish_border<IO, GT, MODE, VEC>(p, q, Borders(q, t0, nv), row, hs, t0, nv, c0, skip, s.b);
    }
}

// The workspace of a call: the tickets 0, every word absent.
__global__ __launch_bounds__(256) void glr_clear_kernel(uint32_t *tickets, int64_t nt, uint64_t *words, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    for (int64_t k = i; k < nt; k += (int64_t)gridDim.x * 256) tickets[k] = 0;
    for (int64_t k = i; k < n; k += (int64_t)gridDim.x * 256) words[k] = kAbsent;
}

// One token: four consecutive channels a thread (16 bytes of the state), the last
// few of the batch one by one.  In a replayed graph 1.8 us at 1 x 2048, which is a
// launch, 3.7 us at 256 x 4096 (14.7 MB, on chip between tokens), 10.6 us at 512 x
// 8192 (5.5 TB/s; one channel a thread: 12.9 us).
constexpr int kThreads = 256;
template <typename IO, typename GT>
__global__ __launch_bounds__(kThreads) void glr_step_kernel(const IO *__restrict__ x, const GT *__restrict__ la,
                                                            float *__restrict__ S, IO *__restrict__ h, int64_t n) {
    const int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 4;
    if (i + 4 <= n) {
        const auto lv = load_raw<GT, 4, true>(la + i);
        const auto xv = load_raw<IO, 4, true>(x + i);
        const auto sv = load_raw<float, 4, true>(S + i);
        float s[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            s[e] = decayed(__expf(raw_at<4>(lv, e)), raw_at<4>(sv, e)) + raw_at<4>(xv, e);
        store_vec<IO, 4>(h + i, s);
        typedef f32x4_t at __attribute__((aligned(4)));
        const f32x4_t r = {s[0], s[1], s[2], s[3]};
        *reinterpret_cast<at *>(S + i) = r;   // read again by the next token: stays in the L2
        return;
    }
    for (int64_t k = i; k < n; ++k) {
        const float s = decayed(__expf(to_f32(la[k])), S[k]) + to_f32(x[k]);
        S[k] = s;
        h[k] = from_f32<IO>(s);
    }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct GlrPlan {
    int vec, lanes;
    int64_t chan_tiles, time_tiles;
};
// Eight bytes of a token a lane (four channels in bf16, two in fp32), or one
// channel.  The channels are split evenly over rows of at most 64 lanes; rows may
// lie across waves.
GlrPlan glr_plan(const GlrArgs &a, int vec, int span) {
    GlrPlan g = {};
    g.vec = vec;
    const int64_t need = ceil_div(a.D, vec);
    g.chan_tiles = ceil_div(need, 64);
    g.lanes = (int)std::max(ceil_div(need, g.chan_tiles), (int64_t)kMinLanes);
    const int64_t tile = (int64_t)(kNT / g.lanes) * span;
    g.time_tiles = a.tokens > tile ? ceil_div(a.tokens, tile) : 1;
    return g;
}
int64_t glr_words(const GlrPlan &g) { return g.time_tiles * g.chan_tiles * g.lanes * g.vec; }
int64_t glr_grid(const GlrPlan &g) {
    return g.time_tiles > 1 ? ceil_div(g.time_tiles, kXcds) * kXcds * g.chan_tiles : g.chan_tiles;
}
// Tiles of a group.  A tile reads up to as many published maps, and a sequence's
// state passes through one group after the other.  With many channel tiles few time
// tiles run at once and the reads count; with few of them the chain does.
int32_t glr_group(const GlrPlan &g) { return g.chan_tiles >= 16 ? 8 : kMaxGroup; }
// The scales of a tile: a row of at least kMinLanes lanes has its channels in one
// block of 128, of more than 32 in at most three.
static_assert(kNT / kMinLanes * 32 <= kMaxScales && kNT / 33 * 32 * 3 <= kMaxScales, "scales of a tile");

// One channel a lane is for what the wide form cannot do: fewer channels than it
// takes, and an overlap of lanes that lies across a border of 128 saved codes (in
// either backward, so that both take the same sums).
int glr_vec(const GlrArgs &a) {
    const int vec = a.io_bf16 ? 4 : 2;
    if (a.D % vec == 0) return vec;
    return a.D < vec || (a.backward && a.D % kAct8Block < vec) ? 1 : vec;
}
// The tilings that a call of these sizes may take: the longest time axis of each.
template <typename F> void glr_each_plan(const GlrArgs &a, F f) {
    f(glr_plan(a, 1, 32));
    f(glr_plan(a, a.io_bf16 ? 4 : 2, kMinSpan));
}

template <typename IO, typename GT, int MODE> hipError_t launch_m(const GlrArgs &a, hipStream_t st) {
    constexpr int kWide = 8 / sizeof(IO), kWideSpan = span_tokens<IO, GT, MODE, kWide>();
    static_assert(kWideSpan >= kMinSpan && span_tokens<IO, GT, MODE, 1>() == 32, "the workspace's plans");
    const int vec = glr_vec(a);
    const GlrPlan g = glr_plan(a, vec, vec > 1 ? kWideSpan : 32);
    // a line that two channel tiles read is read from memory once if it is kept
    // (387 fp32 channels: 192 against 203 us for 139,000 tokens); whole lines are read
    // once and stream past the L2 (65536 x 4096 bf16: 318 against 332 us)
    const bool keep = a.D * sizeof(IO) % 128 != 0 || reinterpret_cast<uintptr_t>(a.x) % 128 != 0;
    GlrParams p = {a.x, a.log_alpha, a.h_in, a.h_scales, a.h0, a.d_hT, a.cu_seqlens, a.out, a.dlog_alpha, a.state_out,
                   a.num_seqs, a.seq_len, a.tokens, a.D, (int32_t)g.chan_tiles, g.lanes, g.time_tiles, nullptr,
                   !a.backward && a.state_out && a.state_out == a.h0, keep,
                   glr_group(g), nullptr};
    if (g.time_tiles > 1) {
        const int64_t nt = g.chan_tiles * kTicketPitch, n = glr_words(g);
        p.tickets = static_cast<uint32_t *>(a.workspace);
        p.words = reinterpret_cast<uint64_t *>(p.tickets + nt);
        hipLaunchKernelGGL(glr_clear_kernel, dim3((unsigned)std::min(ceil_div(n, 256), (int64_t)2048)), dim3(256), 0, st,
                           p.tickets, nt, p.words, n);
    }
    const dim3 grid((unsigned)glr_grid(g));
    if (g.vec > 1) hipLaunchKernelGGL((glr_kernel<IO, GT, MODE, kWide>), grid, dim3(kNT), 0, st, p);
    else hipLaunchKernelGGL((glr_kernel<IO, GT, MODE, 1>), grid, dim3(kNT), 0, st, p);
    return hipGetLastError();
}

template <typename IO, typename GT> hipError_t launch_t(const GlrArgs &a, hipStream_t st) {
    if (!a.backward) return launch_m<IO, GT, kFwd>(a, st);
    return a.h_scales ? launch_m<IO, GT, kBwd8>(a, st) : launch_m<IO, GT, kBwd>(a, st);
}

template <typename IO, typename GT> hipError_t step_t(const GlrStepArgs &a, hipStream_t st) {
    hipLaunchKernelGGL((glr_step_kernel<IO, GT>), dim3((unsigned)ceil_div(a.n, kThreads * 4)), dim3(kThreads), 0, st,
                       (const IO *)a.x, (const GT *)a.log_alpha, a.S, (IO *)a.h, a.n);
    return hipGetLastError();
}

int status(hipError_t e, char *err, size_t err_len) {
    if (e == hipSuccess) return 0;
    snprintf(err, err_len, "%s", hipGetErrorString(e));
    return -1;
}

}  // namespace

size_t glr_workspace_bytes(const GlrArgs &a) {
    size_t need = 0;
    glr_each_plan(a, [&](const GlrPlan &g) {
        if (g.time_tiles > 1)
            need = std::max(need, (size_t)g.chan_tiles * kTicketPitch * sizeof(uint32_t) +
                                      (size_t)glr_words(g) * sizeof(uint64_t));
    });
    return need;
}
bool glr_grids_fit(const GlrArgs &a) {
    bool fit = true;
    glr_each_plan(a, [&](const GlrPlan &g) {
        fit = fit && g.time_tiles <= kMaxWorkItems / kNT / g.chan_tiles && grid_fits(glr_grid(g), kNT);
    });
    return fit;
}
bool glr_step_grids_fit(const GlrStepArgs &a) { return grid_fits(ceil_div(a.n, kThreads * 4), kThreads); }

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
