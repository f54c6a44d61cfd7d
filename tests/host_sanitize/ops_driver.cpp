// Drives the entry points of kda_ops_api.cpp with valid and invalid arguments,
// built with -fsanitize=address,undefined against host-only launchers: only
// valid calls reach one, and a launcher's error text comes back whole.
#include <limits.h>
#include <math.h>
#include <stdio.h>
#include <string.h>

#include "kda.h"
#include "kda_ops_launch.h"

namespace kda {
namespace {
int g_ops = 0;        // launches of this file's launchers
bool g_fail = false;  // they report an error
int note(char *err, size_t len) {
    ++g_ops;
    if (!g_fail) return 0;
    char msg[2048];
    memset(msg, 'x', sizeof(msg) - 1);   // longer than the error buffer
    msg[sizeof(msg) - 1] = '\0';
    snprintf(err, len, "%s", msg);
    return -1;
}
}  // namespace
size_t glr_workspace_bytes(const GlrArgs &a) { return a.tokens > 1024 ? 4096 : 0; }
bool glr_grids_fit(const GlrArgs &) { return true; }
int launch_glr(const GlrArgs &, void *, char *e, size_t n) { return note(e, n); }
bool glr_step_grids_fit(const GlrStepArgs &) { return true; }
int launch_glr_step(const GlrStepArgs &, void *, char *e, size_t n) { return note(e, n); }
bool act8_grids_fit(const Act8Args &) { return true; }
int launch_act8_pack(const Act8Args &, void *, char *e, size_t n) { return note(e, n); }
int launch_act8_unpack(const Act8Args &, void *, char *e, size_t n) { return note(e, n); }
bool norm_grids_fit(const NormArgs &) { return true; }
size_t norm_bwd_workspace_bytes(int64_t, int32_t) { return 1024; }
int launch_norm_fwd(const NormArgs &, void *, char *e, size_t n) { return note(e, n); }
int launch_norm_bwd(const NormArgs &, void *, char *e, size_t n) { return note(e, n); }
extern int g_launches;   // of the chunkwise launchers' stand-ins
}  // namespace kda

namespace {
alignas(256) unsigned char g_buf[1 << 12];   // stands in for device memory; never dereferenced
void *const P = g_buf;
float *const F = reinterpret_cast<float *>(g_buf);
int8_t *const C = reinterpret_cast<int8_t *>(g_buf);
int32_t *const I = reinterpret_cast<int32_t *>(g_buf);
int g_failures = 0;

#define EXPECT(call, want, ops)                                                                  \
    do {                                                                                         \
        const int before_ = kda::g_ops;                                                          \
        const kda_status_t rc_ = (call);                                                         \
        if (rc_ != (want) || kda::g_ops - before_ != (ops)) {                                    \
            fprintf(stderr, "line %d: %s -> %d, %d launches\n", __LINE__, #call, (int)rc_,      \
                    kda::g_ops - before_);                                                       \
            ++g_failures;                                                                        \
        }                                                                                        \
    } while (0)

kda_status_t chunk8(int32_t T, void *ws, size_t wsb, const int8_t *qc = C) {
    return kda_chunk_bwd_act8(qc, F, C, F, C, F, P, P, nullptr, nullptr, 0, P, nullptr, P, P, P, P, P, F, 1, T, 2, 128,
                              128, KDA_BF16, KDA_BF16, ws, wsb, nullptr);
}
}  // namespace

int main() {
    const int b = KDA_BF16;
    EXPECT(kda_glr_fwd(P, P, F, nullptr, 0, P, F, 2, 10, 64, b, b, nullptr, 0, nullptr), KDA_OK, 1);
    EXPECT(kda_glr_fwd(P, P, F, I, 3, P, F, 1, 10, 64, b, b, nullptr, 0, nullptr), KDA_OK, 1);
    EXPECT(kda_glr_fwd(P, P, F, I, 3, P, F, 1, 2000, 64, b, b, nullptr, 0, nullptr), KDA_ERR_WORKSPACE, 0);
    EXPECT(kda_glr_fwd(P, P, F, I, 3, P, F, 1, 2000, 64, b, b, P, 4096, nullptr), KDA_OK, 1);
    EXPECT(kda_glr_fwd(P, P, F, I, INT_MAX, P, F, 1, INT_MAX, INT_MAX, b, b, P, 4096, nullptr),
           KDA_ERR_INVALID_ARGUMENT, 0);
    EXPECT(kda_glr_fwd(P, P, F, nullptr, 0, P, F, INT_MAX, INT_MAX, INT_MAX, b, b, P, 4096, nullptr),
           KDA_ERR_INVALID_ARGUMENT, 0);
    EXPECT(kda_glr_fwd(P, P, F, nullptr, INT_MIN, P, F, 1, INT_MIN, INT_MIN, b, b, P, 4096, nullptr),
           KDA_ERR_INVALID_ARGUMENT, 0);
    EXPECT(kda_glr_bwd(P, P, F, nullptr, 0, P, F, P, P, F, 1, 10, 64, b, b, nullptr, 0, nullptr), KDA_OK, 1);
    EXPECT(kda_glr_bwd(P, nullptr, F, nullptr, 0, P, F, P, P, F, 1, 10, 64, b, b, nullptr, 0, nullptr),
           KDA_ERR_INVALID_ARGUMENT, 0);
    EXPECT(kda_glr_bwd(nullptr, nullptr, F, nullptr, 0, nullptr, F, nullptr, nullptr, F, 3, 0, 64, b, b, nullptr, 0,
                       nullptr), KDA_OK, 1);
    EXPECT(kda_glr_bwd_act8(P, C, F, F, nullptr, 0, P, F, P, P, F, 1, 10, 64, b, b, nullptr, 0, nullptr), KDA_OK, 1);
    EXPECT(kda_glr_bwd_act8(P, C, nullptr, F, nullptr, 0, P, F, P, P, F, 1, 10, 64, b, b, nullptr, 0, nullptr),
           KDA_ERR_INVALID_ARGUMENT, 0);
    EXPECT(kda_glr_step(P, P, F, P, 4, 64, b, b, nullptr), KDA_OK, 1);
    EXPECT(kda_act8_pack(P, C, F, 10, 64, b, nullptr), KDA_OK, 1);
    EXPECT(kda_act8_pack(P, C, F, INT64_MAX, INT_MAX, b, nullptr), KDA_ERR_INVALID_ARGUMENT, 0);
    EXPECT(kda_act8_unpack(C, F, P, 10, 64, b, nullptr), KDA_OK, 1);
    EXPECT(kda_act8_unpack(C, F, nullptr, 0, 64, b, nullptr), KDA_OK, 0);
    EXPECT(kda_rmsnorm_fwd(P, P, P, P, P, F, 10, 64, 1e-6f, b, b, nullptr), KDA_OK, 1);
    EXPECT(kda_rmsnorm_fwd(P, P, P, P, nullptr, F, 10, 64, 1e-6f, b, b, nullptr), KDA_ERR_INVALID_ARGUMENT, 0);
    EXPECT(kda_rmsnorm_fwd_act8(P, nullptr, nullptr, C, F, nullptr, nullptr, 10, 64, 1e-6f, b, b, nullptr), KDA_OK, 1);
    EXPECT(kda_rmsnorm_fwd_act8(P, nullptr, nullptr, C, F, nullptr, nullptr, INT64_MIN, 64, 1e-6f, b, b, nullptr),
           KDA_ERR_INVALID_ARGUMENT, 0);
    EXPECT(kda_rmsnorm_bwd(P, P, F, P, P, P, P, 10, 64, b, b, P, 1024, nullptr), KDA_OK, 1);
    EXPECT(kda_rmsnorm_bwd(P, P, F, P, P, P, P, 10, 64, b, b, P, 1023, nullptr), KDA_ERR_WORKSPACE, 0);
    EXPECT(kda_rmsnorm_bwd(P, P, F, P, P, P, nullptr, 10, 64, b, b, nullptr, 0, nullptr), KDA_OK, 1);
    EXPECT(kda_rmsnorm_bwd(nullptr, P, nullptr, nullptr, nullptr, nullptr, P, 0, 64, b, b, nullptr, 0, nullptr),
           KDA_OK, 1);
    EXPECT(kda_rmsnorm_bwd_act8(C, F, P, F, P, P, P, P, 10, 64, b, b, P, 1024, nullptr), KDA_OK, 1);

    const size_t need = kda_chunk_bwd_act8_workspace_size(1, 128, 2, 128, 128, 0, b);
    int before = kda::g_launches;
    EXPECT(chunk8(128, P, need - 1), KDA_ERR_WORKSPACE, 0);
    EXPECT(chunk8(128, P, need, nullptr), KDA_ERR_INVALID_ARGUMENT, 0);
    EXPECT(chunk8(128, g_buf + 8, need), KDA_ERR_INVALID_ARGUMENT, 0);
    EXPECT(chunk8(INT_MAX, P, need), KDA_ERR_WORKSPACE, 0);
    if (kda::g_launches != before) { fprintf(stderr, "a refused call was launched\n"); ++g_failures; }
    EXPECT(chunk8(128, P, need), KDA_OK, 3);
    if (kda::g_launches != before + 1) { fprintf(stderr, "the backward was not launched once\n"); ++g_failures; }

    kda::g_fail = true;
    EXPECT(kda_glr_step(P, P, F, P, 4, 64, b, b, nullptr), KDA_ERR_HIP, 1);
    const size_t len = strlen(kda_last_hip_error());
    if (len < 100 || len > 1024) { fprintf(stderr, "error text of %zu characters\n", len); ++g_failures; }
    EXPECT(chunk8(128, P, need), KDA_ERR_HIP, 1);
    kda::g_fail = false;
    if (g_failures) return 1;
    printf("ops driver: ok\n");
    return 0;
}
