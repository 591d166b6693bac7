// Host-only driver for the validation and planning code of linear attention,
// the head norm and the moves between slots (linear_abi.cpp, linear_plan.cpp),
// built with AddressSanitizer and UndefinedBehaviorSanitizer on the host side
// only.  As block_fuzz.cpp: edge and random sizes, one output pointer
// misaligned in every call, so that none may reach the kernel launchers
// (stand-ins here, which abort), and the sanitizers report any overflow of the
// size arithmetic.  Exit status 0: no finding.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include "block_internal.h"
#include "linear_internal.h"
#include "ssm.h"

namespace ssm {
[[noreturn]] static void reached(const char* what) {
    fprintf(stderr, "validation let a call through to %s\n", what);
    abort();
}
hipError_t launch_linear_run(const LinearRun&, bool, hipStream_t) { reached("launch_linear_run"); }
hipError_t launch_linear_join(const LinearJoin&, hipStream_t) { reached("launch_linear_join"); }
hipError_t launch_linear_decay_grad(const LinearDecayGrad&, hipStream_t) { reached("launch_linear_decay_grad"); }
hipError_t launch_linear_group_sum(const LinearGroupSum&, hipStream_t) { reached("launch_linear_group_sum"); }
hipError_t launch_linear_step(const LinearStepArgs&, hipStream_t) { reached("launch_linear_step"); }
hipError_t launch_column_sums(const ColumnSums&, hipStream_t) { reached("launch_column_sums"); }
hipError_t launch_head_norm(const HeadNormArgs&, hipStream_t) { reached("launch_head_norm"); }
hipError_t launch_head_norm_bwd(const HeadNormArgs&, hipStream_t) { reached("launch_head_norm_bwd"); }
hipError_t launch_slots_copy(const SlotsArgs&, hipStream_t) { reached("launch_slots_copy"); }
}  // namespace ssm

namespace {

alignas(256) char g_buf[1024];
void* const kOk = g_buf;
float* const kOkF = reinterpret_cast<float*>(g_buf);
int32_t* const kOkI = reinterpret_cast<int32_t*>(g_buf);
void* const kMis = g_buf + 2;

const int64_t kEdge[] = {INT64_MIN, -1, 0, 1, 2, 3, 4, 15, 16, 17, 32, 48, 64, 65, 128, 255, 256, 257, 272, 512, 514,
                         2048, 16384, 65536, 131072, int64_t(1) << 21, int64_t(1) << 22, int64_t(1) << 24,
                         int64_t(1) << 25, int64_t(1) << 30, (int64_t(1) << 31) - 1, int64_t(1) << 31,
                         int64_t(1) << 38, int64_t(1) << 50, int64_t(1) << 58, int64_t(1) << 62, INT64_MAX - 1,
                         INT64_MAX};
constexpr int kNumEdge = sizeof(kEdge) / sizeof(kEdge[0]);

uint64_t g_state = 0x9E3779B97F4A7C15ull;
uint64_t next() {
    uint64_t z = (g_state += 0x9E3779B97F4A7C15ull);
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    return z ^ (z >> 31);
}
int64_t draw() {
    switch (next() % 4) {
        case 0: case 1: return kEdge[next() % kNumEdge];
        case 2: return (int64_t)(next() % 5000);
        default: return (int64_t)(next() >> (next() % 64));
    }
}
// sizes that pass more often
int64_t small() { return next() % 4 ? (int64_t)(next() % 65) : draw(); }
int64_t width() { return next() % 4 ? 16 * (int64_t)(1 + next() % 16) : draw(); }

int g_failures = 0;
void refused(const char* name, int rc, int64_t a, int64_t b, int64_t c) {
    if (rc <= SSM_OK || rc >= SSM_ERR_HIP) {
        fprintf(stderr, "%s(%lld, %lld, %lld): status %d\n", name, (long long)a, (long long)b, (long long)c, rc);
        ++g_failures;
    }
}
void holds(const char* what, bool ok, int64_t a, int64_t b, int64_t c) {
    if (!ok) {
        fprintf(stderr, "%s fails at (%lld, %lld, %lld)\n", what, (long long)a, (long long)b, (long long)c);
        ++g_failures;
    }
}

}  // namespace

int main(int argc, char** argv) {
    const long n = argc > 1 ? atol(argv[1]) : 100000;
    const size_t ws = SIZE_MAX;
    for (long k = 0; k < n && g_failures < 20; ++k) {
        const int64_t B = small(), L = draw(), G = small();
        const int64_t H = G > 0 && G < 100000 && next() % 2 ? G * (int64_t)(1 + next() % 4) : small();
        const int64_t Dk = width(), Dv = width(), qr = draw(), kr = draw(), vr = draw();
        const int dt = (int)(next() % 3), by = (int)(next() % 2);
        refused("linear_attention_fwd",
                ssm_linear_attention_fwd(kOk, kOk, kOk, kOkF, by, 1.0f, kOkF, kMis, kOkF, kOkI, qr, kr, vr, B, L, H, G,
                                         Dk, Dv, dt, kOk, ws, nullptr), B, L, H);
        refused("linear_attention_bwd",
                ssm_linear_attention_bwd(kOk, kOk, kOk, kOkF, by, 1.0f, kOkF, kOk, kOkF, kMis, kOk, kOk, kOkF, kOkF,
                                         kOkI, qr, kr, vr, B, L, H, G, Dk, Dv, dt, kOk, ws, nullptr), B, L, H);
        refused("linear_state_update",
                ssm_linear_state_update(kOkF, kOk, kOk, kOk, kOkF, by, 1.0f, next() % 2 ? kOkI : nullptr, kMis, qr, kr,
                                        vr, B, draw(), H, G, Dk, Dv, dt, nullptr), B, H, Dk);
        const int64_t rows = draw(), hq = small(), hk = small(), w = next() % 4 ? 2 * (int64_t)(next() % 260) : draw();
        const int64_t rot = next() % 2 ? w / 2 / 2 * 2 : draw();
        refused("qk_norm_rope_fwd",
                ssm_qk_norm_rope_fwd(kOk, kOk, kOkF, kOkF, kOkI, kOkF, 0, 1e-6f, kMis, kOk, qr, kr, rows, hq, hk, w, rot,
                                     dt, nullptr), rows, hq, w);
        refused("qk_norm_rope_bwd",
                ssm_qk_norm_rope_bwd(kOk, kOk, kOk, kOk, kOkF, kOkF, kOkI, kOkF, 0, 1e-6f, kMis, kOk, kOkF, kOkF, qr, kr,
                                     rows, hq, hk, w, rot, dt, kOk, ws, nullptr), rows, hq, w);
        const int64_t layers = draw(), slots = draw(), size = draw(), m = draw();
        if (m != 0 && layers != 0 && size != 0)
            refused("state_slots_copy",
                    ssm_state_slots_copy(kOk, kOkI, reinterpret_cast<int32_t*>(kMis), layers, slots, size, m, nullptr),
                    layers, slots, size);
        // whether a launch holds the moves
        if (layers > 0 && layers < (int64_t(1) << 40) && size > 0 && size < (int64_t(1) << 50))
            (void)ssm::slots_copy_fits(ssm::SlotsArgs{kOk, kOkI, kOkI, layers, 1, size, 1 + (int64_t)(next() % 2048)});
        const int seg = ssm_linear_attention_segments(B, L, H, Dk, Dv, dt);
        holds("0 <= segments <= 256", seg >= 0 && seg <= 256, B, L, H);
        const size_t need = ssm_linear_attention_workspace_bytes(B, L, H, Dk, Dv, dt);
        holds("one segment needs nothing", seg > 1 || need == 0, B, L, H);
        holds("segments hold their states", seg <= 1 || need >= (size_t)(seg * B * H * Dk * Dv * 4), B, L, H);
        (void)ssm_linear_attention_bwd_segments(B, L, H, Dk, Dv, dt);
        (void)ssm_linear_attention_bwd_workspace_bytes(B, L, H, G, Dk, Dv, by, dt);
        (void)ssm_qk_norm_rope_bwd_workspace_bytes(rows, w);
    }
    if (g_failures) return 1;
    printf("%ld draws, no finding\n", n);
    return 0;
}
