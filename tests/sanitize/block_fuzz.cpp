// Host-only driver for the validation and planning code of the calls around
// the scan (block_abi.cpp, block_plan.cpp), built with AddressSanitizer and
// UndefinedBehaviorSanitizer on the host side only.  As abi_fuzz.cpp: edge and
// random sizes, one output pointer misaligned in every call, so that none may
// reach the kernel launchers (stand-ins here, which abort), and the sanitizers
// report any overflow of the size arithmetic.  Exit status 0: no finding.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include "block_internal.h"
#include "ssm.h"

namespace ssm {
[[noreturn]] static void reached(const char* what) {
    fprintf(stderr, "validation let a call through to %s\n", what);
    abort();
}
hipError_t launch_gated_fwd(const GatedArgs&, hipStream_t) { reached("launch_gated_fwd"); }
hipError_t launch_gated_bwd(const GatedBwdArgs&, hipStream_t) { reached("launch_gated_bwd"); }
hipError_t launch_gated_step(const GatedStepArgs&, hipStream_t) { reached("launch_gated_step"); }
hipError_t launch_layer_norm(const NormArgs&, hipStream_t) { reached("launch_layer_norm"); }
hipError_t launch_layer_norm_bwd(const NormBwdArgs&, hipStream_t) { reached("launch_layer_norm_bwd"); }
hipError_t launch_conv1d_bwd(const ConvBwdArgs&, hipStream_t) { reached("launch_conv1d_bwd"); }
}  // namespace ssm

namespace {

alignas(256) char g_buf[1024];
void* const kOk = g_buf;
float* const kOkF = reinterpret_cast<float*>(g_buf);
void* const kMis = g_buf + 2;

const int64_t kEdge[] = {INT64_MIN, -1, 0, 1, 2, 3, 4, 7, 63, 64, 65, 127, 128, 129, 255, 256, 257, 768,
                         2048, 65535, 65536, 131072, int64_t(1) << 25, (int64_t(1) << 31) - 1,
                         int64_t(1) << 31, int64_t(1) << 38, int64_t(1) << 50, int64_t(1) << 58,
                         int64_t(1) << 62, INT64_MAX - 1, INT64_MAX};
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

int g_failures = 0;
void refused(const char* name, int rc, int64_t a, int64_t b, int64_t c) {
    if (rc <= SSM_OK || rc >= SSM_ERR_HIP) {
        fprintf(stderr, "%s(%lld, %lld, %lld): status %d\n", name, (long long)a, (long long)b,
                (long long)c, rc);
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
        const int64_t B = draw(), L = draw(), D = draw(), K = (int64_t)(next() % 7);
        const int dt = (int)(next() % 3);
        refused("gated_scan_fwd",
                ssm_gated_scan_fwd(kOk, kOk, kOk, kOkF, kOkF, kOkF, kOkF, kMis, kOkF, kOkF, nullptr, B, L, D,
                                   dt, kOk, ws, nullptr), B, L, D);
        refused("gated_scan_bwd",
                ssm_gated_scan_bwd(kOk, kOk, kOk, kOkF, kOkF, kOkF, kOkF, k % 2 ? kOkF : nullptr, kOk, kOkF,
                                   kMis, kOk, kOk, kOkF, kOkF, kOkF, kOkF, nullptr, B, L, D, dt, kOk, ws,
                                   nullptr), B, L, D);
        refused("gated_state_update",
                ssm_gated_state_update(kOkF, kOk, kOk, kOk, kOkF, kOkF, kOkF, kMis, B, D, dt, nullptr), B, D, 0);
        refused("layer_norm_fwd",
                ssm_layer_norm_fwd(kOk, kOkF, kOkF, kOkF, 1e-5f, kMis, kOkF, kOkF, kOkF, B, D, dt, nullptr),
                B, D, 0);
        refused("layer_norm_bwd",
                ssm_layer_norm_bwd(kOk, SSM_F32, kOk, kOkF, kOkF, kOkF, kOkF, kMis, kOkF, kOkF, kOkF, B, D,
                                   dt, kOk, ws, nullptr), B, D, 0);
        refused("causal_conv1d_silu_bwd",
                ssm_causal_conv1d_silu_bwd(kOk, kOkF, kOkF, kOkF, 1, kOk, kOkF, kMis, kOkF, kOkF, kOkF, B, L,
                                           D, K, dt, kOk, ws, nullptr), B, L, D);
        const int w = ssm_gated_scan_walkers(B, L, D);
        holds("0 <= walkers <= 64", w >= 0 && w <= 64, B, L, D);
        const size_t f = ssm_gated_scan_workspace_bytes(B, L, D, SSM_BF16);
        const size_t with = ssm_gated_scan_bwd_workspace_bytes(B, L, D, SSM_BF16, 1);
        const size_t without = ssm_gated_scan_bwd_workspace_bytes(B, L, D, SSM_BF16, 0);
        holds("one walker shares nothing", w > 1 || f == 0, B, L, D);
        holds("the backward's own sweep adds what the forward needs, and the states",
              without >= with + f && (w == 0 || without >= with + ssm_gated_scan_ckpt_bytes(B, L, D, SSM_BF16)),
              B, L, D);
        (void)ssm_layer_norm_bwd_workspace_bytes(B, D);
        (void)ssm_causal_conv1d_silu_bwd_workspace_bytes(B, L, D, K);
    }
    if (g_failures) return 1;
    printf("%ld draws, no finding\n", n);
    return 0;
}
