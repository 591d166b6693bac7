// C ABI of the calls around the scan in a recurrent block (gated linear
// recurrence, layer norm, the causal conv's backward): argument validation on
// the host before any HIP call, planning, and dispatch to the launchers.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "block_internal.h"
#include "ssm.h"

namespace {

constexpr int64_t kMaxElems = int64_t(1) << 58;   // keeps every byte offset in int64
constexpr int64_t kMaxGrid = 0x7fffffff;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// a * b without overflow; -1 if it would exceed kMaxElems (or a factor is -1)
int64_t mul(int64_t a, int64_t b) {
    if (a < 0 || b < 0) return -1;
    if (a == 0 || b == 0) return 0;
    return a > kMaxElems / b ? -1 : a * b;
}

// every pointer NULL or a multiple of `a`
template <size_t N> bool all_aligned(const void* const (&ptrs)[N], uintptr_t a) {
    for (const void* p : ptrs)
        if (!aligned(p, a)) return false;
    return true;
}

bool is_dtype(int dtype) { return dtype == SSM_F32 || dtype == SSM_BF16; }

int gated_check_sizes(int64_t B, int64_t L, int64_t D, int dtype) {
    if (!is_dtype(dtype)) return SSM_ERR_BAD_DTYPE;
    if (B < 1 || D < 1 || L < 0) return SSM_ERR_BAD_SHAPE;
    if (mul(mul(B, D), L) < 0 || mul(B, D) < 0 || L > kMaxElems) return SSM_ERR_BAD_SHAPE;
    const int64_t strips = mul(B, (D + ssm::gated::kStrip - 1) / ssm::gated::kStrip);
    const int64_t tiles = (L + ssm::gated::kBwdTile - 1) / ssm::gated::kBwdTile;
    if (D > ssm::gated::kMaxRow) return SSM_ERR_UNSUPPORTED;
    if (strips < 0 || strips > kMaxGrid / ssm::gated::kMaxWalkers) return SSM_ERR_UNSUPPORTED;
    if (tiles > (int64_t(1) << 30)) return SSM_ERR_UNSUPPORTED;     // drawn from a 32-bit counter
    if (mul(mul(strips, tiles), 64 * 16) < 0 || mul(mul(B, tiles), mul(D, 32)) < 0)
        return SSM_ERR_BAD_SHAPE;
    return SSM_OK;
}

int norm_check_sizes(int64_t rows, int64_t D, int dtype) {
    if (!is_dtype(dtype)) return SSM_ERR_BAD_DTYPE;
    if (rows < 0 || D < 1) return SSM_ERR_BAD_SHAPE;
    if (mul(rows, D) < 0 || mul(D, 8192) < 0) return SSM_ERR_BAD_SHAPE;
    if (rows > kMaxGrid) return SSM_ERR_UNSUPPORTED;
    if ((D + 63) / 64 > kMaxGrid) return SSM_ERR_UNSUPPORTED;
    return SSM_OK;
}

int norm_bwd_check_sizes(int64_t rows, int64_t D, int dtype) {
    const int rc = norm_check_sizes(rows, D, dtype);
    if (rc != SSM_OK) return rc;
    return D > ssm::kMaxItems - 255 ? SSM_ERR_UNSUPPORTED : SSM_OK;    // the columns, in one launch
}

int conv_bwd_check_sizes(int64_t B, int64_t L, int64_t D, int64_t K, int dtype) {
    if (!is_dtype(dtype)) return SSM_ERR_BAD_DTYPE;
    if (B < 1 || D < 1 || L < 0 || K < 1) return SSM_ERR_BAD_SHAPE;
    if (mul(mul(B, L), D) < 0 || L > kMaxElems) return SSM_ERR_BAD_SHAPE;
    if (K > 4) return SSM_ERR_UNSUPPORTED;
    if (D > ssm::conv::kMaxRow) return SSM_ERR_UNSUPPORTED;
    if (mul(mul(B, D), 16) < 0) return SSM_ERR_BAD_SHAPE;           // states, and their grid
    if ((B * D + 255) / 256 > kMaxGrid) return SSM_ERR_UNSUPPORTED;
    const int64_t cells = mul(B, ssm::conv_bwd_blocks(L));
    if (mul(cells, mul(D, 20)) < 0) return SSM_ERR_BAD_SHAPE;       // partial sums
    if (mul(cells, (D + 63) / 64) < 0 || cells * ((D + 63) / 64) > kMaxGrid) return SSM_ERR_UNSUPPORTED;
    // a batch row, 512 threads to 64 channels of a block, in one launch
    if (ssm::conv_bwd_blocks(L) * ((D + 63) / 64) > ssm::kMaxItems / 512) return SSM_ERR_UNSUPPORTED;
    return SSM_OK;
}

int status(hipError_t e) { return e == hipSuccess ? SSM_OK : SSM_ERR_HIP; }

}  // namespace

extern "C" {

// ------------------------------------------------------------ gated scan

int ssm_gated_scan_walkers(int64_t B, int64_t L, int64_t D) {
    if (gated_check_sizes(B, L, D, SSM_F32) != SSM_OK) return 0;
    return ssm::plan_gated_fwd(B, L, D).walkers;
}

int ssm_gated_scan_bwd_walkers(int64_t B, int64_t L, int64_t D) {
    if (gated_check_sizes(B, L, D, SSM_F32) != SSM_OK) return 0;
    return ssm::plan_gated_bwd(B, L, D).walkers;
}

size_t ssm_gated_scan_workspace_bytes(int64_t B, int64_t L, int64_t D, int dtype) {
    if (gated_check_sizes(B, L, D, dtype) != SSM_OK) return 0;
    return ssm::plan_gated_fwd(B, L, D).chain_bytes;
}

size_t ssm_gated_scan_ckpt_bytes(int64_t B, int64_t L, int64_t D, int dtype) {
    if (gated_check_sizes(B, L, D, dtype) != SSM_OK) return 0;
    return (size_t)(B * ssm::gated_saved(L) * D * 4);
}

int ssm_gated_scan_fwd(const void* x, const void* gate_a, const void* gate_x, const float* A,
                       const float* bias_a, const float* bias_x, const float* h0, void* y,
                       float* h_last, float* ckpt, const int32_t* seq_lens, int64_t B, int64_t L,
                       int64_t D, int dtype, void* workspace, size_t workspace_bytes,
                       void* stream) {
    const int rc = gated_check_sizes(B, L, D, dtype);
    if (rc != SSM_OK) return rc;
    if (!A) return SSM_ERR_NULL_ARG;
    if (L > 0 && (!x || !gate_a || !gate_x || !y)) return SSM_ERR_NULL_ARG;
    if (!all_aligned({x, gate_a, gate_x, y, ckpt}, 16)) return SSM_ERR_MISALIGNED;
    if (!all_aligned({A, bias_a, bias_x, h0, h_last, seq_lens}, 4)) return SSM_ERR_MISALIGNED;
    ssm::GatedArgs a{};
    a.plan = ssm::plan_gated_fwd(B, L, D);
    a.saved = ssm::gated_saved(L);
    if (a.plan.chain_bytes) {
        if (!workspace || workspace_bytes < a.plan.chain_bytes) return SSM_ERR_WORKSPACE;
        if (!aligned(workspace, 256)) return SSM_ERR_MISALIGNED;
        a.chain = workspace;
    }
    a.x = x; a.gate_a = gate_a; a.gate_x = gate_x; a.A = A; a.bias_a = bias_a; a.bias_x = bias_x;
    a.h0 = h0; a.y = y; a.h_last = h_last; a.ckpt = ckpt; a.seq_lens = seq_lens;
    a.B = B; a.L = L; a.D = D; a.bf16 = dtype == SSM_BF16;
    return status(ssm::launch_gated_fwd(a, static_cast<hipStream_t>(stream)));
}

size_t ssm_gated_scan_bwd_workspace_bytes(int64_t B, int64_t L, int64_t D, int dtype,
                                          int with_ckpt) {
    if (gated_check_sizes(B, L, D, dtype) != SSM_OK) return 0;
    return ssm::gated_bwd_workspace_bytes(B, L, D, !with_ckpt);
}

int ssm_gated_scan_bwd(const void* x, const void* gate_a, const void* gate_x, const float* A,
                       const float* bias_a, const float* bias_x, const float* h0,
                       const float* ckpt, const void* dy, const float* dh_last, void* dx,
                       void* dgate_a, void* dgate_x, float* dA, float* dbias_a, float* dbias_x,
                       float* dh0, const int32_t* seq_lens, int64_t B, int64_t L, int64_t D,
                       int dtype, void* workspace, size_t workspace_bytes, void* stream) {
    const int rc = gated_check_sizes(B, L, D, dtype);
    if (rc != SSM_OK) return rc;
    if (!A || !dA) return SSM_ERR_NULL_ARG;
    if (L > 0 && (!x || !gate_a || !gate_x || !dy || !dx || !dgate_a || !dgate_x))
        return SSM_ERR_NULL_ARG;
    if (!all_aligned({x, gate_a, gate_x, dy, dx, dgate_a, dgate_x, ckpt}, 16))
        return SSM_ERR_MISALIGNED;
    if (!all_aligned({A, bias_a, bias_x, h0, dh_last, dA, dbias_a, dbias_x, dh0, seq_lens}, 4))
        return SSM_ERR_MISALIGNED;
    ssm::GatedBwdArgs a{};
    a.own_ckpt = ckpt == nullptr;
    const size_t need = ssm::gated_bwd_workspace_bytes(B, L, D, a.own_ckpt);
    if (need) {
        if (!workspace || workspace_bytes < need) return SSM_ERR_WORKSPACE;
        if (!aligned(workspace, 256)) return SSM_ERR_MISALIGNED;
    }
    a.f.plan = ssm::plan_gated_fwd(B, L, D);
    a.f.saved = ssm::gated_saved(L);
    a.plan = ssm::plan_gated_bwd(B, L, D);
    a.f.x = x; a.f.gate_a = gate_a; a.f.gate_x = gate_x; a.f.A = A; a.f.bias_a = bias_a;
    a.f.bias_x = bias_x; a.f.h0 = h0; a.f.ckpt = const_cast<float*>(ckpt);
    a.f.seq_lens = seq_lens; a.f.B = B; a.f.L = L; a.f.D = D; a.f.bf16 = dtype == SSM_BF16;
    a.dy = dy; a.dh_last = dh_last; a.dx = dx; a.dgate_a = dgate_a; a.dgate_x = dgate_x;
    a.dA = dA; a.dbias_a = dbias_a; a.dbias_x = dbias_x; a.dh0 = dh0;
    if (need) ssm::gated_bwd_carve(a, workspace);
    return status(ssm::launch_gated_bwd(a, static_cast<hipStream_t>(stream)));
}

int ssm_gated_state_update(float* state, const void* x, const void* gate_a, const void* gate_x,
                           const float* A, const float* bias_a, const float* bias_x, void* y,
                           int64_t B, int64_t D, int dtype, void* stream) {
    if (!is_dtype(dtype)) return SSM_ERR_BAD_DTYPE;
    if (B < 1 || D < 1 || mul(B, D) < 0) return SSM_ERR_BAD_SHAPE;
    if ((B * D + 255) / 256 > kMaxGrid) return SSM_ERR_UNSUPPORTED;
    if ((D % 2 == 0 ? D / 2 : D) > ssm::kMaxItems - 255) return SSM_ERR_UNSUPPORTED;   // a row, in one launch
    if (!state || !x || !gate_a || !gate_x || !A || !y) return SSM_ERR_NULL_ARG;
    if (!all_aligned({state, x, gate_a, gate_x, y}, 16)) return SSM_ERR_MISALIGNED;
    if (!all_aligned({A, bias_a, bias_x}, 4)) return SSM_ERR_MISALIGNED;
    ssm::GatedStepArgs a{};
    a.state = state; a.x = x; a.gate_a = gate_a; a.gate_x = gate_x; a.A = A; a.bias_a = bias_a;
    a.bias_x = bias_x; a.y = y; a.B = B; a.D = D; a.bf16 = dtype == SSM_BF16;
    return status(ssm::launch_gated_step(a, static_cast<hipStream_t>(stream)));
}

// ------------------------------------------------------------ layer norm

int ssm_layer_norm_fwd(const void* x, const float* residual, const float* weight,
                       const float* bias, float eps, void* y, float* residual_out, float* mean,
                       float* rstd, int64_t rows, int64_t D, int dtype, void* stream) {
    const int rc = norm_check_sizes(rows, D, dtype);
    if (rc != SSM_OK) return rc;
    if (!(eps >= 0.0f) || isinf(eps)) return SSM_ERR_UNSUPPORTED;
    if (rows > 0 && (!x || !y)) return SSM_ERR_NULL_ARG;
    if (residual_out && !residual) return SSM_ERR_NULL_ARG;
    if (!all_aligned({x, y, residual, residual_out}, 16)) return SSM_ERR_MISALIGNED;
    if (!all_aligned({weight, bias, mean, rstd}, 4)) return SSM_ERR_MISALIGNED;
    ssm::NormArgs a{};
    a.x = x; a.residual = residual; a.weight = weight; a.bias = bias; a.eps = eps; a.y = y;
    a.residual_out = residual_out; a.mean = mean; a.rstd = rstd; a.rows = rows; a.D = D;
    a.bf16 = dtype == SSM_BF16;
    return status(ssm::launch_layer_norm(a, static_cast<hipStream_t>(stream)));
}

size_t ssm_layer_norm_bwd_workspace_bytes(int64_t rows, int64_t D) {
    if (norm_bwd_check_sizes(rows, D, SSM_F32) != SSM_OK) return 0;
    return ssm::norm_bwd_workspace_bytes(rows, D);
}

int ssm_layer_norm_bwd(const void* x, int x_dtype, const void* dy, const float* mean,
                       const float* rstd, const float* weight, const float* dresidual_out,
                       void* dx, float* dresidual, float* dweight, float* dbias, int64_t rows,
                       int64_t D, int dtype, void* workspace, size_t workspace_bytes,
                       void* stream) {
    const int rc = norm_bwd_check_sizes(rows, D, dtype);
    if (rc != SSM_OK) return rc;
    if (!is_dtype(x_dtype)) return SSM_ERR_BAD_DTYPE;
    if (x_dtype != SSM_F32 && x_dtype != dtype) return SSM_ERR_UNSUPPORTED;
    if (rows > 0 && (!x || !dy || !mean || !rstd || !dx)) return SSM_ERR_NULL_ARG;
    if (!all_aligned({x, dy, dx, dresidual_out, dresidual}, 16)) return SSM_ERR_MISALIGNED;
    if (!all_aligned({mean, rstd, weight, dweight, dbias}, 4)) return SSM_ERR_MISALIGNED;
    const size_t need = ssm::norm_bwd_workspace_bytes(rows, D);
    if (need) {
        if (!workspace || workspace_bytes < need) return SSM_ERR_WORKSPACE;
        if (!aligned(workspace, 256)) return SSM_ERR_MISALIGNED;
    }
    ssm::NormBwdArgs a{};
    a.x = x; a.dy = dy; a.mean = mean; a.rstd = rstd; a.weight = weight;
    a.dresidual_out = dresidual_out; a.dx = dx; a.dresidual = dresidual; a.dweight = dweight;
    a.dbias = dbias; a.rows = rows; a.D = D; a.x_bf16 = x_dtype == SSM_BF16;
    a.bf16 = dtype == SSM_BF16; a.groups = ssm::norm_bwd_groups(rows);
    a.part = static_cast<float*>(workspace);
    return status(ssm::launch_layer_norm_bwd(a, static_cast<hipStream_t>(stream)));
}

// ------------------------------------------------------------ conv1d backward

size_t ssm_causal_conv1d_silu_bwd_workspace_bytes(int64_t B, int64_t L, int64_t D, int64_t K) {
    if (conv_bwd_check_sizes(B, L, D, K, SSM_F32) != SSM_OK) return 0;
    return ssm::conv_bwd_workspace_bytes(B, L, D, K);
}

int ssm_causal_conv1d_silu_bwd(const void* x, const float* weight, const float* bias,
                               const float* state_in, int silu, const void* du,
                               const float* dstate_out, void* dx, float* dweight, float* dbias,
                               float* dstate_in, int64_t B, int64_t L, int64_t D, int64_t K,
                               int dtype, void* workspace, size_t workspace_bytes, void* stream) {
    const int rc = conv_bwd_check_sizes(B, L, D, K, dtype);
    if (rc != SSM_OK) return rc;
    if (!weight || !dweight) return SSM_ERR_NULL_ARG;
    if (L > 0 && (!x || !du || !dx)) return SSM_ERR_NULL_ARG;
    if (!all_aligned({x, du, dx}, 16)) return SSM_ERR_MISALIGNED;
    if (!all_aligned({weight, bias, state_in, dstate_out, dweight, dbias, dstate_in}, 4))
        return SSM_ERR_MISALIGNED;
    const size_t need = ssm::conv_bwd_workspace_bytes(B, L, D, K);
    if (need) {
        if (!workspace || workspace_bytes < need) return SSM_ERR_WORKSPACE;
        if (!aligned(workspace, 256)) return SSM_ERR_MISALIGNED;
    }
    ssm::ConvBwdArgs a{};
    a.x = x; a.weight = weight; a.bias = bias; a.state_in = state_in; a.silu = silu != 0;
    a.du = du; a.dstate_out = dstate_out; a.dx = dx; a.dweight = dweight; a.dbias = dbias;
    a.dstate_in = dstate_in; a.B = B; a.L = L; a.D = D; a.K = K; a.bf16 = dtype == SSM_BF16;
    a.blocks = ssm::conv_bwd_blocks(L);
    a.part = static_cast<float*>(workspace);
    return status(ssm::launch_conv1d_bwd(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
