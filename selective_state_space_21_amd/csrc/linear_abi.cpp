// C ABI of linear attention with a decay for each head, of the head norm with
// rotary positions and of the moves between a state pool's slots: argument
// validation on the host before any HIP call, and dispatch to the launchers.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "block_internal.h"
#include "linear_internal.h"
#include "ssm.h"

namespace {

constexpr int64_t kMaxElems = int64_t(1) << 58;   // keeps every byte offset in int64

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// a * b without overflow; -1 if it would exceed kMaxElems (or a factor is -1)
int64_t mul(int64_t a, int64_t b) {
    if (a < 0 || b < 0) return -1;
    if (a == 0 || b == 0) return 0;
    return a > kMaxElems / b ? -1 : a * b;
}

template <size_t N> bool all_aligned(const void* const (&ptrs)[N], uintptr_t a) {
    for (const void* p : ptrs)
        if (!aligned(p, a)) return false;
    return true;
}

bool is_dtype(int dtype) { return dtype == SSM_F32 || dtype == SSM_BF16; }
int status(hipError_t e) { return e == hipSuccess ? SSM_OK : SSM_ERR_HIP; }

// workgroups of 256 threads that go out as one launch
constexpr int64_t kMaxBlocks = int64_t(1) << 24;

int linear_check_sizes(int64_t B, int64_t L, int64_t H, int64_t G, int64_t Dk, int64_t Dv, int dtype) {
    if (!is_dtype(dtype)) return SSM_ERR_BAD_DTYPE;
    if (B < 1 || L < 0 || H < 1 || G < 1 || Dk < 1 || Dv < 1) return SSM_ERR_BAD_SHAPE;
    if (H % G) return SSM_ERR_BAD_SHAPE;
    if (mul(mul(B, H), 65536 * 16) < 0 || mul(mul(mul(B, H), L), 65536) < 0 || L > kMaxElems)
        return SSM_ERR_BAD_SHAPE;
    if (Dk % 16 || Dv % 16 || Dk > ssm::linear::kMaxWidth || Dv > ssm::linear::kMaxWidth) return SSM_ERR_UNSUPPORTED;
    if (H * ssm::linear::kMaxWidth > ssm::linear::kMaxRow) return SSM_ERR_UNSUPPORTED;
    // a head of a row has up to four column tiles of 512 threads, in one launch of less than 2^32
    if (B * H > kMaxBlocks / 16 || L > (int64_t(1) << 30)) return SSM_ERR_UNSUPPORTED;
    return SSM_OK;
}

// the parameters' gradients' last launches hold four elements a thread
bool group_sums_fit(int64_t B, int64_t L, int64_t G, int64_t Dk) {
    return mul(mul(B, L), mul(G, Dk)) >= 0 && B * L * G * (Dk / 4) <= ssm::kMaxItems - 256;
}

// strides between tokens: rows of `width` that do not overlap, within 32-bit offsets of a chunk
bool row_ok(int64_t row, int64_t width, int dtype) {
    return row >= width && row <= ssm::linear::kMaxRow && row % (dtype == SSM_BF16 ? 8 : 4) == 0;
}

}  // namespace

extern "C" {

// ------------------------------------------------------------ linear attention

int ssm_linear_attention_segments(int64_t B, int64_t L, int64_t H, int64_t Dk, int64_t Dv, int dtype) {
    if (linear_check_sizes(B, L, H, H, Dk, Dv, dtype) != SSM_OK) return 0;
    return ssm::plan_linear_fwd(B, L, H, Dk, Dv, dtype == SSM_BF16).segments;
}

int ssm_linear_attention_bwd_segments(int64_t B, int64_t L, int64_t H, int64_t Dk, int64_t Dv, int dtype) {
    if (linear_check_sizes(B, L, H, H, Dk, Dv, dtype) != SSM_OK) return 0;
    return ssm::plan_linear_bwd(B, L, H, Dk, Dv, dtype == SSM_BF16).segments;
}

size_t ssm_linear_attention_workspace_bytes(int64_t B, int64_t L, int64_t H, int64_t Dk, int64_t Dv, int dtype) {
    if (linear_check_sizes(B, L, H, H, Dk, Dv, dtype) != SSM_OK) return 0;
    return ssm::linear_fwd_workspace_bytes(B, L, H, Dk, Dv, dtype == SSM_BF16);
}

int ssm_linear_attention_fwd(const void* q, const void* k, const void* v, const float* log_decay, int by_head,
                             float scale, const float* h0, void* o, float* h_last, const int32_t* seq_lens,
                             int64_t q_row, int64_t k_row, int64_t v_row, int64_t B, int64_t L, int64_t H, int64_t G,
                             int64_t Dk, int64_t Dv, int dtype, void* workspace, size_t workspace_bytes,
                             void* stream) {
    const int rc = linear_check_sizes(B, L, H, G, Dk, Dv, dtype);
    if (rc != SSM_OK) return rc;
    if (!row_ok(q_row, G * Dk, dtype) || !row_ok(k_row, G * Dk, dtype) || !row_ok(v_row, H * Dv, dtype))
        return SSM_ERR_BAD_SHAPE;
    if (!isfinite(scale)) return SSM_ERR_UNSUPPORTED;
    if (L > 0 && (!q || !k || !v || !log_decay || !o)) return SSM_ERR_NULL_ARG;
    if (!all_aligned({q, k, v, o}, 16)) return SSM_ERR_MISALIGNED;
    if (!all_aligned({log_decay, h0, h_last, seq_lens}, 4)) return SSM_ERR_MISALIGNED;
    ssm::LinearArgs a{};
    a.bf16 = dtype == SSM_BF16;
    const size_t need = ssm::linear_fwd_workspace_bytes(B, L, H, Dk, Dv, a.bf16);
    if (need) {
        if (!workspace || workspace_bytes < need) return SSM_ERR_WORKSPACE;
        if (!aligned(workspace, 256)) return SSM_ERR_MISALIGNED;
    }
    a.plan = ssm::plan_linear_fwd(B, L, H, Dk, Dv, a.bf16);
    a.q = q; a.k = k; a.v = v; a.g = log_decay; a.by_head = by_head != 0; a.scale = scale;
    a.h0 = h0; a.o = o; a.h_last = h_last; a.seq_lens = seq_lens;
    a.q_row = q_row; a.k_row = k_row; a.v_row = v_row;
    a.B = B; a.L = L; a.H = H; a.G = G; a.Dk = Dk; a.Dv = Dv;
    a.workspace = workspace;
    return status(ssm::launch_linear_fwd(a, static_cast<hipStream_t>(stream)));
}

size_t ssm_linear_attention_bwd_workspace_bytes(int64_t B, int64_t L, int64_t H, int64_t G, int64_t Dk, int64_t Dv,
                                                int by_head, int dtype) {
    if (linear_check_sizes(B, L, H, G, Dk, Dv, dtype) != SSM_OK) return 0;
    return ssm::linear_bwd_workspace_bytes(B, L, H, G, Dk, Dv, dtype == SSM_BF16, by_head != 0);
}

int ssm_linear_attention_bwd(const void* q, const void* k, const void* v, const float* log_decay, int by_head,
                             float scale, const float* h0, const void* d_o, const float* dh_last, void* dq, void* dk,
                             void* dv, float* dlog_decay, float* dh0, const int32_t* seq_lens, int64_t q_row,
                             int64_t k_row, int64_t v_row, int64_t B, int64_t L, int64_t H, int64_t G, int64_t Dk,
                             int64_t Dv, int dtype, void* workspace, size_t workspace_bytes, void* stream) {
    const int rc = linear_check_sizes(B, L, H, G, Dk, Dv, dtype);
    if (rc != SSM_OK) return rc;
    if (!row_ok(q_row, G * Dk, dtype) || !row_ok(k_row, G * Dk, dtype) || !row_ok(v_row, H * Dv, dtype))
        return SSM_ERR_BAD_SHAPE;
    if (!isfinite(scale)) return SSM_ERR_UNSUPPORTED;
    if (!group_sums_fit(B, L, G, Dk)) return SSM_ERR_UNSUPPORTED;
    if (L > 0 && (!q || !k || !v || !log_decay || !d_o || !dq || !dk || !dv)) return SSM_ERR_NULL_ARG;
    if (!all_aligned({q, k, v, d_o, dq, dk, dv}, 16)) return SSM_ERR_MISALIGNED;
    if (!all_aligned({log_decay, h0, dh_last, dlog_decay, dh0, seq_lens}, 4)) return SSM_ERR_MISALIGNED;
    ssm::LinearBwdArgs a{};
    a.f.bf16 = dtype == SSM_BF16;
    const size_t need = ssm::linear_bwd_workspace_bytes(B, L, H, G, Dk, Dv, a.f.bf16, by_head != 0);
    if (!workspace || workspace_bytes < need) return SSM_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return SSM_ERR_MISALIGNED;
    a.f.plan = ssm::plan_linear_bwd(B, L, H, Dk, Dv, a.f.bf16);
    a.f.q = q; a.f.k = k; a.f.v = v; a.f.g = log_decay; a.f.by_head = by_head != 0; a.f.scale = scale;
    a.f.h0 = h0; a.f.seq_lens = seq_lens;
    a.f.q_row = q_row; a.f.k_row = k_row; a.f.v_row = v_row;
    a.f.B = B; a.f.L = L; a.f.H = H; a.f.G = G; a.f.Dk = Dk; a.f.Dv = Dv;
    a.f.workspace = workspace;
    a.d_o = d_o; a.dh_last = dh_last; a.dq = dq; a.dk = dk; a.dv = dv; a.dg = dlog_decay; a.dh0 = dh0;
    return status(ssm::launch_linear_bwd(a, static_cast<hipStream_t>(stream)));
}

int ssm_linear_state_update(float* state, const void* q, const void* k, const void* v, const float* log_decay,
                            int by_head, float scale, const int32_t* slots, void* o, int64_t q_row, int64_t k_row,
                            int64_t v_row, int64_t B, int64_t n_slots, int64_t H, int64_t G, int64_t Dk, int64_t Dv,
                            int dtype, void* stream) {
    const int rc = linear_check_sizes(B, 1, H, G, Dk, Dv, dtype);
    if (rc != SSM_OK) return rc;
    if (n_slots < 1 || mul(mul(n_slots, H), Dk * Dv) < 0 || (!slots && n_slots < B)) return SSM_ERR_BAD_SHAPE;
    if (n_slots > 0x7fffffff) return SSM_ERR_UNSUPPORTED;
    if (!row_ok(q_row, G * Dk, dtype) || !row_ok(k_row, G * Dk, dtype) || !row_ok(v_row, H * Dv, dtype))
        return SSM_ERR_BAD_SHAPE;
    if (!isfinite(scale)) return SSM_ERR_UNSUPPORTED;
    if (!state || !q || !k || !v || !log_decay || !o) return SSM_ERR_NULL_ARG;
    if (!all_aligned({state, q, k, v, o}, 16)) return SSM_ERR_MISALIGNED;
    if (!all_aligned({log_decay, slots}, 4)) return SSM_ERR_MISALIGNED;
    ssm::LinearStepArgs a{};
    a.state = state; a.q = q; a.k = k; a.v = v; a.g = log_decay; a.by_head = by_head != 0; a.scale = scale;
    a.slots = slots; a.o = o; a.q_row = q_row; a.k_row = k_row; a.v_row = v_row;
    a.B = B; a.n_slots = n_slots; a.H = H; a.G = G; a.Dk = Dk; a.Dv = Dv; a.bf16 = dtype == SSM_BF16;
    return status(ssm::launch_linear_step(a, static_cast<hipStream_t>(stream)));
}

// ------------------------------------------------------------ head norm and rotation

static int head_norm_check(int64_t rows, int64_t q_heads, int64_t k_heads, int64_t width, int64_t rotary,
                           const void* positions, const float* inv_freq, int64_t q_row, int64_t k_row, float eps,
                           int dtype) {
    if (!is_dtype(dtype)) return SSM_ERR_BAD_DTYPE;
    if (rows < 0 || q_heads < 0 || k_heads < 0 || width < 1 || rotary < 0) return SSM_ERR_BAD_SHAPE;
    if (rotary > width || rotary % 2) return SSM_ERR_BAD_SHAPE;
    if (mul(rows, mul(q_heads, width)) < 0 || mul(rows, mul(k_heads, width)) < 0) return SSM_ERR_BAD_SHAPE;
    if (q_row < q_heads * width || k_row < k_heads * width || mul(rows, q_row) < 0 || mul(rows, k_row) < 0)
        return SSM_ERR_BAD_SHAPE;
    if (width % 2 || width > 512) return SSM_ERR_UNSUPPORTED;
    if (q_heads > 65536 || k_heads > 65536 || rows > kMaxBlocks) return SSM_ERR_UNSUPPORTED;
    if (!(eps >= 0.0f) || isinf(eps)) return SSM_ERR_UNSUPPORTED;
    if (rows > 0 && rotary > 0 && (!positions || !inv_freq)) return SSM_ERR_NULL_ARG;
    if (!all_aligned({positions, inv_freq}, 4)) return SSM_ERR_MISALIGNED;
    return SSM_OK;
}

int ssm_qk_norm_rope_fwd(const void* q, const void* k, const float* q_weight, const float* k_weight,
                         const int32_t* positions, const float* inv_freq, int interleaved, float eps, void* q_out,
                         void* k_out, int64_t q_row, int64_t k_row, int64_t rows, int64_t q_heads, int64_t k_heads,
                         int64_t width, int64_t rotary, int dtype, void* stream) {
    const int rc = head_norm_check(rows, q_heads, k_heads, width, rotary, positions, inv_freq, q_row, k_row, eps,
                                   dtype);
    if (rc != SSM_OK) return rc;
    if (rows > 0 && ((q_heads > 0 && (!q || !q_out)) || (k_heads > 0 && (!k || !k_out)))) return SSM_ERR_NULL_ARG;
    if (!all_aligned({q, k}, dtype == SSM_BF16 ? 2 : 4)) return SSM_ERR_MISALIGNED;
    if (!all_aligned({q_out, k_out}, 16) || !all_aligned({q_weight, k_weight}, 4)) return SSM_ERR_MISALIGNED;
    ssm::HeadNormArgs a{};
    a.x[0] = q; a.x[1] = k; a.x_row[0] = q_row; a.x_row[1] = k_row; a.heads[0] = q_heads; a.heads[1] = k_heads;
    a.weight[0] = q_weight; a.weight[1] = k_weight; a.positions = positions; a.inv_freq = inv_freq;
    a.rows = rows; a.width = (int32_t)width; a.rotary = (int32_t)rotary; a.interleaved = interleaved != 0;
    a.eps = eps; a.bf16 = dtype == SSM_BF16;
    a.y[0] = q_out; a.y[1] = k_out;
    return status(ssm::launch_head_norm(a, static_cast<hipStream_t>(stream)));
}

size_t ssm_qk_norm_rope_bwd_workspace_bytes(int64_t rows, int64_t width) {
    if (rows < 0 || rows > kMaxBlocks || width < 1 || width > 512) return 0;
    return (size_t)(ssm::head_norm_groups(rows) * 2 * width * 4);
}

int ssm_qk_norm_rope_bwd(const void* q, const void* k, const void* dq_out, const void* dk_out, const float* q_weight,
                         const float* k_weight, const int32_t* positions, const float* inv_freq, int interleaved,
                         float eps, void* dq, void* dk, float* dq_weight, float* dk_weight, int64_t q_row,
                         int64_t k_row, int64_t rows, int64_t q_heads, int64_t k_heads, int64_t width, int64_t rotary,
                         int dtype, void* workspace, size_t workspace_bytes, void* stream) {
    const int rc = head_norm_check(rows, q_heads, k_heads, width, rotary, positions, inv_freq, q_row, k_row, eps,
                                   dtype);
    if (rc != SSM_OK) return rc;
    if (rows > 0 && ((q_heads > 0 && (!q || !dq_out || !dq)) || (k_heads > 0 && (!k || !dk_out || !dk))))
        return SSM_ERR_NULL_ARG;
    if (!all_aligned({q, k}, dtype == SSM_BF16 ? 2 : 4)) return SSM_ERR_MISALIGNED;
    if (!all_aligned({dq_out, dk_out, dq, dk}, 16)) return SSM_ERR_MISALIGNED;
    if (!all_aligned({q_weight, k_weight, dq_weight, dk_weight}, 4)) return SSM_ERR_MISALIGNED;
    if (!workspace || workspace_bytes < ssm_qk_norm_rope_bwd_workspace_bytes(rows, width)) return SSM_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return SSM_ERR_MISALIGNED;
    ssm::HeadNormArgs a{};
    a.x[0] = q; a.x[1] = k; a.x_row[0] = q_row; a.x_row[1] = k_row; a.heads[0] = q_heads; a.heads[1] = k_heads;
    a.weight[0] = q_weight; a.weight[1] = k_weight; a.positions = positions; a.inv_freq = inv_freq;
    a.rows = rows; a.width = (int32_t)width; a.rotary = (int32_t)rotary; a.interleaved = interleaved != 0;
    a.eps = eps; a.bf16 = dtype == SSM_BF16;
    a.dy[0] = dq_out; a.dy[1] = dk_out; a.dx[0] = dq; a.dx[1] = dk;
    a.dweight[0] = dq_weight; a.dweight[1] = dk_weight;
    a.groups = ssm::head_norm_groups(rows);
    a.group_rows = ssm::head_norm_group_rows(rows);
    a.part = static_cast<float*>(workspace);
    return status(ssm::launch_head_norm_bwd(a, static_cast<hipStream_t>(stream)));
}

// ------------------------------------------------------------ slots of a state pool

int ssm_state_slots_copy(void* pool, const int32_t* src, const int32_t* dst, int64_t layers, int64_t n_slots,
                         int64_t slot_bytes, int64_t n, void* stream) {
    if (layers < 0 || n_slots < 1 || slot_bytes < 0 || n < 0) return SSM_ERR_BAD_SHAPE;
    if (mul(mul(layers, n_slots), slot_bytes) < 0) return SSM_ERR_BAD_SHAPE;
    if (n > ssm::kMaxMoves || n_slots > 0x7fffffff) return SSM_ERR_UNSUPPORTED;
    if (n == 0 || layers == 0 || slot_bytes == 0) return SSM_OK;
    if (!pool || !src || !dst) return SSM_ERR_NULL_ARG;
    if (!all_aligned({src, dst}, 4)) return SSM_ERR_MISALIGNED;
    ssm::SlotsArgs a{pool, src, dst, layers, n_slots, slot_bytes, n};
    if (!ssm::slots_copy_fits(a)) return SSM_ERR_UNSUPPORTED;
    return status(ssm::launch_slots_copy(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
