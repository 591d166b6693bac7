// Internal declarations of linear attention with a decay for each head, of the
// head norm with rotary positions and of the moves between a state pool's
// slots, shared by their C-ABI layer, planner and kernel launchers.  Not part
// of the public interface (include/ssm.h is).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ssm.h"

namespace ssm {

// ---------------------------------------------------------------- linear attention

namespace linear {
constexpr int kMaxWidth = 256;                          // of a key or value row
constexpr int64_t kMaxRow = int64_t(1) << 22;           // elements between tokens: 64 of them within 32-bit byte offsets
constexpr int kColumns = 64;                            // columns of the state per workgroup
constexpr int kSegment = 64;                            // segments are multiples of the longest chunk
}  // namespace linear

// One run of the recurrence S <- e^g S + k v^T, o = q^T S over [B, L] rows of
// heads, forwards or backwards in time.  The gradients are runs of it too, with
// the tensors in other roles; "key" and "value" name the roles here.
struct LinearJob {
    const void* q;               // rows of `kd` elements, contracted with the state
    const void* k;               // rows of `kd`
    const void* v;               // rows of `vd`
    int64_t q_row, k_row, v_row; // elements between tokens
    int32_t q_per, k_per, v_per; // heads that share a row (1: a row for each head)
    int32_t kd, vd;
    void* out;                   // [B, L, H, vd]: dtype, or fp32 with out_f32; NULL: states only
    int32_t out_f32;
    int32_t reversed;            // from the last token to the first; token t then decays by g of t + 1
    int32_t zero_tail;           // rows of out behind a sequence's end are zeroed
    float inner, outer, fresh;   // factors of the products inside a chunk, of those with the state, of new terms in the state
    const float* state_in;       // the state entering each segment, or NULL (zeros)
    float* state_out;            // the state after the last segment, or NULL
    int32_t decay_out;           // state_out is decayed by the first token's g as well
    int64_t in_head, in_seg;     // elements between heads and segments of state_in (0 segments: the first only)
    int64_t out_head;            // between heads of state_out
    int32_t sk, sv;              // between the state's key rows and its value columns
    const void* dot_with;        // [B, L, .] rows of vd: dots[t] = sum of out * dot_with over this workgroup's columns
    int64_t dot_row;
    int32_t dot_per;
    float* dots;                 // [column tiles][B, H, L], or NULL
};

struct LinearRun {
    LinearJob job[3];
    int32_t jobs;
    const float* g;              // [B, L, H] fp32, or [H] with by_head
    int32_t by_head;
    const int32_t* seq_lens;
    int64_t B, L, H;
    int32_t segments;
    int64_t seg_tokens;          // a multiple of kSegment
    int32_t bf16;
    int32_t split;               // scores and state as three bf16 terms each
    float* seg_state[2];         // states-only runs: [B, H, segments][kd][vd] per job, not written for the last segment
    float* seg_decay[2];         // and [B, H, segments], log2 of the segment's decay
};

// How long sequences are cut; a pure function of the sizes.
struct LinearPlan {
    int segments;
    int64_t seg_tokens;
};
LinearPlan plan_linear_fwd(int64_t B, int64_t L, int64_t H, int64_t Dk, int64_t Dv, bool bf16);
LinearPlan plan_linear_bwd(int64_t B, int64_t L, int64_t H, int64_t Dk, int64_t Dv, bool bf16);

struct LinearArgs {
    const void* q;
    const void* k;
    const void* v;
    const float* g;
    int by_head;
    float scale;
    const float* h0;
    void* o;
    float* h_last;
    const int32_t* seq_lens;
    int64_t q_row, k_row, v_row;
    int64_t B, L, H, G, Dk, Dv;
    int bf16;
    LinearPlan plan;
    void* workspace;
};

struct LinearBwdArgs {
    LinearArgs f;                // the forward call's inputs; f.plan is the backward's
    const void* d_o;
    const float* dh_last;
    void* dq;
    void* dk;
    void* dv;
    float* dg;                   // [B, L, H], or [H] with by_head, or NULL
    float* dh0;
};

size_t linear_fwd_workspace_bytes(int64_t B, int64_t L, int64_t H, int64_t Dk, int64_t Dv, bool bf16);
size_t linear_bwd_workspace_bytes(int64_t B, int64_t L, int64_t H, int64_t G, int64_t Dk, int64_t Dv, bool bf16,
                                  bool by_head);
hipError_t launch_linear_fwd(const LinearArgs& a, hipStream_t stream);
hipError_t launch_linear_bwd(const LinearBwdArgs& a, hipStream_t stream);

// The kernels behind them (linear_attention.hip): the jobs of one run, all of
// one padded key width.
hipError_t launch_linear_run(const LinearRun& r, bool states_only, hipStream_t stream);

// seg_state[s] <- the state entering segment s: first (or zeros), then what
// the segments before s leave (after s where reversed); one or two of these.
struct LinearJoin {
    float* seg_state[2];         // [heads, segments][size]
    const float* seg_decay[2];   // [heads, segments]
    const float* first[2];       // [heads][size] or NULL
    int32_t reversed[2];
    int32_t n;
    int64_t heads;
    int32_t segments, size;      // size: elements of a state, a multiple of 4
};
hipError_t launch_linear_join(const LinearJoin& j, hipStream_t stream);

// dg from the tokens' dot products: dg_t = sum over s >= t of (a_s - b_s), from
// <D, S> of the states at each segment's right end on.
struct LinearDecayGrad {
    const float* dot_q;          // [tiles][B, H, L]: q . dq
    const float* dot_k;          // [tiles][B, H, L]: k . dk
    int32_t tiles;
    const float* S;              // states entering segments 1.. and after the last: [B, H, segments][size]
    const float* S_last;         // [B, H][size], after the last segment
    const float* D;              // states entering from the right: [B, H, segments][size]
    const float* D_last;         // dh_last, or NULL
    const float* g;
    int32_t by_head;
    const int32_t* seq_lens;
    int64_t B, L, H;
    int32_t segments, size;
    int64_t seg_tokens;
    float* dg;                   // [B, L, H] or NULL
    float* part;                 // [B * segments][H]: sums over the segment's tokens, or NULL
};
hipError_t launch_linear_decay_grad(const LinearDecayGrad& d, hipStream_t stream);

// out[row][g][c] = sum over the heads of group g of part[row][head][c], of both
struct LinearGroupSum {
    const float* part[2];        // [rows, H, width] fp32
    void* out[2];                // [rows, G, width] dtype
    int64_t rows, H, G;
    int32_t width;               // a multiple of 16
    int bf16;
};
hipError_t launch_linear_group_sum(const LinearGroupSum& s, hipStream_t stream);

struct LinearStepArgs {
    float* state;                // [slots, H, Dk, Dv]
    const void* q;
    const void* k;
    const void* v;
    const float* g;
    int by_head;
    float scale;
    const int32_t* slots;        // [B] or NULL: row b's state is b
    void* o;                     // [B, H, Dv]
    int64_t q_row, k_row, v_row;
    int64_t B, n_slots, H, G, Dk, Dv;
    int bf16;
};
hipError_t launch_linear_step(const LinearStepArgs& a, hipStream_t stream);

// ---------------------------------------------------------------- head norm and rotation

struct HeadNormArgs {
    const void* x[2];            // queries, keys: [rows, heads, width], heads dense within a row
    int64_t x_row[2];            // elements between rows
    int64_t heads[2];
    const float* weight[2];      // [width] or NULL (ones)
    const int32_t* positions;    // [rows]
    const float* inv_freq;       // [rotary / 2] radians a position
    int64_t rows;
    int32_t width, rotary;
    int32_t interleaved;
    float eps;
    int bf16;
    void* y[2];                  // forward: [rows, heads, width]
    const void* dy[2];           // backward: [rows, heads, width]
    void* dx[2];                 // [rows, heads, width]
    float* dweight[2];           // [width] or NULL
    int64_t groups, group_rows;  // backward: workgroups, and the rows that each sums its share of
    float* part;                 // [groups][2][width]
};
int64_t head_norm_group_rows(int64_t rows);
int64_t head_norm_groups(int64_t rows);
hipError_t launch_head_norm(const HeadNormArgs& a, hipStream_t stream);
hipError_t launch_head_norm_bwd(const HeadNormArgs& a, hipStream_t stream);

// ---------------------------------------------------------------- slots of a state pool

struct SlotsArgs {
    void* pool;                  // [layers, slots, slot_bytes]
    const int32_t* src;          // [n]
    const int32_t* dst;          // [n]
    int64_t layers, slots, slot_bytes, n;
};
constexpr int64_t kMaxMoves = 2048;
constexpr int kSlotsHeld = 16;   // units that a thread holds
// How a call is cut: a workgroup's range as wide as its registers hold for all
// entries, at most a unit a thread.
struct SlotsCut {
    int unit, threads, W;        // bytes; a workgroup's; units of a range, a power of two
    int64_t ranges;              // of a slot
};
SlotsCut slots_cut(const SlotsArgs& a);
bool slots_copy_fits(const SlotsArgs& a);   // one launch takes the ranges
hipError_t launch_slots_copy(const SlotsArgs& a, hipStream_t stream);

}  // namespace ssm
