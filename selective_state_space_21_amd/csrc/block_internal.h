// Internal declarations of the calls around the scan in a recurrent block
// (gated linear recurrence, layer norm, the causal conv's backward), shared
// by their C-ABI layer, planners and kernel launchers.  Not part of the
// public interface (include/ssm.h is).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ssm.h"

namespace ssm {

// A launch has at most 2^32 - 1 work-items along an axis (one of more runs
// with its size modulo 2^32, and reports nothing).
constexpr int64_t kMaxItems = 0xffffffff;

// launch(first, count) over `total` rows in slices of at most `most`.
template <typename Launch>
hipError_t in_slices(int64_t total, int64_t most, Launch&& launch) {
    for (int64_t first = 0; first < total; first += most) {
        const hipError_t e = launch(first, total - first < most ? total - first : most);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// p + n elements; NULL stays NULL
template <typename T> T* ahead(T* p, int64_t n) { return p ? p + n : p; }
inline const void* ahead(const void* p, int64_t n, int bytes) { return ahead(static_cast<const char*>(p), n * bytes); }
inline void* ahead(void* p, int64_t n, int bytes) { return ahead(static_cast<char*>(p), n * bytes); }

// ---------------------------------------------------------------- gated scan

// Tiling the planner shares with the kernels.
namespace gated {
constexpr int kFwdTile = 256;           // tokens per tile of the forward walk
constexpr int kBwdTile = SSM_GATED_TILE;   // of the backward walk, which starts from saved states
static_assert(kFwdTile % SSM_GATED_TILE == 0, "a forward tile holds whole saved states");
constexpr int kStrip = 64;              // channels per strip: one workgroup's width
constexpr int kFwdThreads = 1024;
constexpr int kBwdThreads = 1024;
// threads of a workgroup: a sequence of one short tile takes no more than its
// tokens need
constexpr int threads(int64_t L, int tile) { return L <= tile / 4 ? 256 : (L <= tile / 2 ? 512 : 1024); }
// Longest row: a tile's rows are addressed by 32-bit offsets below kNoChannel.
constexpr int64_t kMaxRow = int64_t(1) << 20;
static_assert(kFwdTile * kMaxRow * 4 < int64_t(1) << 31, "a tile's rows end below kNoChannel");
constexpr int kMaxWalkers = 64;         // workgroups per strip at most
constexpr int kBack = 8;                // tiles a walker looks back over for a known state
// What the walkers of a call share, in order: a counter per strip; a map (8
// bytes) per slot; a state (4 bytes) per slot.  A strip has a slot per channel
// and tile, and kBack - 1 empty tiles in front.
__host__ __device__ constexpr int64_t chain_head(int64_t strips) { return (strips * 4 + 255) / 256 * 256; }
__host__ __device__ constexpr int64_t chain_slots(int64_t tiles) { return (tiles + kBack - 1) * kStrip; }
}  // namespace gated

// How a call walks the sequence: every strip (64 channels of one batch row)
// is a chain of tiles, walked by `walkers` workgroups.
struct GatedPlan {
    int64_t strips;        // B * ceil(D / 64)
    int64_t dblocks;       // ceil(D / 64)
    int64_t tiles;         // ceil(L / tile)
    int walkers;           // 1: a workgroup walks its strip alone, nothing is shared
    size_t chain_bytes;    // what the walkers of a strip share (0 for one)
};

// A pure function of the sizes (and the SSM_GATED_WALKERS override).
GatedPlan plan_gated_fwd(int64_t B, int64_t L, int64_t D);
GatedPlan plan_gated_bwd(int64_t B, int64_t L, int64_t D);
inline int64_t gated_saved(int64_t L) { return (L + SSM_GATED_TILE - 1) / SSM_GATED_TILE; }

struct GatedArgs {
    const void* x;
    const void* gate_a;
    const void* gate_x;
    const float* A;
    const float* bias_a;
    const float* bias_x;
    const float* h0;
    void* y;               // NULL: states only
    float* h_last;
    float* ckpt;           // [B, saved, D] or NULL
    int64_t saved;         // ceil(L / SSM_GATED_TILE)
    const int32_t* seq_lens;
    int64_t B, L, D;
    int bf16;
    GatedPlan plan;
    void* chain;           // plan.chain_bytes, or NULL
    bool cleared;          // the caller has zeroed it
};

struct GatedBwdArgs {
    GatedArgs f;           // the forward call's inputs and plan; f.ckpt holds the saved states
    GatedPlan plan;
    const void* dy;
    const float* dh_last;
    void* dx;
    void* dgate_a;
    void* dgate_x;
    float* dA;
    float* dbias_a;
    float* dbias_x;
    float* dh0;
    bool own_ckpt;         // f.ckpt lies in the workspace and the call fills it first
    void* chain;           // the adjoint's, apart from the forward sweep's f.chain
    float* part;           // [B * plan.tiles][3][D]: a tile's sums for dA, dbias_a, dbias_x
};

size_t gated_bwd_workspace_bytes(int64_t B, int64_t L, int64_t D, bool own_ckpt);
void gated_bwd_carve(GatedBwdArgs& a, void* workspace);

// Zeroes what the walkers of a call share (bytes: a multiple of 16).
hipError_t launch_chain_clear(void* chain, size_t bytes, hipStream_t stream);
hipError_t launch_gated_fwd(const GatedArgs& a, hipStream_t stream);
hipError_t launch_gated_bwd(const GatedBwdArgs& a, hipStream_t stream);

struct GatedStepArgs {
    float* state;
    const void* x;
    const void* gate_a;
    const void* gate_x;
    const float* A;
    const float* bias_a;
    const float* bias_x;
    void* y;
    int64_t B, D;
    int bf16;
};

hipError_t launch_gated_step(const GatedStepArgs& a, hipStream_t stream);

// ---------------------------------------------------------------- layer norm

struct NormArgs {
    const void* x;             // [rows, D] dtype
    const float* residual;     // [rows, D] or NULL
    const float* weight;       // [D] or NULL (ones)
    const float* bias;         // [D] or NULL (zeros)
    float eps;
    void* y;
    float* residual_out;       // [rows, D] or NULL
    float* mean;               // [rows] or NULL
    float* rstd;               // [rows] or NULL
    int64_t rows, D;
    int bf16;
};

hipError_t launch_layer_norm(const NormArgs& a, hipStream_t stream);

struct NormBwdArgs {
    const void* x;             // [rows, D] x_bf16 ? bf16 : fp32
    const void* dy;            // [rows, D] dtype
    const float* mean;
    const float* rstd;
    const float* weight;       // or NULL
    const float* dresidual_out;   // [rows, D] or NULL
    void* dx;                  // [rows, D] dtype
    float* dresidual;          // [rows, D] or NULL
    float* dweight;            // [D] or NULL
    float* dbias;              // [D] or NULL
    int64_t rows, D;
    int x_bf16, bf16;
    int64_t groups;            // workgroups that each sum a share of the rows
    float* part;               // [2][groups][D]
};

// Workgroups of a backward call, each with a share of the rows and a row of
// partial sums: a pure function of their number.
int64_t norm_bwd_groups(int64_t rows);
size_t norm_bwd_workspace_bytes(int64_t rows, int64_t D);
hipError_t launch_layer_norm_bwd(const NormBwdArgs& a, hipStream_t stream);

// ---------------------------------------------------------------- conv1d backward

struct ConvBwdArgs {
    const void* x;             // [B, L, D]
    const float* weight;       // [D, K]
    const float* bias;         // [D] or NULL
    const float* state_in;     // [B, D, K-1] or NULL
    const void* du;            // [B, L, D]
    const float* dstate_out;   // [B, D, K-1] or NULL
    void* dx;                  // [B, L, D]
    float* dweight;            // [D, K]
    float* dbias;              // [D] or NULL
    float* dstate_in;          // [B, D, K-1] or NULL
    int64_t B, L, D, K;
    int silu;
    int bf16;
    int64_t blocks;            // token blocks per batch row
    float* part;               // [B * blocks][K + 1][D]
};

namespace conv {
constexpr int kBlockTokens = 256;       // tokens per workgroup of the backward
constexpr int64_t kMaxRow = int64_t(1) << 21;   // 40 rows within 32-bit offsets below kNoChannel
}
int64_t conv_bwd_blocks(int64_t L);
size_t conv_bwd_workspace_bytes(int64_t B, int64_t L, int64_t D, int64_t K);
hipError_t launch_conv1d_bwd(const ConvBwdArgs& a, hipStream_t stream);

// ---------------------------------------------------------------- column sums

// out[j][c] = (sum over n rows of part[row][j][c]) (/ divide[c] for j = 0,
// zero where divide[c] is zero), j < m, in a fixed order: the last step of the
// parameters' gradients.  part: [n][m][D].  out[j] NULL: skipped.  strided:
// out[0] is [D][m - 1] with the last sum in out[1] (the conv's weight layout).
struct ColumnSums {
    const float* part;
    int64_t n, D;
    int m;
    float* out[3];
    const float* divide;
    int strided;
};
hipError_t launch_column_sums(const ColumnSums& a, hipStream_t stream);

}  // namespace ssm
