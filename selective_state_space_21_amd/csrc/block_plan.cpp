// Host-side planning of the calls around the scan: how a gated scan walks its
// sequence, and the workspaces.  Plain host code: pure functions of the sizes
// (and the SSM_GATED_WALKERS override), no HIP call, so the C-ABI layer can
// run them while validating its arguments.
#include <stdint.h>
#include <stdlib.h>

#include "block_internal.h"

namespace ssm {

namespace {
int64_t al256(int64_t bytes) { return (bytes + 255) / 256 * 256; }
}  // namespace

// One workgroup runs on a CU at a time.  Alone on its strip it takes one round
// of the GPU per 256 strips, the last one partly empty; several to a strip
// fill the GPU evenly but clear the chain first and wait for each other, which
// makes a tile cost `handover` percent.  Measured, bf16, L = 2048, forward: 192
// strips 63.6 us alone, 58.3 with two walkers; 256: 67.8, 75.0; 320: 132, 116;
// 448: 128, 131; 32 strips of L = 131072: 3451, 531 with eight (sixteen: 532).
// Backward: 192 strips 117, 122.  With three tiles or fewer (17 us against 22
// for two at 125 strips, both mostly launch) the second launch costs more than
// it gives.
namespace {
constexpr int64_t kCUs = 256;
GatedPlan plan_gated(int64_t B, int64_t L, int64_t D, int tile, int handover) {
    GatedPlan pl{};
    pl.dblocks = (D + gated::kStrip - 1) / gated::kStrip;
    pl.strips = B * pl.dblocks;
    pl.tiles = (L + tile - 1) / tile;
    pl.walkers = 1;
    const int64_t rounds = (pl.strips + kCUs - 1) / kCUs;
    if (pl.tiles > 3 && pl.strips * handover < rounds * kCUs * 100) {
        const int64_t w = (kCUs + pl.strips - 1) / pl.strips;
        pl.walkers = w < 2 ? 2 : (w > gated::kMaxWalkers ? gated::kMaxWalkers : (int)w);
    }
    const char* env = getenv("SSM_GATED_WALKERS");
    if (env && atoi(env) > 0) pl.walkers = atoi(env) < gated::kMaxWalkers ? atoi(env) : gated::kMaxWalkers;
    const int64_t most = kMaxItems / (gated::kFwdThreads * pl.strips);      // what a launch holds
    if (pl.walkers > most) pl.walkers = most > 1 ? (int)most : 1;
    if (pl.walkers > pl.tiles) pl.walkers = pl.tiles > 1 ? (int)pl.tiles : 1;
    if (pl.walkers > 1)
        pl.chain_bytes = (size_t)(gated::chain_head(pl.strips) + pl.strips * gated::chain_slots(pl.tiles) * 12);
    return pl;
}
}  // namespace

GatedPlan plan_gated_fwd(int64_t B, int64_t L, int64_t D) { return plan_gated(B, L, D, gated::kFwdTile, 115); }
GatedPlan plan_gated_bwd(int64_t B, int64_t L, int64_t D) { return plan_gated(B, L, D, gated::kBwdTile, 140); }

namespace {
// byte sizes of the backward's workspace regions, in carve order
struct BwdRegions {
    int64_t part, chain, fwd_chain, ckpt;
};
BwdRegions bwd_regions(int64_t B, int64_t L, int64_t D, bool own_ckpt) {
    const GatedPlan pl = plan_gated_bwd(B, L, D);
    BwdRegions r;
    r.part = al256(B * pl.tiles * 3 * D * 4);
    r.chain = (int64_t)pl.chain_bytes;
    r.fwd_chain = own_ckpt ? (int64_t)plan_gated_fwd(B, L, D).chain_bytes : 0;
    r.ckpt = own_ckpt ? al256(B * gated_saved(L) * D * 4) : 0;
    return r;
}
}  // namespace

size_t gated_bwd_workspace_bytes(int64_t B, int64_t L, int64_t D, bool own_ckpt) {
    const BwdRegions r = bwd_regions(B, L, D, own_ckpt);
    return (size_t)(r.part + r.chain + r.fwd_chain + r.ckpt);
}

void gated_bwd_carve(GatedBwdArgs& a, void* ws) {
    const BwdRegions r = bwd_regions(a.f.B, a.f.L, a.f.D, a.own_ckpt);
    char* p = static_cast<char*>(ws);
    a.part = reinterpret_cast<float*>(p);
    p += r.part;
    a.chain = p;
    p += r.chain;
    a.f.chain = p;
    p += r.fwd_chain;
    if (a.own_ckpt) a.f.ckpt = reinterpret_cast<float*>(p);
}

int64_t norm_bwd_groups(int64_t rows) {
    return rows < kCUs ? rows : kCUs;       // one workgroup per CU
}

size_t norm_bwd_workspace_bytes(int64_t rows, int64_t D) {
    return (size_t)al256(2 * norm_bwd_groups(rows) * D * 4);
}

int64_t conv_bwd_blocks(int64_t L) { return (L + conv::kBlockTokens - 1) / conv::kBlockTokens; }

size_t conv_bwd_workspace_bytes(int64_t B, int64_t L, int64_t D, int64_t K) {
    return (size_t)al256(B * conv_bwd_blocks(L) * (K + 1) * D * 4);
}

}  // namespace ssm
