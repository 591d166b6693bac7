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

GatedPlan plan_gated(int64_t B, int64_t L, int64_t D) {
    GatedPlan pl{};
    pl.dblocks = (D + gated::kStrip - 1) / gated::kStrip;
    pl.strips = B * pl.dblocks;
    pl.tiles = (L + gated::kTile - 1) / gated::kTile;
    pl.walkers = 1;
    pl.chain_bytes = 0;
    return pl;
}

namespace {
// byte sizes of the backward's workspace regions, in carve order
struct BwdRegions {
    int64_t part, chain, fwd_chain, ckpt;
};
BwdRegions bwd_regions(const GatedPlan& pl, int64_t B, int64_t D, bool own_ckpt) {
    BwdRegions r;
    r.part = al256(B * pl.tiles * 3 * D * 4);
    r.chain = (int64_t)pl.chain_bytes;
    r.fwd_chain = own_ckpt ? (int64_t)pl.chain_bytes : 0;
    r.ckpt = own_ckpt ? al256(B * pl.tiles * D * 4) : 0;
    return r;
}
}  // namespace

size_t gated_bwd_workspace_bytes(int64_t B, int64_t L, int64_t D, bool own_ckpt) {
    const BwdRegions r = bwd_regions(plan_gated(B, L, D), B, D, own_ckpt);
    return (size_t)(r.part + r.chain + r.fwd_chain + r.ckpt);
}

void gated_bwd_carve(GatedBwdArgs& a, void* ws) {
    const BwdRegions r = bwd_regions(a.f.plan, a.f.B, a.f.D, a.own_ckpt);
    char* p = static_cast<char*>(ws);
    a.part = reinterpret_cast<float*>(p);
    p += r.part;
    a.chain = p;
    p += r.chain;
    a.f.chain = p;
    p += r.fwd_chain;
    if (a.own_ckpt) a.f.ckpt = reinterpret_cast<float*>(p);
}

int64_t norm_bwd_groups(int64_t rows, int64_t D) {
    (void)D;
    return rows < 512 ? rows : 512;
}

size_t norm_bwd_workspace_bytes(int64_t rows, int64_t D) {
    return (size_t)al256(2 * norm_bwd_groups(rows, D) * D * 4);
}

int64_t conv_bwd_blocks(int64_t L) { return (L + 255) / 256; }

size_t conv_bwd_workspace_bytes(int64_t B, int64_t L, int64_t D, int64_t K) {
    return (size_t)al256(B * conv_bwd_blocks(L) * (K + 1) * D * 4);
}

}  // namespace ssm
