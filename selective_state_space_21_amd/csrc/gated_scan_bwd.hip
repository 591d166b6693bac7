// Backward pass of the gated linear recurrence.  With q the gradient that
// reaches the state before a token (q after the last one is dh_last, before
// the first one dh0), from the right:
//   G = dy_t + q_{t+1}            gradient of h_t
//   q_t = a G
//   dx = G w i,   dgate_x = G w x i (1 - i),          w = sqrt(1 - a^2)
//   E  = (log a) dL/d(log a) = G (la a h_{t-1} - (la / w) a^2 i x)
//   dgate_a = E (1 - r),   dA = (sum E) / A
// E is formed rather than dL/d(log a), whose second term grows like 1/w as a
// nears 1; la / w goes to zero there.  The tile's states come again from the
// state saved before its first token.  Per element the call reads x, two
// gates and dy and writes three gradients: it is bound by those seven streams.
//
// The adjoint is the same kind of recurrence as the states, right to left:
// q_t = a q_{t+1} + a dy_t, so a tile is folded and run as in the forward.  Its
// map needs gate_a and dy alone: it is formed and put up first, and the state
// before it awaited while the others form the rest.
//
// Measured, from saved states: B=1 L=32768 D=2048 fp32 (1.9 GB) 377 us, 5.0
// TB/s, the copy rate; bf16 285 us, 3.3 TB/s; B=8 L=2048 D=1536 bf16 (352 MB)
// 117 us, 3.0 TB/s.  In bf16 the vector instructions bound it: 77 an element,
// eight transcendental, about 60 us of the 117 on the 192 CUs that its 192
// strips fill.  128 registers (16 wavefronts a CU) are what a tile may hold;
// where the values for the gradients are kept over the barriers instead of
// formed again, the registers that spill cost more (bf16 324 -> 317 us long,
// but 122 -> 129 short).  512 threads and tiles of 64 tokens, two workgroups to
// a CU: 314 us long, 132 short (324 and 122 then); looking back over 16 tiles
// with those: 376.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <type_traits>

#include "block_internal.h"
#include "gated_math.h"
#include "gated_tile.h"
#include "lane_ops.h"

namespace ssm {
namespace {

using gated::kStrip;

// THREADS: 1024, or as many as the tokens of a sequence of one short tile need
template <typename T, int V, bool CHAIN, int THREADS>
__global__ __launch_bounds__(THREADS, 4) void gated_bwd(GatedBwdArgs q) {
    constexpr int kTile = gated::kBwdTile * THREADS / gated::kBwdThreads, kWaves = THREADS / 64;
    using S = TileShape<V, kTile, THREADS>;
    using RowT = Row<T, V>;
    constexpr int R = S::kRun;
    const GatedArgs& p = q.f;
    // per wavefront and channel, two copies by turns: the pair of its tokens,
    // then the pair from the tile's start to it (sA, sH); the adjoint's
    // offset, then its pair from the tile's end to it (sP, sQ)
    __shared__ __attribute__((aligned(16))) float sA[2][S::kWaves][kStrip];
    __shared__ __attribute__((aligned(16))) float sH[2][S::kWaves][kStrip];
    __shared__ __attribute__((aligned(16))) float sQ[2][S::kWaves][kStrip];
    __shared__ __attribute__((aligned(16))) float sP[2][S::kWaves][kStrip];
    __shared__ __attribute__((aligned(16))) float sS[2][kStrip];   // state entering the tile
    __shared__ __attribute__((aligned(16))) float sC[2][kStrip];   // adjoint entering it
    __shared__ float sSum[2][kWaves][3][kStrip];                   // wavefronts' sums of a tile
    __shared__ int sNext[2];

    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / 64), lane = tid % 64;
    const int c = tid % S::kLanes, g = tid / S::kLanes;
    const int64_t strip = CHAIN ? blockIdx.x % (unsigned)q.plan.strips : blockIdx.x;
    const int64_t b = strip / q.plan.dblocks;
    const int64_t ds = (strip % q.plan.dblocks) * kStrip;
    const int left = (int)(p.D - ds < kStrip ? p.D - ds : kStrip);  // the strip's channels
    const bool in = c * V < left;
    const int64_t len = row_tokens(p, b);
    const int last = len > 0 ? (int)((len - 1) / kTile) : 0;       // the walk starts there

    GatedChannel ch[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int64_t d = ds + c * V + v;
        ch[v] = gated_channel(in ? p.A[d] : 0.0f, in && p.bias_a ? p.bias_a[d] : 0.0f,
                              in && p.bias_x ? p.bias_x[d] : 0.0f);
    }
    const uint32_t pitch = (uint32_t)(p.D * sizeof(T));
    const uint32_t off = in ? (uint32_t)(g * R) * pitch + (uint32_t)((ds + c * V) * sizeof(T)) : kNoChannel;
    const bool keeper = lane < left;             // a folding lane has channel ds + lane
    // a strip's row of a [rows][D] fp32 tensor; the lane is added last, to a
    // uniform address
    auto row = [&](auto* base, int64_t r) { return base + (r * p.D + ds); };
    const uint32_t ul = lane;

    // tiles behind the row's end: zeros
    for (int64_t t = last + 1 + (CHAIN ? blockIdx.x / (unsigned)q.plan.strips : 0); t < q.plan.tiles;
         t += q.plan.walkers) {
        const __amdgpu_buffer_rsrc_t ox = tile_rows<T>(q.dx, p, b, t * kTile, p.L, kTile);
        const __amdgpu_buffer_rsrc_t oa = tile_rows<T>(q.dgate_a, p, b, t * kTile, p.L, kTile);
        const __amdgpu_buffer_rsrc_t og = tile_rows<T>(q.dgate_x, p, b, t * kTile, p.L, kTile);
        const float z[V] = {};
#pragma unroll
        for (int j = 0; j < R; ++j) {
            RowT::store(ox, off + j * pitch, z);
            RowT::store(oa, off + j * pitch, z);
            RowT::store(og, off + j * pitch, z);
        }
        if (wave < 3 && keeper) row(q.part, (b * q.plan.tiles + t) * 3 + wave)[ul] = 0.0f;
    }

    // wavefront 0 folds the states; wavefront kKeep folds the adjoint, hands
    // it on and waits for it
    constexpr int kKeep = kWaves - 1;
    const bool drawer = tid == kKeep * 64;
    float carry = wave == kKeep && keeper && q.dh_last ? row(q.dh_last, b)[ul] : 0.0f;
    typename RowT::Raw rx[R], ra[R], rg[R], ry[R], nx[R], na[R], ng[R], ny[R];
    float first = 0.0f;                          // wavefront 0: the saved state before the tile
    auto load = [&](int tile) {
        const int64_t t = (int64_t)tile * kTile;
        const int64_t end = tile < 0 ? t : len;
        const __amdgpu_buffer_rsrc_t bx = tile_rows<T>(p.x, p, b, t, end, kTile);
        const __amdgpu_buffer_rsrc_t ba = tile_rows<T>(p.gate_a, p, b, t, end, kTile);
        const __amdgpu_buffer_rsrc_t bg = tile_rows<T>(p.gate_x, p, b, t, end, kTile);
        const __amdgpu_buffer_rsrc_t by = tile_rows<T>(q.dy, p, b, t, end, kTile);
#pragma unroll
        for (int j = 0; j < R; ++j) {
            na[j] = RowT::load(ba, off + j * pitch);
            ny[j] = RowT::load(by, off + j * pitch);
        }
#pragma unroll
        for (int j = 0; j < R; ++j) {
            ng[j] = RowT::load(bg, off + j * pitch);
            nx[j] = RowT::load(bx, off + j * pitch);
        }
        if (wave == 0 && keeper && tile >= 0) first = row(p.ckpt, b * p.saved + tile)[ul];
    };
    auto advance = [&]() {
#pragma unroll
        for (int j = 0; j < R; ++j) {
            rx[j] = nx[j];
            ra[j] = na[j];
            rg[j] = ng[j];
            ry[j] = ny[j];
        }
    };
    // the sums of the tile before: wavefronts' shares in order
    auto put_sums = [&](int buf, int tile) {
        if (wave < 3 && keeper) {
            float t = 0.0f;
#pragma unroll
            for (int m = 0; m < kWaves; ++m) t += sSum[buf][m][wave][lane];
            row(q.part, (b * q.plan.tiles + tile) * 3 + wave)[ul] = t;
        }
    };

    const Chain chain = CHAIN ? chain_of(q.chain, q.plan, strip) : Chain{};
    int tile = last, drawn = last - 1;           // drawn: the tile after this one
    if (CHAIN) {
        if (drawer) {
            sNext[1] = chain_draw(chain);
            drawn = chain_draw(chain);
        }
        lds_barrier();
        tile = last - __builtin_amdgcn_readfirstlane(sNext[1]);
        drawn = last - drawn;
    }
    int before = -1;                             // the tile whose sums are still in LDS
    if (tile >= 0) load(tile);
    int buf = 0;
    for (; tile >= 0; buf ^= 1) {
        advance();
        const int64_t t0 = (int64_t)tile * kTile;
        // what the adjoint's recurrence needs comes first, so that its map is
        // up, and the state before it on its way, while the rest is computed
        float a[R][V], y[R][V], cr[R][V], pa[V], pq[V];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            float av[V];
            RowT::unpack(ra[j], av);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float e = exp_neg_finite(av[v], ch[v].ba), r = sigma_of(e);
                y[j][v] = ch[v].A2 * r;
                a[j][v] = fast_exp2(y[j][v]);
                cr[j][v] = e * r;                // 1 - r
            }
        }
        const bool ragged = t0 + kTile > len;    // tokens that do not exist: the adjoint passes
        if (ragged) {
#pragma unroll
            for (int j = 0; j < R; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (t0 + g * R + j >= len) {
                        a[j][v] = 1.0f;
                        y[j][v] = 0.0f;
                    }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            pa[v] = 1.0f;
            pq[v] = 0.0f;
        }
#pragma unroll
        for (int j = R - 1; j >= 0; --j) {
            float dy[V];
            RowT::unpack(ry[j], dy);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                pa[v] *= a[j][v];
                pq[v] = a[j][v] * (dy[v] + pq[v]);
            }
        }
        // a wavefront's two runs to one map; the lower one starts behind the
        // upper (op, oq), and in the states the upper behind the lower (op, oh)
        float op[V], oq[V], oh[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            op[v] = 1.0f;
            oq[v] = 0.0f;
            if constexpr (S::kPair) {
                op[v] = __shfl_xor(pa[v], 32, 64);
                oq[v] = __shfl_xor(pq[v], 32, 64);
                pq[v] = fmaf(pa[v], oq[v], pq[v]);   // right in the lower half, which stores it
                pa[v] *= op[v];
            }
        }
        if (lane < S::kLanes) {
            lds_put<V>(&sA[buf][wave][c * V], pa);
            lds_put<V>(&sQ[buf][wave][c * V], pq);
        }
        if (drawer) sNext[buf] = CHAIN ? drawn : tile - 1;
        lds_barrier();
        const int next = __builtin_amdgcn_readfirstlane(sNext[buf]);
        if (before >= 0) put_sums(buf ^ 1, before);
        const int pos = last - tile;             // tiles walked before this one
        float P = 1.0f, Q = 0.0f;
        if (wave == kKeep) {
#pragma unroll
            for (int k = S::kWaves - 1; k >= 0; --k) {
                const float ka = sA[buf][k][lane], kq = sQ[buf][k][lane];
                sP[buf][k][lane] = P;
                sQ[buf][k][lane] = Q;
                Q = fmaf(ka, Q, kq);
                P *= ka;
            }
            if (CHAIN && pos > 0) {
                if (tile > 0) chain_put_map(chain, pos, ul, P, Q);
                carry = chain_state_before(chain, pos, ul);
            }
            sC[buf][lane] = carry;
            carry = fmaf(P, carry, Q) + 0.0f;    // -0 is 0
            if (CHAIN && tile > 0) chain_put_state(chain, pos, ul, carry);
            if (keeper && tile == 0 && q.dh0) row(q.dh0, b)[ul] = carry;
        }
        // the weighted inputs, for the state's map; what else the gradients
        // need of them is formed again behind the barriers, which costs less
        // than the registers to keep it in
        float ph[V], e2[R][V];
#pragma unroll
        for (int v = 0; v < V; ++v) ph[v] = 0.0f;
#pragma unroll
        for (int j = 0; j < R; ++j) {
            float xv[V], gv[V];
            RowT::unpack(rx[j], xv);
            RowT::unpack(rg[j], gv);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                e2[j][v] = exp_neg_finite(gv[v], ch[v].bx);
                const float i = sigma_of(e2[j][v]);
                const float w = __builtin_amdgcn_sqrtf(one_minus_sq(y[j][v], a[j][v]));
                ph[v] = fmaf(a[j][v], ph[v], w * (i * xv[v]));
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            oh[v] = 0.0f;
            if constexpr (S::kPair) {
                oh[v] = __shfl_xor(ph[v], 32, 64);
                ph[v] = fmaf(op[v], ph[v], oh[v]);
            }
        }
        if (lane < S::kLanes) lds_put<V>(&sH[buf][wave][c * V], ph);
        lds_barrier();
        if (wave == 0) {
            float Ps = 1.0f, H = 0.0f;
#pragma unroll
            for (int k = 0; k < S::kWaves; ++k) {
                const float ka = sA[buf][k][lane], kh = sH[buf][k][lane];
                sA[buf][k][lane] = Ps;
                sH[buf][k][lane] = H;
                H = fmaf(ka, H, kh);
                Ps *= ka;
            }
            sS[buf][lane] = first;
        }
        load(next);                              // after the chain: loads return in order
        if (CHAIN && drawer) drawn = last - chain_draw(chain);
        lds_barrier();
        const bool upper = lane >= 32;
        float s[V], sp[V], sh[V];                // the state before the thread's run
        lds_get<V>(&sS[buf][c * V], s);
        lds_get<V>(&sA[buf][wave][c * V], sp);
        lds_get<V>(&sH[buf][wave][c * V], sh);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            s[v] = fmaf(sp[v], s[v], sh[v]);
            if (S::kPair && upper) s[v] = fmaf(op[v], s[v], oh[v]);
        }
        float G[V], gp[V], gq[V], sum[3][V];
        lds_get<V>(&sC[buf][c * V], G);
        lds_get<V>(&sP[buf][wave][c * V], gp);
        lds_get<V>(&sQ[buf][wave][c * V], gq);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            G[v] = fmaf(gp[v], G[v], gq[v]);
            if (S::kPair && !upper) G[v] = fmaf(op[v], G[v], oq[v]);
            sum[0][v] = sum[1][v] = sum[2][v] = 0.0f;
        }
        // E = G ef, dgate_a = E (1 - r), dx = G wi, dgate_x = G hc; ef needs the
        // state before the token: left to right
        float ef[R][V], wi[R][V], hc[R][V];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            float xv[V];
            RowT::unpack(rx[j], xv);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                asm volatile("" : "+v"(y[j][v]), "+v"(e2[j][v]));   // not the values from before the barriers
                const float e = e2[j][v], i = sigma_of(e);
                const float w2 = one_minus_sq(y[j][v], a[j][v]);
                // 1 / w; where w^2 leaves fp32's range, so do its terms (a positive A
                // makes w^2 negative: NaN)
                const float rw = fabsf(w2) > 1e-37f ? __builtin_amdgcn_rsqf(w2) : 0.0f;
                const float w = w2 * rw, ix = i * xv[v], h = w * ix;
                // la a h_{t-1} - (la / w) a^2 i x
                ef[j][v] = (y[j][v] * a[j][v]) * kLn2 * fmaf(-(a[j][v] * ix), rw, s[v]);
                wi[j][v] = w * i;
                hc[j][v] = h * (e * i);              // 1 - i = e i
                s[v] = fmaf(a[j][v], s[v], h);
            }
        }
        const __amdgpu_buffer_rsrc_t ox = tile_rows<T>(q.dx, p, b, t0, p.L, kTile);
        const __amdgpu_buffer_rsrc_t oa = tile_rows<T>(q.dgate_a, p, b, t0, p.L, kTile);
        const __amdgpu_buffer_rsrc_t og = tile_rows<T>(q.dgate_x, p, b, t0, p.L, kTile);
        auto gradients = [&](auto partial) {
            const int own = decltype(partial)::value ? (int)(len - t0) - g * R : R;   // tokens that the run has
#pragma unroll
            for (int j = R - 1; j >= 0; --j) {
                float gx[V], ga[V], gg[V], dy[V];
                RowT::unpack(ry[j], dy);
                const bool none = decltype(partial)::value && j >= own;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float gh = dy[v] + G[v];
                    G[v] = a[j][v] * gh;
                    const float E = none ? 0.0f : gh * ef[j][v];
                    gx[v] = none ? 0.0f : gh * wi[j][v];
                    ga[v] = none ? 0.0f : E * cr[j][v];
                    gg[v] = none ? 0.0f : gh * hc[j][v];
                    sum[0][v] += E;
                    sum[1][v] += ga[v];
                    sum[2][v] += gg[v];
                }
                RowT::store(ox, off + j * pitch, gx);
                RowT::store(oa, off + j * pitch, ga);
                RowT::store(og, off + j * pitch, gg);
            }
        };
        // a token that does not exist has no gradient whatever passes it: the
        // adjoint or the state there may be infinite, and a product with its
        // zero weights NaN
        if (ragged) gradients(std::true_type{});
        else gradients(std::false_type{});
#pragma unroll
        for (int k = 0; k < 3; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float t = sum[k][v];
                if constexpr (S::kPair) t += __shfl_xor(t, 32, 64);
                if (lane < S::kLanes) sSum[buf][wave][k][c * V + v] = t;
            }
        before = tile;
        tile = next;
    }
    lds_barrier();
    if (before >= 0) put_sums(buf ^ 1, before);
}

template <typename T, int V>
hipError_t launch_bwd_v(const GatedBwdArgs& a, hipStream_t stream) {
    if (a.plan.walkers > 1) {
        gated_bwd<T, V, true, 1024><<<(unsigned)(a.plan.strips * a.plan.walkers), 1024, 0, stream>>>(a);
        return hipGetLastError();
    }
    // a workgroup to a strip: whole batch rows, as many as a launch holds
    const GatedArgs& f = a.f;
    const int threads = gated::threads(f.L, gated::kBwdTile);
    return in_slices(f.B, kMaxItems / (threads * a.plan.dblocks), [&](int64_t b, int64_t n) {
        GatedBwdArgs s = a;
        s.f.x = ahead(f.x, b * f.L * f.D, sizeof(T));
        s.f.gate_a = ahead(f.gate_a, b * f.L * f.D, sizeof(T));
        s.f.gate_x = ahead(f.gate_x, b * f.L * f.D, sizeof(T));
        s.f.ckpt = ahead(f.ckpt, b * f.saved * f.D);
        s.f.seq_lens = ahead(f.seq_lens, b);
        s.f.B = n;
        s.dy = ahead(a.dy, b * f.L * f.D, sizeof(T));
        s.dx = ahead(a.dx, b * f.L * f.D, sizeof(T));
        s.dgate_a = ahead(a.dgate_a, b * f.L * f.D, sizeof(T));
        s.dgate_x = ahead(a.dgate_x, b * f.L * f.D, sizeof(T));
        s.dh_last = ahead(a.dh_last, b * f.D);
        s.dh0 = ahead(a.dh0, b * f.D);
        s.part = ahead(a.part, b * a.plan.tiles * 3 * f.D);
        s.plan.strips = n * a.plan.dblocks;
        const unsigned strips = (unsigned)s.plan.strips;
        if (threads == 256) gated_bwd<T, V, false, 256><<<strips, 256, 0, stream>>>(s);
        else if (threads == 512) gated_bwd<T, V, false, 512><<<strips, 512, 0, stream>>>(s);
        else gated_bwd<T, V, false, 1024><<<strips, 1024, 0, stream>>>(s);
        return hipGetLastError();
    });
}

template <typename T>
hipError_t launch_bwd(const GatedBwdArgs& a, hipStream_t stream) {
    return a.f.D % 2 == 0 ? launch_bwd_v<T, 2>(a, stream) : launch_bwd_v<T, 1>(a, stream);
}

__global__ __launch_bounds__(256) void gated_bwd_pass(const float* dh_last, float* dh0, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) dh0[i] = dh_last ? dh_last[i] : 0.0f;
}

}  // namespace

hipError_t launch_gated_bwd(const GatedBwdArgs& a, hipStream_t stream) {
    const GatedArgs& f = a.f;
    hipError_t e = hipSuccess;
    if (f.L == 0) {
        const int64_t n = f.B * f.D;
        if (a.dh0) gated_bwd_pass<<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(a.dh_last, a.dh0, n);
        e = hipGetLastError();
    } else {
        // the adjoint's chain and behind it the forward sweep's, at once
        e = launch_chain_clear(a.chain, a.plan.chain_bytes + (a.own_ckpt ? f.plan.chain_bytes : 0), stream);
        if (e != hipSuccess) return e;
        if (a.own_ckpt) {
            GatedArgs sweep = f;
            sweep.cleared = true;
            sweep.y = nullptr;
            sweep.h_last = nullptr;
            e = launch_gated_fwd(sweep, stream);
            if (e != hipSuccess) return e;
        }
        e = f.bf16 ? launch_bwd<uint16_t>(a, stream) : launch_bwd<float>(a, stream);
    }
    if (e != hipSuccess) return e;
    ColumnSums s{};
    s.part = a.part;
    s.n = f.B * a.plan.tiles;
    s.D = f.D;
    s.m = 3;
    s.out[0] = a.dA;
    s.out[1] = a.dbias_a;
    s.out[2] = a.dbias_x;
    s.divide = f.A;
    return launch_column_sums(s, stream);
}

}  // namespace ssm
