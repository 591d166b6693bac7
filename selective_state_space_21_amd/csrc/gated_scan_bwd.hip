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
// q_t = a q_{t+1} + a dy_t, so a tile is folded and run as in the forward.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "block_internal.h"
#include "gated_math.h"
#include "gated_tile.h"
#include "lane_ops.h"

namespace ssm {
namespace {

using gated::kStrip;
using gated::kThreads;
using gated::kTile;
constexpr int kWaves = kThreads / 64;

template <typename T, int V>
__global__ __launch_bounds__(kThreads, 4) void gated_bwd(GatedBwdArgs q) {
    using S = TileShape<V>;
    using RowT = Row<T, V>;
    constexpr int R = S::kRun;
    const GatedArgs& p = q.f;
    __shared__ __attribute__((aligned(16))) float sA[2][S::kGroups][kStrip];   // decay before the group
    __shared__ __attribute__((aligned(16))) float sH[2][S::kGroups][kStrip];   // state entering it
    __shared__ __attribute__((aligned(16))) float sQ[2][S::kGroups][kStrip];   // adjoint entering it
    __shared__ float sSum[kWaves][3][kStrip];

    const int tid = threadIdx.x, wave = tid / 64;
    const int c = tid % S::kLanes, g = tid / S::kLanes;
    const int64_t strip = blockIdx.x;
    const int64_t b = strip / p.plan.dblocks;
    const int64_t ds = (strip % p.plan.dblocks) * kStrip;
    const int64_t d = ds + c * V;
    const bool in = d < p.D;
    const int64_t len = row_tokens(p, b);
    const int64_t last = len > 0 ? (len - 1) / kTile : 0;

    float A[V], ba[V], bx[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        A[v] = in ? p.A[d + v] : 0.0f;
        ba[v] = in && p.bias_a ? p.bias_a[d + v] : 0.0f;
        bx[v] = in && p.bias_x ? p.bias_x[d + v] : 0.0f;
    }
    const int64_t row0 = b * p.L * p.D + d;
    const T* x = static_cast<const T*>(p.x) + row0;
    const T* ga = static_cast<const T*>(p.gate_a) + row0;
    const T* gx = static_cast<const T*>(p.gate_x) + row0;
    const T* dy = static_cast<const T*>(q.dy) + row0;
    T* dx = static_cast<T*>(q.dx) + row0;
    T* dga = static_cast<T*>(q.dgate_a) + row0;
    T* dgx = static_cast<T*>(q.dgate_x) + row0;

    const int64_t dc = ds + tid;
    const bool keeper = tid < kStrip && dc < p.D;
    float carry = keeper && q.dh_last ? q.dh_last[b * p.D + dc] : 0.0f;

    for (int64_t tile = p.plan.tiles - 1; tile >= 0; --tile) {
        const int buf = tile & 1;
        const int64_t t0 = tile * kTile + g * R;
        const int64_t cell = b * p.plan.tiles + tile;
        if (tile > last) {                       // behind the row's end: zeros
            const float z[V] = {};
#pragma unroll
            for (int j = 0; j < R; ++j) {
                if (in && t0 + j < p.L) {
                    const int64_t o = (t0 + j) * p.D;
                    RowT::store(dx + o, z);
                    RowT::store(dga + o, z);
                    RowT::store(dgx + o, z);
                }
            }
            if (keeper)
                for (int k = 0; k < 3; ++k) q.part[(cell * 3 + k) * p.D + dc] = 0.0f;
            continue;
        }
        typename RowT::Raw rx[R], ra[R], rg[R], ry[R];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const bool ok = in && t0 + j < len;
            const int64_t o = (t0 + j) * p.D;
            rx[j] = ok ? RowT::load(x + o) : RowT::zero();
            ra[j] = ok ? RowT::load(ga + o) : RowT::zero();
            rg[j] = ok ? RowT::load(gx + o) : RowT::zero();
            ry[j] = ok ? RowT::load(dy + o) : RowT::zero();
        }
        const float first = keeper ? p.ckpt[cell * p.D + dc] : 0.0f;
        // forward pair and adjoint offset of the thread's run
        float a[R][V], w[R][V], r[R][V], i[R][V], e1[R][V], e2[R][V];
        float pa[V], ph[V], pq[V];
#pragma unroll
        for (int v = 0; v < V; ++v) { pa[v] = 1.0f; ph[v] = 0.0f; pq[v] = 0.0f; }
#pragma unroll
        for (int j = 0; j < R; ++j) {
            float xv[V], av[V], gv[V];
            RowT::unpack(rx[j], xv);
            RowT::unpack(ra[j], av);
            RowT::unpack(rg[j], gv);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                e1[j][v] = exp_neg(av[v] + ba[v]);
                e2[j][v] = exp_neg(gv[v] + bx[v]);
                r[j][v] = sigma_of(e1[j][v]);
                i[j][v] = sigma_of(e2[j][v]);
                const float la = A[v] * r[j][v];
                a[j][v] = fast_exp2(la * kLog2e);
                w[j][v] = __builtin_amdgcn_sqrtf(one_minus_sq(la, a[j][v]));
                float h = w[j][v] * (i[j][v] * xv[v]);
                if (t0 + j >= len) { a[j][v] = 1.0f; h = 0.0f; }
                pa[v] *= a[j][v];
                ph[v] = fmaf(a[j][v], ph[v], h);
            }
        }
#pragma unroll
        for (int j = R - 1; j >= 0; --j) {
            float yv[V];
            RowT::unpack(ry[j], yv);
#pragma unroll
            for (int v = 0; v < V; ++v) pq[v] = a[j][v] * (yv[v] + pq[v]);
        }
        lds_put<V>(&sA[buf][g][c * V], pa);
        lds_put<V>(&sH[buf][g][c * V], ph);
        lds_put<V>(&sQ[buf][g][c * V], pq);
        lds_barrier();
        if (tid < kStrip) {
            float H = first;
#pragma unroll 8
            for (int k = 0; k < S::kGroups; ++k) {
                const float kh = sH[buf][k][tid];
                sH[buf][k][tid] = H;
                H = fmaf(sA[buf][k][tid], H, kh);
            }
#pragma unroll 8
            for (int k = S::kGroups - 1; k >= 0; --k) {
                const float kq = sQ[buf][k][tid];
                sQ[buf][k][tid] = carry;
                carry = fmaf(sA[buf][k][tid], carry, kq);
            }
            if (keeper && tile == 0 && q.dh0) q.dh0[b * p.D + dc] = carry;
        }
        lds_barrier();
        float h[V], G[V], before[R][V], sum[3][V];
        lds_get<V>(&sH[buf][g][c * V], h);
        lds_get<V>(&sQ[buf][g][c * V], G);
#pragma unroll
        for (int v = 0; v < V; ++v) sum[0][v] = sum[1][v] = sum[2][v] = 0.0f;
#pragma unroll
        for (int j = 0; j < R; ++j) {
            float xv[V];
            RowT::unpack(rx[j], xv);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                before[j][v] = h[v];
                h[v] = fmaf(a[j][v], h[v], w[j][v] * (i[j][v] * xv[v]));
            }
        }
#pragma unroll
        for (int j = R - 1; j >= 0; --j) {
            const bool ok = in && t0 + j < len;
            float xv[V], yv[V], ox[V], oa[V], og[V];
            RowT::unpack(rx[j], xv);
            RowT::unpack(ry[j], yv);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float qn = G[v];                     // the adjoint from the right
                const float gh = yv[v] + qn;               // gradient of h_t
                G[v] = t0 + j < len ? a[j][v] * gh : qn;
                const float la = A[v] * r[j][v];
                const float ix = i[j][v] * xv[v];
                // la / w, zero where the decay is one
                const float law = w[j][v] > 0.0f ? la * fast_rcp(w[j][v]) : 0.0f;
                const float E = gh * (la * a[j][v] * before[j][v] - law * (a[j][v] * a[j][v]) * ix);
                ox[v] = gh * w[j][v] * i[j][v];
                og[v] = gh * w[j][v] * ix * (e2[j][v] * i[j][v]);     // 1 - i = e2 i
                oa[v] = E * (e1[j][v] * r[j][v]);                     // 1 - r = e1 r
                sum[0][v] += ok ? E : 0.0f;
                sum[1][v] += ok ? oa[v] : 0.0f;
                sum[2][v] += ok ? og[v] : 0.0f;
                if (!ok) ox[v] = oa[v] = og[v] = 0.0f;
            }
            if (in && t0 + j < p.L) {
                const int64_t o = (t0 + j) * p.D;
                RowT::store(dx + o, ox);
                RowT::store(dga + o, oa);
                RowT::store(dgx + o, og);
            }
        }
        // the tile's sums: over the wavefront's groups, then over wavefronts
#pragma unroll
        for (int k = 0; k < 3; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float s = sum[k][v];
                if constexpr (S::kLanes <= 16) s += __shfl_xor(s, 16, 64);
                if constexpr (S::kLanes <= 32) s += __shfl_xor(s, 32, 64);
                if (tid % 64 < S::kLanes) sSum[wave][k][c * V + v] = s;
            }
        lds_barrier();
        if (tid < 3 * kStrip) {
            const int k = tid / kStrip, ch = tid % kStrip;
            float s = 0.0f;
#pragma unroll
            for (int m = 0; m < kWaves; ++m) s += sSum[m][k][ch];
            if (ds + ch < p.D) q.part[(cell * 3 + k) * p.D + ds + ch] = s;
        }
    }
}

template <typename T>
hipError_t launch_bwd(const GatedBwdArgs& a, hipStream_t stream) {
    const unsigned grid = (unsigned)a.f.plan.strips;
    if (a.f.D % 4 == 0) gated_bwd<T, 4><<<grid, kThreads, 0, stream>>>(a);
    else gated_bwd<T, 1><<<grid, kThreads, 0, stream>>>(a);
    return hipGetLastError();
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
        if (a.own_ckpt) {
            GatedArgs sweep = f;
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
    s.n = f.B * f.plan.tiles;
    s.D = f.D;
    s.m = 3;
    s.out[0] = a.dA;
    s.out[1] = a.dbias_a;
    s.out[2] = a.dbias_x;
    s.divide = f.A;
    return launch_column_sums(s, stream);
}

}  // namespace ssm
