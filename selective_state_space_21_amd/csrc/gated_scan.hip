// The gated linear recurrence, forward and one-token form.  Per batch row b
// and channel d, over tokens t:
//   r = sigma(gate_a + bias_a),  i = sigma(gate_x + bias_x)
//   a = exp(A r),  b = sqrt(1 - a^2) i x,  h <- a h + b,  y = h
// (a diagonal recurrence with one state per channel, decay and input weighed
// by gates of the token; the square root keeps the state's variance at the
// input's).  Per element the call reads x and two gates and writes y: it is
// bound by those four streams.
//
// A map h -> a h + b composes: (a2, b2) o (a1, b1) = (a2 a1, a2 b1 + b2).  A
// workgroup takes a tile of 128 tokens x 64 channels: every thread forms its
// 16 elements' (a, b) in registers, folds its run of tokens to one pair, the
// first wavefront folds the pairs of the tile's token groups in order (one
// lane per channel), and every thread then runs its tokens from the state
// that enters its group.  Inputs are read once.
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

template <typename T, int V>
__global__ __launch_bounds__(kThreads, 4) void gated_fwd(GatedArgs p) {
    using S = TileShape<V>;
    using RowT = Row<T, V>;
    constexpr int R = S::kRun;
    // per token group and channel: the group's pair, then (exclusive) the pair
    // from the tile's start to the group; two copies, by tile parity
    __shared__ __attribute__((aligned(16))) float sA[2][S::kGroups][kStrip];
    __shared__ __attribute__((aligned(16))) float sH[2][S::kGroups][kStrip];
    __shared__ __attribute__((aligned(16))) float sC[2][kStrip];   // state entering the tile

    const int tid = threadIdx.x;
    const int c = tid % S::kLanes, g = tid / S::kLanes;
    const int64_t strip = blockIdx.x;
    const int64_t b = strip / p.plan.dblocks;
    const int64_t ds = (strip % p.plan.dblocks) * kStrip;
    const int64_t d = ds + c * V;
    const bool in = d < p.D;
    const int64_t len = row_tokens(p, b);
    const int64_t last = len > 0 ? (len - 1) / kTile : 0;      // the tile of the last token

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
    T* y = static_cast<T*>(p.y) + row0;

    const int64_t dc = ds + tid;                                // wavefront 0: its lane's channel
    const bool keeper = tid < kStrip && dc < p.D;
    float carry = keeper && p.h0 ? p.h0[b * p.D + dc] : 0.0f;

    for (int64_t tile = 0; tile <= last; ++tile) {
        const int buf = tile & 1;
        const int64_t t0 = tile * kTile + g * R;
        typename RowT::Raw rx[R], ra[R], rg[R];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const bool ok = in && t0 + j < len;
            const int64_t o = (t0 + j) * p.D;
            rx[j] = ok ? RowT::load(x + o) : RowT::zero();
            ra[j] = ok ? RowT::load(ga + o) : RowT::zero();
            rg[j] = ok ? RowT::load(gx + o) : RowT::zero();
        }
        float a[R][V], h[R][V], pa[V], ph[V];
#pragma unroll
        for (int v = 0; v < V; ++v) { pa[v] = 1.0f; ph[v] = 0.0f; }
#pragma unroll
        for (int j = 0; j < R; ++j) {
            float xv[V], av[V], gv[V];
            RowT::unpack(rx[j], xv);
            RowT::unpack(ra[j], av);
            RowT::unpack(rg[j], gv);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                gated_token(xv[v], av[v], gv[v], A[v], ba[v], bx[v], a[j][v], h[j][v]);
                if (t0 + j >= len) { a[j][v] = 1.0f; h[j][v] = 0.0f; }   // no token: the state stays
                pa[v] *= a[j][v];
                ph[v] = fmaf(a[j][v], ph[v], h[j][v]);
            }
        }
        lds_put<V>(&sA[buf][g][c * V], pa);
        lds_put<V>(&sH[buf][g][c * V], ph);
        lds_barrier();
        if (tid < kStrip) {
            float P = 1.0f, H = 0.0f;
#pragma unroll 8
            for (int k = 0; k < S::kGroups; ++k) {
                const float ka = sA[buf][k][tid], kh = sH[buf][k][tid];
                sA[buf][k][tid] = P;
                sH[buf][k][tid] = H;
                H = fmaf(ka, H, kh);
                P *= ka;
            }
            if (keeper && p.ckpt) p.ckpt[(b * p.plan.tiles + tile) * p.D + dc] = carry;
            sC[buf][tid] = carry;
            carry = fmaf(P, carry, H);
            if (keeper && tile == last && p.h_last) p.h_last[b * p.D + dc] = carry;
        }
        lds_barrier();
        if (!p.y) continue;
        float s[V], P[V], H[V];
        lds_get<V>(&sC[buf][c * V], s);
        lds_get<V>(&sA[buf][g][c * V], P);
        lds_get<V>(&sH[buf][g][c * V], H);
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = fmaf(P[v], s[v], H[v]);
#pragma unroll
        for (int j = 0; j < R; ++j) {
#pragma unroll
            for (int v = 0; v < V; ++v) s[v] = fmaf(a[j][v], s[v], h[j][v]);
            if (in && t0 + j < len) RowT::store(y + (t0 + j) * p.D, s);
        }
    }
}

// no tokens: the state passes through (zeros without one)
__global__ __launch_bounds__(256) void gated_pass(const float* h0, float* h_last, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) h_last[i] = h0 ? h0[i] : 0.0f;
}

// One token per sequence against a resident state: V channels per thread.
template <typename T, int V>
__global__ __launch_bounds__(256) void gated_step(GatedStepArgs p) {
    using RowT = Row<T, V>;
    using RowS = Row<float, V>;
    const int64_t vecs = p.D / V;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= p.B * vecs) return;
    const int64_t d = (i % vecs) * V, o = i * V;
    float x[V], ga[V], gx[V], h[V];
    RowT::unpack(RowT::load(static_cast<const T*>(p.x) + o), x);
    RowT::unpack(RowT::load(static_cast<const T*>(p.gate_a) + o), ga);
    RowT::unpack(RowT::load(static_cast<const T*>(p.gate_x) + o), gx);
    RowS::unpack(RowS::load(p.state + o), h);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float a, b;
        gated_token(x[v], ga[v], gx[v], p.A[d + v], p.bias_a ? p.bias_a[d + v] : 0.0f,
                    p.bias_x ? p.bias_x[d + v] : 0.0f, a, b);
        h[v] = fmaf(a, h[v], b);
    }
    RowS::store(p.state + o, h);
    RowT::store(static_cast<T*>(p.y) + o, h);
}

template <typename T>
hipError_t launch_step(const GatedStepArgs& a, hipStream_t stream) {
    const int64_t n = a.B * (a.D % 4 == 0 ? a.D / 4 : a.D);
    const unsigned grid = (unsigned)((n + 255) / 256);
    if (a.D % 4 == 0) gated_step<T, 4><<<grid, 256, 0, stream>>>(a);
    else gated_step<T, 1><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_fwd(const GatedArgs& a, hipStream_t stream) {
    const unsigned grid = (unsigned)a.plan.strips;
    if (a.D % 4 == 0) gated_fwd<T, 4><<<grid, kThreads, 0, stream>>>(a);
    else gated_fwd<T, 1><<<grid, kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gated_fwd(const GatedArgs& a, hipStream_t stream) {
    if (a.L == 0) {
        const int64_t n = a.B * a.D;
        if (a.h_last) gated_pass<<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(a.h0, a.h_last, n);
        return hipGetLastError();
    }
    return a.bf16 ? launch_fwd<uint16_t>(a, stream) : launch_fwd<float>(a, stream);
}

hipError_t launch_gated_step(const GatedStepArgs& a, hipStream_t stream) {
    return a.bf16 ? launch_step<uint16_t>(a, stream) : launch_step<float>(a, stream);
}

}  // namespace ssm
