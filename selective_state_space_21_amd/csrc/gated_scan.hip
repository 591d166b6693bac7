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
// workgroup takes a tile of 256 tokens x 64 channels: every thread forms its
// 16 elements' (a, b) in registers, folds its run of tokens to one pair, the
// first wavefront folds the pairs of the wavefronts' tokens in order and
// learns the state that enters the tile, and every thread then runs its tokens
// from the state that enters its run.  Inputs are read once; the next tile's
// are under way from the moment this one's are folded.
//
// Measured: B=1 L=131072 D=2048 fp32 (4.3 GB) 771 us, 5.6 TB/s, above what a
// copy of as many bytes reaches (5.0); bf16 528 us, 4.1 TB/s; B=8 L=2048 D=1536
// bf16 (201 MB) 58.5 us, 3.4 TB/s, 18 above the copy.  Of those 18 the
// arithmetic (35 vector instructions an element, six of them transcendental)
// accounts for 6: without it the call takes 52.9 us; the clearing launch and
// the hand-over for 6 more: 47.0 without these too, with one workgroup to a
// strip; the last 7 are the phases of one workgroup a CU between its barriers,
// on 192 CUs.  Tried at the bf16 shapes above (long, short) and not kept: 512 threads and tiles of
// 128 tokens, two workgroups to a CU, 547 and 58.7 us; strips of 32 channels,
// whose bf16 rows are half a cache line, 795 and 75.8; the next tile's loads a
// whole tile ahead 585 and 63.3; cached instead of nontemporal accesses 61.2 at
// the short shape and 841 us at the long one in fp32.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "block_internal.h"
#include "gated_math.h"
#include "gated_tile.h"
#include "lane_ops.h"

namespace ssm {
namespace {

using gated::kStrip;
// THREADS: 1024, or as many as the tokens of a sequence of one short tile need
template <typename T, int V, bool CHAIN, int THREADS>
__global__ __launch_bounds__(THREADS, 4) void gated_fwd(GatedArgs p) {
    constexpr int kTile = gated::kFwdTile * THREADS / gated::kFwdThreads;
    constexpr int kSaved = kTile > SSM_GATED_TILE ? kTile / SSM_GATED_TILE : 1;   // states saved per tile
    using S = TileShape<V, kTile, THREADS>;
    using RowT = Row<T, V>;
    constexpr int R = S::kRun;
    // per wavefront and channel: the pair of its tokens, then (exclusive) the
    // pair from the tile's start to it; two copies, by turns
    __shared__ __attribute__((aligned(16))) float sA[2][S::kWaves][kStrip];
    __shared__ __attribute__((aligned(16))) float sH[2][S::kWaves][kStrip];
    __shared__ __attribute__((aligned(16))) float sC[2][kStrip];   // state entering the tile
    __shared__ int sNext[2];                                       // the tile after this one

    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / 64), lane = tid % 64;
    const int c = tid % S::kLanes, g = tid / S::kLanes;            // channels and run of the thread
    const int64_t strip = CHAIN ? blockIdx.x % (unsigned)p.plan.strips : blockIdx.x;
    const int64_t b = strip / p.plan.dblocks;
    const int64_t ds = (strip % p.plan.dblocks) * kStrip;
    const int left = (int)(p.D - ds < kStrip ? p.D - ds : kStrip);  // the strip's channels
    const bool in = c * V < left;
    const int64_t len = row_tokens(p, b);
    const int last = len > 0 ? (int)((len - 1) / kTile) : 0;       // the tile of the last token

    GatedChannel ch[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int64_t d = ds + c * V + v;
        ch[v] = gated_channel(in ? p.A[d] : 0.0f, in && p.bias_a ? p.bias_a[d] : 0.0f,
                              in && p.bias_x ? p.bias_x[d] : 0.0f);
    }
    const uint32_t pitch = (uint32_t)(p.D * sizeof(T));
    const uint32_t off = in ? (uint32_t)(g * R) * pitch + (uint32_t)((ds + c * V) * sizeof(T)) : kNoChannel;

    const bool keeper = wave == 0 && lane < left;                  // wavefront 0: channel ds + lane
    // a strip's row of a [rows][D] fp32 tensor; the lane is added last, to a
    // uniform address
    auto row = [&](auto* base, int64_t r) { return base + (r * p.D + ds); };
    const uint32_t ul = lane;
    float carry = keeper && p.h0 ? row(p.h0, b)[ul] : 0.0f;

    typename RowT::Raw rx[R], ra[R], rg[R];
    auto load = [&](int tile) {
        const int64_t t = (int64_t)tile * kTile;
        const __amdgpu_buffer_rsrc_t bx = tile_rows<T>(p.x, p, b, t, len, kTile);
        const __amdgpu_buffer_rsrc_t ba = tile_rows<T>(p.gate_a, p, b, t, len, kTile);
        const __amdgpu_buffer_rsrc_t bg = tile_rows<T>(p.gate_x, p, b, t, len, kTile);
#pragma unroll
        for (int j = 0; j < R; ++j) {
            ra[j] = RowT::load(ba, off + j * pitch);
            rg[j] = RowT::load(bg, off + j * pitch);
            rx[j] = RowT::load(bx, off + j * pitch);
        }
    };

    const Chain chain = CHAIN ? chain_of(p.chain, p.plan, strip) : Chain{};
    int tile = 0;
    if (CHAIN) {
        if (tid == 0) sNext[1] = chain_draw(chain);
        lds_barrier();
        tile = __builtin_amdgcn_readfirstlane(sNext[1]);
    }
    if (tile <= last) load(tile);
    for (int buf = 0; tile <= last; buf ^= 1) {
        int next = tile + 1;
        if (CHAIN && tid == 0) next = chain_draw(chain);
        const int64_t t0 = (int64_t)tile * kTile;
        float a[R][V], h[R][V], pa[V], ph[V];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            float xv[V], av[V], gv[V];
            RowT::unpack(rx[j], xv);
            RowT::unpack(ra[j], av);
            RowT::unpack(rg[j], gv);
#pragma unroll
            for (int v = 0; v < V; ++v) gated_token(xv[v], av[v], gv[v], ch[v], a[j][v], h[j][v]);
        }
        if (t0 + kTile > len) {                  // no token: the state stays
#pragma unroll
            for (int j = 0; j < R; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (t0 + g * R + j >= len) {
                        a[j][v] = 1.0f;
                        h[j][v] = 0.0f;
                    }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            pa[v] = a[0][v];
            ph[v] = h[0][v];
        }
#pragma unroll
        for (int j = 1; j < R; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                pa[v] *= a[j][v];
                ph[v] = fmaf(a[j][v], ph[v], h[j][v]);
            }
        // a wavefront's two runs to one pair; the upper one starts behind the
        // lower (op, oh)
        float op[V], oh[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            op[v] = 1.0f;
            oh[v] = 0.0f;
            if constexpr (S::kPair) {
                const float xp = __shfl_xor(pa[v], 32, 64), xh = __shfl_xor(ph[v], 32, 64);
                if (lane >= 32) {
                    op[v] = xp;
                    oh[v] = xh;
                }
                ph[v] = fmaf(xp, ph[v], xh);       // right in the lower half, which stores it
                pa[v] *= xp;
            }
        }
        if (lane < S::kLanes) {
            lds_put<V>(&sA[buf][wave][c * V], pa);
            lds_put<V>(&sH[buf][wave][c * V], ph);
        }
        if (CHAIN && tid == 0) sNext[buf] = next;
        lds_barrier();
        if (CHAIN) next = __builtin_amdgcn_readfirstlane(sNext[buf]);
        // the folding wavefront's own loads would hold up the states it waits
        // for (loads return in order): it starts them afterwards
        if (wave != 0) {
            load(next);
        } else {
            float P = 1.0f, H = 0.0f;
#pragma unroll
            for (int k = 0; k < S::kWaves; ++k) {
                const float ka = sA[buf][k][lane], kh = sH[buf][k][lane];
                sA[buf][k][lane] = P;
                sH[buf][k][lane] = H;
                H = fmaf(ka, H, kh);
                P *= ka;
            }
            if (CHAIN && tile > 0) {
                if (tile < last) chain_put_map(chain, tile, ul, P, H);
                carry = chain_state_before(chain, tile, lane);
            }
            sC[buf][lane] = carry;
            const float behind = fmaf(P, carry, H) + 0.0f;       // -0 is 0
            if (CHAIN && tile < last) chain_put_state(chain, tile, ul, behind);
            load(next);
            if (keeper && p.ckpt) {
                constexpr int kStep = S::kWaves / kSaved;
#pragma unroll
                for (int m = 0; m < kSaved; ++m)
                    if (m == 0 || t0 + m * SSM_GATED_TILE < len)
                        row(p.ckpt, b * p.saved + tile * kSaved + m)[ul] =
                            fmaf(sA[buf][m * kStep][lane], carry, sH[buf][m * kStep][lane]);
            }
            carry = behind;
            if (keeper && tile == last && p.h_last) row(p.h_last, b)[ul] = carry;
        }
        lds_barrier();
        if (p.y) {
            float s[V], P[V], H[V];
            lds_get<V>(&sC[buf][c * V], s);
            lds_get<V>(&sA[buf][wave][c * V], P);
            lds_get<V>(&sH[buf][wave][c * V], H);
            const __amdgpu_buffer_rsrc_t by = tile_rows<T>(p.y, p, b, t0, len, kTile);
#pragma unroll
            for (int v = 0; v < V; ++v) s[v] = fmaf(op[v], fmaf(P[v], s[v], H[v]), oh[v]);
#pragma unroll
            for (int j = 0; j < R; ++j) {
#pragma unroll
                for (int v = 0; v < V; ++v) s[v] = fmaf(a[j][v], s[v], h[j][v]);
                RowT::store(by, off + j * pitch, s);
            }
        }
        tile = next;
    }
}

// no tokens: the state passes through (zeros without one)
__global__ __launch_bounds__(256) void gated_pass(const float* h0, float* h_last, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) h_last[i] = h0 ? h0[i] : 0.0f;
}

// V neighbouring elements
template <typename T, int V> __device__ __forceinline__ void get(const T* p, float (&v)[V]) {
    if constexpr (V == 2 && sizeof(T) == 2) {
        Row<T, 2>::unpack(*reinterpret_cast<const uint32_t*>(p), v);
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = Elem<T>::load(p, k);
    }
}
template <typename T, int V> __device__ __forceinline__ void put(T* p, const float (&v)[V]) {
#pragma unroll
    for (int k = 0; k < V; ++k) Elem<T>::store(p, k, v[k]);
}

// One token per sequence against a resident state: V channels per thread.
// (64 sequences x 5120 channels, 5.3 MB: 3.7 us, which is the launch; from
// Python a call takes 10 us.)
template <typename T, int V>
__global__ __launch_bounds__(256) void gated_step(GatedStepArgs p) {
    const int64_t vecs = p.D / V;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= p.B * vecs) return;
    const int64_t d = (i % vecs) * V, o = i * V;
    float x[V], ga[V], gx[V], h[V];
    get<T, V>(static_cast<const T*>(p.x) + o, x);
    get<T, V>(static_cast<const T*>(p.gate_a) + o, ga);
    get<T, V>(static_cast<const T*>(p.gate_x) + o, gx);
    get<float, V>(p.state + o, h);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float a, b;
        gated_token(x[v], ga[v], gx[v],
                    gated_channel(p.A[d + v], p.bias_a ? p.bias_a[d + v] : 0.0f,
                                  p.bias_x ? p.bias_x[d + v] : 0.0f), a, b);
        h[v] = fmaf(a, h[v], b) + 0.0f;
    }
    put<float, V>(p.state + o, h);
    put<T, V>(static_cast<T*>(p.y) + o, h);
}

template <typename T>
hipError_t launch_step(const GatedStepArgs& a, hipStream_t stream) {
    const int64_t vecs = a.D % 2 == 0 ? a.D / 2 : a.D;
    return in_slices(a.B, (kMaxItems - 255) / vecs, [&](int64_t b, int64_t n) {
        GatedStepArgs s = a;
        s.state = ahead(a.state, b * a.D);
        s.x = ahead(a.x, b * a.D, sizeof(T));
        s.gate_a = ahead(a.gate_a, b * a.D, sizeof(T));
        s.gate_x = ahead(a.gate_x, b * a.D, sizeof(T));
        s.y = ahead(a.y, b * a.D, sizeof(T));
        s.B = n;
        const unsigned grid = (unsigned)((n * vecs + 255) / 256);
        if (a.D % 2 == 0) gated_step<T, 2><<<grid, 256, 0, stream>>>(s);
        else gated_step<T, 1><<<grid, 256, 0, stream>>>(s);
        return hipGetLastError();
    });
}

template <typename T, int V>
hipError_t launch_fwd_v(const GatedArgs& a, hipStream_t stream) {
    if (a.plan.walkers > 1) {
        const unsigned grid = (unsigned)(a.plan.strips * a.plan.walkers);
        if (!a.cleared) {
            const hipError_t e = launch_chain_clear(a.chain, a.plan.chain_bytes, stream);
            if (e != hipSuccess) return e;
        }
        gated_fwd<T, V, true, 1024><<<grid, 1024, 0, stream>>>(a);
        return hipGetLastError();
    }
    // a workgroup to a strip: whole batch rows, as many as a launch holds
    const int threads = gated::threads(a.L, gated::kFwdTile);
    return in_slices(a.B, kMaxItems / (threads * a.plan.dblocks), [&](int64_t b, int64_t n) {
        GatedArgs s = a;
        s.x = ahead(a.x, b * a.L * a.D, sizeof(T));
        s.gate_a = ahead(a.gate_a, b * a.L * a.D, sizeof(T));
        s.gate_x = ahead(a.gate_x, b * a.L * a.D, sizeof(T));
        s.y = ahead(a.y, b * a.L * a.D, sizeof(T));
        s.h0 = ahead(a.h0, b * a.D);
        s.h_last = ahead(a.h_last, b * a.D);
        s.ckpt = ahead(a.ckpt, b * a.saved * a.D);
        s.seq_lens = ahead(a.seq_lens, b);
        s.B = n;
        s.plan.strips = n * a.plan.dblocks;
        const unsigned strips = (unsigned)s.plan.strips;
        if (threads == 256) gated_fwd<T, V, false, 256><<<strips, 256, 0, stream>>>(s);
        else if (threads == 512) gated_fwd<T, V, false, 512><<<strips, 512, 0, stream>>>(s);
        else gated_fwd<T, V, false, 1024><<<strips, 1024, 0, stream>>>(s);
        return hipGetLastError();
    });
}

template <typename T>
hipError_t launch_fwd(const GatedArgs& a, hipStream_t stream) {
    return a.D % 2 == 0 ? launch_fwd_v<T, 2>(a, stream) : launch_fwd_v<T, 1>(a, stream);
}

}  // namespace

// a kernel rather than a memset: the call may be captured into a graph
__global__ __launch_bounds__(256) void chain_clear(u32x4* p, int64_t n) {
    const int64_t step = (int64_t)gridDim.x * 256;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += step) p[i] = u32x4{0, 0, 0, 0};
}

hipError_t launch_chain_clear(void* chain, size_t bytes, hipStream_t stream) {
    if (bytes == 0) return hipSuccess;
    const int64_t n = (int64_t)(bytes / 16);
    const int64_t blocks = (n + 255) / 256;
    chain_clear<<<(unsigned)(blocks < 2048 ? blocks : 2048), 256, 0, stream>>>(static_cast<u32x4*>(chain), n);
    return hipGetLastError();
}

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
