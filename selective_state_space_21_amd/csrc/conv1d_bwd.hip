// Backward pass of the short causal depthwise convolution + SiLU, which takes
// the scan's input gradient du to the block's input.  With
//   s_t = bias + sum_k w[k] x_{t-(K-1)+k},   u_t = s_t sigma(s_t)
//   g_t  = du_t sigma(s_t) (1 + s_t (1 - sigma(s_t)))     (du_t without SiLU)
//   dx_t = sum_k w[k] g_{t+(K-1)-k}                       (g = 0 behind the end)
//   dw[k] = sum_t g_t x_{t-(K-1)+k},   dbias = sum_t g_t
// and the K-1 inputs before t = 0 (the carried state) get their share of the
// same sum.  Nothing of the forward is stored: s_t is formed again.  Per
// element the call reads x and du and writes dx: it is bound by those bytes.
//
// A thread owns VEC channels (two where the row length is even) and a run of
// tokens; it walks the run and the K-1 tokens after it (whose g it needs for
// its last outputs) with the last inputs and the last g in registers, and the
// loads of kFlight tokens under way at a time.  Rows are addressed through
// buffer resources that end with the sequence: behind it x and du read as
// zero, g is zero, and stores are dropped.
//
// Measured at B=8 L=2048 D=1536 K=4 bf16 (151 MB): 43.4 us for calls back to
// back, 3.5 TB/s, with the sums' last step (alone, in a kernel trace, 40.8 and
// 4.5 us); one channel a thread and one token in flight 91.  What follows a
// run, up to kTail tokens at a time, is walked apart from its whole batches:
// a check of every token against the end there costs nothing (44.3 us with
// and without), in the batches 45.5, and a second copy of the batch for runs
// that end within it 30 registers (8 x 4096 x 2560 without SiLU 111 -> 117).
// Sixteen tokens in flight 44.8 us for the call against 43.8, the next eight
// loaded ahead 44.2, runs of 64 tokens 45.0, four wavefronts to a workgroup
// 43.9.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <type_traits>

#include "block_internal.h"
#include "gated_tile.h"
#include "lane_ops.h"

namespace ssm {
namespace {

constexpr int kWaves = 8;
constexpr int kRun = 32;                        // tokens per thread
constexpr int kFlight = 8;
constexpr int kTail = 4;                        // at least K - 1
constexpr int kBlockTokens = kWaves * kRun;     // a workgroup: 64 * VEC channels of these
static_assert(kBlockTokens == conv::kBlockTokens && kRun % kFlight == 0, "the planner's blocks");

// du u'(s): the derivative of s sigma(s).  Where e^-s leaves fp32's range sigma
// is zero, and with it the product, however large s is; the bound on e keeps
// e sigma = 1 - sigma a number there.
__device__ __forceinline__ float silu_grad(float du, float s) {
    const float e = fast_exp2(-s * kLog2e);
    const float sg = fast_rcp(1.0f + e);
    return du * (sg * fmaf(s, fminf(e, 0x1p126f) * sg, 1.0f));   // 1 - sigma = e sigma
}

template <typename T, int VEC, int K, bool SILU>
__global__ __launch_bounds__(kWaves * 64) void conv1d_bwd_kernel(ConvBwdArgs p) {
    using V = Row<T, VEC>;
    __shared__ float sSum[kWaves][K + 1][64 * VEC];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int64_t dblocks = (p.D + 64 * VEC - 1) / (64 * VEC);
    const int64_t db = blockIdx.x % dblocks;
    const int64_t cell = blockIdx.x / dblocks;                  // b * blocks + block
    const int64_t b = cell / p.blocks, block = cell % p.blocks;
    const int64_t d0 = (db * 64 + lane) * VEC;
    const bool in = d0 < p.D;
    const int64_t t0 = block * kBlockTokens + wave * kRun;      // t0 >= L: an empty run

    float sum[K + 1][VEC];
#pragma unroll
    for (int k = 0; k <= K; ++k)
#pragma unroll
        for (int c = 0; c < VEC; ++c) sum[k][c] = 0.0f;

    if (t0 < p.L) {
        const uint32_t pitch = (uint32_t)(p.D * sizeof(T));
        const uint32_t off = in ? (uint32_t)(d0 * sizeof(T)) : kNoChannel;
        const int64_t row0 = (b * p.L + t0) * p.D;
        const int64_t n = p.L - t0;                             // tokens from here on
        const int mine = n < kRun ? (int)n : kRun;
        const int there = n < kRun + K - 1 ? (int)n : kRun + K - 1;   // of the tokens walked
        const uint32_t seen = (uint32_t)(there * p.D * sizeof(T));
        const __amdgpu_buffer_rsrc_t rx = make_rsrc(static_cast<const T*>(p.x) + row0, seen);
        const __amdgpu_buffer_rsrc_t ru = make_rsrc(static_cast<const T*>(p.du) + row0, seen);
        const __amdgpu_buffer_rsrc_t ro = make_rsrc(static_cast<T*>(p.dx) + row0, (uint32_t)mine * pitch);
        float w[VEC][K], bias[VEC];
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
#pragma unroll
            for (int k = 0; k < K; ++k) w[c][k] = in ? p.weight[(d0 + c) * K + k] : 0.0f;
            bias[c] = in && p.bias ? p.bias[d0 + c] : 0.0f;
        }
        float win[K][VEC];         // x_{t-(K-1)} .. x_t
        float g[K][VEC];           // g_{t-(K-1)} .. g_t
#pragma unroll
        for (int i = 0; i < K - 1; ++i) {
            const int64_t t = t0 - (K - 1) + i;
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                g[i][c] = 0.0f;
                win[i][c] = 0.0f;
                if (in && t >= 0) win[i][c] = Elem<T>::load(static_cast<const T*>(p.x), (b * p.L + t) * p.D + d0 + c);
                else if (in && p.state_in) win[i][c] = p.state_in[(b * p.D + d0 + c) * (K - 1) + (t + K - 1)];
            }
        }
        // token t0 + u: its own part of the sums (when it is of this run), then
        // the output of token u - (K-1), whose last term it is.  past: it may
        // be behind the run or the end.  Behind the end nothing counts: s and
        // the inputs in the window may be infinite, and g = 0 no help
        auto token = [&](int u, auto past) {
            constexpr bool kPast = decltype(past)::value;
            if (!kPast || u < there) {
#pragma unroll
                for (int c = 0; c < VEC; ++c) {
                    if (SILU) {
                        float s = bias[c];
#pragma unroll
                        for (int k = 0; k < K; ++k) s = fmaf(w[c][k], win[k][c], s);
                        g[K - 1][c] = silu_grad(g[K - 1][c], s);
                    }
                    if (!kPast || u < mine) {
#pragma unroll
                        for (int k = 0; k < K; ++k) sum[k][c] = fmaf(g[K - 1][c], win[k][c], sum[k][c]);
                        sum[K][c] += g[K - 1][c];
                    }
                }
            }
            const int to = u - (K - 1);
            if (to >= 0) {
                float o[VEC];
#pragma unroll
                for (int c = 0; c < VEC; ++c) {
                    o[c] = 0.0f;
#pragma unroll
                    for (int k = 0; k < K; ++k) o[c] = fmaf(w[c][k], g[K - 1 - k][c], o[c]);
                }
                if (p.dstate_out && to + (K - 1) >= n && to < n && in) {     // handed on in the state
#pragma unroll
                    for (int c = 0; c < VEC; ++c)
                        o[c] += p.dstate_out[(b * p.D + d0 + c) * (K - 1) + (to + (K - 1) - n)];
                }
                V::store(ro, off + (uint32_t)to * pitch, o);
            }
#pragma unroll
            for (int i = 0; i < K - 1; ++i)
#pragma unroll
                for (int c = 0; c < VEC; ++c) {
                    win[i][c] = win[i + 1][c];
                    g[i][c] = g[i + 1][c];
                }
        };
        // tokens [u0, u0 + N), N loads of each input under way
        auto batch = [&](int u0, auto count, auto past) {
            constexpr int N = decltype(count)::value;
            typename V::Raw xs[N], us[N];
#pragma unroll
            for (int j = 0; j < N; ++j) {
                xs[j] = V::load(rx, off + (uint32_t)(u0 + j) * pitch);
                us[j] = V::load(ru, off + (uint32_t)(u0 + j) * pitch);
            }
#pragma unroll
            for (int j = 0; j < N; ++j) {
                V::unpack(xs[j], win[K - 1]);
                V::unpack(us[j], g[K - 1]);
                token(u0 + j, past);
            }
        };
        int u0 = 0;
        for (; u0 + kFlight <= mine; u0 += kFlight)
            batch(u0, std::integral_constant<int, kFlight>{}, std::false_type{});
        for (; u0 < mine + K - 1; u0 += kTail)      // what is left of the run, and the tokens after it
            batch(u0, std::integral_constant<int, kTail>{}, std::true_type{});
    }
#pragma unroll
    for (int k = 0; k <= K; ++k)
#pragma unroll
        for (int c = 0; c < VEC; ++c) sSum[wave][k][lane * VEC + c] = sum[k][c];
    lds_barrier();
    for (int i = threadIdx.x; i < (K + 1) * 64 * VEC; i += kWaves * 64) {
        const int k = i / (64 * VEC), ch = i % (64 * VEC);
        float s = 0.0f;
#pragma unroll
        for (int m = 0; m < kWaves; ++m) s += sSum[m][k][ch];
        const int64_t d = db * 64 * VEC + ch;
        if (d < p.D) p.part[(cell * (K + 1) + k) * p.D + d] = s;
    }
}

// The carried state's gradient: slot j is the input at t = j - (K-1), which
// reaches the first j + 1 tokens, and (when the call has fewer than K-1
// tokens) the state that it hands on.  One thread per channel.
template <typename T, int K, bool SILU>
__global__ __launch_bounds__(256) void conv1d_bwd_state(ConvBwdArgs p) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= p.B * p.D) return;
    const int64_t b = i / p.D, d = i % p.D;
    const T* x = static_cast<const T*>(p.x) + b * p.L * p.D + d;
    const T* du = static_cast<const T*>(p.du) + b * p.L * p.D + d;
    float w[K], win[2 * K - 1], g[K];        // win: the state, then the first K-1 inputs
#pragma unroll
    for (int k = 0; k < K; ++k) w[k] = p.weight[d * K + k];
#pragma unroll
    for (int j = 0; j < 2 * (K - 1); ++j) {
        const int64_t t = j - (K - 1);
        win[j] = 0.0f;
        if (t < 0) win[j] = p.state_in ? p.state_in[i * (K - 1) + j] : 0.0f;
        else if (t < p.L) win[j] = Elem<T>::load(x, t * p.D);
    }
#pragma unroll
    for (int t = 0; t < K - 1; ++t) {
        g[t] = 0.0f;
        if (t < p.L) {
            float v = Elem<T>::load(du, t * p.D);
            if (SILU) {
                float s = p.bias ? p.bias[d] : 0.0f;
#pragma unroll
                for (int k = 0; k < K; ++k) s = fmaf(w[k], win[t + k], s);
                v = silu_grad(v, s);
            }
            g[t] = v;
        }
    }
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
        float o = 0.0f;
#pragma unroll
        for (int t = 0; t <= j; ++t) o = fmaf(w[j - t], g[t], o);
        if (p.dstate_out && j >= p.L) o += p.dstate_out[i * (K - 1) + (j - p.L)];
        p.dstate_in[i * (K - 1) + j] = o;
    }
}

template <typename T, int VEC, int K, bool SILU>
hipError_t launch_s(const ConvBwdArgs& a, hipStream_t stream) {
    // whole batch rows, as many at once as a launch holds
    auto slice = [&](int64_t b, int64_t n) {
        ConvBwdArgs s = a;
        s.x = ahead(a.x, b * a.L * a.D, sizeof(T));
        s.du = ahead(a.du, b * a.L * a.D, sizeof(T));
        s.dx = ahead(a.dx, b * a.L * a.D, sizeof(T));
        s.state_in = ahead(a.state_in, b * a.D * (K - 1));
        s.dstate_out = ahead(a.dstate_out, b * a.D * (K - 1));
        s.dstate_in = ahead(a.dstate_in, b * a.D * (K - 1));
        s.part = ahead(a.part, b * a.blocks * (K + 1) * a.D);
        s.B = n;
        return s;
    };
    if (a.blocks > 0) {
        const int64_t groups = (a.D + 64 * VEC - 1) / (64 * VEC) * a.blocks;
        const hipError_t e = in_slices(a.B, kMaxItems / (kWaves * 64 * groups), [&](int64_t b, int64_t n) {
            conv1d_bwd_kernel<T, VEC, K, SILU><<<(unsigned)(groups * n), kWaves * 64, 0, stream>>>(slice(b, n));
            return hipGetLastError();
        });
        if (e != hipSuccess) return e;
    }
    if constexpr (K > 1) {
        if (a.dstate_in)
            return in_slices(a.B, (kMaxItems - 255) / a.D, [&](int64_t b, int64_t n) {
                conv1d_bwd_state<T, K, SILU><<<(unsigned)((n * a.D + 255) / 256), 256, 0, stream>>>(slice(b, n));
                return hipGetLastError();
            });
    }
    return hipSuccess;
}

template <typename T, int VEC>
hipError_t launch_v(const ConvBwdArgs& a, hipStream_t stream) {
    switch (a.K * 2 + (a.silu ? 1 : 0)) {
        case 2: return launch_s<T, VEC, 1, false>(a, stream);
        case 3: return launch_s<T, VEC, 1, true>(a, stream);
        case 4: return launch_s<T, VEC, 2, false>(a, stream);
        case 5: return launch_s<T, VEC, 2, true>(a, stream);
        case 6: return launch_s<T, VEC, 3, false>(a, stream);
        case 7: return launch_s<T, VEC, 3, true>(a, stream);
        case 8: return launch_s<T, VEC, 4, false>(a, stream);
        default: return launch_s<T, VEC, 4, true>(a, stream);
    }
}

}  // namespace

hipError_t launch_conv1d_bwd(const ConvBwdArgs& a, hipStream_t stream) {
    hipError_t e;
    if (a.bf16) e = a.D % 2 == 0 ? launch_v<uint16_t, 2>(a, stream) : launch_v<uint16_t, 1>(a, stream);
    else e = a.D % 2 == 0 ? launch_v<float, 2>(a, stream) : launch_v<float, 1>(a, stream);
    if (e != hipSuccess) return e;
    ColumnSums s{};
    s.part = a.part;
    s.n = a.B * a.blocks;
    s.D = a.D;
    s.m = (int)a.K + 1;
    s.out[0] = a.dweight;
    s.out[1] = a.dbias;
    s.strided = 1;
    return launch_column_sums(s, stream);
}

}  // namespace ssm
