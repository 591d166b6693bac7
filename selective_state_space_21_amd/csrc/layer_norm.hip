// Layer norm over the last axis, forward and backward, with the fp32 residual
// stream's addition in front of it.  Per row s = x (+ residual):
//   mu = mean(s), rstd = 1 / sqrt(mean((s - mu)^2) + eps),  n = (s - mu) rstd
//   y  = n weight + bias
// and backward, with v = dy weight:
//   ds = rstd (v - mean(v) - n mean(v n)) (+ the gradient of s itself)
//   dweight = sum over rows of dy n,   dbias = sum over rows of dy
//
// A row is read once and kept in registers: mean, then the mean square of the
// differences from it (two passes over registers, so nothing cancels).  TPR
// threads share a row (8 lanes for the shortest, a wavefront, a whole
// workgroup for long rows) and each holds NV vectors of VEC elements, vector i
// of thread j being vector i * TPR + j of the row.  Rows too long for that are
// read from memory again for every pass.  Both directions are bound by the
// bytes they move.
//
// Measured with the residual stream, 16384 x 768 bf16: forward (151 MB) 31.8
// us, 4.8 TB/s; backward (201 MB) 40.7 us, 4.9 TB/s, 4 of them the sums' last
// step.  33M elements without it: D = 64 to 16384 bf16 27 to 34 us forward, 42
// to 70 backward (at the copy rate 27 and 40), fp32 45 to 58 and 69 to 93 (54
// and 81).
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "block_internal.h"
#include "device_math.h"
#include "gated_tile.h"
#include "lane_ops.h"

namespace ssm {
namespace {

constexpr int kBwdThreads = 1024;

// VEC elements as fp32: 16-byte vectors of the activations, and for fp32
// operands beside bf16 ones two of them.  Rows of odd length leave a vector at
// any element's alignment, which the hardware's global accesses allow (777
// rows of 2561 fp32 elements, forward and backward without the sums' last
// step: 25.0 us by single elements, 17.3 by vectors).
template <int VEC> struct Bits;                  // VEC bf16 elements
template <> struct Bits<8> {
    typedef uint32_t type __attribute__((ext_vector_type(4), aligned(2)));
};
template <> struct Bits<4> {
    typedef uint32_t type __attribute__((ext_vector_type(2), aligned(2)));
};
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

template <int VEC> __device__ __forceinline__ void load_all(const uint16_t* p, float (&v)[VEC]) {
    const auto r = __builtin_nontemporal_load(reinterpret_cast<const typename Bits<VEC>::type*>(p));
#pragma unroll
    for (int k = 0; k < VEC / 2; ++k) {
        v[2 * k] = __uint_as_float(r[k] << 16);
        v[2 * k + 1] = __uint_as_float(r[k] & 0xffff0000u);
    }
}
template <int VEC> __device__ __forceinline__ void load_all(const float* p, float (&v)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
        const auto r = __builtin_nontemporal_load(reinterpret_cast<const f32x4_any*>(p) + i);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[4 * i + k] = r[k];
    }
}
template <int VEC> __device__ __forceinline__ void store_all(uint16_t* p, const float (&v)[VEC]) {
    typename Bits<VEC>::type r;
#pragma unroll
    for (int k = 0; k < VEC / 2; ++k)
        r[k] = (uint32_t)f32_to_bf16_bits(v[2 * k]) | ((uint32_t)f32_to_bf16_bits(v[2 * k + 1]) << 16);
    __builtin_nontemporal_store(r, reinterpret_cast<typename Bits<VEC>::type*>(p));
}
template <int VEC> __device__ __forceinline__ void store_all(float* p, const float (&v)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
        const f32x4_any r = {v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
        __builtin_nontemporal_store(r, reinterpret_cast<f32x4_any*>(p) + i);
    }
}

// the first n of VEC elements (n <= 0: none), zeros for the others; WHOLE: the
// row is whole vectors, n is VEC or more, or 0 or less
template <bool WHOLE, typename T, int VEC>
__device__ __forceinline__ void get(const T* p, int64_t n, float (&v)[VEC]) {
    if (WHOLE ? n > 0 : n >= VEC) {
        load_all<VEC>(p, v);
    } else {
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[k] = !WHOLE && k < n ? Elem<T>::load(p, k) : 0.0f;
    }
}
template <bool WHOLE, typename T, int VEC>
__device__ __forceinline__ void put(T* p, int64_t n, const float (&v)[VEC]) {
    if (WHOLE ? n > 0 : n >= VEC) {
        store_all<VEC>(p, v);
    } else if (!WHOLE) {
#pragma unroll
        for (int k = 0; k < VEC; ++k)
            if (k < n) Elem<T>::store(p, k, v[k]);
    }
}

// the parameters are read by every row: through the cache
template <bool WHOLE, int VEC>
__device__ __forceinline__ void get_param(const float* p, int64_t d, int64_t n, float (&v)[VEC], float none) {
    if (p && (WHOLE ? n > 0 : n >= VEC)) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[k] = p[d + k];
    } else {
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[k] = !WHOLE && p && k < n ? p[d + k] : none;
    }
}

// the sum over aligned groups of N lanes, in all of them
template <int N> __device__ __forceinline__ float lane_sum(float v) {
    if constexpr (N > 32) v += __shfl_xor(v, 32, 64);
    if constexpr (N > 16) v += lane_xor<16>(v);
    if constexpr (N > 8) v += lane_xor<8>(v);
    if constexpr (N > 4) v += lane_xor<4>(v);
    v += lane_xor<2>(v);
    v += lane_xor<1>(v);
    return v;
}

// the sum over the TPR threads of a row, in all of them; `s` holds one float
// per wavefront of the workgroup, all of whose threads take part
template <int TPR> __device__ __forceinline__ float row_sum(float v, float* s) {
    v = lane_sum<TPR < 64 ? TPR : 64>(v);
    if constexpr (TPR > 64) {
        constexpr int W = TPR / 64;
        const int wave = threadIdx.x / 64, first = wave / W * W;
        lds_barrier();                       // the previous sum has been read
        if (threadIdx.x % 64 == 0) s[wave] = v;
        lds_barrier();
        v = s[first];
#pragma unroll
        for (int k = 1; k < W; ++k) v += s[first + k];
    }
    return v;
}

template <bool WHOLE, typename T, bool RES, int VEC, int NV, int TPR>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void norm_fwd(NormArgs p) {
    constexpr int kThreads = TPR > 256 ? TPR : 256;
    __shared__ float s[kThreads / 64];
    const int j = threadIdx.x % TPR;
    const int64_t at = (int64_t)blockIdx.x * (kThreads / TPR) + threadIdx.x / TPR;
    if (TPR == 64 && at >= p.rows) return;   // a whole wavefront
    const bool there = at < p.rows;          // (the lanes of a wavefront sum together: all stay)
    const int64_t row = there ? at : p.rows - 1, o = row * p.D;
    const T* x = static_cast<const T*>(p.x) + o;
    float v[NV][VEC];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t d = (int64_t)(i * TPR + j) * VEC, n = p.D - d;
        get<WHOLE, T, VEC>(x + d, n, v[i]);
        if (RES) {
            float r[VEC];
            get<WHOLE, float, VEC>(p.residual + o + d, n, r);
#pragma unroll
            for (int k = 0; k < VEC; ++k) v[i][k] += r[k];
        }
#pragma unroll
        for (int k = 0; k < VEC; ++k) sum += v[i][k];
    }
    const float inv = 1.0f / (float)p.D;
    const float mean = row_sum<TPR>(sum, s) * inv;
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t n = p.D - (int64_t)(i * TPR + j) * VEC;
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            const float c = k < n ? v[i][k] - mean : 0.0f;
            sum = fmaf(c, c, sum);
        }
    }
    const float rstd = 1.0f / sqrtf(fmaf(row_sum<TPR>(sum, s), inv, p.eps));
    if (TPR < 64 && !there) return;
    if (j == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t d = (int64_t)(i * TPR + j) * VEC, n = p.D - d;
        if (RES && p.residual_out) put<WHOLE, float, VEC>(p.residual_out + o + d, n, v[i]);
        float w[VEC], b[VEC];
        get_param<WHOLE, VEC>(p.weight, d, n, w, 1.0f);
        get_param<WHOLE, VEC>(p.bias, d, n, b, 0.0f);
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[i][k] = fmaf((v[i][k] - mean) * rstd, w[k], b[k]);
        put<WHOLE, T, VEC>(static_cast<T*>(p.y) + o + d, n, v[i]);
    }
}

// rows of any length: read again for each pass
template <typename T, bool RES>
__global__ __launch_bounds__(1024) void norm_fwd_long(NormArgs p) {
    __shared__ float s[16];
    const int64_t o = (int64_t)blockIdx.x * p.D;
    const T* x = static_cast<const T*>(p.x) + o;
    auto at = [&](int64_t d) {
        const float v = Elem<T>::load(x, d);
        return RES ? v + p.residual[o + d] : v;
    };
    const float inv = 1.0f / (float)p.D;
    float sum = 0.0f;
    for (int64_t d = threadIdx.x; d < p.D; d += 1024) sum += at(d);
    const float mean = row_sum<1024>(sum, s) * inv;
    sum = 0.0f;
    for (int64_t d = threadIdx.x; d < p.D; d += 1024) {
        const float c = at(d) - mean;
        sum = fmaf(c, c, sum);
    }
    const float rstd = 1.0f / sqrtf(fmaf(row_sum<1024>(sum, s), inv, p.eps));
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[blockIdx.x] = mean;
        if (p.rstd) p.rstd[blockIdx.x] = rstd;
    }
    for (int64_t d = threadIdx.x; d < p.D; d += 1024) {
        const float v = at(d);
        if (RES && p.residual_out) p.residual_out[o + d] = v;
        Elem<T>::store(static_cast<T*>(p.y) + o, d,
                       fmaf((v - mean) * rstd, p.weight ? p.weight[d] : 1.0f,
                            p.bias ? p.bias[d] : 0.0f));
    }
}

// X: the type of the normalised input (the fp32 stream, or the activations'),
// T: the activations' type.
// A workgroup of 1024 threads takes 1024 / TPR rows at a time and a share of
// all rows, with its sums for the parameters in registers: one workgroup per
// CU, so that there are few partial sums to write and read (16384 x 2048 bf16:
// 75 us with 512 workgroups of four rows, which leave a CU eight wavefronts).
template <bool WHOLE, typename X, typename T, int VEC, int NV, int TPR>
__global__ __launch_bounds__(kBwdThreads) void norm_bwd(NormBwdArgs p) {
    constexpr int kRows = kBwdThreads / TPR;
    constexpr int kJoin = TPR < 64 ? kBwdThreads / 64 : kRows;      // rows of partial sums left to join
    __shared__ float s[kBwdThreads / 64];
    __shared__ float join[kJoin > 1 ? kJoin : 1][VEC][kJoin > 1 ? TPR : 1];
    const int j = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const float inv = 1.0f / (float)p.D;
    // the weight stays in registers, or is read again (through the cache) for
    // every row where 16 elements a thread at 128 registers leave no room
    constexpr bool HOLD = NV * VEC <= 12;
    float w[HOLD ? NV : 1][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t d = (int64_t)(i * TPR + j) * VEC;
        if (HOLD) get_param<WHOLE, VEC>(p.weight, d, p.D - d, w[HOLD ? i : 0], 1.0f);
#pragma unroll
        for (int k = 0; k < VEC; ++k) dw[i][k] = db[i][k] = 0.0f;
    }
    for (int64_t row0 = (int64_t)blockIdx.x * kRows; row0 < p.rows; row0 += p.groups * kRows) {
        const bool there = row0 + sub < p.rows;                     // all threads sum together
        const int64_t row = there ? row0 + sub : p.rows - 1, o = row * p.D;
        const float mean = p.mean[row], rstd = p.rstd[row];
        float n[NV][VEC], v[NV][VEC];
        float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t d = (int64_t)(i * TPR + j) * VEC, left = p.D - d;
            get<WHOLE, X, VEC>(static_cast<const X*>(p.x) + o + d, left, n[i]);
            get<WHOLE, T, VEC>(static_cast<const T*>(p.dy) + o + d, there ? left : 0, v[i]);   // zero behind the row
            float (&wi)[VEC] = w[HOLD ? i : 0];
            if (!HOLD) get_param<WHOLE, VEC>(p.weight, d, left, wi, 1.0f);
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                n[i][k] = (n[i][k] - mean) * rstd;
                dw[i][k] = fmaf(v[i][k], n[i][k], dw[i][k]);
                db[i][k] += v[i][k];
                v[i][k] *= wi[k];
                c1 = fmaf(v[i][k], n[i][k], c1);
                c2 += v[i][k];
            }
        }
        c1 = row_sum<TPR>(c1, s) * inv;
        c2 = row_sum<TPR>(c2, s) * inv;
        if (!there) continue;                // (no barrier is left in the last round)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t d = (int64_t)(i * TPR + j) * VEC, left = p.D - d;
            float g[VEC];
#pragma unroll
            for (int k = 0; k < VEC; ++k) g[k] = 0.0f;
            if (p.dresidual_out) get<WHOLE, float, VEC>(p.dresidual_out + o + d, left, g);
#pragma unroll
            for (int k = 0; k < VEC; ++k) g[k] = fmaf(rstd, v[i][k] - c2 - n[i][k] * c1, g[k]);
            if (p.dresidual) put<WHOLE, float, VEC>(p.dresidual + o + d, left, g);
            put<WHOLE, T, VEC>(static_cast<T*>(p.dx) + o + d, left, g);
        }
    }
    // join the rows that ran side by side -- a wavefront's by lanes, then the
    // others in order -- for this workgroup's row of part
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            float (&a)[VEC] = which ? db[i] : dw[i];
            if constexpr (TPR < 64) {
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    if constexpr (TPR <= 8) a[k] += lane_xor<8>(a[k]);
                    if constexpr (TPR <= 16) a[k] += lane_xor<16>(a[k]);
                    a[k] += __shfl_xor(a[k], 32, 64);
                }
            }
            const int from = TPR < 64 ? threadIdx.x / 64 : sub;
            const bool puts = TPR >= 64 || threadIdx.x % 64 < TPR;
            if constexpr (kJoin > 1) {
                lds_barrier();
                if (puts) {
#pragma unroll
                    for (int k = 0; k < VEC; ++k) join[from][k][j] = a[k];
                }
                lds_barrier();
                if (puts && from == 0) {
#pragma unroll
                    for (int m = 1; m < kJoin; ++m)
#pragma unroll
                        for (int k = 0; k < VEC; ++k) a[k] += join[m][k][j];
                }
            }
            const int64_t d = (int64_t)(i * TPR + j) * VEC;
            if (puts && from == 0 && d < p.D) {
                float* out = p.part + ((int64_t)blockIdx.x * 2 + which) * p.D + d;
#pragma unroll
                for (int k = 0; k < VEC; ++k)
                    if (WHOLE || d + k < p.D) out[k] = a[k];
            }
        }
    }
}

// rows of any length: dx row by row, then the parameters' sums column by column
template <typename X, typename T>
__global__ __launch_bounds__(1024) void norm_bwd_long(NormBwdArgs p) {
    __shared__ float s[16];
    const int64_t o = (int64_t)blockIdx.x * p.D;
    const X* x = static_cast<const X*>(p.x) + o;
    const T* dy = static_cast<const T*>(p.dy) + o;
    const float mean = p.mean[blockIdx.x], rstd = p.rstd[blockIdx.x], inv = 1.0f / (float)p.D;
    float c1 = 0.0f, c2 = 0.0f;
    for (int64_t d = threadIdx.x; d < p.D; d += 1024) {
        const float v = Elem<T>::load(dy, d) * (p.weight ? p.weight[d] : 1.0f);
        c1 = fmaf(v, (Elem<X>::load(x, d) - mean) * rstd, c1);
        c2 += v;
    }
    c1 = row_sum<1024>(c1, s) * inv;
    c2 = row_sum<1024>(c2, s) * inv;
    for (int64_t d = threadIdx.x; d < p.D; d += 1024) {
        const float v = Elem<T>::load(dy, d) * (p.weight ? p.weight[d] : 1.0f);
        const float n = (Elem<X>::load(x, d) - mean) * rstd;
        const float g = fmaf(rstd, v - c2 - n * c1, p.dresidual_out ? p.dresidual_out[o + d] : 0.0f);
        if (p.dresidual) p.dresidual[o + d] = g;
        Elem<T>::store(static_cast<T*>(p.dx) + o, d, g);
    }
}

template <typename X, typename T>
__global__ __launch_bounds__(256) void norm_bwd_columns(NormBwdArgs p) {
    const int64_t d = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t group = blockIdx.y;
    if (d >= p.D) return;
    float dw = 0.0f, db = 0.0f;
    for (int64_t row = group; row < p.rows; row += p.groups) {
        const float v = Elem<T>::load(static_cast<const T*>(p.dy), row * p.D + d);
        const float n = (Elem<X>::load(static_cast<const X*>(p.x), row * p.D + d) - p.mean[row]) * p.rstd[row];
        dw = fmaf(v, n, dw);
        db += v;
    }
    p.part[(group * 2) * p.D + d] = dw;
    p.part[(group * 2 + 1) * p.D + d] = db;
}

// the rows, as many at once as a launch holds
template <typename T, typename Launch>
hipError_t slices(const NormArgs& a, int64_t most, Launch&& launch) {
    return in_slices(a.rows, most, [&](int64_t row, int64_t n) {
        NormArgs s = a;
        s.x = ahead(a.x, row * a.D, sizeof(T));
        s.residual = ahead(a.residual, row * a.D);
        s.y = ahead(a.y, row * a.D, sizeof(T));
        s.residual_out = ahead(a.residual_out, row * a.D);
        s.mean = ahead(a.mean, row);
        s.rstd = ahead(a.rstd, row);
        s.rows = n;
        launch(s);
        return hipGetLastError();
    });
}

template <bool WHOLE, typename T, bool RES, int VEC, int NV, int TPR>
hipError_t launch_fwd(const NormArgs& a, hipStream_t stream) {
    constexpr int threads = TPR > 256 ? TPR : 256;
    constexpr int rows = threads / TPR;
    return slices<T>(a, kMaxItems / threads * rows, [&](const NormArgs& s) {
        norm_fwd<WHOLE, T, RES, VEC, NV, TPR>
            <<<(unsigned)((s.rows + rows - 1) / rows), threads, 0, stream>>>(s);
    });
}

// the thread layout of a row of `nv` vectors
template <bool WHOLE, typename T, bool RES, int VEC>
hipError_t launch_fwd_v(const NormArgs& a, hipStream_t stream) {
    const int64_t nv = (a.D + VEC - 1) / VEC;
    if (nv <= 8) return launch_fwd<WHOLE, T, RES, VEC, 1, 8>(a, stream);
    if (nv <= 16) return launch_fwd<WHOLE, T, RES, VEC, 1, 16>(a, stream);
    if (nv <= 32) return launch_fwd<WHOLE, T, RES, VEC, 1, 32>(a, stream);
    if (nv <= 64) return launch_fwd<WHOLE, T, RES, VEC, 1, 64>(a, stream);
    if (nv <= 128) return launch_fwd<WHOLE, T, RES, VEC, 2, 64>(a, stream);
    if (nv <= 256) return launch_fwd<WHOLE, T, RES, VEC, 4, 64>(a, stream);
    if (nv <= 512) return launch_fwd<WHOLE, T, RES, VEC, 2, 256>(a, stream);
    if (nv <= 768) return launch_fwd<WHOLE, T, RES, VEC, 3, 256>(a, stream);
    if (nv <= 1024) return launch_fwd<WHOLE, T, RES, VEC, 4, 256>(a, stream);
    if (nv <= 2048) return launch_fwd<WHOLE, T, RES, VEC, 2, 1024>(a, stream);
    if (nv <= 4096) return launch_fwd<WHOLE, T, RES, VEC, 4, 1024>(a, stream);
    return slices<T>(a, kMaxItems / 1024, [&](const NormArgs& s) {
        norm_fwd_long<T, RES><<<(unsigned)s.rows, 1024, 0, stream>>>(s);
    });
}

template <typename T, int VEC>
hipError_t launch_fwd_t(const NormArgs& a, hipStream_t stream) {
    if (a.D % VEC == 0)
        return a.residual ? launch_fwd_v<true, T, true, VEC>(a, stream) : launch_fwd_v<true, T, false, VEC>(a, stream);
    return a.residual ? launch_fwd_v<false, T, true, VEC>(a, stream) : launch_fwd_v<false, T, false, VEC>(a, stream);
}

template <bool WHOLE, typename X, typename T, int VEC, int NV, int TPR>
hipError_t launch_bwd(const NormBwdArgs& a, hipStream_t stream) {
    norm_bwd<WHOLE, X, T, VEC, NV, TPR><<<(unsigned)a.groups, kBwdThreads, 0, stream>>>(a);
    return hipGetLastError();
}

// At most 16 elements a thread: four or five values of each are in registers.
// Where the normalised input is fp32 (bf16 or fp32 around it), vectors of four
// elements, at most four to a thread, and the fewest threads to a row that can
// hold it so: three quarters of them or more have work (the stream's 16384 x
// 768: 40.8 us against 47.5 with vectors of eight, 96 of 128 lanes with work).
// Where all is bf16, 16-byte vectors of eight, two to a thread (16384 x 2048:
// 51 us against 65 with vectors of four).
template <bool WHOLE, typename X, typename T, int TPR>
hipError_t launch_bwd_n(const NormBwdArgs& a, int64_t nv, hipStream_t stream) {
    return nv <= 3 * TPR ? launch_bwd<WHOLE, X, T, 4, 3, TPR>(a, stream) : launch_bwd<WHOLE, X, T, 4, 4, TPR>(a, stream);
}
template <bool WHOLE, typename X, typename T>
hipError_t launch_bwd_w(const NormBwdArgs& a, hipStream_t stream) {
    if constexpr (sizeof(X) == 4) {
        const int64_t nv = (a.D + 3) / 4;
        if (nv <= 16) return launch_bwd<WHOLE, X, T, 4, 1, 16>(a, stream);
        if (nv <= 32) return launch_bwd<WHOLE, X, T, 4, 2, 16>(a, stream);
        if (nv <= 64) return launch_bwd_n<WHOLE, X, T, 16>(a, nv, stream);
        if (nv <= 128) return launch_bwd_n<WHOLE, X, T, 32>(a, nv, stream);
        if (nv <= 256) return launch_bwd_n<WHOLE, X, T, 64>(a, nv, stream);
        if (nv <= 512) return launch_bwd_n<WHOLE, X, T, 128>(a, nv, stream);
        if (nv <= 1024) return launch_bwd_n<WHOLE, X, T, 256>(a, nv, stream);
        if (nv <= 2048) return launch_bwd_n<WHOLE, X, T, 512>(a, nv, stream);
        if (nv <= 4096) return launch_bwd_n<WHOLE, X, T, 1024>(a, nv, stream);
    } else {
        const int64_t nv = (a.D + 7) / 8;
        if (nv <= 8) return launch_bwd<WHOLE, X, T, 8, 1, 8>(a, stream);
        if (nv <= 16) return launch_bwd<WHOLE, X, T, 8, 1, 16>(a, stream);
        if (nv <= 32) return launch_bwd<WHOLE, X, T, 8, 1, 32>(a, stream);
        if (nv <= 64) return launch_bwd<WHOLE, X, T, 8, 1, 64>(a, stream);
        if (nv <= 128) return launch_bwd<WHOLE, X, T, 8, 2, 64>(a, stream);
        if (nv <= 256) return launch_bwd<WHOLE, X, T, 8, 2, 128>(a, stream);
        if (nv <= 512) return launch_bwd<WHOLE, X, T, 8, 2, 256>(a, stream);
        if (nv <= 1024) return launch_bwd<WHOLE, X, T, 8, 2, 512>(a, stream);
        if (nv <= 2048) return launch_bwd<WHOLE, X, T, 8, 2, 1024>(a, stream);
    }
    const hipError_t e = in_slices(a.rows, kMaxItems / 1024, [&](int64_t row, int64_t n) {
        NormBwdArgs s = a;
        s.x = ahead(a.x, row * a.D, sizeof(X));
        s.dy = ahead(a.dy, row * a.D, sizeof(T));
        s.mean = ahead(a.mean, row);
        s.rstd = ahead(a.rstd, row);
        s.dresidual_out = ahead(a.dresidual_out, row * a.D);
        s.dx = ahead(a.dx, row * a.D, sizeof(T));
        s.dresidual = ahead(a.dresidual, row * a.D);
        s.rows = n;
        norm_bwd_long<X, T><<<(unsigned)n, 1024, 0, stream>>>(s);
        return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    norm_bwd_columns<X, T>
        <<<dim3((unsigned)((a.D + 255) / 256), (unsigned)a.groups), 256, 0, stream>>>(a);
    return hipGetLastError();
}

template <typename X, typename T>
hipError_t launch_bwd_t(const NormBwdArgs& a, hipStream_t stream) {
    return a.D % (sizeof(X) == 4 ? 4 : 8) == 0 ? launch_bwd_w<true, X, T>(a, stream) : launch_bwd_w<false, X, T>(a, stream);
}

}  // namespace

hipError_t launch_layer_norm(const NormArgs& a, hipStream_t stream) {
    if (a.rows == 0) return hipSuccess;
    return a.bf16 ? launch_fwd_t<uint16_t, 8>(a, stream) : launch_fwd_t<float, 4>(a, stream);
}

hipError_t launch_layer_norm_bwd(const NormBwdArgs& a, hipStream_t stream) {
    if (a.rows > 0) {
        hipError_t e;
        if (!a.bf16) e = launch_bwd_t<float, float>(a, stream);
        else if (a.x_bf16) e = launch_bwd_t<uint16_t, uint16_t>(a, stream);
        else e = launch_bwd_t<float, uint16_t>(a, stream);
        if (e != hipSuccess) return e;
    }
    if (!a.dweight && !a.dbias) return hipSuccess;
    ColumnSums s{};
    s.part = a.part;
    s.n = a.rows > 0 ? a.groups : 0;
    s.D = a.D;
    s.m = 2;
    s.out[0] = a.dweight;
    s.out[1] = a.dbias;
    return launch_column_sums(s, stream);
}

}  // namespace ssm
