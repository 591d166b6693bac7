// Linear attention with a decay for each head, for gfx950: the chunked
// recurrence behind the forward call and all three gradients.
//
// Per batch row and head, S_t = e^{g_t} S_{t-1} + k_t v_t^T and o_t = q_t^T S_t.
// With G the inclusive sum of g inside a chunk of C tokens and S the state
// that enters it,
//   o_i = sum_{j<=i} (q_i . k_j) e^{G_i - G_j} v_j + e^{G_i} q_i^T S
//   S  <- e^{G_C} S + sum_j e^{G_C - G_j} k_j v_j^T
// The gradients are the same run with other tensors in the roles:
//   dq: q <- do, k <- v, v <- k, the state transposed;
//   dv: q <- k, k <- q, v <- do and dk: q <- v, k <- do, v <- q, from the last
//   token to the first (there token t enters with g of token t + 1).
//
// Work mapping: a workgroup of four wavefronts walks the chunks of one head
// (or of one segment of it) with 64 columns of the state, 16 to a wavefront,
// in fp32 matrix accumulators.  Every wavefront forms the outputs of all C
// tokens for its columns, so the state never leaves its registers: the
// accumulators' rows are laid out so that they are the next product's operand
// as they stand (below).  The scores are shared through LDS.  The next chunk's
// rows are on their way while this one is computed.
//
// Products are v_mfma_f32_16x16x32_bf16, or eight v_mfma_f32_16x16x4_f32 for
// fp32 (element j of every lane's eight makes one of them).  Lane l with
// c = l % 16, g = l / 16: A holds row c, k = 8g..8g+7; B column c, the same k;
// the result rows 4g..4g+3 of column c.  Outputs are formed transposed
// (columns are tokens), so a lane stores four neighbouring elements.  State
// tile (kk, u) holds key rows 32kk + 8a + 4u + b as its rows 4a + b: lane g
// then has rows 32kk + 8g + 0..7 of its column in tiles u = 0, 1, which is the
// A operand of the product with the queries.
//
// Rounding: exponent sums are fp64 and kept as two floats, differences are
// taken of those.  For bf16 the decayed values of the state update are split
// in two bf16 halves (the fp32 state is then off by 2^-18 a term, not 2^-9).
// The scores and the state as an operand are rounded to one bf16 where only
// bf16 outputs come of them, like the outputs themselves, and split too where
// the decay's gradient, an fp32 sum over tokens, is formed (`split`).
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "device_math.h"
#include "lane_ops.h"
#include "linear_internal.h"

namespace ssm {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef short i16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 512, kWaves = 8;
constexpr int kGroups = linear::kColumns / 16;    // column groups: a wavefront of each half of the key rows
constexpr uint32_t kNoOffset = 0x80000000u;      // past every resource's end: loads give zeros
constexpr uint32_t kRecords = 0x7ffffff0u;
constexpr float kMinLog2 = -150.0f;              // 2^-150 is zero in fp32

// Operands and products of a storage type.
template <typename T> struct Mat;

template <> struct Mat<uint16_t> {
    using Frag = bf16x8;
    static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    // eight neighbouring elements of a row
    static __device__ __forceinline__ Frag along(const uint16_t* p) { return *reinterpret_cast<const Frag*>(p); }
    // rows row..row+7 of this lane's column: the 16 columns are first + step * a + b for a, b < 4.
    // A transposing read takes 4 columns of one row from each lane (row r = i / 4, block a = i % 4)
    // and gives lane i column i of the four rows.
    static __device__ __forceinline__ Frag down(const uint16_t* tile, int stride, int row, int first, int step, int i) {
        const uint16_t* p = tile + (row + i / 4) * stride + first + step * (i % 4);
        const i16x4 x = read4(p), y = read4(p + 4 * stride);
        i16x8 z;
#pragma unroll
        for (int j = 0; j < 4; ++j) z[j] = x[j], z[j + 4] = y[j];
        return __builtin_bit_cast(Frag, z);
    }
    static __device__ __forceinline__ i16x4 read4(const uint16_t* p) {
        typedef __attribute__((address_space(3))) i16x4 Shared;
        return __builtin_amdgcn_ds_read_tr16_b64_v4i16((Shared*)(uintptr_t)p);
    }
    static __device__ __forceinline__ f32x8 widen(Frag a) { return __builtin_convertvector(a, f32x8); }
    static __device__ __forceinline__ Frag high(f32x8 x) { return __builtin_convertvector(x, Frag); }
};

template <> struct Mat<float> {
    using Frag = f32x8;
    static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c) {
#pragma unroll
        for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
        return c;
    }
    static __device__ __forceinline__ Frag along(const float* p) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(p), y = *reinterpret_cast<const f32x4*>(p + 4);
        return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    static __device__ __forceinline__ Frag down(const float* tile, int stride, int row, int first, int step, int i) {
        const float* p = tile + row * stride + first + step * (i / 4) + i % 4;
        Frag z;
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = p[j * stride];
        return z;
    }
    static __device__ __forceinline__ f32x8 widen(Frag a) { return a; }
    static __device__ __forceinline__ Frag high(f32x8 x) { return x; }
};

// Inclusive sums over the 64 lanes.
__device__ __forceinline__ double shifted(double x, int row_shr) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    int lo = (int)(uint32_t)b, hi = (int)(uint32_t)(b >> 32);
    switch (row_shr) {
        case 1: lo = __builtin_amdgcn_update_dpp(0, lo, 0x111, 0xf, 0xf, true);
                hi = __builtin_amdgcn_update_dpp(0, hi, 0x111, 0xf, 0xf, true); break;
        case 2: lo = __builtin_amdgcn_update_dpp(0, lo, 0x112, 0xf, 0xf, true);
                hi = __builtin_amdgcn_update_dpp(0, hi, 0x112, 0xf, 0xf, true); break;
        case 4: lo = __builtin_amdgcn_update_dpp(0, lo, 0x114, 0xf, 0xf, true);
                hi = __builtin_amdgcn_update_dpp(0, hi, 0x114, 0xf, 0xf, true); break;
        default: lo = __builtin_amdgcn_update_dpp(0, lo, 0x118, 0xf, 0xf, true);
                 hi = __builtin_amdgcn_update_dpp(0, hi, 0x118, 0xf, 0xf, true); break;
    }
    return __builtin_bit_cast(double, (uint64_t)(uint32_t)lo | (uint64_t)(uint32_t)hi << 32);
}
__device__ __forceinline__ double from_lane(double x, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)lo | (uint64_t)hi << 32);
}
__device__ __forceinline__ double wave_sums(double x, int lane) {
#pragma unroll
    for (int d = 1; d < 16; d *= 2) x += shifted(x, d);
    const double r0 = from_lane(x, 15), r1 = r0 + from_lane(x, 31), r2 = r1 + from_lane(x, 47);
    return x + (lane < 16 ? 0.0 : lane < 32 ? r0 : lane < 48 ? r1 : r2);
}

// An fp32 operand as a sum of N of the storage type, largest first (fp32 is its own).
template <typename T, int N>
struct Terms {
    static constexpr int kN = sizeof(T) == 2 ? N : 1;
    typename Mat<T>::Frag term[kN];
    __device__ __forceinline__ explicit Terms(f32x8 x) {
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            term[n] = Mat<T>::high(x);
            if (n + 1 < kN) x -= Mat<T>::widen(term[n]);
        }
    }
};

template <typename T, int KD, bool STATES, int TERMS>
struct Lds {
    static constexpr int C = linear::chunk(sizeof(T) == 2);
    static constexpr int E = 16 / sizeof(T);                 // elements of a 16-byte piece
    static constexpr int kKey = KD + E, kValue = linear::kColumns + E, kScore = C + E;   // row strides
    alignas(16) T K[C * kKey];
    alignas(16) T V[C * kValue];
    alignas(16) T Q[STATES ? E : C * kKey];
    alignas(16) T P[STATES ? 1 : TERMS][STATES ? E : C * kScore];   // scores, in terms
    alignas(16) f32x4 other[STATES ? 1 : kWaves * C / 32 * 64];     // outputs' parts that the other half finishes
    alignas(16) float hi[C];                                 // log2 of the decay since the chunk's start
    alignas(16) float lo[C];                                 // as two floats
    alignas(16) float since[C];                              // that decay
    alignas(16) float until[C];                              // the decay until the chunk's end (times `fresh`)
    float whole[4];                                          // the chunk's decay
};

// A chunk's rows as 16-byte pieces, spread over the workgroup.
template <typename T, int WIDTH>
struct Rows {
    static constexpr int C = linear::chunk(sizeof(T) == 2), E = 16 / sizeof(T);
    static constexpr int PER_ROW = WIDTH / E, N = C * PER_ROW / kThreads;
    static_assert(C * PER_ROW % kThreads == 0, "whole pieces for every thread");
    u32x4 piece[N];
    // `n` rows from `base` on, `row` elements apart, the first `width` elements of each
    __device__ __forceinline__ void fetch(const T* base, int64_t row, int n, int width, int tid) {
        const __amdgpu_buffer_rsrc_t r = make_rsrc(base, kRecords);
#pragma unroll
        for (int m = 0; m < N; ++m) {
            const int p = tid + m * kThreads, t = p / PER_ROW, c = p % PER_ROW * E;
            const uint32_t at = t < n && c < width ? (uint32_t)((t * (int)row + c) * (int)sizeof(T)) : kNoOffset;
            piece[m] = __builtin_amdgcn_raw_buffer_load_b128(r, (int)at, 0, 0);
        }
    }
    __device__ __forceinline__ void stage(T* tile, int stride, int n, bool reversed, int tid) {
#pragma unroll
        for (int m = 0; m < N; ++m) {
            const int p = tid + m * kThreads, t = p / PER_ROW, c = p % PER_ROW * E;
            const int to = reversed && t < n ? n - 1 - t : t;
            *reinterpret_cast<u32x4*>(&tile[to * stride + c]) = piece[m];
        }
    }
};

// The half that finishes output tile `it`: 0 1 1 0, so both have as many blocks of keys.
__device__ __forceinline__ constexpr int half_of(int it) { return (it ^ it >> 1) & 1; }

template <typename T, int KD, bool STATES, bool SPLIT>
__global__ __launch_bounds__(kThreads, 2) void linear_chunks(LinearRun run) {
    using M = Mat<T>;
    using Frag = typename M::Frag;
    constexpr int TERMS = SPLIT && sizeof(T) == 2 ? 3 : 1;   // of the scores and of the state as an operand
    using L = Lds<T, KD, STATES, TERMS>;
    constexpr int C = L::C, RT = C / 16, KB = C / 32, KK = KD / 64;   // KK: of this half
    constexpr int TILES = RT * (RT + 1) / 2;                 // score tiles on and below the diagonal
    __shared__ L s;

    const LinearJob& job = run.job[blockIdx.y];
    const int ctiles = (job.vd + linear::kColumns - 1) / linear::kColumns;
    // neighbouring ids go to the eight XCDs in turn: the column tiles of a head stay on one, and share its L2
    const int64_t id = blockIdx.x / 8, unit = id / ctiles * 8 + blockIdx.x % 8;
    const int tile = (int)(id % ctiles);
    if (unit >= run.B * run.H * run.segments) return;
    const int seg = (int)(unit % run.segments);
    const int64_t bh = unit / run.segments, b = bh / run.H;
    const int h = (int)(bh % run.H);
    const int tid = threadIdx.x, lane = tid % 64, i = lane % 16, g = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
    const int group = wave % kGroups, half = wave / kGroups, k0 = half * KK;
    const bool rev = job.reversed;
    const int kd = job.kd, vd = job.vd;
    const int col0 = tile * linear::kColumns;                // the workgroup's columns
    const int col = col0 + 16 * group;                       // the wavefront's
    const bool live = col < vd;

    int64_t len = run.L;
    if (run.seq_lens) {
        const int64_t given = run.seq_lens[b];
        len = given < 0 ? 0 : given < len ? given : len;
    }
    const int64_t from = seg * run.seg_tokens;
    const int64_t last = from + run.seg_tokens < run.L ? from + run.seg_tokens : run.L;
    const int64_t to = last < len ? last : len;
    const int64_t chunks = to > from ? (to - from + C - 1) / C : 0;

    // rows of token t: base + t * row
    const T* qb = STATES ? nullptr
                         : static_cast<const T*>(job.q) + b * run.L * job.q_row + (int64_t)(h / job.q_per) * kd;
    const T* kb = static_cast<const T*>(job.k) + b * run.L * job.k_row + (int64_t)(h / job.k_per) * kd;
    const T* vb = static_cast<const T*>(job.v) + b * run.L * job.v_row + (int64_t)(h / job.v_per) * vd + col0;
    const float* gb = run.by_head ? run.g + h : run.g + b * run.L * run.H + h;

    Rows<T, KD> qr, kr;
    Rows<T, linear::kColumns> vr;
    float gr = 0.0f;
    // tokens lo .. lo + n - 1 make chunk c
    const auto place = [&](int64_t c, int64_t& lo, int& n) {
        const int64_t left = (to - from) - c * C;
        n = left < C ? (int)left : C;
        lo = rev ? to - c * C - n : from + c * C;
    };
    const auto fetch = [&](int64_t c) {
        int64_t lo;
        int n;
        place(c, lo, n);
        if constexpr (!STATES) qr.fetch(qb + lo * job.q_row, job.q_row, n, kd, tid);
        kr.fetch(kb + lo * job.k_row, job.k_row, n, kd, tid);
        vr.fetch(vb + lo * job.v_row, job.v_row, n, vd - col0, tid);
        gr = 0.0f;
        if (wave == 0 && lane < n) {
            const int64_t t = rev ? lo + n - lane : lo + lane;       // reversed: the g of the token behind
            if (t < len) gr = run.by_head ? gb[0] : gb[t * run.H];
        }
    };
    if (chunks > 0) fetch(0);

    f32x4 state[KK][2];
    {
        const float* p = job.state_in ? job.state_in + bh * job.in_head + seg * job.in_seg : nullptr;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 32 * (k0 + kk) + 8 * g + 4 * u + r;
                    state[kk][u][r] = p && live && row < kd ? p[(int64_t)row * job.sk + (int64_t)(col + i) * job.sv] : 0.0f;
                }
    }
    if constexpr (!STATES) {
        // the score tiles right of the diagonal that a block of 32 keys reaches are zero throughout
        for (int e = tid; e < RT / 2 * 256; e += kThreads) {
            const int at = (32 * (e / 256) + e % 256 / 16) * L::kScore + 32 * (e / 256) + 16 + e % 16;
#pragma unroll
            for (int n = 0; n < TERMS; ++n) s.P[n][at] = T(0);
        }
    }

    double seg_decay = 0.0;
    for (int64_t c = 0; c < chunks; ++c) {
        int64_t lo;
        int n;
        place(c, lo, n);
        lds_barrier();                                       // the last chunk's rows have been read
        if constexpr (!STATES) qr.stage(s.Q, L::kKey, n, rev, tid);
        kr.stage(s.K, L::kKey, n, rev, tid);
        vr.stage(s.V, L::kValue, n, rev, tid);
        if (wave == 0) {
            double x = (double)gr * 1.4426950408889634074;
            if (x < (double)kMinLog2) x = (double)kMinLog2;          // a NaN stays
            const double sum = wave_sums(x, lane), all = from_lane(sum, 63);
            if (lane < C) {
                const float hi = (float)sum;
                s.hi[lane] = hi;
                s.lo[lane] = (float)(sum - (double)hi);
                s.since[lane] = fast_exp2(hi) * job.outer;
                s.until[lane] = fast_exp2((float)(all - sum)) * job.fresh;
            }
            if (lane == 0) s.whole[0] = fast_exp2((float)all);
            seg_decay += all;
        }
        lds_barrier();
        if (c + 1 < chunks) fetch(c + 1);

        f32x4 out[RT];
        if constexpr (!STATES) {
            // scores, transposed: a lane has four keys of one query
#pragma unroll
            for (int m = 0; m < (TILES + kWaves - 1) / kWaves; ++m) {
                const int idx = kWaves - 1 - wave + m * kWaves;
                if (idx >= TILES) break;
                const int it = (idx >= 1) + (idx >= 3) + (idx >= 6), jt = idx - it * (it + 1) / 2;
                f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int kk = 0; kk < KD / 32; ++kk)
                    acc = M::mma(M::along(&s.K[(16 * jt + i) * L::kKey + 32 * kk + 8 * g]),
                                 M::along(&s.Q[(16 * it + i) * L::kKey + 32 * kk + 8 * g]), acc);
                const int query = 16 * it + i, key = 16 * jt + 4 * g;
                const float hq = s.hi[query], lq = s.lo[query];
                const f32x4 hk = *reinterpret_cast<const f32x4*>(&s.hi[key]);
                const f32x4 lk = *reinterpret_cast<const f32x4*>(&s.lo[key]);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float e = fast_exp2((hq - hk[r]) + (lq - lk[r])) * job.inner;
                    acc[r] = key + r <= query ? acc[r] * e : 0.0f;
                }
#pragma unroll
                for (int n2 = 0; n2 < TERMS; ++n2) {
                    T* p = &s.P[n2][query * L::kScore + key];
                    if constexpr (sizeof(T) == 4) {
                        *reinterpret_cast<f32x4*>(p) = acc;
                    } else {
                        const bf16x4 x = __builtin_convertvector(acc, bf16x4);
                        *reinterpret_cast<bf16x4*>(p) = x;
                        acc -= __builtin_convertvector(x, f32x4);
                    }
                }
            }
            // the entering state's part
#pragma unroll
            for (int it = 0; it < RT; ++it) out[it] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
                const Terms<T, TERMS> x(__builtin_shufflevector(state[kk][0], state[kk][1], 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
                for (int it = 0; it < RT; ++it) {
                    const Frag q = M::along(&s.Q[(16 * it + i) * L::kKey + 32 * (k0 + kk) + 8 * g]);
#pragma unroll
                    for (int n2 = 0; n2 < TERMS; ++n2) out[it] = M::mma(x.term[n2], q, out[it]);
                }
            }
#pragma unroll
            for (int it = 0; it < RT; ++it)
                if (half_of(it) != half) s.other[(wave * (RT / 2) + it / 2) * 64 + lane] = out[it];
            lds_barrier();                                   // the scores and the other half's parts are there
        }

        const float whole = s.whole[0];
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) state[kk][0] *= whole, state[kk][1] *= whole;
        Frag v[KB];
#pragma unroll
        for (int b2 = 0; b2 < KB; ++b2) v[b2] = M::down(s.V, L::kValue, 32 * b2 + 8 * g, 16 * group, 4, i);
#pragma unroll
        for (int b2 = 0; b2 < KB; ++b2) {
            const f32x4 u0 = *reinterpret_cast<const f32x4*>(&s.until[32 * b2 + 8 * g]);
            const f32x4 u1 = *reinterpret_cast<const f32x4*>(&s.until[32 * b2 + 8 * g + 4]);
            const Terms<T, 3> w(M::widen(v[b2]) * __builtin_shufflevector(u0, u1, 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
            for (int kk = 0; kk < KK; ++kk)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const Frag k = M::down(s.K, L::kKey, 32 * b2 + 8 * g, 32 * (k0 + kk) + 4 * u, 8, i);
#pragma unroll
                    for (int n2 = 0; n2 < Terms<T, 3>::kN; ++n2) state[kk][u] = M::mma(k, w.term[n2], state[kk][u]);
                }
        }

        if constexpr (!STATES) {
#pragma unroll
            for (int it = 0; it < RT; ++it) {
                if (half_of(it) != half) continue;
                // wavefront-uniform, and the indices are constants
                f32x4 x = out[it] + s.other[((wave ^ kGroups) * (RT / 2) + it / 2) * 64 + lane];
                const int row = 16 * it + i;
                x *= s.since[row];
#pragma unroll
                for (int b2 = 0; b2 <= it / 2; ++b2) {
#pragma unroll
                    for (int n2 = 0; n2 < TERMS; ++n2)
                        x = M::mma(v[b2], M::along(&s.P[n2][row * L::kScore + 32 * b2 + 8 * g]), x);
                }
                if (!live) continue;
                const int64_t t = rev ? lo + n - 1 - row : lo + row;
                const int64_t at = b * run.L + t;            // of the token
                if (row < n) {
                    const int64_t to2 = (at * run.H + h) * vd + col + 4 * g;
                    if (sizeof(T) == 4 || job.out_f32)
                        *reinterpret_cast<f32x4*>(static_cast<float*>(job.out) + to2) = x;
                    else
                        *reinterpret_cast<bf16x4*>(static_cast<uint16_t*>(job.out) + to2) = __builtin_convertvector(x, bf16x4);
                }
                if (job.dots) {
                    float sum = 0.0f;
                    if (row < n) {
                        const T* y = static_cast<const T*>(job.dot_with) + at * job.dot_row +
                                     (int64_t)(h / job.dot_per) * vd + col + 4 * g;
#pragma unroll
                        for (int r = 0; r < 4; ++r) sum = fmaf(x[r], Elem<T>::load(y, r), sum);
                    }
                    sum += __shfl_xor(sum, 16);
                    sum += __shfl_xor(sum, 32);
                    if (g == 0 && row < n)
                        job.dots[((int64_t)(tile * kGroups + group) * run.B * run.H + bh) * run.L + t] = sum;
                }
            }
        }
    }

    if constexpr (!STATES) {
        if (job.zero_tail) {
            const int width = vd - col0 < linear::kColumns ? vd - col0 : linear::kColumns;
            const int64_t first = from > len ? from : len;
            for (int64_t t = first + wave; t < last; t += kWaves) {
                const int64_t at = ((b * run.L + t) * run.H + h) * vd + col0 + lane;
                if (lane < width) {
                    if (sizeof(T) == 4 || job.out_f32) static_cast<float*>(job.out)[at] = 0.0f;
                    else static_cast<uint16_t*>(job.out)[at] = 0;
                }
            }
        }
    }
    float* p = nullptr;
    float by = 1.0f;
    if constexpr (STATES) {
        p = run.seg_state[blockIdx.y] + unit * kd * vd;
        if (tile == 0 && tid == 0) run.seg_decay[blockIdx.y][unit] = (float)seg_decay;
    } else if (job.state_out && seg == (rev ? 0 : run.segments - 1)) {
        p = job.state_out + bh * job.out_head;
        if (job.decay_out && len > 0) {
            const float x = gb[0] * kLog2e;
            by = fast_exp2(x < kMinLog2 ? kMinLog2 : x);
        }
    }
    if (p && live) {
        const int64_t sk = STATES ? vd : job.sk, sv = STATES ? 1 : job.sv;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 32 * (k0 + kk) + 8 * g + 4 * u + r;
                    if (row < kd) p[row * sk + (col + i) * sv] = state[kk][u][r] * by;
                }
    }
}

template <typename T, int KD>
hipError_t launch_width(const LinearRun& r, bool states_only, hipStream_t stream) {
    int tiles = 0;
    for (int j = 0; j < r.jobs; ++j) {
        const int n = (r.job[j].vd + linear::kColumns - 1) / linear::kColumns;
        tiles = n > tiles ? n : tiles;
    }
    // jobs of fewer tiles leave the last workgroups without a unit
    const int64_t units = (r.B * r.H * r.segments + 7) / 8 * 8;
    const dim3 grid((unsigned)(units * tiles), (unsigned)r.jobs);
    if (states_only) linear_chunks<T, KD, true, false><<<grid, kThreads, 0, stream>>>(r);
    else if (sizeof(T) == 2 && r.split) linear_chunks<T, KD, false, sizeof(T) == 2><<<grid, kThreads, 0, stream>>>(r);
    else linear_chunks<T, KD, false, false><<<grid, kThreads, 0, stream>>>(r);
    return hipGetLastError();
}

// The state entering every segment: a thread folds four elements of one head's
// states over the segments, eight loads ahead of the sums.
__global__ __launch_bounds__(256) void linear_join(LinearJoin j) {
    const int per = j.size / 4;
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (at >= j.heads * per) return;
    const int64_t head = at / per;
    const int e = (int)(at % per) * 4;
    f32x4 carry = {0.0f, 0.0f, 0.0f, 0.0f};
    if (j.first)
#pragma unroll
        for (int r = 0; r < 4; ++r) carry[r] = j.first[head * j.size + e + r];
    for (int n0 = 0; n0 < j.segments; n0 += 8) {
        f32x4 own[8];
        float decay[8];
#pragma unroll
        for (int m = 0; m < 8; ++m)
            if (n0 + m < j.segments) {
                const int64_t s = head * j.segments + (j.reversed ? j.segments - 1 - n0 - m : n0 + m);
                own[m] = *reinterpret_cast<const f32x4*>(j.seg_state + s * j.size + e);
                decay[m] = j.seg_decay[s];
            }
#pragma unroll
        for (int m = 0; m < 8; ++m)
            if (n0 + m < j.segments) {
                const int64_t s = head * j.segments + (j.reversed ? j.segments - 1 - n0 - m : n0 + m);
                *reinterpret_cast<f32x4*>(j.seg_state + s * j.size + e) = carry;
                carry = carry * fast_exp2(decay[m]) + own[m];
            }
    }
}

// The decay's gradient over one segment of a head: from its right end, where
// dg of the token behind is <D, S> of the two states there, the differences
// q . dq - k . dk add up token by token (in fp64: the sums of the two nearly
// cancel where the memory is long).
__global__ __launch_bounds__(256) void linear_decay_grad(LinearDecayGrad d) {
    __shared__ double part[4];
    __shared__ double total[4];
    const int64_t unit = blockIdx.x, bh = unit / d.segments;
    const int seg = (int)(unit % d.segments);
    const int64_t b = bh / d.H;
    const int h = (int)(bh % d.H);
    const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
    int64_t len = d.L;
    if (d.seq_lens) {
        const int64_t given = d.seq_lens[b];
        len = given < 0 ? 0 : given < len ? given : len;
    }
    const int64_t from = seg * d.seg_tokens;
    const int64_t last = from + d.seg_tokens < d.L ? from + d.seg_tokens : d.L;
    const int64_t to = last < len ? last : len;

    const bool end = seg == d.segments - 1;
    const float* S = end ? d.S_last + bh * d.size : d.S + (unit + 1) * d.size;
    const float* D = d.segments > 1 ? d.D + unit * d.size : d.D_last ? d.D_last + bh * d.size : nullptr;
    double sum = 0.0;
    if (D && to > from) {
        for (int e = tid * 4; e < d.size; e += 1024) {
            float x = 0.0f;
#pragma unroll
            for (int r = 0; r < 4; ++r) x = fmaf(S[e + r], D[e + r], x);
            sum += (double)x;
        }
    }
#pragma unroll
    for (int m = 32; m >= 1; m /= 2) sum += __shfl_xor(sum, m);
    if (lane == 0) part[wave] = sum;
    __syncthreads();
    double carry = part[0] + part[1] + part[2] + part[3];
    if (to < len) {                                          // the token behind decays what D brings
        const float x = d.g[d.by_head ? h : (b * d.L + to) * d.H + h] * kLog2e;
        carry *= (double)fast_exp2(x < kMinLog2 ? kMinLog2 : x);
    }

    double all = 0.0;                                       // of this thread's tokens
    for (int64_t hi = to; hi > from; hi -= 256) {
        const int64_t t = hi - 1 - tid;                      // thread 0 has the last token
        double x = 0.0;
        if (t >= from) {
            for (int n = 0; n < d.q_tiles; ++n) x += (double)d.dot_q[((int64_t)n * d.B * d.H + bh) * d.L + t];
            for (int n = 0; n < d.k_tiles; ++n) x -= (double)d.dot_k[((int64_t)n * d.B * d.H + bh) * d.L + t];
        }
        x = wave_sums(x, lane);
        __syncthreads();
        if (lane == 63) total[wave] = x;
        __syncthreads();
        for (int w = 0; w < wave; ++w) x += total[w];
        x += carry;
        carry += total[0] + total[1] + total[2] + total[3];
        if (t >= from) {
            all += x;
            if (d.dg) d.dg[(b * d.L + t) * d.H + h] = (float)x;
        }
    }
    if (d.dg)
        for (int64_t t = (from > len ? from : len) + tid; t < last; t += 256) d.dg[(b * d.L + t) * d.H + h] = 0.0f;
    if (d.part) {
#pragma unroll
        for (int m = 32; m >= 1; m /= 2) all += __shfl_xor(all, m);
        __syncthreads();
        if (lane == 0) part[wave] = all;
        __syncthreads();
        if (tid == 0) d.part[(b * d.segments + seg) * d.H + h] = (float)(part[0] + part[1] + part[2] + part[3]);
    }
}

// Gradients of rows that several heads share: their heads' sum, in order.
__global__ __launch_bounds__(256) void linear_group_sum(LinearGroupSum s) {
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    const int64_t row = s.G * s.width;
    if (at >= s.rows * row) return;
    const int64_t t = at / row;
    const int64_t grp = at % row / s.width;
    const int c = (int)(at % s.width);
    const int per = (int)(s.H / s.G);
    const float* p = s.part + (t * s.H + grp * per) * s.width + c;
    f32x4 x = *reinterpret_cast<const f32x4*>(p);
    for (int n = 1; n < per; ++n) x += *reinterpret_cast<const f32x4*>(p + (int64_t)n * s.width);
    if (s.bf16) {
        uint16_t y[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) y[r] = f32_to_bf16_bits(x[r]);
        *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(s.out) + at) =
            u32x2{y[0] | (uint32_t)y[1] << 16, y[2] | (uint32_t)y[3] << 16};
    } else {
        *reinterpret_cast<f32x4*>(static_cast<float*>(s.out) + at) = x;
    }
}

}  // namespace

hipError_t launch_linear_run(const LinearRun& r, bool states_only, hipStream_t stream) {
    const int kd = r.job[0].kd;
    if (r.bf16)
        return kd <= 64    ? launch_width<uint16_t, 64>(r, states_only, stream)
               : kd <= 128 ? launch_width<uint16_t, 128>(r, states_only, stream)
                           : launch_width<uint16_t, 256>(r, states_only, stream);
    return kd <= 64    ? launch_width<float, 64>(r, states_only, stream)
           : kd <= 128 ? launch_width<float, 128>(r, states_only, stream)
                       : launch_width<float, 256>(r, states_only, stream);
}

hipError_t launch_linear_join(const LinearJoin& j, hipStream_t stream) {
    const int64_t n = j.heads * (j.size / 4);
    linear_join<<<dim3((unsigned)((n + 255) / 256)), 256, 0, stream>>>(j);
    return hipGetLastError();
}

hipError_t launch_linear_decay_grad(const LinearDecayGrad& d, hipStream_t stream) {
    linear_decay_grad<<<dim3((unsigned)(d.B * d.H * d.segments)), 256, 0, stream>>>(d);
    return hipGetLastError();
}

hipError_t launch_linear_group_sum(const LinearGroupSum& s, hipStream_t stream) {
    const int64_t n = s.rows * s.G * (s.width / 4);
    linear_group_sum<<<dim3((unsigned)((n + 255) / 256)), 256, 0, stream>>>(s);
    return hipGetLastError();
}

}  // namespace ssm
