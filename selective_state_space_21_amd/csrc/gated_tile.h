// What the gated scan's forward and backward kernels share: how a workgroup
// of 1024 threads lies over a tile of tokens x 64 channels, the loads and
// stores of its rows, and how workgroups hand the state on.
//
// A thread owns V neighbouring channels and a run of consecutive tokens: V = 2
// for an even row length (4 bytes of bf16, 8 of fp32; 32 threads to a token's
// channels, so that a wavefront's two halves take two runs), else V = 1.
#pragma once

#include "block_internal.h"
#include "device_math.h"

namespace ssm {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// V channels of one token as stored (Raw), widened to fp32, narrowed back,
// through a buffer resource that ends with the tokens there are: loads behind
// it give zeros, stores behind it are dropped.  Every element is read and
// written once: nontemporal accesses.
constexpr int kNontemporal = 2;
template <typename T, int V> struct Row;
template <> struct Row<uint16_t, 2> {
    using Raw = uint32_t;
    static __device__ __forceinline__ Raw load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
        return __builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, kNontemporal);
    }
    static __device__ __forceinline__ void unpack(const Raw& r, float (&v)[2]) {
        v[0] = __uint_as_float(r << 16);
        v[1] = __uint_as_float(r & 0xffff0000u);
    }
    static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, uint32_t off, const float (&v)[2]) {
        const uint32_t w = (uint32_t)f32_to_bf16_bits(v[0]) | ((uint32_t)f32_to_bf16_bits(v[1]) << 16);
        __builtin_amdgcn_raw_buffer_store_b32(w, r, (int)off, 0, kNontemporal);
    }
};
template <> struct Row<float, 2> {
    using Raw = u32x2;
    static __device__ __forceinline__ Raw load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
        return __builtin_amdgcn_raw_buffer_load_b64(r, (int)off, 0, kNontemporal);
    }
    static __device__ __forceinline__ void unpack(const Raw& r, float (&v)[2]) {
        v[0] = __uint_as_float(r.x);
        v[1] = __uint_as_float(r.y);
    }
    static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, uint32_t off, const float (&v)[2]) {
        __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(v[0]), __float_as_uint(v[1])}, r, (int)off, 0,
                                              kNontemporal);
    }
};
template <> struct Row<uint16_t, 1> {
    using Raw = uint16_t;
    static __device__ __forceinline__ Raw load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
        return __builtin_amdgcn_raw_buffer_load_b16(r, (int)off, 0, kNontemporal);
    }
    static __device__ __forceinline__ void unpack(const Raw& r, float (&v)[1]) { v[0] = bf16_bits_to_f32(r); }
    static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, uint32_t off, const float (&v)[1]) {
        __builtin_amdgcn_raw_buffer_store_b16(f32_to_bf16_bits(v[0]), r, (int)off, 0, kNontemporal);
    }
};
template <> struct Row<float, 1> {
    using Raw = uint32_t;
    static __device__ __forceinline__ Raw load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
        return __builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, kNontemporal);
    }
    static __device__ __forceinline__ void unpack(const Raw& r, float (&v)[1]) { v[0] = __uint_as_float(r); }
    static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, uint32_t off, const float (&v)[1]) {
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[0]), r, (int)off, 0, kNontemporal);
    }
};

// Lane offset of channels that do not exist: behind the end of every resource
// (the ABI refuses rows that would reach it).
constexpr uint32_t kNoChannel = 0x80000000u;

template <int V, int TILE, int THREADS> struct TileShape {
    static constexpr int kLanes = gated::kStrip / V;              // threads to a token's channels
    static constexpr int kWaves = THREADS / 64;
    static constexpr int kRun = TILE * kLanes / THREADS;  // consecutive tokens per thread
    static constexpr bool kPair = kLanes == 32;                   // two runs to a wavefront
    static_assert(kRun * THREADS == TILE * kLanes, "a tile is whole runs");
};

// Rows [t, t + tile) of batch row b of a [B, L, D] tensor, as far as `end`.
template <typename T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t tile_rows(const void* base, const GatedArgs& p, int64_t b,
                                                            int64_t t, int64_t end, int tile) {
    int64_t n = end - t;
    n = n < 0 ? 0 : (n > tile ? tile : n);
    return make_rsrc(static_cast<const T*>(base) + (b * p.L + t) * p.D, (uint32_t)(n * p.D * sizeof(T)));
}

// V consecutive floats of an LDS row
template <int V> __device__ __forceinline__ void lds_put(float* p, const float (&v)[V]) {
    if constexpr (V == 2) *reinterpret_cast<f32x2*>(p) = (f32x2){v[0], v[1]};
    else p[0] = v[0];
}
template <int V> __device__ __forceinline__ void lds_get(const float* p, float (&v)[V]) {
    if constexpr (V == 2) {
        const f32x2 r = *reinterpret_cast<const f32x2*>(p);
        v[0] = r.x; v[1] = r.y;
    } else {
        v[0] = p[0];
    }
}

// tokens of batch row b, between 0 and L
__device__ __forceinline__ int64_t row_tokens(const GatedArgs& p, int64_t b) {
    if (!p.seq_lens) return p.L;
    const int64_t n = p.seq_lens[b];
    return n < 0 ? 0 : (n > p.L ? p.L : n);
}

// ------------------------------------------------------------------ chain
// What the workgroups that walk one strip together share.  A strip's tiles are
// numbered in the order of the walk (right to left in the backward).  A tile
// puts up its map of the state, (P, H): state behind = P * state before + H,
// as soon as it has folded it, and the state behind it once it knows the one
// before; a later tile takes the nearest state that is up and folds the maps
// between there and itself onto it.
//
// * Whichever state it starts from, those are the same fused multiply-adds in
//   the same order, so the result does not depend on timing, bit for bit.
// * Every slot is one word, written once with a device-wide atomic store and
//   zero until then (the call clears them first), so a reader sees nothing or
//   the whole value and no other ordering is needed.  A zero P or state is put
//   up as -0 (its bits are not zero) and counts as the same number.
// * Workgroups draw a strip's tiles in order from a counter, one or two ahead,
//   and finish them in that order.  A tile waits for earlier ones only, and of
//   the unfinished tiles that were drawn the earliest waits for nothing: its
//   workgroup is running and on that tile, whatever else the GPU runs.  So
//   every wait ends.  (Two calls at once over one workspace break that, and the
//   rule that forbids it; a wait is given up after some seconds then, with NaN
//   for the state, rather than never.)
struct Chain {
    uint32_t* ticket;     // the strip's counter
    uint64_t* maps;       // [tiles][64], P in the low half; kBack - 1 empty tiles in front
    uint32_t* states;     // [tiles][64], the same
};

__device__ __forceinline__ Chain chain_of(void* base, const GatedPlan& pl, int64_t strip) {
    char* p = static_cast<char*>(base);
    const int64_t head = gated::chain_head(pl.strips), n = gated::chain_slots(pl.tiles);
    const int64_t first = strip * n + (gated::kBack - 1) * gated::kStrip;
    return {reinterpret_cast<uint32_t*>(p) + strip, reinterpret_cast<uint64_t*>(p + head) + first,
            reinterpret_cast<uint32_t*>(p + head + pl.strips * n * 8) + first};
}

__device__ __forceinline__ uint32_t chain_bits(float v) {
    return v == 0.0f ? 0x80000000u : __float_as_uint(v);
}
__device__ __forceinline__ int chain_draw(const Chain& c) {
    return (int)__hip_atomic_fetch_add(c.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void chain_put_map(const Chain& c, int tile, uint32_t lane, float P, float H) {
    __hip_atomic_store(c.maps + (int64_t)tile * gated::kStrip + lane,
                       (uint64_t)chain_bits(P) | ((uint64_t)__float_as_uint(H) << 32), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void chain_put_state(const Chain& c, int tile, uint32_t lane, float h) {
    __hip_atomic_store(c.states + (int64_t)tile * gated::kStrip + lane, chain_bits(h), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
}

// The state before tile `pos` >= 1 of this lane's channel, by one wavefront.
__device__ __forceinline__ float chain_state_before(const Chain& c, int pos, uint32_t lane) {
    constexpr int kBack = gated::kBack;
    constexpr int kPolls = 1 << 22;       // of about two microseconds each
    const uint32_t* states = c.states + (int64_t)(pos - 1) * gated::kStrip + lane;
    const uint64_t* maps = c.maps + (int64_t)(pos - 1) * gated::kStrip + lane;
    float h = 0.0f;
    bool known = false;
    for (int polls = 0; !known && polls < kPolls; ++polls) {
        uint32_t st[kBack];
        uint64_t mp[kBack];
#pragma unroll
        for (int k = 0; k < kBack; ++k) {             // in front of the first tile there are empty slots
            st[k] = __hip_atomic_load(states - k * gated::kStrip, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            mp[k] = __hip_atomic_load(maps - k * gated::kStrip, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
#pragma unroll
        for (int k = kBack - 1; k >= 0; --k) {
            const bool up = st[k] != 0u;
            const float next = fmaf(__uint_as_float((uint32_t)mp[k]), h, __uint_as_float((uint32_t)(mp[k] >> 32)));
            h = up ? __uint_as_float(st[k]) : next;
            known = up || (known && mp[k] != 0ull);
        }
        if (!known) __builtin_amdgcn_s_sleep(1);
    }
    return known ? h + 0.0f : __builtin_nanf("");      // -0 is 0 again
}

}  // namespace ssm
