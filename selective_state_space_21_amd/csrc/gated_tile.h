// What the gated scan's forward and backward kernels share: how a workgroup
// of 512 threads lies over a tile of 128 tokens x 64 channels, and the loads
// and stores of its rows.
//
// A thread owns V neighbouring channels and R consecutive tokens, 16 elements
// either way: V = 4 where the row length allows whole vectors (8 bytes of
// bf16, 16 of fp32, 16 threads to a row's 64 channels, 32 groups of 4 tokens),
// else V = 1 (8 groups of 16 tokens).
#pragma once

#include "block_internal.h"
#include "device_math.h"

namespace ssm {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// V channels of one token as stored (Raw), widened to fp32, narrowed back.
// Every element is read and written once: nontemporal accesses.
template <typename T, int V> struct Row;
template <> struct Row<uint16_t, 4> {
    using Raw = u32x2;
    static __device__ __forceinline__ Raw load(const uint16_t* p) {
        return __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p));
    }
    static __device__ __forceinline__ Raw zero() { return Raw{0, 0}; }
    static __device__ __forceinline__ void unpack(const Raw& r, float (&v)[4]) {
        v[0] = __uint_as_float(r.x << 16);
        v[1] = __uint_as_float(r.x & 0xffff0000u);
        v[2] = __uint_as_float(r.y << 16);
        v[3] = __uint_as_float(r.y & 0xffff0000u);
    }
    static __device__ __forceinline__ void store(uint16_t* p, const float (&v)[4]) {
        const u32x2 r = {(uint32_t)f32_to_bf16_bits(v[0]) | ((uint32_t)f32_to_bf16_bits(v[1]) << 16),
                         (uint32_t)f32_to_bf16_bits(v[2]) | ((uint32_t)f32_to_bf16_bits(v[3]) << 16)};
        __builtin_nontemporal_store(r, reinterpret_cast<u32x2*>(p));
    }
};
template <> struct Row<float, 4> {
    using Raw = f32x4;
    static __device__ __forceinline__ Raw load(const float* p) {
        return __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p));
    }
    static __device__ __forceinline__ Raw zero() { return Raw{0.0f, 0.0f, 0.0f, 0.0f}; }
    static __device__ __forceinline__ void unpack(const Raw& r, float (&v)[4]) {
        v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w;
    }
    static __device__ __forceinline__ void store(float* p, const float (&v)[4]) {
        __builtin_nontemporal_store((f32x4){v[0], v[1], v[2], v[3]}, reinterpret_cast<f32x4*>(p));
    }
};
template <typename T> struct Row<T, 1> {
    using Raw = T;
    static __device__ __forceinline__ Raw load(const T* p) { return __builtin_nontemporal_load(p); }
    static __device__ __forceinline__ Raw zero() { return Raw(0); }
    static __device__ __forceinline__ void unpack(const Raw& r, float (&v)[1]) {
        v[0] = Elem<T>::load(&r, 0);
    }
    static __device__ __forceinline__ void store(T* p, const float (&v)[1]) {
        T r;
        Elem<T>::store(&r, 0, v[0]);
        __builtin_nontemporal_store(r, p);
    }
};

template <int V> struct TileShape {
    static constexpr int kLanes = gated::kStrip / V;              // threads to a token's channels
    static constexpr int kGroups = gated::kThreads / kLanes;      // token groups
    static constexpr int kRun = gated::kTile / kGroups;           // consecutive tokens per thread
    static_assert(kRun * kGroups == gated::kTile, "a tile is whole groups");
};

// V consecutive floats of an LDS row
template <int V> __device__ __forceinline__ void lds_put(float* p, const float (&v)[V]) {
    if constexpr (V == 4) *reinterpret_cast<f32x4*>(p) = (f32x4){v[0], v[1], v[2], v[3]};
    else p[0] = v[0];
}
template <int V> __device__ __forceinline__ void lds_get(const float* p, float (&v)[V]) {
    if constexpr (V == 4) {
        const f32x4 r = *reinterpret_cast<const f32x4*>(p);
        v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w;
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

}  // namespace ssm
