// Moves between the slots of a state pool as one assignment:
// pool[:, dst[i]] <- what pool[:, src[i]] held before the call (zeros for a
// negative src), for any lists: slots may be read and written by the same
// call, and chains and cycles come out right.
//
// A workgroup owns a range of bytes of every slot of one layer, reads it from
// all sources into registers, waits, and writes it to all destinations; ranges
// of different workgroups do not meet.  Bound by the bytes: each moved slot is
// read and written once (64 slots of 2 MB in 8 layers 411 us, 5.2 TB/s: what a
// copy reaches; a few of 18 KB in 4 layers 4.3 us, a launch).  A destination named twice gets its last source: the
// workgroup finds the last namer of each in a hash table in LDS.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "block_internal.h"
#include "lane_ops.h"
#include "linear_internal.h"

namespace ssm {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr int kHeld = kSlotsHeld;                            // units that a thread holds

__host__ __device__ constexpr int table_size(int n) {
    int size = 64;
    while (size < 2 * n) size *= 2;
    return size;
}

// U: the unit that moves, W: units of a workgroup's range (a power of two), n W <= kHeld threads
template <typename U>
__global__ __launch_bounds__(1024) void slots_copy(SlotsArgs a, int W, int64_t ranges, int size) {
    extern __shared__ int shared[];
    const int n = (int)a.n, tid = threadIdx.x, threads = blockDim.x;
    int* from = shared;
    int* to = from + n;
    int* key = to + n;
    int* last = key + size;
    for (int e = tid; e < size; e += threads) key[e] = -1, last[e] = -1;
    for (int e = tid; e < n; e += threads) from[e] = a.src[e], to[e] = a.dst[e];
    lds_barrier();
    const auto home = [&](int slot) { return (int)(((uint32_t)slot * 2654435761u) >> 8) & (size - 1); };
    const auto moves = [&](int e) { return to[e] >= 0 && to[e] < a.slots && from[e] < a.slots; };
    for (int e = tid; e < n; e += threads) {
        if (!moves(e)) continue;
        int at = home(to[e]);                                // at most half of the table is taken: this ends
        while (true) {
            const int was = atomicCAS(&key[at], -1, to[e]);
            if (was == -1 || was == to[e]) break;
            at = (at + 1) & (size - 1);
        }
        atomicMax(&last[at], e);
    }
    lds_barrier();

    const int64_t layer = blockIdx.x / ranges, range = blockIdx.x % ranges;
    const int64_t units = a.slot_bytes / (int64_t)sizeof(U);
    const int64_t at = range * W + tid % W;
    U* base = static_cast<U*>(a.pool) + layer * a.slots * units + at;
    const int per = threads / W, first = tid / W;            // entries of a pass
    U held[kHeld];
    int64_t target[kHeld];
#pragma unroll
    for (int m = 0; m < kHeld; ++m) {
        const int e = first + m * per;
        target[m] = -1;
        held[m] = U{};
        if (e < n && at < units && moves(e)) {
            int find = home(to[e]);
            while (key[find] != to[e]) find = (find + 1) & (size - 1);
            if (last[find] == e && from[e] != to[e]) {
                target[m] = (int64_t)to[e] * units;
                if (from[e] >= 0) held[m] = base[(int64_t)from[e] * units];
            }
        }
    }
    // every source is in a register before any destination is written
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    lds_barrier();
#pragma unroll
    for (int m = 0; m < kHeld; ++m)
        if (target[m] >= 0) base[target[m]] = held[m];
}

template <typename U> hipError_t launch_unit(const SlotsArgs& a, const SlotsCut& c, hipStream_t stream) {
    const int size = table_size((int)a.n);
    const size_t lds = (size_t)(2 * a.n + 2 * size) * 4;
    slots_copy<U><<<dim3((unsigned)(c.ranges * a.layers)), c.threads, lds, stream>>>(a, c.W, c.ranges, size);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_slots_copy(const SlotsArgs& a, hipStream_t stream) {
    const SlotsCut c = slots_cut(a);
    if (c.unit == 16) return launch_unit<u32x4>(a, c, stream);
    if (c.unit == 4) return launch_unit<uint32_t>(a, c, stream);
    return launch_unit<uint8_t>(a, c, stream);
}

}  // namespace ssm
