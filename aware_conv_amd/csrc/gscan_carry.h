// State passed between workgroups that hold successive tiles of a sequence.
//
// Where there are too few rows to fill the device, the tiles of a row are
// spread over workgroups that run at the same time, and the data is still
// read once: a workgroup first composes its tile's map h -> A h + H from what
// it has loaded, publishes it, then collects the state its tile starts from
// and finishes the tile from registers.  The state before tile m is the state
// at the start of its group of kGroup tiles, which the last tile of the group
// before published, put through the maps of the tiles between, in order: a
// fixed order of operations, whatever the timing, and a chain of one wait per
// group, not per tile.
//
// Every wait ends.  Units of work are handed out by a counter, in an order in
// which every tile comes after the tiles that it waits for, so those are held
// by workgroups that already run; one that takes several at a time works them
// off in that order.  A map is published without waiting for
// anything; a group's start waits for maps and the group's start before it:
// by induction over the order, all are published.
//
// A published value is one aligned word that says by itself whether it is
// there (all ones: not yet; a NaN of that pattern is published as another
// one), written and read by relaxed atomics at device scope.  Nothing else
// passes between workgroups, so no fences are needed.  A kernel ahead of the
// scan sets the words.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gsc {

constexpr int kGroup = 16;  // tiles per group

struct Carry {
    unsigned* next;            // shares of units handed out
    unsigned units, share;     // all units; units of a share
    unsigned long long* maps;  // (A, H) of each tile
    unsigned* starts;          // state at the start of each group but the first
};

// First unit of the workgroup's share; `shared` is a word of LDS.
__device__ __forceinline__ unsigned take_share(const Carry& c, unsigned* shared) {
    if (threadIdx.x == 0)
        *shared = c.share * __hip_atomic_fetch_add(c.next, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    // uniform, and known to be: what is derived from it stays scalar
    return __builtin_amdgcn_readfirstlane(*shared);
}

__device__ __forceinline__ void publish_map(unsigned long long* p, float a, float h) {
    unsigned long long w = (unsigned long long)(__float_as_uint(a)) << 32 | __float_as_uint(h);
    if (w == ~0ull) w = 0x7fc000007fc00000ull;
    __hip_atomic_store(p, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void publish_start(unsigned* p, float h) {
    unsigned w = __float_as_uint(h);
    if (w == ~0u) w = 0x7fc00000u;
    __hip_atomic_store(p, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ unsigned long long peek_map(const unsigned long long* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ unsigned peek_start(const unsigned* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float map_a(unsigned long long w) { return __uint_as_float(unsigned(w >> 32)); }
__device__ __forceinline__ float map_h(unsigned long long w) { return __uint_as_float(unsigned(w)); }

// Bytes of the words for `rows` rows of `tiles` tiles, and their places.
inline size_t carry_bytes(size_t rows, int tiles) {
    const size_t groups = (tiles + kGroup - 1) / kGroup;
    return 64 + (sizeof(unsigned long long) * rows * tiles + sizeof(unsigned) * rows * groups + 63) / 64 * 64;
}
// The counter gives out one share in about 12 ns (one address, all XCDs), so
// units that take a workgroup little time are handed out up to `most` at
// once, as long as that leaves a few thousand shares to balance.
inline Carry carry_at(void* ws, size_t rows, int tiles, unsigned units, unsigned most) {
    Carry c;
    c.units = units;
    c.share = units / 4096 < 1 ? 1 : units / 4096 > most ? most : units / 4096;
    c.next = static_cast<unsigned*>(ws);
    c.maps = reinterpret_cast<unsigned long long*>(static_cast<char*>(ws) + 64);
    c.starts = reinterpret_cast<unsigned*>(c.maps + rows * tiles);
    return c;
}
inline unsigned shares(const Carry& c) { return (c.units + c.share - 1) / c.share; }
// Sets the words to "not there" and the counter to 0.
hipError_t clear_carry(void* ws, size_t bytes, hipStream_t st);

}  // namespace gsc
