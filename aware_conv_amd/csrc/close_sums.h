// The last step of sums over positions: P partial sums of each of n values, in
// fp64, in an order that the shape alone sets.
//
// A workgroup takes 16 values and 16 shares of their partial sums, 64 bytes at a
// time, four loads of each thread under way: a few hundred partial sums of a few
// thousand values, the usual end of a backward pass, are read by workgroups on most
// compute units (512 of 2048: 20 us in 8 shares one load at a time, 5 so).
#pragma once

#include <hip/hip_runtime.h>

namespace calls {

// out[k] = sum_p part[p * n + k], k < n; nothing for out = NULL
struct Sums {
    const float* part;
    long long n;
    float* out;
};

inline long long close_blocks(long long na, long long nb, long long nc) {
    return (na + 15) / 16 + (nb + 15) / 16 + (nc + 15) / 16;
}
// Whether one launch, which has fewer than 2^32 threads, closes the sums of so many
// values; asked before anything is enqueued.
inline bool close_fits(long long na, long long nb = 0, long long nc = 0) {
    return close_blocks(na, nb, nc) < (1LL << 24);
}

// `tag` tells the copies of one source file from another's.
template <int tag>
__global__ __launch_bounds__(256) void k_close(Sums a, Sums b, Sums c, long long P) {
    __shared__ double lds[16][17];
    const int i = threadIdx.x & 15, share = threadIdx.x >> 4;
    const long long na = (a.n + 15) / 16, nb = (b.n + 15) / 16;
    const long long block = blockIdx.x;
    const Sums s = block < na ? a : block < na + nb ? b : c;
    const long long k = (block < na ? block : block < na + nb ? block - na : block - na - nb) * 16 + i;
    double v[4] = {0, 0, 0, 0};
    if (k < s.n) {
        const float* const from = s.part + k;
        long long p = share;
        for (; p + 48 < P; p += 64)
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] += from[(p + 16 * q) * s.n];
        for (; p < P; p += 16) v[0] += from[p * s.n];
    }
    lds[share][i] = (v[0] + v[1]) + (v[2] + v[3]);
    __syncthreads();
    if (share || k >= s.n || !s.out) return;
    double sum = 0;
    for (int q = 0; q < 16; ++q) sum += lds[q][i];
    s.out[k] = float(sum);
}

template <int tag>
inline hipError_t close_sums(long long P, hipStream_t st, Sums a, Sums b = {}, Sums c = {}) {
    if (!a.out) a.n = 0;
    if (!b.out) b.n = 0;
    if (!c.out) c.n = 0;
    const long long blocks = close_blocks(a.n, b.n, c.n);
    if (blocks == 0) return hipSuccess;
    k_close<tag><<<unsigned(blocks), 256, 0, st>>>(a, b, c, P);
    return hipGetLastError();
}

}  // namespace calls
