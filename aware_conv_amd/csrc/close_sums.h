// The last step of sums over positions: P partial sums of each of n values, in
// fp64, in an order that the shape alone sets.
//
// A workgroup takes 32 values and 8 shares of their partial sums, so that a few
// hundred partial sums of a few thousand values (the usual ends of a backward
// pass) are read by workgroups on all compute units, 128 bytes at a time.
#pragma once

#include <hip/hip_runtime.h>

namespace calls {

// out[k] = sum_p part[p * stride + k], k < n
template <int TAG>
__global__ __launch_bounds__(256) void k_close(const float* part, long long P, long long stride,
                                               long long n, float* out) {
    __shared__ double lds[8][32];
    const int i = threadIdx.x & 31, share = threadIdx.x >> 5;
    const long long k = (long long)blockIdx.x * 32 + i;
    double v = 0;
    if (k < n)
        for (long long p = share; p < P; p += 8) v += part[p * stride + k];
    lds[share][i] = v;
    __syncthreads();
    if (share || k >= n) return;
    for (int q = 1; q < 8; ++q) v += lds[q][i];
    out[k] = float(v);
}

template <int TAG>
inline hipError_t close_sums(const float* part, long long P, long long stride, long long n,
                             float* out, hipStream_t st) {
    if (n == 0) return hipSuccess;
    k_close<TAG><<<unsigned((n + 31) / 32), 256, 0, st>>>(part, P, stride, n, out);
    return hipGetLastError();
}

}  // namespace calls
