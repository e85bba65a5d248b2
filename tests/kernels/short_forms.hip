// The short root, reciprocal and quotient of the 8-bit update (moments8.h)
// against sqrtf and /, for tests/test_gpu_short_forms.py.  Each kernel adds to
// counts[0] the pairs or values compared and to counts[1] those that differ.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "moments8.h"

namespace zero_shard {
namespace {

typedef unsigned long long u64;
constexpr int kGrid = 2048, kThreads = 256;
constexpr uint32_t kMantissas = 1u << 23;

__device__ __forceinline__ void add(u64* counts, u64 compared, u64 differ) {
    for (int off = 32; off > 0; off >>= 1) {
        compared += __shfl_xor(compared, off, 64);
        differ += __shfl_xor(differ, off, 64);
    }
    if ((threadIdx.x & 63) == 0) {
        atomicAdd(counts, compared);
        if (differ) atomicAdd(counts + 1, differ);
    }
}

__device__ __forceinline__ bool same(float a, float b) { return __float_as_uint(a) == __float_as_uint(b); }

// a, d in [1, 2) with these fractions
__device__ __forceinline__ bool quotient_differs(uint32_t a, uint32_t d) {
    const float x = __uint_as_float(0x3F800000u + a), y = __uint_as_float(0x3F800000u + d);
    return !same(quotient_normal(x, y), x / y);
}

// every float whose bits lie in [lo, hi)
__global__ __launch_bounds__(kThreads) void roots(uint32_t lo, uint32_t hi, u64* counts) {
    u64 compared = 0, differ = 0;
    for (uint64_t b = lo + (uint64_t)blockIdx.x * kThreads + threadIdx.x; b < hi; b += kGrid * kThreads) {
        const float v = __uint_as_float((uint32_t)b);
        ++compared;
        differ += !same(root_normal(v), sqrtf(v));
    }
    add(counts, compared, differ);
}

// every mantissa
__global__ __launch_bounds__(kThreads) void reciprocals(u64* counts) {
    u64 compared = 0, differ = 0;
    for (uint32_t i = blockIdx.x * kThreads + threadIdx.x; i < kMantissas; i += kGrid * kThreads) {
        const float d = __uint_as_float(0x3F800000u + i);
        ++compared;
        differ += !same(reciprocal_normal(d), 1.0f / d);
    }
    add(counts, compared, differ);
}

// Every quotient that lies within radius/(2D) last places of the middle between
// two floats, for every mantissa D of the divisor: 2^(s+1) A = (2K+1) D + delta
// with 0 < |delta| <= radius, s = 23 where A >= D and 24 where A < D.  With
// D = 2^j Do, Do odd, delta has to be a multiple of 2^j, and
// A = ((Do + delta/2^j) / 2) 2^(j-s) modulo Do, where the bracket is even.
__global__ __launch_bounds__(kThreads) void hard_quotients(int radius, u64* counts) {
    u64 compared = 0, differ = 0;
    for (uint32_t i = blockIdx.x * kThreads + threadIdx.x; i < kMantissas; i += kGrid * kThreads) {
        const int64_t D = (int64_t)kMantissas + i;
        const int j = __builtin_ctzll((uint64_t)D);
        const int64_t Do = D >> j;
        for (int s = 23; s <= 24; ++s)
            for (int delta = -radius; delta <= radius; ++delta) {
                if (delta == 0 || (delta & ((1 << j) - 1))) continue;
                const int64_t twice = Do + (delta >> j);
                if (twice & 1) continue;
                int64_t x = (twice / 2 % Do + Do) % Do;
                for (int k = 0; k < s - j; ++k) x = (x & 1) ? (x + Do) / 2 : x / 2;
                for (int64_t A = x; A < 2 * (int64_t)kMantissas; A += Do) {
                    if (A < (int64_t)kMantissas || (A >= D) != (s == 23)) continue;
                    ++compared;
                    differ += quotient_differs((uint32_t)(A - kMantissas), i);
                }
            }
    }
    add(counts, compared, differ);
}

// every numerator over one divisor
__global__ __launch_bounds__(kThreads) void numerators(uint32_t d, u64* counts) {
    u64 compared = 0, differ = 0;
    for (uint32_t a = blockIdx.x * kThreads + threadIdx.x; a < kMantissas; a += kGrid * kThreads) {
        ++compared;
        differ += quotient_differs(a, d);
    }
    add(counts, compared, differ);
}

// n pairs drawn from the exponents that the update's range test lets through:
// the numerator in [2^-74, 2^50) of either sign, the divisor in [2^-48, 2^46).
__global__ __launch_bounds__(kThreads) void exponents(uint64_t n, uint64_t seed, u64* counts) {
    u64 compared = 0, differ = 0;
    for (uint64_t i = (uint64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += kGrid * kThreads) {
        const uint32_t a = dither_bits((uint32_t)i, dither_key(seed, 2 * (i >> 32)));
        const uint32_t b = dither_bits((uint32_t)i, dither_key(seed, 2 * (i >> 32) + 1));
        const uint32_t ea = (uint32_t)(127 - 74) + (a >> 24) % 124u, eb = (uint32_t)(127 - 48) + (b >> 24) % 94u;
        const float x = __uint_as_float((b & 0x800000u) << 8 | ea << 23 | (a & 0x7FFFFFu));
        const float d = __uint_as_float(eb << 23 | (b & 0x7FFFFFu));
        ++compared;
        differ += !same(quotient_normal(x, d), x / d);
    }
    add(counts, compared, differ);
}

}  // namespace
}  // namespace zero_shard

using namespace zero_shard;

extern "C" {

int check_roots(uint32_t lo, uint32_t hi, u64* counts) {
    hipLaunchKernelGGL(roots, dim3(kGrid), dim3(kThreads), 0, 0, lo, hi, counts);
    return (int)hipGetLastError();
}

int check_reciprocals(u64* counts) {
    hipLaunchKernelGGL(reciprocals, dim3(kGrid), dim3(kThreads), 0, 0, counts);
    return (int)hipGetLastError();
}

int check_hard_quotients(int radius, u64* counts) {
    if (radius < 0 || radius > 64) return -1;
    hipLaunchKernelGGL(hard_quotients, dim3(kGrid), dim3(kThreads), 0, 0, radius, counts);
    return (int)hipGetLastError();
}

int check_numerators(uint32_t d, u64* counts) {
    if (d >= kMantissas) return -1;
    hipLaunchKernelGGL(numerators, dim3(kGrid), dim3(kThreads), 0, 0, d, counts);
    return (int)hipGetLastError();
}

int check_exponents(uint64_t n, uint64_t seed, u64* counts) {
    hipLaunchKernelGGL(exponents, dim3(kGrid), dim3(kThreads), 0, 0, n, seed, counts);
    return (int)hipGetLastError();
}

}  // extern "C"
