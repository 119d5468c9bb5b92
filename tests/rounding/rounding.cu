// Exhaustive check of the quantiser's quotients (csrc/mx4_round.cuh) against IEEE
// division. Prints the number of values compared and of those that differ:
//   boundary  every significand of d, at exponents across the range that takes the
//             reciprocal, and the 13 fp32 values nearest to each rounding boundary of
//             E2M1 times d, both signs: the code;
//   silu      every finite fp32 g: SiLU(g) * 1, zeros of either sign being equal.
#include <cstdint>
#include <cstdio>

#include <cuda_runtime.h>

namespace es {
namespace {
#include "mx4_round.cuh"

__device__ unsigned long long differ[2], compared[2];

__global__ void k_boundary(int exponent) {
    const uint32_t m = blockIdx.x * blockDim.x + threadIdx.x;  // the grid is 2^23 threads
    const float d = __uint_as_float(static_cast<uint32_t>(exponent + 127) << 23 | m);
    const float nr = -__frcp_rn(d);
    const float at[8] = {0.25f, 0.75f, 1.25f, 1.75f, 2.5f, 3.5f, 5.0f, 6.0f};
    unsigned long long bad = 0;
    for (int o = -6; o <= 6; ++o) {
        float got[8], want[8];
        for (int j = 0; j < 8; j += 2) {
            float2 x;
            x.x = __uint_as_float(__float_as_uint(__fmul_rn(at[j], d)) + o);
            x.y = -__uint_as_float(__float_as_uint(__fmul_rn(at[j + 1], d)) + o);
            const float2 q = neg_quotient(x, make_float2(d, d), make_float2(nr, nr));
            got[j] = q.x, got[j + 1] = q.y;
            want[j] = __fdiv_rn(-x.x, d), want[j + 1] = __fdiv_rn(-x.y, d);
        }
        const uint32_t a = e2m1_codes(got), b = e2m1_codes(want);
        for (int j = 0; j < 8; ++j) bad += ((a ^ b) >> (4 * j) & 15u) != 0;
    }
    atomicAdd(&compared[0], 8ull * 13);
    if (bad) atomicAdd(&differ[0], bad);
}

__global__ void k_silu() {
    const unsigned long long threads = static_cast<unsigned long long>(gridDim.x) * blockDim.x;
    unsigned long long n = 0, bad = 0;
    for (unsigned long long i = blockIdx.x * static_cast<unsigned long long>(blockDim.x) + threadIdx.x; i < (1ull << 31);
         i += threads) {
        float v[2], g[2];
        const float u[2] = {1.0f, 1.0f};
        for (int j = 0; j < 2; ++j) v[j] = g[j] = __uint_as_float(static_cast<uint32_t>(2 * i + j));
        neg_silu_mul(v, u);
        for (int j = 0; j < 2; ++j) {
            if (!isfinite(g[j])) continue;
            const float want = -__fdiv_rn(g[j], __fadd_rn(1.0f, expf(-g[j])));
            ++n;
            bad += !(v[j] == want);
        }
    }
    atomicAdd(&compared[1], n);
    if (bad) atomicAdd(&differ[1], bad);
}

}  // namespace
}  // namespace es

int main() {
    for (int e : {-59, -30, -1, 0, 17, 58}) es::k_boundary<<<(1 << 23) / 256, 256>>>(e);
    es::k_silu<<<152 * 8, 256>>>();
    unsigned long long n[2], bad[2];
    if (cudaMemcpyFromSymbol(n, es::compared, sizeof(n)) != cudaSuccess ||
        cudaMemcpyFromSymbol(bad, es::differ, sizeof(bad)) != cudaSuccess) {
        std::printf("error %s\n", cudaGetErrorString(cudaGetLastError()));
        return 1;
    }
    std::printf("boundary %llu %llu\nsilu %llu %llu\n", n[0], bad[0], n[1], bad[1]);
    return 0;
}
