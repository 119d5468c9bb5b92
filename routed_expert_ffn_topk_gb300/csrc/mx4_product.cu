// Product of microscaled 4-bit rows with microscaled 4-bit weights:
//   D[r][n] = g * sum_b s_x[r][b] s_w[n][b] sum_{i in b} q_x[r][i] q_w[n][i],
// dense, or grouped by a route map: rows [offsets[p], offsets[p + 1]) meet the
// weights of slot p, rows outside every slot are zero. Sums are held in fp32;
// D is rounded once, to bf16 or fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "estream_internal.h"

namespace es {
namespace {

constexpr int kTile = 64;   // rows and columns of a CTA's tile
constexpr int kStep = 32;   // values of the reduction staged at a time

__device__ __forceinline__ float scale_value(uint8_t s, int fmt) {
    if (fmt == ESTREAM_MX4_E4M3X16) return __half2float(__half(__nv_cvt_fp8_to_halfraw(s, __NV_E4M3)));
    return s == 0xff ? __int_as_float(0x7fc00000)
                     : __uint_as_float(s == 0 ? 0x00400000u : static_cast<uint32_t>(s) << 23);
}

// Slot's rows, kept inside [0, R] whatever the offsets hold.
__device__ __forceinline__ void slot_rows(const Mx4Product& p, int slot, int& lo, int& hi) {
    lo = p.offsets ? min(max(p.offsets[slot], 0), p.R) : 0;
    hi = p.offsets ? min(max(p.offsets[slot + 1], lo), p.R) : p.R;
}

// Plain form: 64 x 64 tiles, both operands widened to fp32 in shared memory,
// 4 x 4 sums a thread.
__global__ void __launch_bounds__(256) k_mx4_product_simple(const Mx4Product p) {
    __shared__ float xs[kStep][kTile + 1], ws[kStep][kTile + 1];
    const int n0 = blockIdx.x * kTile;
    // the block's row tile: tiles of the slots in turn
    int slot = 0, lo = 0, hi = 0, at = blockIdx.y;
    for (; slot < p.P; ++slot) {
        slot_rows(p, slot, lo, hi);
        const int tiles = (hi - lo + kTile - 1) / kTile;
        if (at < tiles) break;
        at -= tiles;
    }
    if (slot == p.P) {
        // rows outside every slot: [0, first) and [last, R)
        if (!p.offsets) return;
        const int first = min(max(p.offsets[0], 0), p.R);
        const int last = min(max(p.offsets[p.P], first), p.R);
        for (int i = threadIdx.x; i < kTile * kTile; i += 256) {
            const int o = at * kTile + i / kTile, n = n0 + i % kTile;
            const int r = o < first ? o : o - first + last;
            if (r >= p.R || n >= p.N) continue;
            if (p.elem == ESTREAM_MX4_F32)
                static_cast<float*>(p.out)[r * p.ld + n] = 0.0f;
            else
                static_cast<__nv_bfloat16*>(p.out)[r * p.ld + n] = __float2bfloat16_rn(0.0f);
        }
        return;
    }
    const int r0 = lo + at * kTile;
    const int Kp = mx4_padded(p.K), blk = mx4_block(p.fmt), nb = Kp / blk;
    const int kt = (p.K + 63) / 64, nt = (p.N + 127) / 128;
    float acc[4][4] = {};
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    for (int k0 = 0; k0 < Kp; k0 += kStep) {
        for (int i = threadIdx.x; i < kTile * (kStep / 2); i += 256) {
            const int t = i / (kStep / 2), c = k0 + i % (kStep / 2) * 2;
            float a = 0.0f, b = 0.0f, wa = 0.0f, wb = 0.0f;
            if (r0 + t < hi) {
                const size_t r = r0 + t;
                const __half2 h(__nv_cvt_fp4x2_to_halfraw2(p.xc[(r * Kp + c) / 2], __NV_E2M1));
                const float s = scale_value(p.xs[r * nb + c / blk], p.fmt);
                a = __low2float(h) * s;
                b = __high2float(h) * s;
            }
            if (n0 + t < p.N) {
                const size_t r = static_cast<size_t>(slot) * p.N + n0 + t;
                const int n = n0 + t;
                const __half2 h(__nv_cvt_fp4x2_to_halfraw2(p.wc[(r * Kp + c) / 2], __NV_E2M1));
                const size_t tile = (static_cast<size_t>(slot) * nt + n / 128) * kt + c / 64;
                const float s = scale_value(
                    p.wt[tile * 512 + n % 32 * 16 + n % 128 / 32 * 4 + c % 64 / 16], p.fmt);
                wa = __low2float(h) * s;
                wb = __high2float(h) * s;
            }
            xs[c - k0][t] = a;
            xs[c - k0 + 1][t] = b;
            ws[c - k0][t] = wa;
            ws[c - k0 + 1][t] = wb;
        }
        __syncthreads();
        for (int k = 0; k < kStep; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = fmaf(xs[k][ty + 16 * i], ws[k][tx + 16 * j], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int r = r0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (r >= hi || n >= p.N) continue;
            const float y = acc[i][j] * p.scale;
            if (p.elem == ESTREAM_MX4_F32)
                static_cast<float*>(p.out)[r * p.ld + n] = y;
            else
                static_cast<__nv_bfloat16*>(p.out)[r * p.ld + n] = __float2bfloat16_rn(y);
        }
}

}  // namespace

cudaError_t launch_mx4_product(const Mx4Product& p, cudaStream_t stream) {
    if (p.R == 0 || p.N == 0) return cudaSuccess;
    // row tiles: at most one ragged tile a slot, and two for rows outside
    const unsigned rows = static_cast<unsigned>((p.R + kTile - 1) / kTile + (p.offsets ? p.P + 2 : 0));
    k_mx4_product_simple<<<dim3((p.N + kTile - 1) / kTile, rows), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace es
