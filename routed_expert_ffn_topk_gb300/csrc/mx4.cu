// Microscaled 4-bit floating point: rows to E2M1 codes with a scale per block,
// back to values, and the layout of a weight's scales for the product
// (mx4_product.cu).
//
// A value is q * s * g with q in {0, .5, 1, 1.5, 2, 3, 4, 6} and a sign (E2M1,
// two codes to a byte, the first in the low half), s the scale of its block
// and g the tensor's:
//   ESTREAM_MX4_E4M3X16  16 values share an E4M3 s = e4m3(amax / (6 g));
//   ESTREAM_MX4_E8M0X32  32 values share s = 2^max(floor(log2(amax / g)) - 2, -126)
//                        (E8M0; the OCP microscaling rule, which lets the top
//                        binade's upper quarter saturate at 6 s).
// With d = fl(s g), q = E2M1 value nearest to fl(x / d), ties to the even code,
// at most 6; d = 0 (an E4M3 block of zeros, or one whose s rounds to 0) gives
// zeros. A block holding a NaN or an infinity gets a NaN scale and zero codes,
// and reads back as NaN.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "estream_internal.h"
#include "overlap.cuh"

namespace es {
namespace {
#include "mx4_round.cuh"

constexpr int kThreads = 256;

template <int kElem>
struct Elem;
template <>
struct Elem<ESTREAM_MX4_BF16> {
    using T = __nv_bfloat16;
    static __device__ __forceinline__ float up(T v) { return __bfloat162float(v); }
    static __device__ __forceinline__ T down(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<ESTREAM_MX4_F16> {
    using T = __half;
    static __device__ __forceinline__ float up(T v) { return __half2float(v); }
    static __device__ __forceinline__ T down(float v) { return __float2half_rn(v); }
};
template <>
struct Elem<ESTREAM_MX4_F32> {
    using T = float;
    static __device__ __forceinline__ float up(T v) { return v; }
    static __device__ __forceinline__ T down(float v) { return v; }
};

// The largest magnitude, NaN if one is NaN.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
    float m;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
    return m;
}

__device__ __forceinline__ float e4m3_value(uint8_t s) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(s, __NV_E4M3)));
}
__device__ __forceinline__ float e8m0_value(uint8_t s) {
    return s == 0xff ? __int_as_float(0x7fc00000)
                     : __uint_as_float(s == 0 ? 0x00400000u : static_cast<uint32_t>(s) << 23);
}

// How a block's warps lie over a matrix: 2^along of them beside each other on a
// row (32 groups of values each), the rest on the rows below, so that a lane's row
// and column need no division.
struct Tiling {
    int groups;  // of a padded row
    int along;
    __host__ __device__ __forceinline__ int rows() const { return kThreads / 32 >> along; }  // of a block
    __device__ __forceinline__ int row() const {
        return blockIdx.x * (kThreads / 32 >> along) + (threadIdx.x >> 5 >> along);
    }
    __device__ __forceinline__ int group() const {
        return ((blockIdx.y << along) + (threadIdx.x >> 5 & ((1 << along) - 1))) * 32 + (threadIdx.x & 31);
    }
};

// Sixteen values a lane: a block of 16, or with its neighbour one of 32, so what
// is done once a block (scale, reciprocal, addresses) is shared by as many values
// as fit a lane's registers. A row is a whole number of 32-value groups, so a block
// never spans rows. A warp goes down its columns, the next row's values on their
// way while it converts a row's.
// Bound by HBM without SwiGLU and by issue slots with it: 8192 rows of 2 x 14336 bf16
// in 120 us (4.4 TB/s of 6.7), 27 instructions a value, 0.69 a clock and scheduler.
// One value at a time with a division each took 50 instructions (190 us); eight values a
// lane, whose block work is shared by half as many, 40 (175); sixteen without the
// next row in flight 28 but 0.57 a clock (150).
constexpr int kVals = 16;
constexpr int kResident = 3;  // blocks an SM
template <int kElem, bool kSwiglu, int kFmt>
__global__ void __launch_bounds__(kThreads, kResident) k_mx4_quantize(const Mx4Quantize q, Tiling tiling, bool wide) {
    using T = typename Elem<kElem>::T;
    constexpr int kRaw = kVals * sizeof(T) / 16;  // 16-byte words
    after_previous();
    const int group = tiling.group(), c = group * kVals, n = q.K - c;
    if (group - static_cast<int>(threadIdx.x & 31) >= tiling.groups) return;  // the whole warp
    // a warp's lanes past the row's end stay for the shuffle
    const bool in = group < tiling.groups;
    const bool whole = wide && n >= kVals;
    const int stride = tiling.rows() * gridDim.x;
    // source row, or -1 past the end and for an index out of range
    auto source = [&](int row) {
        if (row >= q.R) return -1;
        const int src = q.rows ? __ldca(q.rows + row) : row;
        return src < q.n_src ? src : -1;
    };
    auto at = [&](int src) { return static_cast<const T*>(q.x) + static_cast<size_t>(src) * q.ld + c; };
    uint4 raw[kSwiglu ? 2 : 1][kRaw];
    auto fetch = [&](int src) {
        if (!whole || src < 0) return;
#pragma unroll
        for (int h = 0; h < (kSwiglu ? 2 : 1); ++h)
#pragma unroll
            for (int j = 0; j < kRaw; ++j)
                raw[h][j] = __ldca(reinterpret_cast<const uint4*>(at(src) + (h ? q.K : 0)) + j);
    };
    // half h (gate, up) of the row fetched last
    auto values = [&](int src, int h, float (&v)[kVals]) {
        if (whole) {
            const T* t = reinterpret_cast<const T*>(raw[h]);
#pragma unroll
            for (int j = 0; j < kVals; ++j) v[j] = Elem<kElem>::up(t[j]);
        } else {
            const T* p = at(src) + (h ? q.K : 0);
#pragma unroll
            for (int j = 0; j < kVals; ++j) v[j] = j < n ? Elem<kElem>::up(p[j]) : 0.0f;
        }
    };
    int row = tiling.row();
    int src = source(row), next = source(row + stride);
    fetch(src);
    for (; row < q.R; row += stride) {
        const size_t i = static_cast<size_t>(row) * tiling.groups + group;
        float v[kVals];
        if (in && src >= 0) {
            values(src, 0, v);
            if (kSwiglu) {
                float u[kVals];
                values(src, 1, u);
                fetch(next);
                neg_silu_mul(v, u);
            } else {
                fetch(next);
            }
        } else {
            fetch(next);
#pragma unroll
            for (int j = 0; j < kVals; ++j) v[j] = in && n > 0 ? __int_as_float(0x7fc00000) : 0.0f;
        }
        src = next;
        next = source(row + 2 * stride);
        float amax = 0.0f;
#pragma unroll
        for (int j = 0; j < kVals; j += 2) amax = max_abs(v[j], v[j + 1], amax);
        if (kFmt == ESTREAM_MX4_E8M0X32) amax = max_abs(__shfl_xor_sync(0xffffffffu, amax, 1), amax, 0.0f);
        const bool finite = amax < __int_as_float(0x7f800000);
        uint8_t s;
        float d;
        if (kFmt == ESTREAM_MX4_E4M3X16) {
            s = finite ? __nv_cvt_float_to_fp8(__fdiv_rn(amax, __fmul_rn(6.0f, q.scale)), __NV_SATFINITE, __NV_E4M3)
                       : 0x7f;
            d = __fmul_rn(e4m3_value(s), q.scale);
        } else {
            const uint32_t top = __float_as_uint(__fdiv_rn(amax, q.scale));
            s = !finite ? 0xff : static_cast<uint8_t>(min(max(static_cast<int>(top >> 23) - 2, 1), 0xfe));
            d = __fmul_rn(e8m0_value(s), q.scale);
        }
        uint2 codes = make_uint2(0, 0);
        if (finite && d > 0.0f) {
            // One reciprocal for the block. With d's and the block's exponents well inside
            // the range, the corrected quotient gives the division's code for every
            // significand of d and every x next to a rounding boundary of E2M1
            // (tests/rounding/rounding.cu goes through them).
            if (amax < 1e18f && d > 1e-18f && d < 1e18f) {
                const float nr = -__frcp_rn(d);
#pragma unroll
                for (int j = 0; j < kVals; j += 2) {
                    const float2 f = neg_quotient(make_float2(v[j], v[j + 1]), make_float2(d, d), make_float2(nr, nr));
                    v[j] = f.x;
                    v[j + 1] = f.y;
                }
            } else {
#pragma unroll
                for (int j = 0; j < kVals; ++j) v[j] = __fdiv_rn(-v[j], d);
            }
            // the values are negated here, with SwiGLU twice
            const uint32_t sign = kSwiglu ? 0u : 0x88888888u;
            codes = make_uint2(e2m1_codes(v) ^ sign, e2m1_codes(v + 8) ^ sign);
        }
        if (!in) continue;
        reinterpret_cast<uint2*>(q.codes)[i] = codes;
        if (kFmt == ESTREAM_MX4_E4M3X16)
            q.scales[i] = s;
        else if (group % 2 == 0)
            q.scales[i / 2] = s;
    }
}

template <int kElem, int kFmt>
__global__ void __launch_bounds__(kThreads) k_mx4_dequantize(const uint32_t* codes, const uint8_t* scales, float g,
                                                             int R, int K, Tiling tiling, void* out,
                                                             long long ld, bool wide) {
    using T = typename Elem<kElem>::T;
    constexpr int kLanes = kFmt == ESTREAM_MX4_E4M3X16 ? 2 : 4;
    after_previous();
    const int row = tiling.row(), group = tiling.group(), c = group * 8;
    if (row >= R || group >= tiling.groups) return;
    const size_t i = static_cast<size_t>(row) * tiling.groups + group;
    const uint32_t w = __ldca(codes + i);
    const uint8_t s = __ldca(scales + i / kLanes);
    const float d = __fmul_rn(kFmt == ESTREAM_MX4_E4M3X16 ? e4m3_value(s) : e8m0_value(s), g);
    alignas(16) T v[8];
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const __half2 h(__nv_cvt_fp4x2_to_halfraw2(static_cast<uint8_t>(w >> (4 * j)), __NV_E2M1));
        v[j] = Elem<kElem>::down(__fmul_rn(__low2float(h), d));
        v[j + 1] = Elem<kElem>::down(__fmul_rn(__high2float(h), d));
    }
    T* p = static_cast<T*>(out) + static_cast<size_t>(row) * ld + c;
    if (wide && c + 8 <= K) {
#pragma unroll
        for (int j = 0; j < static_cast<int>(sizeof(T)) / 2; ++j)
            reinterpret_cast<uint4*>(p)[j] = reinterpret_cast<const uint4*>(v)[j];
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c + j < K) p[j] = v[j];
    }
}

// One thread a tile byte: tile [n / 128][k / 64] holds, for row r of its 128
// and 16-value group j of its 64, byte (r % 32) * 16 + (r / 32) * 4 + j; rows
// and groups past the matrix are zero. A 32-value block's scale fills two.
__global__ void __launch_bounds__(kThreads) k_mx4_weight_scales(const uint8_t* __restrict__ scales, int P,
                                                                int N, int nb, int fmt, int nt, int kt,
                                                                uint8_t* __restrict__ tiles) {
    const size_t i = static_cast<size_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (i >= static_cast<size_t>(P) * nt * kt * 512) return;
    const int in = static_cast<int>(i % 512);
    const size_t tile = i / 512;
    const int k = static_cast<int>(tile % kt);
    const int n = static_cast<int>(tile / kt % nt) * 128 + in / 16 + in % 16 / 4 * 32;
    const size_t p = tile / kt / nt;
    const int b = fmt == ESTREAM_MX4_E4M3X16 ? k * 4 + in % 4 : (k * 4 + in % 4) / 2;
    tiles[i] = n < N && b < nb ? scales[(p * N + n) * nb + b] : 0;
}

Tiling tile_rows(int R, int K, int vals, dim3& grid) {
    Tiling t{mx4_padded(K) / vals, 0};
    const int warps = (t.groups + 31) / 32;
    // the widest block that leaves at most a sixteenth of its warps without columns
    for (int a = 3; a > 0 && t.along == 0; --a) {
        const int used = (warps + (1 << a) - 1) >> a << a;
        if ((used - warps) * 16 <= used) t.along = a;
    }
    grid = dim3((R + t.rows() - 1) / t.rows(), (warps + (1 << t.along) - 1) >> t.along);
    return t;
}

template <int kElem, bool kSwiglu>
cudaError_t quantize_fmt(const Mx4Quantize& q, const Tiling& t, bool wide, dim3 grid, cudaStream_t s) {
    if (q.fmt == ESTREAM_MX4_E4M3X16)
        return launch_overlapped(k_mx4_quantize<kElem, kSwiglu, ESTREAM_MX4_E4M3X16>, grid, kThreads, 0, s, q, t, wide);
    return launch_overlapped(k_mx4_quantize<kElem, kSwiglu, ESTREAM_MX4_E8M0X32>, grid, kThreads, 0, s, q, t, wide);
}
template <int kElem>
cudaError_t quantize_elem(const Mx4Quantize& q, const Tiling& t, bool wide, dim3 grid, cudaStream_t s) {
    return q.swiglu ? quantize_fmt<kElem, true>(q, t, wide, grid, s)
                    : quantize_fmt<kElem, false>(q, t, wide, grid, s);
}
template <int kElem>
cudaError_t dequantize_elem(const uint8_t* codes, const uint8_t* scales, int fmt, float g, int R, int K,
                            const Tiling& t, void* out, long long ld, bool wide, dim3 grid, cudaStream_t s) {
    const uint32_t* c = reinterpret_cast<const uint32_t*>(codes);
    if (fmt == ESTREAM_MX4_E4M3X16)
        return launch_overlapped(k_mx4_dequantize<kElem, ESTREAM_MX4_E4M3X16>, grid, kThreads, 0, s, c, scales, g, R, K, t, out, ld, wide);
    return launch_overlapped(k_mx4_dequantize<kElem, ESTREAM_MX4_E8M0X32>, grid, kThreads, 0, s, c, scales, g, R, K, t, out, ld, wide);
}

size_t elem_bytes(int elem) { return elem == ESTREAM_MX4_F32 ? 4 : 2; }
bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace

cudaError_t launch_mx4_quantize(const Mx4Quantize& q, cudaStream_t stream) {
    if (q.R == 0) return cudaSuccess;
    dim3 grid;
    const Tiling t = tile_rows(q.R, q.K, kVals, grid);
    int dev = 0, sms = 0;
    cudaError_t rc = cudaGetDevice(&dev);
    if (rc == cudaSuccess) rc = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (rc != cudaSuccess) return rc;
    grid.x = std::min(grid.x, std::max(1u, sms * kResident / grid.y));  // what is resident at once
    // 16-byte loads need every row (and the up half of it) on a 16-byte boundary
    const size_t b = elem_bytes(q.elem);
    const bool wide = on16(q.x) && q.ld * b % 16 == 0 && (!q.swiglu || q.K * b % 16 == 0);
    if (q.elem == ESTREAM_MX4_BF16) return quantize_elem<ESTREAM_MX4_BF16>(q, t, wide, grid, stream);
    if (q.elem == ESTREAM_MX4_F16) return quantize_elem<ESTREAM_MX4_F16>(q, t, wide, grid, stream);
    return quantize_elem<ESTREAM_MX4_F32>(q, t, wide, grid, stream);
}

cudaError_t launch_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int fmt, float scale,
                                  int R, int K, void* out, int elem, long long ld,
                                  cudaStream_t stream) {
    if (R == 0) return cudaSuccess;
    dim3 grid;
    const Tiling t = tile_rows(R, K, 8, grid);
    const bool wide = on16(out) && ld * elem_bytes(elem) % 16 == 0;
    if (elem == ESTREAM_MX4_BF16)
        return dequantize_elem<ESTREAM_MX4_BF16>(codes, scales, fmt, scale, R, K, t, out, ld, wide, grid, stream);
    if (elem == ESTREAM_MX4_F16)
        return dequantize_elem<ESTREAM_MX4_F16>(codes, scales, fmt, scale, R, K, t, out, ld, wide, grid, stream);
    return dequantize_elem<ESTREAM_MX4_F32>(codes, scales, fmt, scale, R, K, t, out, ld, wide, grid, stream);
}

cudaError_t launch_mx4_weight_scales(const uint8_t* scales, int P, int N, int K, int fmt,
                                     uint8_t* tiles, cudaStream_t stream) {
    const int nt = (N + 127) / 128, kt = (K + 63) / 64;
    const size_t total = static_cast<size_t>(P) * nt * kt * 512;
    if (total == 0) return cudaSuccess;
    k_mx4_weight_scales<<<static_cast<unsigned>((total + kThreads - 1) / kThreads), kThreads, 0, stream>>>(
        scales, P, N, mx4_padded(K) / mx4_block(fmt), fmt, nt, kt, tiles);
    return cudaGetLastError();
}

}  // namespace es

using namespace es;

namespace {
bool mx4_fmt_ok(int fmt) { return fmt == ESTREAM_MX4_E4M3X16 || fmt == ESTREAM_MX4_E8M0X32; }
bool mx4_elem_ok(int e) { return e == ESTREAM_MX4_BF16 || e == ESTREAM_MX4_F16 || e == ESTREAM_MX4_F32; }
bool mx4_scale_ok(float s) { return s > 0.0f && s <= 3.402823466e38f; }
bool at(const void* p, size_t a) { return p && reinterpret_cast<uintptr_t>(p) % a == 0; }
constexpr int kMaxWidth = 1 << 24;   // K and N: keeps a row's offsets in 32 bits
constexpr int kMaxRows = 1 << 30;    // keeps a row index and what is added to it (a launch's stride) in 32 bits

// ESTREAM_OK when the current device runs this library's kernels.
estream_status on_device() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return ESTREAM_ERR_CUDA;
    return device_supported(dev) ? ESTREAM_OK : ESTREAM_ERR_UNSUPPORTED;
}
}  // namespace

extern "C" {

size_t estream_mx4_code_bytes(long long rows, int K) {
    if (rows < 0 || K < 1 || K > kMaxWidth) return 0;
    return static_cast<size_t>(rows) * (mx4_padded(K) / 2);
}

size_t estream_mx4_scale_bytes(long long rows, int K, int fmt) {
    if (rows < 0 || K < 1 || K > kMaxWidth || !mx4_fmt_ok(fmt)) return 0;
    return static_cast<size_t>(rows) * (mx4_padded(K) / mx4_block(fmt));
}

size_t estream_mx4_weight_scale_bytes(int P, int N, int K) {
    if (P < 1 || N < 1 || K < 1 || K > kMaxWidth || N > kMaxWidth) return 0;
    return static_cast<size_t>(P) * ((N + 127) / 128) * ((K + 63) / 64) * 512;
}

estream_status estream_mx4_quantize(const void* x, int elem, long long ld, int n_src, int R, int K,
                                    const int32_t* rows, int swiglu, int fmt, float scale,
                                    void* codes, void* scales, void* cuda_stream) {
    NvtxRange range(kNvMx4Quantize, R);
    if (!mx4_elem_ok(elem) || !mx4_fmt_ok(fmt) || !mx4_scale_ok(scale) || R < 0 || R > kMaxRows || n_src < 0 || K < 1 ||
        K > kMaxWidth || ld < (swiglu ? 2ll : 1ll) * K || (!rows && n_src < R))
        return ESTREAM_ERR_INVALID_ARG;
    if (R == 0) return ESTREAM_OK;
    const size_t b = elem == ESTREAM_MX4_F32 ? 4 : 2;
    if ((n_src > 0 && !at(x, b)) || !at(codes, 16) || !scales || (rows && !at(rows, 4)))
        return ESTREAM_ERR_INVALID_ARG;
    const estream_status st = on_device();
    if (st != ESTREAM_OK) return st;
    const Mx4Quantize q{x, elem, ld, n_src, R, K, rows, swiglu != 0, fmt, scale,
                        static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales)};
    return launch_mx4_quantize(q, static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess ? ESTREAM_OK
                                                                                         : ESTREAM_ERR_CUDA;
}

estream_status estream_mx4_dequantize(const void* codes, const void* scales, int fmt, float scale, int R,
                                      int K, void* out, int elem, long long ld, void* cuda_stream) {
    NvtxRange range(kNvMx4Dequantize, R);
    if (!mx4_elem_ok(elem) || !mx4_fmt_ok(fmt) || !mx4_scale_ok(scale) || R < 0 || R > kMaxRows || K < 1 ||
        K > kMaxWidth || ld < K)
        return ESTREAM_ERR_INVALID_ARG;
    if (R == 0) return ESTREAM_OK;
    if (!at(codes, 16) || !scales || !at(out, elem == ESTREAM_MX4_F32 ? 4 : 2)) return ESTREAM_ERR_INVALID_ARG;
    const estream_status st = on_device();
    if (st != ESTREAM_OK) return st;
    return launch_mx4_dequantize(static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales), fmt,
                                 scale, R, K, out, elem, ld, static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess
               ? ESTREAM_OK
               : ESTREAM_ERR_CUDA;
}

estream_status estream_mx4_weight_scales(const void* scales, int P, int N, int K, int fmt, void* tiles,
                                         void* cuda_stream) {
    NvtxRange range(kNvMx4Scales, static_cast<long long>(P) * N);
    if (!mx4_fmt_ok(fmt) || estream_mx4_weight_scale_bytes(P, N, K) == 0 || P > kMaxP || !scales ||
        !at(tiles, 128))
        return ESTREAM_ERR_INVALID_ARG;
    const estream_status st = on_device();
    if (st != ESTREAM_OK) return st;
    return launch_mx4_weight_scales(static_cast<const uint8_t*>(scales), P, N, K, fmt,
                                    static_cast<uint8_t*>(tiles), static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess
               ? ESTREAM_OK
               : ESTREAM_ERR_CUDA;
}

estream_status estream_mx4_product(const void* x_codes, const void* x_scales, int R, const void* w_codes,
                                   const void* w_tiles, int P, int N, int K, int fmt, float scale,
                                   const int32_t* offsets, void* out, int elem, long long ld,
                                   void* cuda_stream) {
    NvtxRange range(kNvMx4Product, R);
    if (!mx4_fmt_ok(fmt) || !mx4_scale_ok(scale) || R < 0 || R > kMaxRows || P < 1 || P > kMaxP || N < 1 ||
        N > kMaxWidth || K < 1 || K > kMaxWidth || (!offsets && P != 1) || ld < N ||
        (elem != ESTREAM_MX4_BF16 && elem != ESTREAM_MX4_F32))
        return ESTREAM_ERR_INVALID_ARG;
    if (R == 0) return ESTREAM_OK;
    if (!at(x_codes, 16) || !at(x_scales, 2) || !at(w_codes, 16) || !at(w_tiles, 128) ||
        (offsets && !at(offsets, 4)) || !at(out, elem == ESTREAM_MX4_F32 ? 4 : 2))
        return ESTREAM_ERR_INVALID_ARG;
    if (static_cast<long long>(P) * N >= (1ll << 31)) return ESTREAM_ERR_CAPACITY;  // weight rows: 32-bit
    const estream_status st = on_device();
    if (st != ESTREAM_OK) return st;
    const Mx4Product p{static_cast<const uint8_t*>(x_codes), static_cast<const uint8_t*>(x_scales),
                       static_cast<const uint8_t*>(w_codes), static_cast<const uint8_t*>(w_tiles),
                       offsets, R, P, N, K, fmt, scale, out, elem, ld};
    return launch_mx4_product(p, static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess ? ESTREAM_OK
                                                                                        : ESTREAM_ERR_CUDA;
}

estream_status estream_mx4_error(void* cuda_stream) {
    const estream_status st = on_device();
    if (st != ESTREAM_OK) return st;
    int code = 0;
    if (read_mx4_error(&code, static_cast<cudaStream_t>(cuda_stream)) != cudaSuccess) return ESTREAM_ERR_CUDA;
    if (code == kDevErrNone) return ESTREAM_OK;
    return code == kDevErrTimeout ? ESTREAM_ERR_TIMEOUT : ESTREAM_ERR_DEVICE;
}

}  // extern "C"
