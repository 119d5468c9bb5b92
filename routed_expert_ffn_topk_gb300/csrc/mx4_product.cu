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
#include "tc_ptx.cuh"

// First error of a product kernel on this device (estream_mx4_error).
__device__ int g_mx4_err;

// ---------------------------------------------------------------------------
// Tensor-core form. tcgen05.mma kind::mxf4nvf4 multiplies the codes and applies
// both operands' block scales itself; a 32-value block is given as two 16-value
// blocks of one scale, so both formats take one path (scale_vec::4X) and differ
// in the scale type alone.
//
// Weights are the M side (128 rows a tile) and x the N side (NT rows), so a
// route map's short segments cost no more than their own rows rounded up to NT.
// A stage is 256 values of K: both operands' codes by TMA (128-byte rows, 128-byte
// swizzle), the weights' scale tiles by one bulk copy. The scales of x come row
// by row (a segment starts anywhere, so no tile layout fits in advance): four
// warps fetch them a stage ahead and place them as the tensor core wants them
// (row r of 128: lane r % 32, byte group r / 32). The issuing thread copies
// scales to tensor memory with tcgen05.cp ahead of the products that use them;
// both run in its issue order, and two column sets alternate.
// ---------------------------------------------------------------------------

constexpr int kMmaThreads = 320;  // producer, MMA, 4 epilogue and 4 scale warps

template <int NT>
struct Tile {
    static constexpr int kGroups = (NT + 127) / 128;   // 128-row groups of x scales
    static constexpr int kA = 128 * 128, kB = NT * 128, kSfA = 2048, kSfB = 2048 * kGroups;
    static constexpr int kStage = kA + kB + kSfA + kSfB;
    static constexpr int kStages = 220 * 1024 / kStage < 8 ? 220 * 1024 / kStage : 8;
    static constexpr int kAccs = NT <= 128 ? 2 : 1;    // accumulators of NT columns
    static constexpr int kSfCols = 16 + 16 * kGroups;  // a stage's scales in tensor memory
};

// Descriptor of a 32-row x 16-byte block of scales (rows of 16 bytes, 8-row
// groups 128 bytes apart, no swizzle).
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(8) << 16) |
           (static_cast<uint64_t>(8) << 32) | (static_cast<uint64_t>(1) << 46);
}
__device__ __forceinline__ void scales_to_tmem(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
__device__ __forceinline__ void mma_mx4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                        uint32_t sfb, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}
// Instruction descriptor of the block-scaled 4-bit kinds: E2M1 operands (1 in
// bits 7-9 and 10-12), both K-major, N >> 3 in bits 17-22, scale type in bit 23
// (0 UE4M3, 1 UE8M0), M >> 4 in bits 24-28, K = 64.
__device__ __forceinline__ uint32_t mx4_idesc(int M, int N, bool e8m0) {
    return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (e8m0 ? 1u << 23 : 0u) |
           (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

// Slot's rows, kept inside [0, R] whatever the offsets hold.
__device__ __forceinline__ void slot_rows(const Mx4Product& p, int slot, int& lo, int& hi) {
    lo = p.offsets ? min(max(p.offsets[slot], 0), p.R) : 0;
    hi = p.offsets ? min(max(p.offsets[slot + 1], lo), p.R) : p.R;
}

template <typename F>
__device__ __forceinline__ void store_out(const Mx4Product& p, size_t at, F v) {
    if (p.elem == ESTREAM_MX4_F32)
        static_cast<float*>(p.out)[at] = v;
    else
        static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v);
}

// Rows before the first slot and after the last are zero; spread over the grid.
__device__ void zero_outside(const Mx4Product& p, int worker, int workers, int tid, int threads) {
    if (!p.offsets) return;
    const int first = min(max(p.offsets[0], 0), p.R), last = min(max(p.offsets[p.P], first), p.R);
    for (int i = worker; i < first + p.R - last; i += workers) {
        const size_t row = static_cast<size_t>(i < first ? i : last + i - first) * p.ld;
        for (int n = tid; n < p.N; n += threads) store_out(p, row + n, 0.0f);
    }
}

// Exclusive prefix of the slots' row tiles of NT rows into base[0 .. P], by the
// whole CTA (warps of 32 slots at a time; P <= kMaxP).
__device__ void tile_prefix(const Mx4Product& p, int nt, int* base, int* sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const int per = (p.P + nw * 32 - 1) / (nw * 32);  // slots a thread
    const int s0 = (warp * 32 + lane) * per;
    int mine = 0;
    for (int s = s0; s < min(p.P, s0 + per); ++s) {
        int lo, hi;
        slot_rows(p, s, lo, hi);
        mine += (hi - lo + nt - 1) / nt;
    }
    int incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    int run = incl - mine;
    for (int w = 0; w < warp; ++w) run += sums[w];
    for (int s = s0; s < min(p.P, s0 + per); ++s) {
        int lo, hi;
        slot_rows(p, s, lo, hi);
        base[s] = run;
        run += (hi - lo + nt - 1) / nt;
        if (s == p.P - 1) base[p.P] = run;
    }
    __syncthreads();
}

struct Work {
    int slot, row, end, n0;  // rows [row, min(row + NT, end)) of x, weight rows from n0 of the slot
};
// Tile i of the launch: row tiles fastest, so the CTAs at work share weight tiles.
__device__ __forceinline__ Work work_at(const Mx4Product& p, const int* base, int nt, int i) {
    const int row_tiles = base[p.P];
    const int q = i % row_tiles;
    int lo = 0, hi = p.P;  // slot: the last with base <= q and rows
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (base[mid] <= q) lo = mid; else hi = mid;
    }
    Work w;
    w.slot = lo;
    slot_rows(p, lo, w.row, w.end);
    w.row += (q - base[lo]) * nt;
    w.n0 = i / row_tiles * 128;
    return w;
}

// The scales of one row of x for a stage: four words, one for each 64 values.
struct RowScales {
    uint32_t w[4];
};
__device__ __forceinline__ RowScales row_scales(const uint8_t* row, int stage, int nb, int fmt, bool wide) {
    RowScales r;
    if (fmt == ESTREAM_MX4_E4M3X16) {
        const int b0 = stage * 16;
        if (wide && b0 + 16 <= nb) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + b0));
            r.w[0] = v.x, r.w[1] = v.y, r.w[2] = v.z, r.w[3] = v.w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int b = b0 + 4 * j;
                const uint32_t lo = b < nb ? __ldg(reinterpret_cast<const uint16_t*>(row + b)) : 0u;
                const uint32_t hi = b + 2 < nb ? __ldg(reinterpret_cast<const uint16_t*>(row + b + 2)) : 0u;
                r.w[j] = lo | (hi << 16);
            }
        }
    } else {
        const int b0 = stage * 8;
        uint32_t v[2] = {0u, 0u};
        if (wide && b0 + 8 <= nb) {
            const uint2 t = __ldg(reinterpret_cast<const uint2*>(row + b0));
            v[0] = t.x, v[1] = t.y;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (b0 + j < nb) v[j / 4] |= static_cast<uint32_t>(__ldg(row + b0 + j)) << (8 * (j % 4));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) r.w[j] = __byte_perm(v[j / 2], 0, j % 2 ? 0x3322 : 0x1100);
    }
    return r;
}

template <int NT>
__global__ void __launch_bounds__(kMmaThreads, 1) k_mx4_product(const __grid_constant__ CUtensorMap tm_w,
                                                               const __grid_constant__ CUtensorMap tm_x,
                                                               const Mx4Product p, int stages) {
    using S = Tile<NT>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * S::kStages + 4];
    __shared__ int base_small[65];
    __shared__ int sums[32];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_word;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    volatile int* abort_flag = &abort_word;
    int* base = p.P <= 64 ? base_small : reinterpret_cast<int*>(smem + stages * S::kStage);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t sbase = smem_addr(smem);
    auto full = [&](int s) { return smem_addr(&bars[s]); };
    auto empty = [&](int s) { return smem_addr(&bars[S::kStages + s]); };
    auto acc_full = [&](int a) { return smem_addr(&bars[2 * S::kStages + a]); };
    auto acc_empty = [&](int a) { return smem_addr(&bars[2 * S::kStages + 2 + a]); };
    if (threadIdx.x == 0) {
        abort_word = 0;
        for (int s = 0; s < stages; ++s) {
            mbar_init(full(s), 1 + 4);  // the producer's expect_tx and the scale warps
            mbar_init(empty(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(acc_full(a), 1);
            mbar_init(acc_empty(a), 4);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(&tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    tile_prefix(p, NT, base, sums);  // ends with a barrier
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const uint32_t sf_col = tmem + S::kAccs * NT;
    const int tiles = base[p.P] * ((p.N + 127) / 128);
    const int kt = (p.K + 63) / 64, n_st = (kt + 3) / 4;
    const int n_blocks = (p.N + 127) / 128;
    int* err = &g_mx4_err;

    if (warp == 0) {
        if (lane == 0) {
            int s = 0, issued = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int i = blockIdx.x; i < tiles && ok; i += gridDim.x) {
                const Work w = work_at(p, base, NT, i);
                const uint8_t* sf = p.wt + (static_cast<size_t>(w.slot) * n_blocks + w.n0 / 128) * kt * 512;
                for (int st = 0; st < n_st; ++st) {
                    if (!(ok = mbar_wait(empty(s), ph ^ 1u, abort_flag, err))) break;
                    const int nk = min(4, kt - 4 * st);
                    const uint32_t at = sbase + s * S::kStage;
                    mbar_arrive_expect_tx(full(s), S::kA + S::kB + nk * 512);
                    tma_load_2d(at, &tm_w, st * 128, w.slot * p.N + w.n0, full(s));
                    tma_load_2d(at + S::kA, &tm_x, st * 128, w.row, full(s));
                    bulk_load(at + S::kA + S::kB, sf + static_cast<size_t>(st) * 2048, nk * 512, full(s));
                    ++issued;
                    if (++s == stages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            // after an abort the copies in flight land before the CTA ends
            if (!ok)
                for (int i = max(0, issued - stages); i < issued; ++i)
                    mbar_wait_drain(full(i % stages), static_cast<uint32_t>(i / stages) & 1u);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = mx4_idesc(128, NT, p.fmt == ESTREAM_MX4_E8M0X32);
            int s = 0, a = 0, it = 0;
            uint32_t ph = 0, aph = 0;
            bool ok = true;
            for (int i = blockIdx.x; i < tiles && ok; i += gridDim.x) {
                if (!(ok = mbar_wait(acc_empty(a), aph ^ 1u, abort_flag, err))) break;
                const uint32_t acc = tmem + a * NT;
                for (int st = 0; st < n_st; ++st, ++it) {
                    if (!(ok = mbar_wait(full(s), ph, abort_flag, err))) break;
                    tc_fence_after();
                    const int nk = min(4, kt - 4 * st);
                    const uint32_t at = sbase + s * S::kStage;
                    const uint32_t sfa = sf_col + (it & 1) * S::kSfCols, sfb = sfa + 16;
                    const uint64_t da = sw128_desc(at), db = sw128_desc(at + S::kA);
                    const uint64_t dsa = scale_desc(at + S::kA + S::kB), dsb = scale_desc(at + S::kA + S::kB + S::kSfA);
                    for (int j = 0; j < nk; ++j) {
                        scales_to_tmem(sfa + 4 * j, dsa + 32 * j);
#pragma unroll
                        for (int q = 0; q < S::kGroups; ++q)
                            scales_to_tmem(sfb + 4 * (j * S::kGroups + q), dsb + 32 * j + 128 * q);
                    }
                    for (int j = 0; j < nk; ++j)
                        mma_mx4(acc, da + 2 * j, db + 2 * j, idesc, sfa + 4 * j, sfb + 4 * j * S::kGroups,
                                st > 0 || j > 0);
                    umma_commit(empty(s));
                    if (++s == stages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (!ok) break;
                umma_commit(acc_full(a));
                if (++a == S::kAccs) {
                    a = 0;
                    aph ^= 1u;
                }
            }
            if (!ok) {
                // what was issued still completes before tensor memory is freed: the
                // last accumulator's barrier gets a commit of everything so far
                umma_commit(acc_full(a));
                mbar_wait_drain(acc_full(a), aph);
            }
        }
    } else if (warp < 6) {
        zero_outside(p, blockIdx.x, gridDim.x, threadIdx.x - 64, 128);
        const int quad = warp % 4;
        int a = 0;
        uint32_t aph = 0;
        for (int i = blockIdx.x; i < tiles; i += gridDim.x) {
            const Work w = work_at(p, base, NT, i);
            if (!__all_sync(0xffffffffu, mbar_wait(acc_full(a), aph, abort_flag, err))) break;
            tc_fence_after();
            const int n = w.n0 + quad * 32 + lane;
            const int rows = min(NT, w.end - w.row);
            for (int c = 0; c < rows; c += 32) {
                uint32_t v[32];
                tmem_ld32(tmem + (static_cast<uint32_t>(quad * 32) << 16) + a * NT + c, v);
                tmem_ld_wait();
                if (c + 32 >= rows) {  // the accumulator is read: the next tile may have it
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(acc_empty(a));
                }
                if (n < p.N) {
                    size_t at = static_cast<size_t>(w.row + c) * p.ld + n;
#pragma unroll
                    for (int x = 0; x < 32; ++x, at += p.ld)
                        if (c + x < rows) store_out(p, at, __uint_as_float(v[x]) * p.scale);
                }
            }
            if (++a == S::kAccs) {
                a = 0;
                aph ^= 1u;
            }
        }
    } else {
        // scales of x: warp lw places rows lw * 32 + lane of each 128-row group
        const int lw = warp - 6, nb = mx4_padded(p.K) / mx4_block(p.fmt);
        const int align = p.fmt == ESTREAM_MX4_E4M3X16 ? 16 : 8;
        const bool wide = nb % align == 0 && reinterpret_cast<uintptr_t>(p.xs) % align == 0;
        int s = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int i = blockIdx.x; i < tiles && ok; i += gridDim.x) {
            const Work w = work_at(p, base, NT, i);
            const uint8_t* row[S::kGroups];
            RowScales next[S::kGroups];
            auto fetch = [&](int st) {
#pragma unroll
                for (int q = 0; q < S::kGroups; ++q)
                    next[q] = row[q] ? row_scales(row[q], st, nb, p.fmt, wide) : RowScales{{0u, 0u, 0u, 0u}};
            };
#pragma unroll
            for (int q = 0; q < S::kGroups; ++q) {
                const int r = q * 128 + lw * 32 + lane;
                row[q] = r < NT && w.row + r < w.end ? p.xs + static_cast<size_t>(w.row + r) * nb : nullptr;
            }
            fetch(0);
            for (int st = 0; st < n_st; ++st) {
                RowScales now[S::kGroups];
#pragma unroll
                for (int q = 0; q < S::kGroups; ++q) now[q] = next[q];
                if (st + 1 < n_st) fetch(st + 1);
                ok = __all_sync(0xffffffffu, mbar_wait(empty(s), ph ^ 1u, abort_flag, err));
                if (!ok) break;
                uint8_t* sf = smem + s * S::kStage + S::kA + S::kB + S::kSfA + lane * 16 + lw * 4;
#pragma unroll
                for (int q = 0; q < S::kGroups; ++q)
#pragma unroll
                    for (int j = 0; j < 4; ++j) *reinterpret_cast<uint32_t*>(sf + q * 2048 + j * 512) = now[q].w[j];
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(full(s));
                if (++s == stages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// Tensor map of rows of codes: 128-byte columns, boxes of `rows` rows.
CUresult codes_map(CUtensorMap* tm, const uint8_t* codes, int K, size_t rows, uint32_t box) {
    return encode_tmap_2d(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, codes, mx4_padded(K) / 2, rows, mx4_padded(K) / 2, 128,
                          box);
}

template <int NT>
cudaError_t launch_mma(const Mx4Product& p, cudaStream_t stream) {
    using S = Tile<NT>;
    CUtensorMap tm_w, tm_x;
    if (codes_map(&tm_w, p.wc, p.K, static_cast<size_t>(p.P) * p.N, 128) != CUDA_SUCCESS ||
        codes_map(&tm_x, p.xc, p.K, static_cast<size_t>(p.R), NT) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    int dev = 0, sms = 0;
    cudaError_t rc = cudaGetDevice(&dev);
    if (rc == cudaSuccess) rc = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (rc != cudaSuccess) return rc;
    // the prefix of more than 64 slots' tiles takes the place of ring stages
    const size_t prefix = p.P > 64 ? sizeof(int) * (p.P + 1) : 0;
    const int stages = static_cast<int>(std::min<size_t>(S::kStages, (225 * 1024 - prefix) / S::kStage));
    const size_t smem = 1024 + static_cast<size_t>(stages) * S::kStage + prefix;
    rc = cudaFuncSetAttribute(k_mx4_product<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (rc != cudaSuccess) return rc;
    // at most one ragged row tile a slot
    const long long tiles = (static_cast<long long>(p.R) / NT + p.P) * ((p.N + 127) / 128);
    const int grid = static_cast<int>(std::min<long long>(sms, std::max(1ll, tiles)));
    k_mx4_product<NT><<<grid, kMmaThreads, smem, stream>>>(tm_w, tm_x, p, stages);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mx4_product(const Mx4Product& p, cudaStream_t stream) {
    if (p.R == 0 || p.N == 0) return cudaSuccess;
    const long long per = p.R / p.P;
    if (per >= 192) return launch_mma<256>(p, stream);
    if (per > 64) return launch_mma<128>(p, stream);
    return launch_mma<64>(p, stream);
}

cudaError_t read_mx4_error(int* code, cudaStream_t stream) {
    cudaError_t rc = cudaStreamSynchronize(stream);
    if (rc == cudaSuccess) rc = cudaMemcpyFromSymbol(code, g_mx4_err, sizeof(int));
    const int none = kDevErrNone;
    if (rc == cudaSuccess && *code != none) rc = cudaMemcpyToSymbol(g_mx4_err, &none, sizeof(int));
    return rc;
}

}  // namespace es
