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
#include <atomic>

#include "estream_internal.h"
#include "overlap.cuh"

namespace es {
namespace {
#include "tc_ptx.cuh"
#include "tc_pair_ptx.cuh"

// One thread of the warp (all 32 call it). The compiler knows what follows to run
// in a single thread, so it need not serialise the tensor-core and copy
// instructions there over possible lanes: 75 clocks an instruction under
// lane == 0.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
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
// Bound by HBM (the weights) and by latency: 1 x 14336 x 4096 streams its 33 MB (a
// tile holds a 32-value block's scale twice) at 6 TB/s for 5.5 us, after 2.5 us until
// the first stage is there (12 us a call back to back, of 4.7 for the data's own
// bytes at HBM's rate), on 112 of the 152 SMs; 64 slots of 128 rows, 2048 x 2048, take 42 us of 29,
// the tensor pipe 22% busy, with about 5 us of it the epilogue's small stores
// (weights are M, so a thread holds a column of D).
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
// whole CTA (warps of 32 slots at a time; P <= kMaxP). Ascending offsets give at
// most R / NT + P tiles. Others may count rows many times over, past 32 bits: the
// sums stop at kMostTiles, above every valid total, and a total past the valid
// ones leaves no tiles at all. (A thread's own slots, at most 16 of 2^30 / 64 + 1
// tiles, and one addition to a sum that has stopped stay within 32 bits.)
constexpr int kMostTiles = 1 << 29;
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
        if (lane >= d) incl = min(incl + o, kMostTiles);
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    int run = incl - mine;
    for (int w = 0; w < warp; ++w) run = min(run + sums[w], kMostTiles);
    for (int s = s0; s < min(p.P, s0 + per); ++s) {
        int lo, hi;
        slot_rows(p, s, lo, hi);
        base[s] = run;
        run += (hi - lo + nt - 1) / nt;
        if (s == p.P - 1) base[p.P] = run > p.R / nt + p.P ? 0 : run;
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
            const uint4 v = __ldca(reinterpret_cast<const uint4*>(row + b0));
            r.w[0] = v.x, r.w[1] = v.y, r.w[2] = v.z, r.w[3] = v.w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int b = b0 + 4 * j;
                const uint32_t lo = b < nb ? __ldca(reinterpret_cast<const uint16_t*>(row + b)) : 0u;
                const uint32_t hi = b + 2 < nb ? __ldca(reinterpret_cast<const uint16_t*>(row + b + 2)) : 0u;
                r.w[j] = lo | (hi << 16);
            }
        }
    } else {
        const int b0 = stage * 8;
        uint32_t v[2] = {0u, 0u};
        if (wide && b0 + 8 <= nb) {
            const uint2 t = __ldca(reinterpret_cast<const uint2*>(row + b0));
            v[0] = t.x, v[1] = t.y;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (b0 + j < nb) v[j / 4] |= static_cast<uint32_t>(__ldca(row + b0 + j)) << (8 * (j % 4));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) r.w[j] = __byte_perm(v[j / 2], 0, j % 2 ? 0x3322 : 0x1100);
    }
    return r;
}

// The scale warps of one CTA over all its tiles (first, first + step, ...): warp
// lw places rows lw * 32 + lane of each 128-row group of a stage. A row's scales
// are fetched kAhead stages before their place in the ring is free, across tiles.
// `slot_free()` waits for the next ring slot and gives its place for x scales (or
// null: stop), `publish()` hands it over.
constexpr int kAhead = 4;
template <int kGroups, int kRows, typename WorkAt, typename Wait, typename Publish>
__device__ __forceinline__ void feed_scales(const Mx4Product& p, int first, int step, int tiles, int n_st, int lw,
                                            int lane, WorkAt work, Wait slot_free, Publish publish) {
    if (first >= tiles) return;
    const int nb = mx4_padded(p.K) / mx4_block(p.fmt);
    const int align = p.fmt == ESTREAM_MX4_E4M3X16 ? 16 : 8;
    const bool wide = nb % align == 0 && reinterpret_cast<uintptr_t>(p.xs) % align == 0;
    const int r0 = lw * 32 + lane;
    int f_tile = first, f_st = 0, f_rows = 0;
    const uint8_t* f_x = p.xs;
    auto enter = [&] {
        if (f_tile >= tiles) return;
        const Work w = work(f_tile);
        f_x = p.xs + static_cast<size_t>(w.row + r0) * nb;
        f_rows = min(kRows, w.end - w.row) - r0;
    };
    RowScales next[kAhead][kGroups];
    auto fetch = [&](RowScales (&to)[kGroups]) {
        if (f_tile >= tiles) return;
#pragma unroll
        for (int q = 0; q < kGroups; ++q)
            to[q] = q * 128 < f_rows ? row_scales(f_x + static_cast<size_t>(q * 128) * nb, f_st, nb, p.fmt, wide)
                                     : RowScales{{0u, 0u, 0u, 0u}};
        if (++f_st == n_st) {
            f_st = 0;
            f_tile += step;
            enter();
        }
    };
    enter();
#pragma unroll
    for (int d = 0; d < kAhead; ++d) fetch(next[d]);
    const int total = ((tiles - first + step - 1) / step) * n_st;
    for (int n = 0; n < total; n += kAhead) {
#pragma unroll
        for (int d = 0; d < kAhead; ++d) {
            if (n + d >= total) break;
            uint8_t* sf = slot_free();
            if (!sf) return;
            sf += lane * 16 + lw * 4;
#pragma unroll
            for (int q = 0; q < kGroups; ++q)
#pragma unroll
                for (int j = 0; j < 4; ++j) *reinterpret_cast<uint32_t*>(sf + q * 2048 + j * 512) = next[d][q].w[j];
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            publish();
            fetch(next[d]);
        }
    }
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
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
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
    after_previous();
    tile_prefix(p, NT, base, sums);  // ends with a barrier
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const uint32_t sf_col = tmem + S::kAccs * NT;
    const int tiles = base[p.P] * ((p.N + 127) / 128);
    const int kt = (p.K + 63) / 64, n_st = (kt + 3) / 4;
    const int n_blocks = (p.N + 127) / 128;
    int* err = &g_mx4_err;

    if (warp == 0) {
        if (elect_one()) {
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
        if (elect_one()) {
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
        const bool pairs_out = p.elem == ESTREAM_MX4_BF16 && p.ld % 2 == 0 && p.N % 2 == 0 &&
                               reinterpret_cast<uintptr_t>(p.out) % 4 == 0;
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
                if (pairs_out) {
                    // neighbouring lanes exchange: the even one stores both columns of row x,
                    // the odd one of row x + 1 (half the stores: 42.1 against 43.4 us, 64 slots)
                    const bool odd = lane & 1;
                    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + static_cast<size_t>(w.row + c + odd) * p.ld + (n & ~1);
#pragma unroll
                    for (int x = 0; x < 32; x += 2, o += 2 * p.ld) {
                        const __nv_bfloat162 q = __floats2bfloat162_rn(__uint_as_float(v[x]) * p.scale,
                                                                       __uint_as_float(v[x + 1]) * p.scale);
                        const uint32_t own = *reinterpret_cast<const uint32_t*>(&q);
                        const uint32_t other = __shfl_xor_sync(0xffffffffu, own, 1);
                        if (n < p.N && c + x + odd < rows)
                            *reinterpret_cast<uint32_t*>(o) = odd ? __byte_perm(other, own, 0x7632) : __byte_perm(own, other, 0x5410);
                    }
                } else if (n < p.N) {
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
        int s = 0;
        uint32_t ph = 0;
        feed_scales<S::kGroups, NT>(
            p, blockIdx.x, gridDim.x, tiles, n_st, warp - 6, lane, [&](int i) { return work_at(p, base, NT, i); },
            [&]() -> uint8_t* {
                if (!__all_sync(0xffffffffu, mbar_wait(empty(s), ph ^ 1u, abort_flag, err))) return nullptr;
                return smem + s * S::kStage + S::kA + S::kB + S::kSfA;
            },
            [&] {
                if (lane == 0) mbar_arrive(full(s));
                if (++s == stages) {
                    s = 0;
                    ph ^= 1u;
                }
            });
    }
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------
// Pair form: clusters of two CTAs on 256 rows of x x 256 weight rows with
// cta_group::2 (M = 256, N = 256). Each CTA holds half of both operands of a stage,
// 32 KB for the 128 x 256 x 256 products that it does, against 48 KB for a CTA
// alone, which would read and fill shared memory at more than its 128 bytes a
// clock and L2 at more than it delivers. The leader (rank 0) issues the products and
// scale copies of both. Here x is the M side: a CTA then places only its own 128
// rows' scales (the weights' come as tiles by TMA), and a thread of the epilogue
// holds a row's neighbouring columns, which leave in whole 128-byte pieces.
// What kept the products waiting, for 4096 x 14336 x 4096 (68 us with neither
// loads, scale fetches nor stores): scale copies issued by the MMA thread, half
// of its time, now from a thread of their own into columns that belong to the
// stage's ring slot; and everything in the load/store unit -- scales fetched by
// loads, whose latency each fence of the placing thread waited for (22 us), and
// the epilogue's stores (27 us). Both go through TMA where the alignment allows.
// One 256-column accumulator and the scales fill tensor memory, so the epilogue
// is not hidden behind the next tile; its eight warps first drain the accumulator
// into registers, 128 columns a thread (the roles' registers are split for that;
// bf16 results are packed on the way, without which they spill: 99 against 94 us),
// and store afterwards.
// 4096 x 14336 x 4096: 94 us back to back, 5.1 PFLOP/s. A stage takes 750 clocks, its
// products 512; the issuing thread waits for operands and scales meanwhile, which
// come at 51 bytes a clock and SM. A kernel of nothing but TMA loads out of L2 into
// every SM reached 40 to 47 (no more with multicast in clusters of 2 or 4), so the
// products are fed as fast as anything measured here was; what would limit them at
// a higher rate is not known. Another 1570 clocks of a tile's 13500 pass between its
// last commit and the next tile's first product.
// ---------------------------------------------------------------------------

// Warpgroups: producer and MMA warps; two of epilogue warps; scale warps. At 128
// registers a thread the launch holds 512 x 128; the split 80 + 168 + 168 + 88
// comes to 504.
constexpr int kPairThreads = 512;
template <int kRegs>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
struct Pair {
    static constexpr int kA = 128 * 128, kB = 128 * 128, kSfA = 2048, kSfB = 4096;
    static constexpr int kStage = kA + kB + kSfA + kSfB;
    static constexpr int kStages = 5;
    static constexpr int kSfCols = 48;
    static constexpr int kOutBytes = 8 * 4096;  // epilogue stage, 4 KB a warp
};

__device__ __forceinline__ void scales_to_tmem_pair(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
__device__ __forceinline__ void mma_mx4_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                             uint32_t sfb, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// 128 bytes of one row a lane (bf16: 64 columns, fp32: 32; the lane's row is
// row0 + lane) through the warp's 4 KB stage (128-byte swizzle) to out columns
// from n on: by TMA, or, where the rows end inside (another slot's follow) or out
// is not aligned for it, by plain stores. Rows from `rows` on and columns from p.N
// on are left out.
template <typename T>
__device__ __forceinline__ void write_rows(const Mx4Product& p, const CUtensorMap* tm, uint8_t* stage,
                                           const uint32_t (&v)[32], int lane, int row0, int rows, int n, bool tma) {
    constexpr int kCols = 128 / sizeof(T), kPiece = 16 / sizeof(T);
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();  // the stage's last use is over
#pragma unroll
    for (int c = 0; c < 8; ++c)
        *reinterpret_cast<uint4*>(stage + lane * 128 + ((c ^ (lane & 7)) * 16)) =
            make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
    if (tma && (rows >= 32 || row0 + rows == p.R)) {  // (the map ends with the last row and column)
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0)
            asm volatile(
                "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];\n\t"
                "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(tm)),
                "r"(n), "r"(row0), "r"(smem_addr(stage))
                : "memory");
        return;
    }
    __syncwarp();
    const int c = lane & 7;
    if (tma && n + kCols <= p.N) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = i * 4 + (lane >> 3);
            const uint4 x = *reinterpret_cast<const uint4*>(stage + r * 128 + ((c ^ (r & 7)) * 16));
            if (r < rows)
                *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + static_cast<size_t>(row0 + r) * p.ld + n + c * kPiece) = x;
        }
    } else {
        for (int r = 0; r < min(32, rows); ++r)
            for (int x = lane; x < kCols && n + x < p.N; x += 32)
                static_cast<T*>(p.out)[static_cast<size_t>(row0 + r) * p.ld + n + x] = *reinterpret_cast<const T*>(
                    stage + r * 128 + (((x / kPiece) ^ (r & 7)) * 16) + x % kPiece * sizeof(T));
    }
}

__global__ void __launch_bounds__(kPairThreads, 1) k_mx4_product_pair(const __grid_constant__ CUtensorMap tm_w,
                                                                     const __grid_constant__ CUtensorMap tm_x,
                                                                     const __grid_constant__ CUtensorMap tm_s,
                                                                     const __grid_constant__ CUtensorMap tm_xs,
                                                                     const __grid_constant__ CUtensorMap tm_out,
                                                                     const Mx4Product p, int stages, bool tma_xs,
                                                                     bool tma_out) {
    using S = Pair;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[4 * S::kStages + 4];
    __shared__ int base_small[65];
    __shared__ int sums[32];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_word;
    // pair instructions and peer addresses need clusters of exactly two
    if (cluster_num_ctas() != 2) {
        if (threadIdx.x == 0) record_error(&g_mx4_err, kDevErrLaunch);
        return;
    }
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    volatile int* abort_flag = &abort_word;
    uint8_t* out_stage = smem + stages * S::kStage;
    int* base = p.P <= 64 ? base_small : reinterpret_cast<int*>(out_stage + S::kOutBytes);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_rank());
    const uint32_t sbase = smem_addr(smem);
    auto full = [&](int s) { return smem_addr(&bars[s]); };            // the leader's
    auto empty = [&](int s) { return smem_addr(&bars[S::kStages + s]); };
    const uint32_t acc_full = smem_addr(&bars[2 * S::kStages]);
    const uint32_t acc_empty = smem_addr(&bars[2 * S::kStages + 1]);   // the leader's
    const uint32_t drained = smem_addr(&bars[2 * S::kStages + 2]), sf_drained = drained + 8;
    auto raw = [&](int s) { return smem_addr(&bars[3 * S::kStages + 4 + s]); };     // x scales as they lie
    auto scaled = [&](int s) { return smem_addr(&bars[2 * S::kStages + 4 + s]); };  // scales in tensor memory
    if (threadIdx.x == 0) {
        abort_word = 0;
        for (int s = 0; s < stages; ++s) {
            mbar_init(full(s), 1 + 4 + 4);  // the leader's expect_tx and both CTAs' scale warps
            mbar_init(empty(s), 1);
            mbar_init(scaled(s), 1);
            mbar_init(raw(s), 1);
        }
        mbar_init(acc_full, 1);
        mbar_init(acc_empty, 8 + 8);
        mbar_init(drained, 1);
        mbar_init(sf_drained, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_addr(&tmem_slot), 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    after_previous();
    tile_prefix(p, 256, base, sums);
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = tmem_slot, sf_col = tmem + 256;
    const int tiles = base[p.P] * ((p.N + 255) / 256);
    const int kt = (p.K + 63) / 64, n_st = (kt + 3) / 4;
    const int n_blocks = (p.N + 127) / 128;
    const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);
    int* err = &g_mx4_err;
    const bool e4m3 = p.fmt == ESTREAM_MX4_E4M3X16;
    // this CTA's rows of a tile, and the tile's first weight row
    auto work = [&](int i) {
        Work w = work_at(p, base, 256, i);
        w.n0 *= 2;
        w.row += 128 * rank;
        return w;
    };

    if (warp < 4) {
        fewer_registers<80>();
        if (warp == 0 && elect_one()) {
            int s = 0, issued = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int i = pair; i < tiles && ok; i += pairs) {
                const Work w = work(i);
                const int sf = (w.slot * n_blocks + w.n0 / 128) * kt;
                for (int st = 0; st < n_st; ++st) {
                    if (!(ok = mbar_wait_cl(empty(s), ph ^ 1u, abort_flag, err))) break;
                    const uint32_t at = sbase + s * S::kStage;
                    const uint32_t bar = map_rank(full(s), 0);
                    if (rank == 0) mbar_arrive_expect_tx(full(s), 2 * (S::kA + S::kB + S::kSfB));
                    if (tma_xs) {  // 16 bytes of each row (32-value blocks: two stages' worth)
                        mbar_arrive_expect_tx(raw(s), S::kSfA);
                        tma_load_2d(at + S::kA + S::kB, &tm_xs, e4m3 ? st * 16 : st / 2 * 16, w.row, raw(s));
                    }
                    tma_load_2d_pair(at, &tm_x, st * 128, w.row, bar);
                    tma_load_2d_pair(at + S::kA, &tm_w, st * 128, w.slot * p.N + w.n0 + 128 * rank, bar);
                    // weight scales of all 256 rows (past the matrix: of rows that are not stored)
                    tma_load_2d_pair(at + S::kA + S::kB + S::kSfA, &tm_s, 0, sf + 4 * st, bar);
                    tma_load_2d_pair(at + S::kA + S::kB + S::kSfA + 2048, &tm_s, 0, sf + kt + 4 * st, bar);
                    ++issued;
                    if (++s == stages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            // after an abort the copies in flight land (on the leader's barriers) before the pair ends
            if (!ok)
                for (int i = max(0, issued - stages); i < issued; ++i) {
                    const uint32_t par = static_cast<uint32_t>(i / stages) & 1u;
                    if (rank == 0) mbar_wait_cl_drain(full(i % stages), par);
                    if (tma_xs) mbar_wait_drain(raw(i % stages), par);
                }
        }
        if (warp == 2 && rank == 0 && elect_one()) {
            int s = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int i = pair; i < tiles && ok; i += pairs)
                for (int st = 0; st < n_st; ++st) {
                    if (!(ok = mbar_wait_cl(full(s), ph, abort_flag, err))) break;
                    tc_fence_after();
                    const uint32_t at = sbase + s * S::kStage + S::kA + S::kB;
                    const uint32_t sfa = sf_col + s * S::kSfCols, sfb = sfa + 16;
                    const uint64_t da = scale_desc(at), db = scale_desc(at + S::kSfA);
                    // (a ragged last stage's pieces past K hold what the slot held before: no product reads them)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        scales_to_tmem_pair(sfa + 4 * j, da + 32 * j);
                        scales_to_tmem_pair(sfb + 8 * j, db + 32 * j);
                        scales_to_tmem_pair(sfb + 8 * j + 4, db + 32 * j + 128);
                    }
                    umma_commit_pair(scaled(s));
                    if (++s == stages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            if (!ok) {
                umma_commit_pair(sf_drained);
                mbar_wait_cl_drain(sf_drained, 0);
            }
        }
        if (warp == 1 && rank == 0 && elect_one()) {
            const uint32_t idesc = mx4_idesc(256, 256, p.fmt == ESTREAM_MX4_E8M0X32);
            int s = 0;
            uint32_t ph = 0, aph = 0;
            bool ok = true;
            for (int i = pair; i < tiles && ok; i += pairs) {
                if (!(ok = mbar_wait_cl(acc_empty, aph ^ 1u, abort_flag, err))) break;
                for (int st = 0; st < n_st; ++st) {
                    if (!(ok = mbar_wait_cl(scaled(s), ph, abort_flag, err))) break;  // after full(s)
                    tc_fence_after();
                    const int nk = min(4, kt - 4 * st);
                    const uint32_t at = sbase + s * S::kStage;
                    const uint32_t sfa = sf_col + s * S::kSfCols, sfb = sfa + 16;
                    const uint64_t da = sw128_desc(at), db = sw128_desc(at + S::kA);
                    if (nk == 4) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            mma_mx4_pair(tmem, da + 2 * j, db + 2 * j, idesc, sfa + 4 * j, sfb + 8 * j, st > 0 || j > 0);
                    } else {
                        for (int j = 0; j < nk; ++j)
                            mma_mx4_pair(tmem, da + 2 * j, db + 2 * j, idesc, sfa + 4 * j, sfb + 8 * j, st > 0 || j > 0);
                    }
                    umma_commit_pair(empty(s));
                    if (++s == stages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (!ok) break;
                umma_commit_pair(acc_full);
                aph ^= 1u;
            }
            if (!ok) {  // what was issued completes before tensor memory is freed
                umma_commit_pair(drained);
                mbar_wait_cl_drain(drained, 0);
            }
        }
    } else if (warp < 12) {
        more_registers<168>();
        zero_outside(p, blockIdx.x, gridDim.x, threadIdx.x - 128, 256);
        const int quad = warp % 4, half = (warp - 4) / 4;  // TMEM lanes; columns [128 half, + 128)
        const uint32_t acc = tmem + (static_cast<uint32_t>(quad * 32) << 16) + half * 128;
        const uint32_t release = map_rank(acc_empty, 0);
        uint8_t* stage = out_stage + (warp - 4) * 4096;
        const bool f32 = p.elem == ESTREAM_MX4_F32;
        uint32_t aph = 0;
        for (int i = pair; i < tiles; i += pairs) {
            const Work w = work(i);
            if (!__all_sync(0xffffffffu, mbar_wait_cl(acc_full, aph, abort_flag, err))) break;
            aph ^= 1u;
            tc_fence_after();
            const int row0 = w.row + quad * 32, rows = w.end - row0, n = w.n0 + half * 128;
            auto drained = [&] {  // the accumulator is read: the next tile may have it
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote_smem_release(release);
            };
            if (rows <= 0) {
                drained();
                continue;
            }
            if (f32) {
                uint32_t v[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(acc + c * 32, v[c]);
                tmem_ld_wait();
                drained();
#pragma unroll
                for (int c = 0; c < 4; ++c) {
#pragma unroll
                    for (int x = 0; x < 32; ++x) v[c][x] = __float_as_uint(__uint_as_float(v[c][x]) * p.scale);
                    if (n + c * 32 < p.N) write_rows<float>(p, &tm_out, stage, v[c], lane, row0, rows, n + c * 32, tma_out);
                }
            } else {
                uint32_t t[2][32];  // 64 columns each
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t v[2][32];
                    tmem_ld32(acc + c * 64, v[0]);
                    tmem_ld32(acc + c * 64 + 32, v[1]);
                    tmem_ld_wait();
#pragma unroll
                    for (int x = 0; x < 32; ++x) {
                        const __nv_bfloat162 q =
                            __floats2bfloat162_rn(__uint_as_float(v[x / 16][x % 16 * 2]) * p.scale,
                                                  __uint_as_float(v[x / 16][x % 16 * 2 + 1]) * p.scale);
                        t[c][x] = *reinterpret_cast<const uint32_t*>(&q);
                    }
                }
                drained();
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    if (n + c * 64 < p.N)
                        write_rows<__nv_bfloat16>(p, &tm_out, stage, t[c], lane, row0, rows, n + c * 64, tma_out);
            }
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // the stage outlives its stores
    } else {
        fewer_registers<88>();
        const int lw = warp - 12;
        int s = 0;
        uint32_t ph = 0;
        auto publish = [&] {
            if (lane == 0) {
                if (rank == 0)
                    mbar_arrive(full(s));
                else
                    mbar_arrive_remote_smem_release(map_rank(full(s), 0));
            }
            if (++s == stages) {
                s = 0;
                ph ^= 1u;
            }
        };
        if (tma_xs) {
            // a row's 16 bytes are four 64-value words: from rows as they lie to the tensor
            // core's order, in place
            bool ok = true;
            for (int i = pair; i < tiles; i += pairs)
                for (int st = 0; st < n_st; ++st) {
                    ok = __all_sync(0xffffffffu, ok && mbar_wait(raw(s), ph, abort_flag, err));
                    uint8_t* sf = smem + s * S::kStage + S::kA + S::kB;
                    uint4 v = *reinterpret_cast<const uint4*>(sf + (lw * 32 + lane) * 16);
                    if (!e4m3) {
                        const uint32_t x = st & 1 ? v.z : v.x, y = st & 1 ? v.w : v.y;
                        v = make_uint4(__byte_perm(x, 0, 0x1100), __byte_perm(x, 0, 0x3322), __byte_perm(y, 0, 0x1100),
                                       __byte_perm(y, 0, 0x3322));
                    }
                    asm volatile("bar.sync 1, 128;" ::: "memory");  // every row is in a register
                    uint32_t* to = reinterpret_cast<uint32_t*>(sf + lane * 16 + lw * 4);
                    to[0] = v.x, to[128] = v.y, to[256] = v.z, to[384] = v.w;
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (ok) publish();
                }
        } else {
            feed_scales<1, 128>(
                p, pair, pairs, tiles, n_st, lw, lane, work,
                [&]() -> uint8_t* {
                    if (!__all_sync(0xffffffffu, mbar_wait_cl(empty(s), ph ^ 1u, abort_flag, err))) return nullptr;
                    return smem + s * S::kStage + S::kA + S::kB;
                },
                publish);
        }
    }
    tc_fence_before();
    __syncwarp();
    cluster_sync();  // neither CTA ends while the other may reach its memory
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// Tensor map of rows of codes: 128-byte columns, boxes of `rows` rows.
CUresult codes_map(CUtensorMap* tm, const uint8_t* codes, int K, size_t rows, uint32_t box) {
    return encode_tmap_2d(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, codes, mx4_padded(K) / 2, rows, mx4_padded(K) / 2, 128,
                          box);
}

// Clusters of two that the device holds at once.
int max_pairs(size_t smem) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    int dev = 0, sms = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    cfg.gridDim = dim3(static_cast<unsigned>(sms & ~1));
    cfg.blockDim = dim3(kPairThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, k_mx4_product_pair, &cfg) != cudaSuccess) return 0;
    return std::min(n, sms / 2);
}

cudaError_t launch_pair(const Mx4Product& p, cudaStream_t stream) {
    CUtensorMap tm_w, tm_x, tm_s, tm_xs, tm_out;
    const uint64_t tiles_s = static_cast<uint64_t>(p.P) * ((p.N + 127) / 128) * ((p.K + 63) / 64);
    if (codes_map(&tm_w, p.wc, p.K, static_cast<size_t>(p.P) * p.N, 128) != CUDA_SUCCESS ||
        codes_map(&tm_x, p.xc, p.K, static_cast<size_t>(p.R), 128) != CUDA_SUCCESS ||
        encode_tmap_2d(&tm_s, CU_TENSOR_MAP_DATA_TYPE_UINT32, p.wt, 128, tiles_s, 512, 128, 4, false) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    // x scales and out by TMA where rows start on 16-byte boundaries; out's also have
    // to end on one (a store fills the 16 bytes that its last column begins)
    const int nb = mx4_padded(p.K) / mx4_block(p.fmt);
    const bool f32 = p.elem == ESTREAM_MX4_F32;
    const bool tma_xs = nb % 16 == 0 && reinterpret_cast<uintptr_t>(p.xs) % 16 == 0;
    const bool tma_out = reinterpret_cast<uintptr_t>(p.out) % 16 == 0 && p.ld * (f32 ? 4 : 2) % 16 == 0 &&
                         p.N * (f32 ? 4 : 2) % 16 == 0;
    tm_xs = tm_out = tm_x;
    if (tma_xs && encode_tmap_2d(&tm_xs, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.xs, nb, static_cast<uint64_t>(p.R), nb, 16, 128,
                                 false) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    if (tma_out &&
        encode_tmap_2d(&tm_out, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.out, p.N,
                       static_cast<uint64_t>(p.R), p.ld * (f32 ? 4 : 2), f32 ? 32 : 64, 32) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    const size_t prefix = p.P > 64 ? sizeof(int) * (p.P + 1) : 0;
    const int stages = static_cast<int>(
        std::min<size_t>(Pair::kStages, (225 * 1024 - Pair::kOutBytes - prefix) / Pair::kStage));
    const size_t smem = 1024 + static_cast<size_t>(stages) * Pair::kStage + Pair::kOutBytes + prefix;
    cudaError_t rc = cudaFuncSetAttribute(k_mx4_product_pair, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          static_cast<int>(smem));
    if (rc != cudaSuccess) return rc;
    int dev = 0;
    rc = cudaGetDevice(&dev);
    if (rc != cudaSuccess) return rc;
    // the query takes as long as a small launch, so a device's answer is kept
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices];
    const bool keep = prefix == 0 && dev < kDevices;
    int most = keep ? known[dev].load(std::memory_order_relaxed) : 0;
    if (most == 0) most = max_pairs(smem);
    if (keep && most > 0) known[dev].store(most, std::memory_order_relaxed);
    if (most < 1) return cudaErrorInvalidConfiguration;
    const long long tiles = (static_cast<long long>(p.R) / 256 + p.P) * ((p.N + 255) / 256);
    const int pairs = static_cast<int>(std::min<long long>(most, tiles));
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1] = overlapped();
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
    cfg.blockDim = dim3(kPairThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_mx4_product_pair, tm_w, tm_x, tm_s, tm_xs, tm_out, p, stages, tma_xs, tma_out);
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
    return launch_overlapped(k_mx4_product<NT>, dim3(grid), kMmaThreads, smem, stream, tm_w, tm_x, p, stages);
}

}  // namespace

cudaError_t launch_mx4_product(const Mx4Product& p, cudaStream_t stream) {
    if (p.R == 0 || p.N == 0) return cudaSuccess;
    // Rows a slot decide (K = 2048, N = 2048 with 64 slots of uneven rows, us a call):
    //   rows   pairs  128  64        one slot, 14336 x 4096:  pairs  128   64
    //   256      63    68             192                      14.9  18.4
    //   192      56.5  56.7           160                      16.6  20.4
    //   160      54    50             128                      16.5  14.4
    //   128      52    45             64                             11.3  11.2
    //   64       -     35   39        32                             13.4  11.0
    //   32       -     31   33
    // With several slots some hold more than the mean, and a tile of 64 rows then
    // reads their weights twice. At both shapes every form has a tile for most SMs.
    // With few weight rows none has (256 rows x N = 256 are one pair's tile); the
    // choice there is this table's all the same, and is not measured.
    const long long per = p.R / p.P;
    if (per >= 192) return launch_pair(p, stream);
    if (per > (p.P == 1 ? 64 : 31)) return launch_mma<128>(p, stream);
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
