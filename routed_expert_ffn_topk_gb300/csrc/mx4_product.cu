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
#include "tc_pair_ptx.cuh"

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
// A stage is 256 values of K, both operands' codes loaded by TMA (128-byte rows,
// 128-byte swizzle). The scales go to tensor memory by another way than
// tcgen05.cp, which runs in line with the products (73 clocks for each of a
// stage's twelve 512-byte pieces of a 256 x 256 tile, against 526 for its
// products: 220 us for 4096 x 14336 x 4096, measured): four warps, one for each
// lane quarter, write them with tcgen05.st, beside the running products, into
// columns that belong to the stage's ring slot (row r of 128: lane r % 32, column
// r / 32; each quarter holds a copy). That also takes the scales of x from where they lie: a
// route map's segments start anywhere, so no layout in advance would fit.
// ---------------------------------------------------------------------------

constexpr int kMmaThreads = 320;  // producer, MMA, 4 epilogue and 4 scale warps

constexpr int kScaleRing = 6;
template <int kGroups>
struct Scales {
    static constexpr int kX = kGroups * 2048, kSlot = kX + 2048;  // x rows of 16 bytes, 4 weight tiles
    static constexpr int kBytes = kScaleRing * kSlot;
};

template <int NT>
struct Tile {
    static constexpr int kGroups = (NT + 127) / 128;   // 128-row groups of x scales
    static constexpr int kA = 128 * 128, kB = NT * 128;
    static constexpr int kStage = kA + kB;
    static constexpr int kStages = (224 * 1024 - Scales<kGroups>::kBytes) / kStage < 8
                                       ? (224 * 1024 - Scales<kGroups>::kBytes) / kStage : 8;
    static constexpr int kAccs = 2;                    // accumulators of NT columns
    static constexpr int kSfCols = 16 + 16 * kGroups;  // a slot's scales in tensor memory
    static_assert(kAccs * NT + kStages * kSfCols <= 512, "tensor memory");
};

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10,"
        "%11, %12, %13, %14, %15, %16};" ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
        "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]),
        "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
                 : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10,"
        "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29,"
        "%30, %31, %32};" ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]),
        "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]),
        "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]),
        "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]),
        "r"(v[30]), "r"(v[31])
                 : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
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

// ---- scales ----
// The four scale warps bring a stage's scales into a shared-memory ring of their
// own, five stages ahead of the tensor core and across tiles (a row of x at a
// time: a thread per row, so that each line is looked up once; all four lane
// quarters then read all rows), and write them to tensor memory from there.
__device__ __forceinline__ void copy_or_zero(uint32_t dst, const void* src, int bytes, bool have) {
    const int n = have ? bytes : 0;
    if (bytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

// All tiles of one CTA (tiles first, first + step, ...), stage after stage, by
// threads tid = 0 .. 127: `slot_free(cols)` waits for the stage's ring slot and
// gives the warp's tensor-memory columns, `publish()` hands them over.
// After a failed wait the warps pass the remaining stages without work, so that
// they meet at the barriers.
template <int kGroups, int kRows, typename WorkAt, typename Wait, typename Publish>
__device__ __forceinline__ void write_scales(const Mx4Product& p, int first, int step, int tiles, int n_blocks,
                                             int kt, uint8_t* ring, int tid, WorkAt work, Wait slot_free,
                                             Publish publish) {
    using S = Scales<kGroups>;
    const int lane = tid & 31, n_st = (kt + 3) / 4;
    const bool e4m3 = p.fmt == ESTREAM_MX4_E4M3X16;
    const int nb = mx4_padded(p.K) / mx4_block(p.fmt), per = e4m3 ? 16 : 8;  // scale bytes of a row, of a stage
    const bool wide = nb % per == 0 && reinterpret_cast<uintptr_t>(p.xs) % per == 0;
    // what is fetched next
    int f_tile = first, f_st = 0, f_slot = 0;
    const uint8_t *f_x = p.xs, *f_w = p.wt;
    int f_rows = 0;  // rows of the tile from this thread's first on
    auto enter = [&] {
        if (f_tile >= tiles) return;
        const Work w = work(f_tile);
        f_x = p.xs + static_cast<size_t>(w.row + tid) * nb;
        f_rows = min(kRows, w.end - w.row) - tid;
        // (a pair's second half may lie past the matrix: it reads the last tile, its rows are not stored)
        f_w = p.wt + (static_cast<size_t>(w.slot) * n_blocks + min(w.n0 / 128, n_blocks - 1)) * kt * 512 + tid * 16;
    };
    auto fetch = [&] {
        if (f_tile < tiles) {
            uint8_t* at = ring + f_slot * S::kSlot + tid * 16;
#pragma unroll
            for (int q = 0; q < kGroups; ++q) {
                const uint8_t* src = f_x + static_cast<size_t>(q * 128) * nb + f_st * per;
                const bool have = q * 128 < f_rows;
                if (wide) {
                    const bool in = have && (f_st + 1) * per <= nb;
                    copy_or_zero(smem_addr(at + q * 2048), in ? src : p.xs, per, in);
                } else {
                    uint32_t v[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (i < per && have && f_st * per + i < nb)
                            v[i / 4] |= static_cast<uint32_t>(__ldg(src + i)) << (8 * (i % 4));
                    *reinterpret_cast<uint4*>(at + q * 2048) = make_uint4(v[0], v[1], v[2], v[3]);
                }
            }
            const bool in = 4 * f_st + tid / 32 < kt;
            copy_or_zero(smem_addr(at + S::kX), in ? f_w + static_cast<size_t>(f_st) * 2048 : p.wt, 16, in);
            if (++f_st == n_st) {
                f_st = 0;
                f_tile += step;
                enter();
            }
        }
        if (++f_slot == kScaleRing) f_slot = 0;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    enter();
    for (int i = 0; i < kScaleRing - 1; ++i) fetch();
    int slot = 0;
    bool ok = true;
    for (int i = first; i < tiles; i += step)
        for (int st = 0; st < n_st; ++st) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kScaleRing - 2) : "memory");
            asm volatile("bar.sync 1, 128;" ::: "memory");
            fetch();  // into the slot that every warp has read by this barrier
            const uint8_t* at = ring + slot * S::kSlot + lane * 16;
            if (++slot == kScaleRing) slot = 0;
            uint32_t va[16], vb[16 * kGroups];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint4 v = *reinterpret_cast<const uint4*>(at + S::kX + j * 512);
                va[4 * j] = v.x, va[4 * j + 1] = v.y, va[4 * j + 2] = v.z, va[4 * j + 3] = v.w;
            }
            // row i * 32 + lane is column i of each 64 values
#pragma unroll
            for (int r = 0; r < 4 * kGroups; ++r) {
                uint4 v;
                if (e4m3) {
                    v = *reinterpret_cast<const uint4*>(at + r * 512);
                } else {
                    const uint2 t = *reinterpret_cast<const uint2*>(at + r * 512);
                    v = make_uint4(__byte_perm(t.x, 0, 0x1100), __byte_perm(t.x, 0, 0x3322),
                                   __byte_perm(t.y, 0, 0x1100), __byte_perm(t.y, 0, 0x3322));
                }
                vb[r] = v.x, vb[4 * kGroups + r] = v.y, vb[8 * kGroups + r] = v.z, vb[12 * kGroups + r] = v.w;
            }
            uint32_t cols = 0;
            ok = ok && slot_free(cols);
            if (!ok) continue;
            tmem_st16(cols, va);
            if constexpr (kGroups == 2)
                tmem_st32(cols + 16, vb);
            else
                tmem_st16(cols + 16, vb);
            tmem_st_wait();
            tc_fence_before();
            publish();
        }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
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
    int* base = p.P <= 64 ? base_small : reinterpret_cast<int*>(smem + stages * S::kStage + Scales<S::kGroups>::kBytes);
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
                for (int st = 0; st < n_st; ++st) {
                    if (!(ok = mbar_wait(empty(s), ph ^ 1u, abort_flag, err))) break;
                    const uint32_t at = sbase + s * S::kStage;
                    mbar_arrive_expect_tx(full(s), S::kA + S::kB);
                    tma_load_2d(at, &tm_w, st * 128, w.slot * p.N + w.n0, full(s));
                    tma_load_2d(at + S::kA, &tm_x, st * 128, w.row, full(s));
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
            int s = 0, a = 0;
            uint32_t ph = 0, aph = 0;
            bool ok = true;
            for (int i = blockIdx.x; i < tiles && ok; i += gridDim.x) {
                if (!(ok = mbar_wait(acc_empty(a), aph ^ 1u, abort_flag, err))) break;
                const uint32_t acc = tmem + a * NT;
                for (int st = 0; st < n_st; ++st) {
                    if (!(ok = mbar_wait(full(s), ph, abort_flag, err))) break;
                    tc_fence_after();
                    const int nk = min(4, kt - 4 * st);
                    const uint32_t at = sbase + s * S::kStage;
                    const uint32_t sfa = sf_col + s * S::kSfCols, sfb = sfa + 16;
                    const uint64_t da = sw128_desc(at), db = sw128_desc(at + S::kA);
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
        const uint32_t quarter = static_cast<uint32_t>(warp % 4 * 32) << 16;
        int s = 0;
        uint32_t ph = 0;
        write_scales<S::kGroups, NT>(
            p, blockIdx.x, gridDim.x, tiles, n_blocks, kt, smem + stages * S::kStage, threadIdx.x - 192,
            [&](int i) { return work_at(p, base, NT, i); },
            [&](uint32_t& cols) {
                if (!__all_sync(0xffffffffu, mbar_wait(empty(s), ph ^ 1u, abort_flag, err))) return false;
                tc_fence_after();
                cols = sf_col + quarter + s * S::kSfCols;
                return true;
            },
            [&] {
                __syncwarp();
                if (lane == 0) mbar_arrive(full(s));
                if (++s == stages) {
                    s = 0;
                    ph ^= 1u;
                }
            });
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------
// Pair form: clusters of two CTAs on 256 weight rows x 256 rows of x with
// cta_group::2 (M = 256, N = 256). Each CTA holds its 128 weight rows and half of
// the x rows of a stage, 32 KB for the 128 x 256 x 256 products that it does,
// against 48 KB in the form above: that one reads and fills shared memory at more
// than its 128 bytes a clock, and L2 at more than it delivers. The leader (rank 0)
// issues the products of both; the scales of x of all 256 rows are written in both
// CTAs. One 256-column accumulator and the scales fill tensor
// memory, so the epilogue is not hidden behind the next tile; its eight warps
// first drain the accumulator into registers (bf16 packed) and store afterwards.
// ---------------------------------------------------------------------------

constexpr int kPairThreads = 448;  // producer, MMA, 8 epilogue and 4 scale warps
struct Pair {
    static constexpr int kA = 128 * 128, kB = 128 * 128;
    static constexpr int kStage = kA + kB;
    static constexpr int kStages = 5;  // 256 accumulator and 5 x 48 scale columns of 512
    static constexpr int kSfCols = 48;
};

__device__ __forceinline__ void mma_mx4_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                             uint32_t sfb, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

__global__ void __launch_bounds__(kPairThreads, 1) k_mx4_product_pair(const __grid_constant__ CUtensorMap tm_w,
                                                                     const __grid_constant__ CUtensorMap tm_x,
                                                                     const Mx4Product p, int stages) {
    using S = Pair;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * S::kStages + 3];
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
    int* base = p.P <= 64 ? base_small : reinterpret_cast<int*>(smem + stages * S::kStage + Scales<2>::kBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_rank());
    const uint32_t sbase = smem_addr(smem);
    auto full = [&](int s) { return smem_addr(&bars[s]); };            // the leader's
    auto empty = [&](int s) { return smem_addr(&bars[S::kStages + s]); };
    const uint32_t acc_full = smem_addr(&bars[2 * S::kStages]);
    const uint32_t acc_empty = smem_addr(&bars[2 * S::kStages + 1]);   // the leader's
    const uint32_t drained = smem_addr(&bars[2 * S::kStages + 2]);
    if (threadIdx.x == 0) {
        abort_word = 0;
        for (int s = 0; s < stages; ++s) {
            mbar_init(full(s), 1 + 4 + 4);  // the leader's expect_tx and both CTAs' scale warps
            mbar_init(empty(s), 1);
        }
        mbar_init(acc_full, 1);
        mbar_init(acc_empty, 8 + 8);
        mbar_init(drained, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_addr(&tmem_slot), 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    tile_prefix(p, 256, base, sums);
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = tmem_slot, sf_col = tmem + 256;
    const int n_pairs_blocks = (p.N + 255) / 256;
    const int tiles = base[p.P] * n_pairs_blocks;
    const int kt = (p.K + 63) / 64, n_st = (kt + 3) / 4;
    const int n_blocks = (p.N + 127) / 128;
    const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);
    int* err = &g_mx4_err;
    auto work = [&](int i) {
        Work w = work_at(p, base, 256, i);
        w.n0 = w.n0 * 2 + 128 * rank;
        return w;
    };

    if (warp == 0) {
        if (lane == 0) {
            int s = 0, issued = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int i = pair; i < tiles && ok; i += pairs) {
                const Work w = work(i);
                for (int st = 0; st < n_st; ++st) {
                    if (!(ok = mbar_wait_cl(empty(s), ph ^ 1u, abort_flag, err))) break;
                    const uint32_t at = sbase + s * S::kStage;
                    const uint32_t bar = map_rank(full(s), 0);
                    if (rank == 0) mbar_arrive_expect_tx(full(s), 2 * (S::kA + S::kB));
                    tma_load_2d_pair(at, &tm_w, st * 128, w.slot * p.N + w.n0, bar);
                    tma_load_2d_pair(at + S::kA, &tm_x, st * 128, w.row + 128 * rank, bar);
                    ++issued;
                    if (++s == stages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            // after an abort the copies in flight land (on the leader's barriers) before the pair ends
            if (!ok && rank == 0)
                for (int i = max(0, issued - stages); i < issued; ++i)
                    mbar_wait_cl_drain(full(i % stages), static_cast<uint32_t>(i / stages) & 1u);
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            const uint32_t idesc = mx4_idesc(256, 256, p.fmt == ESTREAM_MX4_E8M0X32);
            int s = 0;
            uint32_t ph = 0, aph = 0;
            bool ok = true;
            for (int i = pair; i < tiles && ok; i += pairs) {
                if (!(ok = mbar_wait_cl(acc_empty, aph ^ 1u, abort_flag, err))) break;
                tc_fence_after();
                for (int st = 0; st < n_st; ++st) {
                    if (!(ok = mbar_wait_cl(full(s), ph, abort_flag, err))) break;
                    tc_fence_after();
                    const int nk = min(4, kt - 4 * st);
                    const uint32_t at = sbase + s * S::kStage;
                    const uint32_t sfa = sf_col + s * S::kSfCols, sfb = sfa + 16;
                    const uint64_t da = sw128_desc(at), db = sw128_desc(at + S::kA);
                    for (int j = 0; j < nk; ++j)
                        mma_mx4_pair(tmem, da + 2 * j, db + 2 * j, idesc, sfa + 4 * j, sfb + 8 * j, st > 0 || j > 0);
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
    } else if (warp < 10) {
        zero_outside(p, blockIdx.x, gridDim.x, threadIdx.x - 64, 256);
        const int quad = warp % 4, half = (warp - 2) / 4;  // TMEM lanes; columns [128 half, + 128)
        const uint32_t acc = tmem + (static_cast<uint32_t>(quad * 32) << 16) + half * 128;
        const uint32_t release = map_rank(acc_empty, 0);
        uint32_t aph = 0;
        for (int i = pair; i < tiles; i += pairs) {
            const Work w = work(i);
            if (!__all_sync(0xffffffffu, mbar_wait_cl(acc_full, aph, abort_flag, err))) break;
            aph ^= 1u;
            tc_fence_after();
            const int n = w.n0 + quad * 32 + lane;
            const int rows = min(128, w.end - w.row - half * 128);  // may be <= 0
            const size_t row0 = static_cast<size_t>(w.row + half * 128) * p.ld + n;
            auto done = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cl(release);
            };
            if (p.elem == ESTREAM_MX4_BF16) {
                uint32_t v[64];  // two rows a word
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t t[32];
                    if (c * 32 < rows) {
                        tmem_ld32(acc + c * 32, t);
                        tmem_ld_wait();
                    }
#pragma unroll
                    for (int x = 0; x < 16; ++x) {
                        const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(t[2 * x]) * p.scale,
                                                                       __uint_as_float(t[2 * x + 1]) * p.scale);
                        v[c * 16 + x] = *reinterpret_cast<const uint32_t*>(&b);
                    }
                }
                done();
                if (n < p.N) {
                    uint16_t* out = static_cast<uint16_t*>(p.out) + row0;
#pragma unroll
                    for (int x = 0; x < 64; ++x) {
                        if (2 * x < rows) out[2 * x * p.ld] = static_cast<uint16_t>(v[x]);
                        if (2 * x + 1 < rows) out[(2 * x + 1) * p.ld] = static_cast<uint16_t>(v[x] >> 16);
                    }
                }
            } else {
                float* out = static_cast<float*>(p.out) + row0;
                for (int c = 0; c < 4; ++c) {
                    uint32_t t[32];
                    if (c * 32 < rows) {
                        tmem_ld32(acc + c * 32, t);
                        tmem_ld_wait();
                    }
                    if (c == 3) done();
                    if (n < p.N)
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            if (c * 32 + x < rows) out[(c * 32 + x) * p.ld] = __uint_as_float(t[x]) * p.scale;
                }
            }
        }
    } else {
        const uint32_t quarter = static_cast<uint32_t>(warp % 4 * 32) << 16;
        int s = 0;
        uint32_t ph = 0;
        write_scales<2, 256>(
            p, pair, pairs, tiles, n_blocks, kt, smem + stages * S::kStage, threadIdx.x - 320, work,
            [&](uint32_t& cols) {
                if (!__all_sync(0xffffffffu, mbar_wait_cl(empty(s), ph ^ 1u, abort_flag, err))) return false;
                tc_fence_after();
                cols = sf_col + quarter + s * S::kSfCols;
                return true;
            },
            [&] {
                __syncwarp();
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
            });
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
    CUtensorMap tm_w, tm_x;
    if (codes_map(&tm_w, p.wc, p.K, static_cast<size_t>(p.P) * p.N, 128) != CUDA_SUCCESS ||
        codes_map(&tm_x, p.xc, p.K, static_cast<size_t>(p.R), 128) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    const size_t prefix = p.P > 64 ? sizeof(int) * (p.P + 1) : 0;
    const int stages = static_cast<int>(std::min<size_t>(Pair::kStages, (225 * 1024 - Scales<2>::kBytes - prefix) / Pair::kStage));
    const size_t smem = 1024 + static_cast<size_t>(stages) * Pair::kStage + Scales<2>::kBytes + prefix;
    cudaError_t rc = cudaFuncSetAttribute(k_mx4_product_pair, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          static_cast<int>(smem));
    if (rc != cudaSuccess) return rc;
    const int most = max_pairs(smem);
    if (most < 1) return cudaErrorInvalidConfiguration;
    const long long tiles = (static_cast<long long>(p.R) / 256 + p.P) * ((p.N + 255) / 256);
    const int pairs = static_cast<int>(std::min<long long>(most, tiles));
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
    cfg.blockDim = dim3(kPairThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_mx4_product_pair, tm_w, tm_x, p, stages);
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
    const int stages = static_cast<int>(std::min<size_t>(S::kStages, (225 * 1024 - Scales<S::kGroups>::kBytes - prefix) / S::kStage));
    const size_t smem = 1024 + static_cast<size_t>(stages) * S::kStage + Scales<S::kGroups>::kBytes + prefix;
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
    if (per >= 192) return launch_pair(p, stream);
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
