// One MoE layer for the few tokens of a generation step, in one launch.
//
// Y_t = A_t + sum_j alpha_{t,j} W_e^d (SiLU(W_e^g X_t) (*) W_e^u X_t) over the
// token's k experts e_{t,j} (+ shared experts with weight 1), the layer of
// "EStream: Fast and Memory-Efficient MoE Prefill through Expert
// Virtualization on Mobile NPUs" section 3.2, Eq. 1 and Eq. 2, for at most
// kDecodeMaxT tokens over the arena that the prompt pass reads. Optionally
// with the router logits X W_r^T in front.
//
// At these token counts every weight of a chosen expert is read once and used
// for a handful of multiply-adds, so the floor is the HBM time of the chosen
// experts' weights; everything else is latency to hide.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "estream_internal.h"

namespace es {
namespace {
#include "tc_ptx.cuh"
}  // namespace

#include "route_topk.cuh"

namespace {

constexpr uint64_t kDecodeWaitNs = 1000000000ull;  // 1 s: bound of a grid barrier
constexpr int kSimpleThreads = 512;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// Barrier of the whole (cooperative) grid, bounded in time: returns false
// after recording a timeout. sync[0] counts arrivals and only grows within a
// launch; decode_leave zeroes it for the next one.
__device__ bool decode_barrier(int* sync, int generation, int* err, int* ok_flag, bool withhold) {
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        if (!withhold) atomicAdd(sync, 1);
        const int target = generation * static_cast<int>(gridDim.x);
        const uint64_t t0 = global_ns();
        bool ok = true;
        while (true) {
            int seen;
            asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(seen) : "l"(sync) : "memory");
            if (seen >= target) break;
            if (global_ns() - t0 > kDecodeWaitNs) {
                record_error(err, kDevErrTimeout);
                ok = false;
                break;
            }
        }
        __threadfence();
        *ok_flag = ok ? 1 : 0;
    }
    __syncthreads();
    return *ok_flag != 0;
}

// Every CTA passes here last; the one that completes the count leaves both
// words zero, also after a barrier gave up.
__device__ __forceinline__ void decode_leave(int* sync) {
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        if (atomicAdd(sync + 1, 1) == static_cast<int>(gridDim.x) - 1) {
            sync[0] = 0;
            sync[1] = 0;
        }
    }
}

// The call's routes in shared memory, formed by every CTA for itself.
struct Routes {
    int* ids;        // [T k] expert of each route
    float* alpha;    // [T k]
    int* counts;     // [E + 1]
    uint32_t* mask;  // [E] bit t: token t goes to the expert
    int* act;        // [n_act] experts with a token, ascending
    int* row0;       // [n_act] first h row of the expert (one row a token, ascending t)
    int* row_tok;    // [T k] token of each h row
    float* row_alpha;  // [T k] its weight
    int* n_act;
};

__host__ __device__ inline size_t routes_bytes(int R, int E) {
    return (sizeof(int) * (4 * static_cast<size_t>(R) + 4 * static_cast<size_t>(E) + 2) + 15) / 16 * 16;
}

__device__ Routes routes_at(void* smem, int R, int E) {
    Routes r;
    r.ids = static_cast<int*>(smem);
    r.alpha = reinterpret_cast<float*>(r.ids + R);
    r.counts = r.ids + 2 * R;
    r.mask = reinterpret_cast<uint32_t*>(r.counts + E + 1);
    r.act = reinterpret_cast<int*>(r.mask + E);
    r.row0 = r.act + E;
    r.row_tok = r.row0 + E;
    r.row_alpha = reinterpret_cast<float*>(r.row_tok + R);
    r.n_act = r.row_tok + 2 * R;
    return r;
}

// Top-k of every token (a warp per token), then the experts' token masks and
// the list of experts in use. T <= 32 is what lets one word hold a mask, and
// a token's row among its expert's rows be a count of the lower bits.
__device__ void build_routes(const Routes& r, const float* logits, int T, int E, int k, int renorm,
                             int* err) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        r.counts[e] = 0;
        r.mask[e] = 0u;
    }
    __syncthreads();
    for (int t = warp; t < T; t += nw) {
        const float* l = logits + static_cast<size_t>(t) * E;
        if (E <= 64)
            topk_token<2>(t, l, E, k, renorm, nullptr, E, r.ids, r.alpha, r.counts, err);
        else if (E <= 256)
            topk_token<8>(t, l, E, k, renorm, nullptr, E, r.ids, r.alpha, r.counts, err);
        else
            topk_token<kMaxPerLane>(t, l, E, k, renorm, nullptr, E, r.ids, r.alpha, r.counts, err);
        __syncwarp();
        if (lane < k && r.ids[t * k + lane] >= 0) atomicOr(&r.mask[r.ids[t * k + lane]], 1u << t);
    }
    __syncthreads();
    if (warp == 0) {
        int n = 0, rows = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            const int c = e < E ? __popc(r.mask[e]) : 0;
            const unsigned has = __ballot_sync(0xffffffffu, c > 0);
            int incl = c;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += o;
            }
            if (c > 0) {
                const int at = n + __popc(has & ((1u << lane) - 1u));
                r.act[at] = e;
                r.row0[at] = rows + incl - c;
            }
            n += __popc(has);
            rows += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) *r.n_act = n;
    }
    __syncthreads();
    // each route's h row: its expert's first row and the earlier tokens there
    // (counts, now free, holds the experts' first rows)
    for (int a = threadIdx.x; a < *r.n_act; a += blockDim.x) r.counts[r.act[a]] = r.row0[a];
    __syncthreads();
    for (int i = threadIdx.x; i < T * k; i += blockDim.x) {
        const int e = r.ids[i], t = i / k;
        if (e < 0) continue;
        const int row = r.counts[e] + __popc(r.mask[e] & ((1u << t) - 1u));
        r.row_tok[row] = t;
        r.row_alpha[row] = r.alpha[i];
    }
    __syncthreads();
}

template <int kType>
__device__ __forceinline__ float x_at(const void* X, size_t i) {
    return kType == ESTREAM_F32 ? static_cast<const float*>(X)[i]
                                : __bfloat162float(static_cast<const __nv_bfloat16*>(X)[i]);
}

// Router logits (bf16 X and W_r): a warp per (token, expert).
__device__ void router_rows(const DecodeCall& d) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    const __nv_bfloat16* X = static_cast<const __nv_bfloat16*>(d.X);
    const __nv_bfloat16* W = static_cast<const __nv_bfloat16*>(d.W_r);
    for (int p = blockIdx.x * nw + warp; p < d.T * d.E; p += gridDim.x * nw) {
        const int t = p / d.E, e = p % d.E;
        const uint4* x = reinterpret_cast<const uint4*>(X + static_cast<size_t>(t) * d.H);
        const uint4* w = reinterpret_cast<const uint4*>(W + static_cast<size_t>(e) * d.H);
        float s = 0.0f;
#pragma unroll 4
        for (int c = lane; c < d.H / 8; c += 32) {
            const uint4 a = __ldg(x + c), b = __ldg(w + c);
            const uint32_t av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s = fmaf(__uint_as_float(av[i] << 16), __uint_as_float(bv[i] << 16), s);
                s = fmaf(__uint_as_float(av[i] & 0xffff0000u), __uint_as_float(bv[i] & 0xffff0000u), s);
            }
        }
        s = warp_sum(s);
        if (lane == 0) d.logits_out[p] = s;
    }
}

// fp32 planes (row-major): a warp per h row, then a warp per Y column, every
// product an fp32 multiply-add on the CUDA cores.
__global__ void __launch_bounds__(kSimpleThreads) k_layer_decode_simple(const DecodeCall d) {
    extern __shared__ int smem[];
    __shared__ int ok_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    const int gw = blockIdx.x * nw + warp, gn = gridDim.x * nw;
    const int H = d.H, F = d.F, Fs = d.F_shared, T = d.T, k = d.k;
    const Routes r = routes_at(smem, T * k, d.E);
    int gen = 0;
    bool ok = true;
    {
        build_routes(r, d.logits, T, d.E, k, d.renorm, d.err);
        const int n_act = *r.n_act;
        const int routed = n_act * F;
        for (int u = gw; u < routed + d.n_shared * Fs; u += gn) {
            const bool sh = u >= routed;
            const int a = sh ? (u - routed) / Fs : u / F;
            const int f = sh ? (u - routed) % Fs : u % F;
            const int e = sh ? a : r.act[a];
            const size_t slot = sh ? static_cast<size_t>(a) : static_cast<size_t>(d.phi[e]);
            const char* pg = sh ? d.sh_g + slot * d.S_sh : d.plane_g + slot * d.S_gu;
            const char* pu = sh ? d.sh_u + slot * d.S_sh : d.plane_u + slot * d.S_gu;
            const float scale = sh ? d.sh_scale[slot] : d.scale[slot];
            uint32_t m = sh ? (T == 32 ? 0xffffffffu : (1u << T) - 1u) : r.mask[e];
            int row = sh ? a * T : r.row0[a];
            for (; m; m &= m - 1, ++row) {
                const int t = __ffs(m) - 1;
                float g = 0.0f, up = 0.0f;
                for (int c = lane; c < H; c += 32) {
                    const float x = x_at<ESTREAM_F32>(d.X, static_cast<size_t>(t) * H + c);
                    g = fmaf(reinterpret_cast<const float*>(pg)[static_cast<size_t>(f) * H + c], x, g);
                    up = fmaf(reinterpret_cast<const float*>(pu)[static_cast<size_t>(f) * H + c], x, up);
                }
                g = warp_sum(g);
                up = warp_sum(up);
                if (lane == 0) {
                    const float v = scale * (g / (1.0f + expf(-g)) * up);
                    if (sh)
                        static_cast<float*>(d.h_shared)[static_cast<size_t>(row) * Fs + f] = v;
                    else
                        static_cast<float*>(d.h)[static_cast<size_t>(row) * F + f] = r.row_alpha[row] * v;
                }
            }
        }
        ok = decode_barrier(d.sync, ++gen, d.err, &ok_flag, (d.withhold & 2) && blockIdx.x == 0);
    }
    if (ok) {
        const int n_act = *r.n_act;
        for (int o = gw; o < H; o += gn)
            for (int t = 0; t < T; ++t) {
                float y = 0.0f;
                for (int a = 0; a < n_act + d.n_shared; ++a) {
                    const bool sh = a >= n_act;
                    const int e = sh ? a - n_act : r.act[a];
                    if (!sh && !((r.mask[e] >> t) & 1u)) continue;
                    const size_t slot = sh ? static_cast<size_t>(e) : static_cast<size_t>(d.phi[e]);
                    const char* pd = sh ? d.sh_d + slot * d.S_sh : d.plane_d + slot * d.S_d;
                    const int n = sh ? Fs : F;
                    const float* h =
                        sh ? static_cast<const float*>(d.h_shared) + (static_cast<size_t>(e) * T + t) * Fs
                           : static_cast<const float*>(d.h) +
                                 static_cast<size_t>(r.row0[a] + __popc(r.mask[e] & ((1u << t) - 1u))) * F;
                    for (int c = lane; c < n; c += 32)
                        y = fmaf(reinterpret_cast<const float*>(pd)[static_cast<size_t>(o) * n + c], __ldcg(h + c), y);
                }
                y = warp_sum(y);
                if (lane == 0) {
                    const size_t at = static_cast<size_t>(t) * H + o;
                    d.Y[at] = (d.A ? x_at<ESTREAM_F32>(d.A, at) : d.Y[at]) + y;
                }
            }
    }
    decode_leave(d.sync);
}

// ---------------------------------------------------------------------------
// Streaming form (bf16 and 4-bit planes): one persistent CTA per SM, 16
// consumer warps and one producer warp.
//
// The grid splits the h rows of all chosen experts (then the rows of Y) into
// one contiguous range a CTA, to a single row (4-bit: 8 and 4 rows, whose
// scales fill 16 bytes), so every SM streams the same number of weight bytes.
// The producer copies the range's rows, box by box as the arena stores them,
// into a shared-memory ring with cp.async.bulk; it needs the routes but not h,
// so it runs into the down weights while the consumers still wait at the grid
// barrier between the projections, and HBM does not idle there.
//
// A stage holds 16 units, one a consumer warp: 64 reduction values of a row
// tile. The products are mma.sync m16n8k16 with the weights as the 16 rows and
// the tokens as the 8 columns: at 8 columns an instruction covers 512 bytes of
// weights, far above what HBM delivers, so a tcgen05 tile of at least 64 rows
// by 8 columns through tensor memory would add latency and no speed. A tile of
// h is 8 gate rows over 8 up rows, which puts gate and up of one h value in one
// lane. Within 64 values a lane takes runs of 8 (16 bytes) as its k indices, in
// weights and tokens alike, so both come as 16-byte loads without a transpose.
//
// h leaves as three bf16 parts (8 leading bits, the next 8, the next 8), which
// together hold the fp32 value; the down weights, fp16 in the arena, are bf16
// numbers times a power of two and convert to bf16 exactly. So every product of
// both projections is exact and only fp32 sums round. In the down projection
// column t is token t whatever the expert, so the accumulators run on over the
// experts in ascending order and Y needs no atomics.
// ---------------------------------------------------------------------------

constexpr int kConsumers = 16;
constexpr int kStreamThreads = 32 * (kConsumers + 1);
constexpr int kMaxStages = 6;

template <bool kQ4>
struct Stream {
    static constexpr int kHRows = kQ4 ? 32 : 8;    // h rows of a gate/up tile
    static constexpr int kYRows = kQ4 ? 32 : 16;   // Y rows of a down tile
    static constexpr int kHStep = kQ4 ? 8 : 1;     // granularity of a CTA's range
    static constexpr int kYStep = kQ4 ? 4 : 1;
    static constexpr int kHTiles = kHRows / 8;     // m16 tiles (8 gate + 8 up rows)
    static constexpr int kYTiles = kYRows / 16;
    // one plane's part of a unit: rows x 64 weights. 4-bit: two column blocks
    // of 16 bytes a row, then 4 bytes of scales a row.
    static constexpr int kRowBytes = kQ4 ? 36 : 128;
    static constexpr int kHUnit = 2 * kHRows * kRowBytes;
    static constexpr int kYUnit = kYRows * kRowBytes;
    static constexpr int kStage = kConsumers * (kHUnit > kYUnit ? kHUnit : kYUnit);
    static constexpr int kRed = kConsumers * (kHTiles > kYTiles ? kHTiles : kYTiles) * 128;  // floats
};

__device__ __forceinline__ void bulk_row_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
// Two fp16 weights of the down plane as bf16 (exact: see above).
__device__ __forceinline__ uint32_t half2_to_bf162(uint32_t w) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t*>(&b);
}
// Codes p (low half) and p + 1 (high half) of a 4-bit word as bf16 weights: the
// code placed in 128 + q, then - 136 and * d, both exact (d has 5 bits).
__device__ __forceinline__ uint32_t q4_pair(uint32_t word, int p, __nv_bfloat162 d) {
    const uint32_t u = ((word >> (4 * p)) & 0x000f000fu) | 0x43004300u;
    const __nv_bfloat162 q = __hsub2_rn(*reinterpret_cast<const __nv_bfloat162*>(&u),
                                        __floats2bfloat162_rn(136.0f, 136.0f));
    const __nv_bfloat162 v = __hmul2_rn(q, d);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// A run of rows of one expert's plane: rows [r, r + n) of slot-plane p.
struct Rows {
    int at;       // index among the chosen experts, then the shared ones
    int row, n;
};

// The tile of a CTA's h range that starts at `pos` (rows of the chosen experts,
// then of the shared ones): the rest of the expert, of the range, or of the
// aligned tile, whichever ends first.
template <int kRows>
__device__ __forceinline__ Rows h_tile(int pos, int end, int routed, int n_act, int F, int Fs) {
    Rows t;
    const int base = pos < routed ? 0 : routed, len = pos < routed ? F : Fs;
    t.at = (pos - base) / len;
    t.row = (pos - base) % len;
    t.n = min(min(len - t.row, end - pos), kRows - t.row % kRows);
    if (pos >= routed) t.at += n_act;
    return t;
}
// The tile of a CTA's Y range that starts at row o; a down box has 256 rows.
template <int kRows>
__device__ __forceinline__ int y_tile(int o, int end) {
    return min(min(kRows, end - o), 256 - o % 256);
}
__device__ __forceinline__ int share(int total, int step, int part) {
    const long long units = total / step;
    return static_cast<int>(units * part / gridDim.x) * step;
}

// k-blocks of a stage of the gate/up pass: K split evenly into stages of at most 16
__host__ __device__ __forceinline__ int h_chunks(int KB) { return (KB + kConsumers - 1) / kConsumers; }

// kNT: token tiles of 8 that the accumulators have room for (T <= 8 kNT).
template <bool kQ4, int kNT>
__global__ void __launch_bounds__(kStreamThreads, 1) k_layer_decode(const DecodeCall d, int stages) {
    using S = Stream<kQ4>;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * kMaxStages];
    __shared__ int ok_flag;
    __shared__ int abort_word;
    volatile int* abort_flag = &abort_word;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int H = d.H, F = d.F, Fs = d.F_shared, T = d.T, k = d.k;
    const int KB = H / 64, FB = F / 64, FsB = Fs / 64;
    const uint32_t ring = smem_addr(smem_raw);
    float* red = reinterpret_cast<float*>(smem_raw + static_cast<size_t>(stages) * S::kStage);
    const Routes r = routes_at(red + S::kRed, T * k, d.E);
    auto full = [&](int s) { return smem_addr(&bars[s]); };
    auto empty = [&](int s) { return smem_addr(&bars[kMaxStages + s]); };
    if (threadIdx.x == 0) {
        abort_word = 0;
        for (int s = 0; s < stages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), kConsumers);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    int gen = 0;
    bool ok = true;
    if (d.W_r) {
        router_rows(d);
        ok = decode_barrier(d.sync, ++gen, d.err, &ok_flag, (d.withhold & 1) && blockIdx.x == 0);
    }
    if (!ok) {
        decode_leave(d.sync);
        return;
    }
    build_routes(r, d.W_r ? d.logits_out : d.logits, T, d.E, k, d.renorm, d.err);
    const int n_act = *r.n_act;
    const int routed = n_act * F, h_total = routed + d.n_shared * Fs;
    const int h0 = share(h_total, S::kHStep, blockIdx.x), h1 = share(h_total, S::kHStep, blockIdx.x + 1);
    const int y0 = share(H, S::kYStep, blockIdx.x), y1 = share(H, S::kYStep, blockIdx.x + 1);
    const int chunks = h_chunks(KB), per = (KB + chunks - 1) / chunks;
    const int YB = n_act * FB + d.n_shared * FsB;  // k-blocks of a Y row

    if (warp == kConsumers) {
        // ---- producer: the whole warp issues, a lane a copy ----
        int s = 0;
        uint32_t ph = 0;
        int issued = 0;  // stages filled so far
        bool live = true;
        auto wait_empty = [&]() {
            const bool w = mbar_wait(empty(s), ph ^ 1u, abort_flag, d.err);
            return __all_sync(0xffffffffu, w);
        };
        auto next = [&]() {
            ++issued;
            if (++s == stages) {
                s = 0;
                ph ^= 1u;
            }
        };
        for (int pos = h0; pos < h1 && live;) {
            const Rows t = h_tile<S::kHRows>(pos, h1, routed, n_act, F, Fs);
            pos += t.n;
            const bool sh = t.at >= n_act;
            const size_t slot = sh ? static_cast<size_t>(t.at - n_act) : static_cast<size_t>(d.phi[r.act[t.at]]);
            const char* base = lane & 1 ? (sh ? d.sh_u + slot * d.S_sh : d.plane_u + slot * d.S_gu)
                                        : (sh ? d.sh_g + slot * d.S_sh : d.plane_g + slot * d.S_gu);
            base += static_cast<size_t>(t.row / 128) * KB * (128 * S::kRowBytes);
            const int br = t.row % 128, tr = t.row % S::kHRows;
            for (int c = 0; c < chunks && live; ++c) {
                const int kb = c * per + (lane >> 1), nk = min(per, KB - c * per);
                if (!(live = wait_empty())) break;
                if (lane == 0) mbar_arrive_expect_tx(full(s), 2u * nk * t.n * S::kRowBytes);
                __syncwarp();
                if ((lane >> 1) < nk) {
                    const uint32_t dst = ring + s * S::kStage + (lane >> 1) * S::kHUnit +
                                         (lane & 1) * (S::kHRows * S::kRowBytes);
                    const char* src = base + static_cast<size_t>(kb) * (128 * S::kRowBytes);
                    if (kQ4) {
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            bulk_row_load(dst + j * (S::kHRows * 16) + tr * 16, src + j * 2048 + br * 16, t.n * 16,
                                          full(s));
                        bulk_row_load(dst + S::kHRows * 32 + tr * 4, src + 4096 + br * 4, t.n * 4, full(s));
                    } else {
                        bulk_row_load(dst + tr * 128, src + br * 128, t.n * 128, full(s));
                    }
                }
                next();
            }
        }
        for (int o = y0; o < y1 && live;) {
            const int n = y_tile<S::kYRows>(o, y1);
            for (int q0 = 0; q0 < YB && live; q0 += kConsumers) {
                const int nk = min(kConsumers, YB - q0);
                if (!(live = wait_empty())) break;
                if (lane == 0) mbar_arrive_expect_tx(full(s), 1u * nk * n * S::kRowBytes);
                __syncwarp();
                if (lane < nk) {
                    const int q = q0 + lane;
                    const bool sh = q >= n_act * FB;
                    const int len = sh ? FsB : FB, p = sh ? q - n_act * FB : q;
                    const int a = p / len, kb = p % len;
                    const size_t slot = sh ? static_cast<size_t>(a) : static_cast<size_t>(d.phi[r.act[a]]);
                    const char* src = (sh ? d.sh_d + slot * d.S_sh : d.plane_d + slot * d.S_d) +
                                      (static_cast<size_t>(o / 256) * len + kb) * (256 * S::kRowBytes);
                    const uint32_t dst = ring + s * S::kStage + lane * S::kYUnit;
                    const int br = o % 256;
                    if (kQ4) {
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            bulk_row_load(dst + j * (S::kYRows * 16), src + j * 4096 + br * 16, n * 16, full(s));
                        bulk_row_load(dst + S::kYRows * 32, src + 8192 + br * 4, n * 4, full(s));
                    } else {
                        bulk_row_load(dst, src + br * 128, n * 128, full(s));
                    }
                }
                next();
            }
            o += n;
        }
        // after an abort the copies still in flight must land before the CTA ends
        if (!live)
            for (int i = max(0, issued - stages); i < issued; ++i)
                mbar_wait_drain(full(i % stages), static_cast<uint32_t>(i / stages) & 1u);
    } else {
        // ---- consumers ----
        const int g = lane >> 2, tq = lane & 3;
        int s = 0;
        uint32_t ph = 0;
        bool live = true;
        // A wait that gives up raises the abort flag, with which every other wait
        // ends at once; the warp then passes the remaining stages without work,
        // so that all consumers meet at every named barrier.
        auto wait_full = [&]() {
            live = __all_sync(0xffffffffu, live && mbar_wait(full(s), ph, abort_flag, d.err));
            return live;
        };
        auto release = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(empty(s));
            if (++s == stages) {
                s = 0;
                ph ^= 1u;
            }
        };
        auto sync_consumers = [] { asm volatile("bar.sync 1, %0;" ::"n"(32 * kConsumers) : "memory"); };
        // sum of the 16 warps' partial tiles, value i of m16 tile m
        auto reduced = [&](int m, int i) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kConsumers; ++w) v += red[(w * S::kHTiles + m) * 128 + i];
            return v;
        };
        for (int pos = h0; pos < h1;) {
            const Rows t = h_tile<S::kHRows>(pos, h1, routed, n_act, F, Fs);
            pos += t.n;
            const bool sh = t.at >= n_act;
            const int e = sh ? t.at - n_act : r.act[t.at];
            const int cnt = sh ? T : __popc(r.mask[e]);
            const int row0 = sh ? e * T : r.row0[t.at];
            const int nt = (cnt + 7) / 8;
            const __nv_bfloat16* xp[kNT];
#pragma unroll
            for (int j = 0; j < kNT; ++j) {
                const int c = j * 8 + g;
                xp[j] = c < cnt ? static_cast<const __nv_bfloat16*>(d.X) +
                                      static_cast<size_t>(sh ? c : r.row_tok[row0 + c]) * H + tq * 8
                                : nullptr;
            }
            float acc[S::kHTiles][kNT][4];
#pragma unroll
            for (int m = 0; m < S::kHTiles; ++m)
#pragma unroll
                for (int j = 0; j < kNT; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[m][j][i] = 0.0f;
            for (int c = 0; c < chunks; ++c) {
                const int kb = c * per + warp;
                const bool mine = warp < min(per, KB - c * per);
                uint4 x[kNT][2];
#pragma unroll
                for (int j = 0; j < kNT; ++j)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        x[j][b] = mine && xp[j] ? __ldg(reinterpret_cast<const uint4*>(xp[j] + kb * 64 + b * 32))
                                                : make_uint4(0, 0, 0, 0);
                if (wait_full() && mine) {
                    const uint32_t u = ring + s * S::kStage + warp * S::kHUnit;
#pragma unroll
                    for (int m = 0; m < S::kHTiles; ++m)
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            uint32_t wg[4], wu[4];
                            if (kQ4) {
                                const uint32_t p = u + b * (S::kHRows * 16) + (m * 8 + g) * 16 + tq * 4;
                                const uint32_t sc = u + S::kHRows * 32 + (m * 8 + g) * 4;
                                constexpr uint32_t kUp = S::kHRows * S::kRowBytes;
                                const uint32_t qg = ld_shared_u32(p), qu = ld_shared_u32(p + kUp);
                                const uint32_t dg = ld_shared_u32(sc), du = ld_shared_u32(sc + kUp);
                                const uint32_t sg = __byte_perm(dg, 0, b ? 0x3232 : 0x1010);
                                const uint32_t su = __byte_perm(du, 0, b ? 0x3232 : 0x1010);
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    wg[i] = q4_pair(qg, i, *reinterpret_cast<const __nv_bfloat162*>(&sg));
                                    wu[i] = q4_pair(qu, i, *reinterpret_cast<const __nv_bfloat162*>(&su));
                                }
                            } else {
                                const uint32_t p = u + (m * 8 + g) * 128 + b * 64 + tq * 16;
                                const uint4 vg = ld_shared_v4(p), vu = ld_shared_v4(p + S::kHRows * 128);
                                wg[0] = vg.x, wg[1] = vg.y, wg[2] = vg.z, wg[3] = vg.w;
                                wu[0] = vu.x, wu[1] = vu.y, wu[2] = vu.z, wu[3] = vu.w;
                            }
#pragma unroll
                            for (int j = 0; j < kNT; ++j) {
                                if (j >= nt) continue;
                                mma_bf16(acc[m][j], wg[0], wu[0], wg[1], wu[1], x[j][b].x, x[j][b].y);
                                mma_bf16(acc[m][j], wg[2], wu[2], wg[3], wu[3], x[j][b].z, x[j][b].w);
                            }
                        }
                }
                release();
            }
            // the warps' partial sums, SwiGLU and the weights of the routes
            const size_t slot = sh ? static_cast<size_t>(e) : static_cast<size_t>(d.phi[e]);
            const float scale = sh ? d.sh_scale[slot] : d.scale[slot];
            const int len = sh ? Fs : F;
            __nv_bfloat16* hp = static_cast<__nv_bfloat16*>(sh ? d.h_shared : d.h);
#pragma unroll
            for (int j = 0; j < kNT; ++j) {
                if (j >= nt) continue;
                sync_consumers();  // the previous sums have been read
#pragma unroll
                for (int m = 0; m < S::kHTiles; ++m)
                    *reinterpret_cast<float4*>(&red[(warp * S::kHTiles + m) * 128 + lane * 4]) =
                        make_float4(acc[m][j][0], acc[m][j][1], acc[m][j][2], acc[m][j][3]);
                sync_consumers();
                // lane l's values 0, 1 are gate and 2, 3 up of columns 2 (l % 4), + 1
                for (int i = threadIdx.x; i < S::kHTiles * 64; i += 32 * kConsumers) {
                    const int m = i >> 6, l = (i & 63) >> 1, hi = i & 1;
                    const int f = (t.row / S::kHRows) * S::kHRows + m * 8 + (l >> 2);
                    const int c = j * 8 + (l & 3) * 2 + hi;
                    if (f < t.row || f >= t.row + t.n || c >= cnt) continue;
                    const float gate = reduced(m, l * 4 + hi), up = reduced(m, l * 4 + 2 + hi);
                    const float a = sh ? 1.0f : r.row_alpha[row0 + c];
                    const float v = a * scale * (gate / (1.0f + expf(-gate)) * up);
                    __nv_bfloat16* o = hp + static_cast<size_t>(row0 + c) * 3 * len + f;
                    const __nv_bfloat16 p0 = __float2bfloat16_rn(v);
                    const float r1 = v - __bfloat162float(p0);
                    const __nv_bfloat16 p1 = __float2bfloat16_rn(r1);
                    o[0] = p0;
                    o[len] = p1;
                    o[2 * len] = __float2bfloat16_rn(r1 - __bfloat162float(p1));
                }
            }
        }
        // every h row of the call is written: barrier over the consumers of the grid
        {
            sync_consumers();
            if (threadIdx.x == 0) {
                __threadfence();
                if (!*abort_flag && !((d.withhold & 2) && blockIdx.x == 0)) atomicAdd(d.sync, 1);
                const int target = (gen + 1) * static_cast<int>(gridDim.x);
                const uint64_t t0 = global_ns();
                int all = 1;
                while (true) {
                    int seen;
                    asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(seen) : "l"(d.sync) : "memory");
                    if (seen >= target) break;
                    if (*abort_flag || global_ns() - t0 > kDecodeWaitNs) {
                        record_error(d.err, kDevErrTimeout);
                        *abort_flag = 1;
                        all = 0;
                        break;
                    }
                }
                __threadfence();
                ok_flag = all;
            }
            sync_consumers();
            live = ok_flag != 0;
        }
        for (int o = live ? y0 : y1; o < y1;) {
            const int n = y_tile<S::kYRows>(o, y1);
            float acc[S::kYTiles][kNT][4];
#pragma unroll
            for (int m = 0; m < S::kYTiles; ++m)
#pragma unroll
                for (int j = 0; j < kNT; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[m][j][i] = 0.0f;
            for (int q0 = 0; q0 < YB; q0 += kConsumers) {
                const int q = q0 + warp;
                const bool mine = q < YB;
                const bool sh = q >= n_act * FB;
                const int len = sh ? FsB : FB, p = sh ? q - n_act * FB : q;
                const int a = mine ? p / len : 0, kb = mine ? p % len : 0;
                const uint32_t mask = !mine ? 0u
                                      : sh  ? (T == 32 ? 0xffffffffu : (1u << T) - 1u)
                                            : r.mask[r.act[a]];
                const int row0 = !mine ? 0 : sh ? a * T : r.row0[a];
                const __nv_bfloat16* hp = static_cast<const __nv_bfloat16*>(sh ? d.h_shared : d.h) + kb * 64 + tq * 8;
                if (wait_full() && mine) {
                    const uint32_t u = ring + s * S::kStage + warp * S::kYUnit;
                    uint32_t w[S::kYTiles][2][8];  // [.][column block][rows g, g + 8 alternating]
#pragma unroll
                    for (int m = 0; m < S::kYTiles; ++m)
#pragma unroll
                        for (int b = 0; b < 2; ++b)
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                const int row = m * 16 + half * 8 + g;
                                if (kQ4) {
                                    const uint32_t word = ld_shared_u32(u + b * (S::kYRows * 16) + row * 16 + tq * 4);
                                    const uint32_t sc = ld_shared_u32(u + S::kYRows * 32 + row * 4);
                                    const uint32_t s2 = half2_to_bf162(__byte_perm(sc, 0, b ? 0x3232 : 0x1010));
#pragma unroll
                                    for (int i = 0; i < 4; ++i)
                                        w[m][b][2 * i + half] =
                                            q4_pair(word, i, *reinterpret_cast<const __nv_bfloat162*>(&s2));
                                } else {
                                    const uint4 v = ld_shared_v4(u + row * 128 + b * 64 + tq * 16);
                                    w[m][b][half] = half2_to_bf162(v.x);
                                    w[m][b][2 + half] = half2_to_bf162(v.y);
                                    w[m][b][4 + half] = half2_to_bf162(v.z);
                                    w[m][b][6 + half] = half2_to_bf162(v.w);
                                }
                            }
#pragma unroll
                    for (int j = 0; j < kNT; ++j) {
                        if (((mask >> (8 * j)) & 0xffu) == 0u) continue;
                        const int t = 8 * j + g;
                        const bool has = (mask >> t) & 1u;
                        const __nv_bfloat16* hr =
                            hp + static_cast<size_t>(row0 + __popc(mask & ((1u << t) - 1u))) * 3 * (len * 64);
#pragma unroll
                        for (int part = 0; part < 3; ++part)
#pragma unroll
                            for (int b = 0; b < 2; ++b) {
                                const uint4 x = has ? __ldcg(reinterpret_cast<const uint4*>(hr + part * (len * 64) + b * 32))
                                                    : make_uint4(0, 0, 0, 0);
#pragma unroll
                                for (int m = 0; m < S::kYTiles; ++m) {
                                    mma_bf16(acc[m][j], w[m][b][0], w[m][b][1], w[m][b][2], w[m][b][3], x.x, x.y);
                                    mma_bf16(acc[m][j], w[m][b][4], w[m][b][5], w[m][b][6], w[m][b][7], x.z, x.w);
                                }
                            }
                    }
                }
                release();
            }
#pragma unroll
            for (int j = 0; j < kNT; ++j) {
                if (8 * j >= T) continue;
                sync_consumers();
#pragma unroll
                for (int m = 0; m < S::kYTiles; ++m)
                    *reinterpret_cast<float4*>(&red[(warp * S::kHTiles + m) * 128 + lane * 4]) =
                        make_float4(acc[m][j][0], acc[m][j][1], acc[m][j][2], acc[m][j][3]);
                sync_consumers();
                for (int i = threadIdx.x; i < S::kYTiles * 128; i += 32 * kConsumers) {
                    const int m = i >> 7, l = (i & 127) >> 2, v = i & 3;
                    const int row = m * 16 + (l >> 2) + (v >> 1) * 8, t = j * 8 + (l & 3) * 2 + (v & 1);
                    if (row >= n || t >= T || *abort_flag) continue;
                    const size_t at = static_cast<size_t>(t) * H + o + row;
                    d.Y[at] = (d.A ? x_at<ESTREAM_BF16>(d.A, at) : d.Y[at]) + reduced(m, i & 127);
                }
            }
            o += n;
        }
    }
    decode_leave(d.sync);
}

}  // namespace

template <bool kQ4, int kNT>
static cudaError_t launch_stream(const DecodeCall& d, int num_sms, cudaStream_t stream) {
    using S = Stream<kQ4>;
    // the ring takes what the sums and the routes leave of 227 KB (static part: 1 KB)
    const size_t fixed = sizeof(float) * S::kRed + routes_bytes(d.T * d.k, d.E);
    const int stages = static_cast<int>(std::min<size_t>(kMaxStages, (226 * 1024 - fixed) / S::kStage));
    if (stages < 2) return cudaErrorInvalidConfiguration;
    const size_t smem = static_cast<size_t>(stages) * S::kStage + fixed;
    const void* fn = reinterpret_cast<const void*>(k_layer_decode<kQ4, kNT>);
    cudaError_t rc = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (rc != cudaSuccess) return rc;
    DecodeCall call = d;
    int n = stages;
    void* args[] = {&call, &n};
    return cudaLaunchCooperativeKernel(fn, dim3(num_sms), dim3(kStreamThreads), args, smem, stream);
}

cudaError_t launch_layer_decode(const DecodeCall& d, int wdtype, int num_sms, cudaStream_t stream) {
    // up to 8 tokens the accumulators of one token tile suffice
    const bool few = d.T <= 8;
    if (wdtype == ESTREAM_BF16)
        return few ? launch_stream<false, 1>(d, num_sms, stream) : launch_stream<false, 4>(d, num_sms, stream);
    if (wdtype == ESTREAM_Q4)
        return few ? launch_stream<true, 1>(d, num_sms, stream) : launch_stream<true, 4>(d, num_sms, stream);
    const size_t smem = routes_bytes(d.T * d.k, d.E);
    DecodeCall call = d;
    void* args[] = {&call};
    return cudaLaunchCooperativeKernel(reinterpret_cast<const void*>(k_layer_decode_simple), dim3(num_sms),
                                       dim3(kSimpleThreads), args, smem, stream);
}

}  // namespace es
