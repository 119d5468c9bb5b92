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
#include <type_traits>

#include "estream_internal.h"

namespace es {
namespace {
#include "tc_ptx.cuh"
}  // namespace

#include "route_topk.cuh"

namespace {

constexpr uint64_t kDecodeWaitNs = 1000000000ull;  // 1 s: bound of a grid barrier
constexpr uint32_t kSpins = 64;  // polls between two looks at the clock, whose read takes about a microsecond
constexpr int kSimpleThreads = 512;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// mbar_wait that polls for a while before it looks at the clock: a weight copy
// is nearly always a short wait away.
__device__ __forceinline__ bool copy_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err) {
    for (uint32_t i = 0; i < kSpins; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    return mbar_wait(bar, parity, abort_flag, err);
}

// Barrier of the whole (cooperative) grid, bounded in time. sync[0] counts
// arrivals and only grows within a launch; decode_leave zeroes it for the next
// one. Its kFailed bit is the outcome of a barrier that is not met: the first CTA
// whose wait runs out, or whose own work is incomplete (the abort flag), sets it
// while the count is still short, so a barrier is met for every CTA or for none,
// also for one that arrives after others gave up. (A CTA still polling an earlier,
// met barrier may take a later one's failure for its own. It stops there, and only
// the last barrier's outcome decides what is written to Y.)
constexpr int kFailed = 1 << 30;
constexpr uint64_t kLateNs = 3000000000ull;  // test: bound of a late arrival's delay

__device__ __forceinline__ int sync_word(const int* sync) {
    int v;
    asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(sync) : "memory");
    return v;
}
// How this CTA arrives: a test lets one stay away, or come once the others gave up.
enum Arrival { kArrive = 0, kWithhold = 1, kArriveLate = 2 };

__device__ bool decode_barrier(int* sync, int generation, int* err, int* ok_flag, volatile int* abort_flag,
                               Arrival how) {
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        const int target = generation * static_cast<int>(gridDim.x);
        bool give_up = abort_flag && *abort_flag;
        if (how == kArriveLate && !give_up)
            for (const uint64_t t0 = global_ns(); !(sync_word(sync) & kFailed) && global_ns() - t0 < kLateNs;) {}
        if (how != kWithhold && !give_up) atomicAdd(sync, 1);
        uint64_t t0 = 0;
        bool ok = true;
        for (uint32_t spins = 1;; ++spins) {
            const int seen = sync_word(sync);
            if (seen & kFailed) {
                ok = false;
                break;
            }
            if (seen >= target) break;
            if (give_up) {
                // fails only while someone else arrives, at most once a CTA
                if (atomicCAS(sync, seen, seen | kFailed) == seen) record_error(err, kDevErrTimeout);
                continue;
            }
            if (spins % kSpins != 0) continue;  // the clock is slow to read
            if (t0 == 0) t0 = global_ns();
            give_up = global_ns() - t0 > kDecodeWaitNs;
        }
        __threadfence();
        *ok_flag = ok ? 1 : 0;
    }
    __syncthreads();
    return *ok_flag != 0;
}

// CTA 0's arrival at barrier `at` (0 the router's, 1 h's, 2 the sum's) as a test asks for it.
__device__ __forceinline__ Arrival arrival(const DecodeCall& d, int at) {
    return blockIdx.x == 0 ? static_cast<Arrival>(d.arrival >> (2 * at) & 3) : kArrive;
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

// Up to 8 tokens of a chosen expert, or of a shared one after them.
struct Act {
    uint32_t mask;  // bit t: token t is one of them
    int row0;       // the first one's h row (one row a token, ascending t)
    int slot;       // arena slot, or index among the shared experts
    float scale;    // 2^-s of its down weights
};

// The call's routes in shared memory, formed by every CTA for itself.
struct Routes {
    Act* act;          // [act_max] tiles of experts with a token, ascending, then of the shared ones
    Act* expert;       // [E] every expert's entry, with all its tokens
    float* row_alpha;  // [T k] weight of each h row
    int* row_tok;      // [T k] its token
    int* ids;          // [T k] expert of each route; then, a token's h rows in ascending order
    float* alpha;      // [T k] weight of each route
    uint32_t* key;     // [T E] logits as ordered keys (E <= kKeysE)
    int* counts;       // [E + 1] (E > kKeysE)
    int* n_act;
};

constexpr int kKeysE = 128;

__host__ __device__ inline int shared_tiles(int T, int n_shared) { return n_shared * ((T + 7) / 8); }
__host__ __device__ inline int act_max(int T, int k, int E, int n_shared) {
    return E + T * k / 8 + shared_tiles(T, n_shared);
}
__host__ __device__ inline size_t routes_bytes(int T, int k, int E, int n_shared) {
    const size_t R = static_cast<size_t>(T) * k;
    return (sizeof(Act) * (static_cast<size_t>(E) + act_max(T, k, E, n_shared)) +
            sizeof(int) * (4 * R + (E <= kKeysE ? static_cast<size_t>(T) * E : static_cast<size_t>(E) + 1) + 1) + 15) /
           16 * 16;
}

__device__ Routes routes_at(void* smem, int T, int k, int E, int n_shared) {
    const int R = T * k;
    Routes r;
    r.act = static_cast<Act*>(smem);
    r.expert = r.act + act_max(T, k, E, n_shared);
    r.row_alpha = reinterpret_cast<float*>(r.expert + E);
    r.row_tok = reinterpret_cast<int*>(r.row_alpha + R);
    r.ids = r.row_tok + R;
    r.alpha = reinterpret_cast<float*>(r.ids + R);
    r.n_act = reinterpret_cast<int*>(r.alpha + R);
    r.counts = r.n_act + 1;
    r.key = reinterpret_cast<uint32_t*>(r.counts);
    return r;
}

// (A NaN is the largest key, whatever its sign, and a NaN again in key_logit, so its
// token's weights are NaN. The smallest key, of -infinity, is above 0.)
__device__ __forceinline__ uint32_t logit_key(float v) {
    if (isnan(v)) return 0xffffffffu;
    const uint32_t b = __float_as_uint(__fadd_rn(v, 0.0f));  // -0 -> +0
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// What does not depend on the routing: the experts' slots and scales, fetched
// while the logits are on their way.
__device__ void prepare_routes(const Routes& r, const DecodeCall& d) {
    for (int e = threadIdx.x; e < d.E; e += blockDim.x) {
        const int slot = d.phi[e];
        r.expert[e] = {0u, 0, slot, d.scale[slot]};
        if (d.E > kKeysE) r.counts[e] = 0;
    }
    if (threadIdx.x == 0 && d.E > kKeysE) r.counts[d.E] = 0;
}

// An expert's entry as tiles of up to 8 tokens.
__device__ __forceinline__ void list_tiles(Act* act, Act a) {
    for (uint32_t left = a.mask; left; ++act) {
        uint32_t rest = left;
        for (int i = 0; i < 8; ++i) rest &= rest - 1;
        a.mask = left & ~rest;
        *act = a;
        a.row0 += 8;
        left = rest;
    }
}

// Which experts each token takes: the experts' token masks, the list of tiles of up
// to 8 tokens of the experts in use and, with T <= 32, a token's row among its expert's rows as a count of
// the mask's lower bits. A warp a token; up to kKeysE experts its keys stay in
// four registers a lane, a round being the largest key and the lowest expert
// that holds it. The weights of that form are left to route_weights, off the path
// to the first weight copy; more experts take the route build's own selection.
__device__ void build_routes(const Routes& r, const DecodeCall& d, const float* logits) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    const int T = d.T, E = d.E, k = d.k;
    __syncthreads();  // prepare_routes
    for (int t = warp; t < T; t += nw) {
        if (E <= kKeysE) {
            uint32_t key[kKeysE / 32];
#pragma unroll
            for (int j = 0; j < kKeysE / 32; ++j) {
                const int e = lane + 32 * j;
                key[j] = e < E ? logit_key(__ldcg(logits + t * E + e)) : 0u;
            }
#pragma unroll
            for (int j = 0; j < kKeysE / 32; ++j)
                if (lane + 32 * j < E) r.key[t * E + lane + 32 * j] = key[j];
            for (int i = 0; i < k; ++i) {
                uint32_t top = 0u, at = 0xffffffffu;
#pragma unroll
                for (int j = 0; j < kKeysE / 32; ++j)
                    if (key[j] > top) {
                        top = key[j];
                        at = lane + 32 * j;
                    }
                const uint32_t m = __reduce_max_sync(0xffffffffu, top);
                const uint32_t e = __reduce_min_sync(0xffffffffu, top == m ? at : 0xffffffffu);
#pragma unroll
                for (int j = 0; j < kKeysE / 32; ++j)
                    if (static_cast<uint32_t>(lane + 32 * j) == e) key[j] = 0u;
                if (lane == 0) {
                    r.ids[t * k + i] = static_cast<int>(e);
                    atomicOr(&r.expert[e].mask, 1u << t);
                }
            }
        } else {
            topk_token<kMaxPerLane>(t, logits + static_cast<size_t>(t) * E, E, k, d.renorm, nullptr, E, r.ids,
                                    r.alpha, r.counts, d.err);
            __syncwarp();
            if (lane < k && r.ids[t * k + lane] >= 0) atomicOr(&r.expert[r.ids[t * k + lane]].mask, 1u << t);
        }
    }
    __syncthreads();
    if (warp == 0) {
        int n = 0, rows = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            const uint32_t mask = e < E ? r.expert[e].mask : 0u;
            const int c = __popc(mask);
            int incl = c + (((c + 7) / 8) << 16);  // rows and tiles
#pragma unroll
            for (int s = 1; s < 32; s <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, incl, s);
                if (lane >= s) incl += o;
            }
            if (c > 0) {
                Act a = r.expert[e];
                a.row0 = rows + (incl & 0xffff) - c;
                r.expert[e].row0 = a.row0;
                list_tiles(r.act + n + (incl >> 16) - (c + 7) / 8, a);
            }
            const int all = __shfl_sync(0xffffffffu, incl, 31);
            n += all >> 16;
            rows += all & 0xffff;
        }
        if (lane == 0) *r.n_act = n;
        for (int j = lane; j < d.n_shared; j += 32)
            list_tiles(r.act + n + shared_tiles(T, j), {T == 32 ? 0xffffffffu : (1u << T) - 1u, j * T, j, d.sh_scale[j]});
    }
    __syncthreads();
    for (int i = threadIdx.x; i < T * k; i += blockDim.x) {
        const int e = r.ids[i], t = i / k;
        if (e >= 0) r.row_tok[r.expert[e].row0 + __popc(r.expert[e].mask & ((1u << t) - 1u))] = t;
    }
    __syncthreads();
}

// The routes' weights at their h rows, and each token's rows in ascending order
// in place of its experts; by one warp, lane t for token t. Up to kKeysE experts
// the softmax weights are formed here, by topk_token's operations in its order
// (denominator summed in ascending expert order, one division a weight).
__device__ void route_weights(const Routes& r, const DecodeCall& d) {
    const int t = threadIdx.x & 31, E = d.E, k = d.k;
    if (t >= d.T) return;
    float* a = r.alpha + t * k;
    int* id = r.ids + t * k;
    if (E <= kKeysE && id[0] >= 0) {
        const uint32_t* row = r.key + t * E;
        const float m = key_logit(row[id[0]]);
        float s = 0.0f;
#pragma unroll 4
        for (int e = 0; e < E; ++e) s = __fadd_rn(s, route_exp(__fsub_rn(key_logit(row[e]), m)));
        for (int j = 0; j < k; ++j)
            a[j] = id[j] < 0 ? 0.0f : __fdiv_rn(route_exp(__fsub_rn(key_logit(row[id[j]]), m)), s);
        if (d.renorm) {
            float z = 0.0f;  // summed in rank order
            for (int j = 0; j < k; ++j) z = __fadd_rn(z, a[j]);
            for (int j = 0; j < k; ++j) a[j] = __fdiv_rn(a[j], z);
        }
    }
    for (int j = 0; j < k; ++j) {
        const int e = id[j];
        const int row = e < 0 ? -1 : r.expert[e].row0 + __popc(r.expert[e].mask & ((1u << t) - 1u));
        if (e >= 0) r.row_alpha[row] = a[j];
        int x = j;  // insertion by row
        for (; x > 0 && id[x - 1] > row; --x) id[x] = id[x - 1];
        id[x] = row;
    }
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
    // neighbouring pairs on different SMs: few pairs then are few on each
    for (int p = warp * gridDim.x + blockIdx.x; p < d.T * d.E; p += gridDim.x * nw) {
        const int t = p / d.E, e = p % d.E;
        const uint4* x = reinterpret_cast<const uint4*>(X + static_cast<size_t>(t) * d.H);
        const uint4* w = reinterpret_cast<const uint4*>(W + static_cast<size_t>(e) * d.H);
        float s = 0.0f;
#pragma unroll 8
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
    const int H = d.H, F = d.F, Fs = d.F_shared, T = d.T, k = d.k, n_sh = shared_tiles(T, d.n_shared);
    const Routes r = routes_at(smem, T, k, d.E, d.n_shared);
    int gen = 0;
    bool ok = true;
    {
        prepare_routes(r, d);
        build_routes(r, d, d.logits);
        if (warp == 0) route_weights(r, d);
        __syncthreads();
        const int n_act = *r.n_act;
        const int routed = n_act * F;
        for (int u = gw; u < routed + n_sh * Fs; u += gn) {
            const bool sh = u >= routed;
            const int at = sh ? n_act + (u - routed) / Fs : u / F;
            const int f = sh ? (u - routed) % Fs : u % F;
            const Act a = r.act[at];
            const size_t slot = static_cast<size_t>(a.slot);
            const float* pg = reinterpret_cast<const float*>(sh ? d.sh_g + slot * d.S_sh : d.plane_g + slot * d.S_gu);
            const float* pu = reinterpret_cast<const float*>(sh ? d.sh_u + slot * d.S_sh : d.plane_u + slot * d.S_gu);
            int row = a.row0;
            for (uint32_t m = a.mask; m; m &= m - 1, ++row) {
                const int t = __ffs(m) - 1;
                float g = 0.0f, up = 0.0f;
                for (int c = lane; c < H; c += 32) {
                    const float x = x_at<ESTREAM_F32>(d.X, static_cast<size_t>(t) * H + c);
                    g = fmaf(pg[static_cast<size_t>(f) * H + c], x, g);
                    up = fmaf(pu[static_cast<size_t>(f) * H + c], x, up);
                }
                g = warp_sum(g);
                up = warp_sum(up);
                if (lane == 0) {
                    const float v = a.scale * (g / (1.0f + expf(-g)) * up);
                    if (sh)
                        static_cast<float*>(d.h_shared)[static_cast<size_t>(row) * Fs + f] = v;
                    else
                        static_cast<float*>(d.h)[static_cast<size_t>(row) * F + f] = r.row_alpha[row] * v;
                }
            }
        }
        ok = decode_barrier(d.sync, ++gen, d.err, &ok_flag, nullptr, arrival(d, 1));
    }
    if (ok) {
        const int n_act = *r.n_act;
        for (int o = gw; o < H; o += gn)
            for (int t = 0; t < T; ++t) {
                float y = 0.0f;
                for (int at = 0; at < n_act + n_sh; ++at) {
                    const Act a = r.act[at];
                    if (!((a.mask >> t) & 1u)) continue;
                    const bool sh = at >= n_act;
                    const size_t slot = static_cast<size_t>(a.slot);
                    const float* pd =
                        reinterpret_cast<const float*>(sh ? d.sh_d + slot * d.S_sh : d.plane_d + slot * d.S_d);
                    const int n = sh ? Fs : F;
                    const float* h = static_cast<const float*>(sh ? d.h_shared : d.h) +
                                     static_cast<size_t>(a.row0 + __popc(a.mask & ((1u << t) - 1u))) * n;
                    for (int c = lane; c < n; c += 32)
                        y = fmaf(pd[static_cast<size_t>(o) * n + c], __ldcg(h + c), y);
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
// Streaming form (bf16 and 4-bit planes): one persistent CTA of 16 warps per SM.
//
// The h rows of all chosen experts are split into one contiguous range for each
// group of four warps (to a single row; 4-bit: 4, whose scales fill 16 bytes),
// so every SM streams the same number of weight bytes. A unit is 64 (down: 128)
// reduction values of a row tile; a group's warps take a tile's units in turn, each through
// a shared-memory ring of its own that it fills with cp.async.bulk. A copy costs
// its issuing thread about 100 ns and its warp about 30 ns, so one producer warp
// with 1 KB copies would stop at 3.7 TB/s (measured); sixteen issuers reach 6.7.
// Groups of four rather than the whole CTA on a tile: the work per tile that is
// not per unit (pointers, the sum over warps and its barrier) is then paid for 8
// units a warp instead of 2 (H = 2048), and no barrier stops all warps.
// A warp's copies need the routes but not h, so they run into the down weights
// while it still waits at the grid barrier between the projections, and HBM does
// not idle there.
//
// The products are mma.sync m16n8k16 with the weights as the 16 rows and the
// tokens as the 8 columns: at 8 columns an instruction covers 512 bytes of
// weights, far above what HBM delivers, so a tcgen05 tile of at least 64 rows
// by 8 columns through tensor memory would add latency and no speed. A tile of
// h is 8 gate rows over 8 up rows, which puts gate and up of one h value in one
// lane. Within 64 values a lane takes runs of 8 (16 bytes) as its k indices, in
// weights and tokens alike, so both come as 16-byte loads without a transpose.
//
// h leaves as three bf16 parts (8 leading bits, the next 8, the next 8), which
// together hold the fp32 value; the down weights, fp16 in the arena, are bf16
// numbers times a power of two and convert to bf16 exactly. So every product of
// both projections is exact and only fp32 sums round.
//
// More than 8 tokens of an expert are several entries of 8, each with a pass over
// the expert's weights (the second finds many in L2): four column tiles in one pass
// took the same time a tile (it is bound by instructions, not bytes) and twice the
// registers, and left the groups on such experts 30 us behind the others.
//
// Down projection, up to 8 tokens (kByToken): column t is token t whatever the
// expert, so a CTA's Y rows run through all experts in ascending order in one
// accumulator, and Y needs no partial sums. (A column without the expert leaves its
// products out, which are 0 only for finite weights; 1 us of 84 at the DeepSeek
// shape, 3 of 141 at the Mixtral shape in 4 bits, in a captured graph.) With more tokens that would read
// every token's h in every CTA (T = 32, OLMoE shape: 240 MB through L2, 210 us
// of down projection against 47 us of streaming); there the groups split the
// (entry, row) pairs as they do for h, leave a row of Y per route, and sum a
// token's routes in ascending expert order after a second grid barrier.
//
// Measured, L2 cold, of the time that the chosen experts' bytes take at 6.7 TB/s:
//   OLMoE shape (2048 x 1024, 8 of 64), 1 token, router included     36 us of 15
//   DeepSeek shape (2048 x 1408, 6 of 64 and 2), 4 tokens            74-83 us of 59
//   Mixtral shape (4096 x 14336, 2 of 8) in 4 bits, 2 tokens         115-127 us of 52
//   OLMoE shape, 32 tokens                                           161-172 us of 119
// At one token, latency: 8 us until the routes are known in every CTA and the first
// weights are there, and 7 us of down projection after the grid barrier, though its
// weights wait in shared memory by then (every SM reads the same h rows out of L2).
// In 4 bits, issue slots: 26 instructions for 8 weights, of which 9 decode them.
// A call repeats bit for bit. A token's row may differ in its last bits between
// calls whose other tokens choose other experts: which warp sums which unit depends
// on all experts in use.
// ---------------------------------------------------------------------------

constexpr int kWarps = 16;
constexpr int kGroup = 4;  // warps that share a tile
constexpr int kGroups = kWarps / kGroup;
constexpr int kStreamThreads = 32 * kWarps;
constexpr int kMaxStages = 6;

// (4-bit rows are short, so a tile takes more of them)
template <bool kQ4>
struct Stream {
    static constexpr int kHRows = kQ4 ? 48 : 16;  // h rows of a gate/up tile
    static constexpr int kYRows = kQ4 ? 32 : 16;  // Y rows of a down tile
    static constexpr int kStep = kQ4 ? 4 : 1;      // granularity of a range
    static constexpr int kHTiles = kHRows / 8;     // m16 tiles (8 gate + 8 up rows)
    static constexpr int kYTiles = kYRows / 16;
    // one plane's rows x 64 weights. 4-bit: two column blocks of 16 bytes a row,
    // then 4 bytes of scales a row.
    static constexpr int kRowBytes = kQ4 ? 36 : 128;
    static constexpr int kHPart = kHRows * kRowBytes;  // a unit of h: gate, up
    static constexpr int kYPart = kYRows * kRowBytes;  // a unit of Y: two k-blocks
    static constexpr int kUnit = 2 * (kHPart > kYPart ? kHPart : kYPart);
    // the warps' partial sums of a tile, twice: a tile's are written while the last one's are read
    // (two m16 tiles at a time)
    static constexpr int kTiles = 2;
    static constexpr int kRedTile = kWarps * kTiles * 128;  // floats
    static constexpr int kRed = 2 * kRedTile;
};

__device__ __forceinline__ void bulk_row_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <typename T>
__device__ __forceinline__ T as(const uint8_t* p) {
    return *reinterpret_cast<const T*>(p);
}
// Two fp16 weights of the down plane as bf16 (exact: see above).
__device__ __forceinline__ uint32_t half2_to_bf162(uint32_t w) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t*>(&b);
}
// Codes 2 i (low half) and 2 i + 1 (high half) of a 4-bit word as bf16 (q - 8) / 64.
// A half word's low eight bits alone are bf16 numbers below 2^-125, where the format
// is linear: a code in bits 0-3 is q 2^-133, one in bits 4-7 q 2^-129. One
// multiply-add, exact, takes either to its place, so only two of the four pairs of
// a word share a shift. (A code set into the mantissa of 128 needs a shift each.)
constexpr float kQ4Unit = 64.0f;  // what the sums of such products are short of
__device__ __forceinline__ uint32_t q4_pair(uint32_t word, int i) {
    const uint32_t u = (i < 2 ? word : word >> 8) & (i & 1 ? 0x00f000f0u : 0x000f000fu);
    const uint32_t to = i & 1 ? 0x7d007d00u : 0x7f007f00u;  // 2^123, 2^127
    const __nv_bfloat162 v = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&u), *reinterpret_cast<const __nv_bfloat162*>(&to),
                                     __floats2bfloat162_rn(-0.125f, -0.125f));
    return *reinterpret_cast<const uint32_t*>(&v);
}
// The scales of a row's two column blocks (gate and up: bf16; down: fp16).
__device__ __forceinline__ float2 q4_scales(uint32_t bits, bool half) {
    if (half) return __half22float2(*reinterpret_cast<const __half2*>(&bits));
    return make_float2(__uint_as_float(bits << 16), __uint_as_float(bits & 0xffff0000u));
}

// The tiles of a range of rows of the chosen experts (len rows each, `routed`
// in all), then of the shared ones (len_sh each): up to kRows rows of one expert.
template <int kRows>
struct Walk {
    int at;         // index among the chosen experts, then the shared ones
    int row, n;     // the tile's rows [row, row + n) of that expert
    int left;       // rows of the range from the tile's first on
    int len, len_sh, n_act;
    __device__ __forceinline__ void start(int pos, int end, int routed, int n_act_, int len_, int len_sh_) {
        len = len_;
        len_sh = len_sh_;
        n_act = n_act_;
        left = end - pos;
        const bool sh = pos >= routed;
        const int p = sh ? pos - routed : pos;
        at = left > 0 ? p / (sh ? len_sh : len) : 0;
        row = p - at * (sh ? len_sh : len);
        if (sh) at += n_act;
        size();
    }
    __device__ __forceinline__ bool shared() const { return at >= n_act; }
    __device__ __forceinline__ void size() { n = min(min((shared() ? len_sh : len) - row, left), kRows); }
    __device__ __forceinline__ void next() {
        left -= n;
        row += n;
        if (row == (shared() ? len_sh : len)) {
            row = 0;
            ++at;
        }
        size();
    }
};
// First row of part `part` of `parts` of a range of `total` rows.
__device__ __forceinline__ int share(int total, int step, int part, int parts) {
    const long long units = total / step;
    return static_cast<int>(units * part / parts) * step;
}

// kByToken (T <= 8): the down projection's columns are the call's tokens.
template <bool kQ4, bool kByToken>
__global__ void __launch_bounds__(kStreamThreads, 1) k_layer_decode(const DecodeCall d, int stages) {
    using S = Stream<kQ4>;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[kWarps * kMaxStages + 1];  // the last: the routes' weights are there
    __shared__ int ok_flag;
    __shared__ int abort_word;
    volatile int* abort_flag = &abort_word;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int H = d.H, F = d.F, Fs = d.F_shared, T = d.T, k = d.k, n_sh = shared_tiles(T, d.n_shared);
    const int KB = H / 64, FB = F / 64, FsB = Fs / 64;
    const uint8_t* ring_p = smem_raw + warp * stages * S::kUnit;
    const uint32_t ring = smem_addr(ring_p);
    float* red = reinterpret_cast<float*>(smem_raw + static_cast<size_t>(kWarps) * stages * S::kUnit);
    const Routes r = routes_at(red + S::kRed, T, k, d.E, d.n_shared);
    const uint32_t bar0 = smem_addr(&bars[warp * kMaxStages]);
    const uint32_t weights_bar = smem_addr(&bars[kWarps * kMaxStages]);
    if (threadIdx.x == 0) {
        abort_word = 0;
        mbar_init(weights_bar, 1);
    }
    if (lane == 0) {
        for (int s = 0; s < stages; ++s) mbar_init(bar0 + 8 * s, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    prepare_routes(r, d);
    int gen = 0;
    bool ok = true;
    if (d.W_r) {
        router_rows(d);
        ok = decode_barrier(d.sync, ++gen, d.err, &ok_flag, nullptr, arrival(d, 0));
    }
    if (!ok) {
        decode_leave(d.sync);
        return;
    }
    build_routes(r, d, d.W_r ? d.logits_out : d.logits);
    const int n_act = *r.n_act;
    const int routed_h = n_act * F, total_h = routed_h + n_sh * Fs;
    const int wg = warp % kGroup, group = blockIdx.x * kGroups + warp / kGroup;
    const int groups = gridDim.x * kGroups;
    const int h0 = share(total_h, S::kStep, group, groups), h1 = share(total_h, S::kStep, group + 1, groups);
    // Y rows: of Y itself, a range a CTA, or of every (tile, Y) pair, a range a group
    const int routed_y = kByToken ? 0 : n_act * H;
    const int total_y = kByToken ? H : routed_y + n_sh * H;
    const int y_part = kByToken ? blockIdx.x : group, y_parts = kByToken ? gridDim.x : groups;
    const int y0 = share(total_y, S::kStep, y_part, y_parts), y1 = share(total_y, S::kStep, y_part + 1, y_parts);
    constexpr int kYWarps = kByToken ? kWarps : kGroup;  // warps that share a Y tile
    const int wy = kByToken ? warp : wg;
    const int YB = n_act * FB + n_sh * FsB;  // k-blocks of a Y row over all experts
    // Tiles of Y: one expert's rows, or (kByToken, at = 0) Y's own rows.
    auto start_y = [&](Walk<S::kYRows>& t) {
        if (kByToken) {
            t.at = 0;
            t.row = y0;
            t.left = y1 - y0;
            t.n = min(S::kYRows, t.left);
        } else {
            t.start(y0, y1, routed_y, n_act, H, H);
        }
    };
    auto next_y = [&](Walk<S::kYRows>& t) {
        if (kByToken) {
            t.row += t.n;
            t.left -= t.n;
            t.n = min(S::kYRows, t.left);
        } else {
            t.next();
        }
    };

    // ---- the warp's copies, `stages` units ahead of its products ----
    // Kept small: a unit's bookkeeping is the larger part of its instructions.
    constexpr int kParts = kQ4 ? 3 : 1;  // copies of a plane's rows: codes, codes, scales
    Walk<S::kHRows> ih;
    Walk<S::kYRows> iy;
    ih.start(h0, h1, routed_h, n_act, F, Fs);
    start_y(iy);
    int i_stage = 0, issued = 0;
    int i_kb = 0, i_end = 0;   // next unit of the tile, units of the tile
    int i_a = 0, i_akb = 0;    // kByToken: its expert and k-block there
    bool i_down = false, i_fresh = true;  // in the down projection; the tile is yet to be entered
    const char* i_src = nullptr;          // this lane's copy of that unit
    uint32_t i_off = 0, i_bytes = 0, i_tx = 0;
    size_t i_step = 0;
    // this lane's copy of rows [row, row + n) of a box whose rows go to smem rows from `to` on
    auto lane_rows = [&](int part, int box_rows, int smem_rows, int row, int to, int n, size_t& src_off) {
        if (!kQ4) {
            src_off = row * 128;
            i_off = to * 128;
            i_bytes = n * 128;
        } else if (part < 2) {
            src_off = part * (box_rows * 16) + row * 16;
            i_off = part * (smem_rows * 16) + to * 16;
            i_bytes = n * 16;
        } else {
            src_off = box_rows * 32 + row * 4;
            i_off = smem_rows * 32 + to * 4;
            i_bytes = n * 4;
        }
    };
    auto down_src = [&](int at) {
        const size_t slot = static_cast<size_t>(r.act[at].slot);
        return at >= n_act ? d.sh_d + slot * d.S_sh : d.plane_d + slot * d.S_d;
    };
    size_t y_off = 0;  // kByToken: this lane's rows inside a k-block's box, and the box of its Y rows
    int y_box = 0;
    auto issue_next = [&]() {
        while (i_kb >= i_end) {
            if (!i_fresh) {
                if (i_down) next_y(iy); else ih.next();
            }
            i_fresh = false;
            if (!i_down && ih.left <= 0) {
                i_down = true;
                i_fresh = true;
                i_kb = i_end = 0;
                continue;
            }
            if (i_down && iy.left <= 0) {
                i_kb = i_end = 0;
                i_fresh = true;
                return;
            }
            size_t off = 0;
            // a lane a copy: the rows in the first box, then (over) those in the next one
            if (!i_down) {
                i_kb = wg;
                const int here = min(ih.n, 128 - ih.row % 128);
                const bool sh = ih.shared(), up = (lane / kParts) & 1, over = lane >= 2 * kParts;
                const size_t slot = static_cast<size_t>(r.act[ih.at].slot);
                lane_rows(lane % kParts, 128, S::kHRows, over ? 0 : ih.row % 128, over ? here : 0,
                          over ? ih.n - here : here, off);
                if (up) i_off += S::kHPart;
                if (lane >= 4 * kParts) i_bytes = 0;
                i_tx = 2u * ih.n * S::kRowBytes;
                i_step = static_cast<size_t>(kGroup) * (128 * S::kRowBytes);
                i_src = (sh ? (up ? d.sh_u : d.sh_g) + slot * d.S_sh : (up ? d.plane_u : d.plane_g) + slot * d.S_gu) +
                        (static_cast<size_t>(ih.row / 128 + over) * KB + i_kb) * (128 * S::kRowBytes) + off;
                i_end = KB;
            } else {
                i_kb = wy;
                const int here = min(iy.n, 256 - iy.row % 256);
                const bool second = (lane / kParts) & 1, over = lane >= 2 * kParts;
                lane_rows(lane % kParts, 256, S::kYRows, over ? 0 : iy.row % 256, over ? here : 0,
                          over ? iy.n - here : here, off);
                if (second) {
                    i_off += S::kYPart;
                    off += 256 * S::kRowBytes;
                }
                if (lane >= 4 * kParts) i_bytes = 0;
                i_tx = 2u * iy.n * S::kRowBytes;
                i_step = static_cast<size_t>(2 * kYWarps) * (256 * S::kRowBytes);
                y_box = iy.row / 256 + over;
                if (kByToken) {
                    y_off = off;
                    i_a = 0;
                    i_akb = 2 * wy;
                    i_end = YB / 2;
                } else {
                    const int len = iy.shared() ? FsB : FB;
                    i_end = len / 2;
                    i_src = down_src(iy.at) + (static_cast<size_t>(y_box) * len + 2 * i_kb) * (256 * S::kRowBytes) + off;
                }
            }
        }
        if (kByToken && i_down) {
            for (int len = i_a >= n_act ? FsB : FB; i_akb >= len; len = i_a >= n_act ? FsB : FB) {
                i_akb -= len;
                ++i_a;
            }
            i_src = down_src(i_a) +
                    (static_cast<size_t>(y_box) * (i_a >= n_act ? FsB : FB) + i_akb) * (256 * S::kRowBytes) + y_off;
            i_akb += 2 * kYWarps;
        }
        const uint32_t bar = bar0 + 8 * i_stage;
        if (lane == 0) mbar_arrive_expect_tx(bar, i_tx);
        __syncwarp();
        if (i_bytes) bulk_row_load(ring + i_stage * S::kUnit + i_off, i_src, i_bytes, bar);
        i_src += i_step;
        i_kb += i_down ? kYWarps : kGroup;
        ++issued;
        if (++i_stage == stages) i_stage = 0;
    };
    for (int s = 0; s < stages; ++s) issue_next();
    if (warp == kWarps - 1) {
        route_weights(r, d);
        __syncwarp();
        if (lane == 0) mbar_arrive(weights_bar);
    }

    // ---- products ----
    const int g = lane >> 2, tq = lane & 3;
    int stage = 0, used = 0;
    uint32_t ph = 0;
    bool live = true;
    // A wait that gives up raises the abort flag, with which every other wait
    // ends at once; the warp then passes its remaining units without work, so
    // that all warps meet at every barrier.
    auto wait_full = [&]() {
        live = __all_sync(0xffffffffu, live && used < issued && copy_wait(bar0 + 8 * stage, ph, abort_flag, d.err));
        return live;
    };
    auto release = [&]() {
        __syncwarp();
        if (!live) return;
        ++used;
        if (++stage == stages) {
            stage = 0;
            ph ^= 1u;
        }
        issue_next();
    };
    // The partial tiles of the warps that share one meet in one of two buffers in
    // turn: a warp can write to a buffer again only after the barrier of the other
    // one, which every reader of this one has passed by then.
    int turn = 0;
    auto gather = [&](const float (&acc)[4], int m) {
        *reinterpret_cast<float4*>(&red[turn * S::kRedTile + (warp * S::kTiles + m) * 128 + lane * 4]) =
            make_float4(acc[0], acc[1], acc[2], acc[3]);
    };
    // sum over `n` warps from `w0` on, value i of m16 tile m
    auto reduced = [&](int w0, auto n, int m, int i) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < decltype(n)::value; ++w) v += red[turn * S::kRedTile + ((w0 + w) * S::kTiles + m) * 128 + i];
        return v;
    };
    auto sync_group = [&] { asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / kGroup), "n"(32 * kGroup) : "memory"); };
    const int tid_g = threadIdx.x % (32 * kGroup), w_g = warp / kGroup * kGroup;
    Walk<S::kHRows> t;
    t.start(h0, h1, routed_h, n_act, F, Fs);
    for (; t.left > 0; t.next()) {
        const bool sh = t.shared();
        const Act act = r.act[t.at];
        const int cnt = __popc(act.mask), row0 = act.row0;
        // the lane's token; columns past the last one repeat it, and what they sum is
        // not read
        const int col = min(g, cnt - 1);
        const uint4* xp = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(d.X) +
                                                         static_cast<size_t>(sh ? __ffs(act.mask) - 1 + col : r.row_tok[row0 + col]) * H) +
                          tq + wg * 8;
        float acc[S::kHTiles][4] = {};
        uint4 x[2], more[2];
        x[0] = __ldg(xp);
        x[1] = __ldg(xp + 4);
        for (int kb = wg, at = 0; kb < KB; kb += kGroup, at += kGroup * 8) {
            if (wait_full()) {
                const uint8_t* u = ring_p + stage * S::kUnit;
                // the next unit's X is fetched ahead
                const uint4* np = xp + (kb + kGroup < KB ? at + kGroup * 8 : at);
                more[0] = __ldg(np);
                more[1] = __ldg(np + 4);
#pragma unroll
                for (int m = 0; m < S::kHTiles; ++m) {
                    if (m > 0 && m * 8 >= t.n) continue;
                    // a unit's sums join the running ones by rounded additions: the tensor
                    // cores truncate, which over a long chain would bias the sum
                    float part[2][4] = {};  // a chain for each column block
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        uint32_t wg[4], wu[4];
                        if (kQ4) {
                            const uint8_t* p = u + b * (S::kHRows * 16) + (m * 8 + g) * 16 + tq * 4;
                            const uint32_t qg = as<uint32_t>(p), qu = as<uint32_t>(p + S::kHPart);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                wg[i] = q4_pair(qg, i);
                                wu[i] = q4_pair(qu, i);
                            }
                        } else {
                            const uint8_t* p = u + (m * 8 + g) * 128 + b * 64 + tq * 16;
                            const uint4 vg = as<uint4>(p), vu = as<uint4>(p + S::kHPart);
                            wg[0] = vg.x, wg[1] = vg.y, wg[2] = vg.z, wg[3] = vg.w;
                            wu[0] = vu.x, wu[1] = vu.y, wu[2] = vu.z, wu[3] = vu.w;
                        }
                        mma_bf16(part[b], wg[0], wu[0], wg[1], wu[1], x[b].x, x[b].y);
                        mma_bf16(part[b], wg[2], wu[2], wg[3], wu[3], x[b].z, x[b].w);
                    }
                    if (kQ4) {
                        const uint8_t* p = u + S::kHRows * 32 + (m * 8 + g) * 4;
                        const float2 sg = q4_scales(as<uint32_t>(p), false);
                        const float2 su = q4_scales(as<uint32_t>(p + S::kHPart), false);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            acc[m][i] = fmaf(part[0][i], i < 2 ? sg.x : su.x,
                                             fmaf(part[1][i], i < 2 ? sg.y : su.y, acc[m][i]));
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[m][i] += part[0][i] + part[1][i];
                    }
                }
                x[0] = more[0];
                x[1] = more[1];
            }
            release();
        }
        // the warps' partial sums, SwiGLU and the weights of the routes
        const int len = sh ? Fs : F;
        __nv_bfloat16* hp = static_cast<__nv_bfloat16*>(sh ? d.h_shared : d.h);
        copy_wait(weights_bar, 0, abort_flag, d.err);
#pragma unroll
        for (int m0 = 0; m0 < S::kHTiles; m0 += S::kTiles) {
            if (m0 > 0 && m0 * 8 >= t.n) continue;
#pragma unroll
            for (int m = 0; m < S::kTiles; ++m) gather(acc[m0 + m], m);
            sync_group();
            // lane l's values 0, 1 are gate and 2, 3 up of columns 2 (l % 4), + 1
            for (int i = tid_g; i < S::kTiles * 64; i += 32 * kGroup) {
                const int m = i >> 6, l = (i & 63) >> 1, hi = i & 1;
                const int row = (m0 + m) * 8 + (l >> 2), f = t.row + row, c = (l & 3) * 2 + hi;
                if (row >= t.n || c >= cnt) continue;
                const std::integral_constant<int, kGroup> n{};
                constexpr float unit = kQ4 ? kQ4Unit : 1.0f;
                const float gate = unit * reduced(w_g, n, m, l * 4 + hi), up = unit * reduced(w_g, n, m, l * 4 + 2 + hi);
                const float a = sh ? 1.0f : r.row_alpha[row0 + c];
                const float v = a * act.scale * (gate / (1.0f + expf(-gate)) * up);
                __nv_bfloat16* o = hp + static_cast<size_t>(row0 + c) * 3 * len + f;
                // (just below 2^128 rounding up would leave bf16's range; an infinity has no rest)
                const __nv_bfloat16 p0 = fabsf(v) < 0x1.ffp127f ? __float2bfloat16_rn(v) : __float2bfloat16_rz(v);
                const float r1 = isinf(v) ? 0.0f : v - __bfloat162float(p0);
                const __nv_bfloat16 p1 = __float2bfloat16_rn(r1);
                o[0] = p0;
                o[len] = p1;
                o[2 * len] = __float2bfloat16_rn(r1 - __bfloat162float(p1));
            }
            turn ^= 1;
        }
    }
    // every h row of the call is written
    turn = 0;
    const bool met = decode_barrier(d.sync, ++gen, d.err, &ok_flag, abort_flag, arrival(d, 1));
    live = live && met;
    Walk<S::kYRows> ty;
    start_y(ty);
    // (met is the CTA's, live the warp's own: every warp passes every barrier below)
    for (; met && ty.left > 0; next_y(ty)) {
        const bool sh_t = !kByToken && ty.shared();
        const int cnt = kByToken ? T : __popc(r.act[ty.at].mask);
        const int row_t = kByToken ? 0 : r.act[ty.at].row0;
        const int units = (kByToken ? YB : sh_t ? FsB : FB) / 2;
        float acc[S::kYTiles][4] = {};
        // Where the lane finds the h values of unit q for its column: null for a token
        // without the expert (kByToken); columns past the last token repeat it and are
        // not read. l_len: 16-byte words of an h part.
        int l_a = 0, l_kb = 2 * wy;  // kByToken: expert and k-block of the next unit
        uint32_t l_mask = 0;         // kByToken: tokens of the unit whose h values were fetched last
        size_t l_len = (sh_t ? Fs : F) / 8;
        auto h_at = [&](int q) -> const uint4* {
            if (!kByToken)
                return static_cast<const uint4*>(sh_t ? d.h_shared : d.h) +
                       static_cast<size_t>(row_t + min(g, cnt - 1)) * 3 * l_len + q * 16 + tq;
            if (q >= units) return nullptr;
            for (int n = l_a >= n_act ? FsB : FB; l_kb >= n; n = l_a >= n_act ? FsB : FB) {
                l_kb -= n;
                ++l_a;
            }
            const Act act = r.act[l_a];
            const bool sh = l_a >= n_act;
            l_mask = act.mask;
            l_len = (sh ? Fs : F) / 8;
            const uint4* p = static_cast<const uint4*>(sh ? d.h_shared : d.h) +
                             static_cast<size_t>(act.row0 + __popc(act.mask & ((1u << g) - 1u))) * 3 * l_len + l_kb * 8 + tq;
            l_kb += 2 * kYWarps;
            return (act.mask >> g) & 1u ? p : nullptr;
        };
        auto load_h = [&](const uint4* p, size_t len, uint4 (&x)[3][2]) {
#pragma unroll
            for (int q3 = 0; q3 < 3; ++q3)
#pragma unroll
                for (int b = 0; b < 2; ++b) x[q3][b] = p ? __ldcg(p + q3 * len + b * 4) : make_uint4(0, 0, 0, 0);
        };
        uint4 xa[3][2], xb[3][2];  // h values of a unit's first and second k-block, loaded one ahead
        const uint4* hp = wy < units ? h_at(wy) : nullptr;
        load_h(hp, l_len, xa);
        for (int q = wy; q < units; q += kYWarps) {
            const bool full = wait_full();
            // A column without the expert is left out of the sum: 0 times an infinite or NaN
            // weight is not 0. The lane's sums are of columns 2 tq and 2 tq + 1.
            const uint32_t in = kByToken ? l_mask >> (2 * tq) : 3u;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint4 (&x)[3][2] = half ? xb : xa;
                if (half == 0) {
                    load_h(hp ? hp + 8 : nullptr, l_len, xb);
                } else {
                    hp = q + kYWarps < units ? h_at(q + kYWarps) : nullptr;
                    load_h(hp, l_len, xa);
                }
                if (!full) continue;
                const uint8_t* u = ring_p + stage * S::kUnit + half * S::kYPart;
                uint32_t w[S::kYTiles][2][8];  // [.][column block][rows g, g + 8 alternating]
#pragma unroll
                for (int m = 0; m < S::kYTiles; ++m)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int hi = 0; hi < 2; ++hi) {
                            const int row = m * 16 + hi * 8 + g;
                            if (kQ4) {
                                const uint32_t word = as<uint32_t>(u + b * (S::kYRows * 16) + row * 16 + tq * 4);
#pragma unroll
                                for (int i = 0; i < 4; ++i) w[m][b][2 * i + hi] = q4_pair(word, i);
                            } else {
                                const uint4 v = as<uint4>(u + row * 128 + b * 64 + tq * 16);
                                w[m][b][hi] = half2_to_bf162(v.x);
                                w[m][b][2 + hi] = half2_to_bf162(v.y);
                                w[m][b][4 + hi] = half2_to_bf162(v.z);
                                w[m][b][6 + hi] = half2_to_bf162(v.w);
                            }
                        }
                float part[2][S::kYTiles][4] = {};  // a chain for each column block
#pragma unroll
                for (int q3 = 0; q3 < 3; ++q3)
#pragma unroll
                    for (int m = 0; m < S::kYTiles; ++m)
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            mma_bf16(part[b][m], w[m][b][0], w[m][b][1], w[m][b][2], w[m][b][3], x[q3][b].x, x[q3][b].y);
                            mma_bf16(part[b][m], w[m][b][4], w[m][b][5], w[m][b][6], w[m][b][7], x[q3][b].z, x[q3][b].w);
                        }
#pragma unroll
                for (int m = 0; m < S::kYTiles; ++m) {
                    if (kQ4) {
                        const uint8_t* p = u + S::kYRows * 32 + (m * 16 + g) * 4;
                        const float2 lo = q4_scales(as<uint32_t>(p), true), hi = q4_scales(as<uint32_t>(p + 32), true);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (in >> (i & 1) & 1u)
                                acc[m][i] = fmaf(part[0][m][i], i < 2 ? lo.x : hi.x,
                                                 fmaf(part[1][m][i], i < 2 ? lo.y : hi.y, acc[m][i]));
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (in >> (i & 1) & 1u) acc[m][i] += part[0][m][i] + part[1][m][i];
                    }
                }
            }
            release();
        }
#pragma unroll
        for (int m = 0; m < S::kYTiles; ++m) gather(acc[m], m);
        if (kByToken)
            __syncthreads();
        else
            sync_group();
        for (int i = kByToken ? threadIdx.x : tid_g; i < S::kYTiles * 128; i += 32 * kYWarps) {
            const int m = i >> 7, l = (i & 127) >> 2, v = i & 3;
            const int row = m * 16 + (l >> 2) + (v >> 1) * 8, c = (l & 3) * 2 + (v & 1);
            if (row >= ty.n || c >= cnt || *abort_flag) continue;
            const float y = (kQ4 ? kQ4Unit : 1.0f) *
                            reduced(kByToken ? 0 : w_g, std::integral_constant<int, kYWarps>{}, m, i & 127);
            if (kByToken) {
                const size_t at = static_cast<size_t>(c) * H + ty.row + row;
                d.Y[at] = (d.A ? x_at<ESTREAM_BF16>(d.A, at) : d.Y[at]) + y;
            } else {
                (sh_t ? d.y_shared : d.y_rows)[static_cast<size_t>(row_t + c) * H + ty.row + row] = y;
            }
        }
        turn ^= 1;
    }
    if (!kByToken) {
        const bool summed = met && decode_barrier(d.sync, ++gen, d.err, &ok_flag, abort_flag, arrival(d, 2));
        // Y[t] = A[t] (or Y[t]) + the token's routes in ascending expert order + the shared experts
        const int n4 = T * (H / 4);
        for (int i = blockIdx.x * kStreamThreads + threadIdx.x; summed && i < n4; i += gridDim.x * kStreamThreads) {
            const int t = i / (H / 4), c = (i - t * (H / 4)) * 4;
            float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            auto add = [&](const float* rows, size_t row) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(rows + row * H + c));
                y.x += v.x, y.y += v.y, y.z += v.z, y.w += v.w;
            };
            for (int j = 0; j < k; ++j) {
                const int row = r.ids[t * k + j];
                if (row >= 0) add(d.y_rows, row);
            }
            for (int e = 0; e < d.n_shared; ++e) add(d.y_shared, static_cast<size_t>(e) * T + t);
            const size_t at = static_cast<size_t>(t) * H + c;
            float4* out = reinterpret_cast<float4*>(d.Y + at);
            float4 a;
            if (d.A) {
                const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(d.A) + at);
                a = make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                                __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
            } else {
                a = *out;
            }
            *out = make_float4(a.x + y.x, a.y + y.y, a.z + y.z, a.w + y.w);
        }
    }
    // after an abort the copies still in flight must land before the CTA ends
    for (; used < issued; ++used) {
        mbar_wait_drain(bar0 + 8 * stage, ph);
        if (++stage == stages) {
            stage = 0;
            ph ^= 1u;
        }
    }
    decode_leave(d.sync);
}

}  // namespace

template <bool kQ4, bool kByToken>
static cudaError_t launch_stream(const DecodeCall& d, int num_sms, cudaStream_t stream) {
    using S = Stream<kQ4>;
    // the ring takes what the sums and the routes leave of 227 KB (static part: 1 KB)
    const size_t fixed = sizeof(float) * S::kRed + routes_bytes(d.T, d.k, d.E, d.n_shared);
    const int stages = static_cast<int>(std::min<size_t>(kMaxStages, (226 * 1024 - fixed) / (kWarps * S::kUnit)));
    if (stages < 2) return cudaErrorInvalidConfiguration;
    const size_t smem = static_cast<size_t>(stages) * kWarps * S::kUnit + fixed;
    const void* fn = reinterpret_cast<const void*>(k_layer_decode<kQ4, kByToken>);
    cudaError_t rc = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (rc != cudaSuccess) return rc;
    DecodeCall call = d;
    int n = stages;
    void* args[] = {&call, &n};
    return cudaLaunchCooperativeKernel(fn, dim3(num_sms), dim3(kStreamThreads), args, smem, stream);
}

cudaError_t launch_layer_decode(const DecodeCall& d, int wdtype, int num_sms, cudaStream_t stream) {
    // up to 8 tokens fill the 8 columns of a product
    const bool few = d.T <= 8;
    if (wdtype == ESTREAM_BF16)
        return few ? launch_stream<false, true>(d, num_sms, stream) : launch_stream<false, false>(d, num_sms, stream);
    if (wdtype == ESTREAM_Q4)
        return few ? launch_stream<true, true>(d, num_sms, stream) : launch_stream<true, false>(d, num_sms, stream);
    const size_t smem = routes_bytes(d.T, d.k, d.E, d.n_shared);
    const void* fn = reinterpret_cast<const void*>(k_layer_decode_simple);
    if (smem > 47 * 1024) {
        const cudaError_t rc =
            cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (rc != cudaSuccess) return rc;
    }
    DecodeCall call = d;
    void* args[] = {&call};
    return cudaLaunchCooperativeKernel(fn, dim3(num_sms), dim3(kSimpleThreads), args, smem, stream);
}

}  // namespace es
