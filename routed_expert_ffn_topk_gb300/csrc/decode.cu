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

// Weight (row, c) of one expert's [rows][cols] plane as the arena stores it:
// fp32 row-major; bf16 / fp16 tile-major boxes of tile_rows x 64; 4-bit boxes
// (see estream_pack_experts).
template <int kType, bool kDown>
__device__ __forceinline__ float plane_weight(const char* p, int row, int c, int cols) {
    constexpr int tr = kDown ? 256 : 128;
    if (kType == ESTREAM_F32) return reinterpret_cast<const float*>(p)[static_cast<size_t>(row) * cols + c];
    const size_t box = static_cast<size_t>(row / tr) * (cols / 64) + c / 64;
    const int r = row % tr, kk = c % 64;
    if (kType == ESTREAM_BF16) {
        const size_t at = (box * tr + r) * 64 + kk;
        return kDown ? __half2float(reinterpret_cast<const __half*>(p)[at])
                     : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[at]);
    }
    const char* b = p + box * (tr * 36);
    const int j = kk / 32, in = kk % 32;
    const uint32_t word = *reinterpret_cast<const uint32_t*>(b + j * tr * 16 + r * 16 + 4 * (in / 8));
    const int q = (word >> (16 * (in & 1) + 4 * ((in % 8) / 2))) & 15;
    const uint16_t bits = *reinterpret_cast<const uint16_t*>(b + tr * 32 + (r * 2 + j) * 2);
    const float d = kDown ? __half2float(__ushort_as_half(bits))
                          : __uint_as_float(static_cast<uint32_t>(bits) << 16);
    return static_cast<float>(q - 8) * d;
}

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
    int* n_act;
};

__host__ __device__ inline size_t routes_bytes(int R, int E) {
    return sizeof(int) * (2 * static_cast<size_t>(R) + 4 * static_cast<size_t>(E) + 2);
}

__device__ Routes routes_at(void* smem, int R, int E) {
    Routes r;
    r.ids = static_cast<int*>(smem);
    r.alpha = reinterpret_cast<float*>(r.ids + R);
    r.counts = r.ids + 2 * R;
    r.mask = reinterpret_cast<uint32_t*>(r.counts + E + 1);
    r.act = reinterpret_cast<int*>(r.mask + E);
    r.row0 = r.act + E;
    r.n_act = r.row0 + E;
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
}

// alpha of token t's route to expert e.
__device__ __forceinline__ float route_alpha(const Routes& r, int t, int e, int k) {
    float a = 0.0f;
    for (int j = 0; j < k; ++j)
        if (r.ids[t * k + j] == e) a = r.alpha[t * k + j];
    return a;
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
        float s = 0.0f;
        for (int c = lane; c < d.H; c += 32)
            s = fmaf(__bfloat162float(X[static_cast<size_t>(t) * d.H + c]),
                     __bfloat162float(W[static_cast<size_t>(e) * d.H + c]), s);
        s = warp_sum(s);
        if (lane == 0) d.logits_out[p] = s;
    }
}

// Plain form: a warp per h row, then a warp per Y column, every product an
// fp32 multiply-add on the CUDA cores.
template <int kType>
__global__ void __launch_bounds__(kSimpleThreads) k_layer_decode_simple(const DecodeCall d) {
    extern __shared__ int smem[];
    __shared__ int ok_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    const int gw = blockIdx.x * nw + warp, gn = gridDim.x * nw;
    const int H = d.H, F = d.F, Fs = d.F_shared, T = d.T, k = d.k;
    const Routes r = routes_at(smem, T * k, d.E);
    int gen = 0;
    bool ok = true;
    if (d.W_r) {
        router_rows(d);
        ok = decode_barrier(d.sync, ++gen, d.err, &ok_flag, (d.withhold & 1) && blockIdx.x == 0);
    }
    if (ok) {
        build_routes(r, d.W_r ? d.logits_out : d.logits, T, d.E, k, d.renorm, d.err);
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
            float* h = sh ? d.h_shared + static_cast<size_t>(a) * T * Fs + f
                          : d.h + static_cast<size_t>(r.row0[a]) * F + f;
            for (; m; m &= m - 1, h += sh ? Fs : F) {
                const int t = __ffs(m) - 1;
                float g = 0.0f, up = 0.0f;
                for (int c = lane; c < H; c += 32) {
                    const float x = x_at<kType>(d.X, static_cast<size_t>(t) * H + c);
                    g = fmaf(plane_weight<kType, false>(pg, f, c, H), x, g);
                    up = fmaf(plane_weight<kType, false>(pu, f, c, H), x, up);
                }
                g = warp_sum(g);
                up = warp_sum(up);
                if (lane == 0)
                    *h = (sh ? 1.0f : route_alpha(r, t, e, k)) * scale * (g / (1.0f + expf(-g)) * up);
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
                        sh ? d.h_shared + (static_cast<size_t>(e) * T + t) * Fs
                           : d.h + static_cast<size_t>(r.row0[a] + __popc(r.mask[e] & ((1u << t) - 1u))) * F;
                    for (int c = lane; c < n; c += 32)
                        y = fmaf(plane_weight<kType, true>(pd, o, c, n), __ldcg(h + c), y);
                }
                y = warp_sum(y);
                if (lane == 0) {
                    const size_t at = static_cast<size_t>(t) * H + o;
                    d.Y[at] = (d.A ? x_at<kType>(d.A, at) : d.Y[at]) + y;
                }
            }
    }
    decode_leave(d.sync);
}

}  // namespace

cudaError_t launch_layer_decode(const DecodeCall& d, int wdtype, int num_sms, cudaStream_t stream) {
    const void* fn = wdtype == ESTREAM_F32  ? reinterpret_cast<const void*>(k_layer_decode_simple<ESTREAM_F32>)
                     : wdtype == ESTREAM_Q4 ? reinterpret_cast<const void*>(k_layer_decode_simple<ESTREAM_Q4>)
                                            : reinterpret_cast<const void*>(k_layer_decode_simple<ESTREAM_BF16>);
    const size_t smem = routes_bytes(d.T * d.k, d.E);
    DecodeCall call = d;
    void* args[] = {&call};
    return cudaLaunchCooperativeKernel(fn, dim3(num_sms), dim3(kSimpleThreads), args, smem, stream);
}

}  // namespace es
