// The next token of each row of logits from a given random number: temperature,
// top-k, top-p and min-p, then the first token in the vocabulary's order at which
// the kept weight exceeds u times the whole.
//
// Which token that is has to be what exact arithmetic says: with 10^5 tokens a
// cumulative weight that is off by 1e-7 names another one in a row of a hundred. So
// weights are integers, 2^42 for the largest, within 2^-38 of their value or one unit, and
// their sums are exact and the same in every order.
//
// A cluster of CTAs holds a row's logits in its shared memory (they are read from
// HBM once) and goes over them in passes, between which the CTAs exchange a few
// numbers. A cut (the k-th largest logit, or the logit at which top_p of the weight
// is reached) is found by bins: first of equal width in the logit, which spreads
// the logits over the bins, then, inside the bin with the cut, of equal width in
// the ordered bit pattern until a bin is a single value.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "estream_internal.h"
#include "overlap.cuh"

namespace es {
namespace {
namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 1024;
constexpr int kMaxCtas = 8;  // of a cluster
constexpr int kOne = 42;     // log2 of the largest weight

struct Sample {
    const void* logits;
    long long ld;
    int V, slice;  // logits of a CTA, a multiple of 8
    bool wide;     // rows lie on 16 bytes
    const float* u;
    float temperature, top_p, min_p;
    int top_k;
    const float *temperatures, *top_ps, *min_ps;
    const int32_t* top_ks;
    int32_t* ids;
    float* prob;
};

template <int kElem>
__device__ __forceinline__ float widen(const void* p, long long i) {
    if constexpr (kElem == ESTREAM_MX4_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    else if constexpr (kElem == ESTREAM_MX4_F16) return __half2float(static_cast<const __half*>(p)[i]);
    else return static_cast<const float*>(p)[i];
}

// Bit patterns in the order of the values, -0 as 0, NaN above all.
__device__ __forceinline__ uint32_t key_of(float x) {
    if (x != x) return ~0u;
    const uint32_t u = __float_as_uint(x + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// 2^-(2^-j) for j = 1 .. 8, 63 fractional bits.
__constant__ uint64_t kRoots[8] = {0x5a827999fcef3242ull, 0x6ba27e656b4eb57aull, 0x75606373ee921c97ull,
                                   0x7a92be8a92436616ull, 0x7d41d96db915019dull, 0x7e9f06067a4360baull,
                                   0x7f4f08ae3dc7c426ull, 0x7fa765aca88f6453ull};

// Weights of a row: exp((l - max) / temperature) = 2^-t, t = (max - l) c, c = log2 e / temperature.
// max - l and c are held as sums of two floats, so t is good to 2^-40; it is cut into
// whole, 1/256ths (a table) and a rest r < 2^-8, whose 2^-r is a short series.
struct Weights {
    float top, c, c_low;
    const uint64_t* table;  // 2^(42 - i / 256)
    // The weight is the result times 2^-s.
    __device__ __forceinline__ uint64_t parts(float l, int& s) const {
        s = 0;
        const float d = top - l;
        const float z = d - top, low = (top - (d - z)) - (l + z);  // what rounding took from d
        const float p = d * c;
        if (!(p < kOne + 2.0f)) return 0;
        const float q = fmaf(d, c, -p) + fmaf(d, c_low, low * c);
        const float n = floorf(p), f = p - n;
        const int i = static_cast<int>(f * 256.0f);
        const float r = f - static_cast<float>(i) * (1.0f / 256.0f);
        constexpr float kLn2 = 0.693147182464599609375f, kLn2Low = -1.904654299957767e-9f;
        const float xh = r * kLn2, xl = fmaf(r, kLn2, -xh) + fmaf(r, kLn2Low, q * kLn2), x = xh + xl;
        // e^-x - 1 + xh, without its leading -xh
        const float tail = fmaf(x * x, fmaf(x, fmaf(x, 1.0f / 24.0f, -1.0f / 6.0f), 0.5f), -xl);
        const long long change = static_cast<long long>(rintf(tail * 0x1p39f)) - static_cast<long long>(rintf(xh * 0x1p39f));
        const uint64_t t = table[i];
        const uint64_t w = t + static_cast<uint64_t>((static_cast<long long>(t >> 11) * change) >> 28);
        s = static_cast<int>(n);
        return w;
    }
    __device__ __forceinline__ uint64_t of(float l) const {
        int s;
        const uint64_t w = parts(l, s);
        return (w + (1ull << s >> 1)) >> s;
    }
};

template <typename T, typename F>
__device__ __forceinline__ T warp_reduce(T v, F&& join) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = join(v, __shfl_xor_sync(~0u, v, o));
    return v;
}
template <typename T>
__device__ __forceinline__ T add(T a, T b) {
    return a + b;
}

struct Exchange {  // a CTA's numbers that its cluster reads
    uint64_t best;   // key of its largest logit, then the complement of its index
    float least;     // its smallest finite logit
    uint32_t lo, hi; // keys of a bin
    uint64_t mass;
    uint32_t ties;
};

// The cut: kept are logits with key > tau, and the first `ties` in the vocabulary's
// order of those with key == tau.
struct Cut {
    uint32_t tau, ties;
};

struct Shared {
    uint64_t table[256];
    uint64_t bins[2][kBins];  // of this CTA, read by its cluster; used in turn
    uint64_t warp[kWarps];
    uint32_t warp2[kWarps];
    uint64_t found[2];
    double min_below;         // temperature ln(min_p)
    float c, c_low;           // log2 e / temperature
    Exchange exchange[2];     // used in turn
};

template <int kElem>
__global__ void __launch_bounds__(kThreads) k_sample(const Sample a) {
    extern __shared__ __align__(16) uint8_t raw[];
    Shared& sh = *reinterpret_cast<Shared*>(raw);
    float* logits = reinterpret_cast<float*>(raw + (sizeof(Shared) + 15) / 16 * 16);
    after_previous();
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int row = blockIdx.x / ctas, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int first = rank * a.slice, n = max(0, min(a.slice, a.V - first));
    const float given = a.temperatures ? a.temperatures[row] : a.temperature, temperature = given > 0x1p100f ? 0x1p100f : given;
    const int top_k = a.top_ks ? a.top_ks[row] : a.top_k;
    const float top_p = a.top_ps ? a.top_ps[row] : a.top_p;
    const float min_p = a.min_ps ? a.min_ps[row] : a.min_p;

    // in 64 bits by one thread: an SM does two such operations a clock
    if (tid == kThreads - 1) {
        const double c = 1.4426950408889634074 / static_cast<double>(fmaxf(temperature, 0x1p-100f));
        sh.c = static_cast<float>(c);
        sh.c_low = static_cast<float>(c - static_cast<double>(sh.c));
        if (min_p > 0.0f && min_p < 1.0f) sh.min_below = static_cast<double>(temperature) * log(static_cast<double>(min_p));
    }

    int turn = 0;  // of the exchanges: a number is written again only after a further meeting of the cluster
    // One value of every CTA, joined.
    auto across = [&](auto pick, auto join) {
        cluster.sync();
        auto v = pick(*cluster.map_shared_rank(&sh.exchange[turn], 0));
        for (int r = 1; r < ctas; ++r) v = join(v, pick(*cluster.map_shared_rank(&sh.exchange[turn], r)));
        turn ^= 1;
        return v;
    };

    // The logits, and the largest of them.
    uint64_t best = 0;
    float least = INFINITY;
    {
        const uint8_t* from = static_cast<const uint8_t*>(a.logits) + (row * a.ld + first) * (kElem == ESTREAM_MX4_F32 ? 4 : 2);
        constexpr int kPer = kElem == ESTREAM_MX4_F32 ? 4 : 8;
        auto take = [&](int i, float x) {
            logits[i] = x;
            best = max(best, static_cast<uint64_t>(key_of(x)) << 32 | ~static_cast<uint32_t>(first + i));
            if (x > -INFINITY) least = fminf(least, x);
        };
        const int vec = a.wide ? n / kPer * kPer : 0;
        for (int i = tid * kPer; i < vec; i += kThreads * kPer) {
            const uint4 w = *reinterpret_cast<const uint4*>(from + static_cast<size_t>(i) * (16 / kPer));
#pragma unroll
            for (int j = 0; j < kPer; ++j) take(i + j, widen<kElem>(&w, j));
        }
        for (int i = vec + tid; i < n; i += kThreads) take(i, widen<kElem>(from, i));
    }
    best = warp_reduce(best, [](uint64_t x, uint64_t y) { return max(x, y); });
    least = warp_reduce(least, [](float x, float y) { return fminf(x, y); });
    if (lane == 0) {
        sh.warp[warp] = best;
        sh.warp2[warp] = __float_as_uint(least);
    }
    if (tid < 256) {  // the table
        uint64_t v = 1ull << 63;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (tid >> (7 - j) & 1) v = __umul64hi(v, kRoots[j] << 1);
        sh.table[tid] = (v + (1ull << (62 - kOne))) >> (63 - kOne);
    }
    __syncthreads();
    if (tid == 0) {
        Exchange& e = sh.exchange[turn];
        e.best = 0;
        e.least = INFINITY;
        for (int w = 0; w < kWarps; ++w) {
            e.best = max(e.best, sh.warp[w]);
            e.least = fminf(e.least, __uint_as_float(sh.warp2[w]));
        }
    }
    const int seen = turn;
    best = across([](const Exchange& e) { return e.best; }, [](uint64_t x, uint64_t y) { return max(x, y); });
    least = INFINITY;
    for (int r = 0; r < ctas; ++r) least = fminf(least, cluster.map_shared_rank(&sh.exchange[seen], r)->least);

    const uint32_t top_key = static_cast<uint32_t>(best >> 32);
    const float top = value_of(top_key);
    const bool none = !(fabsf(top) < INFINITY) || top_key == ~0u, greedy = !(temperature > 0x1p-100f);
    if (none || greedy) {
        if (rank == 0 && tid == 0) {
            a.ids[row] = none ? -1 : static_cast<int>(~static_cast<uint32_t>(best));
            if (a.prob) a.prob[row] = none ? NAN : 1.0f;
        }
        cluster.sync();  // nobody leaves while others read its numbers
        return;
    }

    const Weights w{top, sh.c, sh.c_low, sh.table};

    // Finds where the measure of the tokens before reaches `target` > 0: by bins over
    // all logits of some weight and key >= floor_key, each bin's measure from `measure`.
    int which = 0;
    auto find = [&](auto measure, uint32_t floor_key, uint64_t target) {
        const float span = fminf(top - least, (kOne + 2.0f) / w.c);
        const float scale = span > 0.0f ? static_cast<float>(kBins) / span : 0.0f;
        auto linear = [&](float x) { return static_cast<int>(fminf((top - x) * scale, kBins - 1.0f)); };
        uint32_t lo = 0, hi = top_key;  // keys of the bin that holds the cut
        uint64_t before = 0;
        int shift = -1;                 // -1: bins over the logit
        for (;;) {
            uint64_t* bins = sh.bins[which];
            for (int b = tid; b < kBins; b += kThreads) bins[b] = 0;
            __syncthreads();
            for (int i = tid; i < n; i += kThreads) {
                const float x = logits[i];
                const uint32_t k = key_of(x);
                if (k < lo || k > hi || k < floor_key || x == -INFINITY) continue;
                const uint64_t m = measure(x, k);
                if (m == 0) continue;
                const int b = shift < 0 ? linear(x) : static_cast<int>((hi - k) >> shift);
                atomicAdd(reinterpret_cast<unsigned long long*>(bins + b), static_cast<unsigned long long>(m));
            }
            cluster.sync();
            // every CTA adds up all CTAs' bins; a thread two neighbouring ones
            uint64_t v[2] = {0, 0};
            for (int r = 0; r < ctas; ++r) {
                const uint64_t* other = cluster.map_shared_rank(bins, r);
                v[0] += other[2 * tid];
                v[1] += other[2 * tid + 1];
            }
            uint64_t upto = v[0] + v[1];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t y = __shfl_up_sync(~0u, upto, o);
                if (lane >= o) upto += y;
            }
            if (lane == 31) sh.warp[warp] = upto;
            if (tid == 0) sh.found[0] = ~0ull;
            __syncthreads();
            uint64_t base = before;
            for (int q = 0; q < warp; ++q) base += sh.warp[q];
            uint64_t at = base + upto - v[0] - v[1];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (at < target && at + v[j] >= target) {
                    sh.found[0] = 2 * tid + j;
                    sh.found[1] = at;
                }
                at += v[j];
            }
            __syncthreads();
            which ^= 1;
            const uint64_t bin = sh.found[0];
            if (bin == ~0ull) return Cut{floor_key ? floor_key - 1 : 0, 0};  // less than that in all: no cut
            before = sh.found[1];
            if (shift == 0) {
                const uint32_t tau = hi - static_cast<uint32_t>(bin);
                const uint64_t each = measure(value_of(tau), tau);
                return Cut{tau, static_cast<uint32_t>((target - before + each - 1) / each)};
            }
            if (shift < 0) {
                // the keys that the bin holds
                uint32_t small = ~0u, large = 0;
                for (int i = tid; i < n; i += kThreads) {
                    const float x = logits[i];
                    if (x == -INFINITY || linear(x) != static_cast<int>(bin)) continue;
                    small = min(small, key_of(x));
                    large = max(large, key_of(x));
                }
                small = __reduce_min_sync(~0u, small);
                large = __reduce_max_sync(~0u, large);
                if (lane == 0) sh.warp[warp] = static_cast<uint64_t>(small) << 32 | large;
                __syncthreads();
                if (tid == 0) {
                    Exchange& e = sh.exchange[turn];
                    e.lo = ~0u;
                    e.hi = 0;
                    for (int q = 0; q < kWarps; ++q) {
                        e.lo = min(e.lo, static_cast<uint32_t>(sh.warp[q] >> 32));
                        e.hi = max(e.hi, static_cast<uint32_t>(sh.warp[q]));
                    }
                }
                const uint64_t both = across([](const Exchange& e) { return static_cast<uint64_t>(~e.lo) << 32 | e.hi; },
                                             [](uint64_t x, uint64_t y) {
                                                 return max(x >> 32, y >> 32) << 32 | max(x & 0xffffffffu, y & 0xffffffffu);
                                             });
                lo = ~static_cast<uint32_t>(both >> 32);
                hi = static_cast<uint32_t>(both);
            } else {
                hi -= static_cast<uint32_t>(bin) << shift;
                lo = max(lo, hi - ((1u << shift) - 1));
            }
            shift = 0;
            while ((hi - lo) >> shift >= kBins) ++shift;
        }
    };
    // The kept weight, by warps (each a run of the CTA's logits) and over the cluster.
    const int run = (n + kWarps - 1) / kWarps, r0 = min(n, warp * run), r1 = min(n, r0 + run);
    auto kept = [&](Cut cut, uint64_t& above, uint32_t& ties) {
        above = 0;
        ties = 0;
        for (int i = r0 + lane; i < r1; i += 32) {
            const float x = logits[i];
            const uint32_t k = key_of(x);
            if (k > cut.tau) above += w.of(x);
            else if (k == cut.tau) ++ties;
        }
        above = warp_reduce(above, add<uint64_t>);
        ties = warp_reduce(ties, add<uint32_t>);
        __syncthreads();
        if (lane == 0) {
            sh.warp[warp] = above;
            sh.warp2[warp] = ties;
        }
        __syncthreads();
        if (tid == 0) {
            Exchange& e = sh.exchange[turn];
            e.mass = 0;
            e.ties = 0;
            for (int q = 0; q < kWarps; ++q) {
                e.mass += sh.warp[q];
                e.ties += sh.warp2[q];
            }
        }
    };

    Cut cut{0, 0};  // everything
    uint64_t above;
    uint32_t ties;
    if (top_k > 0 && top_k < a.V)
        cut = find([](float, uint32_t) { return 1ull; }, 0u, static_cast<uint64_t>(top_k));
    if (top_p < 1.0f || top_p != top_p) {
        kept(cut, above, ties);
        const int t = turn;
        uint64_t whole = across([](const Exchange& e) { return e.mass; }, add<uint64_t>);
        uint32_t all_ties = 0;
        for (int r = 0; r < ctas; ++r) all_ties += cluster.map_shared_rank(&sh.exchange[t], r)->ties;
        const uint64_t each = w.of(value_of(cut.tau));
        if (cut.ties) whole += min(cut.ties, all_ties) * each;
        // before < p whole, for integers: before < ceil(p whole)
        uint64_t target = 0;
        if (top_p > 0.0f) {
            const uint64_t p = __float2ull_rz(top_p * 0x1p64f);
            target = __umul64hi(p, whole) + (p * whole != 0);
        }
        if (target == 0) cut = Cut{top_key, 1};
        // the target is at most what the first cut keeps: where that ends among equal
        // logits, this one ends there or before
        else cut = find([&](float x, uint32_t) { return w.of(x); }, cut.tau + (cut.ties == 0), target);
    }
    if (min_p > 0.0f) {
        // w >= min_p, as a smallest logit: max + temperature ln(min_p)
        if (!(min_p < 1.0f)) {
            if (cut.tau < top_key) cut = Cut{top_key - 1, 0};
        } else {
            const uint32_t k = key_of(__double2float_ru(static_cast<double>(top) + sh.min_below));
            if (k > cut.tau) cut = Cut{k - 1, 0};
        }
    }
    kept(cut, above, ties);
    {
        cluster.sync();
        const uint64_t each = cut.ties ? w.of(value_of(cut.tau)) : 0;
        uint64_t whole = 0, my_start = 0, my_mass = 0;
        uint32_t ties_left = cut.ties, my_ties = 0;
        for (int r = 0; r < ctas; ++r) {
            const Exchange& e = *cluster.map_shared_rank(&sh.exchange[turn], r);
            const uint32_t t = min(ties_left, e.ties);
            const uint64_t m = e.mass + t * each;
            if (r == rank) {
                my_start = whole;
                my_mass = m;
                my_ties = ties_left;
            }
            ties_left -= t;
            whole += m;
        }
        const float u = a.u[row];
        uint64_t target = 0;  // the first token whose cumulative weight exceeds this
        if (u >= 1.0f) target = whole - 1;
        else if (u > 0.0f) target = __umul64hi(__float2ull_rz(u * 0x1p64f), whole);
        cluster.sync();  // the others' numbers have been read
        if (target < my_start || target >= my_start + my_mass) return;
        // the run with it
        uint64_t at = my_start;
        int q = 0;
        for (;; ++q) {
            const uint32_t t = min(my_ties, sh.warp2[q]);
            const uint64_t m = sh.warp[q] + t * each;
            if (target < at + m) break;
            at += m;
            my_ties -= t;
        }
        if (warp != q) return;
        for (int i0 = r0;; i0 += 32) {
            const int i = i0 + lane;
            const float x = i < r1 ? logits[i] : -INFINITY;
            const uint32_t k = key_of(x);
            const bool tie = i < r1 && cut.ties && k == cut.tau;
            const uint32_t tied = __ballot_sync(~0u, tie);
            const bool keep = i < r1 && (k > cut.tau || (tie && __popc(tied & ((1u << lane) - 1)) < my_ties));
            const uint64_t weight = keep ? w.of(x) : 0;
            uint64_t upto = weight;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t y = __shfl_up_sync(~0u, upto, o);
                if (lane >= o) upto += y;
            }
            const uint32_t over = __ballot_sync(~0u, at + upto > target);
            if (over) {
                if (lane == __ffs(over) - 1) {
                    a.ids[row] = first + i;
                    if (a.prob) {  // from the weight before it became a whole number of units
                        int s;
                        const double mine = static_cast<double>(w.parts(x, s));
                        a.prob[row] = static_cast<float>(mine / (static_cast<double>(1ull << s) * static_cast<double>(whole)));
                    }
                }
                return;
            }
            at += __shfl_sync(~0u, upto, 31);
            my_ties -= min(my_ties, static_cast<uint32_t>(__popc(tied)));
            if (i0 + 32 >= r1) return;
        }
    }
}

bool at(const void* p, size_t a) { return p && reinterpret_cast<uintptr_t>(p) % a == 0; }

template <int kElem>
cudaError_t launch(const Sample& s, int B, int ctas, cudaStream_t stream) {
    const size_t smem = (sizeof(Shared) + 15) / 16 * 16 + static_cast<size_t>(s.slice) * 4;
    cudaError_t rc = cudaFuncSetAttribute(k_sample<kElem>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (rc != cudaSuccess) return rc;
    cudaLaunchAttribute attr[2] = {overlapped(), {}};
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(B) * ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_sample<kElem>, s);
}

}  // namespace
}  // namespace es

using namespace es;

extern "C" estream_status estream_sample_tokens(const void* logits, int elem, long long ld, int B, int V, const float* u,
                                                float temperature, const float* temperature_rows, int top_k,
                                                const int32_t* top_k_rows, float top_p, const float* top_p_rows,
                                                float min_p, const float* min_p_rows, int32_t* ids, float* prob,
                                                void* cuda_stream) {
    NvtxRange range(kNvSample, B);
    if ((elem != ESTREAM_MX4_BF16 && elem != ESTREAM_MX4_F16 && elem != ESTREAM_MX4_F32) || B < 0 || B > 1 << 20 || V < 1 ||
        V > ESTREAM_SAMPLE_MAX_V || ld < 0)
        return ESTREAM_ERR_INVALID_ARG;
    if (B == 0) return ESTREAM_OK;
    const size_t size = elem == ESTREAM_MX4_F32 ? 4 : 2;
    if (!at(logits, size) || !at(u, 4) || !at(ids, 4) || (prob && !at(prob, 4)) ||
        (temperature_rows && !at(temperature_rows, 4)) || (top_k_rows && !at(top_k_rows, 4)) ||
        (top_p_rows && !at(top_p_rows, 4)) || (min_p_rows && !at(min_p_rows, 4)))
        return ESTREAM_ERR_INVALID_ARG;
    const estream_status st = on_device();
    if (st != ESTREAM_OK) return st;
    // as many CTAs a row as keep the device busy, of 2048 logits at least, and as many as hold the row
    int ctas = 1;
    while (ctas < kMaxCtas && (V > ctas * 24576 || (B * ctas < 152 && V > ctas * 2048))) ctas *= 2;
    Sample s{logits, ld, V, ((V + ctas - 1) / ctas + 7) / 8 * 8, at(logits, 16) && ld * size % 16 == 0, u,
             temperature, top_p, min_p, top_k, temperature_rows, top_p_rows, min_p_rows, top_k_rows, ids, prob};
    const cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
    const cudaError_t rc = elem == ESTREAM_MX4_BF16  ? launch<ESTREAM_MX4_BF16>(s, B, ctas, stream)
                           : elem == ESTREAM_MX4_F16 ? launch<ESTREAM_MX4_F16>(s, B, ctas, stream)
                                                     : launch<ESTREAM_MX4_F32>(s, B, ctas, stream);
    return rc == cudaSuccess ? ESTREAM_OK : ESTREAM_ERR_CUDA;
}
