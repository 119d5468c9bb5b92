// The next token of each row of logits from a given random number: temperature,
// top-k, top-p and min-p, then the first token in the vocabulary's order at which
// the kept weight exceeds u times the whole.
//
// Which token that is has to be what exact arithmetic says: with 10^5 tokens a
// cumulative weight that is off by 1e-7 names another one in a row of a hundred. So
// weights are integers, 2^45 for the largest, within 2^-37 of their value and half a unit, and
// their sums are exact and the same in every order. 2^45 is the most that 2^18.6 tokens
// leave 64 bits: half units add up to V 2^-46 of the largest weight where tokens far
// below it share one logit, at most 5.6e-9 (with 2^42, 4.5e-8 and a wrong token where u lay that near).
//
// A cluster of CTAs goes over a row in passes, between which the CTAs exchange a few numbers. Where a
// row may have a cut, it holds the row's logits in its shared memory, so they are read from HBM once.
//
// A cut (the k-th largest logit, or the one at which top_p of the weight is reached)
// is found by bins of equal width in the logit below the largest, counted and weighed by
// shared-memory atomics and added up over the cluster. Where few tokens lie up to
// the cut's bin, as after most prompts, they are gathered in one CTA, which does
// the rest alone: up to 128 by comparing each with all (sorting them took 32 rows of
// 102400 with top-k 40 from 17 to 21 us), more by sorting. Else the bin with the cut is divided again until its tokens
// can be sorted or are all equal, and the kept tokens are weighed and searched
// where they are.
//
// Without cuts the logits are not kept, so that more rows are under way: what may hold a kept
// token is read again, out of L2. With min-p or temperature 0 that is little: each lane notes
// the largest of each part (8 or more reads of 16 bytes), and the warp shares out those with a hit (reading whole runs
// of a warp again took 256 rows of 151936 fp32 with min-p 1.4 times as long). Without any choice all is weighed. Such rows
// take 30 us with temperature 0, 42 with min-p 0.02 and 111 without a choice.
//
// What bounds it: for few rows the meetings of the cluster (about 1 us each: three for a
// list, two without cuts), for many the weights. With each float operation of two logits'
// weights in one instruction, 256 rows without a choice take a tenth less.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>
#include <utility>

#include "estream_internal.h"
#include "overlap.cuh"

namespace es {
namespace {
namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
template <bool kCuts>
constexpr int kThreadsOf = kCuts ? kThreads : 256;  // without cuts: four CTAs an SM instead of two
constexpr int kBins = kThreads;  // one a thread
constexpr int kMaxCtas = 8;      // of a cluster
constexpr int kFew = 2 * kThreads;  // tokens that one CTA sorts
constexpr int kOne = 45;         // log2 of the largest weight
static_assert(ESTREAM_SAMPLE_MAX_V <= ~0ull >> kOne, "sums stay below 2^64");

struct Sample {
    const void* logits;
    long long ld;
    int V, slice;  // logits of a CTA, a multiple of 8
    const float* u;
    float temperature, top_p, min_p;
    int top_k;
    const float *temperatures, *top_ps, *min_ps;
    const int32_t* top_ks;
    int32_t* ids;
    float* prob;
};

template <int kElem>
struct Elem {
    static constexpr int kBytes = kElem == ESTREAM_MX4_F32 ? 4 : 2;
    static constexpr int kPer = 16 / kBytes;  // in 16 bytes
    static __device__ __forceinline__ float at(const void* p, int i) {
        if constexpr (kElem == ESTREAM_MX4_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
        else if constexpr (kElem == ESTREAM_MX4_F16) return __half2float(static_cast<const __half*>(p)[i]);
        else return static_cast<const float*>(p)[i];
    }
    static __device__ __forceinline__ void put(void* p, int i, float x) {
        if constexpr (kElem == ESTREAM_MX4_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(x);
        else if constexpr (kElem == ESTREAM_MX4_F16) static_cast<__half*>(p)[i] = __float2half_rn(x);
        else static_cast<float*>(p)[i] = x;
    }
};

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

// Two floats that one instruction works on.
struct F2 {
    uint64_t v;
    __device__ __forceinline__ F2() {}
    __device__ __forceinline__ F2(float x, float y) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y)); }
    __device__ __forceinline__ explicit F2(float x) : F2(x, x) {}
    __device__ __forceinline__ float2 get() const {
        float2 f;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
        return f;
    }
};
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// Weights of a row: exp((l - max) / temperature) = 2^-t, t = (max - l) c, c = log2 e / temperature.
// max - l and c are held as sums of two floats, so t is good to 2^-40; it is cut into
// whole, 1/256ths (a table) and a rest |r| <= 2^-9, whose 2^-r is a short series. Whole
// numbers come out of floats by adding 1.5 * 2^23, whose last bit is 1: conversions
// go through a unit of a quarter of the rate.
struct Weights {
    float top, c, c_low, past;  // past: a distance from the top at which weights are 0
    const uint64_t* table;      // 2^(kOne + 1 - i / 256)
    struct Two {
        uint64_t of[2];
        int s[2];
    };
    // Twice a weight is the result times 2^-s. Without branches, so that several are on their way, and for two logits
    // at once, whose floats' steps are one instruction for both.
    __device__ __forceinline__ Two parts(float l0, float l1) const {
        constexpr float kRound = 12582912.0f;
        constexpr int kRoundBits = 0x4b400000;
        constexpr float kLn2 = 0.693147182464599609375f, kLn2Low = -1.904654299957767e-9f;
        const F2 l(l0, l1), t(top), minus(-1.0f);
        const float2 full = fma(l, minus, t).get();
        const bool near[2] = {full.x < past, full.y < past};
        const F2 d(near[0] ? full.x : past, near[1] ? full.y : past);
        const F2 z = d + F2(-top);
        // what rounding took from d: (top - (d - z)) - (l + z)
        const float2 off = fma(l + z, minus, fma(fma(z, minus, d), minus, t)).get();
        const F2 low(near[0] ? off.x : 0.0f, near[1] ? off.y : 0.0f);
        const F2 np = d * F2(-c);  // -t, rounded, and what that leaves of t
        const F2 q = fma(d, F2(c), np) + fma(d, F2(c_low), low * F2(c));
        const F2 rounded = fma(np, F2(-256.0f), F2(kRound));
        const F2 nr = fma(rounded + F2(-kRound), F2(1.0f / 256.0f), np);  // -r
        const F2 xh = nr * F2(-kLn2);
        // -xl, where the exponent x is xh + xl
        const F2 nxl = fma(nr, F2(kLn2), xh) + fma(nr, F2(kLn2Low), q * F2(-kLn2));
        const F2 x = fma(nxl, minus, xh);
        // e^-x - 1 + xh, without its leading -xh; the next term is below 2^-42
        const F2 tail = fma(x * x, fma(x, F2(-1.0f / 6.0f), F2(0.5f)), nxl);
        const float2 small = fma(tail, F2(0x1p39f), F2(kRound)).get(), large = (xh * F2(0x1p39f)).get(), k2 = rounded.get();
        Two two;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int k = __float_as_int(i ? k2.y : k2.x) - kRoundBits;
            const int change = __float_as_int(i ? small.y : small.x) - kRoundBits - __float2int_rn(i ? large.y : large.x);
            const uint64_t w = table[k & 255];
            two.s[i] = k >> 8;
            two.of[i] = w + static_cast<uint64_t>((static_cast<long long>(static_cast<int>(w >> (kOne - 29))) * change) >> (68 - kOne));
        }
        return two;
    }
    __device__ __forceinline__ void of(float l0, float l1, uint64_t& w0, uint64_t& w1) const {
        const Two two = parts(l0, l1);
        w0 = ((two.of[0] >> two.s[0]) + 1) >> 1;
        w1 = ((two.of[1] >> two.s[1]) + 1) >> 1;
    }
    __device__ __forceinline__ uint64_t of(float l) const {
        uint64_t w, again;
        of(l, l, w, again);
        return w;
    }
    // A kept token's probability, from its weight before that became a whole number of units.
    __device__ __forceinline__ float share(float l, uint64_t whole) const {
        const Two two = parts(l, l);
        return static_cast<float>(static_cast<double>(two.of[0]) / (static_cast<double>(2ull << two.s[0]) * static_cast<double>(whole)));
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
template <typename T>
__device__ __forceinline__ T warp_scan(T v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(~0u, v, o);
        if (lane >= o) v += y;
    }
    return v;
}
__device__ __forceinline__ float max_or_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}
// The largest of 16 bytes' logits, NaN if one is NaN; packed types as they lie.
template <int kElem>
__device__ __forceinline__ float largest(const uint4& w) {
    if constexpr (kElem == ESTREAM_MX4_F32) {
        float m;
        asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(__uint_as_float(w.x)), "f"(__uint_as_float(w.y)), "f"(__uint_as_float(w.z)));
        return max_or_nan(m, __uint_as_float(w.w));
    } else if constexpr (kElem == ESTREAM_MX4_BF16) {
        const auto* h = reinterpret_cast<const __nv_bfloat162*>(&w);
        const float2 m = __bfloat1622float2(__hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3])));
        return max_or_nan(m.x, m.y);
    } else {
        const auto* h = reinterpret_cast<const __half2*>(&w);
        const float2 m = __half22float2(__hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3])));
        return max_or_nan(m.x, m.y);
    }
}

// The cut: kept are logits above `at`, and of those equal to it, `all` in number, the
// first `ties` in the vocabulary's order.
struct Cut {
    float at;
    uint32_t ties, all;
};

// What a search found: nothing, all tokens up to the cut's bin, listed in the leading CTA, or the cut.
enum Found { kNothing, kListed, kFound };

// A CTA's numbers that its cluster needs: each CTA stores its own in all of them, so that they are local
// when the cluster has met, and nobody has to stay for the others.
struct Exchange {
    float top, least;  // its largest logit (NaN if it has one), and smallest finite one
    int first;         // its first largest logit's index
    uint32_t lo, hi;   // keys of a bin
    uint32_t ties;
    uint64_t mass;
    Cut cut;
};

// A bin's measure: the number of its tokens, and their weight in three parts of 16 bits (a CTA has fewer than 2^16
// logits, so a part's sum stays in 32 bits), which native 32-bit atomics add up (an SM has none of 64 bits on shared memory, and loops instead: bins of
// 32000 logits took 11 us).
constexpr int kPart = 16;
static_assert(3 * kPart > kOne, "the largest weight fits its parts");
struct Bins {
    uint32_t count[kBins], part[3][kBins];
};
constexpr int kSlots = 8;  // parts of what a lane reads, at most
struct Shared {
    uint64_t table[256];
    union {
        struct {
            Bins bins;            // of this CTA, read by its cluster; else room for a list
            uint64_t sum[kBins];  // all CTAs' bins, added up
            uint32_t sum_count[kBins];
            uint64_t list[kFew];  // the leading CTA's: tokens to sort
        };
        struct {  // without cuts
            float tops[kSlots][kThreadsOf<false>];  // the largest logit of each part of what a lane reads
            uint16_t hits[kThreadsOf<false> / 32][32 * kSlots];  // a warp's parts with a kept token: part * 32 + lane
        };
    };
    uint64_t warp[kWarps];
    uint32_t warp2[kWarps];
    uint64_t before;
    Cut cut;
    uint32_t bin, members, upto, listed, collected, listed_at;
    float min_below, min_below_low;  // temperature ln(min_p)
    float c, c_low;                  // log2 e / temperature
    Exchange exchange[2][kMaxCtas];  // used in turn
};

__device__ __forceinline__ uint32_t cta_min(uint32_t v, uint32_t* room) {  // room: kWarps values
    v = __reduce_min_sync(~0u, v);
    if (threadIdx.x % 32 == 0) room[threadIdx.x / 32] = v;
    __syncthreads();
    v = __reduce_min_sync(~0u, room[threadIdx.x % kWarps]);
    __syncthreads();
    return v;
}

// Puts the list's n <= kFew different values in ascending order. Of a few, each value's place is
// the number of smaller ones. More are first dealt into as many bins of equal width in the
// upper word as there are threads, so that a value is compared with those of its bin alone.
__device__ __forceinline__ void sort(Shared& sh, int n) {
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    uint64_t* v = sh.list;
    __syncthreads();
    if (n <= kFew / 8) {
        int size = 16;
        while (size < n) size *= 2;
        const int share = kThreads / size, i = tid / share, part = tid % share;  // threads of a value
        const uint64_t mine = i < n ? v[i] : 0;
        int place = 0;
        if (i < n)
            for (int j = part; j < n; j += share) place += v[j] < mine;
        for (int o = share / 2; o; o >>= 1) place += __shfl_xor_sync(~0u, place, o);
        __syncthreads();
        if (i < n && part == 0) v[place] = mine;
        __syncthreads();
        return;
    }
    static_assert(sizeof(Bins) >= kFew * sizeof(uint64_t) && kBins >= kFew / 4, "a list fits the bins, two short ones the sums");
    uint64_t* dealt = reinterpret_cast<uint64_t*>(&sh.bins);
    uint32_t* count = sh.sum_count;
    uint64_t x[2];
    uint32_t small = ~0u, small_not = ~0u;
#pragma unroll
    for (int j = 0; j < 2; ++j)
        if (tid + j * kThreads < n) {
            x[j] = v[tid + j * kThreads];
            small = min(small, static_cast<uint32_t>(x[j] >> 32));
            small_not = min(small_not, ~static_cast<uint32_t>(x[j] >> 32));
        }
    count[tid] = 0;
    small = cta_min(small, sh.warp2);
    small_not = cta_min(small_not, sh.warp2);
    int shift = 0;
    while ((~small_not - small) >> shift >= kThreads) ++shift;
    uint32_t at[2], bin[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
        if (tid + j * kThreads < n) {
            bin[j] = (static_cast<uint32_t>(x[j] >> 32) - small) >> shift;
            at[j] = atomicAdd(&count[bin[j]], 1u);
        }
    __syncthreads();
    const uint32_t mine = count[tid], upto = warp_scan(mine, lane);
    if (lane == 31) sh.warp2[warp] = upto;
    __syncthreads();
    uint32_t before = upto - mine;
    for (int q = 0; q < warp; ++q) before += sh.warp2[q];
    uint32_t* start = reinterpret_cast<uint32_t*>(sh.sum);  // [kThreads + 1]
    start[tid] = before;
    if (tid == 0) start[kThreads] = n;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 2; ++j)
        if (tid + j * kThreads < n) dealt[start[bin[j]] + at[j]] = x[j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 2; ++j)
        if (tid + j * kThreads < n) {
            const uint32_t from = start[bin[j]], to = start[bin[j] + 1];
            uint32_t place = from;
            for (uint32_t q = from; q < to; ++q) place += dealt[q] < x[j];
            v[place] = x[j];
        }
    __syncthreads();
}

// kCuts: some row may have a top-k or a top-p. Without, logits are read again where a part's largest
// allows a kept token, out of L2, and a row needs no shared memory, so that more rows are under way.
template <int kElem, bool kCuts>
__global__ void __launch_bounds__(kThreadsOf<kCuts>, 1024 / kThreadsOf<kCuts>) k_sample(const Sample a) {
    using E = Elem<kElem>;
    constexpr int kThreads = kThreadsOf<kCuts>, kWarps = kThreads / 32;
    extern __shared__ __align__(16) uint8_t raw[];
    Shared& sh = *reinterpret_cast<Shared*>(raw);
    uint8_t* logits = raw + (sizeof(Shared) + 15) / 16 * 16;
    after_previous();
    cg::cluster_group cluster = cg::this_cluster();
    auto begun = cluster.barrier_arrive();  // nobody stores in a CTA that has not begun
    const int ctas = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int row = blockIdx.x / ctas, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    // Without cuts the CTA's logits are counted from the 16-byte boundary before them: `skew` of what lies from there
    // on is not the row's and never read. So rows of any alignment are read 16 bytes at a time (256 rows of
    // 151937 fp32 with min-p take as long as of 151936, with single reads 1.4 times as long). With cuts a row that is not on 16 bytes is read singly: it
    // costs 5 to 15% where it happens, and the counting 3% everywhere.
    const uint8_t* const start = static_cast<const uint8_t*>(a.logits) + (row * a.ld + rank * a.slice) * E::kBytes;
    const int past16 = static_cast<int>(reinterpret_cast<uintptr_t>(start) % 16 / E::kBytes), skew = kCuts ? 0 : past16;
    const uint8_t* const from = start - skew * E::kBytes;
    const int first = rank * a.slice - skew, n = max(0, min(a.slice, a.V - rank * a.slice)) + skew;

    const float given = a.temperatures ? a.temperatures[row] : a.temperature, temperature = given > 0x1p100f ? 0x1p100f : given;
    const int top_k = a.top_ks ? a.top_ks[row] : a.top_k;
    const float top_p = a.top_ps ? a.top_ps[row] : a.top_p;
    const float min_p = a.min_ps ? a.min_ps[row] : a.min_p;
    // a min-p above 1 leaves the first largest logit, too
    const bool greedy = !(temperature > 0x1p-100f) || min_p > 1.0f;
    const bool use_p = kCuts && !(top_p >= 1.0f);
    const bool use_k = kCuts && top_k > 0 && top_k < a.V;
    // in 64 bits by one thread: an SM does two such operations a clock
    if (tid == kThreads - 1) {
        const double c = 1.4426950408889634074 / static_cast<double>(fmaxf(temperature, 0x1p-100f));
        sh.c = static_cast<float>(c);
        sh.c_low = static_cast<float>(c - static_cast<double>(sh.c));
        if (min_p > 0.0f && min_p < 1.0f) {
            const double below = static_cast<double>(temperature) * log(static_cast<double>(min_p));
            sh.min_below = static_cast<float>(below);
            sh.min_below_low = static_cast<float>(below - static_cast<double>(sh.min_below));
        }
        sh.listed = 0;
    }
    for (int i = tid; i < 256; i += kThreads) {  // the table
        uint64_t v = 1ull << 63;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (i >> (7 - j) & 1) v = __umul64hi(v, kRoots[j] << 1);
        sh.table[i] = (v + (1ull << (61 - kOne))) >> (62 - kOne);
    }
    auto given_at = [&](int i) { return i >= skew && i < n ? E::at(from, i) : -INFINITY; };
    auto at = [&](int i) { return kCuts ? E::at(logits, i) : given_at(i); };
    auto chunk = [&](int i) {  // 16 bytes from logit i on
        if constexpr (kCuts) return *reinterpret_cast<const uint4*>(logits + static_cast<size_t>(i) * E::kBytes);
        if (i >= skew && i + E::kPer <= n) return *reinterpret_cast<const uint4*>(from + static_cast<size_t>(i) * E::kBytes);
        uint4 w;
#pragma unroll
        for (int j = 0; j < E::kPer; ++j) E::put(&w, j, at(i + j));
        return w;
    };
    // A warp has a run of the CTA's logits; runs begin and end at multiples of 8 (past the row's end lies -infinity).
    const int padded = (n + 7) / 8 * 8, length = ((padded + kWarps - 1) / kWarps + 7) / 8 * 8;
    const int run_begin = min(padded, warp * length), run_end = min(padded, run_begin + length);
    float run_top = -INFINITY;  // its largest
    // the run's whole 16 bytes are [vec_begin, vec)
    const int vec_begin = run_begin / E::kPer + (run_begin < skew), vec = kCuts && past16 ? 0 : min(n, run_end) / E::kPer;
    constexpr int kAtOnce = 8;  // 16 bytes that a lane reads at a time
    const int batches = (vec - vec_begin + 32 * kAtOnce - 1) / (32 * kAtOnce);  // of a warp; none or less: none
    const int per_slot = max(1, (batches + kSlots - 1) / kSlots);
    int turn = 0;  // of the exchanges: a number is stored again only after a further meeting of the cluster
    // This CTA's numbers to the others: by the first warp, a CTA a lane. Then the cluster meets, and
    // warps read a CTA a lane, and join them.
    auto give = [&](auto set) {
        if (warp == 0 && lane < ctas) set(cluster.map_shared_rank(&sh.exchange[turn][rank], lane));
        cluster.sync();
        turn ^= 1;
    };
    auto given_by = [&](int r) -> const Exchange& { return sh.exchange[turn ^ 1][r]; };
    constexpr float kLowest = -3.402823466e38f;  // what can be drawn is finite
    // f(16 bytes' logits, i) where one of them may be at or above `lowest`
    constexpr int kAhead = 4;  // reads that a lane has under way, without cuts (one alone: 4% longer without a choice)
    auto chunks_of_run = [&](float lowest, auto f) {
        if (!(run_top >= lowest)) return;
        int i = run_begin;
        if (!kCuts && lowest > kLowest) {
            // the warp shares out what its lanes with a hit have read
            int hits = 0;
            for (int slot = 0; slot * per_slot < batches; ++slot) {
                const bool hit = sh.tops[slot][tid] >= lowest;
                const uint32_t mask = __ballot_sync(~0u, hit);
                if (hit) sh.hits[warp][hits + __popc(mask & ((1u << lane) - 1))] = slot * 32 + lane;
                hits += __popc(mask);
            }
            __syncwarp();
            const int each = per_slot * kAtOnce;                       // reads of a part
            const uint32_t over = 0xffffffffu / max(1, hits) + 1;  // 2^32 / hits: e * hits < 2^32, so quotients are exact
            for (int e0 = lane; e0 < hits * each; e0 += 32 * kAhead) {
                uint4 w[kAhead];
                int c[kAhead];
#pragma unroll
                for (int q = 0; q < kAhead; ++q) {
                    const int e = e0 + 32 * q;
                    c[q] = vec;
                    if (e < hits * each) {
                        const int j = hits == 1 ? e : __umulhi(e, over), h = sh.hits[warp][e - j * hits];
                        c[q] = vec_begin + ((h >> 5) * each + j) * 32 + (h & 31);
                    }
                    if (c[q] < vec) w[q] = reinterpret_cast<const uint4*>(from)[c[q]];
                }
#pragma unroll
                for (int q = 0; q < kAhead; ++q)
                    if (c[q] < vec) f(w[q], c[q] * E::kPer);
            }
            __syncwarp();
            if (run_begin < skew && lane == 0) f(chunk(run_begin), run_begin);
            i = max(vec_begin, vec) * E::kPer;
        }
        constexpr int kStep = 32 * E::kPer;
        if (!kCuts)
            for (; i + kAhead * kStep <= run_end; i += kAhead * kStep) {
                uint4 w[kAhead];
#pragma unroll
                for (int q = 0; q < kAhead; ++q) w[q] = chunk(i + q * kStep + lane * E::kPer);
#pragma unroll
                for (int q = 0; q < kAhead; ++q) f(w[q], i + q * kStep + lane * E::kPer);
            }
        for (i += lane * E::kPer; i < run_end; i += kStep) f(chunk(i), i);
    };
    // f(x, i) for four logits from i on, where one of them is at or above `lowest`
    auto fours_of_run = [&](float lowest, auto f) {
        chunks_of_run(lowest, [&](const uint4& w, int i) {
            if (!(largest<kElem>(w) >= lowest)) return;
#pragma unroll
            for (int j = 0; j < E::kPer; j += 4) {
                const float x[4] = {E::at(&w, j), E::at(&w, j + 1), E::at(&w, j + 2), E::at(&w, j + 3)};
                f(x);
            }
        });
    };
    auto each_of_run = [&](float lowest, auto f) {
        chunks_of_run(lowest, [&](const uint4& w, int i) {
            if (!(largest<kElem>(w) >= lowest)) return;
#pragma unroll
            for (int j = 0; j < E::kPer; ++j) {
                const float x = E::at(&w, j);
                if (x >= lowest) f(x, i + j);
            }
        });
    };
    // the warps' v, a lane of each warp
    auto of_warps = [&](uint64_t v) {
        if (lane == 0) sh.warp[warp] = v;
        __syncthreads();
        return sh.warp[lane % kWarps];
    };

    // The largest logit and the range; with cuts the logits come to shared memory on the way.
    float top = -INFINITY, least = INFINITY;
    {
        const bool ranged = use_k || use_p;
        auto low = [&](float x) {
            if (x > -INFINITY) least = fminf(least, x);
        };
        for (int batch = 0; batch < batches; ++batch) {
            const int i0 = vec_begin + batch * kAtOnce * 32 + lane;
            uint4 v[kAtOnce];
            float batch_top = -INFINITY;
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j)
                if (i0 + j * 32 < vec) v[j] = reinterpret_cast<const uint4*>(from)[i0 + j * 32];
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j)
                if (i0 + j * 32 < vec) {
                    if constexpr (kCuts) reinterpret_cast<uint4*>(logits)[i0 + j * 32] = v[j];
                    batch_top = max_or_nan(batch_top, largest<kElem>(v[j]));
                    if (ranged)
#pragma unroll
                        for (int q = 0; q < E::kPer; ++q) low(E::at(&v[j], q));
                }
            run_top = max_or_nan(run_top, batch_top);
            if constexpr (!kCuts) {
                float& slot_top = sh.tops[batch / per_slot][tid];
                slot_top = batch % per_slot ? max_or_nan(slot_top, batch_top) : batch_top;
            }
        }
        auto one = [&](int i) {
            const float x = given_at(i);
            run_top = max_or_nan(run_top, x);
            if (ranged) low(x);
            if constexpr (kCuts) E::put(logits, i, x);
        };
        if (run_begin < skew && lane < E::kPer) one(lane);
        for (int i = max(vec_begin, vec) * E::kPer + lane; i < run_end; i += 32) one(i);
        top = run_top = warp_reduce(run_top, max_or_nan);
        least = warp_reduce(least, fminf);
        const uint64_t both = of_warps(static_cast<uint64_t>(__float_as_uint(top)) << 32 | __float_as_uint(least));
        top = __uint_as_float(static_cast<uint32_t>(both >> 32));
        least = __uint_as_float(static_cast<uint32_t>(both));
        if (warp == 0) {
            top = warp_reduce(top, max_or_nan);
            least = warp_reduce(least, fminf);
        }
        cluster.barrier_wait(std::move(begun));
        give([&](Exchange* e) {
            e->top = top;
            e->least = least;
        });
        top = warp_reduce(lane < ctas ? given_by(lane).top : -INFINITY, max_or_nan);
        least = warp_reduce(lane < ctas ? given_by(lane).least : INFINITY, fminf);
    }
    const bool none = !(fabsf(top) < INFINITY);
    if (none || greedy) {
        int mine = 0x7fffffff;
        if (!none) each_of_run(top, [&](float, int i) { mine = min(mine, first + i); });
        mine = __reduce_min_sync(~0u, static_cast<uint32_t>(mine));
        mine = static_cast<int>(of_warps(static_cast<uint64_t>(mine)));
        if (warp == 0) mine = __reduce_min_sync(~0u, static_cast<uint32_t>(mine));
        give([&](Exchange* e) { e->first = mine; });
        if (rank == 0 && tid == 0) {
            for (int r = 0; r < ctas; ++r) mine = min(mine, given_by(r).first);
            a.ids[row] = none ? -1 : mine;
            if (a.prob) a.prob[row] = none ? NAN : 1.0f;
        }
        return;
    }

    const Weights w{top, sh.c, sh.c_low, (kOne + 3.0f) / sh.c, sh.table};
    const float u = a.u[row];
    // the first token whose cumulative weight exceeds this is drawn
    auto point = [&](uint64_t whole) {
        return u >= 1.0f ? whole - 1 : u > 0.0f ? __umul64hi(__float2ull_rz(u * 0x1p64f), whole) : 0;
    };
    // before < top_p whole, for integers: before < this
    auto share = [&](uint64_t whole) -> uint64_t {
        if (!(top_p > 0.0f)) return 0;
        const uint64_t p = __float2ull_rz(top_p * 0x1p64f);
        return __umul64hi(p, whole) + (p * whole != 0);
    };
    // w >= min_p as a smallest logit: max + temperature ln(min_p)
    float least_kept = -INFINITY;
    if (min_p > 0.0f) {
        least_kept = top;
        if (min_p < 1.0f) {
            const float y = sh.min_below, sum = top + y, z = sum - top;
            const float rest = ((top - (sum - z)) + (y - z)) + sh.min_below_low;  // of the sum in full
            const float up = rest > 0.0f ? value_of(key_of(sum) + 1) : sum;     // rounded up
            least_kept = fminf(top, up);
        }
    }
    auto item = [&](float x, int i) { return static_cast<uint64_t>(~key_of(x)) << 32 | static_cast<uint32_t>(first + i); };
    auto logit_of = [&](uint64_t it) { return value_of(~static_cast<uint32_t>(it >> 32)); };
    // Sums of two values a thread, in the threads' order: what lies before them, and all.
    auto scan = [&](uint64_t v0, uint64_t v1, uint64_t& before, uint64_t& whole) {
        const uint64_t upto = warp_scan(v0 + v1, lane);
        __syncthreads();
        if (lane == 31) sh.warp[warp] = upto;
        __syncthreads();
        before = upto - v0 - v1;
        whole = 0;
        for (int q = 0; q < kWarps; ++q) {
            if (q < warp) before += sh.warp[q];
            whole += sh.warp[q];
        }
    };

    // Where the measure (each token's weight, or 1) reaches a target: bins over the logits
    // at or above `floor`, then over those of the bin with the cut. The target is formed
    // from the whole measure; with may_list, tokens up to the first bin's end are
    // only listed where they are few.
    uint64_t target = 0;
    Cut cut{-INFINITY, 0, 0};  // everything
    // This CTA's tokens that are wanted go where the bins are; room for kFew. sh.collected is 0 before.
    uint64_t* const staged = reinterpret_cast<uint64_t*>(&sh.bins);
    auto append = [&](bool wanted, float x, int i) {  // by the lanes that come here together
        const uint32_t here = __activemask(), mask = __ballot_sync(here, wanted);
        if (!mask) return;
        uint32_t to = 0;
        if (lane == __ffs(mask) - 1) to = atomicAdd(&sh.collected, static_cast<uint32_t>(__popc(mask)));
        to = __shfl_sync(here, to, __ffs(mask) - 1) + __popc(mask & ((1u << lane) - 1));
        if (wanted && to < kFew) staged[to] = item(x, i);
    };
    auto hand_over = [&](uint32_t at) {  // to the leading CTA's list
        uint64_t* list = cluster.map_shared_rank(sh.list, 0);
        for (uint32_t i = tid; i < sh.collected; i += kThreads) list[at + i] = staged[i];
    };
    auto find = [&](auto weighs, float floor, auto aim, bool may_list) {
        constexpr bool kWeigh = decltype(weighs)::value;
        const float span = fminf(top - least, (kOne + 2.0f) / w.c);
        const float scale = span > 0.0f ? static_cast<float>(kBins) / span : 0.0f;
        auto bin_of = [&](float x) { return fminf((top - x) * scale, static_cast<float>(kBins)); };  // kBins: as kBins - 1
        float base = 0.0f;     // of the second division's bin
        uint32_t lo = 0, hi = 0;  // keys that later ones divide
        int shift = 0;
        uint64_t before = 0;
        for (int level = 0;; ++level) {
            Bins& bins = sh.bins;
            bins.count[tid] = bins.part[0][tid] = bins.part[1][tid] = bins.part[2][tid] = 0;
            __syncthreads();
            auto place = [&](float x) {  // -1: not in question
                if (level >= 2) {
                    const uint32_t k = key_of(x);
                    return k < lo || k > hi ? -1 : static_cast<int>((hi - k) >> shift);
                }
                const int b = min(kBins - 1, static_cast<int>(bin_of(x)));
                if (level == 0) return b;
                return b != static_cast<int>(base) ? -1 : min(kBins - 1, static_cast<int>((bin_of(x) - base) * kBins));
            };
            fours_of_run(floor, [&](const float (&x)[4]) {
                int b[4];
                uint64_t m[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    b[q] = x[q] >= floor ? place(x[q]) : -1;
                    m[q] = 1;
                }
                if constexpr (kWeigh) {
                    w.of(x[0], x[1], m[0], m[1]);
                    w.of(x[2], x[3], m[2], m[3]);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (b[q] < 0 || m[q] == 0) continue;
                    if constexpr (kWeigh) {
#pragma unroll
                        for (int j = 0; j < 3; ++j)
                            atomicAdd(&bins.part[j][b[q]], static_cast<uint32_t>(m[q] >> kPart * j) & (1u << kPart) - 1);
                    }
                    atomicAdd(&bins.count[b[q]], 1u);
                }
            });
            cluster.sync();
            // A CTA adds up its share of the bins, a thread a bin of one of the CTAs, and stores the sums in all.
            uint64_t v = 0;
            uint32_t c = 0;
            {
                const int r = tid & (ctas - 1), b = rank * (kBins / ctas) + tid / ctas;
                const Bins& theirs = *cluster.map_shared_rank(&bins, r);
                c = theirs.count[b];
                if constexpr (kWeigh) {
#pragma unroll
                    for (int j = 0; j < 3; ++j) v += static_cast<uint64_t>(theirs.part[j][b]) << kPart * j;
                }
                for (int o = 1; o < ctas; o *= 2) {
                    c += __shfl_xor_sync(~0u, c, o);
                    if constexpr (kWeigh) v += __shfl_xor_sync(~0u, v, o);
                }
                cluster.map_shared_rank(sh.sum_count, r)[b] = c;
                if constexpr (kWeigh) cluster.map_shared_rank(sh.sum, r)[b] = v;
            }
            cluster.sync();
            c = sh.sum_count[tid];
            v = kWeigh ? sh.sum[tid] : c;
            const uint64_t upto = warp_scan(v, lane);
            const uint32_t counted = warp_scan(c, lane);
            if (lane == 31) {
                sh.warp[warp] = upto;
                sh.warp2[warp] = counted;
            }
            if (tid == 0) sh.bin = ~0u;
            __syncthreads();
            uint64_t start = before, whole = 0;
            uint32_t ahead = 0;
            for (int q = 0; q < kWarps; ++q) {
                if (q < warp) {
                    start += sh.warp[q];
                    ahead += sh.warp2[q];
                }
                whole += sh.warp[q];
            }
            if (level == 0) target = aim(whole);
            start += upto - v;
            if (start < target && start + v >= target) {
                sh.bin = tid;
                sh.before = start;
                sh.members = c;
                sh.upto = ahead + counted;
            }
            __syncthreads();
            const int bin = static_cast<int>(sh.bin);
            if (bin < 0) return kNothing;  // less than that in all, or a target of 0
            before = sh.before;
            const uint32_t members = sh.members;
            const bool all = may_list && level == 0 && sh.upto <= kFew;
            if (all || members <= kFew) {
                // nothing outside the bin's ends, with room for roundings, can be in it
                float from = floor, to = INFINITY;
                if (level == 0) {
                    const float width = 1.0f / scale, slack = width * 0.01f + fabsf(top) * 1e-6f;
                    if (bin < kBins - 1) from = fmaxf(floor, top - static_cast<float>(bin + 1) * width - slack);
                    if (!all) to = top - static_cast<float>(bin) * width + slack;
                }
                if (tid == 0) sh.collected = 0;
                __syncthreads();  // and all have read the bins' sums
                each_of_run(from, [&](float x, int i) {
                    if (x > to) return;
                    const int b = place(x);
                    if (b != bin && !(all && b < bin && b >= 0)) return;
                    append(!(kWeigh && w.of(x) == 0), x, i);  // as they were counted
                });
                __syncthreads();
                if (tid == 0) sh.listed_at = atomicAdd(cluster.map_shared_rank(&sh.listed, 0), sh.collected);
                __syncthreads();
                hand_over(sh.listed_at);
                cluster.sync();
                if (all) return kListed;
                if (rank == 0) {
                    const int m = static_cast<int>(sh.listed);
                    sort(sh, m);
                    uint64_t v2[2], lead, sum;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int p = 2 * tid + j;
                        v2[j] = p >= m ? 0 : kWeigh ? w.of(logit_of(sh.list[p])) : 1;
                    }
                    scan(v2[0], v2[1], lead, sum);
                    lead += before;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if (lead < target && lead + v2[j] >= target) {
                            const int p = 2 * tid + j;
                            const uint64_t key = sh.list[p] >> 32;
                            auto bound = [&](uint64_t k) {  // the first with a key at or behind k
                                int x = 0, y = m;
                                while (x < y) {
                                    const int mid = (x + y) / 2;
                                    if (sh.list[mid] >> 32 < k) x = mid + 1;
                                    else y = mid;
                                }
                                return x;
                            };
                            const int from = bound(key), to = bound(key + 1);
                            sh.cut = Cut{logit_of(sh.list[p]), static_cast<uint32_t>(p + 1 - from), static_cast<uint32_t>(to - from)};
                        }
                        lead += v2[j];
                    }
                    __syncthreads();
                    cut = sh.cut;
                    if (tid == 0) sh.listed = 0;
                    if (warp == 0 && lane < ctas) cluster.map_shared_rank(&sh.exchange[turn][0], lane)->cut = cut;
                }
                cluster.sync();
                turn ^= 1;
                cut = given_by(0).cut;
                return kFound;
            }
            if (level >= 2 && shift == 0) {  // equal logits
                const float x = value_of(hi - static_cast<uint32_t>(bin));
                const uint64_t m = kWeigh ? w.of(x) : 1;
                cut = Cut{x, static_cast<uint32_t>((target - before + m - 1) / m), members};
                return kFound;
            }
            if (level == 0) {
                base = static_cast<float>(bin);
                continue;
            }
            if (level == 1) {  // the keys that the bin holds
                uint32_t small = ~0u, large = 0;
                each_of_run(floor, [&](float x, int) {
                    if (place(x) != bin) return;
                    small = min(small, key_of(x));
                    large = max(large, key_of(x));
                });
                small = __reduce_min_sync(~0u, small);
                large = __reduce_max_sync(~0u, large);
                const uint64_t both = of_warps(static_cast<uint64_t>(small) << 32 | large);
                small = static_cast<uint32_t>(both >> 32);
                large = static_cast<uint32_t>(both);
                if (warp == 0) {
                    small = __reduce_min_sync(~0u, small);
                    large = __reduce_max_sync(~0u, large);
                }
                give([&](Exchange* e) {
                    e->lo = small;
                    e->hi = large;
                });
                lo = __reduce_min_sync(~0u, lane < ctas ? given_by(lane).lo : ~0u);
                hi = __reduce_max_sync(~0u, lane < ctas ? given_by(lane).hi : 0u);
            } else {
                hi -= static_cast<uint32_t>(bin) << shift;
                lo = max(lo, hi - ((1u << shift) - 1));
            }
            shift = 0;
            while ((hi - lo) >> shift >= kBins) ++shift;
        }
    };
    // What the leading CTA does with a list of the likeliest tokens: the first `most` of them
    // are what top-k keeps; limit: the target of top-p, or 0 to form it from their weight.
    auto finish = [&](int most, uint64_t limit) {
        const int m = static_cast<int>(sh.listed);
        if (m <= kFew / 8) {
            // Nothing is sorted: every token meets every other, by several threads a token. First what is likelier,
            // or as likely and earlier; then what is kept and earlier.
            uint64_t* weights = sh.sum;
            uint64_t* kept = sh.sum + kFew / 8;
            int size = 16;
            while (size < m) size *= 2;
            const int parts = kThreads / size, i = tid / parts, part = tid % parts;
            __syncthreads();  // the list is whole
            const uint64_t mine = i < m ? sh.list[i] : 0;
            const float x = i < m ? logit_of(mine) : -INFINITY;
            const uint64_t weight = w.of(x);
            if (i < m && part == 0) weights[i] = weight;
            __syncthreads();
            int place = 0;
            uint64_t lead = 0;
            if (i < m)
                for (int j = part; j < m; j += parts) {
                    const bool ahead = sh.list[j] < mine;
                    place += ahead;
                    lead += ahead ? weights[j] : 0;
                }
            for (int o = parts / 2; o; o >>= 1) {
                place += __shfl_xor_sync(~0u, place, o);
                lead += __shfl_xor_sync(~0u, lead, o);
            }
            if (use_p && limit == 0) {
                uint64_t before, whole;
                scan(i < m && part == 0 && place < most ? weight : 0, 0, before, whole);
                limit = share(whole);
            }
            const bool keep = i < m && (place == 0 || (place < most && x >= least_kept && (!use_p || lead < limit)));
            if (i < m && part == 0) kept[i] = keep ? weight : 0;
            __syncthreads();
            uint64_t upto = 0, whole = 0;
            for (int j = part; j < m; j += parts) {
                whole += kept[j];
                upto += static_cast<uint32_t>(sh.list[j]) <= static_cast<uint32_t>(mine) ? kept[j] : 0;
            }
            for (int o = parts / 2; o; o >>= 1) {
                whole += __shfl_xor_sync(~0u, whole, o);
                upto += __shfl_xor_sync(~0u, upto, o);
            }
            const uint64_t goal = point(whole);
            if (keep && part == 0 && upto > goal && upto - weight <= goal) {
                a.ids[row] = static_cast<int>(static_cast<uint32_t>(mine));
                if (a.prob) a.prob[row] = w.share(x, whole);
            }
            return;
        }
        sort(sh, m);
        most = min(most, m);
        float x[2];
        uint64_t v[2], lead, whole;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int p = 2 * tid + j;
            x[j] = p < most ? logit_of(sh.list[p]) : -INFINITY;
            v[j] = w.of(x[j]);
        }
        scan(v[0], v[1], lead, whole);
        if (use_p && limit == 0) limit = share(whole);
        const bool keep[2] = {tid == 0 || (2 * tid < most && x[0] >= least_kept && (!use_p || lead < limit)),
                              2 * tid + 1 < most && x[1] >= least_kept && (!use_p || lead + v[0] < limit)};
        // kept tokens are the first ones
        const int kept = __syncthreads_count(keep[0]) + __syncthreads_count(keep[1]);
        uint64_t to[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint64_t it = sh.list[2 * tid + j];
            to[j] = it << 32 | it >> 32;  // index first
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (keep[j]) sh.list[2 * tid + j] = to[j];
        sort(sh, kept);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int p = 2 * tid + j;
            to[j] = p < kept ? sh.list[p] : 0;
            x[j] = value_of(~static_cast<uint32_t>(to[j]));
            v[j] = p < kept ? w.of(x[j]) : 0;
        }
        scan(v[0], v[1], lead, whole);
        const uint64_t goal = point(whole);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (lead <= goal && lead + v[j] > goal) {
                a.ids[row] = static_cast<int>(to[j] >> 32);
                if (a.prob) a.prob[row] = w.share(x[j], whole);
            }
            lead += v[j];
        }
    };

    if constexpr (kCuts) {
        int most = 0;        // listed: the leading CTA's list has the cut
        uint64_t limit = 0;  // its target, for top-p alone
        if (use_k) {
            const Found f = find(std::false_type{}, kLowest, [&](uint64_t) { return static_cast<uint64_t>(top_k); }, true);
            if (f == kListed) most = top_k;
        }
        if (use_p && !most) {
            // equal logits that top-k leaves out are weighed with the others
            const uint64_t surplus = cut.ties ? (cut.all - cut.ties) * w.of(cut.at) : 0;
            const Found f = find(std::true_type{}, fmaxf(cut.at, kLowest), [&](uint64_t whole) { return share(whole - surplus); }, cut.ties == 0);
            if (f == kListed) {
                most = kFew;
                limit = target;
            }
            if (f == kNothing) cut = Cut{top, 1, 1};  // top_p of 0
        }
        if (most) {
            if (rank == 0) finish(most, limit);
            return;
        }
    }
    if (least_kept > cut.at) cut = Cut{-INFINITY, 0, 0};
    // The kept weight, by warps, each of which has a run of the CTA's logits, and over the cluster.
    const float lowest = fmaxf(fmaxf(cut.at, least_kept), kLowest);
    auto weigh_chunk = [&](const uint4& v, uint64_t& mass, uint32_t& ties) {
        if (!(largest<kElem>(v) >= lowest)) return;
#pragma unroll
        for (int j = 0; j < E::kPer; j += 4) {
            const float x[4] = {E::at(&v, j), E::at(&v, j + 1), E::at(&v, j + 2), E::at(&v, j + 3)};
            uint64_t m[4];
            w.of(x[0], x[1], m[0], m[1]);
            w.of(x[2], x[3], m[2], m[3]);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const bool tied = cut.ties && x[q] == cut.at;
                ties += tied;
                mass += x[q] >= lowest && !tied ? m[q] : 0;
            }
        }
    };
    const uint64_t tie = cut.ties ? w.of(cut.at) : 0;
    uint64_t mass = 0;
    uint32_t ties = 0;
    chunks_of_run(lowest, [&](const uint4& v, int) { weigh_chunk(v, mass, ties); });
    mass = warp_reduce(mass, add<uint64_t>);
    ties = __reduce_add_sync(~0u, ties);
    // What precedes, of this lane's value in its warp: (mass, ties) in the vocabulary's order, of which only the
    // first `left` ties count.
    struct Before {
        uint64_t start, mass;
        uint32_t left;
    };
    auto line_up = [&](uint64_t m, uint32_t n_ties, uint64_t start, uint32_t left) {
        const uint32_t earlier = warp_scan(n_ties, lane) - n_ties;
        Before b;
        b.left = left - min(left, earlier);
        b.mass = m + min(b.left, n_ties) * tie;
        b.start = start + warp_scan(b.mass, lane) - b.mass;
        return b;
    };
    // The lane whose value has the goal, and what precedes it there.
    auto pick = [&](Before& b, uint64_t goal) {
        const int who = __ffs(__ballot_sync(~0u, goal >= b.start && goal < b.start + b.mass)) - 1;
        b.start = __shfl_sync(~0u, b.start, max(who, 0));
        b.left = __shfl_sync(~0u, b.left, max(who, 0));
        return who;
    };
    if (lane == 0) {
        sh.warp[warp] = mass;
        sh.warp2[warp] = ties;
    }
    __syncthreads();
    if (warp == 0) {
        mass = warp_reduce(lane < kWarps ? sh.warp[lane] : 0, add<uint64_t>);
        ties = __reduce_add_sync(~0u, lane < kWarps ? sh.warp2[lane] : 0);
    }
    give([&](Exchange* e) {
        e->mass = mass;
        e->ties = ties;
    });
    Before b = line_up(lane < ctas ? given_by(lane).mass : 0, lane < ctas ? given_by(lane).ties : 0, 0, cut.ties);
    const uint64_t whole = __shfl_sync(~0u, b.start + b.mass, 31), goal = point(whole);
    if (pick(b, goal) != rank) return;
    // The run with it, a thread's share of that run, and the token.
    b = line_up(lane < kWarps ? sh.warp[lane] : 0, lane < kWarps ? sh.warp2[lane] : 0, b.start, b.left);
    const int run = pick(b, goal), begin = run * length, end = min(padded, begin + length);
    const int part = ((end - begin + kThreads - 1) / kThreads + 7) / 8 * 8, mine = begin + tid * part;
    uint64_t of_part = 0;
    uint32_t ties_of_part = 0;
    for (int i = mine; i < min(end, mine + part); i += E::kPer) weigh_chunk(chunk(i), of_part, ties_of_part);
    mass = warp_reduce(of_part, add<uint64_t>);
    ties = __reduce_add_sync(~0u, ties_of_part);
    __syncthreads();
    if (lane == 0) {
        sh.warp[warp] = mass;
        sh.warp2[warp] = ties;
    }
    __syncthreads();
    b = line_up(lane < kWarps ? sh.warp[lane] : 0, lane < kWarps ? sh.warp2[lane] : 0, b.start, b.left);
    if (pick(b, goal) != warp) return;
    b = line_up(of_part, ties_of_part, b.start, b.left);
    const int from_here = begin + (warp * 32 + pick(b, goal)) * part, to_here = min(end, from_here + part);
    for (int i0 = from_here; i0 < to_here; i0 += 32) {
        const int i = i0 + lane;
        const float x = i < to_here ? at(i) : -INFINITY;
        const bool tied = cut.ties && x == cut.at;
        Before c = line_up(!tied && x >= lowest ? w.of(x) : 0, tied, b.start, b.left);
        const uint32_t over = __ballot_sync(~0u, c.start + c.mass > goal);
        if (over) {
            if (lane == __ffs(over) - 1) {
                a.ids[row] = first + i;
                if (a.prob) a.prob[row] = w.share(x, whole);
            }
            return;
        }
        b.start = __shfl_sync(~0u, c.start + c.mass, 31);
        b.left = __shfl_sync(~0u, c.left - min(c.left, static_cast<uint32_t>(tied)), 31);
    }
}

bool at(const void* p, size_t a) { return p && reinterpret_cast<uintptr_t>(p) % a == 0; }

template <int kElem, bool kCuts>
cudaError_t launch(const Sample& s, int B, int ctas, cudaStream_t stream) {
    const size_t smem = (sizeof(Shared) + 15) / 16 * 16 + (kCuts ? static_cast<size_t>(s.slice) * Elem<kElem>::kBytes : 0);
    const auto kernel = k_sample<kElem, kCuts>;
    cudaError_t rc = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (rc != cudaSuccess) return rc;
    cudaLaunchAttribute attr[2] = {overlapped(), {}};
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(B) * ctas);
    cfg.blockDim = dim3(kThreadsOf<kCuts>);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, s);
}
template <int kElem>
cudaError_t launch(const Sample& s, bool cuts, int B, int ctas, cudaStream_t stream) {
    return cuts ? launch<kElem, true>(s, B, ctas, stream) : launch<kElem, false>(s, B, ctas, stream);
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
    const bool cuts = top_k_rows || top_p_rows || (top_k > 0 && top_k < V) || !(top_p >= 1.0f);
    // as many CTAs a row as keep the device busy, of 2048 logits at least, and with cuts as many as hold the row in 96 KB
    // each (256 rows of 151936: bf16 with top-p 0.9, 4 CTAs a row 294 us, 8 366; fp32 with min-p, in two waves of which one
    // reads while the other meets, 4 CTAs 42 us, 2 53, 8 51)
    int ctas = 1, sms = 0;
    if (sm_count(&sms) != cudaSuccess) return ESTREAM_ERR_CUDA;
    while (ctas < kMaxCtas && ((cuts && V * static_cast<long long>(size) > ctas * 98304ll) ||
                               (B * ctas < (cuts ? sms : 4 * sms) && V > ctas * 2048)))
        ctas *= 2;
    const Sample s{logits, ld, V, ((V + ctas - 1) / ctas + 7) / 8 * 8, u, temperature, top_p, min_p, top_k,
                   temperature_rows, top_p_rows, min_p_rows, top_k_rows, ids, prob};
    const cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
    const cudaError_t rc = elem == ESTREAM_MX4_BF16  ? launch<ESTREAM_MX4_BF16>(s, cuts, B, ctas, stream)
                           : elem == ESTREAM_MX4_F16 ? launch<ESTREAM_MX4_F16>(s, cuts, B, ctas, stream)
                                                     : launch<ESTREAM_MX4_F32>(s, cuts, B, ctas, stream);
    return rc == cudaSuccess ? ESTREAM_OK : ESTREAM_ERR_CUDA;
}
