// Attention of one new token per sequence over a paged key-value cache.
//
// With z_i = scale (q . k_i): out = sum_i e^{z_i - m} v_i / l, l = sum_i e^{z_i - m}, m = max z.
// (m, l, sum) of two sets of positions join as
//   m = max(m1, m2), l = l1 e^{m1 - m} + l2 e^{m2 - m}, the sums alike,
// so a sequence may be cut anywhere. Exponents are held in base 2, and m is the next whole number from the
// largest on: it loses nothing when it is subtracted from a score, when sums by two of them are joined, or when lse is
// formed, and a unit's sums are rescaled by powers of two.
//
// The work is all (row, key head) units' blocks of 16 or 32 positions, one unit behind
// another; every warp takes an equal, contiguous share of them, found from the
// lengths on the device (so a captured graph keeps its balance as sequences grow), with
// a ring of its own that cp.async fills ahead over units' ends. A unit that lies in one
// share is finished there; the pieces of others go through the workspace to a
// second kernel. With shares of CTAs, whose warps took turns at the blocks and met
// at a unit's end, a batch with many short sequences waited for its slowest CTA
// twice as long as the average one took.
//
// Where all units fit on the device with a cluster of CTAs each and the table allows no
// long sequence, a unit is split over its cluster's warps instead, whose pieces meet
// through distributed shared memory: one launch, no workspace.
//
// The matrix instructions take keys and transposed values as their 16 rows and the query heads of
// a key head as their 8 columns (a wider group of heads: two tiles of 8, and units of 16),
// so a group of 8 heads or fewer wastes no row: with the heads as rows, it took twice the
// instructions and registers (64 ragged sequences over E4M3 243 us instead of 208).
//
// Bound by HBM: 131072 positions of 8 heads of 128 bf16 in 82 us (6.5 TB/s, 96% of the copy rate) and
// 5 us of joining; 64 ragged sequences up to 16384 in E4M3 124 us (5.9 TB/s), 32 in fp16 60 us (6.2).
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>

#include "estream_internal.h"
#include "overlap.cuh"

namespace es {
namespace {
namespace cg = cooperative_groups;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kGroup = 16;  // positions that lie in one page together where page_size is a multiple of it
constexpr int kRows = 16;   // query heads that meet a key together, at most
// What a unit costs a warp beside its blocks (queries, results), in blocks: without it the warps with the short
// sequences of a ragged batch end last (140 us instead of 134, 64 sequences over E4M3).
constexpr int kOver = 1;

struct Attend {
    const void* q;
    void* out;
    float* lse;
    const uint8_t *k, *v;
    const int32_t *table, *lens;
    float *part, *ml;  // workspace: pieces' sums [2 warps][rows][kDim], and their (m, l) [2 warps][rows][2]
    int2* pieces;      // [B * heads * tiles]: the warp with a unit's first piece, and how many further pieces there are
    long long q_row, q_head, out_row, out_head, table_row;
    long long k_page, k_token, k_head, v_page, v_token, v_head;  // bytes
    float scale, v_scale;  // scale * k_scale * log2 e
    float back, back_low;  // what a score in base 2 is worth: (scale * k_scale) / Attend::scale in two floats, which undoes its rounding
    int B, Hq, heads, group, tiles, rows, dim, chunks, M, max_len, num_pages, window;
    int ctas;  // of the cluster that has a unit to itself; 0: shares of all units
    int out_f16, q_words;  // type of q and out; q rows lie on 4 bytes
    FastDiv page;
};

// What differs by the cache's type (ESTREAM_KV_*) and the padded width.
template <int kElem, int kDim>
struct Shape {
    static constexpr bool kBytes = kElem == ESTREAM_KV_E4M3;
    static constexpr bool kBf16 = kElem == ESTREAM_KV_BF16;  // the matrix instructions' type; else fp16
    static constexpr int kRowBytes = kDim * (kBytes ? 1 : 2);
    static constexpr int kBlock = kRowBytes <= 128 ? 32 : 16;  // positions a warp takes at a time
    static constexpr int kStageBytes = 2 * kBlock * kRowBytes;  // keys, then values
    static constexpr int kStages = kRowBytes == 64 ? 6 : 3;
    static constexpr int kSmem = kWarps * kStages * kStageBytes;
    static constexpr int kResident = std::min(4, 228 * 1024 / (kSmem + 1024 + 128));  // 1 KB a CTA is the system's
    // fp16 weights are 2^14 times as large as the formula's: their smallest normal
    // value is then 2^-28 of the largest weight, not 2^-14
    static constexpr float kBias = kBf16 ? 0.0f : 14.0f;
    static constexpr float kUnit = kBf16 ? 1.0f : 0x1p-14f;  // 2^-kBias
};

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float finite_or_zero(float m) { return m == -INFINITY ? 0.0f : m; }

__device__ __forceinline__ void ldmatrix(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldmatrix_trans(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
template <bool kBf16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (kBf16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 16 bytes to shared memory, zeros when !there (then `from` is not read).
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}
// Four E4M3 values as fp16, exactly: the lower two, and the upper two.
__device__ __forceinline__ void from_e4m3(uint32_t four, uint32_t& low, uint32_t& high) {
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h;}"
        : "=r"(low), "=r"(high) : "r"(four));
}
template <bool kBf16>
__device__ __forceinline__ uint32_t pack(float x, float y) {
    if constexpr (kBf16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __half2 h = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}
template <bool kBf16>
__device__ __forceinline__ float2 unpack(uint32_t w) {
    if constexpr (kBf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    else return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
// Where 16-byte chunk c of row r lies in a tile: eight rows' chunks of one c are on
// different banks.
template <int kRowBytes>
__device__ __forceinline__ uint32_t in_tile(int r, int c) {
    const int x = kRowBytes == 64 ? (r >> 1) & 3 : r & 7;
    return r * kRowBytes + ((c ^ x) << 4);
}

__device__ __forceinline__ uint32_t transpose(uint32_t x) {  // 8 x 8 values of 16 bits
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// A row's attended positions [lo, len) and its blocks, which begin at a multiple of 16.
struct Span {
    int len, lo, first, blocks;
};
template <int kBlock>
__device__ __forceinline__ Span span_of(const Attend& a, int b) {
    Span s;
    s.len = a.lens[b];
    s.lo = a.window > 0 && s.len > a.window ? s.len - a.window : 0;
    s.first = s.lo & ~(kGroup - 1);
    s.blocks = s.len > 0 && s.len <= a.max_len ? (s.len - s.first + kBlock - 1) / kBlock : 0;
    return s;
}

// A unit: row, key head and tile of 16 query heads. Shares are cut from all units' costs,
// one unit's kOver + blocks behind the other's.
struct Unit {
    int b, head;  // head = key head * tiles + tile
    Span span;
    long long start;  // its cost's beginning
    __device__ __forceinline__ long long cost() const { return span.blocks + kOver; }
    // Its blocks [from, to) of a share [begin, end).
    __device__ __forceinline__ int from(long long begin) const {
        return static_cast<int>(max(0ll, begin - start - kOver));
    }
    __device__ __forceinline__ int to(long long end) const {
        return static_cast<int>(min(static_cast<long long>(span.blocks), end - start - kOver));
    }
    // To the next unit with blocks in the share; false: there is none.
    template <int kBlock>
    __device__ __forceinline__ bool next(const Attend& a, long long end) {
        start += cost();
        if (start + kOver >= end) return false;
        if (++head == a.heads * a.tiles) {
            head = 0;
            do span = span_of<kBlock>(a, ++b);
            while (span.blocks == 0);
        }
        return true;
    }
};

// What a row's (m, l, sum) gives: the factor of its sums, and lse; unit: what a weight of 1 is worth.
struct Finish {
    float by, lse;
};
__device__ __forceinline__ Finish finish(const Attend& a, float m, float l, float unit) {
    if (l == 0.0f) return {0.0f, -INFINITY};
    return {l > 0.0f ? a.v_scale / l : NAN, fmaf(m, a.back, fmaf(m, a.back_low, log2f(l * unit) * 0.69314718055994531f))};
}
// One value of the result; sums of nothing may be anything.
__device__ __forceinline__ void put(const Attend& a, int b, int h, int d, float sum, const Finish& f) {
    if (d >= a.dim) return;
    const float y = f.by == 0.0f ? 0.0f : sum * f.by;
    static_cast<uint16_t*>(a.out)[b * a.out_row + h * a.out_head + d] =
        a.out_f16 ? __half_as_ushort(__float2half_rn(y)) : __bfloat16_as_ushort(__float2bfloat16_rn(y));
}
__device__ __forceinline__ void put_lse(const Attend& a, int b, int h, const Finish& f) {
    if (a.lse) a.lse[static_cast<long long>(b) * a.Hq + h] = f.lse;
}

// kTiles: tiles of 8 query heads (2 only where a group has more than 8). kWhole: page_size is a
// multiple of 16, so 16 positions from a multiple of 16 on lie in one page.
template <int kElem, int kDim, int kTiles, bool kWhole>
__global__ void __launch_bounds__(kThreads, Shape<kElem, kDim>::kResident) k_kv_attend(const Attend a) {
    using S = Shape<kElem, kDim>;
    constexpr int kSteps = kDim / 16, kBlock = S::kBlock;
    constexpr int kChunks = S::kRowBytes / 16;                 // of a padded row
    constexpr int kPerCopy = kChunks < 32 ? 32 / kChunks : 1;  // rows that a warp's copy covers
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long scan[kWarps];
    __shared__ Unit first_unit[kWarps];
    __shared__ float2 stats[kWarps][kRows];  // of a cluster's unit: the warps' (m, l)
    after_previous();
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t = lane % 4;
    const int units = a.heads * a.tiles;  // of a row

    const int worker = blockIdx.x * kWarps + warp;
    Unit u;
    long long begin, end, share = 0;
    if (a.ctas) {
        const int id = blockIdx.x / a.ctas;
        u.b = id / units;
        u.head = id % units;
        u.start = 0;
        u.span = span_of<kBlock>(a, u.b);
        const int workers = a.ctas * kWarps, mine = worker % workers, each = (u.span.blocks + workers - 1) / workers;
        begin = kOver + mine * each;
        end = min(kOver + u.span.blocks, static_cast<int>(begin) + each);
        if (u.span.blocks == 0) {  // nothing to attend: zeros, or NaN where the length is out of range
            const Finish f = finish(a, 0.0f, u.span.len == 0 ? 0.0f : NAN, 1.0f);
            const int h0 = u.head / a.tiles * a.group + u.head % a.tiles * kRows;
            const int rows = min(kRows, a.group - u.head % a.tiles * kRows);
            for (int i = mine / kWarps * kThreads + tid; i < rows * kDim; i += a.ctas * kThreads) {
                put(a, u.b, h0 + i / kDim, i % kDim, 1.0f, f);
                if (i % kDim == 0) put_lse(a, u.b, h0 + i / kDim, f);
            }
            return;
        }
    } else {
        // Rows with nothing to attend: zeros, or NaN where the length is out of range.
        for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
            const Span s = span_of<kBlock>(a, b);
            if (s.blocks) continue;
            for (int i = tid; i < units; i += kThreads) a.pieces[static_cast<long long>(b) * units + i] = make_int2(0, 0);
            const Finish f = finish(a, 0.0f, s.len == 0 ? 0.0f : NAN, 1.0f);
            for (int i = tid; i < a.Hq * a.dim; i += kThreads) {
                const int h = i / a.dim, d = i - h * a.dim;
                put(a, b, h, d, 1.0f, f);
                if (d == 0) put_lse(a, b, h, f);
            }
        }

        // This warp's share, and the unit it begins in.
        const int per_thread = (a.B + kThreads - 1) / kThreads, mine = tid * per_thread, past = min(a.B, mine + per_thread);
        auto cost_of = [&](int b) {
            const int n = span_of<kBlock>(a, b).blocks;
            return n ? n + kOver : 0;
        };
        long long count = 0;
        for (int b = mine; b < past; ++b) count += cost_of(b);
        long long upto = count;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(~0u, upto, o);
            if (lane >= o) upto += v;
        }
        if (lane == 31) scan[warp] = upto;
        __syncthreads();
        long long total = 0, before = 0;
        for (int w = 0; w < kWarps; ++w) {
            if (w == warp) before = total;
            total += scan[w];
        }
        total *= units;
        before = (before + upto - count) * units;
        const int workers = gridDim.x * kWarps;
        share = (total + workers - 1) / workers;
        for (int w = 0; w < kWarps; ++w) {
            const long long begin = (blockIdx.x * kWarps + w) * share;
            if (begin < before || begin >= before + count * units) continue;
            Unit u;
            u.b = mine;
            u.start = before;
            for (;; ++u.b) {
                const long long n = static_cast<long long>(cost_of(u.b)) * units;
                if (begin < u.start + n) break;
                u.start += n;
            }
            u.span = span_of<kBlock>(a, u.b);
            u.head = static_cast<int>((begin - u.start) / u.cost());
            u.start += u.head * u.cost();
            first_unit[w] = u;
        }
        __syncthreads();
        begin = worker * share;
        end = min(total, begin + share);
        if (begin >= end) return;
        u = first_unit[warp];
        if (u.from(begin) >= u.to(end) && !u.template next<kBlock>(a, end)) return;
    }

    // The warp's loads run ahead of its products, over units' ends.
    Unit ahead = u;
    int next = ahead.from(begin), stop = ahead.to(end);  // of the unit's blocks
    bool more = next < stop;
    // The page (-1: not attended, -2: out of range) and the place in it of the next block's
    // position lane % kBlock, or where a page holds whole groups, of its group's first one.
    int page = -1, slot = 0;
    auto look_up = [&] {
        int at = ahead.span.first + next * kBlock + lane % kBlock;
        if constexpr (kWhole) at &= ~(kGroup - 1);
        page = -1;
        const int entry = static_cast<int>(a.page.div(at));
        slot = at - entry * static_cast<int>(a.page.d);
        if (at < ahead.span.len && (kWhole || at >= ahead.span.lo)) {
            page = a.table[ahead.b * a.table_row + entry];
            if (page < 0 || page >= a.num_pages) page = -2;
        }
    };
    const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + warp * S::kStages * S::kStageBytes;
    const int my_chunk = lane % kChunks, my_row = lane / kChunks;
    uint32_t bad = 0;  // by stage: a page out of range
    auto issue = [&](int stage) {
        if (more) {
            const uint32_t to = ring + stage * S::kStageBytes;
            const int h = ahead.head / a.tiles;
            const uint8_t* kb = a.k + h * a.k_head + my_chunk * 16;
            const uint8_t* vb = a.v + h * a.v_head + my_chunk * 16;
            const bool in = my_chunk < a.chunks;
            bad = (bad & ~(1u << stage)) | (__any_sync(~0u, page == -2) ? 1u << stage : 0u);
            if constexpr (kWhole) {
                const int at = ahead.span.first + next * kBlock;
                const uint8_t *kf[kBlock / kGroup], *vf[kBlock / kGroup];
                bool there[kBlock / kGroup];
#pragma unroll
                for (int j = 0; j < kBlock / kGroup; ++j) {
                    const int p = __shfl_sync(~0u, page, j * kGroup), s = __shfl_sync(~0u, slot, j * kGroup) + my_row;
                    there[j] = in && p >= 0;
                    kf[j] = kb + max(p, 0) * a.k_page + s * a.k_token;
                    vf[j] = vb + max(p, 0) * a.v_page + s * a.v_token;
                }
                const long long k_step = kPerCopy * a.k_token, v_step = kPerCopy * a.v_token;
                if (at >= ahead.span.lo && at + kBlock <= ahead.span.len) {  // all rows are attended
#pragma unroll
                    for (int j = 0; j < kBlock / kGroup; ++j)
#pragma unroll
                        for (int i = 0; i < kGroup / kPerCopy; ++i) {
                            const int r = j * kGroup + i * kPerCopy + my_row;
                            copy16(to + in_tile<S::kRowBytes>(r, my_chunk), kf[j], there[j]);
                            copy16(to + kBlock * S::kRowBytes + in_tile<S::kRowBytes>(r, my_chunk), vf[j], there[j]);
                            kf[j] += k_step;
                            vf[j] += v_step;
                        }
                } else {
                    const int lo = ahead.span.lo - at, len = ahead.span.len - at;
#pragma unroll
                    for (int j = 0; j < kBlock / kGroup; ++j)
#pragma unroll
                        for (int i = 0; i < kGroup / kPerCopy; ++i) {
                            const int r = j * kGroup + i * kPerCopy + my_row;
                            const bool one = there[j] && r >= lo && r < len;
                            copy16(to + in_tile<S::kRowBytes>(r, my_chunk), kf[j], one);
                            copy16(to + kBlock * S::kRowBytes + in_tile<S::kRowBytes>(r, my_chunk), vf[j], one);
                            kf[j] += k_step;
                            vf[j] += v_step;
                        }
                }
            } else {
#pragma unroll
                for (int i = 0; i < kBlock / kPerCopy; ++i) {
                    const int r = i * kPerCopy + my_row;
                    const int p = __shfl_sync(~0u, page, r), s = __shfl_sync(~0u, slot, r);
                    const bool there = in && p >= 0;
                    const uint8_t* kf = kb + max(p, 0) * a.k_page + s * a.k_token;
                    const uint8_t* vf = vb + max(p, 0) * a.v_page + s * a.v_token;
                    copy16(to + in_tile<S::kRowBytes>(r, my_chunk), kf, there);
                    copy16(to + kBlock * S::kRowBytes + in_tile<S::kRowBytes>(r, my_chunk), vf, there);
                }
            }
            if (++next == stop) {
                more = ahead.template next<kBlock>(a, end);
                next = 0;
                stop = ahead.to(end);
            }
            if (more) look_up();
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    if (more) look_up();
#pragma unroll
    for (int s = 0; s < S::kStages - 1; ++s) issue(s);

    int stage = 0;
    for (;;) {
        const int from = u.from(begin), to = u.to(end);
        const int kv_head = u.head / a.tiles, row0 = u.head % a.tiles * kRows;  // first query head of this unit in its group
        const int rows = min(kRows, a.group - row0);
        // Of heads 2t and 2t + 1 of each tile: the maximum, rounded up (the same in all lanes of one t), this
        // lane's part of the sum of weights, and of the values' dims g and g + 8 of each 16 (E4M3: 2g, 2g + 1).
        float m[kTiles][2], base[kTiles][2], l[kTiles][2], o[kTiles][kSteps][4];  // base: finite m, less the bias
#pragma unroll
        for (int j = 0; j < kTiles; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[j][i] = -INFINITY;
                base[j][i] = -S::kBias;
                l[j][i] = 0.0f;
#pragma unroll
                for (int s = 0; s < kSteps; ++s) o[j][s][i] = o[j][s][i + 2] = 0.0f;
            }
        bool poison = false;
        if (from < to) {
            // Query fragments. An E4M3 key's four neighbouring values lie in one lane, so pairs
            // (2t, 2t + 1) and (2t + 8, 2t + 9) of the product are values (4t, 4t + 1) and (4t + 2, 4t + 3).
            uint32_t qb[kTiles][kSteps][2];
            float c[kTiles][2];  // scale of heads 2t and 2t + 1
#pragma unroll
            for (int j = 0; j < kTiles; ++j) {
                const int h = 8 * j + g;
                const uint16_t* qr = static_cast<const uint16_t*>(a.q) + u.b * a.q_row +
                                     static_cast<long long>(kv_head * a.group + row0 + min(h, rows - 1)) * a.q_head;
#pragma unroll
                for (int s = 0; s < kSteps; ++s)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int d = 16 * s + (S::kBytes ? 4 * t + 2 * i : 2 * t + 8 * i);
                        uint32_t w = 0;
                        if (d < a.dim && h < rows)
                            w = a.q_words ? *reinterpret_cast<const uint32_t*>(qr + d)
                                          : qr[d] | static_cast<uint32_t>(qr[d + 1]) << 16;
                        qb[j][s][i] = w;
                    }
                c[j][0] = c[j][1] = a.scale;
                if constexpr (S::kBytes) {
                    // to fp16, by the power of two that puts the head's largest at 2^10 to 2^11
                    auto wide = [&](uint32_t w) {
                        return a.out_f16 ? __half22float2(*reinterpret_cast<__half2*>(&w))
                                         : __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&w));
                    };
                    float top = 0.0f;
#pragma unroll
                    for (int s = 0; s < kSteps; ++s)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float2 f = wide(qb[j][s][i]);
                            top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                        }
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
                    const int e = min(126, max(-126, 137 - static_cast<int>(__float_as_uint(top) >> 23)));
                    const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
                    for (int s = 0; s < kSteps; ++s)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float2 f = wide(qb[j][s][i]);
                            qb[j][s][i] = pack<false>(f.x * up, f.y * up);
                        }
                    const float down = a.scale * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // head g's
                    c[j][0] = __shfl_sync(~0u, down, 8 * t);
                    c[j][1] = __shfl_sync(~0u, down, 8 * t + 4);
                }
            }
            for (int at = u.span.first + from * kBlock, past = u.span.first + to * kBlock; at < past; at += kBlock) {
                asm volatile("cp.async.wait_group %0;" ::"n"(S::kStages - 2) : "memory");
                __syncwarp();  // every lane's copies are there, and every lane has read the stage that is filled next
                issue(stage == 0 ? S::kStages - 1 : stage - 1);
                const uint32_t kt = ring + stage * S::kStageBytes, vt = kt + kBlock * S::kRowBytes;
                poison |= bad >> stage & 1;
                stage = stage + 1 == S::kStages ? 0 : stage + 1;
                const bool edge = at < u.span.lo || at + kBlock > u.span.len;
#pragma unroll
                for (int half = 0; half < kBlock / 16; ++half) {
                    // z: positions g and g + 8 of heads 2t and 2t + 1
                    float z[kTiles][4];
#pragma unroll
                    for (int j = 0; j < kTiles; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) z[j][i] = 0.0f;
                    const int row = 16 * half + (lane & 15), side = lane >> 4;
                    if constexpr (S::kBytes) {
#pragma unroll
                        for (int s = 0; s < kSteps; s += 2) {
                            uint32_t r[4];
                            ldmatrix(r, kt + in_tile<S::kRowBytes>(row, s + side));
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                uint32_t f[4];
                                from_e4m3(r[2 * i], f[0], f[2]);
                                from_e4m3(r[2 * i + 1], f[1], f[3]);
#pragma unroll
                                for (int j = 0; j < kTiles; ++j) mma<false>(z[j], f, qb[j][s + i][0], qb[j][s + i][1]);
                            }
                        }
                    } else {
#pragma unroll
                        for (int s = 0; s < kSteps; ++s) {
                            uint32_t r[4];
                            ldmatrix(r, kt + in_tile<S::kRowBytes>(row, 2 * s + side));
#pragma unroll
                            for (int j = 0; j < kTiles; ++j) mma<S::kBf16>(z[j], r, qb[j][s][0], qb[j][s][1]);
                        }
                    }
                    bool above = false;
#pragma unroll
                    for (int j = 0; j < kTiles; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float x = z[j][i] * c[j][i & 1];
                            if (edge) {
                                const int p = at + 16 * half + g + (i & 2) * 4;
                                if (p < u.span.lo || p >= u.span.len) x = -INFINITY;
                            }
                            z[j][i] = x;
                            above |= x > m[j][i & 1];
                        }
                    if (__any_sync(~0u, above)) {  // seldom, after the first blocks
#pragma unroll
                        for (int j = 0; j < kTiles; ++j)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                float top = fmaxf(z[j][i], z[j][i + 2]);
#pragma unroll
                                for (int x = 4; x < 32; x *= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, x));
                                const float now = fmaxf(m[j][i], ceilf(top)), shrink = exp2_fast(m[j][i] - finite_or_zero(now));
                                m[j][i] = now;
                                base[j][i] = finite_or_zero(now) - S::kBias;
                                l[j][i] *= shrink;
#pragma unroll
                                for (int s = 0; s < kSteps; ++s) {
                                    o[j][s][i] *= shrink;
                                    o[j][s][i + 2] *= shrink;
                                }
                            }
                    }
                    // A weight enters the products as two terms, what the type holds of it and what that leaves: 16 bits for
                    // bf16, 22 for fp16. With one fp16 term results were 2 to 6% less exact (2.20e-4 of the norm instead of
                    // 2.07e-4, fp16 pages) for at most 1% of the time, next to 8-bit pages for 1 to 4%.
                    uint32_t hi[kTiles][2], lo[kTiles][2];
#pragma unroll
                    for (int j = 0; j < kTiles; ++j)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {  // positions g, then g + 8
                            const float x = exp2_fast(z[j][2 * i] - base[j][0]);
                            const float y = exp2_fast(z[j][2 * i + 1] - base[j][1]);
                            l[j][0] += x;
                            l[j][1] += y;
                            const uint32_t w = pack<S::kBf16>(x, y);
                            hi[j][i] = transpose(w);
                            const float2 first = unpack<S::kBf16>(w);
                            lo[j][i] = transpose(pack<S::kBf16>(x - first.x, y - first.y));
                        }
                    if constexpr (S::kBytes) {
#pragma unroll
                        for (int s = 0; s < kSteps; s += 2) {
                            uint32_t r[4];
                            ldmatrix_trans(r, vt + in_tile<S::kRowBytes>(row, s + side));
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                // values (2g, 2g + 1) of positions 2t and 2t + 1: to pairs of positions
                                uint32_t f[4];
                                from_e4m3(__byte_perm(r[2 * i], 0, 0x3120), f[0], f[1]);
                                from_e4m3(__byte_perm(r[2 * i + 1], 0, 0x3120), f[2], f[3]);
#pragma unroll
                                for (int j = 0; j < kTiles; ++j) {
                                    mma<false>(o[j][s + i], f, hi[j][0], hi[j][1]);
                                    mma<false>(o[j][s + i], f, lo[j][0], lo[j][1]);
                                }
                            }
                        }
                    } else {
                        const int vrow = 16 * half + (lane & 7) + (lane >> 4) * 8, vside = lane >> 3 & 1;
#pragma unroll
                        for (int s = 0; s < kSteps; ++s) {
                            uint32_t r[4];
                            ldmatrix_trans(r, vt + in_tile<S::kRowBytes>(vrow, 2 * s + vside));
#pragma unroll
                            for (int j = 0; j < kTiles; ++j) {
                                mma<S::kBf16>(o[j][s], r, hi[j][0], hi[j][1]);
                                mma<S::kBf16>(o[j][s], r, lo[j][0], lo[j][1]);
                            }
                        }
                    }
                }
            }
        }
        // The unit's result, or this piece of it.
        if (a.ctas) {  // the cluster's pieces meet
            cg::cluster_group cluster = cg::this_cluster();
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncwarp();
            float* const mine = reinterpret_cast<float*>(smem + warp * S::kStages * S::kStageBytes);  // the warp's ring, as [kRows][kDim]
#pragma unroll
            for (int j = 0; j < kTiles; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
#pragma unroll
                    for (int x = 4; x < 32; x *= 2) l[j][i] += __shfl_xor_sync(~0u, l[j][i], x);
                    const int row = 8 * j + 2 * t + i;
                    if (g == 0) stats[warp][row] = make_float2(m[j][i], poison ? NAN : l[j][i]);
                    if (row >= rows) continue;
#pragma unroll
                    for (int s = 0; s < kSteps; ++s) {
                        const int d = 16 * s + (S::kBytes ? 2 * g : g);
                        mine[row * kDim + d] = o[j][s][i];
                        mine[row * kDim + d + (S::kBytes ? 1 : 8)] = o[j][s][i + 2];
                    }
                }
            cluster.sync();
            const int rank = static_cast<int>(cluster.block_rank());
            for (int e = rank * kThreads + tid; e < rows * kDim; e += a.ctas * kThreads) {
                const int row = e / kDim, d = e % kDim;
                float top = -INFINITY, sum = 0.0f, weight = 0.0f;
                for (int r = 0; r < a.ctas; ++r) {
                    const float2* theirs = cluster.map_shared_rank(&stats[0][0], r);
                    const float* sums = reinterpret_cast<const float*>(cluster.map_shared_rank(smem, r)) + e;
                    float2 s[kWarps];
                    float x[kWarps];
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        s[w] = theirs[w * kRows + row];
                        x[w] = sums[w * (S::kStages * S::kStageBytes / 4)];
                    }
                    float now = top;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) now = fmaxf(now, s[w].x);
                    const float at = finite_or_zero(now), shrink = exp2_fast(top - at);
                    top = now;
                    sum *= shrink;
                    weight *= shrink;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        const float f = exp2_fast(s[w].x - at);
                        sum += f * x[w];
                        weight += f * s[w].y;
                    }
                }
                const Finish f = finish(a, top, weight, S::kUnit);
                const int h = kv_head * a.group + row0 + row;
                put(a, u.b, h, d, sum, f);
                if (d == 0) put_lse(a, u.b, h, f);
            }
            cluster.sync();  // nobody leaves while others read its piece
            return;
        }
        const bool whole = from == 0 && to == u.span.blocks;
        const long long piece = 2ll * worker + (from == 0);
#pragma unroll
        for (int j = 0; j < kTiles; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int x = 4; x < 32; x *= 2) l[j][i] += __shfl_xor_sync(~0u, l[j][i], x);
                if (poison) l[j][i] = NAN;
                const int row = 8 * j + 2 * t + i;
                if (row >= rows) continue;
                const int h = kv_head * a.group + row0 + row;
                if (whole) {
                    const Finish f = finish(a, m[j][i], l[j][i], S::kUnit);
#pragma unroll
                    for (int s = 0; s < kSteps; ++s) {
                        const int d = 16 * s + (S::kBytes ? 2 * g : g);
                        put(a, u.b, h, d, o[j][s][i], f);
                        put(a, u.b, h, d + (S::kBytes ? 1 : 8), o[j][s][i + 2], f);
                    }
                    if (g == 0) put_lse(a, u.b, h, f);
                } else {
                    float* to = a.part + (piece * a.rows + row) * kDim;
#pragma unroll
                    for (int s = 0; s < kSteps; ++s) {
                        const int d = 16 * s + (S::kBytes ? 2 * g : g);
                        to[d] = o[j][s][i];
                        to[d + (S::kBytes ? 1 : 8)] = o[j][s][i + 2];
                    }
                    if (g == 0) reinterpret_cast<float2*>(a.ml)[piece * a.rows + row] = make_float2(m[j][i], l[j][i]);
                }
            }
        if (from == 0 && lane == 0)
            a.pieces[static_cast<long long>(u.b) * units + u.head] =
                make_int2(worker, static_cast<int>((u.start + kOver + u.span.blocks - 1) / share) - worker);
        if (!u.template next<kBlock>(a, end)) break;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// The results of units in pieces: the first piece of one warp's share, then the leading pieces
// of those that follow. An item is a unit's query head; a warp joins one of few pieces, a
// block one of many (or, where items are few, any): 8 pieces a warp are under way at a time.
// Neighbouring items, of one unit, go to different blocks.
constexpr int kJoinWarps = 16;
constexpr int kAtOnce = 8;
template <int kDim>
struct Joined {
    static constexpr int kPer = kDim / 32;  // columns a lane, beside each other
    float m = -INFINITY, l = 0.0f, sum[kPer] = {};
    __device__ __forceinline__ void add(const Attend& a, int worker, int row, int lane, int first, int last, int step) {
        const float2* ml = reinterpret_cast<const float2*>(a.ml);
        for (int i0 = first; i0 <= last; i0 += kAtOnce * step) {
            float2 s[kAtOnce];
            float x[kAtOnce][kPer];
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const int i = i0 + j * step;
                s[j] = make_float2(-INFINITY, 0.0f);
#pragma unroll
                for (int c = 0; c < kPer; ++c) x[j][c] = 0.0f;
                if (i <= last) {
                    const long long at = (2ll * (worker + i) + (i == 0)) * a.rows + row;  // piece i's row
                    s[j] = ml[at];
                    const float* from = a.part + at * kDim + lane * kPer;
                    if constexpr (kPer == 2) {
                        *reinterpret_cast<float2*>(x[j]) = *reinterpret_cast<const float2*>(from);
                    } else {
#pragma unroll
                        for (int c = 0; c < kPer; c += 4)
                            *reinterpret_cast<float4*>(x[j] + c) = *reinterpret_cast<const float4*>(from + c);
                    }
                }
            }
            float now = m;
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) now = fmaxf(now, s[j].x);
            const float base = finite_or_zero(now), shrink = exp2_fast(m - base);
            m = now;
            l *= shrink;
#pragma unroll
            for (int c = 0; c < kPer; ++c) sum[c] *= shrink;
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const float f = exp2_fast(s[j].x - base);
                l += f * s[j].y;
#pragma unroll
                for (int c = 0; c < kPer; ++c) sum[c] += f * x[j][c];
            }
        }
    }
};
template <int kDim>
__global__ void __launch_bounds__(32 * kJoinWarps) k_kv_join(const Attend a, float unit, int items, int per_block) {
    using J = Joined<kDim>;
    __shared__ float sums[kJoinWarps][kDim];
    __shared__ float2 stats[kJoinWarps];
    __shared__ bool many[kJoinWarps];
    after_previous();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int units = a.heads * a.tiles, rows = a.rows;
    // item i of this block: row, query head, that head's place in its unit, and the pieces; false: it has none, or one
    auto item = [&](int i, int& b, int& h, int& row, int2& pieces) {
        const int it = i * gridDim.x + blockIdx.x;
        if (i >= per_block || it >= items) return false;
        const int unit = it / rows, head = unit % units, row0 = head % a.tiles * kRows;
        row = it % rows;
        if (row0 + row >= a.group) return false;
        pieces = a.pieces[unit];
        b = unit / units;
        h = head / a.tiles * a.group + row0 + row;
        return pieces.y > 0;
    };
    int b, h, row;
    int2 pieces = {};
    uint32_t left = 1;  // items that the block joins
    if (per_block > 1) {
        const bool any = item(warp, b, h, row, pieces), few = pieces.y < 4 * kAtOnce;
        if (any && few) {
            J r;
            r.add(a, pieces.x, row, lane, 0, pieces.y, 1);
            const Finish f = finish(a, r.m, r.l, unit);
#pragma unroll
            for (int c = 0; c < J::kPer; ++c) put(a, b, h, lane * J::kPer + c, r.sum[c], f);
            if (lane == 0) put_lse(a, b, h, f);
        }
        if (lane == 0) many[warp] = any && !few;
        __syncthreads();
        left = __ballot_sync(~0u, lane < kJoinWarps && many[lane]);
    }
    for (; left; left &= left - 1) {
        if (!item(__ffs(left) - 1, b, h, row, pieces)) return;
        J r;
        r.add(a, pieces.x, row, lane, warp, pieces.y, kJoinWarps);
        __syncthreads();  // all have read those before
#pragma unroll
        for (int c = 0; c < J::kPer; ++c) sums[warp][lane * J::kPer + c] = r.sum[c];
        if (lane == 0) stats[warp] = make_float2(r.m, r.l);
        __syncthreads();
        const int d = threadIdx.x;
        if (d >= kDim) continue;
        float m = -INFINITY, l = 0.0f, sum = 0.0f;
        for (int w = 0; w < kJoinWarps; ++w) m = fmaxf(m, stats[w].x);
        const float base = finite_or_zero(m);
        for (int w = 0; w < kJoinWarps; ++w) {
            const float f = exp2_fast(stats[w].x - base);
            sum += f * sums[w][d];
            l += f * stats[w].y;
        }
        const Finish f = finish(a, m, l, unit);
        put(a, b, h, d, sum, f);
        if (d == 0) put_lse(a, b, h, f);
    }
}

int padded_dim(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

// How a call is laid out: CTAs, those of a unit's cluster (0: shares of all units), and the workspace's parts.
struct Layout {
    int grid, ctas;
    size_t ml, pieces, bytes;  // offsets behind the sums
};
template <template <int, int> class F, int kElem>
int by_dim(int dim) {
    switch (padded_dim(dim)) {
        case 64: return F<kElem, 64>::value;
        case 128: return F<kElem, 128>::value;
        default: return F<kElem, 256>::value;
    }
}
template <template <int, int> class F>
int by_shape(const estream_kv_cache* c) {
    return c->elem == ESTREAM_KV_BF16  ? by_dim<F, ESTREAM_KV_BF16>(c->dim)
           : c->elem == ESTREAM_KV_F16 ? by_dim<F, ESTREAM_KV_F16>(c->dim)
                                       : by_dim<F, ESTREAM_KV_E4M3>(c->dim);
}
template <int kElem, int kDim>
struct Resident {
    static constexpr int value = Shape<kElem, kDim>::kResident;
};
template <int kElem, int kDim>
struct Block {
    static constexpr int value = Shape<kElem, kDim>::kBlock;
};

// A unit gets a cluster while all fit on the device at once and its warps have 128 positions or fewer: one launch
// and no workspace (9 us a call instead of 17 for 1 x 500). In a graph, cluster against shares, us: 8 key heads of 500
// positions 5.6 / 8.9, 2048 8.0 / 9.6, 4096 10.6 / 10.4, 8192 16.3 / 12.0; 32 of 4096 11.9 / 14.4, 8192
// 24.9 / 28.1, where equal lengths fill the device either way but a cluster of a short sequence would leave it idle;
// 8 in E4M3 of 4096 9.6 / 10.8, 8192 13.7 / 11.4.
constexpr int kMaxCtas = 8;
constexpr int kDeep = 128;  // positions of a cluster's warp, at most

Layout layout(const estream_kv_cache* c, int B, int Hq, int M, int window, int sms) {
    const int group = Hq / c->heads, tiles = (group + kRows - 1) / kRows, kd = padded_dim(c->dim);
    const int block = by_shape<Block>(c), resident = by_shape<Resident>(c);
    long long blocks = (static_cast<long long>(M) * c->page_size + block - 1) / block;
    if (window > 0) blocks = std::min(blocks, window / block + 2ll);
    const long long units = static_cast<long long>(B) * c->heads * tiles, room = static_cast<long long>(sms) * resident;
    Layout l{};
    int ctas = 1;
    while (ctas < kMaxCtas && ctas * kWarps < blocks) ctas *= 2;
    if (units * ctas <= room && blocks * block <= ctas * kWarps * kDeep) {
        l.ctas = ctas;
        l.grid = static_cast<int>(units) * ctas;
        return l;
    }
    l.grid = static_cast<int>(std::max(1ll, std::min((blocks * units + kWarps - 1) / kWarps, room)));
    const size_t workers = static_cast<size_t>(l.grid) * kWarps, rows = std::min(group, kRows);
    l.ml = workers * 2 * rows * kd * 4;
    l.pieces = l.ml + workers * 2 * rows * 8;
    l.bytes = (l.pieces + static_cast<size_t>(units) * 8 + 15) / 16 * 16;
    return l;
}

template <int kElem, int kDim, int kTiles, bool kWhole>
cudaError_t launch(const Attend& a, int grid, cudaStream_t stream) {
    using S = Shape<kElem, kDim>;
    const auto kernel = k_kv_attend<kElem, kDim, kTiles, kWhole>;
    cudaError_t rc = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (rc != cudaSuccess) return rc;
    cudaLaunchAttribute attr[2] = {overlapped(), {}};
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(a.ctas);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = a.ctas ? 2 : 1;
    rc = cudaLaunchKernelEx(&cfg, kernel, a);
    if (rc != cudaSuccess || a.ctas) return rc;
    // a block an item while all are on the device at once, else a warp
    const int items = a.B * a.heads * a.tiles * a.rows, per_block = items <= 2 * grid ? 1 : kJoinWarps;
    return launch_overlapped(k_kv_join<kDim>, dim3((items + per_block - 1) / per_block), 32 * kJoinWarps, 0, stream, a, S::kUnit,
                             items, per_block);
}
template <int kElem, int kDim>
cudaError_t launch(const Attend& a, bool whole, int grid, cudaStream_t stream) {
    if (a.group > 8) return whole ? launch<kElem, kDim, 2, true>(a, grid, stream) : launch<kElem, kDim, 2, false>(a, grid, stream);
    return whole ? launch<kElem, kDim, 1, true>(a, grid, stream) : launch<kElem, kDim, 1, false>(a, grid, stream);
}
template <int kElem>
cudaError_t launch(const Attend& a, bool whole, int grid, cudaStream_t stream) {
    switch (padded_dim(a.dim)) {
        case 64: return launch<kElem, 64>(a, whole, grid, stream);
        case 128: return launch<kElem, 128>(a, whole, grid, stream);
        default: return launch<kElem, 256>(a, whole, grid, stream);
    }
}

bool at(const void* p, size_t a) { return p && reinterpret_cast<uintptr_t>(p) % a == 0; }

bool sizes_ok(const estream_kv_cache* c, int B, int Hq, int M) {
    return kv_cache_ok(c) && B >= 0 && Hq >= 1 && Hq % c->heads == 0 && Hq <= 1 << 16 && M >= 0 &&
           static_cast<long long>(B) * Hq <= 1 << 24 && static_cast<long long>(M) * c->page_size < (1ll << 31) - 4096;
}

}  // namespace
}  // namespace es

using namespace es;

extern "C" {

size_t estream_kv_attend_workspace_bytes(const estream_kv_cache* c, int B, int Hq, int M, int window) {
    int sms = 0;
    if (!sizes_ok(c, B, Hq, M) || B == 0 || window < 0 || sm_count(&sms) != cudaSuccess) return 0;
    return layout(c, B, Hq, M, window, sms).bytes;
}

estream_status estream_kv_attend(const estream_kv_cache* c, int elem, int B, int Hq, const void* q, long long q_row,
                                 long long q_head, const int32_t* table, int M, long long table_row,
                                 const int32_t* lens, float scale, int window, void* out, long long out_row,
                                 long long out_head, float* lse, void* workspace, size_t workspace_bytes,
                                 void* cuda_stream) {
    NvtxRange range(kNvKvAttend, B);
    if (!sizes_ok(c, B, Hq, M) || (elem != ESTREAM_KV_BF16 && elem != ESTREAM_KV_F16) ||
        (c->elem != ESTREAM_KV_E4M3 && c->elem != elem) || table_row < 0 || window < 0)
        return ESTREAM_ERR_INVALID_ARG;
    const double natural = static_cast<double>(scale) * c->k_scale;  // base 2's factor is to be finite
    if (!(std::fabs(natural) * 1.4426950408889634 <= 3.4028234e38)) return ESTREAM_ERR_INVALID_ARG;
    if (B == 0) return ESTREAM_OK;
    if (!at(q, 2) || !at(out, 2) || (M > 0 && !at(table, 4)) || !at(lens, 4) || (lse && !at(lse, 4)))
        return ESTREAM_ERR_INVALID_ARG;
    const estream_status st = on_device();
    if (st != ESTREAM_OK) return st;
    int sms = 0;
    if (sm_count(&sms) != cudaSuccess) return ESTREAM_ERR_CUDA;
    const Layout l = layout(c, B, Hq, M, window, sms);
    if (l.bytes && (workspace_bytes < l.bytes || !at(workspace, 16))) return ESTREAM_ERR_INVALID_ARG;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const int size = c->elem == ESTREAM_KV_E4M3 ? 1 : 2, group = Hq / c->heads;
    const float base2 = static_cast<float>(natural * 1.4426950408889634);
    const double back = base2 == 0.0f ? 0.69314718055994531 : natural / base2;
    const Attend a{q, out, lse, static_cast<const uint8_t*>(c->k), static_cast<const uint8_t*>(c->v), table, lens,
                   reinterpret_cast<float*>(ws), reinterpret_cast<float*>(ws + l.ml), reinterpret_cast<int2*>(ws + l.pieces),
                   q_row, q_head, out_row, out_head, table_row, c->k_page * size, c->k_token * size, c->k_head * size,
                   c->v_page * size, c->v_token * size, c->v_head * size,
                   base2, c->v_scale, static_cast<float>(back),
                   static_cast<float>(back - static_cast<double>(static_cast<float>(back))), B, Hq, c->heads, group, (group + kRows - 1) / kRows, std::min(group, kRows), c->dim, c->dim * size / 16, M,
                   M * c->page_size, c->num_pages, window, l.ctas, elem == ESTREAM_KV_F16,
                   at(q, 4) && q_row % 2 == 0 && q_head % 2 == 0, FastDiv(c->page_size)};
    const bool whole = c->page_size % kGroup == 0;
    const cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
    const cudaError_t rc = c->elem == ESTREAM_KV_BF16  ? launch<ESTREAM_KV_BF16>(a, whole, l.grid, stream)
                           : c->elem == ESTREAM_KV_F16 ? launch<ESTREAM_KV_F16>(a, whole, l.grid, stream)
                                                       : launch<ESTREAM_KV_E4M3>(a, whole, l.grid, stream);
    return rc == cudaSuccess ? ESTREAM_OK : ESTREAM_ERR_CUDA;
}

}  // extern "C"
