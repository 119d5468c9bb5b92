// New tokens' keys and values into a paged cache, keys (and the tokens' queries)
// rotated by their position on the way.
//
// Pair i of a rotated row, (a, b), becomes (a cos t - b sin t, b cos t + a sin t)
// with t = position * inv_freq[i]. Far positions make many turns, of which only the
// last, unfinished one counts: inv_freq / 2 pi is taken to 64 fractional bits, where
// the product with the position drops whole turns by itself. Of what is left the top 32
// bits are taken: a quarter turn and a rest of at most pi / 4, whose sine and cosine
// are Taylor series with the leading terms in two floats each, right to about 0.6 of
// fp32's half step (sincospi of the fraction as one float is off by four times that,
// which an 8-bit cache's rounding borders show). The angle's error is 2^-64 position
// (2^-53 position inv_freq / 2 pi from an inv_freq of 2 on) + 2^-33 turns.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

#include "estream_internal.h"
#include "overlap.cuh"

namespace es {
namespace {

struct Append {
    const void *k, *v, *q;
    void *q_out, *kc, *vc;
    long long k_token, k_head, v_token, v_head, q_token, q_head, qo_token, qo_head;
    long long kc_page, kc_token, kc_head, vc_page, vc_token, vc_head;
    const int32_t *positions, *rows, *table;
    const float* inv_freq;
    long long table_row;
    float k_inv, v_inv;  // 1 / scale
    int T, B, M, num_pages, Hq, heads, dim, rot, interleaved;
    int per_head, per_v;  // units of a rotated and of a value head
    int parts;            // log2 of the warps that share a token's heads
    FastDiv page;
};

template <bool kF16>
__device__ __forceinline__ float2 up2(uint32_t w) {
    if constexpr (kF16) return __half22float2(*reinterpret_cast<__half2*>(&w));
    else return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&w));
}
template <bool kF16>
__device__ __forceinline__ uint32_t down2(float x, float y) {
    if constexpr (kF16) {
        const __half2 h = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}
template <bool kF16>
__device__ __forceinline__ float up1(uint16_t v) {
    if constexpr (kF16) return __half2float(__ushort_as_half(v));
    else return __bfloat162float(__ushort_as_bfloat16(v));
}
template <bool kF16>
__device__ __forceinline__ uint16_t down1(float v) {
    if constexpr (kF16) return __half_as_ushort(__float2half_rn(v));
    else return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// Eight values that lie together.
struct Eight {
    float x[8];
};
template <bool kF16>
__device__ __forceinline__ Eight widen(uint4 w) {
    Eight e;
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = up2<kF16>(u[i]);
        e.x[2 * i] = f.x;
        e.x[2 * i + 1] = f.y;
    }
    return e;
}
template <bool kF16>
__device__ __forceinline__ void store16(void* to, const Eight& e) {
    *static_cast<uint4*>(to) = make_uint4(down2<kF16>(e.x[0], e.x[1]), down2<kF16>(e.x[2], e.x[3]),
                                          down2<kF16>(e.x[4], e.x[5]), down2<kF16>(e.x[6], e.x[7]));
}
__device__ __forceinline__ uint32_t e4m3x2(float x, float y) {
    return __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
}
// To the cache, whose elements are of the input's type or E4M3.
template <bool kF16, bool kE4m3>
__device__ __forceinline__ void keep8(void* base, long long at, const Eight& e, float inv) {
    if constexpr (kE4m3) {
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = e4m3x2(e.x[4 * i] * inv, e.x[4 * i + 1] * inv) |
                   e4m3x2(e.x[4 * i + 2] * inv, e.x[4 * i + 3] * inv) << 16;
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(base) + at) = make_uint2(w[0], w[1]);
    } else {
        store16<kF16>(static_cast<uint16_t*>(base) + at, e);
    }
}
template <bool kF16, bool kE4m3>
__device__ __forceinline__ void keep1(void* base, long long at, float x, float inv) {
    if constexpr (kE4m3) static_cast<uint8_t*>(base)[at] = __nv_cvt_float_to_fp8(x * inv, __NV_SATFINITE, __NV_E4M3);
    else static_cast<uint16_t*>(base)[at] = down1<kF16>(x);
}

// f / 2 pi turns, 64 fractional bits, rounded down, of a finite f (of others: any). In integers below 2: with double's
// operations, of which an SM does two a clock, 4096 tokens took 5 us longer.
__device__ __forceinline__ uint64_t turns_of(float f) {
    const uint32_t u = __float_as_uint(f), e = u >> 23 & 0xff;
    uint64_t w;
    if (e < 128) {
        // f = m 2^(max(e, 1) - 150); 2^88 / 2 pi in two words
        constexpr uint64_t kHigh = 0x28be60, kLow = 0xdb9391054a7f09d6ull;
        const uint64_t m = (u & 0x7fffff) | (e ? 0x800000u : 0u);
        const uint64_t low = m * kLow, high = m * kHigh + __umul64hi(m, kLow);
        const uint32_t s = 174 - max(e, 1u);  // 47 for the largest
        w = s < 64 ? high << (64 - s) | low >> s : s < 128 ? high >> (s - 64) : 0;
    } else {
        double turns = static_cast<double>(fminf(fabsf(f), 3.402823466e38f)) * 0.15915494309189533577;
        turns -= floor(turns);
        w = static_cast<uint64_t>(turns * 18446744073709551616.0);
    }
    return u >> 31 ? ~w + 1 : w;
}

// cos, sin of a fraction of a turn, 32 bits.
__device__ __forceinline__ float2 cos_sin(uint32_t turn) {
    const uint32_t quarter = (turn + 0x20000000u) >> 30;
    const int rest = static_cast<int>(turn - (quarter << 30));  // of 2^32, in [-2^29, 2^29)
    const float r = static_cast<float>(rest), r_low = static_cast<float>(rest - static_cast<int>(r));
    constexpr float kUnit = 1.4629180e-9f;  // 2 pi / 2^32, rounded, and what that leaves
    constexpr float kUnitLow = static_cast<float>(1.4629180792671596e-9 - static_cast<double>(kUnit));
    const float x = r * kUnit, x_low = fmaf(r, kUnit, -x) + fmaf(r, kUnitLow, r_low * kUnit);
    const float q = x * x, q_low = fmaf(x, x, -q) + 2.0f * x * x_low;
    // x - x^3/6 + x^5/120 - ... : next term x^13/13! < 2^-36
    float s = fmaf(q, -1.0f / 39916800.0f, 1.0f / 362880.0f);
    s = fmaf(q, s, -1.0f / 5040.0f);
    s = fmaf(q, s, 1.0f / 120.0f);
    s = fmaf(q, s, -1.0f / 6.0f);
    s = x + fmaf(x * q, s, x_low);
    // 1 - x^2/2 + x^4/24 - ... : next term x^12/12! < 2^-32
    float c = fmaf(q, -1.0f / 3628800.0f, 1.0f / 40320.0f);
    c = fmaf(q, c, -1.0f / 720.0f);
    c = fmaf(q, c, 1.0f / 24.0f);
    const float lead = fmaf(q, -0.5f, 1.0f), lead_low = fmaf(q, -0.5f, 1.0f - lead);
    c = lead + fmaf(q * q, c, fmaf(q_low, -0.5f, lead_low));
    if (quarter & 1) {
        const float t = c;
        c = -s;
        s = t;
    }
    return quarter & 2 ? make_float2(-c, -s) : make_float2(c, s);
}

// How a lane's unit of work lies in a row: one pair or value; eight pairs whose
// halves are rot / 2 apart (or eight values that are not rotated); eight values
// that hold four neighbouring pairs.
enum Mode { kSingles, kHalves, kNeighbours };

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Bound by HBM for many tokens and by latency for few. A warp has a token, or where tokens
// are few a part of its heads: it goes over the heads with several steps' values under way, and
// forms the token's sines and cosines, one pair a lane, behind the first loads; a lane has the same unit of
// every head it comes to, so sines, cosines and strides stay in registers. Nothing
// waits for another warp. 4096 tokens of 16 + 32 heads of 128: 16.7 us (101 MB, 6.0 TB/s), 114
// instructions a unit; a block a token, with a division and sines from shared memory for
// every unit, took 169 and 24 us. One token of 32 + 16 heads: 3.0 us in a graph.
template <Mode kMode, bool kF16, bool kE4m3>
__global__ void __launch_bounds__(kThreads, kMode == kHalves ? 3 : 4) k_kv_append(const Append a) {
    constexpr int kPairs = kMode == kSingles ? 1 : kMode == kHalves ? 8 : 4;  // of a unit
    constexpr int kBytes = kE4m3 ? 1 : 2;                                     // of a cache element
    constexpr int kAtOnce = kMode == kHalves ? 2 : 4;                         // heads whose values a lane has under way
    using Raw = std::conditional_t<kMode == kSingles, uint16_t, uint4>;
    __shared__ __align__(16) float2 turn[kWarps][kKvMaxDim / 2];  // cos, sin
    after_previous();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int item = blockIdx.x * kWarps + warp, t = item >> a.parts, part = item & ((1 << a.parts) - 1);
    if (t >= a.T) return;
    const int pos = a.positions[t], row = a.rows ? a.rows[t] : t, pairs = a.rot / 2;
    if (pos < 0) return;  // padding
    const int entry = static_cast<int>(a.page.div(pos)), slot = pos - entry * static_cast<int>(a.page.d);
    int page = -1;
    if (row >= 0 && row < a.B && entry < a.M) page = a.table[row * a.table_row + entry];
    const bool ok = page >= 0 && page < a.num_pages;
    const float nan = __int_as_float(0x7fc00000);
    bool formed = false;
    auto form_angles = [&] {  // once the first values are under way
        if (formed) return;
        formed = true;
        for (int p = lane; p < pairs; p += 32) {
            const float f = a.inv_freq[p];
            const uint64_t angle = turns_of(f) * static_cast<uint64_t>(pos);
            turn[warp][p] = fabsf(f) < INFINITY ? cos_sin(static_cast<uint32_t>((angle + 0x80000000u) >> 32)) : make_float2(nan, nan);
        }
        __syncwarp();
    };
    int steps = 0;  // of the kinds of heads before; the parts of a token take turns at all of them
    // The heads of one kind: from `from` (of this token), heads from_head elements apart, to `to`,
    // to_head bytes apart; into the cache, or as queries.
    auto go = [&](auto rotated, auto cached, int heads, int per_head, const void* from, long long from_head, void* to,
                  long long to_head, float inv) {
        constexpr bool kRotated = decltype(rotated)::value, kCached = decltype(cached)::value;
        const int together = per_head < 32 ? 32 / per_head : 1;  // heads of a step
        const int parts = 1 << a.parts, mine = part - steps & parts - 1;  // this warp's first step
        steps += (heads + together - 1) / together;
        for (int j0 = 0; j0 < per_head; j0 += 32) {
            if (mine * together >= heads) break;
            const int sub = per_head < 32 ? lane / per_head : 0, j = per_head < 32 ? lane - sub * per_head : j0 + lane;
            const bool active = sub < together && j < per_head;
            const bool turns = kRotated && active && j * kPairs < pairs;
            int d0, d1;  // where the unit's values lie
            if constexpr (kMode == kSingles) {
                d0 = !kRotated ? j : !turns ? j + pairs : a.interleaved ? 2 * j : j;
                d1 = !turns ? d0 : a.interleaved ? d0 + 1 : j + pairs;
            } else if constexpr (kMode == kHalves && kRotated) {
                d0 = turns ? 8 * j : 8 * j + pairs;
                d1 = turns ? 8 * j + pairs : d0;
            } else {
                d0 = d1 = 8 * j;
            }
            float2 cs[kPairs];
            const int first = active ? mine * together + sub : heads, step = together << a.parts;
            const uint16_t* f = static_cast<const uint16_t*>(from) + first * from_head;
            uint8_t* o = static_cast<uint8_t*>(to) + first * to_head;
            const long long f_step = step * from_head, o_step = step * to_head;
            constexpr bool kTwo = kMode != kNeighbours && kRotated;
            bool begun = false;
            for (int h = first; h < heads || !begun; h += kAtOnce * step) {  // at least once, for the angles
                Raw raw[kAtOnce][kTwo ? 2 : 1];
#pragma unroll
                for (int q = 0; q < kAtOnce; ++q)
                    if (h + q * step < heads) {
                        raw[q][0] = *reinterpret_cast<const Raw*>(f + d0);
                        if constexpr (kTwo) raw[q][1] = *reinterpret_cast<const Raw*>(f + d1);
                        f += f_step;
                    }
                if (!begun) {
                    begun = true;
                    if constexpr (kRotated) form_angles();
                    if (turns) {
#pragma unroll
                        for (int q = 0; q < kPairs; ++q) cs[q] = turn[warp][j * kPairs + q];  // past the last pair: not used
                    }
                    if (kCached && !ok) return;
                }
#pragma unroll
                for (int q = 0; q < kAtOnce; ++q) {
                    if (h + q * step >= heads) break;
                    if constexpr (kMode == kSingles) {
                        float x = up1<kF16>(raw[q][0]), y = 0.0f;
                        if (turns) {
                            y = up1<kF16>(raw[q][kTwo ? 1 : 0]);
                            const float lo = x * cs[0].x - y * cs[0].y;
                            y = y * cs[0].x + x * cs[0].y;
                            x = lo;
                        }
                        if (!kCached && !ok) x = y = nan;
                        if constexpr (kCached) {
                            keep1<kF16, kE4m3>(o, d0, x, inv);
                            if (turns) keep1<kF16, kE4m3>(o, d1, y, inv);
                        } else {
                            reinterpret_cast<uint16_t*>(o)[d0] = down1<kF16>(x);
                            if (turns) reinterpret_cast<uint16_t*>(o)[d1] = down1<kF16>(y);
                        }
                    } else if (kRotated || (kCached && kE4m3)) {
                        Eight x = widen<kF16>(raw[q][0]), y;
                        if (turns) {
                            if constexpr (kTwo) {
                                y = widen<kF16>(raw[q][1]);
#pragma unroll
                                for (int e = 0; e < 8; ++e) {
                                    const float2 c = cs[e % kPairs];
                                    const float lo = x.x[e] * c.x - y.x[e] * c.y;
                                    y.x[e] = y.x[e] * c.x + x.x[e] * c.y;
                                    x.x[e] = lo;
                                }
                            } else {
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    // pairs behind the rotated ones stay as they are: by (1, 0), an infinity's neighbour would be NaN
                                    if (j * kPairs + e >= pairs) continue;
                                    const float2 c = cs[e % kPairs];
                                    const float lo = x.x[2 * e] * c.x - x.x[2 * e + 1] * c.y;
                                    x.x[2 * e + 1] = x.x[2 * e + 1] * c.x + x.x[2 * e] * c.y;
                                    x.x[2 * e] = lo;
                                }
                            }
                        }
                        if (!kCached && !ok)
#pragma unroll
                            for (int e = 0; e < 8; ++e) x.x[e] = y.x[e] = nan;
                        if constexpr (kCached) {
                            keep8<kF16, kE4m3>(o, d0, x, inv);
                            if constexpr (kTwo)
                                if (turns) keep8<kF16, kE4m3>(o, d1, y, inv);
                        } else {
                            store16<kF16>(o + 2 * d0, x);
                            if constexpr (kTwo)
                                if (turns) store16<kF16>(o + 2 * d1, y);
                        }
                    } else {
                        *reinterpret_cast<Raw*>(o + 2 * d0) = raw[q][0];  // as it is
                    }
                    o += o_step;
                }
            }
        }
    };
    using yes = std::true_type;
    using no = std::false_type;
    if (a.Hq)
        go(yes{}, no{}, a.Hq, a.per_head, static_cast<const uint16_t*>(a.q) + t * a.q_token, a.q_head,
           static_cast<uint16_t*>(a.q_out) + t * a.qo_token, 2 * a.qo_head, 1.0f);
    go(yes{}, yes{}, a.heads, a.per_head, static_cast<const uint16_t*>(a.k) + t * a.k_token, a.k_head,
       static_cast<uint8_t*>(a.kc) + (page * a.kc_page + slot * a.kc_token) * kBytes, kBytes * a.kc_head, a.k_inv);
    go(no{}, yes{}, a.heads, a.per_v, static_cast<const uint16_t*>(a.v) + t * a.v_token, a.v_head,
       static_cast<uint8_t*>(a.vc) + (page * a.vc_page + slot * a.vc_token) * kBytes, kBytes * a.vc_head, a.v_inv);
}

template <Mode kMode, bool kF16>
cudaError_t launch(const Append& a, bool e4m3, int grid, cudaStream_t stream) {
    return e4m3 ? launch_overlapped(k_kv_append<kMode, kF16, true>, dim3(grid), kThreads, 0, stream, a)
                : launch_overlapped(k_kv_append<kMode, kF16, false>, dim3(grid), kThreads, 0, stream, a);
}
template <bool kF16>
cudaError_t launch(const Append& a, Mode mode, bool e4m3, int grid, cudaStream_t stream) {
    switch (mode) {
        case kSingles: return launch<kSingles, kF16>(a, e4m3, grid, stream);
        case kHalves: return launch<kHalves, kF16>(a, e4m3, grid, stream);
        default: return launch<kNeighbours, kF16>(a, e4m3, grid, stream);
    }
}

bool at(const void* p, size_t a) { return p && reinterpret_cast<uintptr_t>(p) % a == 0; }
// Rows of 16-bit values at `p` that start on 16 bytes.
bool on16(const void* p, long long token, long long head) { return at(p, 16) && token % 8 == 0 && head % 8 == 0; }

}  // namespace

bool kv_cache_ok(const estream_kv_cache* c) {
    if (!c || c->elem < ESTREAM_KV_BF16 || c->elem > ESTREAM_KV_E4M3 || c->num_pages < 0 || c->num_pages > 1 << 30 ||
        c->page_size < 1 || c->page_size > 1 << 30 || c->heads < 1 || c->heads > kKvMaxHeads || c->dim < 16 ||
        c->dim > kKvMaxDim || c->dim % 16)
        return false;
    auto scale = [&](float s) { return s >= 0x1p-100f && s <= 0x1p100f && (c->elem == ESTREAM_KV_E4M3 || s == 1.0f); };
    if (!scale(c->k_scale) || !scale(c->v_scale)) return false;
    if (c->num_pages > 0 && (!at(c->k, 16) || !at(c->v, 16))) return false;
    const long long unit = c->elem == ESTREAM_KV_E4M3 ? 16 : 8, most = 1ll << 40;
    auto stride = [&](long long s, int n) { return n == 1 || (s >= c->dim && s <= most && s % unit == 0); };
    return stride(c->k_page, c->num_pages) && stride(c->v_page, c->num_pages) && stride(c->k_token, c->page_size) &&
           stride(c->v_token, c->page_size) && stride(c->k_head, c->heads) && stride(c->v_head, c->heads);
}

}  // namespace es

using namespace es;

extern "C" estream_status estream_kv_append(const estream_kv_cache* c, int elem, int T, const void* k, long long k_token,
                                            long long k_head, const void* v, long long v_token, long long v_head,
                                            const int32_t* positions, const int32_t* rows, const int32_t* table,
                                            int B, int M, long long table_row, const void* q, long long q_token,
                                            long long q_head, int Hq, void* q_out, long long qo_token,
                                            long long qo_head, const float* inv_freq, int rot, int interleaved,
                                            void* cuda_stream) {
    NvtxRange range(kNvKvAppend, T);
    if (!kv_cache_ok(c) || (elem != ESTREAM_KV_BF16 && elem != ESTREAM_KV_F16) ||
        (c->elem != ESTREAM_KV_E4M3 && c->elem != elem) || T < 0 || T > 1 << 24 || B < 0 || M < 0 || table_row < 0 ||
        Hq < 0 || Hq > kKvMaxHeads || rot < 0 || rot % 2 || rot > c->dim)
        return ESTREAM_ERR_INVALID_ARG;
    if (T == 0) return ESTREAM_OK;
    const bool entries = B > 0 && M > 0;
    if (!at(k, 2) || !at(v, 2) || !at(positions, 4) || (rows && !at(rows, 4)) || (entries && !at(table, 4)) ||
        (Hq && (!at(q, 2) || !at(q_out, 2))) || (rot && !at(inv_freq, 4)))
        return ESTREAM_ERR_INVALID_ARG;
    const estream_status st = on_device();
    if (st != ESTREAM_OK) return st;
    const bool wide = on16(k, k_token, k_head) && on16(v, v_token, v_head) &&
                      (!Hq || (on16(q, q_token, q_head) && on16(q_out, qo_token, qo_head)));
    const bool neighbours = interleaved || rot == 0;
    const Mode mode = !wide || (!neighbours && rot % 16) ? kSingles : neighbours ? kNeighbours : kHalves;
    const int dim = c->dim;
    const int per_head = mode == kSingles ? dim - rot / 2 : mode == kHalves ? rot / 16 + (dim - rot) / 8 : dim / 8;
    const int per_v = mode == kSingles ? dim : dim / 8;
    // warps for a token: one while tokens alone fill the device with 32 warps an SM, at most 16 (32 tokens 3.8 us;
    // with 32 warps 4.2, and 1 token 3.0 with either)
    int parts = 0, sms = 0;
    if (sm_count(&sms) != cudaSuccess) return ESTREAM_ERR_CUDA;
    while (parts < 4 && (static_cast<long long>(T) << parts) < sms * 32) ++parts;
    const Append a{k, v, q, q_out, c->k, c->v, k_token, k_head, v_token, v_head, q_token, q_head, qo_token, qo_head,
                   c->k_page, c->k_token, c->k_head, c->v_page, c->v_token, c->v_head, positions, rows, table,
                   inv_freq, table_row, 1.0f / c->k_scale, 1.0f / c->v_scale, T, entries ? B : 0, M, c->num_pages, Hq,
                   c->heads, dim, rot, interleaved != 0, per_head, per_v, parts, FastDiv(c->page_size)};
    const int grid = static_cast<int>(((static_cast<long long>(T) << parts) + kWarps - 1) / kWarps);
    const cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
    const bool e4m3 = c->elem == ESTREAM_KV_E4M3;
    const cudaError_t rc = elem == ESTREAM_KV_F16 ? launch<true>(a, mode, e4m3, grid, stream)
                                                  : launch<false>(a, mode, e4m3, grid, stream);
    return rc == cudaSuccess ? ESTREAM_OK : ESTREAM_ERR_CUDA;
}
