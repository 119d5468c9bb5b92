// Softmax top-k of one token's router logits by one warp, shared by the route
// build (route.cu) and the few-token layer kernel (decode.cu): the written
// fp32 exponential, the selection order and the weights.
// Included inside `namespace es` after tc_ptx.cuh.
#pragma once

// ---------------------------------------------------------------------------
// Written fp32 exponential, the same written definition the CPU oracle uses,
// implemented here on its own so both sides round identically:
//   x < -87 -> 0; n = nearest-even(fl(x * LOG2E));
//   r = fma(-n, LN2_HI, x); r = fma(-n, LN2_LO, r)   (Cody & Waite, 1980)
//   p = Horner of sum_{j<=7} r^j/j!, one fma per step;  result = p * 2^n.
// LN2_HI = fp32(ln 2) with its 8 low significand bits cleared, LN2_LO =
// fp32(ln 2 - LN2_HI); LOG2E and 1/j! are round-to-nearest fp32 values.
// Every operation is an explicit round-to-nearest intrinsic (no contraction).
// ---------------------------------------------------------------------------
__device__ __forceinline__ float route_exp(float x) {
    if (x < -87.0f) return 0.0f;
    const float kLog2e = 0x1.715476p+0f;
    const float kLn2Hi = 0x1.62e4p-1f;
    const float kLn2Lo = 0x1.7f7d1cp-20f;
    const int n = __float2int_rn(__fmul_rn(x, kLog2e));
    const float nf = static_cast<float>(n);
    float r = __fmaf_rn(-nf, kLn2Hi, x);
    r = __fmaf_rn(-nf, kLn2Lo, r);
    float p = 0x1.a01a02p-13f;           // 1/7!
    p = __fmaf_rn(p, r, 0x1.6c16c2p-10f);  // 1/6!
    p = __fmaf_rn(p, r, 0x1.111112p-7f);   // 1/5!
    p = __fmaf_rn(p, r, 0x1.555556p-5f);   // 1/4!
    p = __fmaf_rn(p, r, 0x1.555556p-3f);   // 1/3!
    p = __fmaf_rn(p, r, 0.5f);             // 1/2!
    p = __fmaf_rn(p, r, 1.0f);             // 1/1!
    p = __fmaf_rn(p, r, 1.0f);             // 1/0!
    return __fmul_rn(p, __int_as_float((n + 127) << 23));
}

// One warp per token; lane l holds the logits of experts l, l+32, l+64, ...
// The softmax denominator is summed in ascending expert order (the same
// sequence of fp32 additions as the written definition): the warp streams the
// per-expert exponentials to every lane with shuffles, one expert at a time.
// Selection walks the strict total order (logit descending, expert id
// ascending): round j takes the best expert after round j-1's pick in that
// order. Each logit is mapped to an unsigned key of the same order (-0 taken
// as +0, which compares equal to it), so a round is one warp-wide max of the
// keys and one min of the ids holding it. Lane j then forms route j's weight.
constexpr int kMaxPerLane = kMaxE / 32;

// kJ: logits held per lane (E <= 32 kJ), so that small E keeps the arrays in
// registers.
// l: the token's E logits (global or shared memory).
template <int kJ>
__device__ __forceinline__ void topk_token(
    int t, const float* l, int E, int k, int renorm,
    const int32_t* __restrict__ phi, int P, int32_t* __restrict__ topk_ids,
    float* __restrict__ alpha, int* counts, int* __restrict__ err) {
    const int lane = threadIdx.x & 31;
    const int nj = (E + 31) >> 5;
    const float kNegInf = __int_as_float(0xff800000);
    float v[kJ];
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
        const int e = lane + 32 * j;
        v[j] = (j < nj && e < E) ? l[e] : kNegInf;
    }
    float m = kNegInf;
#pragma unroll
    for (int j = 0; j < kJ; ++j) m = fmaxf(m, v[j]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));

    // denominator: sequential fp32 sum over e = 0, 1, ..., E-1
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
        if (j >= nj) break;
        const int e = lane + 32 * j;
        const float p = (e < E) ? route_exp(__fsub_rn(v[j], m)) : 0.0f;
        const int n_here = min(32, E - 32 * j);
        if (n_here == 32) {
#pragma unroll
            for (int src = 0; src < 32; ++src) s = __fadd_rn(s, __shfl_sync(0xffffffffu, p, src));
        } else {
            for (int src = 0; src < n_here; ++src)
                s = __fadd_rn(s, __shfl_sync(0xffffffffu, p, src));
        }
    }

    // order-preserving keys (entries past E are never candidates)
    uint32_t key[kJ];
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
        const uint32_t b = __float_as_uint(__fadd_rn(v[j], 0.0f));  // -0 -> +0
        key[j] = (j < nj && lane + 32 * j < E) ? ((b & 0x80000000u) ? ~b : (b | 0x80000000u)) : 0u;
    }
    uint32_t prev_k = 0xffffffffu;  // every expert comes after it
    uint32_t prev_i = 0u;           // with prev_k = max, ids compare as "after" from 0 on
    bool first = true;
    uint32_t key_mine = 0u;  // lane j keeps route j's key and expert
    int id_mine = -1;
    for (int r = 0; r < k; ++r) {
        uint32_t bk = 0u, bi = 0xffffffffu;
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
            if (j >= nj) break;
            const uint32_t e = static_cast<uint32_t>(lane + 32 * j);
            if (static_cast<int>(e) >= E) break;
            const bool after_prev =
                first || key[j] < prev_k || (key[j] == prev_k && e > prev_i);
            if (after_prev && (key[j] > bk || (key[j] == bk && e < bi))) {
                bk = key[j];
                bi = e;
            }
        }
        const uint32_t mk = __reduce_max_sync(0xffffffffu, bk);
        const uint32_t mi = __reduce_min_sync(0xffffffffu, bk == mk ? bi : 0xffffffffu);
        prev_k = mk;
        prev_i = mi;
        first = false;
        if (lane == r) {
            key_mine = mk;
            id_mine = static_cast<int>(mi);
        }
    }
    float a_mine = 0.0f;
    if (lane < k) {
        const float bv = __uint_as_float((key_mine & 0x80000000u) ? (key_mine & 0x7fffffffu) : ~key_mine);
        a_mine = __fdiv_rn(route_exp(__fsub_rn(bv, m)), s);
    }
    if (renorm) {
        float z = 0.0f;  // summed in rank order
        for (int r = 0; r < k; ++r) z = __fadd_rn(z, __shfl_sync(0xffffffffu, a_mine, r));
        a_mine = __fdiv_rn(a_mine, z);
    }
    if (lane < k) {
        const int i = t * k + lane;
        topk_ids[i] = id_mine;
        alpha[i] = a_mine;
        // no candidate is selected only for logits outside the contract (a
        // row of NaNs with every bit set): file the route as unresolved
        int slot = id_mine < 0 ? P + 1 : (phi ? phi[id_mine] : id_mine);
        if (slot < -1 || slot >= P) {
            record_error(err, kDevErrSlotRange);
            slot = -1;
        }
        const int b = slot < 0 ? P : slot;
        atomicAdd(&counts[b], 1);
    }
}
