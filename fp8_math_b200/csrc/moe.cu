// moe.cu -- kernels of a mixture-of-experts layer's training step that stand
// between the quantizers and the grouped GEMM: the router (top-k, weights,
// counts, row order, balance loss) and its gradient, the combine of expert
// rows in bf16 and its gradients, the gated SiLU whose input is kept in MXFP8
// for the backward pass.  All sums are in fp32 and in a fixed order, so a call
// gives the same bits every time.
#include <algorithm>

#include <cooperative_groups.h>

#include "common.cuh"
#include "moe.cuh"

namespace bsq {

namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kChunk = 64;  // tokens of one router CTA: their choice of an expert is one 64-bit mask

BSQ_DEV float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}
BSQ_DEV uint32_t pack_bf16(float lo, float hi) {
    __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&b);
}
BSQ_DEV float load_logit(const float *p) { return __ldg(p); }
BSQ_DEV float load_logit(const uint16_t *p) { return __uint_as_float((uint32_t)__ldg(p) << 16); }
BSQ_DEV void store_logit(uint16_t *p, float v) { *p = (uint16_t)(pack_bf16(v, 0.0f) & 0xFFFFu); }

// a * b + c on an fp32 pair
BSQ_DEV f32x2 f2_fma(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// 2^x (relative error 2^-22, results below 2^-126 are 0) and 1/x of a normal x (1 ulp).
BSQ_DEV float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
BSQ_DEV float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.44269504088896341f;

// n / d for the grid's 32-bit unit numbers: multiply-shift with a
// precomputed multiplier (Granlund and Montgomery, PLDI'94).
struct UnitDiv {
    uint32_t d, mul, sh1, sh2;
};
UnitDiv unit_div(uint32_t d) {
    int l = 0;
    while (l < 32 && (uint64_t(1) << l) < d) l++;
    const uint64_t m = ((uint64_t(1) << 32) * ((uint64_t(1) << l) - d)) / d + 1;
    return UnitDiv{d, (uint32_t)m, (uint32_t)std::min(l, 1), (uint32_t)std::max(l - 1, 0)};
}
BSQ_DEV uint32_t divide(uint32_t n, const UnitDiv &v) {
    const uint32_t t = __umulhi(v.mul, n);
    return (t + ((n - t) >> v.sh1)) >> v.sh2;
}

// min(a, b), NaN when one of them is NaN
BSQ_DEV float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Sum and maximum over the LPT neighbouring lanes that share a token.
template <int LPT>
BSQ_DEV float group_sum(float v) {
#pragma unroll
    for (int o = LPT / 2; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}
template <int LPT>
BSQ_DEV float group_max(float v) {
#pragma unroll
    for (int o = LPT / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}

// A lane's logits of one token: LPT lanes hold a row in quads of four
// consecutive experts, lane `sub` the quads sub, sub + LPT, ...  Experts past
// E are -inf.  `vec`: E % 4 == 0 and every row starts on a quad's alignment.
template <typename In, int LPT, int Q>
struct Row;

template <int LPT, int Q>
struct Row<uint16_t, LPT, Q> {
    uint2 w[Q];
    BSQ_DEV void load(const uint16_t *row, int E, int sub, bool vec, bool live) {
#pragma unroll
        for (int q = 0; q < Q; q++) {
            const int e = 4 * (q * LPT + sub);
            w[q] = make_uint2(0xFF80FF80u, 0xFF80FF80u);
            if (!live || e >= E) continue;
            if (vec) {
                w[q] = __ldg(reinterpret_cast<const uint2 *>(row + e));
            } else {  // (32-bit words and a shift were slower: neighbouring rows part ways)
                uint32_t v[4];
#pragma unroll
                for (int i = 0; i < 4; i++) v[i] = e + i < E ? (uint32_t)__ldg(row + e + i) : 0xFF80u;
                w[q] = make_uint2(v[0] | (v[1] << 16), v[2] | (v[3] << 16));
            }
        }
    }
    BSQ_DEV void clear() {
#pragma unroll
        for (int q = 0; q < Q; q++) w[q] = make_uint2(0xFF80FF80u, 0xFF80FF80u);
    }
    BSQ_DEV float quad_max(int q) const {
        uint32_t m;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(w[q].x), "r"(w[q].y));
        return fmaxf(bf16_lo(m), bf16_hi(m));
    }
    BSQ_DEV void get(int q, float z[4]) const {
        z[0] = bf16_lo(w[q].x);
        z[1] = bf16_hi(w[q].x);
        z[2] = bf16_lo(w[q].y);
        z[3] = bf16_hi(w[q].y);
    }
};

template <int LPT, int Q>
struct Row<float, LPT, Q> {
    float4 w[Q];
    BSQ_DEV void load(const float *row, int E, int sub, bool vec, bool live) {
#pragma unroll
        for (int q = 0; q < Q; q++) {
            const int e = 4 * (q * LPT + sub);
            w[q] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (!live || e >= E) continue;
            if (vec) {
                w[q] = __ldg(reinterpret_cast<const float4 *>(row + e));
            } else {
                w[q].x = __ldg(row + e);
                if (e + 1 < E) w[q].y = __ldg(row + e + 1);
                if (e + 2 < E) w[q].z = __ldg(row + e + 2);
                if (e + 3 < E) w[q].w = __ldg(row + e + 3);
            }
        }
    }
    BSQ_DEV void clear() {
#pragma unroll
        for (int q = 0; q < Q; q++) w[q] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    }
    BSQ_DEV float quad_max(int q) const {
        return fmaxf(fmaxf(w[q].x, w[q].y), fmaxf(w[q].z, w[q].w));
    }
    BSQ_DEV void get(int q, float z[4]) const {
        z[0] = w[q].x;
        z[1] = w[q].y;
        z[2] = w[q].z;
        z[3] = w[q].w;
    }
};

// max(a, b), NaN when one of them is NaN
BSQ_DEV float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// e^d = 2^t (1 + (d - t ln 2)) with t = fl(d log2 e): the second factor takes
// back the roundings of t and of log2 e, which alone would be |d| 2^-23 (ln 2 in
// fp32 leaves |d| 2^-28).  d is held at -150, where 2^t is 0: a logit of -inf,
// or one so low that the difference overflows, would give a factor of NaN.
constexpr float kLn2 = 0.693147180559945309f, kLowest = -150.0f;

BSQ_DEV float exp_of(float d) {
    d = max_nan(d, kLowest);
    const float t = d * kLog2e, p = ex2(t);
    return fmaf(p, fmaf(t, -kLn2, d), p);
}
// exp(x[i] - top); -inf gives 0.
BSQ_DEV void exp_below4(float x[4], f32x2 top2) {
    const f32x2 l2 = f2_pack(kLog2e, kLog2e), ln2 = f2_pack(-kLn2, -kLn2);
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        float a, b;
        f2_unpack(f2_sub(f2_pack(x[i], x[i + 1]), top2), a, b);
        const f32x2 d = f2_pack(max_nan(a, kLowest), max_nan(b, kLowest)), t = f2_mul(d, l2);
        f2_unpack(t, a, b);
        const f32x2 p = f2_pack(ex2(a), ex2(b));
        f2_unpack(f2_fma(p, f2_fma(t, ln2, d), p), x[i], x[i + 1]);
    }
}

// ------------------------------------------------------------------ router
// A lane's best D candidates among its logits, in the order (-logit, expert),
// so that each of the k rounds is one maximum over the token's lanes; a lane
// that has given all D looks at its logits again.  D is chosen so that with k
// near 8 few tokens need that: the lanes give k / LPT each on average.  -inf
// is never a candidate.
//
// bf16 logits leave 16 bits of an fp32 free: the expert goes there, so that
// one float comparison orders (logit, expert) and no two are equal.  Larger
// low bits make a positive float larger and a negative one smaller; adding 0
// turns -0 into +0 first.  -inf with low bits is a NaN, which maxima pass
// over (and min_nan hands on to them).
template <typename In, int LPT, int Q>
struct Candidates;

template <int LPT>
constexpr int kDepth = LPT == 8 ? 4 : LPT == 16 ? 3 : 2;

template <int LPT, int Q>
struct Candidates<uint16_t, LPT, Q> {
    static constexpr int D = kDepth<LPT>;
    float m[D];
    int left;
    template <bool AGAIN>
    BSQ_DEV void fill(const Row<uint16_t, LPT, Q> &row, int sub, float limit) {
        left = D;
#pragma unroll
        for (int d = 0; d < D; d++) m[d] = -INFINITY;
#pragma unroll
        for (int q = 0; q < Q; q++) {
            float z[4];
            row.get(q, z);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const uint32_t b = __float_as_uint(__fadd_rn(z[i], 0.0f));
                const uint32_t e = (uint32_t)(4 * (q * LPT + sub) + i);
                float key = __uint_as_float(b | (e ^ (~(uint32_t)((int32_t)b >> 31) & 0xFFFFu)));
                if (AGAIN) key = key < limit ? key : -INFINITY;
#pragma unroll
                for (int d = D - 1; d > 0; d--) m[d] = fmaxf(m[d], min_nan(m[d - 1], key));
                m[0] = fmaxf(m[0], key);
            }
        }
    }
    // The best candidate of the token's lanes leaves: its logit (-inf: there is none) and expert.
    BSQ_DEV float pop(const Row<uint16_t, LPT, Q> &row, int sub, int &e) {
        const float best = group_max<LPT>(m[0]);
        const uint32_t b = __float_as_uint(best);
        e = (int)((b ^ ~(uint32_t)((int32_t)b >> 31)) & 0xFFFFu);
        if (!(best > -INFINITY)) return -INFINITY;
        if (m[0] == best) {
#pragma unroll
            for (int d = 0; d + 1 < D; d++) m[d] = m[d + 1];
            m[D - 1] = -INFINITY;
            if (4 * Q > D && --left == 0) fill<true>(row, sub, best);
        }
        return __uint_as_float(b & 0xFFFF0000u);
    }
};

template <int LPT, int Q>
struct Candidates<float, LPT, Q> {
    static constexpr int D = kDepth<LPT>;
    float m[D];
    int at[D], left;
    template <bool AGAIN>
    BSQ_DEV void fill(const Row<float, LPT, Q> &row, int sub, float limit, int limit_e = 0) {
        left = D;
#pragma unroll
        for (int d = 0; d < D; d++) {
            m[d] = -INFINITY;
            at[d] = 0xFFFF;
        }
#pragma unroll
        for (int q = 0; q < Q; q++) {
            float z[4];
            row.get(q, z);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int e = 4 * (q * LPT + sub) + i;
                float x = z[i];
                if (AGAIN) x = x < limit || (x == limit && e > limit_e) ? x : -INFINITY;
                // a lane's experts come in rising order: equal logits stay behind the earlier one
#pragma unroll
                for (int d = D - 1; d > 0; d--) {
                    at[d] = x > m[d - 1] ? at[d - 1] : x > m[d] ? e : at[d];
                    m[d] = fmaxf(m[d], min_nan(m[d - 1], x));
                }
                at[0] = x > m[0] ? e : at[0];
                m[0] = fmaxf(m[0], x);
            }
        }
    }
    BSQ_DEV float pop(const Row<float, LPT, Q> &row, int sub, int &e) {
        const float best = group_max<LPT>(m[0]);
        // the lowest expert among the lanes that hold this logit
        int cand = m[0] == best ? at[0] : 0xFFFF;
#pragma unroll
        for (int o = LPT / 2; o; o >>= 1) cand = min(cand, __shfl_xor_sync(kFull, cand, o));
        e = cand;
        if (!(best > -INFINITY)) return -INFINITY;
        if (m[0] == best && at[0] == cand) {
#pragma unroll
            for (int d = 0; d + 1 < D; d++) {
                m[d] = m[d + 1];
                at[d] = at[d + 1];
            }
            m[D - 1] = -INFINITY;
            if (4 * Q > D && --left == 0) fill<true>(row, sub, best, cand);
        }
        return best;
    }
};

// For k <= L: a sorted list of the token's L best, built without a branch: a
// lane sorts its logits by networks of maxima and minima, and log2(LPT)
// exchanges merge the lanes' lists (the larger of a[i] and b[L-1-i] are the L
// best of two sorted lists, in bitonic order).  The whole call at 131072x256,
// k = 8: 63 us, with rounds of one maximum each 92; at 64x64 4.4 and 6.2.  The
// entries are logits with the expert in their low bits, as above.
// An fp32 logit gives its lowest ceil(log2 E) bits for it; where two such
// truncated logits meet in the list or at its end, the order is not certain and
// the warp's tokens go through the rounds instead.  NaN entries (-inf logits)
// sink to the end.
BSQ_DEV void order2(float &a, float &b) {
    const float lo = min_nan(a, b);
    a = fmaxf(a, b);
    b = lo;
}
// Batcher's odd-even merge sort, descending, for N = 4 or 8.
template <int N>
BSQ_DEV void sort_desc(float *v) {
#pragma unroll
    for (int p = 1; p < N; p <<= 1)
#pragma unroll
        for (int k = p; k; k >>= 1)
#pragma unroll
            for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; i++)
                    if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) order2(v[i + j], v[i + j + k]);
}
// v becomes the N best of the sorted lists v and w, sorted.
template <int N>
BSQ_DEV void keep_best(float *v, const float *w) {
#pragma unroll
    for (int i = 0; i < N; i++) v[i] = fmaxf(v[i], w[N - 1 - i]);
#pragma unroll
    for (int h = N / 2; h; h >>= 1)
#pragma unroll
        for (int i = 0; i < N; i++)
            if (!(i & h)) order2(v[i], v[i + h]);
}
template <int N>
BSQ_DEV float entry(const float *v, int i) {  // v[i % N]
    float w[N];
#pragma unroll
    for (int j = 0; j < N; j++) w[j] = v[j];
#pragma unroll
    for (int h = 1; h < N; h <<= 1)
#pragma unroll
        for (int j = 0; j < N; j += 2 * h) w[j] = i & h ? w[j + h] : w[j];
    return w[0];
}
template <typename In>
BSQ_DEV uint32_t expert_bits(int E) {
    return sizeof(In) == 2 ? 0xFFFFu : (2u << (31 - __clz(max(E - 1, 1)))) - 1u;
}
BSQ_DEV float with_expert(float z, uint32_t e, uint32_t bits) {
    const uint32_t b = __float_as_uint(__fadd_rn(z, 0.0f));
    return __uint_as_float((b & ~bits) | (e ^ (~(uint32_t)((int32_t)b >> 31) & bits)));
}
BSQ_DEV int expert_of(uint32_t b, uint32_t bits) { return (int)((b ^ ~(uint32_t)((int32_t)b >> 31)) & bits); }

// The token's L best, the same list in all of its lanes.
template <int L, typename In, int LPT, int Q>
BSQ_DEV void best_list(const Row<In, LPT, Q> &row, int sub, uint32_t bits, float v[L]) {
    constexpr int kQuads = L / 4;  // quads that make a list
#pragma unroll
    for (int q0 = 0; q0 < Q; q0 += kQuads) {
        float w[L];
#pragma unroll
        for (int d = 0; d < kQuads; d++) {
            const int q = q0 + d;
            float z[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            if (q < Q) row.get(q, z);
#pragma unroll
            for (int i = 0; i < 4; i++)
                w[4 * d + i] = q < Q ? with_expert(z[i], (uint32_t)(4 * (q * LPT + sub) + i), bits) : -INFINITY;
        }
        sort_desc<L>(w);
        if (q0 == 0) {
#pragma unroll
            for (int i = 0; i < L; i++) v[i] = w[i];
        } else {
            keep_best<L>(v, w);
        }
    }
#pragma unroll
    for (int o = 1; o < LPT; o <<= 1) {
        float w[L];
#pragma unroll
        for (int i = 0; i < L; i++) w[i] = __shfl_xor_sync(kFull, v[i], o);
        keep_best<L>(v, w);
    }
}

// The same for many logits per lane, in two steps: the L quads with the best
// maxima hold the L best logits (a quad before which L others come has L
// logits before each of its own), so lists of quads come first, then lane i
// reads quad i's four logits again, and lists are made of those.  Five and
// more quads a lane: the call takes 63 us instead of 73 at 131072x256, k = 8, 53
// instead of 55 at 131072x160.  The list is that of the lanes sub < L alone.
template <int L, typename In, int LPT, int Q>
BSQ_DEV void best_of_quads(const Row<In, LPT, Q> &row, const In *logits, int sub, int E, bool vec, uint32_t bits,
                           float v[L]) {
    const uint32_t qbits = expert_bits<In>((E + 3) >> 2);
#pragma unroll
    for (int q0 = 0; q0 < Q; q0 += L) {
        float w[L];
#pragma unroll
        for (int i = 0; i < L; i++)
            w[i] = q0 + i < Q ? with_expert(row.quad_max(q0 + i), (uint32_t)((q0 + i) * LPT + sub), qbits) : -INFINITY;
        sort_desc<L>(w);
        if (q0 == 0) {
#pragma unroll
            for (int i = 0; i < L; i++) v[i] = w[i];
        } else {
            keep_best<L>(v, w);
        }
    }
#pragma unroll
    for (int o = 1; o < LPT; o <<= 1) {
        float w[L];
#pragma unroll
        for (int i = 0; i < L; i++) w[i] = __shfl_xor_sync(kFull, v[i], o);
        keep_best<L>(v, w);
    }
    const float mine = entry<L>(v, sub);
    const bool some = sub < L && mine > -INFINITY;
    const int quad = some ? expert_of(__float_as_uint(mine), qbits) : 0;
    Row<In, 1, 1> one;
    one.load(logits + 4 * quad, E - 4 * quad, 0, vec, some);
    float z[4];
    one.get(0, z);
#pragma unroll
    for (int i = 0; i < 4; i++) v[i] = with_expert(z[i], (uint32_t)(4 * quad + i), bits);
    sort_desc<4>(v);
    if (L == 8) {  // two lists of four make one of eight
#pragma unroll
        for (int i = 0; i < 4; i++) v[L - 1 - i] = __shfl_xor_sync(kFull, v[i], 1);
#pragma unroll
        for (int h = L / 2; h; h >>= 1)
#pragma unroll
            for (int i = 0; i < L; i++)
                if (!(i & h)) order2(v[i], v[i + h]);
    }
#pragma unroll
    for (int o = L / 4; o < L; o <<= 1) {
        float w[L];
#pragma unroll
        for (int i = 0; i < L; i++) w[i] = __shfl_xor_sync(kFull, v[i], o);
        keep_best<L>(v, w);
    }
}

// Slot `sub` of the token by such a list: its expert (-1: none) and logit.
// False where the order is not certain.
template <int L, typename In, int LPT, int Q>
BSQ_DEV bool choose(const Row<In, LPT, Q> &row, const In *logits, int sub, int E, bool vec, int k, int &e, float &z) {
    const uint32_t bits = expert_bits<In>(E);
    float v[L];
    if (Q >= 5) best_of_quads<L>(row, logits, sub, E, vec, bits, v);
    else best_list<L>(row, sub, bits, v);
    const float mine = entry<L>(v, sub);
    const uint32_t b = __float_as_uint(mine);
    e = sub < k && mine > -INFINITY ? expert_of(b, bits) : -1;
    if (sizeof(In) == 2) {
        z = __uint_as_float(b & ~bits);
        return true;
    }
    z = e >= 0 ? load_logit(logits + e) : 0.0f;
    const uint32_t next = __shfl_down_sync(kFull, b, 1, LPT);
    bool bad = sub + 1 < k && e >= 0 && ((b ^ next) & ~bits) == 0;
    // the last slot's truncated logit: nothing else may have it
    const float last = __shfl_sync(kFull, entry<L>(v, k - 1), 0, LPT);
    const uint32_t lb = __float_as_uint(last);
    const float least = __uint_as_float((lb >> 31) ? lb | bits : lb & ~bits);
    int n = 0;
#pragma unroll
    for (int q = 0; q < Q; q++) {
        float x[4];
        row.get(q, x);
#pragma unroll
        for (int i = 0; i < 4; i++) n += x[i] >= least;
    }
#pragma unroll
    for (int o = LPT / 2; o; o >>= 1) n += __shfl_xor_sync(kFull, n, o);
    bad |= last > -INFINITY && n != k;
    return !__any_sync(kFull, bad);
}

// Exclusive scan of n[0..E) (PAD128: each rounded up to 128) into off[0..E]
// by the CTA's first warp, 32 consecutive experts at a time.
template <bool PAD128, class Count>
BSQ_DEV void warp_scan(Count n, int E, int32_t *off) {
    const int lane = threadIdx.x & 31;
    int carry = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
        const int e = e0 + lane;
        int v = e < E ? n(e) : 0;
        if (PAD128) v = (v + 127) & ~127;
        int s = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(kFull, s, o);
            if (lane >= o) s += u;
        }
        if (e < E) off[e] = carry + s - v;
        carry += __shfl_sync(kFull, s, 31);
    }
    if (lane == 0) off[E] = carry;
}

// coef E / (k n^2) sum_e c_e sum_t p_te, by divisions of fp32 size.
BSQ_DEV float balance_loss(float weighted, int tokens, float coef, int E, int k) {
    return tokens > 0 ? coef * (float)E * (weighted / (float)tokens) / ((float)k * (float)tokens) : 0.0f;
}

// Bytes of one chunk's row of 8-bit counts (E experts and the tokens).
__host__ __device__ __forceinline__ int hist_row(int E) { return (E + 1 + 3) & ~3; }

struct RouteOut {
    int32_t *ids;
    float *weights;
    int32_t *rows, *row_index, *row_off, *sf_row_off, *counts;
    float *prob_sums, *loss;
};

// The rest of the call by the CTAs of one cluster, 64 tokens each: every one adds
// up all masks' counts, those of the CTAs before it apart, and places its slots.
// Against a second launch: 512x128, k = 8, 7.2 us on the device instead of 8.4 (with
// 1000 experts 25.7 and 25.5), and a launch's host time less.
BSQ_DEV void finish_route(unsigned long long *masks, float *red, int32_t *off, const uint16_t *sel, const float *sel_x,
                          const float *inv, int64_t T, UnitDiv kd, int E, int ctas, int want_p, const RouteOut &out,
                          float coef) {
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, k = (int)kd.d, rank = blockIdx.x;
    const int t0 = rank * kChunk, here = max(0, min(kChunk, (int)T - t0)) * k;
    int32_t *all = off + E + 1, *before = all + E + 1, *first_token = before + E + 1;
    auto sync = [&] {
        if (ctas > 1) cluster.sync();
        else __syncthreads();
    };
    sync();  // masks and sums of all CTAs are there
    for (int e = threadIdx.x; e <= E; e += blockDim.x) {
        int n = 0, b = 0;
        for (int r = 0; r < ctas; r++) {
            const int c = __popcll(cluster.map_shared_rank(masks, r)[e]);
            n += c;
            b += r < rank ? c : 0;
        }
        all[e] = n;
        before[e] = b;
    }
    if (threadIdx.x == 0) *first_token = 0;
    __syncthreads();
    if (warp == 0) warp_scan<false>([&](int e) { return all[e]; }, E, off);
    __syncthreads();
    const int total = off[E];
    for (int i = threadIdx.x; i < here; i += blockDim.x) {
        const int tl = (int)divide((uint32_t)i, kd);
        const int e = (int16_t)sel[i];
        int row = -1;
        if (e >= 0) {
            row = off[e] + before[e] + __popcll(masks[e] & ((1ull << tl) - 1ull));
            out.row_index[row] = t0 + tl;
        }
        out.ids[t0 * k + i] = e;
        out.weights[t0 * k + i] = sel_x[i] * inv[tl];
        out.rows[t0 * k + i] = row;
    }
    if (t0 * k + here > total) {  // rows without a slot repeat the first row's token
        for (int e = threadIdx.x; e < E; e += blockDim.x)
            if (off[e] == 0 && off[e + 1] > 0) {  // one expert has the first row
                int r = 0;
                while (cluster.map_shared_rank(masks, r)[e] == 0) r++;
                *first_token = r * kChunk + __ffsll(cluster.map_shared_rank(masks, r)[e]) - 1;
            }
        __syncthreads();
        for (int i = max(t0 * k, total) + threadIdx.x; i < t0 * k + here; i += blockDim.x)
            out.row_index[i] = *first_token;
    }
    if (rank == 0) {
        __syncthreads();
        float *sums = reinterpret_cast<float *>(before);
        for (int e = threadIdx.x; e <= E; e += blockDim.x) {
            out.counts[e] = all[e];
            out.row_off[e] = off[e];
            if (want_p && e < E) {
                float v = 0.0f;
                for (int r = 0; r < ctas; r++) v += cluster.map_shared_rank(red, r)[e];
                sums[e] = v;
                if (out.prob_sums) out.prob_sums[e] = v;
            }
        }
        __syncthreads();
        if (warp == 0) warp_scan<true>([&](int e) { return all[e]; }, E, out.sf_row_off);
        if (warp == 1 && out.loss) {
            float v = 0.0f;
            for (int e = lane; e < E; e += 32) v += (float)all[e] * sums[e];
            v = warp_sum(v);
            if (lane == 0) *out.loss = balance_loss(v, all[E], coef, E, k);
        }
    }
    sync();  // no CTA leaves while another reads its shared memory
}

// Pass 1.  A CTA takes chunks of kChunk consecutive tokens in turn, LPT lanes a
// token; the sums of probabilities stay in its registers (with 32 fp32 logits a
// lane, 193 to 256 and 385 experts and more, some spill).  The softmax sum runs
// over the same registers as the choice.  The chosen experts go into one 64-bit
// mask of tokens per expert, whose population count is the chunk's count and
// whose bits below a token are that token's rank in the chunk: the order "by
// expert, then token" needs no sort.  Row E of the counts is the number of tokens
// with at least one expert.  With `ctas` > 0 the chunks are one cluster, a CTA
// each, which finishes the call (rows, offsets, loss) from one another's masks and
// sums in shared memory.  L: k <= L by sorted lists; 0: rounds for any k.
// 131072x256, k = 8: three quarters of the call's 63 us.  261 instructions a token; a
// third of the issue slots stay empty, with three CTAs (24 warps) on an SM.
// (The launch bound is there for the registers: 64 where a lane has few logits, so
// that two CTAs of 512 threads share an SM, else 80.)
template <typename In, int LPT, int Q, int L>
__global__ void __launch_bounds__(Q <= 2 ? 1024 : 768)
    route_topk_kernel(const In *__restrict__ logits, int64_t T, int E, int64_t ldl,
                                                         int vec, const uint8_t *__restrict__ mask, UnitDiv kd,
                                                         int renorm, int want_p, int ctas, RouteOut out, int64_t nchunk,
                                                         uint8_t *__restrict__ hist, float *__restrict__ psum,
                                                         float coef) {
    grid_dependents_launch();
    grid_dependency_wait();
    extern __shared__ unsigned long long smem[];
    const int k = (int)kd.d, nwarps = blockDim.x >> 5;
    unsigned int *words = reinterpret_cast<unsigned int *>(smem);      // [(E + 1) * 2]
    float *sel_x = reinterpret_cast<float *>(words + 2 * (E + 1));     // [kChunk][k] exp(logit - top)
    float *inv = sel_x + kChunk * k;                                   // [kChunk]
    float *red = inv + kChunk;                                         // [nwarps][E] when want_p
    int32_t *off = reinterpret_cast<int32_t *>(red + (want_p ? nwarps * E : 0));  // 3 [E + 1] + 1 when ctas > 0
    uint16_t *sel = reinterpret_cast<uint16_t *>(off + (ctas ? 3 * (E + 1) + 1 : 0));  // [kChunk][k]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % LPT;
    constexpr int kGroups = 32 / LPT;
    auto pick = [&](int tl, int j, int e, float x) {
        sel[tl * k + j] = (uint16_t)e;
        sel_x[tl * k + j] = x;
        if (e >= 0) atomicOr(&words[2 * e + (tl >> 5)], 1u << (tl & 31));
        if (j == 0 && e >= 0) atomicOr(&words[2 * E + (tl >> 5)], 1u << (tl & 31));
    };
    f32x2 acc[Q][2];
#pragma unroll
    for (int q = 0; q < Q; q++) acc[q][0] = acc[q][1] = f2_pack(0.0f, 0.0f);
    for (int i = threadIdx.x; i < 2 * (E + 1); i += blockDim.x) words[i] = 0;
    __syncthreads();
    for (int64_t chunk = blockIdx.x; chunk < nchunk; chunk += gridDim.x) {
        const int64_t t0 = chunk * kChunk;
        const int here = (int)min((int64_t)kChunk, T - t0);
        for (int w0 = warp * kGroups; w0 < here; w0 += nwarps * kGroups) {
            const int tl = w0 + lane / LPT;
            const bool in = tl < here;
            const bool live = in && (!mask || __ldg(mask + t0 + tl) != 0);
            Row<In, LPT, Q> row;
            row.load(logits + (t0 + tl) * ldl, E, sub, vec, live);
            float top = 0.0f, chosen = 0.0f;
            bool done = false;
            if (L > 0) {
                int e;
                float z;
                done = choose<L == 0 ? 4 : L>(row, logits + (t0 + tl) * ldl, sub, E, vec, k, e, z);
                if (done) {  // the same for the whole warp
                    top = __shfl_sync(kFull, e >= 0 ? z : 0.0f, lane & ~(LPT - 1));
                    const float x = e >= 0 ? exp_of(z - top) : 0.0f;
                    chosen = group_sum<LPT>(x);
                    if (in && sub < k) pick(tl, sub, e, x);
                }
            }
            if (!done) {
                Candidates<In, LPT, Q> c;
                c.template fill<false>(row, sub, 0.0f);
                for (int j0 = 0; j0 < k; j0 += LPT) {
                    int my_e = -1;
                    float my_x = 0.0f;
                    for (int j = j0; j < min(k, j0 + LPT); j++) {
                        int e;
                        const float z = c.pop(row, sub, e);
                        const bool ok = z > -INFINITY;
                        if (j == 0 && ok) top = z;
                        const float x = ok ? exp_of(z - top) : 0.0f;
                        chosen += x;
                        if (ok && sub == j - j0) {
                            my_e = e;
                            my_x = x;
                        }
                    }
                    if (in && j0 + sub < k) pick(tl, j0 + sub, my_e, my_x);  // a lane per slot
                }
            }
            if (want_p || !renorm) {
                const f32x2 top2 = f2_pack(top, top);
                f32x2 s2 = f2_pack(0.0f, 0.0f), p[Q][2];
#pragma unroll
                for (int q = 0; q < Q; q++) {
                    float x[4];
                    row.get(q, x);
                    exp_below4(x, top2);
                    p[q][0] = f2_pack(x[0], x[1]);
                    p[q][1] = f2_pack(x[2], x[3]);
                    s2 = f2_add(s2, f2_add(p[q][0], p[q][1]));
                }
                float s, s_odd;
                f2_unpack(s2, s, s_odd);
                s = group_sum<LPT>(s + s_odd);
                const float r = s > 0.0f ? rcp(s) : 0.0f;
                const f32x2 r2 = f2_pack(r, r);
                if (want_p)
#pragma unroll
                    for (int q = 0; q < Q; q++) {
                        acc[q][0] = f2_fma(p[q][0], r2, acc[q][0]);
                        acc[q][1] = f2_fma(p[q][1], r2, acc[q][1]);
                    }
                if (!renorm) chosen = s;
            }
            if (in && sub == 0) inv[tl] = chosen > 0.0f ? rcp(chosen) : 0.0f;
        }
        __syncthreads();
        if (ctas) break;
        for (int i = threadIdx.x; i < here * k; i += blockDim.x) {
            const int tl = (int)divide((uint32_t)i, kd);
            const int e = (int16_t)sel[i];
            out.ids[t0 * k + i] = e;
            out.weights[t0 * k + i] = sel_x[i] * inv[tl];
            out.rows[t0 * k + i] = e < 0 ? -1 : __popcll(smem[e] & ((1ull << tl) - 1ull));
        }
        // a row of counts and a row of first tokens per chunk
        uint8_t *to = hist + chunk * 2 * hist_row(E);
        for (int e = threadIdx.x; e <= E; e += blockDim.x) {
            const unsigned long long m = smem[e];
            to[e] = (uint8_t)__popcll(m);
            to[hist_row(E) + e] = (uint8_t)(m ? __ffsll(m) - 1 : 0);
        }
        if (chunk + gridDim.x < nchunk) {
            __syncthreads();
            for (int i = threadIdx.x; i < 2 * (E + 1); i += blockDim.x) words[i] = 0;
            __syncthreads();
        }
    }
    if (want_p) {
#pragma unroll
        for (int q = 0; q < Q; q++) {
            float a4[4];
            f2_unpack(acc[q][0], a4[0], a4[1]);
            f2_unpack(acc[q][1], a4[2], a4[3]);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                float v = a4[i];
#pragma unroll
                for (int o = LPT; o < 32; o <<= 1) v += __shfl_xor_sync(kFull, v, o);
                const int e = 4 * (q * LPT + sub) + i;
                if (lane < LPT && e < E) red[warp * E + e] = v;
            }
        }
        __syncthreads();
    }
    if (want_p)
        for (int e = threadIdx.x; e < E; e += blockDim.x) {
            float v = 0.0f;
            for (int w = 0; w < nwarps; w++) v += red[w * E + e];
            if (ctas) red[e] = v;  // this thread's own column
            else psum[(int64_t)blockIdx.x * E + e] = v;
        }
    if (ctas) finish_route(smem, red, off, sel, sel_x, inv, T, kd, E, ctas, want_p, out, coef);
}

// Pass 2, for many chunks.  A CTA takes kBlock consecutive chunks and 32 experts
// (row E, the tokens, among them), a lane one expert and a warp a run of the
// chunks, all loads in flight at once: the exclusive prefix of every chunk
// inside the block, and the block's counts.  The first pass's rows of sums of
// probabilities are added up along the way, spread over the blocks.
constexpr int kBlock = 64, kRun = kBlock / 8;

__global__ void __launch_bounds__(256) route_block_kernel(const uint8_t *__restrict__ hist,
                                                          const float *__restrict__ psum, int64_t rows, int64_t nchunk,
                                                          int E, uint16_t *__restrict__ prefix,
                                                          int32_t *__restrict__ count,
                                                          float *__restrict__ psum_block) {
    grid_dependents_launch();
    grid_dependency_wait();
    __shared__ int run[8][32];
    __shared__ float fsum[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int e = blockIdx.y * 32 + lane, row = hist_row(E);
    const int64_t c = (int64_t)blockIdx.x * kBlock + warp * kRun;
    int v[kRun], n = 0;
    float p = 0.0f;
#pragma unroll
    for (int i = 0; i < kRun; i++) v[i] = c + i < nchunk && e <= E ? __ldg(hist + (c + i) * 2 * row + e) : 0;
    if (psum && e < E)
#pragma unroll 4
        for (int64_t i = blockIdx.x + (int64_t)warp * gridDim.x; i < rows; i += 8 * (int64_t)gridDim.x)
            p += __ldg(psum + i * E + e);
#pragma unroll
    for (int i = 0; i < kRun; i++) n += v[i];
    run[warp][lane] = n;
    fsum[warp][lane] = p;
    __syncthreads();
    int at = 0;
    for (int w = 0; w < warp; w++) at += run[w][lane];
    if (e > E) return;
    if (warp == 7) {
        count[(int64_t)blockIdx.x * (E + 1) + e] = at + n;
        if (e < E && psum) {
            float all = 0.0f;
#pragma unroll
            for (int w = 0; w < 8; w++) all += fsum[w][lane];
            psum_block[(int64_t)blockIdx.x * E + e] = all;
        }
    }
    if (e == E) return;
#pragma unroll
    for (int i = 0; i < kRun; i++) {
        if (c + i < nchunk) prefix[(c + i) * E + e] = (uint16_t)at;  // 64 chunks of 64 tokens
        at += v[i];
    }
}

// Sum of n values `stride` apart, 16 loads in flight; *part that of the first m.
// (n stride < 2^31: a block of 4096 tokens has at most 1025 values.)
template <typename V>
BSQ_DEV V column_sum(const V *p, int stride, int n, int m, V *part) {
    V s = 0, first = 0;
    for (int b = 0; b < n; b += 16, p += 16 * stride) {
        V v[16];
#pragma unroll
        for (int i = 0; i < 16; i++) v[i] = b + i < n ? __ldg(p + i * stride) : V(0);
#pragma unroll
        for (int i = 0; i < 16; i++) {
            s += v[i];
            if (b + i < m) first += v[i];
        }
    }
    *part = first;
    return s;
}

// Exclusive scan of n[0..E), E <= 1024, into off[0..E] by a CTA of 256
// threads, four neighbouring experts each.
BSQ_DEV void cta_scan(const int32_t *n, int E, int32_t *off, int *wsum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e0 = threadIdx.x * 4;
    int v[4], s = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        v[i] = e0 + i < E ? n[e0 + i] : 0;
        s += v[i];
    }
    int inc = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFull, inc, o);
        if (lane >= o) inc += u;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    int at = inc - s;
    for (int w = 0; w < warp; w++) at += wsum[w];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        if (e0 + i <= E) off[e0 + i] = at;
        at += v[i];
    }
    if (E == 1024 && threadIdx.x == 255) off[E] = at;
    __syncthreads();
}

// Pass 3.  Row of a slot = its expert's offset + the prefix of the blocks
// before + the chunk's prefix in its block + the rank inside the chunk; the
// rows past the last routed one repeat the first row's token.  A CTA takes
// `span` chunks of one block; one more writes the offsets and the loss.
__global__ void __launch_bounds__(256) route_place_kernel(int64_t T, UnitDiv kd, int E, int64_t nchunk, int span,
                                                          const uint8_t *__restrict__ hist,
                                                          const uint16_t *__restrict__ prefix,
                                                          const int32_t *__restrict__ count,
                                                          const float *__restrict__ psum_block, RouteOut out,
                                                          float coef) {
    grid_dependents_launch();
    grid_dependency_wait();
    __shared__ int32_t base[kRouteMaxExperts], all[kRouteMaxExperts + 1], off[kRouteMaxExperts + 1];
    __shared__ float sums[kRouteMaxExperts];
    __shared__ int wsum[8], first_chunk;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t blocks = gridDim.x - 1, b = blockIdx.x;  // the last column's first CTA has no chunks
    if (b == blocks && blockIdx.y > 0) return;
    const int64_t c0 = min(b * kBlock + blockIdx.y * span, nchunk);
    const int64_t c1 = max(c0, min(min(c0 + span, (b + 1) * kBlock), nchunk));
    const uint32_t k = kd.d, i0 = (uint32_t)(min(c0 * kChunk, T) * k);  // slots i0 .. i0 + here, below 2^31
    const int here = (int)((min(c1 * kChunk, T) - min(c0 * kChunk, T)) * k);
    const uint16_t *at = prefix + c0 * E;
    for (int e = threadIdx.x; e < E; e += 256) {
        int before;
        all[e] = column_sum(count + e, E + 1, (int)blocks, (int)b, &before);
        base[e] = before;
    }
    __syncthreads();
    cta_scan(all, E, off, wsum);
    for (int e = threadIdx.x; e < E; e += 256) base[e] += off[e];
    const int total = off[E];
    __syncthreads();
    // four slots at a time, so that their loads overlap
    for (int x0 = threadIdx.x; x0 < here; x0 += 1024) {
        int e[4], r[4];
        uint32_t t[4];
#pragma unroll
        for (int u = 0; u < 4; u++) {
            const int x = x0 + 256 * u;
            e[u] = x < here ? __ldg(out.ids + i0 + x) : -1;
            r[u] = x < here ? out.rows[i0 + x] : 0;
            t[u] = divide(x, kd);
        }
#pragma unroll
        for (int u = 0; u < 4; u++)
            if (e[u] >= 0) r[u] += base[e[u]] + __ldg(at + (t[u] / kChunk) * E + e[u]);
#pragma unroll
        for (int u = 0; u < 4; u++) {
            if (e[u] < 0) continue;
            out.rows[i0 + x0 + 256 * u] = r[u];
            out.row_index[r[u]] = (int)(c0 * kChunk) + (int)t[u];
        }
    }
    if (here > 0 && (int64_t)i0 + here > total) {
        int token = 0;
        if (total > 0) {  // the first chunk that has the first row's expert, and its first token there
            int e0 = 0;
            while (all[e0] == 0) e0++;
            int64_t b0 = 0;
            while (__ldg(count + b0 * (E + 1) + e0) == 0) b0++;
            if (threadIdx.x == 0) first_chunk = kBlock;
            __syncthreads();
            if (threadIdx.x < kBlock && b0 * kBlock + threadIdx.x < nchunk &&
                __ldg(hist + (b0 * kBlock + threadIdx.x) * 2 * hist_row(E) + e0))
                atomicMin(&first_chunk, (int)threadIdx.x);
            __syncthreads();
            const int64_t c = b0 * kBlock + first_chunk;
            token = (int)(c * kChunk) + __ldg(hist + c * 2 * hist_row(E) + hist_row(E) + e0);
        }
        for (int x = threadIdx.x; x < here; x += 256)
            if ((int64_t)i0 + x >= total) out.row_index[i0 + x] = token;
    }
    if (b < blocks) return;
    for (int e = threadIdx.x; e <= E; e += 256) {
        int none;
        if (e == E) all[E] = column_sum(count + E, E + 1, (int)blocks, 0, &none);
        out.counts[e] = all[e];
        out.row_off[e] = off[e];
        if (psum_block && e < E) {
            float part;
            sums[e] = column_sum(psum_block + e, E, (int)blocks, 0, &part);
            if (out.prob_sums) out.prob_sums[e] = sums[e];
        }
    }
    __syncthreads();
    if (warp == 0) warp_scan<true>([&](int e) { return all[e]; }, E, out.sf_row_off);
    if (warp == 1 && out.loss) {
        float v = 0.0f;
        for (int e = lane; e < E; e += 32) v += (float)all[e] * sums[e];
        v = warp_sum(v);
        if (lane == 0) *out.loss = balance_loss(v, all[E], coef, E, (int)k);
    }
}

// Passes 2 and 3 in one launch, for few chunks: a CTA per chunk adds up all
// chunks' 8-bit counts (kSmallHist bytes at most, from L2), those before its own
// apart, which gives the experts' offsets and its own prefix, and places its
// slots.  Three bytes are added before they are widened (64 a chunk), and two
// counts share a 32-bit sum (512 chunks at most).  One more CTA writes the
// offsets, the sums of the probabilities and the loss.  The whole call against
// passes 2 and 3 apart: 8.7 and 9.3 us at 2048x128 (4 KB of counts), 13.6 and 13.9
// at 16384x64 (17 KB); nearer the limit the passes apart are the faster ones, 15.1
// and 12.9 at 16384x96 (26 KB), 24.5 and 16.0 at 16384x160 (42 KB).
constexpr int kSmallHist = 48 * 1024, kSmallChunks = 512;

__global__ void __launch_bounds__(256) route_scan_place_kernel(int64_t T, UnitDiv kd, int E, int nchunk,
                                                               UnitDiv wd, const uint8_t *__restrict__ hist,
                                                               const float *__restrict__ psum, int64_t rows,
                                                               RouteOut out,
                                                               float coef) {
    grid_dependents_launch();
    grid_dependency_wait();
    // counts of the chunks before this one, and of this one and the ones after it
    __shared__ int32_t before[kRouteMaxExperts + 4], rest[kRouteMaxExperts + 4], off[kRouteMaxExperts + 1];
    __shared__ float sums[kRouteMaxExperts];
    __shared__ int first_chunk;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, k = (int)kd.d;
    const int row = hist_row(E), words = (int)wd.d, chunk = blockIdx.x;
    const uint32_t slot0 = (uint32_t)chunk * kChunk * k;
    const int here = (int)max((int64_t)0, min((int64_t)kChunk, T - (int64_t)chunk * kChunk)) * k;
    // this chunk's slots, read ahead of the sums
    int e_s[2], rank_s[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const int j = threadIdx.x + 256 * i;
        e_s[i] = j < here ? out.ids[slot0 + j] : -1;
        rank_s[i] = j < here ? out.rows[slot0 + j] : 0;
    }
    for (int e = threadIdx.x; e < row; e += 256) before[e] = rest[e] = 0;
    if (threadIdx.x == 0) first_chunk = nchunk;
    if (chunk == nchunk && psum) {
        // 16 rows of partial sums in flight per thread; E <= 256 here: 256 / E threads share an expert
        __shared__ float part[256];
        const int parts = 256 / E, e = threadIdx.x % E, g = threadIdx.x / E;
        float p = 0.0f;
        if (g < parts)
            for (int c0 = g; c0 < rows; c0 += 16 * parts) {
                float v[16];
#pragma unroll
                for (int i = 0; i < 16; i++) {
                    const int c = c0 + i * parts;
                    v[i] = c < rows ? __ldg(psum + c * E + e) : 0.0f;
                }
#pragma unroll
                for (int i = 0; i < 16; i++) p += v[i];
            }
        part[threadIdx.x] = p;
        __syncthreads();
        if (threadIdx.x < E) {
            for (int i = 1; i < parts; i++) p += part[threadIdx.x + i * E];
            sums[threadIdx.x] = p;
            if (out.prob_sums) out.prob_sums[threadIdx.x] = p;
        }
    }
    __syncthreads();
    const int parts = max(1, 256 / words);  // threads that share a word, each with every parts-th chunk
    for (int u = threadIdx.x; u < words * parts; u += 256) {
        const int part = (int)divide((uint32_t)u, wd), w = u - part * words;
        auto add_up = [&](int c0, int c1, int32_t *to) {
            const uint32_t *p = reinterpret_cast<const uint32_t *>(hist) + w;
            uint32_t even = 0, odd = 0;
            const int step = parts * 2 * words;
            p += (c0 + part) * 2 * words;
            int left = c1 - c0 - part;  // rows of this thread: every parts-th of them
            for (; left > 5 * parts; left -= 6 * parts, p += 6 * step) {
                const uint32_t x0 = __ldg(p), x1 = __ldg(p + step), x2 = __ldg(p + 2 * step), x3 = __ldg(p + 3 * step),
                               x4 = __ldg(p + 4 * step), x5 = __ldg(p + 5 * step);
                const uint32_t y = x0 + x1 + x2, z = x3 + x4 + x5;
                even += (y & 0x00FF00FFu) + (z & 0x00FF00FFu);
                odd += ((y >> 8) & 0x00FF00FFu) + ((z >> 8) & 0x00FF00FFu);
            }
            for (; left > 0; left -= parts, p += step) {
                const uint32_t x = __ldg(p);
                even += x & 0x00FF00FFu;
                odd += (x >> 8) & 0x00FF00FFu;
            }
            if (even & 0xFFFFu) atomicAdd(to + 4 * w, (int)(even & 0xFFFFu));
            if (odd & 0xFFFFu) atomicAdd(to + 4 * w + 1, (int)(odd & 0xFFFFu));
            if (even >> 16) atomicAdd(to + 4 * w + 2, (int)(even >> 16));
            if (odd >> 16) atomicAdd(to + 4 * w + 3, (int)(odd >> 16));
        };
        add_up(0, chunk, before);
        add_up(chunk, nchunk, rest);
    }
    __syncthreads();
    if (warp == 0) warp_scan<false>([&](int e) { return before[e] + rest[e]; }, E, off);
    __syncthreads();
    const int total = off[E];
    for (int j = threadIdx.x, i = 0; j < here; j += 256, i++) {
        const int e = i < 2 ? e_s[i] : out.ids[slot0 + j];
        if (e < 0) continue;
        const int r = off[e] + before[e] + (i < 2 ? rank_s[i] : out.rows[slot0 + j]);
        out.rows[slot0 + j] = r;
        out.row_index[r] = chunk * kChunk + (int)divide((uint32_t)j, kd);
    }
    if (here > 0 && (int64_t)slot0 + here > total) {  // rows without a slot repeat the first row's token
        int token = 0;
        if (total > 0) {
            int e0 = 0;
            while (off[e0 + 1] == 0) e0++;
            for (int c = threadIdx.x; c < nchunk; c += 256)
                if (hist[c * 2 * row + e0]) {
                    atomicMin(&first_chunk, c);
                    break;
                }
            __syncthreads();
            token = first_chunk * kChunk + hist[first_chunk * 2 * row + row + e0];
        }
        for (int j = threadIdx.x; j < here; j += 256)
            if ((int)slot0 + j >= total) out.row_index[slot0 + j] = token;
    }
    if (chunk < nchunk) return;
    // the CTA past the chunks: `before` holds the counts
    for (int e = threadIdx.x; e <= E; e += 256) {
        out.counts[e] = before[e];
        out.row_off[e] = off[e];
    }
    if (warp == 0) warp_scan<true>([&](int e) { return before[e]; }, E, out.sf_row_off);
    if (warp == 1 && out.loss) {
        float v = 0.0f;
        for (int e = lane; e < E; e += 32) v += (float)before[e] * sums[e];
        v = warp_sum(v);
        if (lane == 0) *out.loss = balance_loss(v, before[E], coef, E, k);
    }
}

// ------------------------------------------------------------------ router, backward
BSQ_DEV void store4(float *p, const float d[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(d[0], d[1], d[2], d[3]);
}
BSQ_DEV void store4(uint16_t *p, const float d[4]) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(d[0], d[1]), pack_bf16(d[2], d[3]));
}

// A row of E values by LPT lanes, at any alignment of whole elements.
template <int LPT>
BSQ_DEV void store_row(float *to, const float *row, int E, int sub) {
    for (int e = sub; e < E; e += LPT) to[e] = row[e];
}
template <int LPT>
BSQ_DEV void store_row(uint16_t *to, const float *row, int E, int sub) {
    const int mid = (reinterpret_cast<uintptr_t>(to) & 2u) ? 1 : 0;  // words of elements (2i - mid, 2i + 1 - mid)
    for (int e = 2 * sub - mid; e < E; e += 2 * LPT) {
        if (e >= 0 && e + 1 < E) *reinterpret_cast<uint32_t *>(to + e) = pack_bf16(row[e], row[e + 1]);
        else if (e >= 0) store_logit(to + e, row[e]);
        else store_logit(to, row[0]);
    }
}

// CTAs per SM, and the grid is no larger: five at 48 registers where a lane's
// logits leave that many free, six where the softmax is not needed (shared
// memory).  With eight CTAs per SM in turns, 131072x256 takes 37 us instead of 34
// and 100003x160 19.9 instead of 18.7 (bf16; fp32 logits at 131072x256 48 instead
// of 53).
template <int Q, bool NEED_P>
constexpr int bwd_ctas() {
    return !NEED_P ? 6 : Q <= 5 ? 5 : 3;
}

// LPT lanes per token.  With q the weights' distribution (the softmax over all
// experts, or over the chosen ones) and a_e = dL/dweight of expert e (zero
// where it was not chosen): dz_e = q_e (a_e - sum q a).  The balance loss adds
// the softmax's gradient of sum_e b_e p_e with b_e = dloss coef E c_e / (k n^2),
// kept in shared memory for the CTA.  The chosen experts' own terms reach the
// lanes that hold those experts through a row of shared memory per token,
// which is zero between tokens.
template <typename In, int LPT, int Q, bool NEED_P>
__global__ void __launch_bounds__(256, bwd_ctas<Q, NEED_P>())
    route_bwd_kernel(const In *__restrict__ logits, int64_t T, int E, int64_t ldl, int vec, int k, int renorm,
                     const int32_t *__restrict__ ids, const float *__restrict__ weights,
                     const float *__restrict__ dweights, const int32_t *__restrict__ counts, float coef,
                     const float *__restrict__ dloss, In *__restrict__ dlogits, int64_t ldd) {
    grid_dependents_launch();
    grid_dependency_wait();
    constexpr int kGroups = 32 / LPT, kCols = 4 * LPT * Q;
    // rows 32 bytes apart in the banks, for the groups' reads of single values
    __shared__ __align__(16) float own_rows[8 * kGroups][kCols + 8];
    __shared__ __align__(16) float bias[NEED_P ? kCols : 4];
    const int lane = threadIdx.x & 31, sub = lane % LPT;
    const int group = threadIdx.x / LPT;
    float *own_row = own_rows[group];
    for (int e = sub; e < kCols; e += LPT) own_row[e] = 0.0f;
    if (NEED_P) {
        float bscale = 0.0f;
        if (dloss) {
            const int n = __ldg(counts + E);
            bscale = n > 0 ? __ldg(dloss) * coef * (float)E / (float)n / ((float)k * (float)n) : 0.0f;
        }
        for (int e = threadIdx.x; e < kCols; e += 256)
            bias[e] = dloss && e < E ? bscale * (float)__ldg(counts + e) : 0.0f;
    }
    __syncthreads();
    const int64_t stride = (int64_t)gridDim.x * 8 * kGroups;
    // a warp's tokens start together: the shuffles want whole warps
    for (int64_t t0 = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * kGroups; t0 < T; t0 += stride) {
        const int64_t t = t0 + lane / LPT;
        const bool in = t < T;
        Row<In, LPT, Q> row;
        if (NEED_P) row.load(logits + t * ldl, E, sub, vec, in);  // in flight with the choice
        // slot sub in registers, slots sub + LPT, ... (k > LPT) by the loops
        const uint32_t slot = (uint32_t)t * (uint32_t)k + sub;  // T k < 2^31
        int e0 = -1;
        float w0 = 0.0f, a0 = 0.0f;
        if (in && sub < k) {
            e0 = __ldg(ids + slot);
            if (dweights) {
                w0 = __ldg(weights + slot);
                a0 = __ldg(dweights + slot);
            }
        }
        const bool has = (unsigned)e0 < (unsigned)E;
        bool live = has;
        float dot = has ? w0 * a0 : 0.0f;
        for (int j = LPT; sub + j < k; j += LPT) {
            const int e = in ? __ldg(ids + slot + j) : -1;
            if ((unsigned)e >= (unsigned)E) continue;
            live = true;
            if (dweights) dot = fmaf(__ldg(weights + slot + j), __ldg(dweights + slot + j), dot);
        }
        const unsigned any = __ballot_sync(kFull, live);
        const unsigned mine = LPT == 32 ? kFull : ((1u << (LPT & 31)) - 1u) << (lane & ~(LPT - 1));
        live = (any & mine) != 0;
        if (NEED_P && !live) row.clear();  // a masked token's logits may be anything
        dot = group_sum<LPT>(dot);  // sum over the chosen of q a: both kinds of q have q_ej = w_j
        // the chosen experts' own term: w_j (a_j - dot), or w_j a_j where dot goes over all experts
        const float all = renorm ? dot : 0.0f;
        if (dweights) {
            if (has) own_row[e0] = w0 * (a0 - all);
            for (int j = LPT; sub + j < k; j += LPT) {
                const int e = in ? __ldg(ids + slot + j) : -1;
                if ((unsigned)e < (unsigned)E)
                    own_row[e] = __ldg(weights + slot + j) * (__ldg(dweights + slot + j) - all);
            }
        }
        float d[Q][4], sub_all = 0.0f, inv = 0.0f;
        if (NEED_P) {
            float top = -INFINITY;
#pragma unroll
            for (int q = 0; q < Q; q++) {
                row.get(q, d[q]);
                top = fmaxf(fmaxf(top, fmaxf(d[q][0], d[q][1])), fmaxf(d[q][2], d[q][3]));
            }
            top = group_max<LPT>(top);
            if (!(top > -INFINITY)) top = 0.0f;
            const f32x2 top2 = f2_pack(top, top);
            f32x2 s2 = f2_pack(0.0f, 0.0f), pb2 = s2;
#pragma unroll
            for (int q = 0; q < Q; q++) {
                exp_below4(d[q], top2);
                const float4 b = *reinterpret_cast<const float4 *>(bias + 4 * (q * LPT + sub));
                const f32x2 p0 = f2_pack(d[q][0], d[q][1]), p1 = f2_pack(d[q][2], d[q][3]);
                s2 = f2_add(s2, f2_add(p0, p1));
                pb2 = f2_fma(p0, f2_pack(b.x, b.y), f2_fma(p1, f2_pack(b.z, b.w), pb2));
            }
            float s, pb, odd;
            f2_unpack(s2, s, odd);
            s = group_sum<LPT>(s + odd);
            inv = s > 0.0f ? rcp(s) : 0.0f;
            f2_unpack(pb2, pb, odd);
            sub_all = group_sum<LPT>(pb + odd) * inv + (renorm ? 0.0f : dot);
        }
        __syncwarp();
        const f32x2 inv2 = f2_pack(inv, inv), sub2 = f2_pack(sub_all, sub_all);
#pragma unroll
        for (int q = 0; q < Q; q++) {
            const int e = 4 * (q * LPT + sub);
            const float4 o = *reinterpret_cast<const float4 *>(own_row + e);
            if (NEED_P) {
                const float4 b = *reinterpret_cast<const float4 *>(bias + e);
                const f32x2 p0 = f2_mul(f2_pack(d[q][0], d[q][1]), inv2), p1 = f2_mul(f2_pack(d[q][2], d[q][3]), inv2);
                f2_unpack(f2_fma(p0, f2_sub(f2_pack(b.x, b.y), sub2), f2_pack(o.x, o.y)), d[q][0], d[q][1]);
                f2_unpack(f2_fma(p1, f2_sub(f2_pack(b.z, b.w), sub2), f2_pack(o.z, o.w)), d[q][2], d[q][3]);
            } else {
                d[q][0] = o.x;
                d[q][1] = o.y;
                d[q][2] = o.z;
                d[q][3] = o.w;
            }
            if (vec && in && e < E) store4(dlogits + t * ldd + e, d[q]);
        }
        if (!vec) {  // the row's values go through its shared memory, to be written side by side
#pragma unroll
            for (int q = 0; q < Q; q++)
                *reinterpret_cast<float4 *>(own_row + 4 * (q * LPT + sub)) =
                    make_float4(d[q][0], d[q][1], d[q][2], d[q][3]);
            __syncwarp();
            if (in) store_row<LPT>(dlogits + t * ldd, own_row, E, sub);
            __syncwarp();
#pragma unroll
            for (int q = 0; q < Q; q++)
                *reinterpret_cast<float4 *>(own_row + 4 * (q * LPT + sub)) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            __syncwarp();
            continue;
        }
        __syncwarp();
        if (dweights) {
            if (has) own_row[e0] = 0.0f;
            for (int j = LPT; sub + j < k; j += LPT) {
                const int e = in ? __ldg(ids + slot + j) : -1;
                if ((unsigned)e < (unsigned)E) own_row[e] = 0.0f;
            }
        }
        __syncwarp();
    }
}

// ------------------------------------------------------------------ combine
// out[t] = sum_j w_tj y[rows_tj]: a CTA of 128 threads takes 1024 columns of
// one token, each thread eight of them over all k rows.  Memory bound:
// 16384x8x4096 takes 185 us, the measured copy rate.  B rows in flight: with one it
// takes 201 us; k = 2 with B = 4, half of them empty, 76 us at 16384x2x4096 instead of 70.
template <int B>
__global__ void __launch_bounds__(128) combine_kernel(const uint16_t *__restrict__ y, int64_t R, int64_t H, int64_t ldy,
                                                      const int32_t *__restrict__ rows,
                                                      const float *__restrict__ weights, int k,
                                                      uint16_t *__restrict__ out, int64_t ldo) {
    grid_dependents_launch();
    grid_dependency_wait();
    const int64_t t = blockIdx.x;
    const int64_t c = ((int64_t)blockIdx.y * 128 + threadIdx.x) * 8;
    if (c >= H) return;
    f32x2 acc[4];
#pragma unroll
    for (int i = 0; i < 4; i++) acc[i] = f2_pack(0.0f, 0.0f);
    rows += t * k;
    if (weights) weights += t * k;
    for (int j0 = 0; j0 < k; j0 += B) {  // B rows in flight
        uint4 q[B];
        float w[B];
#pragma unroll
        for (int j = 0; j < B; j++) {
            const int64_t r = j0 + j < k ? __ldg(rows + j0 + j) : -1;
            const bool has = r >= 0 && r < R;
            w[j] = !has ? 0.0f : weights ? __ldg(weights + j0 + j) : 1.0f;
            q[j] = has ? __ldg(reinterpret_cast<const uint4 *>(y + r * ldy + c)) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int j = 0; j < B; j++) {
            const uint32_t v[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
            const f32x2 w2 = f2_pack(w[j], w[j]);
#pragma unroll
            for (int i = 0; i < 4; i++) acc[i] = f2_fma(w2, f2_pack(bf16_lo(v[i]), bf16_hi(v[i])), acc[i]);
        }
    }
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        float lo, hi;
        f2_unpack(acc[i], lo, hi);
        o[i] = pack_bf16(lo, hi);
    }
    *reinterpret_cast<uint4 *>(out + t * ldo + c) = make_uint4(o[0], o[1], o[2], o[3]);
}

// 2^(code - 127) of an E8M0 code (0: 2^-127, a subnormal).
BSQ_DEV float e8m0_value(uint32_t code) { return __uint_as_float(code ? code << 23 : 0x00400000u); }

// 16 E4M3 codes as fp32 pairs, without their block's scale.
BSQ_DEV void e4m3x16(uint4 q, f32x2 v[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        float a, b, c, d;
        e4m3x2_to_f32(w[i] & 0xFFFFu, a, b);
        e4m3x2_to_f32(w[i] >> 16, c, d);
        v[2 * i] = f2_pack(a, b);
        v[2 * i + 1] = f2_pack(c, d);
    }
}

// Eight columns: the dot product's terms, and w times dout in bf16.
BSQ_DEV void bwd8(uint4 dq, const f32x2 v[4], f32x2 w2, f32x2 &dot2, uint16_t *to) {
    const uint32_t d[4] = {dq.x, dq.y, dq.z, dq.w};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const f32x2 d2 = f2_pack(bf16_lo(d[i]), bf16_hi(d[i]));
        dot2 = f2_fma(d2, v[i], dot2);
        float a, b;
        f2_unpack(f2_mul(d2, w2), a, b);
        o[i] = pack_bf16(a, b);
    }
    *reinterpret_cast<uint4 *>(to) = make_uint4(o[0], o[1], o[2], o[3]);
}

// dy[rows_tj] = w_tj dout_t and dw_tj = <dout_t, y[rows_tj]>: one warp per
// slot, so that empty slots cost nothing and no sum leaves the warp; a
// token's dout is read from DRAM by one of its warps and by the others from
// L1.  Memory bound: y read once, dy written once.  16384x8x4096: 351 us, the
// measured copy rate (354 with eight warps a CTA instead of four); from 8-bit rows
// 310 us (321).
template <bool MX>
__global__ void __launch_bounds__(128) combine_bwd_kernel(const uint16_t *__restrict__ dout, int64_t ldo,
                                                          const uint16_t *__restrict__ y, int64_t ldy,
                                                          const uint8_t *__restrict__ codes,
                                                          const uint8_t *__restrict__ sf, int64_t R, int64_t H,
                                                          const int32_t *__restrict__ rows,
                                                          const float *__restrict__ weights, uint32_t slots, UnitDiv k,
                                                          uint16_t *__restrict__ dy, int64_t lddy,
                                                          float *__restrict__ dweights) {
    grid_dependents_launch();
    grid_dependency_wait();
    const uint32_t slot = blockIdx.x * 4 + (threadIdx.x >> 5);
    if (slot >= slots) return;
    const int lane = threadIdx.x & 31;
    const int64_t r = __ldg(rows + slot);
    const f32x2 zero2 = f2_pack(0.0f, 0.0f);
    f32x2 dot2 = zero2;
    if (r >= 0 && r < R) {
        const float w = __ldg(weights + slot);
        const f32x2 w2 = f2_pack(w, w);
        const uint16_t *drow = dout + (int64_t)divide(slot, k) * ldo;
        uint16_t *to = dy + r * lddy;
        const int cols = (int)H;  // at most 2^25
        if (MX) {
            const uint8_t *crow = codes + r * H;
            const uint8_t *srow = sf + sf_offset(r, 0, H >> 5);
#pragma unroll 2
            for (int c = lane * 16; c < cols; c += 512) {
                const uint4 q = __ldg(reinterpret_cast<const uint4 *>(crow + c));
                const uint4 d0 = __ldg(reinterpret_cast<const uint4 *>(drow + c));
                const uint4 d1 = __ldg(reinterpret_cast<const uint4 *>(drow + c + 8));
                const float scale = e8m0_value(__ldg(srow + ((c >> 7) << 9) + ((c >> 5) & 3)));  // atoms of 4 blocks
                f32x2 v[8], part2 = zero2;
                e4m3x16(q, v);
                bwd8(d0, v, w2, part2, to + c);
                bwd8(d1, v + 4, w2, part2, to + c + 8);
                dot2 = f2_fma(part2, f2_pack(scale, scale), dot2);
            }
        } else {
            const uint16_t *yrow = y + r * ldy;
#pragma unroll 4
            for (int c = lane * 8; c < cols; c += 256) {
                const uint4 d = __ldg(reinterpret_cast<const uint4 *>(drow + c));
                const uint4 q = __ldg(reinterpret_cast<const uint4 *>(yrow + c));
                const f32x2 v[4] = {f2_pack(bf16_lo(q.x), bf16_hi(q.x)), f2_pack(bf16_lo(q.y), bf16_hi(q.y)),
                                    f2_pack(bf16_lo(q.z), bf16_hi(q.z)), f2_pack(bf16_lo(q.w), bf16_hi(q.w))};
                bwd8(d, v, w2, dot2, to + c);
            }
        }
    }
    float dot, odd;
    f2_unpack(dot2, dot, odd);
    dot = warp_sum(dot + odd);
    if (lane == 0) dweights[slot] = dot;
}

// ------------------------------------------------------------------ gated SiLU with an MXFP8 checkpoint
// sigmoid of a pair and g times it, through q = 2^(g log2 e / 2) with the exponent held at 32 (g = 44, where the
// sigmoid is 1 to 2^-63): s = q r, g s = (g r) q with r = q / (1 + q^2).  No factor leaves the normal numbers before
// the last product does, so s is right below 2^-126 (g < -87.3) too.  Relative error (13 + 2 |g|) 2^-24 at most, the
// |g| from the rounding of the exponent, and one step more for g s; results are rounded to 2^-8.
BSQ_DEV f32x2 sigmoid2(f32x2 g, f32x2 &gs) {
    float a, b;
    f2_unpack(f2_mul(g, f2_pack(0.5f * kLog2e, 0.5f * kLog2e)), a, b);
    const f32x2 q = f2_pack(ex2(fminf(a, 32.0f)), ex2(fminf(b, 32.0f)));
    f2_unpack(f2_fma(q, q, f2_pack(1.0f, 1.0f)), a, b);
    const f32x2 r = f2_mul(q, f2_pack(rcp(a), rcp(b)));
    gs = f2_mul(f2_mul(g, r), q);
    return f2_mul(q, r);
}

// Larger of two bf16 pairs of magnitudes, lane by lane.
BSQ_DEV uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
constexpr uint32_t kAbs2 = 0x7FFF7FFFu;

// Row-wise MXFP8 of 16 values, two lanes per block of 32 (the bytes of
// bsq_quant_mxfp8 with nearest rounding).  The block maximum is taken on the
// bf16 words; its exponent field minus 8 is the scale code (0 where that
// would be below 0, and for an all-zero block, whose codes are +0), and the
// products with 2^-E are exact.
BSQ_DEV uint4 mx_encode16(const uint32_t w[8], uint32_t *scale_code) {
    uint32_t m = w[0] & kAbs2;
#pragma unroll
    for (int i = 1; i < 8; i++) m = max_bf16x2(m, w[i] & kAbs2);
    m = max_bf16x2(m, __shfl_xor_sync(kFull, m, 1));
    m = max(m & 0xFFFFu, m >> 16);
    const uint32_t sb = (uint32_t)max((int)(m >> 7) - 8, 0);
    *scale_code = sb;
    const float inv = __uint_as_float((254u - sb) << 23);
    const f32x2 inv2 = f2_pack(inv, inv);
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        float a, b, c, d;
        f2_unpack(f2_mul(f2_pack(bf16_lo(w[2 * i]), bf16_hi(w[2 * i])), inv2), a, b);
        f2_unpack(f2_mul(f2_pack(bf16_lo(w[2 * i + 1]), bf16_hi(w[2 * i + 1])), inv2), c, d);
        q[i] = cvt_e4m3x2(a, b) | (cvt_e4m3x2(c, d) << 16);  // saturating: +-448 beyond
    }
    const uint32_t keep = m ? 0xFFFFFFFFu : 0u;
    return make_uint4(q[0] & keep, q[1] & keep, q[2] & keep, q[3] & keep);
}

BSQ_DEV void load16(const uint16_t *p, uint32_t w[8]) { load_words16(p, w); }
BSQ_DEV void store16(uint16_t *p, const uint32_t w[8]) {
    reinterpret_cast<uint4 *>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4 *>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

__global__ void zero_word_kernel(unsigned int *p) {
    grid_dependents_launch();
    grid_dependency_wait();
    *p = 0;
}

// Threads of a gated SiLU CTA; with 256, 131072x768 takes 129 us instead of 127, its backward 156 instead of 149.
constexpr int kGlu = 128;

// Memory bound: 8.06 bytes per h.  A thread takes 16 columns of the gate and
// the same 16 of v (64 bytes in flight), so two lanes share a block of 32 and
// write one scale byte each.  131072x768: 127 us, 98 % of the measured copy rate.
__global__ void __launch_bounds__(kGlu, 1024 / kGlu)
    swiglu_ckpt_kernel(const uint16_t *__restrict__ u, int64_t M, int64_t F, int64_t ldu, UnitDiv per,
                       const int32_t *__restrict__ n_rows, uint16_t *__restrict__ h, int64_t ldh,
                       uint8_t *__restrict__ codes, uint8_t *__restrict__ sf, unsigned int *__restrict__ amax) {
    grid_dependents_launch();
    grid_dependency_wait();
    const int64_t rows = n_rows ? min(M, (int64_t)max(__ldg(n_rows), 0)) : M;
    const int64_t n = rows * per.d;  // even: a block's two lanes go together
    const int64_t i = (int64_t)blockIdx.x * kGlu + threadIdx.x;
    if ((i & ~int64_t(31)) >= n) return;  // whole warps: the shuffles want all of their lanes
    const uint32_t unit = i < n ? (uint32_t)i : 0u;
    const uint32_t r = divide(unit, per);
    const int64_t c = (int64_t)(unit - r * per.d) * 16;
    uint32_t g[8], v[8], o[8], top = 0;
    load16(u + r * ldu + c, g);
    load16(u + r * ldu + F + c, v);
    uint32_t sg, sv;
    const uint4 cg = mx_encode16(g, &sg), cv = mx_encode16(v, &sv);
#pragma unroll
    for (int q = 0; q < 8; q++) {
        const f32x2 gq = f2_pack(bf16_lo(g[q]), bf16_hi(g[q]));
        f32x2 gs;
        sigmoid2(gq, gs);
        float a, b;
        f2_unpack(f2_mul(gs, f2_pack(bf16_lo(v[q]), bf16_hi(v[q]))), a, b);
        o[q] = pack_bf16(a, b);
        top = max_bf16x2(top, o[q] & kAbs2);
    }
    if (i < n) {
        store16(h + r * ldh + c, o);
        uint8_t *row = codes + (int64_t)r * 2 * F + c;
        *reinterpret_cast<uint4 *>(row) = cg;
        *reinterpret_cast<uint4 *>(row + F) = cv;
        const bool odd = threadIdx.x & 1;
        sf[sf_offset(r, (c + (odd ? F : 0)) >> 5, F >> 4)] = (uint8_t)(odd ? sv : sg);
    }
    if (amax) {
        top = __reduce_max_sync(kFull, max(top & 0xFFFFu, top >> 16)) << 16;
        // non-negative floats order as their bits; most warps find a larger one there already
        if ((threadIdx.x & 31) == 0 && top > *reinterpret_cast<volatile unsigned int *>(amax)) atomicMax(amax, top);
    }
}

// From the checkpoint's g and v: du = (dh v s (1 + g (1 - s)), dh g s), and,
// when h is wanted, h = g s v again.  Memory bound: 8.06 bytes per element of
// dh, 10.06 with h (131072x768: 118 and 149 us).
template <bool AGAIN>
__global__ void __launch_bounds__(kGlu) swiglu_ckpt_bwd_kernel(const uint16_t *__restrict__ dh, int64_t lddh,
                                                              const uint8_t *__restrict__ codes,
                                                              const uint8_t *__restrict__ sf, int64_t M, int64_t F,
                                                              UnitDiv per, const int32_t *__restrict__ n_rows,
                                                              uint16_t *__restrict__ du, int64_t lddu,
                                                              uint16_t *__restrict__ h, int64_t ldh) {
    grid_dependents_launch();
    grid_dependency_wait();
    const int64_t rows = n_rows ? min(M, (int64_t)max(__ldg(n_rows), 0)) : M;
    const int64_t n = rows * per.d;
    const int64_t i = (int64_t)blockIdx.x * kGlu + threadIdx.x;
    if (i >= n) return;
    const uint32_t r = divide((uint32_t)i, per);
    const int64_t c = (int64_t)((uint32_t)i - r * per.d) * 16;
    const uint8_t *row = codes + (int64_t)r * 2 * F + c;
    uint32_t d[8], x[8], y[8], w[8];
    f32x2 g[8], v[8];
    load16(dh + r * lddh + c, d);
    const uint4 qg = __ldg(reinterpret_cast<const uint4 *>(row));
    const uint4 qv = __ldg(reinterpret_cast<const uint4 *>(row + F));
    const uint32_t sg = __ldg(sf + sf_offset(r, c >> 5, F >> 4));
    const uint32_t sv = __ldg(sf + sf_offset(r, (c + F) >> 5, F >> 4));
    e4m3x16(qg, g);
    e4m3x16(qv, v);
    const float fg = e8m0_value(sg), fv = e8m0_value(sv);
    const f32x2 fg2 = f2_pack(fg, fg), fv2 = f2_pack(fv, fv);
#pragma unroll
    for (int q = 0; q < 8; q++) {
        g[q] = f2_mul(g[q], fg2);
        v[q] = f2_mul(v[q], fv2);
    }
#pragma unroll
    for (int q = 0; q < 8; q++) {
        f32x2 gs;
        const f32x2 dd = f2_pack(bf16_lo(d[q]), bf16_hi(d[q])), sg2 = sigmoid2(g[q], gs);
        float a, b;
        f2_unpack(f2_mul(dd, gs), a, b);
        y[q] = pack_bf16(a, b);
        // s (1 + g (1 - s)) = s + gs (1 - s)
        const f32x2 slope = f2_fma(gs, f2_sub(f2_pack(1.0f, 1.0f), sg2), sg2);
        f2_unpack(f2_mul(f2_mul(dd, v[q]), slope), a, b);
        x[q] = pack_bf16(a, b);
        if (AGAIN) {
            f2_unpack(f2_mul(gs, v[q]), a, b);
            w[q] = pack_bf16(a, b);
        }
    }
    store16(du + r * lddu + c, x);
    store16(du + r * lddu + F + c, y);
    if (AGAIN) store16(h + r * ldh + c, w);
}

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// Whether quads of four logits are aligned in every row.
template <typename In>
bool quads(const void *p, int64_t E, int64_t ld) {
    return E % 4 == 0 && ld % 4 == 0 && reinterpret_cast<uintptr_t>(p) % (4 * sizeof(In)) == 0;
}

// f.template operator()<LPT, Q>() with LPT lanes per token, Q quads of logits per
// lane.  Eight lanes per token wherever 32 logits per lane are enough: a round
// of the choice serves four tokens of a warp.  Against the next larger step the
// ones at 96, 160, 192 and 384 take 131072 tokens, k = 8, from 50 to 45, 60 to 54,
// 61 to 56 and 105 to 98 us (bf16; fp32 57 to 53, 80 to 65, 82 to 70, 135 to 117), the
// gradient from 20 to 18, 31 to 24, 33 to 29 and 58 to 51 (fp32 22 to 21, 35 both,
// 38 both, 70 to 76).
template <class F>
int by_experts(int64_t E, F f) {
    if (E <= 32) return f.template operator()<8, 1>();
    if (E <= 64) return f.template operator()<8, 2>();
    if (E <= 96) return f.template operator()<8, 3>();
    if (E <= 128) return f.template operator()<8, 4>();
    if (E <= 160) return f.template operator()<8, 5>();
    if (E <= 192) return f.template operator()<8, 6>();
    if (E <= 256) return f.template operator()<8, 8>();
    if (E <= 384) return f.template operator()<16, 6>();
    if (E <= 512) return f.template operator()<16, 8>();
    return f.template operator()<32, 8>();
}

bool small_hist(int64_t nchunk, int E) {
    return E <= 256 && nchunk <= kSmallChunks && nchunk * hist_row(E) <= kSmallHist;
}

// First pass: 16 warps take a chunk in half as many turns as 8, up to two chunks
// an SM.  Up to 64 experts both chunks fit on it at once (64 registers); with
// more experts the second waits for the first, and 16 warps are the faster all
// the same.  The call with 16 and 8 warps, k = 8: 11.4 and 16.0 us at 16384x64,
// 19.6 and 20.6 at 16384x128, 18.3 and 22.1 at 16384x256, 47 and 90 at
// 16384x1000 (bf16; fp32 alike); 8 warps win a few sizes of 96 to 160 experts, by
// 13 % at most (12000x160: 20.9 and 18.2).
// Many experts and more chunks: two chunks a CTA, so that the sums of
// probabilities leave the registers half as often: 131072x256 takes 63.4 us, 64.5
// with a chunk a CTA, 66.5 with as many CTAs as fit at once (40000x256: 30.3, 27.6
// and 30.6).
int topk_threads(int64_t nchunk, int num_sms) { return nchunk <= 2 * num_sms ? 512 : 256; }
int64_t topk_grid(int64_t nchunk, int64_t E, int num_sms) {
    return E > 128 && topk_threads(nchunk, num_sms) == 256 ? (nchunk + 1) / 2 : nchunk;
}

// CTAs of the cluster that takes all chunks (a power of two, eight at most: the
// portable size), or 0: more chunks than that.
int cluster_ctas(int64_t nchunk) {
    return nchunk > 8 ? 0 : nchunk > 4 ? 8 : nchunk > 2 ? 4 : (int)nchunk;
}

// Shared memory of the first pass, all of it dynamic (a variable of static size would count towards the 48 KB that
// need no attribute); at most 98,584 bytes (1024 experts, 32 slots, 16 warps).
constexpr int kRouteSmem = 100 * 1024;

template <typename In>
struct TopkLaunch {
    const RouteArgs &a;
    const RouteWorkspace &w;
    int want_p, num_sms;
    cudaStream_t s;
    template <int LPT, int Q>
    int operator()() const {
        return a.topk <= 4   ? run(route_topk_kernel<In, LPT, Q, 4>)
               : a.topk <= 8 ? run(route_topk_kernel<In, LPT, Q, 8>)
                             : run(route_topk_kernel<In, LPT, Q, 0>);
    }
    template <class K>
    int run(K kern) const {
        const int E = (int)a.E, k = a.topk;
        const int threads = topk_threads(w.nchunk, num_sms), ctas = cluster_ctas(w.nchunk);
        const size_t smem = 8 * (size_t)(E + 1) + 4 * kChunk * (size_t)(k + 1) +
                            (want_p ? threads / 32 * 4 * (size_t)E : 0) + (ctas ? 12 * (size_t)(E + 1) + 4 : 0) +
                            2 * kChunk * (size_t)k;
        if (smem > 48 * 1024 && smem_attr_once(reinterpret_cast<const void *>(kern), kRouteSmem) != BSQ_OK) return 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(ctas ? ctas : topk_grid(w.nchunk, E, num_sms)));
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        cudaLaunchAttribute attr[2];
        if (kernel_choice(BSQ_KNOB_LAUNCH_OVERLAP) != 0) {  // as launch_dependent()
            attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
        }
        if (ctas > 1) {
            attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
            attr[cfg.numAttrs].val.clusterDim.x = (unsigned)ctas;
            attr[cfg.numAttrs].val.clusterDim.y = 1;
            attr[cfg.numAttrs++].val.clusterDim.z = 1;
        }
        cfg.attrs = attr;
        const RouteOut out{a.ids, a.weights, a.rows, a.row_index, a.row_off, a.sf_row_off, a.counts, a.prob_sums,
                           a.loss};
        return cudaLaunchKernelEx(&cfg, kern, static_cast<const In *>(a.logits), a.T, E, a.ldl,
                                  (int)quads<In>(a.logits, E, a.ldl), a.mask, unit_div((uint32_t)k), (int)a.renorm,
                                  want_p, ctas, out, w.nchunk, a.ws + w.hist,
                                  reinterpret_cast<float *>(a.ws + w.psum), a.coef) != cudaSuccess;
    }
};

template <typename In, bool NEED_P>
struct BwdLaunch {
    const RouteBwdArgs &a;
    int num_sms;
    cudaStream_t s;
    template <int LPT, int Q>
    int operator()() const {
        constexpr int per_cta = 8 * (32 / LPT);
        const int64_t most = (int64_t)num_sms * bwd_ctas<Q, NEED_P>();
        const unsigned grid = (unsigned)std::min<int64_t>((a.T + per_cta - 1) / per_cta, most);
        const bool vec = quads<In>(a.logits, a.E, a.ldl) && quads<In>(a.dlogits, a.E, a.ldd);
        return launch_dependent(route_bwd_kernel<In, LPT, Q, NEED_P>, dim3(grid), dim3(256), 0, s,
                                static_cast<const In *>(a.logits), a.T, (int)a.E, a.ldl, (int)vec, a.topk,
                                (int)a.renorm, a.ids, a.weights, a.dweights, a.counts, a.coef, a.dloss,
                                static_cast<In *>(a.dlogits), a.ldd) != cudaSuccess;
    }
};

}  // namespace

RouteWorkspace route_workspace(int64_t T, int64_t E) {
    RouteWorkspace w;
    w.nchunk = std::max<int64_t>((T + kChunk - 1) / kChunk, 1);
    const int64_t blocks = (w.nchunk + kBlock - 1) / kBlock;
    w.hist = 0;
    w.prefix = up(w.nchunk * 2 * hist_row((int)E), 256);
    w.psum = up(w.prefix + 2 * E * w.nchunk, 256);
    w.count = up(w.psum + 4 * E * w.nchunk, 256);
    w.psum_block = up(w.count + 4 * (E + 1) * blocks, 256);
    w.bytes = up(w.psum_block + 4 * E * blocks, 256);
    return w;
}

int launch_moe_route(const RouteArgs &a, int num_sms, cudaStream_t s) {
    const RouteWorkspace w = route_workspace(a.T, a.E);
    const int want_p = a.prob_sums || a.loss;
    if (a.bf16 ? by_experts(a.E, TopkLaunch<uint16_t>{a, w, want_p, num_sms, s})
               : by_experts(a.E, TopkLaunch<float>{a, w, want_p, num_sms, s}))
        return 1;
    if (cluster_ctas(w.nchunk)) return 0;  // done
    const int64_t rows = topk_grid(w.nchunk, a.E, num_sms);  // of sums of probabilities
    const int E = (int)a.E;
    float *psum = want_p ? reinterpret_cast<float *>(a.ws + w.psum) : nullptr;
    const RouteOut out{a.ids, a.weights, a.rows, a.row_index, a.row_off, a.sf_row_off, a.counts, a.prob_sums, a.loss};
    if (small_hist(w.nchunk, E))
        return launch_dependent(route_scan_place_kernel, dim3((unsigned)w.nchunk + 1), dim3(256), 0, s, a.T,
                                unit_div((uint32_t)a.topk), E, (int)w.nchunk,
                                unit_div((uint32_t)hist_row(E) / 4), (const uint8_t *)(a.ws + w.hist),
                                (const float *)psum, rows, out, a.coef) != cudaSuccess;
    const int64_t blocks = (w.nchunk + kBlock - 1) / kBlock;
    uint16_t *prefix = reinterpret_cast<uint16_t *>(a.ws + w.prefix);
    int32_t *count = reinterpret_cast<int32_t *>(a.ws + w.count);
    float *psum_block = want_p ? reinterpret_cast<float *>(a.ws + w.psum_block) : nullptr;
    if (launch_dependent(route_block_kernel, dim3((unsigned)blocks, E / 32 + 1), dim3(256), 0, s,
                         (const uint8_t *)(a.ws + w.hist), (const float *)psum, rows, w.nchunk, E, prefix, count,
                         psum_block) != cudaSuccess)
        return 1;
    // about three CTAs per SM: each adds up all blocks' counts
    const int parts = (int)std::max<int64_t>(1, std::min<int64_t>(kBlock, 3 * num_sms / blocks));
    const int span = (kBlock + parts - 1) / parts;
    return launch_dependent(route_place_kernel, dim3((unsigned)blocks + 1, (kBlock + span - 1) / span), dim3(256), 0, s,
                            a.T, unit_div((uint32_t)a.topk), E, w.nchunk, span, (const uint8_t *)(a.ws + w.hist),
                            (const uint16_t *)prefix, (const int32_t *)count, (const float *)psum_block, out,
                            a.coef) != cudaSuccess;
}

int launch_moe_route_bwd(const RouteBwdArgs &a, int num_sms, cudaStream_t s) {
    // the softmax over the chosen experts alone needs their weights, not the logits
    if (!a.renorm || a.dloss)
        return a.bf16 ? by_experts(a.E, BwdLaunch<uint16_t, true>{a, num_sms, s})
                      : by_experts(a.E, BwdLaunch<float, true>{a, num_sms, s});
    return a.bf16 ? by_experts(a.E, BwdLaunch<uint16_t, false>{a, num_sms, s})
                  : by_experts(a.E, BwdLaunch<float, false>{a, num_sms, s});
}

int launch_moe_combine(const uint16_t *y, int64_t R, int64_t H, int64_t ldy, const int32_t *rows, const float *weights,
                       int64_t T, int topk, uint16_t *out, int64_t ldo, cudaStream_t s) {
    auto run = [&](auto kern) {
        return launch_dependent(kern, dim3((unsigned)T, (unsigned)((H + 1023) / 1024)), dim3(128), 0, s, y, R, H, ldy,
                                rows, weights, topk, out, ldo) != cudaSuccess;
    };
    return topk <= 2 ? run(combine_kernel<2>) : run(combine_kernel<4>);  // no loads for slots that are not there
}

int launch_moe_combine_bwd(const uint16_t *dout, int64_t ldo, const uint16_t *y, int64_t ldy, const uint8_t *codes,
                           const uint8_t *sf, int64_t R, int64_t H, const int32_t *rows, const float *weights,
                           int64_t T, int topk, uint16_t *dy, int64_t lddy, float *dweights, cudaStream_t s) {
    const uint32_t slots = (uint32_t)(T * topk);
    auto run = [&](auto kern) {
        return launch_dependent(kern, dim3((slots + 3) / 4), dim3(128), 0, s, dout, ldo, y, ldy, codes, sf, R, H, rows,
                                weights, slots, unit_div((uint32_t)topk), dy, lddy, dweights) != cudaSuccess;
    };
    return codes ? run(combine_bwd_kernel<true>) : run(combine_bwd_kernel<false>);
}

int launch_swiglu_ckpt(const uint16_t *u, int64_t M, int64_t F, int64_t ldu, const int32_t *n_rows, uint16_t *h,
                       int64_t ldh, uint8_t *codes, uint8_t *sf, unsigned int *amax, cudaStream_t s) {
    const unsigned grid = (unsigned)((M * (F / 16) + kGlu - 1) / kGlu);
    const UnitDiv per = unit_div((uint32_t)(F / 16));
    if (amax && launch_dependent(zero_word_kernel, dim3(1), dim3(1), 0, s, amax) != cudaSuccess) return 1;
    return launch_dependent(swiglu_ckpt_kernel, dim3(grid), dim3(kGlu), 0, s, u, M, F, ldu, per, n_rows, h, ldh, codes,
                            sf, amax) != cudaSuccess;
}

int launch_swiglu_ckpt_bwd(const uint16_t *dh, int64_t lddh, const uint8_t *codes, const uint8_t *sf, int64_t M,
                           int64_t F, const int32_t *n_rows, uint16_t *du, int64_t lddu, uint16_t *h, int64_t ldh,
                           cudaStream_t s) {
    const unsigned grid = (unsigned)((M * (F / 16) + kGlu - 1) / kGlu);
    const UnitDiv per = unit_div((uint32_t)(F / 16));
    auto run = [&](auto kern) {
        return launch_dependent(kern, dim3(grid), dim3(kGlu), 0, s, dh, lddh, codes, sf, M, F, per, n_rows, du, lddu, h,
                                ldh) != cudaSuccess;
    };
    return h ? run(swiglu_ckpt_bwd_kernel<true>) : run(swiglu_ckpt_bwd_kernel<false>);
}

}  // namespace bsq
