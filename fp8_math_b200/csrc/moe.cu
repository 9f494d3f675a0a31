// moe.cu -- kernels of a mixture-of-experts layer's training step that stand
// between the quantizers and the grouped GEMM: the router (top-k, weights,
// counts, row order, balance loss) and its gradient, the combine of expert
// rows in bf16 and its gradients, the gated SiLU whose input is kept in MXFP8
// for the backward pass.  All sums are in fp32 and in a fixed order, so a call
// gives the same bits every time.
#include <algorithm>

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
BSQ_DEV float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}
BSQ_DEV uint32_t pack_bf16(float lo, float hi) {
    __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&b);
}
BSQ_DEV float load_logit(const float *p) { return __ldg(p); }
BSQ_DEV float load_logit(const uint16_t *p) { return __uint_as_float((uint32_t)__ldg(p) << 16); }
BSQ_DEV void store_logit(float *p, float v) { *p = v; }
BSQ_DEV void store_logit(uint16_t *p, float v) { *p = (uint16_t)(pack_bf16(v, 0.0f) & 0xFFFFu); }

// 2^x (relative error 2^-22, subnormal results kept) and 1/x (1 ulp).
BSQ_DEV float ex2(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
BSQ_DEV float rcp(float x) {
    float y;
    asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
BSQ_DEV float ex2_ftz(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
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

// max over the warp; NaN operands are passed over
BSQ_DEV float warp_max_redux(float v) {
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// min(a, b), NaN when one of them is NaN
BSQ_DEV float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// exp(x[i] - top) for all i, through 2^x; -inf gives 0.
template <int N>
BSQ_DEV void exp_below(float x[N], float top) {
    const f32x2 t2 = f2_pack(top, top), l2 = f2_pack(kLog2e, kLog2e);
#pragma unroll
    for (int i = 0; i + 1 < N; i += 2) {
        f2_unpack(f2_mul(f2_sub(f2_pack(x[i], x[i + 1]), t2), l2), x[i], x[i + 1]);
        x[i] = ex2_ftz(x[i]);
        x[i + 1] = ex2_ftz(x[i + 1]);
    }
    if (N & 1) x[N - 1] = ex2_ftz((x[N - 1] - top) * kLog2e);
}

// ------------------------------------------------------------------ router
// A lane's two best candidates of its EPL logits, and the next best once both
// are gone: k rounds of one warp maximum each then need no second look at
// the logits, except in the few tokens where one lane holds three of the top
// k.  Ordered by (-logit, expert); -inf is never a candidate.
//
// bf16 logits leave 16 bits of an fp32 free: the expert goes there, so that
// one float comparison orders (logit, expert) and no two are equal.  Larger
// low bits make a positive float larger and a negative one smaller; adding 0
// turns -0 into +0 first.  -inf with low bits is a NaN, which maxima pass
// over (and the minimum below hands on to them).
template <typename In, int EPL>
struct Candidates;

template <int EPL>
struct Candidates<uint16_t, EPL> {
    float key[EPL], m1, m2;
    int left;
    BSQ_DEV void init(const float z[EPL], int lane) {
        m1 = m2 = -INFINITY;
        left = 2;
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            const uint32_t b = __float_as_uint(__fadd_rn(z[i], 0.0f));
            key[i] = __uint_as_float(b | ((uint32_t)(i * 32 + lane) ^ (~(uint32_t)((int32_t)b >> 31) & 0xFFFFu)));
            m2 = fmaxf(m2, min_nan(m1, key[i]));
            m1 = fmaxf(m1, key[i]);
        }
    }
    // The best candidate of the warp leaves: its logit (-inf: there is none) and expert.
    BSQ_DEV float pop(int, int &e) {
        const float best = warp_max_redux(m1);
        const uint32_t b = __float_as_uint(best);
        e = (int)((b ^ ~(uint32_t)((int32_t)b >> 31)) & 0xFFFFu);
        if (m1 == best) {
            m1 = m2;
            m2 = -INFINITY;
            if (EPL > 2 && --left <= 0)
#pragma unroll
                for (int i = 0; i < EPL; i++) m1 = fmaxf(m1, key[i] < best ? key[i] : -INFINITY);
        }
        return best > -INFINITY ? __uint_as_float(b & 0xFFFF0000u) : -INFINITY;
    }
};

template <int EPL>
struct Candidates<float, EPL> {
    float z[EPL], m1, m2;
    int e1, e2, left;
    BSQ_DEV void init(const float x[EPL], int) {
        m1 = m2 = -INFINITY;
        e1 = e2 = 0;
        left = 2;
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            z[i] = x[i];
            const bool first = x[i] > m1, second = x[i] > m2;
            e2 = first ? e1 : second ? i : e2;
            m2 = fmaxf(m2, fminf(m1, x[i]));
            e1 = first ? i : e1;
            m1 = first ? x[i] : m1;
        }
    }
    BSQ_DEV float pop(int lane, int &e) {
        const float best = warp_max_redux(m1);
        // the lowest expert among the lanes that hold this logit
        e = (int)__reduce_min_sync(kFull, m1 == best ? (unsigned)(e1 * 32 + lane) : 0xFFFFu);
        if (e == e1 * 32 + lane && m1 == best) {
            const int at = e1;
            m1 = m2;
            e1 = e2;
            m2 = -INFINITY;
            if (EPL > 2 && --left <= 0) {
#pragma unroll
                for (int i = 0; i < EPL; i++)
                    if ((z[i] < best || (z[i] == best && i > at)) && z[i] > m1) {
                        m1 = z[i];
                        e1 = i;
                    }
            }
        }
        return best;
    }
};

// Pass 1.  A CTA takes kChunk consecutive tokens, a warp one token at a time;
// lane l holds the logits of experts l, l + 32, ...  The softmax sum runs over
// the same registers.  The chosen experts go into one 64-bit mask of tokens
// per expert, whose population count is the chunk's count and whose bits below
// a token are that token's rank in the chunk: the order "by expert, then
// token" needs no sort.  Row E of the counts is the number of tokens with at
// least one expert.
template <typename In, int EPL>
__global__ void __launch_bounds__(256) route_topk_kernel(const In *__restrict__ logits, int64_t T, int E, int64_t ldl,
                                                         const uint8_t *__restrict__ mask, int k, int renorm,
                                                         int want_p, int32_t *__restrict__ ids,
                                                         float *__restrict__ weights, int32_t *__restrict__ rows,
                                                         int64_t nchunk, uint32_t *__restrict__ hist,
                                                         float *__restrict__ psum) {
    grid_dependents_launch();
    extern __shared__ unsigned long long smem[];
    unsigned int *words = reinterpret_cast<unsigned int *>(smem);               // [(E + 1) * 2]
    uint16_t *sel = reinterpret_cast<uint16_t *>(words + 2 * (E + 1));          // [kChunk][k]
    float *red = reinterpret_cast<float *>(sel + kChunk * k);                   // [8][E] when want_p
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < 2 * (E + 1); i += 256) words[i] = 0;
    __syncthreads();
    const int64_t t0 = (int64_t)blockIdx.x * kChunk;
    float acc[EPL];
#pragma unroll
    for (int i = 0; i < EPL; i++) acc[i] = 0.0f;
    for (int tl = warp; tl < kChunk; tl += 8) {
        const int64_t t = t0 + tl;
        if (t >= T) break;
        float my_z = -INFINITY, sum = 0.0f, top = 0.0f;
        int my_e = -1;
        if (!mask || __ldg(mask + t) != 0) {
            float z[EPL];
#pragma unroll
            for (int i = 0; i < EPL; i++) {
                const int e = i * 32 + lane;
                z[i] = e < E ? load_logit(logits + t * ldl + e) : -INFINITY;
            }
            Candidates<In, EPL> c;
            c.init(z, lane);
            for (int j = 0; j < k; j++) {
                int e;
                const float best = c.pop(lane, e);
                if (!(best > -INFINITY)) break;
                if (j == 0) top = best;
                if (lane == j) {
                    my_z = best;
                    my_e = e;
                }
            }
            if (want_p || !renorm) {
                exp_below<EPL>(z, top);
#pragma unroll
                for (int i = 0; i < EPL; i++) sum += z[i];
                sum = warp_sum(sum);
                const float inv = sum > 0.0f ? rcp(sum) : 0.0f;
                if (want_p)
#pragma unroll
                    for (int i = 0; i < EPL; i++) acc[i] = fmaf(z[i], inv, acc[i]);
            }
        }
        const float x = my_e >= 0 ? ex2_ftz((my_z - top) * kLog2e) : 0.0f;
        if (renorm) sum = warp_sum(x);
        if (lane < k) {
            ids[t * k + lane] = my_e;
            weights[t * k + lane] = my_e >= 0 ? x * rcp(sum) : 0.0f;
            sel[tl * k + lane] = (uint16_t)my_e;
            if (my_e >= 0) atomicOr(&words[2 * my_e + (tl >> 5)], 1u << (tl & 31));
            if (lane == 0 && my_e >= 0) atomicOr(&words[2 * E + (tl >> 5)], 1u << (tl & 31));
        }
    }
    if (want_p) {
#pragma unroll
        for (int i = 0; i < EPL; i++)
            if (i * 32 + lane < E) red[warp * E + i * 32 + lane] = acc[i];
    }
    __syncthreads();
    const int here = (int)min((int64_t)kChunk, T - t0);
    for (int i = threadIdx.x; i < here * k; i += 256) {
        const int e = (int16_t)sel[i];
        rows[t0 * k + i] = e < 0 ? -1 : __popcll(smem[e] & ((1ull << (i / k)) - 1ull));
    }
    for (int e = threadIdx.x; e <= E; e += 256) {
        const unsigned long long m = smem[e];
        // count in the low byte, the chunk's first token of the expert above it
        hist[(int64_t)e * nchunk + blockIdx.x] = (uint32_t)__popcll(m) | (m ? (uint32_t)(__ffsll(m) - 1) << 8 : 0u);
        if (want_p && e < E) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < 8; w++) v += red[w * E + e];
            psum[(int64_t)e * nchunk + blockIdx.x] = v;
        }
    }
}

// Pass 2.  One CTA per expert (and one for the token count): its counts per
// chunk become exclusive prefixes in place, their total goes to counts[e];
// the first token that chose e, and the sum of its probabilities, go along.
__global__ void __launch_bounds__(256) route_scan_kernel(uint32_t *__restrict__ hist, const float *__restrict__ psum,
                                                         int64_t nchunk, int E, int32_t *__restrict__ counts,
                                                         int32_t *__restrict__ first, float *__restrict__ psum_total) {
    grid_dependents_launch();
    grid_dependency_wait();
    __shared__ int wsum[8];
    __shared__ float fsum[8];
    __shared__ int sfirst;
    const int e = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t *h = hist + (int64_t)e * nchunk;
    if (threadIdx.x == 0) sfirst = 0x7FFFFFFF;
    __syncthreads();
    int carry = 0;
    float p = 0.0f;
    for (int64_t c0 = 0; c0 < nchunk; c0 += 256) {
        const int64_t c = c0 + threadIdx.x;
        const uint32_t v = c < nchunk ? h[c] : 0u;
        const int n = (int)(v & 0xFFu);
        if (n) atomicMin(&sfirst, (int)(c * kChunk) + (int)(v >> 8));
        if (psum && e < E && c < nchunk) p += psum[(int64_t)e * nchunk + c];
        int s = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(kFull, s, o);
            if (lane >= o) s += u;
        }
        if (lane == 31) wsum[warp] = s;
        __syncthreads();
        int before = 0, all = 0;
#pragma unroll
        for (int w = 0; w < 8; w++) {
            if (w < warp) before += wsum[w];
            all += wsum[w];
        }
        if (c < nchunk) h[c] = (uint32_t)(carry + before + s - n);
        carry += all;
        __syncthreads();
    }
    p = warp_sum(p);
    if (lane == 0) fsum[warp] = p;
    __syncthreads();
    if (threadIdx.x == 0) {
        counts[e] = carry;
        if (e < E) {
            first[e] = sfirst;
            if (psum) {
                float v = 0.0f;
                for (int w = 0; w < 8; w++) v += fsum[w];
                psum_total[e] = v;
            }
        }
    }
}

// Exclusive scan over e < E of counts[e] (PAD128: each rounded up to 128)
// into off[0..E], by one CTA of 256 threads holding four experts each.
template <bool PAD128>
BSQ_DEV void scan_counts(const int32_t *counts, int E, int32_t *off, int *wsum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int n[4], s = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int e = threadIdx.x * 4 + i;
        n[i] = e < E ? counts[e] : 0;
        if (PAD128) n[i] = (n[i] + 127) & ~127;
        s += n[i];
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
        const int e = threadIdx.x * 4 + i;
        if (e <= E) off[e] = at;
        at += n[i];
    }
    if (E == 1024 && threadIdx.x == 255) off[E] = at;
    __syncthreads();
}

// Pass 3.  Row of a slot = its expert's offset + the chunk's prefix + the
// rank inside the chunk; the rows past the last routed one repeat the first
// row's token.  CTA 0 also writes the offsets and the loss.
__global__ void __launch_bounds__(256) route_place_kernel(const int32_t *__restrict__ ids, int32_t *__restrict__ rows,
                                                          uint32_t n, UnitDiv k, int E, int64_t nchunk,
                                                          const uint32_t *__restrict__ hist,
                                                          const int32_t *__restrict__ counts,
                                                          const int32_t *__restrict__ first,
                                                          const float *__restrict__ psum_total, float coef,
                                                          int32_t *__restrict__ row_index,
                                                          int32_t *__restrict__ row_off,
                                                          int32_t *__restrict__ sf_row_off,
                                                          float *__restrict__ prob_sums, float *__restrict__ loss) {
    grid_dependency_wait();
    __shared__ int32_t off[kRouteMaxExperts + 1];
    __shared__ int wsum[8];
    __shared__ int first_token;
    if (threadIdx.x == 0) first_token = 0;
    scan_counts<false>(counts, E, off, wsum);
    for (int e = threadIdx.x; e < E; e += 256)
        if (off[e] == 0 && off[e + 1] > 0) first_token = first[e];  // one expert only
    __syncthreads();
    const uint32_t total = (uint32_t)off[E];
    for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256) {  // n < 2^31
        const int e = ids[i];
        const uint32_t t = divide(i, k);
        if (e >= 0) {
            const int row = off[e] + (int)hist[(int64_t)e * nchunk + t / kChunk] + rows[i];
            rows[i] = row;
            row_index[row] = (int32_t)t;
        }
        if (i >= total) row_index[i] = first_token;
    }
    if (blockIdx.x == 0) {
        for (int e = threadIdx.x; e <= E; e += 256) row_off[e] = off[e];
        float part = 0.0f;
        if (psum_total)
            for (int e = threadIdx.x; e < E; e += 256) {
                const float p = psum_total[e];
                if (prob_sums) prob_sums[e] = p;
                part += (float)counts[e] * p;
            }
        __syncthreads();
        if (loss) {
            __shared__ float fsum[8];
            part = warp_sum(part);
            if ((threadIdx.x & 31) == 0) fsum[threadIdx.x >> 5] = part;
            __syncthreads();
            if (threadIdx.x == 0) {
                float v = 0.0f;
                for (int w = 0; w < 8; w++) v += fsum[w];
                const float tokens = (float)counts[E];
                // E / (k n^2) * sum c_e sum_t p_te, by two divisions: n^2 may pass 2^24
                *loss = counts[E] > 0 ? coef * (float)E * (v / tokens) / ((float)k.d * tokens) : 0.0f;
            }
        }
        scan_counts<true>(counts, E, off, wsum);
        for (int e = threadIdx.x; e <= E; e += 256) sf_row_off[e] = off[e];
    }
}

// ------------------------------------------------------------------ router, backward
// One warp per token.  With q the weights' distribution (the softmax over all
// experts, or over the chosen ones) and a_e = dL/dweight of expert e (zero
// where it was not chosen): dz_e = q_e (a_e - sum q a).  The balance loss adds
// the softmax's gradient of sum_e b_e p_e with b_e = dloss coef E c_e / (k n^2),
// kept in shared memory for the CTA.  The chosen experts' own terms reach the
// lanes that hold those experts through a row of shared memory per warp, which
// is zero between tokens.
template <typename In, int EPL, bool NEED_P>
__global__ void __launch_bounds__(256) route_bwd_kernel(const In *__restrict__ logits, int64_t T, int E, int64_t ldl,
                                                        int k, int renorm, const int32_t *__restrict__ ids,
                                                        const float *__restrict__ weights,
                                                        const float *__restrict__ dweights,
                                                        const int32_t *__restrict__ counts, float coef,
                                                        const float *__restrict__ dloss, In *__restrict__ dlogits,
                                                        int64_t ldd) {
    __shared__ float own_rows[8][EPL * 32];
    __shared__ float bias[NEED_P ? EPL * 32 : 1];
    const int lane = threadIdx.x & 31;
    float *own_row = own_rows[threadIdx.x >> 5];
#pragma unroll
    for (int i = 0; i < EPL; i++) own_row[i * 32 + lane] = 0.0f;
    if (NEED_P) {
        float bscale = 0.0f;
        if (dloss) {
            const int n = __ldg(counts + E);
            bscale = n > 0 ? __ldg(dloss) * coef * (float)E / (float)n / ((float)k * (float)n) : 0.0f;
        }
        for (int e = threadIdx.x; e < EPL * 32; e += 256)
            bias[e] = dloss && e < E ? bscale * (float)__ldg(counts + e) : 0.0f;
    }
    __syncthreads();
    const int64_t stride = (int64_t)gridDim.x * 8;
    for (int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); t < T; t += stride) {
        int e_j = -1;
        float w_j = 0.0f, a_j = 0.0f;
        if (lane < k) {
            e_j = __ldg(ids + t * k + lane);
            if ((unsigned)e_j >= (unsigned)E) e_j = -1;
            if (e_j >= 0) {
                w_j = __ldg(weights + t * k + lane);
                a_j = dweights ? __ldg(dweights + t * k + lane) : 0.0f;
            }
        }
        float p[EPL];
        const bool live = __any_sync(kFull, e_j >= 0);  // a masked token's logits are not read
        if (NEED_P && live) {
#pragma unroll
            for (int i = 0; i < EPL; i++) {
                const int e = i * 32 + lane;
                p[i] = e < E ? load_logit(logits + t * ldl + e) : -INFINITY;
            }
        }
        const float dot = warp_sum(w_j * a_j);  // sum over chosen of q a: both kinds of q have q_ej = w_j
        // the chosen experts' own term: w_j (a_j - dot), or w_j a_j where dot goes over all experts
        if (e_j >= 0) own_row[e_j] = renorm ? w_j * (a_j - dot) : w_j * a_j;
        float d[EPL];
        if (NEED_P && live) {
            float top = p[0];
#pragma unroll
            for (int i = 1; i < EPL; i++) top = fmaxf(top, p[i]);
            top = warp_max_redux(top);
            exp_below<EPL>(p, top);
            float s = 0.0f, pb = 0.0f;
#pragma unroll
            for (int i = 0; i < EPL; i++) {
                d[i] = bias[i * 32 + lane];
                s += p[i];
                pb = fmaf(p[i], d[i], pb);
            }
            const float inv = rcp(warp_sum(s));
            const float sub = warp_sum(pb) * inv + (renorm ? 0.0f : dot);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < EPL; i++) d[i] = fmaf(p[i] * inv, d[i] - sub, own_row[i * 32 + lane]);
        } else {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < EPL; i++) d[i] = own_row[i * 32 + lane];
        }
        __syncwarp();
        if (e_j >= 0) own_row[e_j] = 0.0f;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < EPL; i++)
            if (i * 32 + lane < E) store_logit(dlogits + t * ldd + i * 32 + lane, d[i]);
    }
}

// ------------------------------------------------------------------ combine
// out[t] = sum_j w_tj y[rows_tj]: a CTA of 128 threads takes 1024 columns of
// one token, each thread eight of them over all k rows.
__global__ void __launch_bounds__(128) combine_kernel(const uint16_t *__restrict__ y, int64_t R, int64_t H, int64_t ldy,
                                                      const int32_t *__restrict__ rows,
                                                      const float *__restrict__ weights, int k,
                                                      uint16_t *__restrict__ out, int64_t ldo) {
    const int64_t t = blockIdx.x;
    const int64_t c = ((int64_t)blockIdx.y * 128 + threadIdx.x) * 8;
    if (c >= H) return;
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; i++) acc[i] = 0.0f;
    for (int j = 0; j < k; j++) {
        const int64_t r = __ldg(rows + t * k + j);
        if (r < 0 || r >= R) continue;
        const float w = weights ? __ldg(weights + t * k + j) : 1.0f;
        float v[8];
        load8_bf16(y + r * ldy + c, v);
#pragma unroll
        for (int i = 0; i < 8; i++) acc[i] += w * v[i];
    }
    *reinterpret_cast<uint4 *>(out + t * ldo + c) = make_uint4(pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]),
                                                               pack_bf16(acc[4], acc[5]), pack_bf16(acc[6], acc[7]));
}

// Eight values of an MXFP8 row: codes times 2^(scale code - 127).
BSQ_DEV void load8_mx(const uint8_t *codes, const uint8_t *sf, int64_t r, int64_t c, int64_t K, float v[8]) {
    const uint2 q = __ldg(reinterpret_cast<const uint2 *>(codes + r * K + c));
    const float scale = exp2i((int)__ldg(sf + sf_offset(r, c >> 5, K >> 5)) - 127);
    e4m3x2_to_f32(q.x & 0xFFFFu, v[0], v[1]);
    e4m3x2_to_f32(q.x >> 16, v[2], v[3]);
    e4m3x2_to_f32(q.y & 0xFFFFu, v[4], v[5]);
    e4m3x2_to_f32(q.y >> 16, v[6], v[7]);
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] *= scale;
}

// dy[rows_tj] = w_tj dout_t and dw_tj = <dout_t, y[rows_tj]>: one CTA per
// token, row by row; the dot product is summed per warp, then over the warps.
template <bool MX>
__global__ void __launch_bounds__(256) combine_bwd_kernel(const uint16_t *__restrict__ dout, int64_t ldo,
                                                          const uint16_t *__restrict__ y, int64_t ldy,
                                                          const uint8_t *__restrict__ codes,
                                                          const uint8_t *__restrict__ sf, int64_t R, int64_t H,
                                                          const int32_t *__restrict__ rows,
                                                          const float *__restrict__ weights, int k,
                                                          uint16_t *__restrict__ dy, int64_t lddy,
                                                          float *__restrict__ dweights) {
    __shared__ float part[kRouteMaxTopk][8];
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int j = 0; j < k; j++) {
        const int64_t r = __ldg(rows + t * k + j);
        float dot = 0.0f;
        if (r >= 0 && r < R) {
            const float w = __ldg(weights + t * k + j);
            for (int64_t c = threadIdx.x * 8; c < H; c += 256 * 8) {
                float d[8], v[8];
                load8_bf16(dout + t * ldo + c, d);
                if (MX) load8_mx(codes, sf, r, c, H, v);
                else load8_bf16(y + r * ldy + c, v);
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    dot += d[i] * v[i];
                    d[i] *= w;
                }
                *reinterpret_cast<uint4 *>(dy + r * lddy + c) = make_uint4(
                    pack_bf16(d[0], d[1]), pack_bf16(d[2], d[3]), pack_bf16(d[4], d[5]), pack_bf16(d[6], d[7]));
            }
        }
        dot = warp_sum(dot);
        if (lane == 0) part[j][warp] = dot;
    }
    __syncthreads();
    if (threadIdx.x < k) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; w++) s += part[threadIdx.x][w];
        dweights[t * k + threadIdx.x] = s;
    }
}

// ------------------------------------------------------------------ gated SiLU with an MXFP8 checkpoint
// sigmoid(g) as r or e r with e = exp(-|g|), r = 1 / (1 + e): e never
// overflows and r lies in [1/2, 1].  Relative error (8 + |g|) 2^-24 at most,
// the |g| from the rounding of the exponent; results are rounded to 2^-8.
BSQ_DEV float sigmoid(float g) {
    const float e = ex2(-fabsf(g) * kLog2e);
    const float r = rcp(1.0f + e);
    return g >= 0.0f ? r : e * r;
}

// max(|a|, |b|) of two bf16 pairs
BSQ_DEV uint32_t absmax_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a & 0x7FFF7FFFu), "r"(b & 0x7FFF7FFFu));
    return r;
}

// Row-wise MXFP8 of 16 values, two lanes per block of 32 (the bytes of
// bsq_quant_mxfp8 with nearest rounding).  The block maximum is taken on the
// bf16 words; its exponent field minus 8 is the scale code (0 where that
// would be below 0, and for an all-zero block, whose codes are +0), and the
// products with 2^-E are exact.
BSQ_DEV uint4 mx_encode16(const uint32_t w[8], uint32_t *scale_code) {
    uint32_t m = absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(w[0], w[1]), absmax_bf16x2(w[2], w[3])),
                               absmax_bf16x2(absmax_bf16x2(w[4], w[5]), absmax_bf16x2(w[6], w[7])));
    m = absmax_bf16x2(m, __shfl_xor_sync(kFull, m, 1));
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

// Memory bound: 8.06 bytes per h.  A thread takes 16 columns of the gate and
// the same 16 of v (64 bytes in flight), so two lanes share a block of 32 and
// write one scale byte each.
__global__ void __launch_bounds__(256) swiglu_ckpt_kernel(const uint16_t *__restrict__ u, int64_t M, int64_t F,
                                                          int64_t ldu, UnitDiv per, const int32_t *__restrict__ n_rows,
                                                          uint16_t *__restrict__ h, int64_t ldh,
                                                          uint8_t *__restrict__ codes, uint8_t *__restrict__ sf,
                                                          unsigned int *__restrict__ amax) {
    __shared__ unsigned int part[8];
    const int64_t rows = n_rows ? min(M, (int64_t)max(__ldg(n_rows), 0)) : M;
    const int64_t n = rows * per.d;  // even: a block's two lanes go together
    uint32_t top = 0;
    const int64_t round = (n + 31) & ~int64_t(31);  // the shuffle wants whole warps
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < round; i += (int64_t)gridDim.x * 256) {
        const uint32_t unit = i < n ? (uint32_t)i : 0u;
        const uint32_t r = divide(unit, per);
        const int64_t c = (int64_t)(unit - r * per.d) * 16;
        uint32_t g[8], v[8], o[8];
        load16(u + r * ldu + c, g);
        load16(u + r * ldu + F + c, v);
        uint32_t sg, sv;
        const uint4 cg = mx_encode16(g, &sg), cv = mx_encode16(v, &sv);
        if (i >= n) continue;
#pragma unroll
        for (int q = 0; q < 8; q++) {
            const float g0 = bf16_lo(g[q]), g1 = bf16_hi(g[q]);
            o[q] = pack_bf16(g0 * sigmoid(g0) * bf16_lo(v[q]), g1 * sigmoid(g1) * bf16_hi(v[q]));
            top = absmax_bf16x2(top, o[q]);
        }
        store16(h + r * ldh + c, o);
        uint8_t *row = codes + (int64_t)r * 2 * F + c;
        *reinterpret_cast<uint4 *>(row) = cg;
        *reinterpret_cast<uint4 *>(row + F) = cv;
        const bool odd = threadIdx.x & 1;
        sf[sf_offset(r, (c + (odd ? F : 0)) >> 5, F >> 4)] = (uint8_t)(odd ? sv : sg);
    }
    if (amax) {
        top = max(top & 0xFFFFu, top >> 16);
        top = __reduce_max_sync(kFull, top);
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < 8; w++) top = max(top, part[w]);
            atomicMax(amax, top << 16);  // non-negative floats order as their bits
        }
    }
}

// 16 values of an MXFP8 row from their codes and the block's scale code.
BSQ_DEV void mx_decode16(uint4 q, uint32_t sb, f32x2 v[8]) {
    const float scale = exp2i((int)sb - 127);
    const f32x2 s2 = f2_pack(scale, scale);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        float a, b, c, d;
        e4m3x2_to_f32(w[i] & 0xFFFFu, a, b);
        e4m3x2_to_f32(w[i] >> 16, c, d);
        v[2 * i] = f2_mul(f2_pack(a, b), s2);
        v[2 * i + 1] = f2_mul(f2_pack(c, d), s2);
    }
}

// From the checkpoint's g and v: du = (dh v s (1 + g (1 - s)), dh g s), and,
// when h is wanted, h = g s v again.  Memory bound: 8.06 bytes per element of
// dh, 10.06 with h.
template <bool AGAIN>
__global__ void __launch_bounds__(256) swiglu_ckpt_bwd_kernel(const uint16_t *__restrict__ dh, int64_t lddh,
                                                              const uint8_t *__restrict__ codes,
                                                              const uint8_t *__restrict__ sf, int64_t M, int64_t F,
                                                              UnitDiv per, const int32_t *__restrict__ n_rows,
                                                              uint16_t *__restrict__ du, int64_t lddu,
                                                              uint16_t *__restrict__ h, int64_t ldh) {
    const int64_t rows = n_rows ? min(M, (int64_t)max(__ldg(n_rows), 0)) : M;
    const int64_t n = rows * per.d;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const uint32_t r = divide((uint32_t)i, per);
        const int64_t c = (int64_t)((uint32_t)i - r * per.d) * 16;
        const uint8_t *row = codes + (int64_t)r * 2 * F + c;
        uint32_t d[8], x[8], y[8], w[8];
        f32x2 g[8], v[8];
        load16(dh + r * lddh + c, d);
        const uint4 qg = __ldg(reinterpret_cast<const uint4 *>(row)), qv = __ldg(reinterpret_cast<const uint4 *>(row + F));
        const uint32_t sg = __ldg(sf + sf_offset(r, c >> 5, F >> 4)), sv = __ldg(sf + sf_offset(r, (c + F) >> 5, F >> 4));
        mx_decode16(qg, sg, g);
        mx_decode16(qv, sv, v);
#pragma unroll
        for (int q = 0; q < 8; q++) {
            float gg[2], vv[2], dx[2], dy[2], again[2];
            f2_unpack(g[q], gg[0], gg[1]);
            f2_unpack(v[q], vv[0], vv[1]);
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const float dd = e ? bf16_hi(d[q]) : bf16_lo(d[q]);
                const float s = sigmoid(gg[e]), gs = gg[e] * s;
                dy[e] = dd * gs;
                // s (1 + g (1 - s)) = s + gs - gs s
                dx[e] = dd * vv[e] * fmaf(gs, 1.0f - s, s);
                again[e] = gs * vv[e];
            }
            x[q] = pack_bf16(dx[0], dx[1]);
            y[q] = pack_bf16(dy[0], dy[1]);
            if (AGAIN) w[q] = pack_bf16(again[0], again[1]);
        }
        store16(du + r * lddu + c, x);
        store16(du + r * lddu + F + c, y);
        if (AGAIN) store16(h + r * ldh + c, w);
    }
}

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

int launched() { return cudaGetLastError() == cudaSuccess ? 0 : 1; }

template <typename In>
int route_topk(const RouteArgs &a, const RouteWorkspace &w, int want_p, cudaStream_t s) {
    const int E = (int)a.E, k = a.topk;
    // at most 45064 bytes (1024 experts, 32 slots): within the default limit
    const size_t smem = 8 * (size_t)(E + 1) + 2 * kChunk * (size_t)k + (want_p ? 32 * (size_t)E : 0);
    auto run = [&](auto kern) {
        kern<<<(unsigned)w.nchunk, 256, smem, s>>>(
            static_cast<const In *>(a.logits), a.T, E, a.ldl, a.mask, k, a.renorm, want_p, a.ids, a.weights, a.rows,
            w.nchunk, reinterpret_cast<uint32_t *>(a.ws + w.hist), reinterpret_cast<float *>(a.ws + w.psum));
        return launched();
    };
    if (E <= 32) return run(route_topk_kernel<In, 1>);
    if (E <= 64) return run(route_topk_kernel<In, 2>);
    if (E <= 96) return run(route_topk_kernel<In, 3>);
    if (E <= 128) return run(route_topk_kernel<In, 4>);
    if (E <= 192) return run(route_topk_kernel<In, 6>);
    if (E <= 256) return run(route_topk_kernel<In, 8>);
    if (E <= 384) return run(route_topk_kernel<In, 12>);
    if (E <= 512) return run(route_topk_kernel<In, 16>);
    return run(route_topk_kernel<In, 32>);
}

template <typename In, bool NEED_P>
int route_bwd(const RouteBwdArgs &a, int num_sms, cudaStream_t s) {
    const unsigned grid = (unsigned)std::min<int64_t>((a.T + 7) / 8, (int64_t)num_sms * 8);
    auto run = [&](auto kern) {
        kern<<<grid, 256, 0, s>>>(static_cast<const In *>(a.logits), a.T, (int)a.E, a.ldl, a.topk, a.renorm, a.ids,
                                  a.weights, a.dweights, a.counts, a.coef, a.dloss, static_cast<In *>(a.dlogits),
                                  a.ldd);
        return launched();
    };
    if (a.E <= 32) return run(route_bwd_kernel<In, 1, NEED_P>);
    if (a.E <= 64) return run(route_bwd_kernel<In, 2, NEED_P>);
    if (a.E <= 96) return run(route_bwd_kernel<In, 3, NEED_P>);
    if (a.E <= 128) return run(route_bwd_kernel<In, 4, NEED_P>);
    if (a.E <= 192) return run(route_bwd_kernel<In, 6, NEED_P>);
    if (a.E <= 256) return run(route_bwd_kernel<In, 8, NEED_P>);
    if (a.E <= 384) return run(route_bwd_kernel<In, 12, NEED_P>);
    if (a.E <= 512) return run(route_bwd_kernel<In, 16, NEED_P>);
    return run(route_bwd_kernel<In, 32, NEED_P>);
}

}  // namespace

RouteWorkspace route_workspace(int64_t T, int64_t E) {
    RouteWorkspace w;
    w.nchunk = std::max<int64_t>((T + kChunk - 1) / kChunk, 1);
    w.hist = 0;
    w.psum = up(w.hist + 4 * (E + 1) * w.nchunk, 256);
    w.first = up(w.psum + 4 * E * w.nchunk, 256);
    w.psum_total = up(w.first + 4 * E, 256);
    w.bytes = up(w.psum_total + 4 * E, 256);
    return w;
}

int launch_moe_route(const RouteArgs &a, int num_sms, cudaStream_t s) {
    const RouteWorkspace w = route_workspace(a.T, a.E);
    const int want_p = a.prob_sums || a.loss;
    if (a.bf16 ? route_topk<uint16_t>(a, w, want_p, s) : route_topk<float>(a, w, want_p, s)) return 1;
    const int E = (int)a.E;
    uint32_t *hist = reinterpret_cast<uint32_t *>(a.ws + w.hist);
    int32_t *first = reinterpret_cast<int32_t *>(a.ws + w.first);
    float *psum = want_p ? reinterpret_cast<float *>(a.ws + w.psum) : nullptr;
    float *total = want_p ? reinterpret_cast<float *>(a.ws + w.psum_total) : nullptr;
    if (launch_dependent(route_scan_kernel, dim3(E + 1), dim3(256), 0, s, hist, (const float *)psum, w.nchunk, E,
                         a.counts, first, total) != cudaSuccess)
        return 1;
    const int64_t n = a.T * a.topk;
    const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>((n + 1023) / 1024, (int64_t)num_sms * 8));
    if (launch_dependent(route_place_kernel, dim3(grid), dim3(256), 0, s, (const int32_t *)a.ids, a.rows, (uint32_t)n,
                         unit_div((uint32_t)a.topk), E, w.nchunk, (const uint32_t *)hist, (const int32_t *)a.counts, (const int32_t *)first,
                         (const float *)total, a.coef, a.row_index, a.row_off, a.sf_row_off, a.prob_sums,
                         a.loss) != cudaSuccess)
        return 1;
    return launched();
}

int launch_moe_route_bwd(const RouteBwdArgs &a, int num_sms, cudaStream_t s) {
    // the softmax over the chosen experts alone needs their weights, not the logits
    if (!a.renorm || a.dloss)
        return a.bf16 ? route_bwd<uint16_t, true>(a, num_sms, s) : route_bwd<float, true>(a, num_sms, s);
    return a.bf16 ? route_bwd<uint16_t, false>(a, num_sms, s) : route_bwd<float, false>(a, num_sms, s);
}

int launch_moe_combine(const uint16_t *y, int64_t R, int64_t H, int64_t ldy, const int32_t *rows, const float *weights,
                       int64_t T, int topk, uint16_t *out, int64_t ldo, int, cudaStream_t s) {
    combine_kernel<<<dim3((unsigned)T, (unsigned)((H + 1023) / 1024)), 128, 0, s>>>(y, R, H, ldy, rows, weights, topk,
                                                                                     out, ldo);
    return launched();
}

int launch_moe_combine_bwd(const uint16_t *dout, int64_t ldo, const uint16_t *y, int64_t ldy, const uint8_t *codes,
                           const uint8_t *sf, int64_t R, int64_t H, const int32_t *rows, const float *weights,
                           int64_t T, int topk, uint16_t *dy, int64_t lddy, float *dweights, int, cudaStream_t s) {
    if (y)
        combine_bwd_kernel<false><<<(unsigned)T, 256, 0, s>>>(dout, ldo, y, ldy, codes, sf, R, H, rows, weights, topk,
                                                              dy, lddy, dweights);
    else
        combine_bwd_kernel<true><<<(unsigned)T, 256, 0, s>>>(dout, ldo, y, ldy, codes, sf, R, H, rows, weights, topk,
                                                             dy, lddy, dweights);
    return launched();
}

int launch_swiglu_ckpt(const uint16_t *u, int64_t M, int64_t F, int64_t ldu, const int32_t *n_rows, uint16_t *h,
                       int64_t ldh, uint8_t *codes, uint8_t *sf, unsigned int *amax, int num_sms, cudaStream_t s) {
    const unsigned grid = (unsigned)std::min<int64_t>((M * (F / 16) + 255) / 256, (int64_t)num_sms * 8);
    swiglu_ckpt_kernel<<<grid, 256, 0, s>>>(u, M, F, ldu, unit_div((uint32_t)(F / 16)), n_rows, h, ldh, codes, sf,
                                            amax);
    return launched();
}

int launch_swiglu_ckpt_bwd(const uint16_t *dh, int64_t lddh, const uint8_t *codes, const uint8_t *sf, int64_t M,
                           int64_t F, const int32_t *n_rows, uint16_t *du, int64_t lddu, uint16_t *h, int64_t ldh,
                           int num_sms, cudaStream_t s) {
    const unsigned grid = (unsigned)std::min<int64_t>((M * (F / 16) + 255) / 256, (int64_t)num_sms * 8);
    const UnitDiv per = unit_div((uint32_t)(F / 16));
    if (h) swiglu_ckpt_bwd_kernel<true><<<grid, 256, 0, s>>>(dh, lddh, codes, sf, M, F, per, n_rows, du, lddu, h, ldh);
    else swiglu_ckpt_bwd_kernel<false><<<grid, 256, 0, s>>>(dh, lddh, codes, sf, M, F, per, n_rows, du, lddu, h, ldh);
    return launched();
}

}  // namespace bsq
