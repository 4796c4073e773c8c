// What trains on decoded tokens: the log-probability of one token of every row (with the entropy of the row's
// distribution), the clipped policy loss and the preference loss made of it, and their gradients.
//
// With s = x / T, y the row's token, R = sum of e^{s_v} over v != y and d = log R - s_y:
//   log p_y = -log(1 + e^d),  q = 1 - p_y = 1 / (1 + e^-d),  log p_v = s_v - log R + log q   (v != y)
//   H = p_y log(1 + e^d) + q (log(1 + e^-d) + H_R),  H_R the entropy of the others among themselves
// The token is left out of the sum, which has the maximum of what is in it, so that 1 - p_y of a token that has
// nearly all the mass (most tokens of a trained model) is a quotient and no difference.  For dL/dlog p_y = a,
// dL/dH = h:
//   dL/dx_v = -p_v (a + h (log p_v + H)) / T,   dL/dx_y = (a q - h p_y (log p_y + H)) / T
//
// stats_kernel streams a row and leaves what the gradient needs (32 bytes a row), grad_kernel streams it again.
#include <cmath>

#include "vocab_rows.cuh"

namespace dspark {

namespace {

constexpr int kTokVec = 4;                                   // vectors a thread holds at a time
constexpr int kGradVecs = 2048;                              // vectors of a row that a CTA of the gradient takes
constexpr float kLn2 = 0.693147180559945f;

enum TokenOp : int { kScore, kPolicy, kPreference };

// What a row leaves for its gradient (the caller's saved array).
struct __align__(16) RowSaved {
    float m, f;                                              // the others' maximum; q / (R T) by it, negative: gradient 0
    float level;                                             // log p_v + H less the exponent's part (preference: log p_y)
    float q, py;                                             // q / T, p_y (log p_y + H) / T (preference: log p_y's low part)
    float a, h;                                              // dL/dlog p_y, dL/dH before the upstream gradient
    int pair;                                                // (preference) whose upstream gradient, -1: none
};
static_assert(sizeof(RowSaved) == 4 * DSPARK_SAVED_FLOATS, "the header's size");

struct TokArgs {
    int V, op;
    float c, inv_t;                                          // log2(e) / T, 1 / T
    long long x_stride, g_stride;
    const void* x;
    void* g;
    const int* tokens;
    const float* weights;                                    // (policy) a row of weight 0 is not read
    float* logp;
    float* entropy;
    float* loss;
    float* kl;
    RowSaved* saved;
    int* row_status;
    const float* old_lp;
    const float* ref_lp;
    const float* adv;
    float low, high, kl_coef, ent_coef;                      // 1 - clip_low, 1 + clip_high
    const float* up;                                         // upstream gradients, null: 1
    const float* up_entropy;                                 // (score) null: 0
    int n_up;                                                // (preference) entries of up
    int log_c, splits;                                       // stats: log2 of the CTAs of a row; gradient: CTAs of a row
};

// A sum of exponentials e by ExpRef(m), and the sum w of e times its exponent (base 2).
struct EntSum {
    float m, sum, w;
};
// what a sum by `from` scales by to be by `to`, and what its exponents gain
__device__ __forceinline__ float shift_of(float from, float to, float c) {
    const ExpRef a(from, c), b(to, c);
    return fmaxf(a.whole && b.whole ? a.r - b.r : (from - to) * c, -16384.f);
}
template <bool ENT>
__device__ __forceinline__ void rebase_to(EntSum& a, float to, float c) {
    if (a.m > -INFINITY) {
        const float by = shift_of(a.m, to, c), k = ex2_approx(by);
        if (ENT) a.w = fmaf(a.sum, by, a.w) * k;
        a.sum *= k;
    }
    a.m = to;
}
// The sum over groups of `lanes` lanes, in each of them.
template <bool ENT>
__device__ __forceinline__ EntSum lanes_join(EntSum a, int lanes, float c) {
    float m = a.m;
    for (int o = lanes / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (m > -INFINITY) rebase_to<ENT>(a, m, c);
    for (int o = lanes / 2; o; o >>= 1) {
        a.sum += __shfl_xor_sync(0xffffffffu, a.sum, o);
        if (ENT) a.w += __shfl_xor_sync(0xffffffffu, a.w, o);
    }
    return a;
}

// Add U vectors whose maximum is bm.
template <int SX, bool ENT, int U>
__device__ __forceinline__ void add_vecs(RunSum& es, float& w, const uint4 (&v)[U], float bm, float c) {
    constexpr int VE = 16 / SX;
    if (!ENT) {
        add_exps<SX>(es, v, bm, c);
        return;
    }
    const float m = fmaxf(es.m, bm), t = m * c, r = ceilf(t);
    EntSum was{es.m, es.sum, w};
    if (m > -INFINITY) rebase_to<true>(was, m, c);
    if (fabsf(t) < 4194304.f) {
        const unsigned long long c2 = pack2(c, c), r2 = pack2(-r, -r);
        unsigned long long acc = pack2(was.sum, 0.f), accw = pack2(was.w, 0.f);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < VE / 2; ++k) {
                float lo, hi;
                unpack2(fma2(pair_of<SX>(v[u], k), c2, r2), lo, hi);
                const unsigned long long e = pack2(ex2_approx(lo), ex2_approx(hi));
                acc = add2(acc, e);
                accw = fma2(e, pack2(fmaxf(lo, -16384.f), fmaxf(hi, -16384.f)), accw);   // (0 times -inf)
            }
        float lo, hi;
        unpack2(acc, lo, hi);
        es.sum = lo + hi;
        unpack2(accw, lo, hi);
        w = lo + hi;
    } else {
        const float ref = m > -INFINITY ? m : 0.f;
        es.sum = was.sum;
        w = was.w;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int q = 0; q < VE; ++q) {
                const float z = (elem<SX>(v[u], q) - ref) * c, e = ex2_approx(z);
                es.sum += e;
                w = fmaf(e, fmaxf(z, -16384.f), w);
            }
    }
    es.m = m;
    es.r = r;
}

// Replace logit i of a vector whose first is i0.
template <int SX>
__device__ __forceinline__ void patch(uint4& v, int lane, uint32_t bits) {
#pragma unroll
    for (int q = 0; q < 16 / SX; ++q)
        if (q == lane) put_bits<SX>(v, q, bits);
}

// log(1 + e^d) and 1 / (1 + e^-d)
__device__ __forceinline__ TwoFloat softplus(const TwoFloat& d) {
    if (!(d.hi > -INFINITY)) return TwoFloat{d.hi == d.hi ? 0.f : NAN, 0.f};
    if (d.hi > 0.f) {
        const float t = log1pf(expf(-d.hi));
        if (!(d.hi < INFINITY)) return TwoFloat{d.hi, 0.f};
        const TwoFloat s = two_sum(d.hi, t);
        return TwoFloat{s.hi, s.lo + d.lo * (1.f - t)};
    }
    const float e = expf(d.hi);
    return TwoFloat{log1pf(fmaf(e, d.lo, e)), 0.f};
}
__device__ __forceinline__ float sigmoid(float d) { return d > 0.f ? 1.f / (1.f + expf(-d)) : expf(d) / (1.f + expf(d)); }

// e^D - D - 1 without the difference of near ones: its series where D is small (relative remainder below 2^-24)
__device__ __forceinline__ float k3_of(float D) {
    if (fabsf(D) < 0.25f) {
        float s = 1.f + D * (1.f / 9.f);
        s = fmaf(D * s, 1.f / 8.f, 1.f);
        s = fmaf(D * s, 1.f / 7.f, 1.f);
        s = fmaf(D * s, 1.f / 6.f, 1.f);
        s = fmaf(D * s, 1.f / 5.f, 1.f);
        s = fmaf(D * s, 1.f / 4.f, 1.f);
        s = fmaf(D * s, 1.f / 3.f, 1.f);
        return 0.5f * D * D * s;
    }
    return expm1f(D) - D;
}

struct PolicyRow {
    float w, old, ref, adv;
};

// One row's results from its sum over the other tokens and its token's logit, by one thread.
template <bool ENT>
__device__ __forceinline__ RowSaved row_end(const TokArgs& a, long long row, const EntSum& es, float xy, const PolicyRow& pr) {
    RowSaved s{0.f, -1.f, 0.f, 0.f, 0.f, 0.f, 0.f, -1};
    int status = 0;
    const bool none = !(es.m > -INFINITY) && es.sum == es.sum;   // no other token has any mass
    TwoFloat d{-INFINITY, 0.f};
    if (!(xy < INFINITY) || es.sum != es.sum || !(es.m < INFINITY) || (none && !(xy > -INFINITY))) {
        status = DSPARK_ROW_NONFINITE;
    } else if (!none) {
        const ExpRef ref(es.m, a.c);
        if (!(xy > -INFINITY)) {
            d.hi = INFINITY;
        } else if (ref.whole) {
            const TwoFloat p = two_prod(xy, a.c), by = two_sum(ref.r, -p.hi);
            d = fabsf(p.hi) < INFINITY ? TwoFloat{by.hi, by.lo - p.lo} * ln2_two() + log_two(es.sum)
                                       : TwoFloat{xy > 0.f ? -INFINITY : INFINITY, 0.f};
        } else {
            const float by = (es.m - xy) * a.c;
            d = fabsf(by) < INFINITY ? TwoFloat{by, 0.f} * ln2_two() + log_two(es.sum) : TwoFloat{by, 0.f};
        }
    }
    TwoFloat lp{NAN, 0.f};
    float H = NAN;
    if (!status) {
        const TwoFloat sp = softplus(d);
        lp = -sp;
        const float py = sigmoid(-d.hi), q = sigmoid(d.hi), sm = softplus(-d).hi;   // -log q
        const float lr = none ? 0.f : logf(es.sum);
        H = 0.f;
        if (ENT) H = (py > 0.f ? py * sp.hi : 0.f) + (none || q == 0.f ? 0.f : q * (sm + (lr - kLn2 * (es.w / es.sum))));
        s.m = none ? 0.f : es.m;
        s.f = none ? 0.f : q / es.sum * a.inv_t;
        s.level = none || !(sm < INFINITY) ? 0.f : H - lr - sm;
        s.q = q * a.inv_t;
        s.py = py > 0.f ? py * (lp.hi + H) * a.inv_t : 0.f;
    }
    const float logp = lp.hi + lp.lo;
    if (a.op == kPolicy) {
        float loss = NAN, kl = 0.f;
        if (!status) {
            const float rho = expf((lp.hi - pr.old) + lp.lo);
            // the smaller of rho A and the clipped rho times A; clipping binds above for a gain, below for a loss
            float gain = 0.f, by_lp = 0.f;
            if (pr.adv != 0.f) {
                const bool binds = pr.adv > 0.f ? rho > a.high : rho < a.low;
                gain = (binds ? (pr.adv > 0.f ? a.high : a.low) : rho) * pr.adv;
                by_lp = binds ? 0.f : -gain;
            }
            loss = -gain;
            if (a.ref_lp) {
                const float D = (pr.ref - lp.hi) - lp.lo;
                kl = k3_of(D);
                if (a.kl_coef != 0.f) {
                    loss = fmaf(a.kl_coef, kl, loss);
                    by_lp = fmaf(-a.kl_coef, expm1f(D), by_lp);
                }
            }
            if (a.ent_coef != 0.f) loss = fmaf(-a.ent_coef, H, loss);
            loss *= pr.w;
            s.a = pr.w * by_lp;
            s.h = -pr.w * a.ent_coef;
            if (!(fabsf(loss) < INFINITY) || !(fabsf(s.a) < INFINITY)) {
                status = DSPARK_ROW_NONFINITE;
                loss = NAN;
                s.f = -1.f;
            }
        }
        a.loss[row] = loss;
        if (a.kl) a.kl[row] = status ? NAN : kl;
    } else if (a.op == kScore) {
        s.a = 1.f;
        s.h = ENT ? 1.f : NAN;                               // an entropy's gradient needs a call that asked for the entropy
    } else if (!status) {
        s.level = lp.hi;                                     // a sequence's log ratios cancel: the sum takes both parts
        s.py = lp.lo;
    }
    if (status && a.op != kPolicy) s.f = -1.f;
    if (a.logp) a.logp[row] = status ? NAN : logp;
    if (ENT && a.entropy) a.entropy[row] = status ? NAN : H;
    a.row_status[row] = status;
    return s;
}

// A row that is not read: without a token, of weight 0, or (status) with a token out of range.
__device__ __forceinline__ void row_skipped(const TokArgs& a, long long row, int status) {
    const float v = status ? NAN : 0.f;
    if (a.logp) a.logp[row] = v;
    if (a.entropy) a.entropy[row] = v;
    if (a.loss) a.loss[row] = v;
    if (a.kl) a.kl[row] = v;
    if (a.saved) a.saved[row] = RowSaved{0.f, -1.f, 0.f, 0.f, 0.f, 0.f, 0.f, -1};
    a.row_status[row] = status;
}

template <int SX, bool ENT>
__global__ void __launch_bounds__(kRowThreads) stats_kernel(TokArgs a) {
    __shared__ EntSum s_warp[kRowWarps];
    __shared__ EntSum s_peer[kMaxCluster];                   // (in the row's first CTA) written by the cluster's
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = 1 << a.log_c, rank = blockIdx.x & (C - 1);
    const long long row = blockIdx.x >> a.log_c;
    if (C > 1) cluster_arrive_relaxed();
    pdl_wait();
    const int y = a.tokens[row];
    PolicyRow pr{1.f, 0.f, 0.f, 0.f};
    if (a.op == kPolicy && a.weights) pr.w = a.weights[row];
    const bool bad = y < -1 || y >= a.V;
    if (bad || y < 0 || pr.w == 0.f) {                       // the same branch in every CTA of the row
        if (rank == 0 && tid == 0) row_skipped(a, row, bad ? DSPARK_ROW_BAD_TOKEN : 0);
        if (C > 1) cluster_wait();
        return;
    }
    const VocabRow<SX> x(a.x, row, a.x_stride, a.V);
    const int k0 = static_cast<int>(static_cast<long long>(x.nvec) * rank >> a.log_c);
    const int k1 = static_cast<int>(static_cast<long long>(x.nvec) * (rank + 1) >> a.log_c);
    constexpr int VE = VocabRow<SX>::VE;
    const int ky = (y + x.a0) / VE, qy = (y + x.a0) % VE;    // the token's vector and lane
    float xy = 0.f;
    if (rank == 0 && tid == 0) {
        xy = load_logit<SX>(x, y);
        if (a.op == kPolicy) {
            pr.old = a.old_lp[row];
            pr.adv = a.adv[row];
            if (a.ref_lp) pr.ref = a.ref_lp[row];
        }
    }
    RunSum run;
    float w = 0.f;
    int k = k0 + tid;
    for (; k + (kTokVec - 1) * kRowThreads < k1; k += kTokVec * kRowThreads) {
        uint4 v[kTokVec];
#pragma unroll
        for (int u = 0; u < kTokVec; ++u) v[u] = load_vec<SX>(x, k + u * kRowThreads, k1);
#pragma unroll
        for (int u = 0; u < kTokVec; ++u)
            if (k + u * kRowThreads == ky) patch<SX>(v[u], qy, ninf_bits<SX>());
        add_vecs<SX, ENT>(run, w, v, vecs_max<SX>(v), a.c);
    }
    for (; k < k1; k += kRowThreads) {
        uint4 v[1] = {load_vec<SX>(x, k, k1)};
        if (k == ky) patch<SX>(v[0], qy, ninf_bits<SX>());
        add_vecs<SX, ENT>(run, w, v, vecs_max<SX>(v), a.c);
    }
    EntSum es = lanes_join<ENT>(EntSum{run.m, run.sum, w}, 32, a.c);
    if (lane == 0) s_warp[warp] = es;
    __syncthreads();
    if (warp == 0) es = lanes_join<ENT>(s_warp[lane & (kRowWarps - 1)], kRowWarps, a.c);
    if (C > 1) {
        cluster_wait();                                      // the row's first CTA is there
        if (tid == 0) {
            const unsigned at = peer_addr(&s_peer[rank], 0);
            asm volatile("st.shared::cluster.f32 [%0], %1;" :: "r"(at), "f"(es.m) : "memory");
            asm volatile("st.shared::cluster.f32 [%0], %1;" :: "r"(at + 4), "f"(es.sum) : "memory");
            asm volatile("st.shared::cluster.f32 [%0], %1;" :: "r"(at + 8), "f"(es.w) : "memory");
        }
        cluster_arrive();
        cluster_wait();
        if (rank == 0 && warp == 0)
            es = lanes_join<ENT>((lane & (kMaxCluster - 1)) < C ? s_peer[lane & (kMaxCluster - 1)] : EntSum{-INFINITY, 0.f, 0.f},
                                 kMaxCluster, a.c);
    }
    if (rank == 0 && tid == 0) {
        const RowSaved s = row_end<ENT>(a, row, es, xy, pr);
        if (a.saved) a.saved[row] = s;
    }
}

template <int SX>
__device__ __forceinline__ void store_vec(const VocabRow<SX>& g, int i0, const uint4& w, bool same_phase) {
    constexpr int VE = 16 / SX;
    unsigned char* p = const_cast<unsigned char*>(g.p);
    if (same_phase && i0 >= 0 && i0 + VE <= g.V) {
        st_vec16(p + static_cast<long long>(i0) * SX, w);
        return;
    }
#pragma unroll
    for (int q = 0; q < VE; ++q) {
        const int i = i0 + q;
        if (i < 0 || i >= g.V) continue;
        if (SX == 2) reinterpret_cast<unsigned short*>(p)[i] = static_cast<unsigned short>(word_of(w, q >> 1) >> (16 * (q & 1)));
        else reinterpret_cast<unsigned*>(p)[i] = word_of(w, q);
    }
}

// What a row's gradient is made with: e_v (a0 + a1 z_v) for exponentials e_v = 2^z_v, and the token's own.
struct RowGrad {
    float a0, a1, at_y;
};
__device__ __forceinline__ RowGrad row_grad(const RowSaved& s, float a, float h) {
    return RowGrad{-s.f * fmaf(h, s.level, a), -s.f * h * kLn2, a * s.q - h * s.py};
}

template <int SX, bool ENT>
__device__ __forceinline__ uint4 grad_vec(const uint4& v, const ExpRef& ref, const RowGrad& rg) {
    constexpr int VE = 16 / SX;
    float f[VE];
    const unsigned long long c2 = pack2(ref.c, ref.c), r2 = pack2(-ref.r, -ref.r);
#pragma unroll
    for (int h = 0; h < VE / 2; ++h) {
        float lo, hi;
        if (ref.whole) {
            unpack2(fma2(pair_of<SX>(v, h), c2, r2), lo, hi);
        } else {
            lo = (elem<SX>(v, 2 * h) - ref.m) * ref.c;
            hi = (elem<SX>(v, 2 * h + 1) - ref.m) * ref.c;
        }
        const unsigned long long e = pack2(ex2_approx(lo), ex2_approx(hi));
        unsigned long long k = pack2(rg.a0, rg.a0);
        if (ENT) k = fma2(pack2(fmaxf(lo, -16384.f), fmaxf(hi, -16384.f)), pack2(rg.a1, rg.a1), k);
        unpack2(mul2(e, k), f[2 * h], f[2 * h + 1]);
    }
    if (SX == 2) return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4 % VE], f[5 % VE]), pack_bf16(f[6 % VE], f[7 % VE]));
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}

template <int SX, bool ENT>
__global__ void __launch_bounds__(kRowThreads) grad_kernel(TokArgs a) {
    constexpr int VE = VocabRow<SX>::VE;
    const long long row = blockIdx.x / a.splits;
    const int part = blockIdx.x % a.splits;
    pdl_wait();
    const VocabRow<SX> x(a.x, row, a.x_stride, a.V), g(a.g, row, a.g_stride, a.V);
    const bool same_phase = x.a0 == g.a0;
    const int k0 = part * kGradVecs, k1 = min(x.nvec, k0 + kGradVecs);
    RowSaved s = a.saved[row];
    const int y = a.tokens[row];
    if (a.op == kPreference) s.level = s.py = 0.f;
    float ga = s.a, gh = s.h;
    if (a.op == kScore) {
        ga = a.up ? a.up[row] : 0.f;
        gh = ENT && a.up_entropy ? s.h * a.up_entropy[row] : 0.f;
    } else if (a.op == kPolicy) {
        const float u = a.up ? a.up[row] : 1.f;
        ga *= u;
        gh *= u;
    } else if (a.up) {
        ga = s.pair >= 0 && s.pair < a.n_up ? ga * a.up[s.pair] : 0.f;
    }
    if (s.f < 0.f || (ga == 0.f && gh == 0.f)) {
        for (int k = k0 + threadIdx.x; k < k1; k += kRowThreads) store_vec<SX>(g, x.first(k), make_uint4(0, 0, 0, 0), same_phase);
        return;
    }
    const RowGrad rg = row_grad(s, ga, gh);
    const ExpRef ref(s.m, a.c);
    const int ky = (y + x.a0) / VE, qy = (y + x.a0) % VE;
    int k = k0 + threadIdx.x;
    for (; k + (kTokVec - 1) * kRowThreads < k1; k += kTokVec * kRowThreads) {
        uint4 v[kTokVec];
#pragma unroll
        for (int u = 0; u < kTokVec; ++u) v[u] = load_vec<SX>(x, k + u * kRowThreads, k1);
#pragma unroll
        for (int u = 0; u < kTokVec; ++u) {
            uint4 o = grad_vec<SX, ENT>(v[u], ref, rg);
            if (k + u * kRowThreads == ky) patch<SX>(o, qy, to_bits<SX>(rg.at_y));
            store_vec<SX>(g, x.first(k + u * kRowThreads), o, same_phase);
        }
    }
    for (; k < k1; k += kRowThreads) {
        uint4 o = grad_vec<SX, ENT>(load_vec<SX>(x, k, k1), ref, rg);
        if (k == ky) patch<SX>(o, qy, to_bits<SX>(rg.at_y));
        store_vec<SX>(g, x.first(k), o, same_phase);
    }
}

// ---------------------------------------------------------------- pairs of sequences
struct PairArgs {
    int R, P, mean;
    float beta, margin, smoothing;
    const int* offsets;
    const int* tokens;
    const float* ref_lp;
    const float* weights;
    const int* row_status;
    float* loss;
    float* rewards;
    int* pair_status;
    RowSaved* saved;
};

// A CTA to a pair: the two sequences' sums in pairs of floats (they cancel), the loss, and each row's dL/dlog p.
__global__ void __launch_bounds__(kRowThreads) pair_kernel(PairArgs a) {
    __shared__ TwoFloat s_sum[2][kRowWarps];
    __shared__ int s_count[2][kRowWarps];
    __shared__ float s_coef[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, p = blockIdx.x;
    pdl_wait();
    // the offsets up to this pair's last ascend and stay inside the rows
    bool bad = false;
    for (int k = tid; k < 2 * p + 2; k += kRowThreads) bad = bad || a.offsets[k] > a.offsets[k + 1];
    const int lo = a.offsets[2 * p], mid = a.offsets[2 * p + 1], hi = a.offsets[2 * p + 2];
    if (__syncthreads_or(bad || a.offsets[0] < 0 || hi > a.R)) {
        if (tid == 0) {
            a.loss[p] = NAN;
            if (a.rewards) a.rewards[2 * p] = a.rewards[2 * p + 1] = NAN;
            a.pair_status[p] = DSPARK_ROW_BAD_PARAMS;
        }
        return;
    }
    int status = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        TwoFloat sum{0.f, 0.f};
        int count = 0;
        for (int r = (k ? mid : lo) + tid; r < (k ? hi : mid); r += kRowThreads) {
            status |= a.row_status[r];
            if (a.tokens[r] < 0) continue;
            ++count;
            const float lp = a.saved[r].level;
            TwoFloat gain = a.ref_lp ? two_sum(lp, -a.ref_lp[r]) : TwoFloat{lp, 0.f};
            gain.lo += a.saved[r].py;
            sum = fabsf(gain.hi) < INFINITY && fabsf(sum.hi) < INFINITY ? sum + gain : TwoFloat{sum.hi + gain.hi, 0.f};
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const TwoFloat other{__shfl_xor_sync(0xffffffffu, sum.hi, o), __shfl_xor_sync(0xffffffffu, sum.lo, o)};
            sum = fabsf(other.hi) < INFINITY && fabsf(sum.hi) < INFINITY ? sum + other : TwoFloat{sum.hi + other.hi, 0.f};
            count += __shfl_xor_sync(0xffffffffu, count, o);
        }
        if (lane == 0) {
            s_sum[k][warp] = sum;
            s_count[k][warp] = count;
        }
    }
    status = __reduce_or_sync(0xffffffffu, status);
    __shared__ int s_status[kRowWarps];
    if (lane == 0) s_status[warp] = status;
    __syncthreads();
    if (tid == 0) {
        TwoFloat reward[2];
        float norm[2];
        int st = 0;
        for (int w = 0; w < kRowWarps; ++w) st |= s_status[w];
        for (int k = 0; k < 2; ++k) {
            TwoFloat sum{0.f, 0.f};
            int count = 0;
            for (int w = 0; w < kRowWarps; ++w) {
                const TwoFloat other = s_sum[k][w];
                sum = fabsf(other.hi) < INFINITY && fabsf(sum.hi) < INFINITY ? sum + other : TwoFloat{sum.hi + other.hi, 0.f};
                count += s_count[k][w];
            }
            norm[k] = a.mean ? static_cast<float>(max(count, 1)) : 1.f;
            reward[k] = fabsf(sum.hi) < INFINITY ? sum * TwoFloat{a.beta, 0.f} / TwoFloat{norm[k], 0.f} : TwoFloat{sum.hi, 0.f};
        }
        TwoFloat z{(reward[0].hi - reward[1].hi) - a.margin, 0.f};
        if (fabsf(z.hi) < INFINITY) z = reward[0] + -reward[1] + TwoFloat{-a.margin, 0.f};
        if (!st && z.hi != z.hi) st = DSPARK_ROW_NONFINITE;
        const float w = a.weights ? a.weights[p] : 1.f, e = a.smoothing;
        const TwoFloat down = softplus(-z), up = softplus(z);   // -log sigma(z), -log sigma(-z)
        float loss = 0.f, by_z = 0.f;
        if (w != 0.f) {
            loss = (1.f - e) * (down.hi + down.lo);
            if (e > 0.f) loss += e * (up.hi + up.lo);
            loss *= w;
            by_z = w * (e * sigmoid(z.hi) - (1.f - e) * sigmoid(-z.hi));
        }
        a.loss[p] = st ? NAN : loss;
        if (a.rewards)
            for (int k = 0; k < 2; ++k) a.rewards[2 * p + k] = st ? NAN : reward[k].hi + reward[k].lo;
        a.pair_status[p] = st;
        s_coef[0] = st ? 0.f : by_z * a.beta / norm[0];
        s_coef[1] = st ? 0.f : -by_z * a.beta / norm[1];
    }
    __syncthreads();
    for (int r = lo + tid; r < hi; r += kRowThreads) {
        a.saved[r].a = s_coef[r >= mid];
        a.saved[r].pair = p;
    }
}

// ---------------------------------------------------------------- host
dspark_status_t token_args(const void* logits, const dspark_token_params_t* p, const void* grad, TokArgs* a, int* sx) {
    if (!logits || !p || !p->tokens) return DSPARK_ERR_INVALID_ARG;
    if (p->n_rows < 1 || p->n_rows > DSPARK_MAX_ROWS || p->V < 1 || p->V > DSPARK_MAX_V) return DSPARK_ERR_INVALID_ARG;
    if (p->logits_dtype != DSPARK_BF16 && p->logits_dtype != DSPARK_FP32) return DSPARK_ERR_INVALID_ARG;
    const float c = kLog2E / p->temperature, inv_t = 1.f / p->temperature;
    if (!(p->temperature > 0.f) || !(c > 0.f) || !(c < INFINITY) || !(inv_t < INFINITY)) return DSPARK_ERR_INVALID_ARG;
    *sx = p->logits_dtype == DSPARK_BF16 ? 2 : 4;
    if (p->logits_stride < p->V || reinterpret_cast<uintptr_t>(logits) % *sx) return DSPARK_ERR_INVALID_ARG;
    if (grad && (p->grad_stride < p->V || reinterpret_cast<uintptr_t>(grad) % *sx)) return DSPARK_ERR_INVALID_ARG;
    if (grad == logits && p->grad_stride != p->logits_stride) return DSPARK_ERR_INVALID_ARG;
    a->V = p->V;
    a->c = c;
    a->inv_t = inv_t;
    a->x = logits;
    a->x_stride = p->logits_stride;
    a->g = const_cast<void*>(grad);
    a->g_stride = p->grad_stride;
    a->tokens = p->tokens;
    a->row_status = p->row_status;
    return DSPARK_OK;
}

bool misplaced(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

dspark_status_t launch_stats(TokArgs& a, int sx, bool entropy, const dspark_token_params_t* p) {
    const int nvec = max_vectors(p->V, sx);
    int C = 1;
    a.log_c = 0;
    while (C < kMaxCluster && nvec >= C * 512 && static_cast<long long>(p->n_rows) * 2 * C <= 640) {
        C *= 2;
        ++a.log_c;
    }
    auto kern = sx == 2 ? (entropy ? stats_kernel<2, true> : stats_kernel<2, false>)
                        : (entropy ? stats_kernel<4, true> : stats_kernel<4, false>);
    const cudaError_t e = launch_cluster(kern, static_cast<unsigned>(p->n_rows) * C, kRowThreads, C, 0,
                                         static_cast<cudaStream_t>(p->stream), a);
    return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

dspark_status_t launch_grad(TokArgs& a, int sx, bool entropy, const dspark_token_params_t* p) {
    a.splits = (max_vectors(p->V, sx) + kGradVecs - 1) / kGradVecs;
    const long long grid = static_cast<long long>(p->n_rows) * a.splits;
    if (grid > 0x7fffffffLL) return DSPARK_ERR_UNSUPPORTED;
    auto kern = sx == 2 ? (entropy ? grad_kernel<2, true> : grad_kernel<2, false>)
                        : (entropy ? grad_kernel<4, true> : grad_kernel<4, false>);
    const cudaError_t e = launch_cluster(kern, static_cast<unsigned>(grid), kRowThreads, 1, 0, static_cast<cudaStream_t>(p->stream), a);
    return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

dspark_status_t policy_args(const dspark_policy_t* o, TokArgs* a) {
    if (!o || !o->old_logprobs || !o->advantages) return DSPARK_ERR_INVALID_ARG;
    if (!(o->clip_low >= 0.f) || !(o->clip_low <= 1.f) || !(o->clip_high >= 0.f) || !(o->clip_high < INFINITY)) return DSPARK_ERR_INVALID_ARG;
    if (!std::isfinite(o->kl_coef) || !std::isfinite(o->entropy_coef)) return DSPARK_ERR_INVALID_ARG;
    if (o->kl_coef != 0.f && !o->ref_logprobs) return DSPARK_ERR_INVALID_ARG;
    a->op = kPolicy;
    a->old_lp = o->old_logprobs;
    a->ref_lp = o->ref_logprobs;
    a->adv = o->advantages;
    a->weights = o->weights;
    a->low = 1.f - o->clip_low;
    a->high = 1.f + o->clip_high;
    a->kl_coef = o->kl_coef;
    a->ent_coef = o->entropy_coef;
    return DSPARK_OK;
}

}  // namespace
}  // namespace dspark

using namespace dspark;

extern "C" {

dspark_status_t dspark_token_logprobs(const void* logits, const dspark_token_params_t* params, float* out_logprobs,
                                      float* out_entropy, float* out_saved) {
    TokArgs a{};
    int sx = 0;
    if (const dspark_status_t st = token_args(logits, params, nullptr, &a, &sx); st != DSPARK_OK) return st;
    if (!out_logprobs || !params->row_status || misplaced(out_saved, 16)) return DSPARK_ERR_INVALID_ARG;
    a.op = kScore;
    a.logp = out_logprobs;
    a.entropy = out_entropy;
    a.saved = reinterpret_cast<RowSaved*>(out_saved);
    return launch_stats(a, sx, out_entropy != nullptr, params);
}

dspark_status_t dspark_token_logprobs_backward(const void* logits, const dspark_token_params_t* params, const float* saved,
                                               const float* grad_logprobs, const float* grad_entropy, void* out_grad) {
    TokArgs a{};
    int sx = 0;
    if (!out_grad || !saved || misplaced(saved, 16) || (!grad_logprobs && !grad_entropy)) return DSPARK_ERR_INVALID_ARG;
    if (const dspark_status_t st = token_args(logits, params, out_grad, &a, &sx); st != DSPARK_OK) return st;
    a.op = kScore;
    a.saved = reinterpret_cast<RowSaved*>(const_cast<float*>(saved));
    a.up = grad_logprobs;
    a.up_entropy = grad_entropy;
    return launch_grad(a, sx, grad_entropy != nullptr, params);
}

dspark_status_t dspark_policy_loss(const void* logits, const dspark_policy_t* policy, const dspark_token_params_t* params,
                                   float* out_loss, float* out_logprobs, float* out_entropy, float* out_kl, float* out_saved,
                                   void* out_grad) {
    TokArgs a{};
    int sx = 0;
    if (const dspark_status_t st = token_args(logits, params, out_grad, &a, &sx); st != DSPARK_OK) return st;
    if (const dspark_status_t st = policy_args(policy, &a); st != DSPARK_OK) return st;
    if (!out_loss || !params->row_status || misplaced(out_saved, 16)) return DSPARK_ERR_INVALID_ARG;
    if ((out_grad && !out_saved) || (out_kl && !policy->ref_logprobs)) return DSPARK_ERR_INVALID_ARG;
    a.loss = out_loss;
    a.logp = out_logprobs;
    a.entropy = out_entropy;
    a.kl = out_kl;
    a.saved = reinterpret_cast<RowSaved*>(out_saved);
    const dspark_status_t st = launch_stats(a, sx, out_entropy || policy->entropy_coef != 0.f, params);
    if (st != DSPARK_OK || !out_grad) return st;
    return launch_grad(a, sx, policy->entropy_coef != 0.f, params);
}

dspark_status_t dspark_policy_loss_backward(const void* logits, const dspark_policy_t* policy, const dspark_token_params_t* params,
                                            const float* saved, const float* grad_loss, void* out_grad) {
    TokArgs a{};
    int sx = 0;
    if (!out_grad || !saved || misplaced(saved, 16)) return DSPARK_ERR_INVALID_ARG;
    if (const dspark_status_t st = token_args(logits, params, out_grad, &a, &sx); st != DSPARK_OK) return st;
    if (const dspark_status_t st = policy_args(policy, &a); st != DSPARK_OK) return st;
    a.saved = reinterpret_cast<RowSaved*>(const_cast<float*>(saved));
    a.up = grad_loss;
    return launch_grad(a, sx, policy->entropy_coef != 0.f, params);
}

dspark_status_t dspark_preference_loss(const void* logits, const dspark_preference_t* pref, const dspark_token_params_t* params,
                                       float* out_loss, float* out_rewards, int32_t* pair_status, float* out_logprobs,
                                       float* out_saved, void* out_grad) {
    TokArgs a{};
    int sx = 0;
    if (const dspark_status_t st = token_args(logits, params, out_grad, &a, &sx); st != DSPARK_OK) return st;
    if (!pref || !pref->row_offsets || pref->n_pairs < 1 || pref->n_pairs > DSPARK_MAX_PAIRS) return DSPARK_ERR_INVALID_ARG;
    if (!(pref->beta > 0.f) || !(pref->beta < INFINITY) || !std::isfinite(pref->margin)) return DSPARK_ERR_INVALID_ARG;
    if (!(pref->label_smoothing >= 0.f) || !(pref->label_smoothing < 1.f)) return DSPARK_ERR_INVALID_ARG;
    if (!out_loss || !pair_status || !out_saved || !params->row_status || misplaced(out_saved, 16)) return DSPARK_ERR_INVALID_ARG;
    a.op = kPreference;
    a.logp = out_logprobs;
    a.saved = reinterpret_cast<RowSaved*>(out_saved);
    if (const dspark_status_t st = launch_stats(a, sx, false, params); st != DSPARK_OK) return st;
    PairArgs b{params->n_rows, pref->n_pairs, pref->mean, pref->beta, pref->margin, pref->label_smoothing, pref->row_offsets,
               params->tokens, pref->ref_logprobs, pref->weights, params->row_status, out_loss, out_rewards,
               pair_status, a.saved};
    if (launch_cluster(pair_kernel, static_cast<unsigned>(pref->n_pairs), kRowThreads, 1, 0,
                       static_cast<cudaStream_t>(params->stream), b) != cudaSuccess)
        return DSPARK_ERR_CUDA;
    return out_grad ? launch_grad(a, sx, false, params) : DSPARK_OK;
}

dspark_status_t dspark_preference_loss_backward(const void* logits, const dspark_token_params_t* params, int32_t n_pairs,
                                                const float* saved, const float* grad_loss, void* out_grad) {
    TokArgs a{};
    int sx = 0;
    if (!out_grad || !saved || misplaced(saved, 16) || n_pairs < 1 || n_pairs > DSPARK_MAX_PAIRS) return DSPARK_ERR_INVALID_ARG;
    if (const dspark_status_t st = token_args(logits, params, out_grad, &a, &sx); st != DSPARK_OK) return st;
    a.op = kPreference;
    a.saved = reinterpret_cast<RowSaved*>(const_cast<float*>(saved));
    a.up = grad_loss;
    a.n_up = n_pairs;
    return launch_grad(a, sx, false, params);
}

}  // extern "C"
