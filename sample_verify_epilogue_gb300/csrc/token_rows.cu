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
// stats_kernel streams a row and leaves what the gradient needs (32 bytes a row), grad_kernel streams it again, kept_kernel
// does both with the row in shared memory, pair_kernel makes the pairs of a preference from their rows.  All but the last are
// bound by bandwidth where there is enough to read: of the copy bandwidth stats 0.91 to 0.98 (4096 rows of 151936 bf16 with the
// entropy 181 us, a tenth of them without a token), the gradient 0.93 to 1, both in one 0.98 (351 us; 0.93, 375 us, with an
// entropy bonus).  Where a CTA has little to read its latencies bound it: token, first vectors, joins, the row's end.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <limits>

#include "vocab_rows.cuh"

namespace dspark {

namespace {

constexpr int kTokVec = 2;                                   // vectors a thread takes at a time from shared memory
constexpr int kGradVec = 4;                                  // vectors a thread of the gradient has on their way
constexpr int kShortRow = 2048;                              // vectors of a row that 128 threads take, where rows are many
constexpr int kSlimRow = 1024;                               // those that 64 take
constexpr float kLn2 = 0.693147180559945f;
// what a sum of the exponential unit's results lacks on average, relative: added to its logarithm.  (2^20 arguments between whole
// exponents: 5.06e-8, from 9e-8 too large to 1.4e-7 too small; sums of 262144 normal logits over 0.7, 1 and 1.3, by a
// reference above them: 4.6e-8 to 5.1e-8.)
constexpr float kEx2Lacks = 5.06e-8f;

constexpr float kAbove = 5.f;

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
    float c, c_low, inv_c, inv_t;                            // log2(e) / T and what it lacks of it, 1 / c, 1 / T
    float above;                                             // kAbove / c, a distance of logits
    float c_head, c_tail;                                    // log2(e) / T in two positive parts, 16 bits and the rest
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
    int log_c, splits;                                       // log2 of the CTAs of a row (stats); CTAs of a row (gradient, fused)
    int span;                                                // vectors of each (fused)
    float most;                                              // a sum of vectors from which on the reference is raised
    unsigned zero;                                           // 0
};

// A sum of exponentials e by ExpRef(m), and the sum w of e times its exponent (base 2).  m is about the largest logits'
// size, kAbove powers of two above those it was taken from, so that few that come later are larger: exponents above -1 lose their
// last bits in the exponential unit (sums by the largest of a thousand logits lacked 5e-9 to 4e-8 of what is below, by one
// above all of them 5e-8).
struct EntSum {
    float m, sum, w;
};
// What a sum by `from` scales by to be by `to`, a power of two, and what its exponents gain: the difference of what was taken from
// the exponents, a whole number or (logits of 2.9 million T) m log2(e) / T itself, to its low part, with the constant's second part where
// the exponents have it.
__device__ __forceinline__ float shift_of(float from, float to, float c, float low) {
    const float t = from * c, u = to * c;
    const bool t_whole = fabsf(t) < 4194304.f, u_whole = fabsf(u) < 4194304.f;
    float by = (t_whole ? ceilf(t) : t) - (u_whole ? ceilf(u) : u);
    if (!t_whole) by += fmaf(from, low, fmaf(from, c, -t));
    if (!u_whole) by -= fmaf(to, low, fmaf(to, c, -u));
    return from == to ? 0.f : fmaxf(by, -16384.f);           // (NaN, of the types' lowest values: nothing is left)
}
template <bool ENT>
__device__ __forceinline__ void rebase_to(EntSum& a, float to, float c, float low) {
    if (a.m > -INFINITY) {
        const float by = shift_of(a.m, to, c, ENT ? 0.f : low), k = ex2_approx(by);
        if (ENT) a.w = fmaf(a.sum, by, a.w) * k;
        a.sum *= k;
    }
    a.m = to;
}
// The sum over groups of N lanes, in each of them.
template <bool ENT, int N>
__device__ __forceinline__ EntSum lanes_join(EntSum a, const TokArgs& args) {
    float m = a.m;
    if (N == 32) m = key_to_f(__reduce_max_sync(0xffffffffu, fkey(m)));
    else
#pragma unroll
        for (int o = N / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (m > -INFINITY) rebase_to<ENT>(a, m, args.c, args.c_low);
#pragma unroll
    for (int o = N / 2; o; o >>= 1) {
        a.sum += __shfl_xor_sync(0xffffffffu, a.sum, o);
        if (ENT) a.w += __shfl_xor_sync(0xffffffffu, a.w, o);
    }
    return a;
}

// A thread's sum while it streams.
//
// Vectors are added by the reference that is there, whatever their maximum: where that makes a sum of a.most or more
// (the first vectors, a maximum above the reference) they are added again by a reference above it.  The reference's whole exponent r
// makes the exponent's one rounding that of the fma; -inf stands for none.  (With the running
// maximum of every batch of vectors in the way: 191 us where this takes 181, 4096 rows of 151936 with the entropy.)
//
// A row's log-probability may be off by 1e-7 at random, but not to one side: sums of a thousand log ratios follow.  So
// the vectors' sum joins the rest in a pair of floats (added one by one, small terms are lost more often than gained:
// 2e-8 of a row of 151936), and log2(e) / T is not rounded to one float (which makes every log-probability off by up to
// 2^-24 of the distance between logits): it has a head of 16 bits, whose product with a bf16 is exact, and a tail whose product is
// large beside an exponent's last bit (of 24 bits and the rest the rest would be rounded away, the same way in every row); with
// the entropy, whose sum gives the mean logit, what the one float lacks is made up for in row_end.
template <int SX, bool ENT>
struct RunEnt {
    static constexpr int VE = 16 / SX;
    float m = -INFINITY, r = -INFINITY, sum = 0.f, low = 0.f, w = 0.f;
    uint32_t least = 0u;                                     // (bf16, entropy) logits below have e = 0: a pair of it

    __device__ __forceinline__ EntSum get() const { return EntSum{m, sum + low, w}; }

    __device__ __forceinline__ void rebase(float to, const ExpRef& ref, const TokArgs& a) {
        EntSum was = get();
        rebase_to<ENT>(was, to, a.c, a.c_low);
        m = to;
        r = ref.whole ? ref.r : -INFINITY;
        sum = was.sum;
        low = 0.f;
        w = was.w;
    }

    // Before the first vectors, by a whole warp: the largest of them all is a reference that hardly ever has to be raised
    // (a thread's own: 4096 policy rows of 151936 389 -> 435 us).
    template <int U>
    __device__ __forceinline__ void seed(const uint4 (&v)[U], const TokArgs& a) {
        const float to = key_to_f(__reduce_max_sync(0xffffffffu, fkey(vecs_max<SX>(v)))) + a.above;
        const ExpRef ref(to, a.c);
        if (!ref.whole) return;
        m = to;
        r = ref.r;
        if (ENT && SX == 2) least = least_pair(ref, a.inv_c);
    }

    // U vectors from shared memory, `stride` apart: read again where the reference has to be raised.
    template <int U>
    __device__ __forceinline__ void add_from(const uint4* p, int stride, const TokArgs& a) {
        float ws, s;
        {
            uint4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = p[u * stride];
            s = sum_of(v, a, ws);
        }
        if (!(s < a.most)) {
#pragma unroll 1
            for (int u = 0; u < U; ++u) {
                uint4 v[1] = {p[u * stride]};
                add(v, a);
            }
            return;
        }
        take(s, ws);
    }
    __device__ __forceinline__ void take(float s, float ws) {
        const TwoFloat t = two_sum(sum, s);
        sum = t.hi;
        low += t.lo;
        if (ENT) w += ws;
    }

    template <int U>
    __device__ __forceinline__ void add(uint4 (&v)[U], const TokArgs& a) {
        float ws, s = sum_of(v, a, ws);
        if (!(s < a.most)) {
            // (a zero that the compiler does not know: else it keeps the first sum's conversions for the second, in registers
            // that are not there)
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = make_uint4(v[u].x ^ a.zero, v[u].y ^ a.zero, v[u].z ^ a.zero, v[u].w ^ a.zero);
            const float to = fmaxf(m, vecs_max<SX>(v) + a.above);
            const ExpRef ref(to, a.c);
            if (!ref.whole) {
#pragma unroll 1
                for (int u = 0; u < U; ++u) {
                    uint4 one = v[0];
#pragma unroll
                    for (int k = 1; k < U; ++k)
                        if (k == u) one = v[k];
                    add_far(one, a);
                }
                return;
            }
            rebase(to, ref, a);
            if (ENT && SX == 2) least = least_pair(ref, a.inv_c);
            s = sum_of(v, a, ws);                            // (NaN stays)
        }
        take(s, ws);
    }

    template <int U>
    __device__ __forceinline__ float sum_of(const uint4 (&v)[U], const TokArgs& a, float& ws) const {
        const float c = ENT ? a.c : a.c_head;
        const unsigned long long c2 = pack2(c, c), l2 = pack2(a.c_tail, a.c_tail), r2 = pack2(-r, -r);
        unsigned long long acc[2] = {0ull, 0ull}, accw = 0ull;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < VE / 2; ++h) {
                unsigned long long x;
                float lo, hi;
                if (ENT && SX == 2) {                        // (0 times -inf)
                    const __nv_bfloat162 b = __hmax2_nan(reinterpret_cast<const __nv_bfloat162*>(&v[u])[h], *reinterpret_cast<const __nv_bfloat162*>(&least));
                    const uint32_t bits = *reinterpret_cast<const uint32_t*>(&b);
                    x = pack2(bf16_lo(bits), bf16_hi(bits));
                } else {
                    x = pair_of<SX>(v[u], h);
                }
                unsigned long long z = fma2(x, c2, r2);
                if (!ENT) z = fma2(x, l2, z);
                unpack2(z, lo, hi);
                const unsigned long long e = pack2(ex2_approx(lo), ex2_approx(hi));
                acc[h & 1] = add2(acc[h & 1], e);
                if (ENT) accw = fma2(e, SX == 2 ? z : pack2(fmaxf(lo, -16384.f), fmaxf(hi, -16384.f)), accw);
            }
        float lo, hi;
        if (ENT) {
            unpack2(accw, lo, hi);
            ws = lo + hi;
        }
        unpack2(add2(acc[0], acc[1]), lo, hi);
        return lo + hi;
    }

    // Vectors of infinities, of the type's lowest values.
    __device__ __forceinline__ void add_far(const uint4& v, const TokArgs& a) {
        const float to = fmaxf(m, vec_max<SX>(v));
        if (!(to > -INFINITY)) {                             // nothing yet; a NaN among it counts
            float t = 0.f;
#pragma unroll
            for (int q = 0; q < VE; ++q) t += elem<SX>(v, q);
            if (t != t) sum = t;
            return;
        }
        const ExpRef ref(to, a.c);
        rebase(to, ref, a);
#pragma unroll
        for (int q = 0; q < VE; ++q) {
            const float x = elem<SX>(v, q), z = !ref.whole ? (x - ref.m) * a.c : ENT ? fmaf(x, a.c, -ref.r) : fmaf(x, a.c_tail, fmaf(x, a.c_head, -ref.r));
            const float e = ex2_approx(z);
            sum += e;
            if (ENT) w = fmaf(e, fmaxf(z, -16384.f), w);
        }
        if (ENT && SX == 2 && ref.whole) least = least_pair(ref, a.inv_c);
    }

    // a logit whose exponential by the reference is 0, not below the type's lowest value (rounded down: of logits of a million
    // the next one above may be the largest)
    static __device__ __forceinline__ uint32_t least_pair(const ExpRef& ref, float inv_c) {
        const uint32_t x = __bfloat16_as_ushort(__float2bfloat16_rd(fmaxf((ref.r - 4096.f) * inv_c, -3.38e38f)));
        return x | x << 16;
    }
};

// log(v), v > 0 normal, to some 2^-31: the exponent's part, and 2 atanh((m - 1) / (m + 1)) of what is left in [0.75, 1.5).
// (logf's error there, 2^-25, would be the same for every row whose sum is about as large: a sequence's sum has it
// hundreds of times.)
__device__ __forceinline__ TwoFloat log_fine(float v) {
    const int e = (__float_as_int(v) - 0x3F400000) >> 23;
    const float m = __int_as_float(__float_as_int(v) - (e << 23)), num = m - 1.f;
    const TwoFloat den = two_sum(m, 1.f);
    const float f = num / den.hi, low = (fmaf(-f, den.hi, num) - f * den.lo) / den.hi, s = f * f;
    float p = fmaf(s, 1.f / 13.f, 1.f / 11.f);
    p = fmaf(s, p, 1.f / 9.f);
    p = fmaf(s, p, 1.f / 7.f);
    p = fmaf(s, p, 1.f / 5.f);
    p = fmaf(s, p, 1.f / 3.f);
    const TwoFloat l = TwoFloat{static_cast<float>(e), 0.f} * ln2_two() + TwoFloat{2.f * f, 2.f * fmaf(f * s, p, low)};
    return two_sum(l.hi, l.lo);
}

// Replace logit `lane` of a vector.
template <int SX>
__device__ __forceinline__ void patch(uint4& v, int lane, uint32_t bits) {
#pragma unroll
    for (int q = 0; q < 16 / SX; ++q)
        if (q == lane) put_bits<SX>(v, q, bits);
}

// e^D - D - 1 without the difference of near ones: its series where D is small (relative remainder below 2^-24);
// em1 is expm1f(D)
__device__ __forceinline__ float k3_of(float D, float em1) {
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
    return D > 64.f ? em1 : em1 - D;                         // (an infinite D has an infinite e^D)
}

struct PolicyRow {
    float w, old, ref, adv;
};

// The smaller gain of rho A and the clipped rho times A: clipping binds above for A > 0, below for A < 0.  A ratio at
// the border, or past it by what two fp32 log-probabilities' rounding makes of it, keeps its gradient (2^-24 |log p| for each of them and
// 2e-7 of the sums: with clip 0 half of a rollout's rows would have none on the policy that drew them).
struct Clipped {
    float ratio, edge;                                       // clipped; from where clipping binds
    bool binds;
    __device__ __forceinline__ Clipped(const TokArgs& a, float rho, float logp, float adv) {
        const float border = adv > 0.f ? a.high : a.low, slack = fmaf(fabsf(logp), 0x1p-22f, 0x1p-20f);
        edge = fmaf(border, adv > 0.f ? slack : -slack, border);
        binds = adv > 0.f ? rho > edge : rho < edge;
        ratio = (adv > 0.f ? rho > border : rho < border) ? border : rho;
    }
};

// A row's results, of which `saved` goes to its gradient.
struct RowEnd {
    RowSaved saved;
    float logp, entropy, loss, kl;
    int status;
};

// What log R - s_y is made of: log(1 + e^d) and log(1 + e^-d), 1 / (1 + e^-d) and 1 / (1 + e^d).
struct Odds {
    TwoFloat sp;
    float sm, q, p;
    __device__ __forceinline__ explicit Odds(const TwoFloat& d) {
        // (d.lo is up to 2^-24 d: of a sure token's q 16 u)
        const bool up = d.hi > 0.f;
        const float t = expf(-fabsf(d.hi)), l = log1pf(t), by = fabsf(d.hi) < INFINITY ? fmaf(t, up ? -d.lo : d.lo, t) : t;
        const float inv = 1.f / (1.f + by), small = by * inv;
        q = up ? inv : small;
        p = up ? small : inv;
        sm = up ? l : l - d.hi;
        sp = up ? two_sum(d.hi, l) : TwoFloat{l, 0.f};
        if (d.hi < INFINITY) sp.lo += d.lo * q;              // (the sum with an infinity has no error term)
        else sp.lo = 0.f;
    }
};

// What the gradient's exponentials, relative to those of the sum, have to be multiplied with for c_low (as much as 2% for
// logits of a million T): fp32's gradient has all of log2(e) / T in its exponents, bf16's does not; a sum with the entropy does not.
// by_low is what it adds to the sum's logarithm; without the entropy the largest logit stands for all that count.  (H, a
// difference of two that have it or have it not, is the same.)
template <int SX, bool ENT>
__device__ __forceinline__ float by_low_of(const TokArgs& a, float m, float by_low) {
    if (ENT) return SX == 4 ? ex2_approx(-kLog2E * by_low) : 1.f;
    return SX == 4 ? 1.f : fabsf(m * a.c) < 4194304.f ? ex2_approx(m * a.c_low) : 1.f;
}

// From a row's sum over the other tokens and its token's logit, by one thread.
template <int SX, bool ENT>
__device__ __forceinline__ RowEnd row_end(const TokArgs& a, const EntSum& es, float xy, const PolicyRow& pr) {
    RowEnd o{RowSaved{0.f, -1.f, 0.f, 0.f, 0.f, 0.f, 0.f, -1}, NAN, NAN, NAN, NAN, DSPARK_ROW_NONFINITE};
    const bool none = !(es.m > -INFINITY) && es.sum == es.sum;   // no other token has any mass
    if (!(xy < INFINITY) || es.sum != es.sum || !(es.m < INFINITY) || (none && !(xy > -INFINITY))) return o;
    o.status = 0;
    RowSaved& s = o.saved;
    TwoFloat d{-INFINITY, 0.f}, lr{0.f, 0.f};
    float mean = 0.f, by_low = 0.f;                          // of the others' exponents; what c_low adds to log R
    if (!none) {
        const ExpRef ref(es.m, a.c);
        lr = log_fine(es.sum);
        lr.lo += kEx2Lacks;
        if (ENT) {
            mean = es.w / es.sum;
            if (ref.whole) by_low = a.c_low * a.inv_c * kLn2 * (mean + ref.r);
        }
        if (!(xy > -INFINITY)) {
            d.hi = INFINITY;
        } else if (ref.whole) {
            const TwoFloat p = two_prod(xy, a.c), by = two_sum(ref.r, -p.hi);
            d = fabsf(p.hi) < INFINITY ? TwoFloat{by.hi, by.lo - fmaf(xy, a.c_low, p.lo)} * ln2_two() + TwoFloat{lr.hi, lr.lo + by_low}
                                       : TwoFloat{fmaf(-xy, a.inv_t, ref.r * kLn2), 0.f};   // the types' lowest values
        } else {
            const float by = (es.m - xy) * a.inv_t;
            d = fabsf(by) < INFINITY ? TwoFloat{by, 0.f} + lr : TwoFloat{by, 0.f};
        }
        if (fabsf(d.hi) < INFINITY) d = two_sum(d.hi, d.lo);   // (what c_low adds is not small beside logits of thousands)
        s.m = es.m;
    }
    const Odds k(d);
    const TwoFloat lp = -k.sp;
    float H = 0.f;
    if (ENT) H = (k.p > 0.f ? k.p * k.sp.hi : 0.f) + (none || k.q == 0.f ? 0.f : k.q * (k.sm + fmaf(-kLn2, mean, lr.hi + lr.lo)));
    s.f = none ? 0.f : k.q / es.sum * a.inv_t * by_low_of<SX, ENT>(a, es.m, by_low);
    s.level = none || !(k.sm < INFINITY) ? 0.f : H - (SX == 4 ? lr.hi + by_low : lr.hi) - k.sm;
    s.q = k.q * a.inv_t;
    s.py = k.p > 0.f ? k.p * (lp.hi + H) * a.inv_t : 0.f;
    o.logp = lp.hi + lp.lo;
    o.entropy = H;
    if (a.op == kPolicy) {
        const float rho = expf((lp.hi - pr.old) + lp.lo);
        float gain = 0.f, by_lp = 0.f;
        if (pr.adv != 0.f) {
            const Clipped k(a, rho, lp.hi, pr.adv);
            gain = k.ratio * pr.adv;
            by_lp = k.binds ? 0.f : -rho * pr.adv;
        }
        float loss = -gain;
        o.kl = 0.f;
        if (a.ref_lp) {
            const float D = (pr.ref - lp.hi) - lp.lo, em1 = expm1f(D);
            o.kl = k3_of(D, em1);
            if (a.kl_coef != 0.f) {
                loss = fmaf(a.kl_coef, o.kl, loss);
                by_lp = fmaf(-a.kl_coef, em1, by_lp);
            }
        }
        if (a.ent_coef != 0.f) loss = fmaf(-a.ent_coef, H, loss);
        o.loss = loss * pr.w;
        s.a = pr.w * by_lp;
        s.h = -pr.w * a.ent_coef;
        if (!(fabsf(o.loss) < INFINITY) || !(fabsf(s.a) < INFINITY) || !(fabsf(s.h) < INFINITY)) {
            o = RowEnd{s, NAN, NAN, NAN, NAN, DSPARK_ROW_NONFINITE};
            o.saved.f = -1.f;
        }
    } else if (a.op == kScore) {
        s.a = 1.f;
        s.h = ENT ? 1.f : NAN;                               // an entropy's gradient needs a call that asked for the entropy
    } else {
        s.level = lp.hi;                                     // a sequence's log ratios cancel: the sum takes both parts
        s.py = lp.lo;
    }
    return o;
}
__device__ __forceinline__ void row_write(const TokArgs& a, long long row, const RowEnd& o, bool entropy) {
    if (a.logp) a.logp[row] = o.logp;
    if (entropy && a.entropy) a.entropy[row] = o.entropy;
    if (a.loss) a.loss[row] = o.loss;
    if (a.kl) a.kl[row] = o.kl;
    if (a.saved) a.saved[row] = o.saved;
    a.row_status[row] = o.status;
}

// A row that is not read: without a token, of weight 0, or (status) with a token out of range.
__device__ __forceinline__ void row_skipped(const TokArgs& a, long long row, int status) {
    const float v = status ? NAN : 0.f;
    row_write(a, row, RowEnd{RowSaved{0.f, -1.f, 0.f, 0.f, 0.f, 0.f, 0.f, -1}, v, v, v, v, status}, true);
}

// The place of logit i of a row among its vectors.
template <int SX>
struct Place {
    int k, lane;
    __device__ __forceinline__ Place(const VocabRow<SX>& x, int i) : k((i + x.a0) / VocabRow<SX>::VE), lane((i + x.a0) % VocabRow<SX>::VE) {}
};

__device__ __forceinline__ RowEnd row_bad(int status) {
    return RowEnd{RowSaved{0.f, -1.f, 0.f, 0.f, 0.f, 0.f, 0.f, -1}, NAN, NAN, NAN, NAN, status};
}

// Sums between the CTAs of a row: each pushes its own to those that want it, where an mbarrier counts the bytes.
struct __align__(16) PeerSum {
    EntSum es;
    uint32_t after;
};
__device__ __forceinline__ void expect_peers(uint64_t* bar, int n) {
    if (threadIdx.x == 0) {
        mbar_init(bar, 1);
        fence_mbar_init();
        mbar_arrive_expect_tx(bar, sizeof(PeerSum) * n);
    }
    cluster_arrive_relaxed();                                // before a peer can push here (the fence above orders it)
}
// after: something whose load has to be done before a peer may write
__device__ __forceinline__ void push_sum(PeerSum* slot, uint64_t* bar, int to, const EntSum& es, uint32_t after) {
    peer_push128(peer_addr(slot, to), peer_addr(bar, to), __float_as_uint(es.m), __float_as_uint(es.sum), __float_as_uint(es.w),
                 after);
}
template <bool ENT>
__device__ __forceinline__ EntSum peers_join(const PeerSum* s, int C, const TokArgs& args) {
    const int k = threadIdx.x & (kMaxCluster - 1);
    return lanes_join<ENT, kMaxCluster>(k < C ? s[k].es : EntSum{-INFINITY, 0.f, 0.f}, args);
}

template <int SX, bool ENT, int NT, int U>
__global__ void __launch_bounds__(NT, U == 4 ? 1536 / NT : 1024 / NT) stats_kernel(TokArgs a) {
    __shared__ EntSum s_warp[(NT / 32)];
    __shared__ PeerSum s_peer[kMaxCluster];                  // (in the row's first CTA) written by the cluster's
    __shared__ uint64_t s_bar;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = 1 << a.log_c, rank = blockIdx.x & (C - 1);
    const long long row = blockIdx.x >> a.log_c;
    if (C > 1) expect_peers(&s_bar, C - 1);
    pdl_wait();
    if (a.op == kPreference) pdl_trigger();                  // the pairs' few CTAs may come while the last rows are read
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
    float xy = 0.f;
    if (rank == 0 && tid == 0) {
        xy = load_logit<SX>(x, y);
        if (a.op == kPolicy) {
            pr.old = a.old_lp[row];
            pr.adv = a.adv[row];
            if (a.ref_lp) pr.ref = a.ref_lp[row];
        }
    }
    // whole vectors [w0, w1) go straight through; the token's is its owner's business
    const int w0 = k0 + (k0 < k1 && !x.whole(k0)), w1 = k1 - (k1 > w0 && !x.whole(k1 - 1));
    const Place<SX> at(x, y);
    const int own = (at.k - w0) % NT == tid ? at.k : -1;
    RunEnt<SX, ENT> run;
    int k = w0 + tid;
    const uint4* p = reinterpret_cast<const uint4*>(x.p + static_cast<long long>(x.first(k)) * SX);
    for (; k + (U - 1) * NT < w1; k += U * NT, p += U * NT) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = ld_vec16(p + u * NT);
        if (own >= k && own < k + U * NT) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (k + u * NT == own) patch<SX>(v[u], at.lane, ninf_bits<SX>());
        }
        if (k == w0 + tid && w0 + (tid | 31) + (U - 1) * NT < w1) run.seed(v, a);
        run.add(v, a);
    }
    if (k < w1) {                                            // what is left, on its way together too (1 to 8% of rows of 5000 to 32000)
        uint4 v[U - 1][1];
#pragma unroll
        for (int u = 0; u < U - 1; ++u)
            if (k + u * NT < w1) v[u][0] = ld_vec16(p + u * NT);
#pragma unroll
        for (int u = 0; u < U - 1; ++u)
            if (k + u * NT < w1) {
                if (k + u * NT == own) patch<SX>(v[u][0], at.lane, ninf_bits<SX>());
                run.add(v[u], a);
            }
    }
    if (tid < 2) {                                           // the ragged ends
        const int e = tid ? w1 : k0;
        if (tid ? w1 < k1 : k0 < w0) {
            uint4 v[1] = {load_vec<SX>(x, e, k1)};
            if (e == at.k) patch<SX>(v[0], at.lane, ninf_bits<SX>());
            run.add(v, a);
        }
    }
    EntSum es = lanes_join<ENT, 32>(run.get(), a);
    if (lane == 0) s_warp[warp] = es;
    __syncthreads();
    if (C > 1) cluster_wait();
    if (warp != 0) return;
    es = lanes_join<ENT, (NT / 32)>(s_warp[lane & ((NT / 32) - 1)], a);
    bool late = false;
    if (C > 1) {
        if (rank != 0) {                                     // to the row's first CTA, which is there and waits
            if (lane == 0) push_sum(&s_peer[rank], &s_bar, 0, es, 0u);
            return;
        }
        if (lane == 0) s_peer[0].es = es;
        __syncwarp();
        late = !bar_wait(&s_bar, 0, kPeerMs);
        es = peers_join<ENT>(s_peer, C, a);
    }
    if (lane == 0) row_write(a, row, late ? row_bad(DSPARK_ROW_INTERNAL) : row_end<SX, ENT>(a, es, xy, pr), ENT);
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
template <int SX>
__device__ __forceinline__ void store_one(const VocabRow<SX>& g, int i, float v) {
    unsigned char* p = const_cast<unsigned char*>(g.p);
    if (SX == 2) reinterpret_cast<unsigned short*>(p)[i] = static_cast<unsigned short>(to_bits<SX>(v));
    else reinterpret_cast<float*>(p)[i] = v;
}

// What a row's gradient is made with: e_v (a0 + a1 z_v) for exponentials e_v = 2^z_v, and the token's own.
template <int SX, bool ENT>
struct RowGrad {
    static constexpr int VE = 16 / SX;
    ExpRef ref;
    float head, tail, a0, a1, at_y;                          // of log2(e) / T
    uint32_t least;

    __device__ __forceinline__ RowGrad(const TokArgs& a, const RowSaved& s, float da, float dh)
        : ref(s.m, a.c), head(SX == 4 ? a.c_head : a.c), tail(a.c_tail), a0(-s.f * fmaf(dh, s.level, da)), a1(-s.f * dh * kLn2), at_y(da * s.q - dh * s.py) {
        if (!ENT) {
            a0 = -s.f * da;
            at_y = da * s.q;
        }
        least = ENT && SX == 2 ? RunEnt<SX, ENT>::least_pair(ref, a.inv_c) : 0u;
    }
    __device__ __forceinline__ static uint4 pack(const float (&f)[VE]) {
        if (SX == 2) return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4 % VE], f[5 % VE]), pack_bf16(f[6 % VE], f[7 % VE]));
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
    // by a reference with a whole exponent
    __device__ __forceinline__ uint4 of(const uint4& v) const {
        float f[VE];
        const unsigned long long c2 = pack2(head, head), l2 = pack2(tail, tail), r2 = pack2(-ref.r, -ref.r);
#pragma unroll
        for (int h = 0; h < VE / 2; ++h) {
            unsigned long long x;
            if (ENT && SX == 2) {
                const __nv_bfloat162 b = __hmax2(reinterpret_cast<const __nv_bfloat162*>(&v)[h], *reinterpret_cast<const __nv_bfloat162*>(&least));
                const uint32_t bits = *reinterpret_cast<const uint32_t*>(&b);
                x = pack2(bf16_lo(bits), bf16_hi(bits));
            } else {
                x = pair_of<SX>(v, h);
            }
            unsigned long long z = fma2(x, c2, r2);
            if (SX == 4) z = fma2(x, l2, z);                 // (bf16 holds nothing that the second part would change)
            float lo, hi;
            unpack2(z, lo, hi);
            unsigned long long k = pack2(a0, a0);
            if (ENT) k = fma2(SX == 2 ? z : pack2(fmaxf(lo, -16384.f), fmaxf(hi, -16384.f)), pack2(a1, a1), k);
            unpack2(mul2(pack2(ex2_approx(lo), ex2_approx(hi)), k), f[2 * h], f[2 * h + 1]);
        }
        return pack(f);
    }
    // by the types' lowest values
    __device__ __forceinline__ uint4 far_of(const uint4& v) const {
        float f[VE];
#pragma unroll
        for (int q = 0; q < VE; ++q) {
            const float z = (elem<SX>(v, q) - ref.m) * ref.c;
            f[q] = ex2_approx(z) * (ENT ? fmaf(fmaxf(z, -16384.f), a1, a0) : a0);
        }
        return pack(f);
    }
};

// The gradient of vectors [k0, k1) of a row (or zeros), by the CTA's threads in turn; src is where vector k0 lies, in global
// or shared memory (kept: whole there, ragged ones too); the token's entry by the thread that has its vector.
template <int SX, bool ENT, bool KEPT, int U, int NT>
__device__ __forceinline__ void write_grad(const VocabRow<SX>& x, const VocabRow<SX>& g, int k0, int k1, int y, bool zero,
                                           const RowGrad<SX, ENT>& rg, const uint4* src) {
    const int tid = threadIdx.x;
    const bool same_phase = x.a0 == g.a0;
    int k = k0 + tid;
    if (zero) {
        for (; k < k1; k += NT) store_vec<SX>(g, x.first(k), make_uint4(0, 0, 0, 0), same_phase);
        return;
    }
    auto get = [&](int k) { return KEPT ? src[k - k0] : load_vec<SX>(x, k, k1); };
    if (same_phase && rg.ref.whole) {
        // whole vectors go straight through, by the threads that have them
        const int w0 = k0 + (k0 < k1 && !x.whole(k0)), w1 = k1 - (k1 > w0 && !x.whole(k1 - 1));
        if (k < w0) k += NT;
        unsigned char* p = const_cast<unsigned char*>(g.p) + static_cast<long long>(x.first(k)) * SX;
        const uint4* q = src + (k - k0);
        const uint4* const end = src + (w1 - k0);
        if (U == 1 || SX == 4)
            for (; q + (U - 1) * NT < end; q += U * NT, p += 16 * U * NT) {
                uint4 v[U];
#pragma unroll
                for (int u = 0; u < U; ++u) v[u] = KEPT ? q[u * NT] : ld_vec16(q + u * NT);
#pragma unroll
                for (int u = 0; u < U; ++u) st_vec16(p + 16 * u * NT, rg.of(v[u]));
            }
        // the last ones on their way together too (one by one: 16000 rows of 5000 bf16 83 us, 60 so); of bf16, whose registers are
        // short, all of them here
        if (U > 1)
            for (; q < end; q += U * NT, p += 16 * U * NT) {
                uint4 v[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (q + u * NT < end) v[u] = KEPT ? q[u * NT] : ld_vec16(q + u * NT);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (q + u * NT < end) st_vec16(p + 16 * u * NT, rg.of(v[u]));
            }
        if (tid == 0 && k0 < w0) store_vec<SX>(g, x.first(k0), rg.of(get(k0)), false);
        if (w1 < k1 && (k1 - 1 - k0) % NT == tid) store_vec<SX>(g, x.first(k1 - 1), rg.of(get(k1 - 1)), false);
    } else {
        for (; k < k1; k += NT) {
            const uint4 v = get(k);
            store_vec<SX>(g, x.first(k), rg.ref.whole ? rg.of(v) : rg.far_of(v), same_phase);
        }
    }
    const Place<SX> at(x, y);
    // (a token that changed after the call that saved the row may be out of range)
    if (y >= 0 && y < x.V && at.k >= k0 && at.k < k1 && (at.k - k0) % NT == tid) store_one<SX>(g, y, rg.at_y);
}

// The gradient alone, VECS vectors of a row to a CTA.  Rows whose gradient is 0 are not read.  Threads to an SM, where they are
// set (without the entropy): of fp32 1536 (unset: 800 rows of 12000 14.9 us for 14.0), by 64 1280 (1536: 16000 of 5000 97 for 94),
// of bf16 1152 (unset: 2629 rows of 34007 56.5 for 55.0); with the entropy 1152 and 1024 take 1 and 4% more than the compiler's choice.
template <int SX, bool ENT, int NT, int VECS>
__global__ void __launch_bounds__(NT, (ENT ? 0 : SX == 2 ? 1152 : NT == 64 ? 1280 : 1536) / NT) grad_kernel(TokArgs a) {
    const long long row = blockIdx.x / a.splits;
    const int part = blockIdx.x % a.splits;
    pdl_wait();
    const VocabRow<SX> x(a.x, row, a.x_stride, a.V), g(a.g, row, a.g_stride, a.V);
    const int k0 = part * VECS, k1 = min(x.nvec, k0 + VECS);
    RowSaved s = a.saved[row];
    const int y = a.tokens[row];
    if (a.op == kPreference) s.level = s.py = 0.f;
    float da = s.a, dh = s.h;
    if (a.op == kScore) {
        da = a.up ? a.up[row] : 0.f;
        dh = ENT && a.up_entropy ? s.h * a.up_entropy[row] : 0.f;
    } else if (a.op == kPolicy) {
        const float u = a.up ? a.up[row] : 1.f;
        da *= u;
        dh *= u;
    } else if (a.up) {
        da = s.pair >= 0 && s.pair < a.n_up ? da * a.up[s.pair] : 0.f;
    }
    const RowGrad<SX, ENT> rg(a, s, da, dh);
    write_grad<SX, ENT, false, kGradVec, NT>(x, g, k0, k1, y, s.f < 0.f || (da == 0.f && dh == 0.f), rg,
                                                      reinterpret_cast<const uint4*>(x.p + static_cast<long long>(x.first(k0)) * SX));
}

// ---------------------------------------------------------------- loss and gradient in one
// What a policy row's gradient is made with, on the way between its sum and its gradient, where the whole CTA waits: base 2
// and the hardware's functions, a third of row_end's steps (its chain of dependent instructions, run by one warp
// among forty, took 42 of 434 us of 4096 rows of 151936).  Logarithms are split from their exponents, what cancels has two parts.
// For fp32 logarithms and e^D - 1 by series, corrected reciprocals: the gradient at the token is off by 9e-8 relative (5e-7 at most), as by
// row_end (1000 rows, V of 2 to 32003), for 0.4 to 1% of the time.  For bf16 the units' own: 1.7e-7 (7e-7, and 2e-6 of a KL
// term's e^D - 1), where the result's rounding is 2e-3.
struct QuickRow {
    TwoFloat old2, ref2;                                     // log-probabilities by log2(e)
    float w, adv;
};
__device__ __forceinline__ TwoFloat base2(float v) {
    const TwoFloat p = two_prod(v, kLog2E);
    return TwoFloat{p.hi, fabsf(p.hi) < INFINITY ? fmaf(v, 1.9259629e-8f, p.lo) : 0.f};
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2_approx(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 1 / x and 2^x without what the units lack: a step of Newton's; the exponential's mean error
__device__ __forceinline__ float rcp_fine(float x) {
    const float r = rcp_approx(x);
    return fmaf(r, fmaf(-x, r, 1.f), r);
}
__device__ __forceinline__ float ex2_fine(float x, float more = 0.f) {   // times 1 + more
    const float e = ex2_approx(x);
    return fmaf(e, more + kEx2Lacks, e);
}
// log2((den + num) / (den - num)) = 2 / ln 2 atanh(num / den), by K terms of atanh's series
template <int K>
__device__ __forceinline__ float lg2_ratio(float num, float den) {
    const float r = rcp_approx(den), g = num * r, f = fmaf(r, fmaf(-g, den, num), g), s = f * f, c = 2.f * kLog2E * f;
    float p = 1.f / (2 * K - 1);
#pragma unroll
    for (int k = K - 1; k > 1; --k) p = fmaf(s, p, 1.f / (2 * k - 1));
    return fmaf(c * s, p, c);
}
// log2 of m in [0.75, 1.5) and of 1 + t, t up to 1, the series' remainders 1e-8 relative; for bf16 2^-22 absolute (4096 rows of
// 32000 81.7 us, by the series 82.9)
template <int SX>
__device__ __forceinline__ float lg2_near1(float m) {
    return SX == 4 ? lg2_ratio<5>(m - 1.f, m + 1.f) : lg2_approx(m);
}
template <int SX>
__device__ __forceinline__ float lg2_1p(float t) {
    if (SX == 4) return lg2_ratio<7>(t, 2.f + t);
    return t < 0.03125f ? t * kLog2E * fmaf(t, fmaf(t, fmaf(t, -0.25f, 1.f / 3.f), -0.5f), 1.f) : lg2_approx(1.f + t);
}
// Whether quick_end takes the row: the others have a whole exponent and a sum, the token a logit among them.  What is a matter of
// the last bits it leaves to row_end (sure = false), whose loss and status the row reports: a ratio within 2^-19 of where
// clipping binds (its own is off by 6e-7 at most, row_end's by 3e-7), and what may leave fp32's range.
constexpr float kSureRange = 0x1p120f;
__device__ __forceinline__ bool is_quick(const EntSum& es, float xy, float c) {
    return fabsf(es.m * c) < 4194304.f && es.sum > 0x1p-60f && es.sum < 0x1p60f && fabsf(xy * c) < 4194304.f;
}
template <int SX, bool ENT>
__device__ __forceinline__ RowSaved quick_end(const TokArgs& a, const EntSum& es, float xy, const QuickRow& pr, bool& sure) {
    RowSaved s{es.m, -1.f, 0.f, 0.f, 0.f, 0.f, 0.f, -1};
    const float r = ceilf(es.m * a.c), by_sum = rcp_fine(es.sum), mean = ENT ? es.w * by_sum : 0.f;
    const int e = (__float_as_int(es.sum) - 0x3F400000) >> 23;
    const float l = lg2_near1<SX>(__int_as_float(__float_as_int(es.sum) - (e << 23))) + kEx2Lacks * kLog2E;
    const float by_low = ENT ? a.c_low * a.inv_c * (mean + r) : 0.f;
    const TwoFloat p = two_prod(xy, a.c), top = two_sum(r + static_cast<float>(e), -p.hi);
    const float rest = top.lo + (l + by_low - fmaf(xy, a.c_low, p.lo)), d = top.hi + rest;   // log2 of R / e^s_y
    const bool up = d > 0.f;
    const float d_low = kLn2 * ((top.hi - d) + rest);
    const float t = ex2_fine(-fabsf(d), up ? -d_low : d_low), inv = rcp_fine(1.f + t), small = t * inv;
    const float q = up ? inv : small, py = up ? small : inv;
    const float lu = lg2_1p<SX>(t);
    const TwoFloat lp{up ? -top.hi : 0.f, up ? -(rest + lu) : -lu};   // log2 of p
    float H = 0.f;
    if (ENT) {
        const float sm = kLn2 * (up ? lu : lu - d), lr = kLn2 * (static_cast<float>(e) + l);
        H = fmaf(q, sm + fmaf(-kLn2, mean, lr), -py * kLn2 * (lp.hi + lp.lo));
        s.level = H - (SX == 4 ? fmaf(kLn2, by_low, lr) : lr) - sm;
        s.py = py * fmaf(kLn2, lp.hi + lp.lo, H) * a.inv_t;
    }
    s.q = q * a.inv_t;
    const float rho = ex2_fine((lp.hi - pr.old2.hi) + (lp.lo - pr.old2.lo));
    float gain = 0.f, by_lp = 0.f;
    if (pr.adv != 0.f) {
        const Clipped k(a, rho, kLn2 * (lp.hi + lp.lo), pr.adv);
        gain = k.ratio * pr.adv;
        by_lp = k.binds ? 0.f : -rho * pr.adv;
        sure = fabsf(gain) < kSureRange && !(fabsf(rho - k.edge) <= 0x1p-19f * k.edge);
    }
    float loss = -gain;
    if (a.kl_coef != 0.f) {
        const float D2 = (pr.ref2.hi - lp.hi) + (pr.ref2.lo - lp.lo), D = kLn2 * D2;
        const float em1 = SX == 4 ? expm1f(D)
                          : fabsf(D) < 0.0625f ? D * fmaf(D, fmaf(D, fmaf(D, fmaf(D, 1.f / 120.f, 1.f / 24.f), 1.f / 6.f), 0.5f), 1.f) : ex2_approx(D2) - 1.f;
        loss = fmaf(a.kl_coef, em1 - D, loss);
        by_lp = fmaf(-a.kl_coef, em1, by_lp);
    }
    if (ENT) loss = fmaf(-a.ent_coef, H, loss);
    s.a = pr.w * by_lp;
    s.h = -pr.w * a.ent_coef;
    sure = sure && fabsf(loss * pr.w) < kSureRange && fabsf(s.a) < kSureRange && fabsf(s.h) < kSureRange;
    s.f = q * by_sum * a.inv_t * by_low_of<SX, ENT>(a, es.m, kLn2 * by_low);
    return s;
}

// A policy row's loss and gradient without reading it twice: a cluster of C CTAs keeps the row in shared memory, a span
// each, between the sum and the gradient.  A span comes by one bulk copy (copies of 16 bytes by the threads that read them:
// 8% slower, 4096 rows of 151936; the row read twice: half as long again); a thread reads the same vectors for both, so
// that only the joins of the sums wait for others.  An SM moves as many bytes as it holds over how long it holds them: some
// 200 KB for 9.5 us at the copy bandwidth, so what stands between copy and gradient is kept short.
constexpr int kFusedSpan = 14000;                            // vectors of a span at most: 224,000 bytes
constexpr int kFusedCtas = 5;                                // CTAs of 256 threads to an SM at most

#ifdef DSPARK_TEST_EXPIRED_PEERS
constexpr unsigned kExpirePeerMs = 50;                       // test build: a second wait of the row's second CTA, for what nobody sends
#else
constexpr unsigned kExpirePeerMs = 0;
#endif

template <int SX, bool ENT, int NT>
__global__ void __launch_bounds__(NT, kFusedCtas * 256 / NT) kept_kernel(TokArgs a) {
    __shared__ EntSum s_warp[(NT / 32)];
    __shared__ PeerSum s_peer[kMaxCluster];                  // written by the row's CTAs
    __shared__ RowSaved s_row;
    __shared__ uint64_t s_bar, s_copy;
    extern __shared__ uint4 s_x[];                           // [span]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = a.splits, rank = static_cast<int>(cluster_rank());
    const long long row = cluster_id();
    if (tid == 0) {
        mbar_init(&s_copy, 1);
        fence_mbar_init();
    }
    if (C > 1) expect_peers(&s_bar, C);
    __syncthreads();
    pdl_wait();
    const int y = a.tokens[row];
    PolicyRow pr{1.f, 0.f, 0.f, 0.f};
    if (a.weights) pr.w = a.weights[row];
    const bool bad = y < -1 || y >= a.V, dead = bad || y < 0 || pr.w == 0.f;   // the same in every CTA of the row
    const VocabRow<SX> x(a.x, row, a.x_stride, a.V), g(a.g, row, a.g_stride, a.V);
    const int k0 = min(x.nvec, rank * a.span), cnt = min(x.nvec, k0 + a.span) - k0;
    if (dead) {
        if (rank == 0 && tid == 0) row_skipped(a, row, bad ? DSPARK_ROW_BAD_TOKEN : 0);
        for (int k = tid; k < cnt; k += NT) store_vec<SX>(g, x.first(k0 + k), make_uint4(0, 0, 0, 0), x.a0 == g.a0);
        if (C > 1) cluster_wait();
        return;
    }
    if (warp == 0) fetch_piece<SX>(x, k0, k0 + cnt, s_x, &s_copy);
    float xy = 0.f;
    if (warp == 0) {
        xy = load_logit<SX>(x, y);
        pr.old = a.old_lp[row];
        pr.adv = a.adv[row];
        if (a.ref_lp) pr.ref = a.ref_lp[row];
    }
    const Place<SX> at(x, y);
    RunEnt<SX, ENT> run;
    bool late = !copy_wait(&s_copy, 0);
    if (late) bar_wait(&s_copy, 0);                          // once more: it is in flight
    // the token leaves the sum (and the gradient's loop) here
    if (at.k >= k0 && at.k < k0 + cnt && (at.k - k0) % NT == tid) patch<SX>(s_x[at.k - k0], at.lane, ninf_bits<SX>());
    const uint4* const end = s_x + cnt;
    const uint4* q = s_x + tid;
    if ((tid | 31) < cnt) {
        const uint4 v[1] = {*q};
        run.seed(v, a);
    }
    for (; q + (kTokVec - 1) * NT < end; q += kTokVec * NT) run.template add_from<kTokVec>(q, NT, a);
    for (; q < end; q += NT) run.template add_from<1>(q, NT, a);
    EntSum es = lanes_join<ENT, 32>(run.get(), a);
    if (lane == 0) s_warp[warp] = es;
    late = __syncthreads_or(late);
    if (C > 1) cluster_wait();                               // the row's CTAs are there
    if (warp == 0) {
        es = lanes_join<ENT, (NT / 32)>(s_warp[lane & ((NT / 32) - 1)], a);
        if (C > 1) {
            // the token's logit has been read: its place may be written, where the gradient takes the logits' place
            const uint32_t after = (__float_as_uint(xy) & ~1u) | late;
            if (lane < C) push_sum(&s_peer[rank], &s_bar, lane, es, after);
            late = !bar_wait(&s_bar, 0, kPeerMs) || (kExpirePeerMs && rank == 1 && !bar_wait(&s_bar, 1, kExpirePeerMs)) || late;
            late = __any_sync(0xffffffffu, lane < C && (s_peer[lane & (kMaxCluster - 1)].after & 1u)) || late;
            es = peers_join<ENT>(s_peer, C, a);
        }
        if (lane == 0) {
            bool sure = late || is_quick(es, xy, a.c);
            if (late) s_row = row_bad(DSPARK_ROW_INTERNAL).saved;
            else if (sure) s_row = quick_end<SX, ENT>(a, es, xy, QuickRow{base2(pr.old), base2(pr.ref), pr.w, pr.adv}, sure);
            if (!sure) s_row = row_end<SX, ENT>(a, es, xy, pr).saved;
        }
    }
    __syncthreads();
    const RowGrad<SX, ENT> rg(a, s_row, s_row.a, s_row.h);
    const bool zero = s_row.f < 0.f;
    write_grad<SX, ENT, true, 1, NT>(x, g, k0, k0 + cnt, y, zero, rg, s_x);
    // the first CTA's business, but one whose wait for the others ran out has written zeros: it says so, seconds after it
    if (tid == 0 && (rank == 0 || late)) {
        row_write(a, row, late ? row_bad(DSPARK_ROW_INTERNAL) : row_end<SX, ENT>(a, es, xy, pr), ENT);
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

// A CTA to a pair, half of its warps to a sequence: the sums in pairs of floats (they cancel), the loss, and each row's
// dL/dlog p.  4 us, most of it its launch and three trips to L2 in a row.  More pairs than fit the GPU at once go to its CTAs in
// runs, so that the offsets before a pair are looked through once for a run (for each pair: 2040 us for 65536, 160 in runs).
constexpr int kPairCtas = 152 * 8;
struct __align__(16) SeqSum {
    TwoFloat sum;
    int count, status;
};
__device__ __forceinline__ TwoFloat add_finite(const TwoFloat& a, const TwoFloat& b) {   // infinities and NaN have no low part
    return fabsf(a.hi) < INFINITY && fabsf(b.hi) < INFINITY ? a + b : TwoFloat{a.hi + b.hi, 0.f};
}
__device__ __forceinline__ void one_pair(const PairArgs& a, int p, int lo, int mid, int hi, SeqSum* s_part, float* s_coef, bool* s_none) {
    constexpr int kHalf = kRowThreads / 2;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    SeqSum q{TwoFloat{0.f, 0.f}, 0, 0};
    const int half = tid / kHalf;
    for (int r = (half ? mid : lo) + tid % kHalf; r < (half ? hi : mid); r += kHalf) {
        q.status |= a.row_status[r];
        const float lp = a.saved[r].level, low = a.saved[r].py, ref = a.ref_lp ? a.ref_lp[r] : 0.f;
        if (a.tokens[r] < 0) continue;
        ++q.count;
        TwoFloat gain = a.ref_lp ? two_sum(lp, -ref) : TwoFloat{lp, 0.f};
        gain.lo += low;
        q.sum = add_finite(q.sum, gain);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        q.sum = add_finite(q.sum, TwoFloat{__shfl_xor_sync(0xffffffffu, q.sum.hi, o), __shfl_xor_sync(0xffffffffu, q.sum.lo, o)});
    }
    q.count = __reduce_add_sync(0xffffffffu, q.count);
    q.status = __reduce_or_sync(0xffffffffu, q.status);
    if (lane == 0) s_part[warp] = q;
    __syncthreads();
    if (tid == 0) {
        TwoFloat reward[2];
        float norm[2];
        int st = 0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            SeqSum s = s_part[k * kRowWarps / 2];
#pragma unroll
            for (int w = 1; w < kRowWarps / 2; ++w) {
                const SeqSum& o = s_part[k * kRowWarps / 2 + w];
                s = SeqSum{add_finite(s.sum, o.sum), s.count + o.count, s.status | o.status};
            }
            st |= s.status;
            norm[k] = a.mean ? static_cast<float>(max(s.count, 1)) : 1.f;
            // the mean before beta, which may leave fp32's range; what has left it has no low part
            if (a.mean && fabsf(s.sum.hi) < INFINITY) s.sum = s.sum / TwoFloat{norm[k], 0.f};
            reward[k] = fabsf(s.sum.hi) < INFINITY ? s.sum * TwoFloat{a.beta, 0.f} : TwoFloat{s.sum.hi, 0.f};
            if (!(fabsf(reward[k].hi) < INFINITY)) reward[k].lo = 0.f;
        }
        TwoFloat z{(reward[0].hi - reward[1].hi) - a.margin, 0.f};
        if (fabsf(z.hi) < INFINITY) z = reward[0] + -reward[1] + TwoFloat{-a.margin, 0.f};
        if (!st && z.hi != z.hi) st = DSPARK_ROW_NONFINITE;
        const float w = a.weights ? a.weights[p] : 1.f, e = a.smoothing;
        const Odds of(z);                                    // -log sigma(z) = log(1 + e^-z), -log sigma(-z) = log(1 + e^z)
        float loss = 0.f, by_z = 0.f;
        if (w != 0.f) {
            loss = (1.f - e) * (of.sm - (z.lo * of.p));
            if (e > 0.f) loss += e * (of.sp.hi + of.sp.lo);
            loss *= w;
            by_z = w * (e * of.q - (1.f - e) * of.p);
        }
        s_coef[0] = by_z * a.beta / norm[0];
        s_coef[1] = -by_z * a.beta / norm[1];
        *s_none = st != 0 || w == 0.f;
        a.loss[p] = st ? NAN : loss;
        if (a.rewards)
            for (int k = 0; k < 2; ++k) a.rewards[2 * p + k] = st ? NAN : reward[k].hi + reward[k].lo;
        a.pair_status[p] = st;
    }
    __syncthreads();
    // (a pair without a gradient, of weight 0 too, has none whatever comes from upstream: its NaN loss comes back as NaN)
    const bool none = *s_none;
    for (int r = lo + tid; r < hi; r += kRowThreads) {
        a.saved[r].a = s_coef[r >= mid];
        a.saved[r].pair = p;
        if (none) a.saved[r].f = -1.f;
    }
}
__global__ void __launch_bounds__(kRowThreads) pair_kernel(PairArgs a) {
    __shared__ SeqSum s_part[kRowWarps];
    __shared__ float s_coef[2];
    __shared__ bool s_none;
    const int tid = threadIdx.x;
    pdl_wait();
    const int p0 = static_cast<int>(static_cast<long long>(a.P) * blockIdx.x / gridDim.x);
    const int p1 = static_cast<int>(static_cast<long long>(a.P) * (blockIdx.x + 1) / gridDim.x);
    // the offsets up to a pair's last ascend and stay inside the rows
    int lo = a.offsets[2 * p0], mid = a.offsets[2 * p0 + 1], hi = a.offsets[2 * p0 + 2];
    bool bad = a.offsets[0] < 0;
#pragma unroll 4
    for (int k = tid; k < 2 * p0; k += kRowThreads) bad |= a.offsets[k] > a.offsets[k + 1];
    bad = __syncthreads_or(bad);
    for (int p = p0; p < p1; ++p) {
        if (p > p0) {
            lo = hi;
            mid = a.offsets[2 * p + 1];
            hi = a.offsets[2 * p + 2];
        }
        bad = bad || lo > mid || mid > hi || hi > a.R;
        if (!bad) {
            one_pair(a, p, lo, mid, hi, s_part, s_coef, &s_none);
        } else if (tid == 0) {
            a.loss[p] = NAN;
            if (a.rewards) a.rewards[2 * p] = a.rewards[2 * p + 1] = NAN;
            a.pair_status[p] = DSPARK_ROW_BAD_PARAMS;
        }
    }
}

// ---------------------------------------------------------------- host
// Whether a gradient that does not take the logits' place shares elements with them: a row's gradient would be made of another's.
bool overlaps(const void* logits, const void* grad, const dspark_token_params_t* p, int sx) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(logits), g = reinterpret_cast<uintptr_t>(grad);
    const auto bytes = [&](int64_t stride) { return (static_cast<uintptr_t>(p->n_rows - 1) * stride + p->V) * sx; };
    if (g >= x ? g - x >= bytes(p->logits_stride) : x - g >= bytes(p->grad_stride)) return false;
    if (p->logits_stride != p->grad_stride) return true;     // (rows among each other: not looked into)
    const uintptr_t stride = static_cast<uintptr_t>(p->logits_stride) * sx, row = static_cast<uintptr_t>(p->V) * sx;
    const uintptr_t on = g >= x ? (g - x) % stride : (x - g) % stride;
    return on < row || stride - on < row;
}
dspark_status_t token_args(const void* logits, const dspark_token_params_t* p, const void* grad, TokArgs* a, int* sx) {
    if (!logits || !p || !p->tokens) return DSPARK_ERR_INVALID_ARG;
    if (p->n_rows < 1 || p->n_rows > DSPARK_MAX_ROWS || p->V < 1 || p->V > DSPARK_MAX_V) return DSPARK_ERR_INVALID_ARG;
    if (p->logits_dtype != DSPARK_BF16 && p->logits_dtype != DSPARK_FP32) return DSPARK_ERR_INVALID_ARG;
    const double exact = 1.44269504088896340736 / p->temperature;
    const float c = static_cast<float>(exact);
    const float inv_t = 1.f / p->temperature;
    if (!(p->temperature > 0.f) || !(c > 0.f) || !(c < INFINITY) || !(inv_t < INFINITY)) return DSPARK_ERR_INVALID_ARG;
    *sx = p->logits_dtype == DSPARK_BF16 ? 2 : 4;
    if (p->logits_stride < p->V || reinterpret_cast<uintptr_t>(logits) % *sx) return DSPARK_ERR_INVALID_ARG;
    if (grad && (p->grad_stride < p->V || reinterpret_cast<uintptr_t>(grad) % *sx)) return DSPARK_ERR_INVALID_ARG;
    if (grad && (grad != logits ? overlaps(logits, grad, p, *sx) : p->grad_stride != p->logits_stride)) return DSPARK_ERR_INVALID_ARG;
    a->V = p->V;
    a->c = c;
    a->c_low = static_cast<float>(exact - c);
    float head = c > exact ? std::nextafter(c, 0.f) : c;
    uint32_t bits;
    std::memcpy(&bits, &head, sizeof bits);
    bits &= 0xFFFFFF00u;
    std::memcpy(&head, &bits, sizeof bits);
    a->c_head = head;                                        // the tail is not 0, so that -inf times both is -inf
    a->c_tail = std::max(static_cast<float>(exact - head), std::numeric_limits<float>::denorm_min());
    a->inv_t = inv_t;
    a->inv_c = std::min(1.f / c, std::numeric_limits<float>::max());
    a->above = std::min(kAbove / c, std::numeric_limits<float>::max());
    a->x = logits;
    a->x_stride = p->logits_stride;
    a->g = const_cast<void*>(grad);
    a->g_stride = p->grad_stride;
    a->tokens = p->tokens;
    a->row_status = p->row_status;
    return DSPARK_OK;
}

bool misplaced(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

// A row is a CTA's work where there are rows enough: 456, 912, 1824 or 3648 of them are on the GPU at a time, by CTAs of 512, 256,
// 128 or 64 threads, and take the longer the more they are.
//   - rows for one wave of 512 threads are theirs (400 rows of 151936: 23 us, 27 by 256 threads; 150 of 32000: 4.0 and 4.7; but
//     509 of 50001 fp32: 22 and 20);
//   - rows whose last wave of 256 threads makes them an even number of waves take half as many of 128 (1024 rows of
//     151936: 54 us, 63 by 256; 3600: 167 and 170; more than four: 195 and 188);
//     up to eight of these to an SM have six vectors on their way in place of four (1024 rows: 52 us, and of 50001 fp32 34, 36, 41);
//   - short rows too (700 rows of 12470: 6.1 and 6.5 us; 200 of 16000: 4.8 and 4.1);
//   - what takes little more than one wave of 128 threads is a wave by 64, up to three waves of 256 (by 64, 128, 256: 1900 rows of 12470
//     fp32 19.6, 22.6, 22.5; 2100 of 151936 104, 118, 105; of 20000 fp32 2300 32.7, 34.9, 33.7, 2500 34.6, 36.0, 35.6, 2700 36.9, 37.5,
//     37.8; beyond, as fast or slower: 2828 of 32347 fp32 with the entropy 64.6, 63.1, 66.2, 3600 of 20000 51.0, 49.6, 51.1), of long rows up to
//     two and a half (2300 of 60000 fp32 87.0, 92.9, 85.0), and rows so short that their latencies are most of their time are
//     theirs too (9000 rows of 7200: 37.4 and 31.6 us by 128 and 64; of 10000 39.1 and 38.7, 4096 of them 21.4 and 22.8);
//   - the others are by 256, six to an SM (five: 2% less for 4096 rows of 151936, 900 rows 58 us instead of 46).
// Fewer rows still are split over clusters (9 rows of 151936 in 1, 2, 4, 8 CTAs of 256: 11.4, 7.9, 5.8, 4.5 us; 8 of 512:
// 3.9; shorter rows only where they are a handful: 9 of 32000 whole, in 2, 4, 8 3.7, 4.4, 3.6, 3.2 us, 40 of them 3.9, 4.4, 4.1, 4.2).
constexpr int kWave = 152 * 6;                               // rows by 256 threads
template <int NT, int U = 4>
cudaError_t launch_stats_by(const TokArgs& a, int sx, bool entropy, unsigned grid, int C, cudaStream_t s) {
    auto kern = sx == 2 ? (entropy ? stats_kernel<2, true, NT, U> : stats_kernel<2, false, NT, U>)
                        : (entropy ? stats_kernel<4, true, NT, U> : stats_kernel<4, false, NT, U>);
    return launch_cluster(kern, grid, NT, C, 0, s, a);
}
dspark_status_t launch_stats(TokArgs& a, int sx, bool entropy, const dspark_token_params_t* p) {
    const int nvec = max_vectors(p->V, sx);
    const long long rows = p->n_rows;
    const bool wide = rows <= kWave / 2 && nvec >= 2048;
    const bool thin = rows > kWave / 2 && (nvec <= kShortRow || (rows <= 4 * kWave && (rows + kWave - 1) / kWave % 2 == 0));
    const bool slim = rows > 2 * kWave && (nvec <= kSlimRow || rows <= (nvec <= 8192 ? 3 * kWave : 5 * kWave / 2));
    int C = 1;
    a.log_c = 0;
    const int least = wide && rows <= 16 && nvec <= 8192 ? 512 : 4096;   // vectors that are worth one more CTA
    while (C < kMaxCluster && nvec >= C * least && rows * 2 * C <= (wide ? kWave / 2 : 640)) {
        C *= 2;
        ++a.log_c;
    }
    a.most = 1.f;
    const unsigned grid = static_cast<unsigned>(p->n_rows) * C;
    const cudaStream_t s = static_cast<cudaStream_t>(p->stream);
    const cudaError_t e = wide ? launch_stats_by<512>(a, sx, entropy, grid, C, s)
                          : slim ? launch_stats_by<64>(a, sx, entropy, grid, C, s)
                          : thin ? (rows > kWave && rows <= 1216 ? launch_stats_by<128, 6>(a, sx, entropy, grid, C, s)
                                                                 : launch_stats_by<128>(a, sx, entropy, grid, C, s))
                                 : launch_stats_by<256>(a, sx, entropy, grid, C, s);
    return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

// Of fp32 32 KB of a row to a CTA of 256 threads (16 KB: 3% slower for 509 rows of 50001, 8 KB: 34%); of bf16, with twice the
// instructions to a byte, 16 KB to one of 128 (2000 rows of 151936 with the entropy 177 us, 32 KB to 256 threads 200; without
// it 335 and 332 for 3843); of many short rows 16 KB to one of 64 (16000 rows of 5000 bf16: 51 us, 57 by 128; 500 of them 3.0, 2.7).
template <int SX, int NT, int VECS>
cudaError_t launch_grad_by(TokArgs& a, bool entropy, const dspark_token_params_t* p) {
    a.splits = (max_vectors(p->V, SX) + VECS - 1) / VECS;
    auto kern = entropy ? grad_kernel<SX, true, NT, VECS> : grad_kernel<SX, false, NT, VECS>;
    return launch_cluster(kern, static_cast<unsigned>(p->n_rows) * a.splits, NT, 1, 0, static_cast<cudaStream_t>(p->stream), a);
}
dspark_status_t launch_grad(TokArgs& a, int sx, bool entropy, const dspark_token_params_t* p) {
    const int nvec = max_vectors(p->V, sx);
    if (static_cast<long long>(p->n_rows) * ((nvec + 1023) / 1024) > 0x7fffffffLL) return DSPARK_ERR_UNSUPPORTED;
    const bool slim = nvec <= kShortRow && p->n_rows > kWave;
    const cudaError_t e = sx == 2 ? (slim ? launch_grad_by<2, 64, 1024>(a, entropy, p) : launch_grad_by<2, 128, 1024>(a, entropy, p))
                                  : (slim ? launch_grad_by<4, 64, 1024>(a, entropy, p) : launch_grad_by<4, 256, 2048>(a, entropy, p));
    return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

// CTAs of a row whose span stays in shared memory; 0 when the row is too long for eight of them.  Of the splits that fit, the
// one by which an SM holds the most bytes (4096 rows of 151936 bf16 in 4, 5, 6, 7, 8: 407, 443, 411, 392, 409 us for 152,
// 182, 203, 217, 190 KB; 2048 fp32 rows of it in eighths of 76 KB: 412 us, read twice 525); few rows in more
// (100 of 32000 in 1, 2, 4, 8: 6.2, 6.3, 5.7, 8.3 us, 37 of them 6.1, 5.3, 5.0, 4.8).
int fused_split(int nvec, long long rows) {
    int C = 1;
    while (C < kMaxCluster && nvec >= C * 512 && rows * 2 * C <= 400) C *= 2;
    int best = 0;
    for (int c = C, most = 0; c <= kMaxCluster; ++c) {
        const int span = (nvec + c - 1) / c;
        if (c > C && span < 512) break;
        if (span > kFusedSpan) continue;
        const int held = span * std::min(kFusedCtas, 228 * 1024 / (16 * span + 2 * 1024));
        if (held >= most) {
            most = held;
            best = c;
        }
    }
    return best;
}

template <int NT>
cudaError_t launch_kept_by(TokArgs& a, int sx, bool entropy, const dspark_token_params_t* p) {
    auto kern = sx == 2 ? (entropy ? kept_kernel<2, true, NT> : kept_kernel<2, false, NT>)
                        : (entropy ? kept_kernel<4, true, NT> : kept_kernel<4, false, NT>);
    const size_t smem = static_cast<size_t>(a.span) * 16;
    // beyond what a launch gets unasked; the same for every call, as another thread's may come between
    if (smem > 32 * 1024)
        if (const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 16 * kFusedSpan); e != cudaSuccess) return e;
    return launch_cluster(kern, static_cast<unsigned>(p->n_rows) * a.splits, NT, a.splits, smem, static_cast<cudaStream_t>(p->stream), a);
}
dspark_status_t launch_kept(TokArgs& a, int sx, bool entropy, const dspark_token_params_t* p, int C) {
    a.splits = C;
    a.span = (max_vectors(p->V, sx) + C - 1) / C;
    a.most = 64.f;                                           // (1: 387 us for 377, 4096 rows of 151936; no row's loss is a long sum)
    const cudaError_t e = C == 1 && a.span <= kShortRow ? launch_kept_by<128>(a, sx, entropy, p) : launch_kept_by<256>(a, sx, entropy, p);
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
    const bool entropy = out_entropy || policy->entropy_coef != 0.f;
    if (out_grad)
        if (const int C = fused_split(max_vectors(params->V, sx), params->n_rows); C > 0) return launch_kept(a, sx, entropy, params, C);
    const dspark_status_t st = launch_stats(a, sx, entropy, params);
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
    if (launch_cluster(pair_kernel, static_cast<unsigned>(std::min(pref->n_pairs, kPairCtas)), kRowThreads, 1, 0,
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
