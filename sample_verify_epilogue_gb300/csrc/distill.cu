// distill_kernel: the divergence of a student's softmax from a teacher known by its top logits,
// its gradient, or both in one launch; each row split over a cluster of C CTAs.
//
// With e_v = exp(s_v / T) up to a factor of the row, Z = sum e_v, R = sum of e_v outside the record's
// set S:
//   L = sum_S p_i (log p_i - log e_i + log Z) + p_r log(p_r Z / R)
//   dL/ds_v = (e_v a - p_v / T) in S, e_v b outside,  a = M / (Z T),  b = (M/Z - p_r/R) / T
// R is summed without the members of S rather than taken as Z less their sum, which cancels when
// they carry nearly all mass, and both sums have a maximum of their own: by the row's, R would vanish where a
// member lies 87 T above everything outside S, with p_r log(p_r Z / R) and the gradient there, which then is
// -p_r e_v / R.  Only where R / Z is below 2^-kDisApart (masks of the type's lowest value) does it count as 0.
//
// Bound by bandwidth: s is read once and the gradient written once (4096 rows of 151936 bf16, a tenth
// of weight 0: 358 us, 0.98 of what the copy bandwidth takes for the same bytes).  For both results a CTA's
// span of the row comes to shared memory by bulk copies and stays there between the sum and the gradient,
// so that the row is not read twice; an SM holds some 200 KB of rows.  What bounds the rate is how long a
// CTA lives, so everything between copy and store is kept short and wide.  The record is one thread's
// work per entry; while the span arrives they make the teacher's probabilities, then take the members out:
// each notes its logit and leaves -inf in its place, so that the two loops over the span know nothing of
// S, and writes its member's gradient over at the end.  (The record by one warp: 6000 cycles of a CTA's
// 24600; the members looked up from inside the loops: 2800.)
// For one result a CTA streams its span through two 16 KB buffers, six CTAs to an SM (2048 rows of 151936,
// loss alone: 96 us, 0.86 of the bandwidth; of 32000: 30 us, 0.65, and the gradient alone 43 us, 0.89:
// there a CTA waits for its row's ids, first pieces and joins about as long as it reads).  Spans too
// long to keep go through the buffers twice; the second read is then from L2.
//
// Sums that meet cancellation (p_i log p_i/e_i) are held as pairs of floats, and by 2^-k so that logits of
// the types' lowest values do not pass fp32's range on the way.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "vocab_rows.cuh"

namespace dspark {

namespace {

constexpr int kDisVec = 4;                                   // vectors a thread holds at a time
constexpr int kDisSpan = 4608;                               // vectors of a span kept in one piece at most
constexpr int kDisPiece = 1024;                              // vectors of a piece of a longer one
constexpr int kDisCtas = 5;                                  // CTAs of one-piece spans an SM takes at most
constexpr int kSmSmem = 228 * 1024, kCtaSmem = 4 * 1024;     // an SM's shared memory; what a CTA takes beside its span
static_assert(DSPARK_MAX_TOP_LOGITS <= kRowThreads, "a thread per record entry");

enum DistillPass : int { kLoss = 1, kGrad = 2 };

struct DisArgs {
    int V, n, log_c, target_V;                               // log_c: log2 of C, rounded up
    int piece, np, log_slots;                                // vectors of a piece, pieces of a span; buffers (1 or 2)
    float c;                                                 // log2(e) / T
    float inv_t, inv_t_low;                                  // 1 / T in two parts
    float down, up_again;                                    // 2^-k, 2^k
    float unit2, unit2_low;                                  // 2 ln 2 times c, by 2^-k: the sums' own 1/T (c is rounded)
    long long s_stride, g_stride;
    const void* s;
    void* g;
    const int* ids;
    const float* tl;
    const float* lse;
    const int* t2d;
    const float* weights;
    const float* up;                                         // upstream gradient of each row or null
    float* loss;
    float* saved_out;
    const float* saved;
    int* row_status;
    int C, span;                                             // CTAs of a row, vectors of each
};

struct __align__(16) DisCross {                              // a CTA's part of the loss
    TwoFloat sum;
    int flags, unused;                                       // status bits, or kDisInf
};
constexpr int kDisInf = 1 << 30;                             // a member with p > 0 has a logit of -inf
constexpr int kDisStopped = 1 << 29;                         // a copy was late: no further one is asked for
// powers of two between the units of Z and R: from here on R is nothing beside Z; up to here fp32 holds R by Z's
constexpr float kDisApart = 4194304.f, kDisNear = 96.f;

struct DisRow {                                              // a row's sums
    ExpSum out;                                              // outside S, by the maximum there
    float m, apart;                                          // the row's maximum; powers of two by which its unit is larger than out's
    float in_m, out_m, total;                                // the sums by m; Z by m, NaN when there is none
};

struct __align__(16) DisSmem {
    alignas(16) ExpSum all[2 * kMaxCluster];                 // sums in S, then outside: written by the cluster's CTAs
    alignas(16) ExpSum warp[2 * kRowWarps];
    DisCross cross_all[kMaxCluster];                         // (in the row's first CTA) written by the cluster's
    TwoFloat cross[kRowWarps];
    uint64_t bar[2], part_bar, cross_bar;
    alignas(16) unsigned wkey[kRowWarps];                    // largest key of 32 entries' logits
    alignas(16) TwoFloat wsum[kRowWarps];                    // sum of their probabilities
    DisRow row;
    float wt, scale_in, scale_out;
    float by, out;                                           // outside S: maximum that its exponentials are by, their factor
    TwoFloat log_z, log_sum;                                 // the loss's parts by 2^-k: log Z, log of the record's sum,
    float last;                                              // the last class's term
    int flags;                                               // of this CTA
    int id[DSPARK_MAX_TOP_LOGITS];                           // draft ids of the record, -1: none
    unsigned seen[kRowThreads];                              // 8192 bits: hashes of the ids met
};
static_assert(sizeof(DisSmem) + 1024 <= kCtaSmem, "the system takes 1 KB of a CTA's");
constexpr unsigned kSeenBits = 32 * kRowThreads;

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

// ONE: the span is one piece.
template <int SX, int PASS, bool ONE>
__global__ void __launch_bounds__(kRowThreads, ONE ? kDisCtas : 6) distill_kernel(DisArgs a) {
    constexpr int VE = VocabRow<SX>::VE;
    constexpr bool kWantLoss = (PASS & kLoss) != 0, kWantGrad = (PASS & kGrad) != 0;
    __shared__ DisSmem s;
    extern __shared__ uint4 s_x[];                           // [slots][piece]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // only spans kept whole come in other numbers than a power of two: the streaming forms have no registers
    // to spare at six CTAs to an SM (backward of 2048 rows of 32000: 1.5 us for two spilled)
    constexpr bool kAnyC = ONE && kWantLoss && kWantGrad;
    const int C = kAnyC ? a.C : 1 << a.log_c;
    const int rank = kAnyC ? static_cast<int>(cluster_rank()) : static_cast<int>(blockIdx.x & (C - 1));
    const long long row = kAnyC ? cluster_id() : blockIdx.x >> a.log_c;
    const VocabRow<SX> x(a.s, row, a.s_stride, a.V);
    const VocabRow<SX> g(a.g, row, a.g_stride, a.V);
    const int k0 = kAnyC ? min(x.nvec, rank * a.span) : x.nvec * rank >> a.log_c;   // nvec * C < 2^31
    const int k1 = kAnyC ? min(x.nvec, k0 + a.span) : x.nvec * (rank + 1) >> a.log_c;
    const bool same_phase = x.a0 == g.a0;

    if (tid == 0) {
        s.flags = 0;
        mbar_init(&s.bar[0], 1);
        mbar_init(&s.bar[1], 1);
        if (kWantLoss && C > 1) {
            mbar_init(&s.part_bar, 1);
            mbar_init(&s.cross_bar, 1);
        }
        fence_mbar_init();
        if (kWantLoss && C > 1) {
            mbar_arrive_expect_tx(&s.part_bar, sizeof(ExpSum) * 2 * C);
            mbar_arrive_expect_tx(&s.cross_bar, sizeof(DisCross) * C);
        }
    }
    s.seen[tid] = 0u;
    if (kWantLoss && C > 1) cluster_arrive_relaxed();        // before a peer can push here (the fence above orders it)
    pdl_wait();                                              // what came before in the stream
    const float w = a.weights ? a.weights[row] : 1.f;
    // the record's entries go to the last warp first, so that the first one fetches and joins meanwhile (0.3 to
    // 0.6 us a call, but 0.5 more for n = 256); the gradient alone has no joins, and no registers to spare
    const int ent = kWantLoss ? tid ^ (kRowThreads - 32) : tid, part = ent >> 5;
    int id = ent < a.n ? a.ids[row * a.n + ent] : -1;
    const float t = ent < a.n ? a.tl[row * a.n + ent] : 0.f;
    const float lse = a.lse ? a.lse[row] : 0.f;

    auto zeros = [&]() {
        for (int k = k0 + tid; k < k1; k += kRowThreads) store_vec<SX>(g, x.first(k), make_uint4(0, 0, 0, 0), same_phase);
    };
    // a row that is not reduced: loss, status and gradient; the same branch in every CTA of the row
    auto leave = [&](int status) {
        if (kWantLoss && rank == 0 && tid == 0) {
            a.loss[row] = status ? NAN : 0.f;
            a.row_status[row] = status;
            if (a.saved_out)
                for (int k = 0; k < 4; ++k) a.saved_out[4 * row + k] = 0.f;
        }
        if (kWantGrad) zeros();
        if (kWantLoss && C > 1) cluster_wait();
    };
    // The span in np pieces (the last may be short, or empty); copy number f (the pieces in turn, then
    // again for a second pass) goes to buffer f mod slots; warp 0 fetches.
    const int np = ONE ? 1 : a.np, log_slots = ONE ? 0 : a.log_slots, slots = 1 << log_slots;
    auto lo = [&](int j) { return min(k1, k0 + j * a.piece); };
    auto hi = [&](int j) { return min(k1, k0 + (j + 1) * a.piece); };
    auto buffer = [&](int f) { return s_x + (f & (slots - 1)) * a.piece; };
    auto fetch = [&](int f) {
        const int j = f < np ? f : f - np;
        fetch_piece<SX>(x, lo(j), hi(j), buffer(f), &s.bar[f & (slots - 1)]);
    };
    if (w == 0.f) {
        leave(0);
        return;
    }
    if (warp == 0)
        for (int f = 0; f < min(np, slots); ++f) fetch(f);

    // ---- the record, a thread to an entry; warps past it have nothing to do
    const bool entries = 32 * part < a.n;
    const int n_warps = (a.n + 31) >> 5;
    bool bad = !isfinite(lse);
    if (entries) {
        if (id < -1 || id >= (a.t2d ? a.target_V : a.V)) { bad = true; id = -1; }
        if (a.t2d && id >= 0) {
            id = a.t2d[id];
            if (id < -1 || id >= a.V) { bad = true; id = -1; }
        }
        if (id >= 0 && !(t < INFINITY)) { bad = true; id = -1; }
        s.id[ent] = id;
        const unsigned key = __reduce_max_sync(0xffffffffu, id >= 0 ? fkey(t) : 0u);   // 0: no entry
        if (lane == 0) s.wkey[part] = key;
    }
    __syncthreads();
    unsigned top = 0u;
    for (int k = 0; k < n_warps; ++k) top = max(top, s.wkey[k]);
    float lp = -INFINITY, lp_low = 0.f, p = 0.f;             // log p in two parts
    if (entries) {
        const float tmax = key_to_f(top);
        if (id >= 0) {
            if (t > -INFINITY) {
                const float ih = a.inv_t, il = a.inv_t_low;
                if (a.lse) {                                 // 1 - sum p is what is left of the mass: p to its last bits
                    const float prod = t * ih, rest = fmaf(t, ih, -prod);
                    const TwoFloat d = two_sum(prod, -lse);
                    lp = d.hi;
                    lp_low = lp > -INFINITY ? d.lo + fmaf(t, il, rest) : 0.f;   // (the lowest value over T below 1)
                    p = expf(lp);
                    p = fmaf(p, lp_low, p);
                } else {
                    const float d = t - tmax;
                    lp = d * ih;
                    lp_low = fmaf(d, il, fmaf(d, ih, -lp));
                    p = expf(lp);
                }
            }
        }
        // a repeated id: the warp looks for the entries whose hash was met before, one after the other
        // (an entry by itself through the record: 65 us where this takes 44, 2048 rows of 32000, n = 256)
        const unsigned h = (static_cast<unsigned>(id) * 2654435761u) >> 19;
        static_assert(kSeenBits == 1u << 13, "the hash has 13 bits");
        unsigned met = __ballot_sync(0xffffffffu, id >= 0 && (atomicOr(&s.seen[h >> 5], 1u << (h & 31)) >> (h & 31) & 1u));
        for (; met; met &= met - 1) {
            const int from = __ffs(met) - 1, other = __shfl_sync(0xffffffffu, id, from);
            for (int k = lane; k < a.n; k += 32) bad = bad || (s.id[k] == other && k != 32 * part + from);
        }
        // only -inf in the record, a log-sum-exp far below its logits
        bad = bad || (top != 0u && !a.lse && !(tmax > -INFINITY)) || !(p < INFINITY);
        TwoFloat ws{p, 0.f};
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const float hi = __shfl_xor_sync(0xffffffffu, ws.hi, o), lo = __shfl_xor_sync(0xffffffffu, ws.lo, o);
            const TwoFloat d = two_sum(ws.hi, hi);
            ws = TwoFloat{d.hi, d.lo + (ws.lo + lo)};
        }
        if (lane == 0) s.wsum[part] = ws;
    }
    const int status0 = __syncthreads_or(bad) ? DSPARK_ROW_BAD_TEACHER : 0;
    TwoFloat sum{0.f, 0.f};
    for (int k = 0; k < n_warps; ++k) {
        const TwoFloat d = two_sum(sum.hi, s.wsum[k].hi);
        sum = TwoFloat{d.hi, d.lo + (sum.lo + s.wsum[k].lo)};
    }
    // the entries' p stand as they are; with a log-sum-exp the rest of the mass is p_r, without one
    // their sum is what they are relative to
    float mass = sum.hi, p_r = 0.f;                          // M = sum of p + p_r
    if (a.lse) {
        p_r = fmaxf((1.f - sum.hi) - sum.lo, 0.f);
        if (p_r > 0.f) mass = 1.f;
    }
    // p_r Z / R - 1 for Z = R + in (both by one maximum), p_r = 1 - sum: without the difference of the two near ones
    auto tail_excess = [&](float rest, float in) {
        const float z = sum.hi * rest;
        return ((fmaf(p_r, in, -z) - fmaf(sum.hi, rest, -z)) - sum.lo * rest) / rest;
    };
    if (status0 || top == 0u) {
        bool late = false;
        if (warp == 0)
            for (int f = 0; f < min(np, slots); ++f)
                if (!bar_wait(&s.bar[f], 0)) {
                    late = true;
                    bar_wait(&s.bar[f], 0);                  // once more: it is in flight
                }
        late = __syncthreads_or(late);
        leave(status0 ? status0 : late ? DSPARK_ROW_INTERNAL : 0);
        return;
    }
    if (kWantLoss && C > 1) cluster_wait();                  // the peers' barriers stand

    float v = -INFINITY;                                     // this thread's member: its logit
    bool here = false;                                       // ... is in this span
    constexpr bool kTwice = kWantLoss && kWantGrad && !ONE;  // the pieces come again for the gradient
    // Wait for copy f of piece j; its members are noted and replaced by -inf.  Ends with a barrier.
    auto arrive = [&](int f, int j, bool note) {
        const int i0 = x.first(lo(j));
        const bool in = entries && id >= max(0, i0) && id < min(a.V, x.first(hi(j)));
        auto parity = [&](int k) { return static_cast<unsigned>(k >> log_slots) & 1u; };
        if ((warp == 0 || (entries && __any_sync(0xffffffffu, in))) &&
            !copy_wait(&s.bar[f & (slots - 1)], parity(f), ONE ? nullptr : &s.flags)) {
            if (warp == 0 && !(s.flags & kDisStopped)) {     // those in flight arrive before the CTA ends
                for (int k = f; k < min(f + slots, kTwice ? 2 * np : np); ++k) bar_wait(&s.bar[k & (slots - 1)], parity(k));
                atomicOr(&s.flags, kDisStopped);
            }
            atomicOr(&s.flags, DSPARK_ROW_INTERNAL);
        }
        if (in && note) {
            using Bits = std::conditional_t<SX == 2, unsigned short, unsigned>;
            Bits* const at = reinterpret_cast<Bits*>(buffer(f)) + (id - i0);
            v = __uint_as_float(static_cast<uint32_t>(*at) << (SX == 2 ? 16 : 0));
            *at = static_cast<Bits>(ninf_bits<SX>());
            here = true;
        }
        __syncthreads();
    };
    // The buffer of copy f - slots is free for copy f (entry warps have written to it).
    auto refill = [&](int f) {
        if (entries) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        const bool late = (s.flags & kDisStopped) != 0;
        __syncthreads();
        if (warp != 0) return;
        if (!late) fetch(f);
    };
    auto has_tail = [&](const DisRow& r) { return p_r > 0.f && r.out.sum > 0.f && r.apart < kDisApart; };

    // the gradient's factor outside S, b T, by one thread
    auto outside = [&](const DisRow& r) {
        const bool tail = has_tail(r);                       // M/Z - p_r/R, M = 1
        s.by = tail ? r.out.m : r.m;
        if (tail && r.apart >= kDisNear) return s.out = -p_r / r.out.sum;
        return s.out = !tail ? mass / r.total : -(tail_excess(r.out_m, r.in_m) / r.total) * ex2_approx(-r.apart);
    };
    // what the gradient is made with, by one thread
    auto scales = [&](float total, float out) {
        float wt = (a.up ? w * a.up[row] : w) * a.inv_t;
        if (!a.lse) wt /= sum.hi;
        s.wt = wt;
        s.scale_in = wt * (mass / total);
        s.scale_out = wt * out;
    };

    // what the loss is made of, by one thread
    auto logs = [&](const DisRow& r) {
        auto scaled = [&](const TwoFloat& l) { return TwoFloat{l.hi * a.down, l.lo * a.down}; };
        const ExpRef ref(r.m, a.c);
        const TwoFloat log_z = scaled(log_two(r.total));
        s.log_z = ref.whole ? TwoFloat{ref.r * a.down, 0.f} * ln2_two() + log_z : log_z;
        if (!a.lse) s.log_sum = scaled(log_two(sum.hi));
        float last = 0.f;
        if (has_tail(r)) {
            const bool near = r.apart < kDisNear;
            const float x = near ? tail_excess(r.out_m, r.in_m) : 1.f;
            last = fabsf(x) < 0.5f ? log1pf(x) : fmaf(near ? 0.f : r.apart, ln2_two().hi, logf(p_r * (r.total / (near ? r.out_m : r.out.sum))));
            last *= p_r * a.down;
        }
        s.last = last;
    };

    // the CTA's part of the loss to the row's first, by one warp
    auto push_cross = [&]() {
        if (warp != 0) return;
        TwoFloat cross = lane < kRowWarps ? s.cross[lane] : TwoFloat{0.f, 0.f};
#pragma unroll
        for (int i = kRowWarps / 2; i; i >>= 1)
            cross = cross + TwoFloat{__shfl_xor_sync(0xffffffffu, cross.hi, i), __shfl_xor_sync(0xffffffffu, cross.lo, i)};
        if (lane != 0) return;
        if (C > 1)
            peer_push128(peer_addr(&s.cross_all[rank], 0), peer_addr(&s.cross_bar, 0), __float_as_uint(cross.hi),
                         __float_as_uint(cross.lo), static_cast<uint32_t>(s.flags), 0u);
        else s.cross_all[0] = DisCross{cross, s.flags, 0};
    };

    // ---- Z and R
    if (kWantLoss) {
        RunSum run;
        for (int j = 0; j < np; ++j) {
            arrive(j, j, true);
            const uint4* const q0 = buffer(j);
            const int cnt = hi(j) - lo(j);
            int k = tid;
            for (; k + (kDisVec - 1) * kRowThreads < cnt; k += kDisVec * kRowThreads) {
                uint4 q[kDisVec];
#pragma unroll
                for (int u = 0; u < kDisVec; ++u) q[u] = q0[k + u * kRowThreads];
                add_exps<SX>(run, q, vecs_max<SX>(q), a.c);
            }
            for (; k < cnt; k += kRowThreads) {
                const uint4 q[1] = {q0[k]};
                add_exps<SX>(run, q, vecs_max<SX>(q), a.c);
            }
            if (!ONE && j + slots < (kTwice ? 2 * np : np)) refill(j + slots);
        }
        const ExpSum es = run.get();
        // the warp's part, then the CTA's to every CTA of the row, then the row's
        const bool mine = entries && __any_sync(0xffffffffu, here);
        {
            const float m_out = key_to_f(__reduce_max_sync(0xffffffffu, fkey(es.m)));
            const float rest = warp_sum(m_out > -INFINITY ? es.sum * rebase(es.m, m_out, a.c) : es.sum);
            ExpSum in{-INFINITY, 0.f};
            if (mine) {
                in.m = key_to_f(__reduce_max_sync(0xffffffffu, fkey(v)));
                in.sum = warp_sum(here ? ExpRef(in.m > -INFINITY ? in.m : 0.f, a.c).of(v) : 0.f);   // NaN for NaN and +inf
            }
            if (lane == 0) {
                s.warp[warp] = in;
                s.warp[kRowWarps + warp] = ExpSum{m_out, rest};
            }
        }
        __syncthreads();
        // by one warp, in lane order: the sums in S in lanes 0 to 7, outside in 8 to 15; every lane has both maxima
        static_assert(kRowWarps == 8 && kMaxCluster == 8, "eight lanes to a join");
        float m_in = -INFINITY, m_out = -INFINITY;
        auto join = [&](const ExpSum* parts, int count) {
            const bool used = lane < 16 && (lane & 7) < count;
            ExpSum o{-INFINITY, 0.f};
            if (used) o = parts[lane];
            const unsigned key = fkey(o.m);
            m_in = key_to_f(__reduce_max_sync(0xffffffffu, lane < 8 ? key : 0u));
            m_out = key_to_f(__reduce_max_sync(0xffffffffu, lane < 8 ? 0u : key));
            const float m = lane < 8 ? m_in : m_out;
            if (m > -INFINITY) o.sum *= rebase(o.m, m, a.c);
#pragma unroll
            for (int i = 4; i; i >>= 1) o.sum += __shfl_xor_sync(0xffffffffu, o.sum, i);
            o.m = m;
            return o;
        };
        // the row's sums of what join gives, in lane 0
        auto row_of = [&](float joined) {
            const ExpRef i(m_in, a.c), o(m_out, a.c);
            const float x = i.whole && o.whole ? i.r - o.r : (m_in - m_out) * a.c;   // NaN for a row of -inf
            const float by_m = joined * ex2_approx(fminf(lane < 8 ? x : -x, 0.f));
            const float out = __shfl_sync(0xffffffffu, joined, 8), out_m = __shfl_sync(0xffffffffu, by_m, 8);
            return DisRow{ExpSum{m_out, out}, fmaxf(m_in, m_out), fmaxf(x, 0.f), by_m, out_m, x == x ? by_m + out_m : NAN};
        };
        ExpSum o;
        if (warp == 0) {
            o = join(s.warp, kRowWarps);
            if (s.flags & DSPARK_ROW_INTERNAL) o.sum = NAN;  // no gradient from any CTA
            if (C > 1 && lane < 16 && (lane & 7) < C)
                peer_push64(peer_addr(&s.all[(lane & 8) + rank], lane & 7), peer_addr(&s.part_bar, lane & 7), pack2(o.m, o.sum));
        }
        // sum p_i (log p_i - (v_i - from) / T) of the warp's members
        auto cross_from = [&](float from) {
            TwoFloat cross{0.f, 0.f};
            if (mine) {
                if (here && p > 0.f && !(v > -INFINITY)) {
                    atomicOr(&s.flags, kDisInf);             // (or NaN, which no loss comes of either)
                } else if (here && p > 0.f) {
                    const TwoFloat to = two_prod(p, lp * a.down);
                    cross = TwoFloat{to.hi, fmaf(p, lp_low * a.down, to.lo)} +
                            -(two_prod(p, v * 0.5f - from * 0.5f) * TwoFloat{a.unit2, a.unit2_low});   // halves: in range
                }
#pragma unroll
                for (int o = 16; o; o >>= 1)
                    cross = cross + TwoFloat{__shfl_xor_sync(0xffffffffu, cross.hi, o), __shfl_xor_sync(0xffffffffu, cross.lo, o)};
            }
            if (lane == 0) s.cross[warp] = cross;
        };
        cross_from(0.f);                                     // while the parts are on their way
        if (warp == 0) {
            bool none = false;
            if (C > 1) {
                none = !bar_wait(&s.part_bar, 0, kPeerMs);
                o = join(s.all, C);
            }
            DisRow r = row_of(o.sum);
            if (lane == 0) {
                if (none) {
                    atomicOr(&s.flags, DSPARK_ROW_INTERNAL);
                    r.total = NAN;
                }
                s.row = r;
                if (kWantGrad) scales(r.total, outside(r));
                else logs(r);
            }
        }
        __syncthreads();
        if (!ExpRef(s.row.m, a.c).whole) {                   // logits of the lowest values: what is left of them counts
            cross_from(s.row.m);
            __syncthreads();
        }
        if (!kTwice) push_cross();
    }

    // ---- the gradient
    if (kWantGrad) {
        const float* const saved = kWantLoss ? nullptr : a.saved + 4 * row;
        const float total = kWantLoss ? s.row.total : saved[1], by = kWantLoss ? s.by : saved[2];
        const bool ok = total > 0.f;                         // NaN for a row that cannot be normalised
        if (!kWantLoss) {
            if (tid == 0) {
                s.row.m = saved[0];
                scales(total, saved[3]);
            }
            __syncthreads();
        }
        const float scale = s.scale_out;
        const ExpRef ref(by, a.c);                           // of what lies outside S
        const unsigned long long c2 = pack2(a.c, a.c), r2 = pack2(-ref.r, -ref.r), s2 = pack2(scale, scale);
        auto pack = [&](const float (&f)[VE]) {
            if (SX == 2) return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4 % VE], f[5 % VE]), pack_bf16(f[6 % VE], f[7 % VE]));
            return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
        };
        auto grad_whole = [&](const uint4& q) {
            float f[VE];
#pragma unroll
            for (int h = 0; h < VE / 2; ++h) {
                float lo, hi;
                unpack2(fma2(pair_of<SX>(q, h), c2, r2), lo, hi);
                unpack2(mul2(pack2(ex2_approx(lo), ex2_approx(hi)), s2), f[2 * h], f[2 * h + 1]);
            }
            return pack(f);
        };
        auto grad_far = [&](const uint4& q) {                // logits of the type's lowest values
            float f[VE];
#pragma unroll
            for (int h = 0; h < VE; ++h) f[h] = ref.of(elem<SX>(q, h)) * scale;
            return pack(f);
        };
        // one piece is still in its buffer from the sum
        for (int j = 0; j < np; ++j) {
            const int f = kWantLoss ? np + j : j;
            if (!kWantLoss || !ONE) arrive(f, j, !kWantLoss);
            const uint4* const q0 = buffer(f);
            const int b = lo(j), cnt = hi(j) - b;
            // whole vectors of rows that lie alike go straight through
            int w0 = 0, w1 = 0;
            if (ok && ref.whole && same_phase) {
                w0 = !x.whole(b);
                w1 = cnt - (cnt > w0 && !x.whole(b + cnt - 1));   // both 0 or 1 from the ends
                unsigned char* gp = const_cast<unsigned char*>(g.p) + static_cast<long long>(x.first(b + w0 + tid)) * SX;
                const uint4* const end = q0 + w1;
#pragma unroll 2
                for (const uint4* q = q0 + w0 + tid; q < end; q += kRowThreads, gp += 16 * kRowThreads) st_vec16(gp, grad_whole(*q));
            }
            // the ragged ones, or all of them
            auto one = [&](int k) {
                store_vec<SX>(g, x.first(b + k), !ok ? make_uint4(0, 0, 0, 0) : ref.whole ? grad_whole(q0[k]) : grad_far(q0[k]), same_phase);
            };
            if (w1 > w0) {
                if (tid < w0) one(0);
                if (tid < cnt - w1) one(cnt - 1);
            } else {
                for (int k = tid; k < cnt; k += kRowThreads) one(k);
            }
            if (!ONE && j + slots < np) refill(f + slots);
        }
        __syncthreads();                                     // the members' gradients go over the span's
        // a piece that did not come in time leaves no gradient
        const bool in_time = (kWantLoss && ONE) || !(s.flags & DSPARK_ROW_INTERNAL);
        if (!in_time) zeros();
        else if (here && ok) {
            const float d = fmaf(-p, s.wt, ExpRef(s.row.m, a.c).of(v) * s.scale_in);
            unsigned char* const gp = const_cast<unsigned char*>(g.p);
            if (SX == 2) reinterpret_cast<unsigned short*>(gp)[id] = static_cast<unsigned short>(to_bits<SX>(d));
            else reinterpret_cast<float*>(gp)[id] = d;
        }
        if (kTwice) push_cross();                            // with what the second look at the pieces met
        if (!kWantLoss && tid == 0 && !in_time && a.row_status) a.row_status[row] = DSPARK_ROW_INTERNAL;
    }
    if (kWantLoss && rank == 0 && warp == 0) {               // the loss
        const bool none = C > 1 && !bar_wait(&s.cross_bar, 0, kPeerMs);
        __syncwarp();
        if (lane == 0) {
            if (kWantGrad) logs(s.row);
            TwoFloat loss = sum * s.log_z;
            int flags = none ? DSPARK_ROW_INTERNAL : 0;
            for (int k = 0; k < C; ++k) {
                loss = loss + s.cross_all[k].sum;
                flags |= s.cross_all[k].flags;
            }
            const int status = flags & DSPARK_ROW_INTERNAL ? DSPARK_ROW_INTERNAL : s.row.total == s.row.total ? 0 : DSPARK_ROW_NONFINITE;
            if (!a.lse) loss = loss / sum + -s.log_sum;
            loss = loss + TwoFloat{s.last, 0.f};
            loss = loss * TwoFloat{w, 0.f};
            a.loss[row] = status ? NAN : flags & kDisInf ? w * INFINITY : fabsf(loss.hi) < INFINITY ? (loss.hi + loss.lo) * a.up_again : loss.hi;
            a.row_status[row] = status;
            if (a.saved_out) {
                if (!kWantGrad) outside(s.row);
                a.saved_out[4 * row + 3] = s.out;
                a.saved_out[4 * row] = s.row.m;
                a.saved_out[4 * row + 1] = status ? NAN : s.row.total;
                a.saved_out[4 * row + 2] = s.by;
            }
        }
    }
}

// Checks shared by the two entry points; on success *a and *sx are set.
dspark_status_t distill_args(const void* student, const dspark_teacher_t* t, const dspark_distill_params_t* p, const void* grad,
                             bool both, DisArgs* a, int* sx) {
    if (!student || !t || !p || !t->ids || !t->logits) return DSPARK_ERR_INVALID_ARG;
    if (p->n_rows < 1 || p->n_rows > DSPARK_MAX_ROWS || p->V < 1 || p->V > DSPARK_MAX_V) return DSPARK_ERR_INVALID_ARG;
    if (t->n < 1 || t->n > DSPARK_MAX_TOP_LOGITS) return DSPARK_ERR_INVALID_ARG;
    if (t->t2d && (t->target_V < 1 || t->target_V > DSPARK_MAX_V)) return DSPARK_ERR_INVALID_ARG;
    if (p->logits_dtype != DSPARK_BF16 && p->logits_dtype != DSPARK_FP32) return DSPARK_ERR_INVALID_ARG;
    const float c = kLog2E / p->temperature;
    if (!(p->temperature > 0.f) || !(c > 0.f) || !(c < INFINITY)) return DSPARK_ERR_INVALID_ARG;
    *sx = p->logits_dtype == DSPARK_BF16 ? 2 : 4;
    if (p->student_stride < p->V || reinterpret_cast<uintptr_t>(student) % *sx) return DSPARK_ERR_INVALID_ARG;
    if (grad && (p->grad_stride < p->V || reinterpret_cast<uintptr_t>(grad) % *sx)) return DSPARK_ERR_INVALID_ARG;
    if (grad == student && p->grad_stride != p->student_stride) return DSPARK_ERR_INVALID_ARG;
    a->V = p->V; a->n = t->n; a->target_V = t->target_V;
    a->c = c;
    const double inv_t = 1.0 / p->temperature, unit = 0.69314718055994530942 * c;
    a->inv_t = static_cast<float>(inv_t);
    a->inv_t_low = static_cast<float>(inv_t - static_cast<double>(a->inv_t));
    // logits of up to 2^128 over T, p of up to 256 in sum
    const int k = std::min(126, std::max(10, std::ilogb(unit) + 11));
    a->down = std::ldexp(1.f, -k);
    a->up_again = std::ldexp(1.f, k);
    a->unit2 = static_cast<float>(std::ldexp(unit, 1 - k));
    a->unit2_low = static_cast<float>(std::ldexp(unit, 1 - k) - static_cast<double>(a->unit2));
    a->s = student; a->s_stride = p->student_stride;
    a->g = const_cast<void*>(grad ? grad : student);         // the row's phase alone is read without a gradient
    a->g_stride = grad ? p->grad_stride : p->student_stride;
    a->ids = t->ids; a->tl = t->logits; a->lse = t->lse; a->t2d = t->t2d;
    a->weights = p->weights; a->row_status = p->row_status;
    // CTAs per row.  For one result a span streams through two buffers and may be as long as the row: a
    // CTA's latencies cost about what 40 KB do (2048 rows of 304 KB, loss alone: 101 us whole, 138 us in
    // quarters, 198 us in eighths).  Smaller spans while that makes no more than four CTAs per SM (150 such
    // rows: 25.7 us whole, 18.7 in halves, 16.2 in quarters, 21.7 in eighths), or two for both results.
    const int nvec = max_vectors(p->V, *sx);
    int C = 1;
    while (C < kMaxCluster && nvec >= C * 512 && static_cast<long long>(p->n_rows) * 2 * C <= (both ? 320 : 640)) C *= 2;
    // Both results: spans kept in one piece, of which an SM holds the more bytes the better (1024 rows
    // of 128256 bf16 in 4, 5, 6, 7, 8: 90, 85, 83, 88, 94 us for 188, 200, 209, 180, 157 KB; of 151936 in
    // 5 to 8: 108, 100, 108, 102 us for 178, 198, 170, 186).  kCtaSmem is a few hundred bytes more than a CTA takes now:
    // five sixths of 128256 would just fit an SM, and the rule, which counts four, goes in fifths.
    if (both)
        for (int c = C, most = 0; c <= kMaxCluster; ++c) {
            const int span = (nvec + c - 1) / c;
            if (c > C && span < 512) break;
            if (span > kDisSpan && c < kMaxCluster) continue;
            const int held = span * min(kDisCtas, kSmSmem / (16 * span + kCtaSmem));
            if (held >= most) {
                most = held;
                C = c;
            }
        }
    a->C = C;
    while ((1 << a->log_c) < C) ++a->log_c;
    a->span = a->piece = (nvec + C - 1) / C;
    a->np = 1;
    if (a->span > (both ? kDisSpan : kDisPiece)) {
        a->np = (a->span + kDisPiece - 1) / kDisPiece;
        a->piece = kDisPiece;
        a->log_slots = 1;
    }
    return DSPARK_OK;
}

template <int SX, int PASS>
dspark_status_t distill_launch(const DisArgs& a, int rows, void* stream) {
    const size_t smem = static_cast<size_t>(a.piece) * 16 << a.log_slots;
    auto kern = a.np == 1 ? distill_kernel<SX, PASS, true> : distill_kernel<SX, PASS, false>;
    // beyond what a launch gets unasked; the same for every call, as another thread's may come between
    if (smem > 32 * 1024 && cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 16 * kDisSpan) != cudaSuccess)
        return DSPARK_ERR_CUDA;
    const unsigned grid = static_cast<unsigned>(rows) * a.C;
    const cudaError_t e = launch_cluster(kern, grid, kRowThreads, a.C, smem, static_cast<cudaStream_t>(stream), a);
    return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

}  // namespace
}  // namespace dspark

using namespace dspark;

extern "C" {

dspark_status_t dspark_distill(const void* student, const dspark_teacher_t* teacher, const dspark_distill_params_t* params,
                               float* out_loss, float* out_saved, void* out_grad) {
    DisArgs a{};
    int sx = 0;
    if (const dspark_status_t st = distill_args(student, teacher, params, out_grad, out_grad != nullptr, &a, &sx); st != DSPARK_OK) return st;
    if (!out_loss || !params->row_status) return DSPARK_ERR_INVALID_ARG;
    a.loss = out_loss;
    a.saved_out = out_saved;
    if (out_grad)
        return sx == 2 ? distill_launch<2, kLoss | kGrad>(a, params->n_rows, params->stream)
                       : distill_launch<4, kLoss | kGrad>(a, params->n_rows, params->stream);
    return sx == 2 ? distill_launch<2, kLoss>(a, params->n_rows, params->stream)
                   : distill_launch<4, kLoss>(a, params->n_rows, params->stream);
}

dspark_status_t dspark_distill_backward(const void* student, const dspark_teacher_t* teacher,
                                        const dspark_distill_params_t* params, const float* saved, const float* grad_loss,
                                        void* out_grad) {
    DisArgs a{};
    int sx = 0;
    if (!out_grad || !saved) return DSPARK_ERR_INVALID_ARG;
    if (const dspark_status_t st = distill_args(student, teacher, params, out_grad, false, &a, &sx); st != DSPARK_OK) return st;
    a.saved = saved;
    a.up = grad_loss;
    return sx == 2 ? distill_launch<2, kGrad>(a, params->n_rows, params->stream)
                   : distill_launch<4, kGrad>(a, params->n_rows, params->stream);
}

}  // extern "C"
