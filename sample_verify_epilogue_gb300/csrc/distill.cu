// distill_kernel: the divergence of a student's softmax from a teacher known by its top logits,
// its gradient, or both in one launch; each row split over a cluster of C CTAs.
//
// With e_v = exp(s_v / T) up to a factor of the row, Z = sum e_v, R = sum of e_v outside the record's
// set S:
//   L = sum_S p_i (log p_i - log e_i + log Z) + p_r log(p_r Z / R)
//   dL/ds_v = (e_v a - p_v / T) in S, e_v b outside,  a = M / (Z T),  b = (M/Z - p_r/R) / T
// R is summed without the members of S rather than taken as Z less their sum, which cancels when
// they carry nearly all mass.
//
// Bound by bandwidth: s is read once and the gradient written once.  A CTA's span of the row
// comes to shared memory by bulk copies and stays there between the sum and the gradient, so that
// a call for both does not read the row twice.  While it arrives, one warp makes the teacher's
// probabilities from the record.  That warp then takes the span's members out: it notes their
// logits and puts -inf in their place, so that the two loops over the span know nothing of S; the
// members' gradients are written over afterwards.  (Longer spans go through the buffer in pieces,
// twice when both results are wanted; the second read is then from L2.)
//
// Sums that meet cancellation (of p, of p_i log p_i/e_i) are held in 64 bits, by one warp: this
// GPU's 64-bit rate is 1/64 of its 32-bit one.
#include <type_traits>

#include "vocab_rows.cuh"

namespace dspark {

namespace {

constexpr int kDisVec = 4;                                   // vectors a thread holds at a time
constexpr int kDisSpan = 4608;                               // vectors of a span kept in one piece at most
constexpr int kDisPiece = 2560;                              // vectors of a piece of a longer one
constexpr int kDisEntries = DSPARK_MAX_TOP_LOGITS / 32;      // record entries per lane

enum DistillPass : int { kLoss = 1, kGrad = 2 };

struct DisArgs {
    int V, n, log_c, target_V;                               // log_c: of the cluster's size
    int piece;                                               // vectors of the buffer
    float c;                                                 // log2(e) / T
    double inv_t;
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
};

struct __align__(16) DisPart {                               // what a CTA tells its cluster
    float m, rest, in;                                       // maximum; sums of e outside and inside S, by it
    int status;
    double cross;                                            // sum over its members of p_i (log p_i - log e_i)
    double pad;
};
constexpr unsigned kDisPartBytes = 24;

struct __align__(16) DisSmem {
    DisPart all[kMaxCluster];                                // written by the cluster's CTAs
    uint64_t bar, part_bar;
    int id[DSPARK_MAX_TOP_LOGITS];                           // draft ids of the row's record, -1: none
    float p[DSPARK_MAX_TOP_LOGITS];
    float lv[DSPARK_MAX_TOP_LOGITS];                         // log p; once taken out, the student's logit
    ExpSum es[kRowWarps];
    float psum, p_r, mass;                                   // sum of p, 1 - sum, their sum
    int status, any;
    float m, total, rest;                                    // the row's
};

// log(v), v > 0 normal: the exponent's part in 64 bits, logf of what is left in [0.75, 1.5).
__device__ __forceinline__ double log_split(float v) {
    const int e = (__float_as_int(v) - 0x3F400000) >> 23;
    return kLn2 * e + static_cast<double>(logf(__int_as_float(__float_as_int(v) - (e << 23))));
}

template <int SX>
__device__ __forceinline__ void store_vec(const VocabRow<SX>& g, int k, int i0, const uint4& w, bool same_phase) {
    constexpr int VE = 16 / SX;
    unsigned char* p = const_cast<unsigned char*>(g.p);
    if (same_phase && i0 >= 0 && i0 + VE <= g.V) {
        st_stream(p + static_cast<long long>(i0) * SX, w);
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

// The teacher's record of a row, by one warp: draft ids, probabilities and their logarithms.
struct Record {
    int id[kDisEntries];
    float t[kDisEntries], lse;
    __device__ __forceinline__ void load(const DisArgs& a, long long row);
    __device__ __forceinline__ void take(const DisArgs& a, DisSmem& s, long long row);
};
__device__ __forceinline__ void Record::load(const DisArgs& a, long long row) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int q = 0; q < kDisEntries; ++q) {
        const int e = lane + 32 * q;
        id[q] = e < a.n ? a.ids[row * a.n + e] : -1;
        t[q] = e < a.n ? a.tl[row * a.n + e] : 0.f;
    }
    lse = a.lse ? a.lse[row] : 0.f;
}
__device__ __forceinline__ void Record::take(const DisArgs& a, DisSmem& s, long long row) {
    const int lane = threadIdx.x & 31;
    int status = 0;
    float tmax = -INFINITY;
#pragma unroll
    for (int q = 0; q < kDisEntries; ++q) {
        if (id[q] < -1 || id[q] >= (a.t2d ? a.target_V : a.V)) { status = DSPARK_ROW_BAD_TEACHER; id[q] = -1; }
        if (a.t2d && id[q] >= 0) id[q] = a.t2d[id[q]];
    }
    bool any = false;
#pragma unroll
    for (int q = 0; q < kDisEntries; ++q) {
        if (id[q] < -1 || id[q] >= a.V || (id[q] >= 0 && !(t[q] < INFINITY))) { status = DSPARK_ROW_BAD_TEACHER; id[q] = -1; }
        if (id[q] >= 0) {
            any = true;
            tmax = fmaxf(tmax, t[q]);
        }
    }
    any = __any_sync(0xffffffffu, any);
    tmax = warp_max(tmax);
    if (!isfinite(lse) || (any && !a.lse && !(tmax > -INFINITY))) status = DSPARK_ROW_BAD_TEACHER;
    // log p: t / T is a product with 1/T in two parts, the first one exact inside the fma
    const float ih = static_cast<float>(a.inv_t), il = static_cast<float>(a.inv_t - static_cast<double>(ih));
    float lp[kDisEntries], p[kDisEntries];
    double sum = 0.0;
#pragma unroll
    for (int q = 0; q < kDisEntries; ++q) {
        lp[q] = -INFINITY;
        p[q] = 0.f;
        if (id[q] >= 0 && t[q] > -INFINITY) {
            lp[q] = a.lse ? fmaf(t[q], il, fmaf(t[q], ih, -lse)) : (t[q] - tmax) * ih;
            p[q] = expf(lp[q]);
        }
        if (32 * q < a.n) sum += p[q];
    }
    sum = warp_sum_d(sum);
    if (!(sum < INFINITY)) status = DSPARK_ROW_BAD_TEACHER;  // a log-sum-exp far below its logits
    float psum = static_cast<float>(sum), p_r = 0.f, mass = psum;
    if (a.lse) {
        if (sum < 1.0) { p_r = static_cast<float>(1.0 - sum); mass = 1.f; }
    } else if (any) {
        const float ls = logf(psum), inv = 1.f / psum;
#pragma unroll
        for (int q = 0; q < kDisEntries; ++q) {
            lp[q] -= ls;
            p[q] *= inv;
        }
        psum = mass = 1.f;
    }
#pragma unroll
    for (int q = 0; q < kDisEntries; ++q) {
        const int e = lane + 32 * q;
        if (e < a.n) {
            s.id[e] = id[q];
            s.p[e] = p[q];
            s.lv[e] = lp[q];
        }
    }
    status = __reduce_or_sync(0xffffffffu, static_cast<unsigned>(status));
    if (lane == 0) {
        s.psum = psum;
        s.p_r = p_r;
        s.mass = mass;
        s.status = status;
        s.any = any;
    }
}

template <int SX, int PASS>
__global__ void __launch_bounds__(kRowThreads, 5) distill_kernel(DisArgs a) {
    constexpr int VE = VocabRow<SX>::VE;
    constexpr bool kWantLoss = (PASS & kLoss) != 0, kWantGrad = (PASS & kGrad) != 0;
    __shared__ DisSmem s;
    extern __shared__ uint4 s_x[];                           // [piece]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = 1 << a.log_c, rank = static_cast<int>(blockIdx.x & (C - 1));
    const long long row = blockIdx.x >> a.log_c;
    const VocabRow<SX> x(a.s, row, a.s_stride, a.V);
    const VocabRow<SX> g(a.g, row, a.g_stride, a.V);
    const int k0 = x.nvec * rank >> a.log_c, k1 = x.nvec * (rank + 1) >> a.log_c;   // nvec * C < 2^31
    const bool same_phase = x.a0 == g.a0;
    const float w = a.weights ? a.weights[row] : 1.f;

    if (kWantLoss && C > 1) {                                // before a peer can push here
        if (tid == 0) {
            mbar_init(&s.part_bar, 1);
            fence_mbar_init();
            mbar_arrive_expect_tx(&s.part_bar, kDisPartBytes * C);
        }
        cluster_arrive();
    }
    // a row that is not reduced: loss, status and gradient; the same branch in every CTA of the row
    auto leave = [&](int status) {
        if (kWantLoss && rank == 0 && tid == 0) {
            a.loss[row] = status ? NAN : 0.f;
            a.row_status[row] = status;
            if (a.saved_out)
                for (int k = 0; k < 4; ++k) a.saved_out[4 * row + k] = 0.f;
        }
        if (kWantGrad)
            for (int k = k0 + tid; k < k1; k += kRowThreads) store_vec<SX>(g, k, x.first(k), make_uint4(0, 0, 0, 0), same_phase);
        if (kWantLoss && C > 1) cluster_wait();
    };
    // vectors [b, e) of the row into the buffer: whole ones by a bulk copy, the row's ragged first
    // and last by two threads of the warp that takes the members out
    auto fetch = [&](int b, int e) {
        const int wb = b + !x.whole(b), we = e - (e > wb && !x.whole(e - 1));
        if (tid == 0) {
            const unsigned bytes = we > wb ? 16u * static_cast<unsigned>(we - wb) : 0u;
            mbar_arrive_expect_tx(&s.bar, bytes);
            if (bytes) bulk_g2s(s_x + (wb - b), x.p + static_cast<long long>(x.first(wb)) * SX, bytes, &s.bar);
        }
        if (tid == 1 && wb > b) s_x[0] = load_vec<SX>(x, b, e);
        if (tid == 2 && we < e && we >= wb) s_x[we - b] = load_vec<SX>(x, we, e);
    };
    Record rec;
    if (warp == 0) rec.load(a, row);
    if (w == 0.f) {
        leave(0);
        return;
    }
    if (tid == 0) {
        mbar_init(&s.bar, 1);
        fence_mbar_init();
    }
    int b = k0, e = min(k1, k0 + a.piece);
    unsigned parity = 0;
    if (k0 < k1) fetch(b, e);
    if (warp == 0) rec.take(a, s, row);
    __syncthreads();
    bool late = false;
    if (!s.any || s.status) {
        if (warp == 0 && k0 < k1) late = !bar_wait(&s.bar, 0);
        late = __syncthreads_or(late);
        leave(s.status ? s.status : late ? DSPARK_ROW_INTERNAL : 0);
        return;
    }

    if (kWantLoss && C > 1) cluster_wait();                  // the peers' barriers stand

    ExpSum es{-INFINITY, 0.f};
    double cross = 0.0;
    int status = 0;
    const double ln_c = kLn2 * a.c;                          // the sums' own 1/T: c rounds log2(e)/T to fp32
    // One warp notes the logits of the members among the buffer's vectors [b, e) and puts -inf in
    // their place.  A repeated id finds the mark of the first (a NaN that is cleared at the end).
    auto take_members = [&](int b, int e) {
        __syncwarp();
        constexpr uint32_t kMark = SX == 2 ? 0x7FD5u : 0x7FD5AB31u;
        using Bits = std::conditional_t<SX == 2, unsigned short, unsigned>;
        Bits* const buf = reinterpret_cast<Bits*>(s_x);
        const int i0 = x.first(b), i_lo = max(0, i0), i_hi = min(a.V, x.first(e));
        for (int r0 = 0; r0 < a.n; r0 += 32) {
            const int r = r0 + lane, id = r < a.n ? s.id[r] : -1;
            const bool in = id >= i_lo && id < i_hi;
            if (!__any_sync(0xffffffffu, in)) continue;
            if (__popc(__match_any_sync(0xffffffffu, in ? id : -2 - lane)) > 1) status = DSPARK_ROW_BAD_TEACHER;
            if (in) {
                const uint32_t bits = buf[id - i0];
                if (bits == kMark) status = DSPARK_ROW_BAD_TEACHER;
                const float v = __uint_as_float(SX == 2 ? bits << 16 : bits), p = s.p[r];
                if (p > 0.f) cross += p * (s.lv[r] - v * ln_c);
                s.lv[r] = v;
            }
            __syncwarp();
            if (in) buf[id - i0] = static_cast<Bits>(kMark);
            __syncwarp();
        }
        for (int r = lane; r < a.n; r += 32) {
            const int id = s.id[r];
            if (id >= i_lo && id < i_hi) buf[id - i0] = static_cast<Bits>(ninf_bits<SX>());
        }
    };
    double row_cross = 0.0;
    int row_status = 0;
    if (kWantLoss) {
        while (true) {
            if (warp == 0 && k0 < k1) {                      // the others sleep at the barrier
                late |= !bar_wait(&s.bar, parity);
                take_members(b, e);
            }
            parity ^= 1;
            __syncthreads();
            int k = tid;
            for (; k + (kDisVec - 1) * kRowThreads < e - b; k += kDisVec * kRowThreads) {
                uint4 v[kDisVec];
#pragma unroll
                for (int u = 0; u < kDisVec; ++u) v[u] = s_x[k + u * kRowThreads];
                add_exps<SX>(es, v, vecs_max<SX>(v), a.c);
            }
            for (; k < e - b; k += kRowThreads) {
                const uint4 v[1] = {s_x[k]};
                add_exps<SX>(es, v, vecs_max<SX>(v), a.c);
            }
            if (e >= k1) break;
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncthreads();
            b = e;
            e = min(k1, b + a.piece);
            fetch(b, e);
        }
        es = warp_merge(es, a.c);
        if (lane == 0) s.es[warp] = es;
        __syncthreads();
        if (warp == 0) {                                     // the CTA's part, to every CTA of the row
            es = lane < kRowWarps ? s.es[lane] : ExpSum{-INFINITY, 0.f};
            const int i_lo = max(0, x.first(k0)), i_hi = min(a.V, x.first(k1));
            float m = es.m;
            for (int r = lane; r < a.n; r += 32)
                if (s.id[r] >= i_lo && s.id[r] < i_hi) m = fmaxf(m, s.lv[r]);
            m = key_to_f(__reduce_max_sync(0xffffffffu, fkey(m)));
            const ExpRef ref(m > -INFINITY ? m : 0.f, a.c);
            float in = 0.f;
            for (int r = lane; r < a.n; r += 32)
                if (s.id[r] >= i_lo && s.id[r] < i_hi) in += ref.of(s.lv[r]);   // NaN for NaN and +inf
            in = warp_sum(in);
            const float rest = warp_sum(m > -INFINITY ? es.sum * rebase(es.m, m, a.c) : es.sum);
            cross = warp_sum_d(cross);
            status = __reduce_or_sync(0xffffffffu, static_cast<unsigned>(status));
            if (late) status |= DSPARK_ROW_INTERNAL;
            if (C > 1) {
                if (lane < C) {
                    const unsigned to = peer_addr(&s.all[rank], lane), bar = peer_addr(&s.part_bar, lane);
                    peer_push128(to, bar, __float_as_uint(m), __float_as_uint(rest), __float_as_uint(in), static_cast<uint32_t>(status));
                    peer_push64(to + 16, bar, static_cast<unsigned long long>(__double_as_longlong(cross)));
                }
                late = !bar_wait(&s.part_bar, 0);
            } else if (lane == 0) {
                s.all[0] = DisPart{m, rest, in, status, cross, 0.0};
            }
            __syncwarp();
            // the row: every CTA joins the C parts alike
            DisPart o{-INFINITY, 0.f, 0.f, 0, 0.0, 0.0};
            if (lane < C) o = s.all[lane];
            m = key_to_f(__reduce_max_sync(0xffffffffu, fkey(o.m)));
            const float f = m > -INFINITY ? rebase(o.m, m, a.c) : 1.f;
            const float rest_r = warp_sum(lane < C ? o.rest * f : 0.f), total = rest_r + warp_sum(lane < C ? o.in * f : 0.f);
            row_status = __reduce_or_sync(0xffffffffu, static_cast<unsigned>(o.status));
            if (late) row_status |= DSPARK_ROW_INTERNAL;
            if (!row_status && !(total == total && m > -INFINITY)) row_status = DSPARK_ROW_NONFINITE;
            row_cross = o.cross;
            if (lane == 0) {
                s.m = m;
                s.total = row_status ? NAN : total;
                s.rest = rest_r;
            }
        }
        __syncthreads();
    }

    // ---- the gradient
    if (kWantGrad) {
        const float m = kWantLoss ? s.m : a.saved[4 * row], total = kWantLoss ? s.total : a.saved[4 * row + 1];
        const float rest = kWantLoss ? s.rest : a.saved[4 * row + 2];
        const bool ok = total > 0.f && m > -INFINITY;        // total is NaN for a row that cannot be normalised
        const float wt = (a.up ? w * a.up[row] : w) * static_cast<float>(a.inv_t);
        const float scale_in = wt * (s.mass / total);
        // (M R - p_r Z) / (Z R): the two products cancel where the student's tail is nearly right
        float scale_out = scale_in;
        if (s.p_r > 0.f && rest > 0.f) {
            const float z = s.p_r * total, ze = fmaf(s.p_r, total, -z);
            scale_out = wt * (((fmaf(s.mass, rest, -z) - ze) / rest) / total);
        }
        const ExpRef ref(m, a.c);
        // with a loss the last piece is in the buffer; the others, if any, come again
        const bool kept = kWantLoss && e - b == k1 - k0;
        if (kWantLoss && !kept) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncthreads();
            b = k0;
            e = min(k1, k0 + a.piece);
            if (k0 < k1) fetch(b, e);
        }
        bool lost = false;
        while (true) {
            if (!kept) {
                if (warp == 0 && k0 < k1) {
                    lost |= !bar_wait(&s.bar, parity);
                    if (!kWantLoss) take_members(b, e);
                }
                parity ^= 1;
                lost = __syncthreads_or(lost);
            }
            for (int k = b + tid; k < e; k += kRowThreads) {
                const uint4 v = s_x[k - b];
                uint4 o = make_uint4(0, 0, 0, 0);
                if (ok && !lost) {
                    float f[VE];
                    if (ref.whole) {
                        const unsigned long long c2 = pack2(a.c, a.c), r2 = pack2(-ref.r, -ref.r), s2 = pack2(scale_out, scale_out);
#pragma unroll
                        for (int h = 0; h < VE / 2; ++h) {
                            float lo, hi;
                            unpack2(fma2(pair_of<SX>(v, h), c2, r2), lo, hi);
                            unpack2(mul2(pack2(ex2_approx(lo), ex2_approx(hi)), s2), f[2 * h], f[2 * h + 1]);
                        }
                    } else {
#pragma unroll
                        for (int q = 0; q < VE; ++q) f[q] = ref.of(elem<SX>(v, q)) * scale_out;
                    }
                    if (SX == 2) o = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4 % VE], f[5 % VE]), pack_bf16(f[6 % VE], f[7 % VE]));
                    else o = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
                }
                store_vec<SX>(g, k, x.first(k), o, same_phase);
            }
            if (kept || e >= k1) break;
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncthreads();
            b = e;
            e = min(k1, b + a.piece);
            fetch(b, e);
        }
        __syncthreads();                                     // the members' gradients go over the span's
        if (warp == 0 && ok && !lost) {
            const int i_lo = max(0, x.first(k0)), i_hi = min(a.V, x.first(k1));
            for (int r = lane; r < a.n; r += 32) {
                const int id = s.id[r];
                if (id < i_lo || id >= i_hi) continue;
                const float v = fmaf(-s.p[r], wt, ref.of(s.lv[r]) * scale_in);
                unsigned char* p = const_cast<unsigned char*>(g.p);
                if (SX == 2) reinterpret_cast<unsigned short*>(p)[id] = static_cast<unsigned short>(to_bits<SX>(v));
                else reinterpret_cast<float*>(p)[id] = v;
            }
        }
    }
    if (kWantLoss && rank == 0 && warp == 0) {               // the loss, off the gradient's path
        row_cross = warp_sum_d(lane < C ? row_cross : 0.0);
        if (lane == 0) {
            const float m = s.m, total = s.total, rest = s.rest;
            const ExpRef ref(m, a.c);
            double loss = row_cross + s.psum * ((ref.whole ? kLn2 * ref.r : m * ln_c) + log_split(total));
            if (s.p_r > 0.f && rest > 0.f) loss += s.p_r * logf(s.p_r * (total / rest));
            a.loss[row] = row_status ? NAN : static_cast<float>(w * loss);
            a.row_status[row] = row_status;
            if (a.saved_out) {
                a.saved_out[4 * row] = m;
                a.saved_out[4 * row + 1] = total;
                a.saved_out[4 * row + 2] = rest;
                a.saved_out[4 * row + 3] = 0.f;
            }
        }
    }
}

// Checks shared by the two entry points; on success *a and *sx are set.
dspark_status_t distill_args(const void* student, const dspark_teacher_t* t, const dspark_distill_params_t* p, const void* grad,
                             DisArgs* a, int* sx) {
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
    a->c = c; a->inv_t = 1.0 / p->temperature;
    a->s = student; a->s_stride = p->student_stride;
    a->g = const_cast<void*>(grad ? grad : student);         // the row's phase alone is read without a gradient
    a->g_stride = grad ? p->grad_stride : p->student_stride;
    a->ids = t->ids; a->tl = t->logits; a->lse = t->lse; a->t2d = t->t2d;
    a->weights = p->weights; a->row_status = p->row_status;
    // CTAs per row: spans of at most 72 KB (three CTAs to an SM), and smaller ones while the rows alone
    // do not make two CTAs per SM.  2048 rows of 64 KB, loss then gradient: 114 us whole, 139 us in
    // halves, 227 us in quarters: a CTA's latencies cost more than its share of the row.
    const int nvec = max_vectors(p->V, *sx);
    int cluster = 1;
    while (cluster < kMaxCluster && (nvec > cluster * kDisSpan ||
                                        (nvec >= cluster * 512 && static_cast<long long>(p->n_rows) * cluster < 304)))
        cluster *= 2;
    for (a->log_c = 0; (1 << a->log_c) < cluster;) ++a->log_c;
    // a longer span comes in pieces of 40 KB
    a->piece = nvec / cluster + 1;
    if (a->piece > kDisSpan) a->piece = kDisPiece;
    return DSPARK_OK;
}

template <int SX, int PASS>
dspark_status_t distill_launch(const DisArgs& a, int rows, void* stream) {
    const size_t smem = static_cast<size_t>(a.piece) * 16;
    if (smem > 32 * 1024 &&                                  // beyond what a launch gets unasked
        cudaFuncSetAttribute(distill_kernel<SX, PASS>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
        return DSPARK_ERR_CUDA;
    const unsigned grid = static_cast<unsigned>(rows) << a.log_c;
    const cudaError_t e = launch_cluster(distill_kernel<SX, PASS>, grid, 1 << a.log_c, smem, static_cast<cudaStream_t>(stream), a);
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
    if (const dspark_status_t st = distill_args(student, teacher, params, out_grad, &a, &sx); st != DSPARK_OK) return st;
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
    if (const dspark_status_t st = distill_args(student, teacher, params, out_grad, &a, &sx); st != DSPARK_OK) return st;
    a.saved = saved;
    a.up = grad_loss;
    return sx == 2 ? distill_launch<2, kGrad>(a, params->n_rows, params->stream)
                   : distill_launch<4, kGrad>(a, params->n_rows, params->stream);
}

}  // extern "C"
