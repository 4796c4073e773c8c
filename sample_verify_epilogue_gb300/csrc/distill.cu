// distill_kernel: the divergence of a student's softmax from a teacher known by its top logits,
// its gradient, or both in one launch; each row split over a cluster of CTAs.
//
// With e_v = 2^((s_v - m) log2(e)/T), Z = sum e_v, R = sum of e_v outside the record's set S:
//   L = sum_S p_i (log p_i - s_i/T + m/T + log Z) + p_r log(p_r Z / R)
//   dL/ds_v = (e_v a - p_v / T) in S, e_v b outside,  a = M / (Z T),  b = (M/Z - p_r/R) / T
// so the row is needed twice: once for Z and R, once for the gradient.  R is summed without the
// members of S rather than taken as Z less their sum, which cancels when they carry nearly
// all mass.  A bit per 16-byte vector says whether the vector holds a member; only those vectors
// (at most n of a row) look their lanes up in the CTA's part of the record.
//
// Bound by bandwidth: s is read once, the gradient written once.  When both come from one call
// the second read of a row follows the first at once and finds it in L2: the cluster's size
// bounds the rows in flight.  Teacher probabilities are made by every CTA of the row, one thread
// for each of the record's n entries; the sums that meet cancellation (of p, of p_i log p_i/q_i)
// are held in 64 bits, by one warp: this GPU's 64-bit rate is 1/64 of its 32-bit one.
#include "vocab_rows.cuh"

namespace dspark {

namespace {

constexpr int kDisVec = 4;
constexpr int kDisBatch = kDisVec * kRowThreads;
static_assert(DSPARK_MAX_TOP_LOGITS <= kRowThreads, "one record entry per thread");

enum DistillPass : int { kLoss = 1, kGrad = 2 };

struct DisArgs {
    int V, n, cluster, target_V, words;                      // words: of the per-vector bitmap
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

struct DisPart {                                             // what a CTA tells its cluster
    float m, rest, in;                                       // maximum; sums of e relative to it
    int pad;
    double cross;                                            // sum over its members of p_i (log p_i - s_i/T)
};

struct __align__(16) DisSmem {
    DisPart part;
    alignas(16) int id[DSPARK_MAX_TOP_LOGITS];                     // draft ids of the row's record, -1: none
    float p[DSPARK_MAX_TOP_LOGITS];                          // its probabilities (renormalised later where wanted)
    int m_id[DSPARK_MAX_TOP_LOGITS];                         // members inside this CTA's span:
    float m_p[DSPARK_MAX_TOP_LOGITS];                        //   probability, its logarithm
    float m_lp[DSPARK_MAX_TOP_LOGITS];
    int wmem[kRowWarps];
    float wmax[kRowWarps];
    ExpSum es[kRowWarps];
    double psum;                                             // sum of p
    float m, total, rest;                                    // the row's
};

__device__ __forceinline__ int find_member(const DisSmem& s, int n_mem, int i) {
    for (int e = 0; e < n_mem; ++e)
        if (s.m_id[e] == i) return e;
    return -1;
}

// log(v), v > 0 normal: the exponent's part in 64 bits, logf of what is left in [0.75, 1.5).
__device__ __forceinline__ double log_split(float v) {
    const int e = (__float_as_int(v) - 0x3F400000) >> 23;
    return kLn2 * e + static_cast<double>(logf(__int_as_float(__float_as_int(v) - (e << 23))));
}

template <int SX>
__device__ __forceinline__ void store_vec(const VocabRow<SX>& g, int i0, const float (&v)[16 / SX], bool vec) {
    constexpr int VE = 16 / SX;
    unsigned char* p = const_cast<unsigned char*>(g.p);
    if (vec) {
        uint4 w;
        if (SX == 2) w = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4 % VE], v[5 % VE]), pack_bf16(v[6 % VE], v[7 % VE]));
        else w = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
        st_stream(p + static_cast<long long>(i0) * SX, w);
        return;
    }
#pragma unroll
    for (int q = 0; q < VE; ++q) {
        const int i = i0 + q;
        if (i < 0 || i >= g.V) continue;
        if (SX == 2) reinterpret_cast<unsigned short*>(p)[i] = static_cast<unsigned short>(to_bits<SX>(v[q]));
        else reinterpret_cast<float*>(p)[i] = v[q];
    }
}

template <int SX, int PASS>
__global__ void __launch_bounds__(kRowThreads) distill_kernel(DisArgs a) {
    constexpr int VE = VocabRow<SX>::VE;
    constexpr bool kWantLoss = (PASS & kLoss) != 0, kWantGrad = (PASS & kGrad) != 0;
    __shared__ DisSmem s;
    extern __shared__ unsigned s_bits[];                     // [words]: bit k - k0 of vector k
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = a.cluster, rank = static_cast<int>(blockIdx.x % C);
    const long long row = blockIdx.x / C;
    const VocabRow<SX> x(a.s, row, a.s_stride, a.V);
    const VocabRow<SX> g(a.g, row, a.g_stride, a.V);
    const int k0 = static_cast<int>(static_cast<long long>(x.nvec) * rank / C);
    const int k1 = static_cast<int>(static_cast<long long>(x.nvec) * (rank + 1) / C);
    const int i_lo = max(0, x.first(k0)), i_hi = min(a.V, x.first(k1));
    const bool same_phase = x.a0 == g.a0;

    // gradient of a row that has none
    auto zero_grad = [&]() {
        const float zero[VE] = {};
        for (int k = k0 + tid; k < k1; k += kRowThreads) store_vec<SX>(g, x.first(k), zero, same_phase && x.whole(k));
    };
    // loss and status of a row that is not reduced; the same branch in every CTA of the row
    auto leave = [&](int status) {
        if (kWantLoss && rank == 0 && tid == 0) {
            a.loss[row] = status ? NAN : 0.f;
            a.row_status[row] = status;
            if (a.saved_out)
                for (int k = 0; k < 4; ++k) a.saved_out[4 * row + k] = 0.f;
        }
        if (kWantGrad) zero_grad();
    };

    // ---- the teacher's record: draft ids, probabilities, the CTA's members
    const float w = a.weights ? a.weights[row] : 1.f;
    int id = tid < a.n ? a.ids[row * a.n + tid] : -1;
    float t = tid < a.n ? a.tl[row * a.n + tid] : 0.f;
    if (w == 0.f) {
        leave(0);
        return;
    }
    uint4 nxt[kDisVec];
    if (kWantLoss) {
#pragma unroll
        for (int u = 0; u < kDisVec; ++u) nxt[u] = load_vec<SX>(x, k0 + u * kRowThreads + tid, k1);
    }
    int bad = id < -1 || id >= (a.t2d ? a.target_V : a.V);
    if (bad) id = -1;
    if (a.t2d && id >= 0) {
        id = a.t2d[id];
        if (id < -1 || id >= a.V) { bad = 1; id = -1; }
    }
    if (id >= 0 && !(t < INFINITY)) { bad = 1; id = -1; }
    s.id[tid] = id;
    for (int i = tid; i < a.words; i += kRowThreads) s_bits[i] = 0u;
    float tmax = id >= 0 ? t : -INFINITY;
    tmax = warp_max(tmax);
    if (lane == 0) s.wmax[warp] = tmax;
    const int any = __syncthreads_or(id >= 0);
#pragma unroll
    for (int k = 0; k < kRowWarps; ++k) tmax = fmaxf(tmax, s.wmax[k]);
    if (id >= 0) {                                           // a repeated id
        int same = 0;
        for (int e = 0; e < a.n; e += 4) {
            const int4 o = *reinterpret_cast<const int4*>(&s.id[e]);
            same += (o.x == id) + (o.y == id) + (o.z == id) + (o.w == id);
        }
        bad |= same != 1;
    }
    // log p: the product t / T is exact inside the fma but for the rounding of 1 / T, put back
    const float ih = static_cast<float>(a.inv_t), il = static_cast<float>(a.inv_t - static_cast<double>(ih));
    float logp = -INFINITY;
    if (id >= 0 && t > -INFINITY) {
        if (a.lse) logp = fmaf(t, il, fmaf(t, ih, -a.lse[row]));
        else logp = (t - tmax) * ih;
    }
    if (a.lse && !isfinite(a.lse[row])) bad = 1;
    if (!a.lse && any && !(tmax > -INFINITY)) bad = 1;       // nothing above -inf in the record
    float p = id >= 0 ? expf(logp) : 0.f;
    if (!(p < INFINITY)) bad = 1;                            // a log-sum-exp far below its logits
    s.p[tid] = p;
    bad = __syncthreads_or(bad);
    if (bad || !any) {
        leave(bad ? DSPARK_ROW_BAD_TEACHER : 0);
        return;
    }
    if (warp == 0) {
        double ps = 0.0;
        for (int e = lane; e < a.n; e += 32) ps += s.p[e];
        ps = warp_sum_d(ps);
        if (lane == 0) s.psum = ps;
    }
    // the members of this span, in the record's order
    const bool here = id >= i_lo && id < i_hi;
    const unsigned vote = __ballot_sync(0xffffffffu, here);
    if (lane == 0) s.wmem[warp] = __popc(vote);
    if (here) {
        const int k = (id + x.a0) / VE - k0;
        atomicOr(&s_bits[k >> 5], 1u << (k & 31));
    }
    __syncthreads();
    int mine = __popc(vote & ((1u << lane) - 1u)), n_mem = 0;
#pragma unroll
    for (int k = 0; k < kRowWarps; ++k) {
        if (k < warp) mine += s.wmem[k];
        n_mem += s.wmem[k];
    }
    // psum, p_r, mass = psum + p_r
    float psum = static_cast<float>(s.psum), p_r = 0.f, mass = 1.f;
    if (a.lse) {
        p_r = s.psum < 1.0 ? static_cast<float>(1.0 - s.psum) : 0.f;
        mass = s.psum < 1.0 ? 1.f : psum;
    } else {
        logp -= logf(psum);
        p /= psum;
        psum = 1.f;
    }
    if (here) {
        s.m_id[mine] = id;
        s.m_p[mine] = p;
        s.m_lp[mine] = logp;
    }
    __syncthreads();

    // ---- Z and R
    if (kWantLoss) {
        ExpSum es{-INFINITY, 0.f};
        uint4 cur[kDisVec];
        for (int b0 = k0; b0 < k1; b0 += kDisBatch) {
#pragma unroll
            for (int u = 0; u < kDisVec; ++u) cur[u] = nxt[u];
            if (b0 + kDisBatch < k1) {
#pragma unroll
                for (int u = 0; u < kDisVec; ++u) nxt[u] = load_vec<SX>(x, b0 + kDisBatch + u * kRowThreads + tid, k1);
            }
            float bm = -INFINITY;
#pragma unroll
            for (int u = 0; u < kDisVec; ++u) {
                const int k = b0 + u * kRowThreads + tid, kb = k - k0;
                if (k < k1 && ((s_bits[kb >> 5] >> (kb & 31)) & 1u)) {
                    const int i0 = x.first(k);
#pragma unroll
                    for (int q = 0; q < VE; ++q)
                        if (find_member(s, n_mem, i0 + q) >= 0) put_bits<SX>(cur[u], q, ninf_bits<SX>());
                }
                bm = fmaxf(bm, vec_max<SX>(cur[u]));
            }
            if (bm > es.m) {
                es.sum *= rebase(es.m, bm, a.c);
                es.m = bm;
            }
            const float ref = es.m > -INFINITY ? es.m : 0.f;
#pragma unroll
            for (int u = 0; u < kDisVec; ++u)
#pragma unroll
                for (int q = 0; q < VE; ++q) es.sum += exp_of(elem<SX>(cur[u], q), ref, a.c);
        }
        for (int o = 16; o; o >>= 1)
            es = merge(es, ExpSum{__shfl_xor_sync(0xffffffffu, es.m, o), __shfl_xor_sync(0xffffffffu, es.sum, o)}, a.c);
        if (lane == 0) s.es[warp] = es;
        __syncthreads();
        if (warp == 0) {                                     // the members, and the CTA's part
            es = s.es[lane & (kRowWarps - 1)];
            for (int o = kRowWarps / 2; o; o >>= 1)
                es = merge(es, ExpSum{__shfl_xor_sync(0xffffffffu, es.m, o), __shfl_xor_sync(0xffffffffu, es.sum, o)}, a.c);
            float v[DSPARK_MAX_TOP_LOGITS / 32], m = es.m;
#pragma unroll
            for (int q = 0; q < DSPARK_MAX_TOP_LOGITS / 32; ++q) {
                const int e = lane + 32 * q;
                v[q] = e < n_mem ? load_logit<SX>(x, s.m_id[e]) : -INFINITY;
                m = fmaxf(m, v[q]);
            }
            m = warp_max(m);
            const float ref = m > -INFINITY ? m : 0.f;
            float in = 0.f;
            double cross = 0.0;
#pragma unroll
            for (int q = 0; q < DSPARK_MAX_TOP_LOGITS / 32; ++q) {
                const int e = lane + 32 * q;
                if (e >= n_mem) break;
                in += exp_of(v[q], ref, a.c);                // NaN for NaN and +inf
                const float pe = s.m_p[e];
                // the student's exponent as the sums have it: c is log2(e)/T rounded to fp32
                if (pe > 0.f) cross += pe * (s.m_lp[e] - static_cast<double>(v[q]) * (kLn2 * a.c));
            }
            in = warp_sum(in);
            cross = warp_sum_d(cross);
            if (lane == 0) {
                s.part.m = m;
                s.part.rest = m > -INFINITY ? es.sum * rebase(es.m, m, a.c) : es.sum;
                s.part.in = in;
                s.part.cross = cross;
            }
        }
        if (C > 1) {
            __syncthreads();
            cluster_arrive();
            cluster_wait();
        }
        if (warp == 0) {                                     // the row: every CTA joins the C parts alike
            __syncwarp();
            DisPart o{-INFINITY, 0.f, 0.f, 0, 0.0};
            if (C > 1) {
                if (lane < C) {
                    const unsigned from = peer_addr(&s.part, lane);
                    o.m = __uint_as_float(peer_ld32(from));
                    o.rest = __uint_as_float(peer_ld32(from + 4));
                    o.in = __uint_as_float(peer_ld32(from + 8));
                    if (rank == 0) o.cross = __longlong_as_double(static_cast<long long>(peer_ld64(from + 16)));
                }
            } else if (lane == 0) {
                o = s.part;
            }
            const float m = warp_max(o.m);
            const float f = m > -INFINITY ? rebase(o.m, m, a.c) : 1.f;
            const float rest = warp_sum(o.rest * f), total = rest + warp_sum(o.in * f);
            if (lane == 0) { s.m = m; s.total = total; s.rest = rest; }
            if (rank == 0) {
                const double cross = warp_sum_d(o.cross);
                if (lane == 0) {
                    const bool ok = total == total && m > -INFINITY;
                    double loss = cross + psum * (m * (kLn2 * a.c) + log_split(total));
                    if (p_r > 0.f && rest > 0.f) loss += p_r * logf(p_r * (total / rest));
                    a.loss[row] = ok ? static_cast<float>(w * loss) : NAN;
                    a.row_status[row] = ok ? 0 : DSPARK_ROW_NONFINITE;
                    if (a.saved_out) {
                        a.saved_out[4 * row] = m;
                        a.saved_out[4 * row + 1] = total;
                        a.saved_out[4 * row + 2] = rest;
                        a.saved_out[4 * row + 3] = 0.f;
                    }
                }
            }
        }
        if (kWantGrad) __syncthreads();
        if (C > 1) cluster_arrive();                         // waited for at the end: peers have read this CTA's part
    }

    // ---- the gradient
    if (kWantGrad) {
        const float m = kWantLoss ? s.m : a.saved[4 * row], total = kWantLoss ? s.total : a.saved[4 * row + 1];
        const float rest = kWantLoss ? s.rest : a.saved[4 * row + 2];
        if (total > 0.f && m > -INFINITY) {                  // total is NaN for a row that cannot be normalised
            const float wt = (a.up ? w * a.up[row] : w) * ih;
            const float scale_in = wt * (mass / total);
            // (M R - p_r Z) / (Z R): the two products cancel where the student's tail is nearly right
            float scale_out = scale_in;
            if (p_r > 0.f && rest > 0.f) {
                const float z = p_r * total, ze = fmaf(p_r, total, -z);
                scale_out = wt * (((fmaf(mass, rest, -z) - ze) / rest) / total);
            }
            for (int b0 = k0; b0 < k1; b0 += kDisBatch) {
                uint4 v[kDisVec];
#pragma unroll
                for (int u = 0; u < kDisVec; ++u) v[u] = load_vec<SX>(x, b0 + u * kRowThreads + tid, k1);
#pragma unroll
                for (int u = 0; u < kDisVec; ++u) {
                    const int k = b0 + u * kRowThreads + tid, kb = k - k0;
                    if (k >= k1) break;
                    const int i0 = x.first(k);
                    float o[VE];
#pragma unroll
                    for (int q = 0; q < VE; ++q) o[q] = exp_of(elem<SX>(v[u], q), m, a.c) * scale_out;
                    if ((s_bits[kb >> 5] >> (kb & 31)) & 1u) {
#pragma unroll
                        for (int q = 0; q < VE; ++q) {
                            const int e = find_member(s, n_mem, i0 + q);
                            if (e >= 0) o[q] = fmaf(-s.m_p[e], wt, exp_of(elem<SX>(v[u], q), m, a.c) * scale_in);
                        }
                    }
                    store_vec<SX>(g, i0, o, same_phase && x.whole(k));
                }
            }
        } else {
            zero_grad();
        }
    }
    if (kWantLoss && C > 1) cluster_wait();
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
    // CTAs per row: one batch of vectors each at least
    const int nvec = max_vectors(p->V, *sx);
    a->cluster = 1;
    while (a->cluster < kMaxCluster && nvec >= 2 * a->cluster * kDisBatch) a->cluster *= 2;
    a->words = (nvec / a->cluster + 1 + 31) / 32;
    return DSPARK_OK;
}

template <int SX, int PASS>
dspark_status_t distill_launch(const DisArgs& a, int rows, void* stream) {
    const size_t smem = static_cast<size_t>(a.words) * sizeof(unsigned);
    if (smem > 32 * 1024 &&                                  // beyond what a launch gets unasked
        cudaFuncSetAttribute(distill_kernel<SX, PASS>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
        return DSPARK_ERR_CUDA;
    const unsigned grid = static_cast<unsigned>(rows) * static_cast<unsigned>(a.cluster);
    const cudaError_t e = launch_cluster(distill_kernel<SX, PASS>, grid, a.cluster, smem, static_cast<cudaStream_t>(stream), a);
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
