// top_logits_kernel: the n largest logits of every row (value descending, id ascending among
// equals) and log sum exp(x / T), one launch, each row split over a cluster of C CTAs.
//
// One pass over the row, bound by bandwidth: while a CTA streams its span, each thread keeps the sum
// of its exponentials and the maxima of the groups of vectors it sees, and nothing else.
// The row's 512 group maxima then give a threshold: their n-th largest is reached by at least n
// logits, and by few more (G groups, n of them at or above: about -G ln(1 - n/G) logits, 69 for
// n = 64), so
//   1. group maxima go to shared memory; every CTA reads the row's 512 through distributed shared
//      memory and finds their n-th largest by bisection on the upper 16 bits of its key (one warp);
//   2. only the threads whose maximum reaches it read their vectors again (L2) and list the
//      logits that do;
//   3. every CTA reads the row's whole list and ranks its own entries in it: the rank is the place
//      in the record.
// Rows whose list would be too long (equal values, few distinct values, values bunched in one
// group) take an exact path: bisection on the value over counts of the whole row, from that
// threshold up to the maximum; then the logits above the n-th value, and in id order as many equal
// to it as are wanted.
#include "vocab_rows.cuh"

namespace dspark {

namespace {

constexpr int kTopVec = 4;
constexpr int kTopBatch = kTopVec * kRowThreads;             // vectors per batch
constexpr int kTopGroups = 512;                              // of a row, whatever its cluster
constexpr int kTopOwn = 2 * DSPARK_MAX_TOP_LOGITS;           // entries a CTA lists at most
constexpr int kTopAll = 1024;                                // entries of a row on the short path
constexpr int kTopBuf = DSPARK_MAX_TOP_LOGITS * (kMaxCluster + 1);   // ... on the exact path: < n above, n equal per CTA

// (order-preserving value key, id reversed), ids below 2^24.
__device__ __forceinline__ unsigned long long top_key(float v, int id) { return ckey(v, id); }

struct TopArgs {
    int V, n, cluster;
    float c;                                                 // log2(e) / T
    double inv_t;
    long long stride;
    const void* x;
    float* values;
    int* ids;
    float* lse;
    int* row_status;
};

struct __align__(16) TopSmem {
    unsigned long long own[kTopOwn];
    unsigned long long all[kTopBuf];
    unsigned short gmax[kTopGroups];                         // this CTA's 512/C group maxima: upper halves of their keys
    ExpSum es[kRowWarps];
    ExpSum part;                                             // this CTA's sum
    int n;                                                   // entries listed (passes kTopOwn when they do not fit)
    int n_all;                                               // -1: the row takes the exact path
    int cnt;                                                 // exact path: this CTA's count
    int wcnt[kRowWarps];
    unsigned th;                                             // threshold key
    ExpSum row;
};

__device__ __forceinline__ float key_floor(unsigned k) {     // value of a key, never -inf
    return fmaxf(key_to_f(k), -3.402823466e38f);
}

// Largest k with at least n of the warp's 32*Q keys >= k, on 16-bit keys; 0 when fewer are set.
template <int Q>
__device__ unsigned warp_nth_key16(const unsigned (&key)[Q], int n) {
    unsigned lo = 0;
    for (int bit = 15; bit >= 0; --bit) {
        const unsigned mid = lo | (1u << bit);
        int c = 0;
#pragma unroll
        for (int q = 0; q < Q; ++q) c += key[q] >= mid;
        if (__reduce_add_sync(0xffffffffu, c) >= n) lo = mid;
    }
    return lo;
}

// Barrier of the cluster, or of the block when the row has one CTA.
__device__ __forceinline__ void row_sync(int C) {
    if (C > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
}

template <int SX>
__global__ void __launch_bounds__(kRowThreads, 4) top_logits_kernel(TopArgs a) {
    constexpr int VE = VocabRow<SX>::VE;
    __shared__ TopSmem s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = a.cluster, rank = static_cast<int>(blockIdx.x % C);
    const long long row = blockIdx.x / C;
    const VocabRow<SX> x(a.x, row, a.stride, a.V);
    const int k0 = static_cast<int>(static_cast<long long>(x.nvec) * rank / C);
    const int k1 = static_cast<int>(static_cast<long long>(x.nvec) * (rank + 1) / C);
    if (tid == 0) s.n = 0;

    // ---- the stream
    RunSum run;
    float g[2] = {-INFINITY, -INFINITY};                     // maxima of the thread's even and odd vectors
    {
        uint4 cur[kTopVec], nxt[kTopVec];
#pragma unroll
        for (int u = 0; u < kTopVec; ++u) nxt[u] = load_vec<SX>(x, k0 + u * kRowThreads + tid, k1);
        for (int base = k0; base < k1; base += kTopBatch) {
#pragma unroll
            for (int u = 0; u < kTopVec; ++u) cur[u] = nxt[u];
            if (base + kTopBatch < k1) {
#pragma unroll
                for (int u = 0; u < kTopVec; ++u) nxt[u] = load_vec<SX>(x, base + kTopBatch + u * kRowThreads + tid, k1);
            }
            float bm[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int u = 0; u < kTopVec; ++u) bm[u & 1] = fmaxf(bm[u & 1], vec_max<SX>(cur[u]));
            add_exps<SX>(run, cur, fmaxf(bm[0], bm[1]), a.c);
            g[0] = fmaxf(g[0], bm[0]);
            g[1] = fmaxf(g[1], bm[1]);
        }
    }
    const float tmax = fmaxf(g[0], g[1]);
    ExpSum es = run.get();

    // ---- group maxima: 512/C of this CTA; a group is a thread's half, a thread, or 2 or 4 threads
    {
        float gm = tmax;
        if (C == 1) {
            s.gmax[tid] = static_cast<unsigned short>(fkey(g[0]) >> 16);
            s.gmax[tid + kRowThreads] = static_cast<unsigned short>(fkey(g[1]) >> 16);
        } else {
            if (C >= 4) gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, 1));
            if (C >= 8) gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, 2));
            const int per = C / 2;                           // threads of a group
            if (tid % per == 0) s.gmax[tid / per] = static_cast<unsigned short>(fkey(gm) >> 16);
        }
        for (int o = 16; o; o >>= 1)
            es = merge(es, ExpSum{__shfl_xor_sync(0xffffffffu, es.m, o), __shfl_xor_sync(0xffffffffu, es.sum, o)}, a.c);
        if (lane == 0) s.es[warp] = es;
        __syncthreads();
        if (warp == 0) {
            es = s.es[lane & (kRowWarps - 1)];
            for (int o = kRowWarps / 2; o; o >>= 1)
                es = merge(es, ExpSum{__shfl_xor_sync(0xffffffffu, es.m, o), __shfl_xor_sync(0xffffffffu, es.sum, o)}, a.c);
            if (lane == 0) s.part = es;
        }
    }
    row_sync(C);

    // ---- threshold, and the row's sum
    if (warp == 0) {
        unsigned key[kTopGroups / 32];
        if (C > 1) {
            // two 16-bit maxima per word; CTA p has 256/C words
            const int per = kTopGroups / 2 / C;
#pragma unroll
            for (int q = 0; q < kTopGroups / 64; ++q) {
                const int w = q * 32 + lane;
                const unsigned v = peer_ld32(peer_addr(reinterpret_cast<const unsigned*>(s.gmax) + w % per, w / per));
                key[2 * q] = v & 0xFFFFu;
                key[2 * q + 1] = v >> 16;
            }
            es = ExpSum{-INFINITY, 0.f};
            if (lane < C) {
                const unsigned from = peer_addr(&s.part, lane);
                es = ExpSum{__uint_as_float(peer_ld32(from)), __uint_as_float(peer_ld32(from + 4))};
            }
            for (int o = kMaxCluster / 2; o; o >>= 1)
                es = merge(es, ExpSum{__shfl_xor_sync(0xffffffffu, es.m, o), __shfl_xor_sync(0xffffffffu, es.sum, o)}, a.c);
        } else {
#pragma unroll
            for (int q = 0; q < kTopGroups / 32; ++q) key[q] = s.gmax[q * 32 + lane];
        }
        const unsigned th = warp_nth_key16(key, a.n) << 16;
        if (lane == 0) {
            s.th = th;
            s.row = es;
        }
    }
    __syncthreads();
    es = s.row;
    // a row with NaN or +inf has a NaN sum, one with nothing above -inf a maximum of -inf
    const bool ok = es.sum == es.sum && es.m > -INFINITY;

    // ---- list the logits that reach the threshold: flagged threads' vectors, a warp to a thread
    const float th = key_floor(s.th);
    if (ok) {
        unsigned flagged = __ballot_sync(0xffffffffu, tmax >= th);
        while (flagged) {
            const int t = warp * 32 + __ffs(flagged) - 1;
            flagged &= flagged - 1;
            for (int k = k0 + t + lane * kRowThreads; k < k1; k += 32 * kRowThreads) {
                const uint4 w = load_vec<SX>(x, k, k1);
                if (!(vec_max<SX>(w) >= th)) continue;
#pragma unroll
                for (int q = 0; q < VE; ++q) {
                    const float v = elem<SX>(w, q);
                    if (v >= th) {
                        const int at = atomicAdd(&s.n, 1);
                        if (at < kTopOwn) s.own[at] = top_key(v, x.first(k) + q);
                    }
                }
            }
            if (*reinterpret_cast<volatile int*>(&s.n) > kTopOwn) break;   // the exact path counts anew
        }
    }
    row_sync(C);

    // ---- the row's list
    const long long out = row * a.n;
    int total = 0, before = 0, mine = 0;
    auto gather = [&](int cap) {                             // false: a CTA's entries or all of them are too many
        const int np = C > 1 ? (lane < C ? static_cast<int>(peer_ld32(peer_addr(&s.n, lane))) : 0) : (lane == 0 ? s.n : 0);
        int incl = np;
#pragma unroll
        for (int o = 1; o < kMaxCluster; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        total = __shfl_sync(0xffffffffu, incl, kMaxCluster - 1);
        mine = __shfl_sync(0xffffffffu, np, rank);
        before = __shfl_sync(0xffffffffu, incl, rank) - mine;
        if (__any_sync(0xffffffffu, np > kTopOwn) || total > cap) return false;
        for (int i0 = warp * 32; i0 < total; i0 += kRowThreads) {
            const int i = i0 + lane;
            int p = 0, start = 0;                            // entry i is number i - start of CTA p
#pragma unroll
            for (int t = 0; t < kMaxCluster - 1; ++t) {
                const int end = __shfl_sync(0xffffffffu, incl, t);
                if (i >= end) { p = t + 1; start = end; }
            }
            if (i < total) s.all[i] = C > 1 ? peer_ld64(peer_addr(&s.own[i - start], p)) : s.own[i];
        }
        return true;
    };
    if (ok && !gather(kTopAll)) {
        // exact path (the same for every CTA of the row): v, the n-th largest value, is the largest
        // with at least n logits at or above it
        row_sync(C);                                         // the counts have been read
        unsigned lo = fkey(th), hi = fkey(es.m);
        while (lo < hi) {
            const unsigned mid = lo + ((hi - lo) >> 1) + 1;
            const float v = key_to_f(mid);
            int c = 0;
            for (int k = k0 + tid; k < k1; k += kRowThreads) {
                const uint4 w = load_vec<SX>(x, k, k1);
#pragma unroll
                for (int q = 0; q < VE; ++q) c += elem<SX>(w, q) >= v;
            }
            c = __reduce_add_sync(0xffffffffu, c);
            if (lane == 0) s.wcnt[warp] = c;
            __syncthreads();
            if (tid == 0) {
                int t = 0;
                for (int w = 0; w < kRowWarps; ++w) t += s.wcnt[w];
                s.cnt = t;
            }
            __syncthreads();
            row_sync(C);
            int all = 0;
            for (int p = 0; p < C; ++p) all += C > 1 ? static_cast<int>(peer_ld32(peer_addr(&s.cnt, p))) : s.cnt;
            row_sync(C);
            if (all >= a.n) lo = mid; else hi = mid - 1;
        }
        const float v = key_to_f(lo);
        if (tid == 0) s.n = 0;
        __syncthreads();
        // above v: fewer than n in the row.  Equal: the span's first n in id order
        for (int k = k0 + tid; k < k1; k += kRowThreads) {
            const uint4 w = load_vec<SX>(x, k, k1);
#pragma unroll
            for (int q = 0; q < VE; ++q) {
                const float e = elem<SX>(w, q);
                if (e > v) s.own[atomicAdd(&s.n, 1)] = top_key(e, x.first(k) + q);
            }
        }
        __syncthreads();
        const int above = s.n;
        int equal = 0;
        for (int base = k0; base < k1 && equal < a.n; base += kRowThreads) {
            const int k = base + tid;
            const uint4 w = load_vec<SX>(x, k, k1);
            int c = 0;
#pragma unroll
            for (int q = 0; q < VE; ++q) c += elem<SX>(w, q) == v;
            int incl = c;
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            if (lane == 31) s.wcnt[warp] = incl;
            __syncthreads();
            int at = equal + incl - c;
            for (int p = 0; p < kRowWarps; ++p) {
                if (p < warp) at += s.wcnt[p];
                equal += s.wcnt[p];
            }
#pragma unroll
            for (int q = 0; q < VE; ++q)
                if (elem<SX>(w, q) == v) {
                    if (at < a.n) s.own[above + at] = top_key(v, x.first(k) + q);
                    ++at;
                }
            __syncthreads();
        }
        if (tid == 0) s.n = above + min(equal, a.n);
        __syncthreads();
        row_sync(C);
        gather(kTopBuf);
    }
    __syncthreads();

    // ---- places: an entry's rank in the row's list, a warp to an entry
    if (ok) {
        for (int i = warp; i < mine; i += kRowWarps) {
            const unsigned long long k = s.all[before + i];
            int at = 0;
            for (int e = lane; e < total; e += 32) at += s.all[e] > k;
            at = __reduce_add_sync(0xffffffffu, at);
            if (lane == 0 && at < a.n) {
                a.values[out + at] = ckey_v(k);
                a.ids[out + at] = ckey_id(k);
            }
        }
    }
    if (rank == 0) {
        for (int i = (ok ? total : 0) + tid; i < a.n; i += kRowThreads) {
            a.values[out + i] = -INFINITY;
            a.ids[out + i] = -1;
        }
        if (tid == 0) {
            a.row_status[row] = ok ? 0 : DSPARK_ROW_NONFINITE;
            if (a.lse)
                a.lse[row] = ok ? static_cast<float>(ExpRef(es.m, a.c).log_unit(a.inv_t) + log(static_cast<double>(es.sum))) : NAN;
        }
    }
    if (C > 1) {                                             // peers' shared memory is read until here
        cluster_arrive();
        cluster_wait();
    }
}

}  // namespace
}  // namespace dspark

using namespace dspark;

extern "C" dspark_status_t dspark_top_logits(const void* logits, const dspark_top_params_t* p, float* out_values,
                                             int32_t* out_ids, float* out_lse) {
    if (!p || !logits || !out_values || !out_ids || !p->row_status) return DSPARK_ERR_INVALID_ARG;
    if (p->n_rows < 1 || p->n_rows > DSPARK_MAX_ROWS || p->V < 1 || p->V > DSPARK_MAX_V) return DSPARK_ERR_INVALID_ARG;
    if (p->n < 1 || p->n > DSPARK_MAX_TOP_LOGITS) return DSPARK_ERR_INVALID_ARG;
    if (p->logits_dtype != DSPARK_BF16 && p->logits_dtype != DSPARK_FP32) return DSPARK_ERR_INVALID_ARG;
    const float c = kLog2E / p->temperature;
    if (!(p->temperature > 0.f) || !(c > 0.f) || !(c < INFINITY)) return DSPARK_ERR_INVALID_ARG;
    const int sx = p->logits_dtype == DSPARK_BF16 ? 2 : 4;
    if (p->logits_stride < p->V || reinterpret_cast<uintptr_t>(logits) % sx) return DSPARK_ERR_INVALID_ARG;

    TopArgs a{};
    a.V = p->V; a.n = p->n; a.c = c; a.inv_t = 1.0 / p->temperature; a.stride = p->logits_stride;
    a.x = logits; a.values = out_values; a.ids = out_ids; a.lse = out_lse; a.row_status = p->row_status;
    // CTAs per row: spans of at most 256 KB, and smaller ones, down to a batch of vectors, while the
    // rows alone do not make two CTAs per SM.  A CTA's part after the stream costs about as much as
    // streaming 128 KB: 576 rows of 512 KB take 91 us in halves and 132 us in eighths, 9 rows of
    // 304 KB 24 us whole and 12 us in eighths.
    const int nvec = max_vectors(p->V, sx);
    a.cluster = 1;
    while (a.cluster < kMaxCluster && (nvec > a.cluster * 16384 ||
                                       (nvec >= 2 * a.cluster * kTopBatch && static_cast<long long>(p->n_rows) * a.cluster < 304)))
        a.cluster *= 2;
    const unsigned grid = static_cast<unsigned>(p->n_rows) * static_cast<unsigned>(a.cluster);
    cudaStream_t s = static_cast<cudaStream_t>(p->stream);
    const cudaError_t e = sx == 2 ? launch_cluster(top_logits_kernel<2>, grid, kRowThreads, a.cluster, 0, s, a)
                                  : launch_cluster(top_logits_kernel<4>, grid, kRowThreads, a.cluster, 0, s, a);
    return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}
