// top_logits_kernel: the n largest logits of every row (value descending, id ascending among
// equals) and log sum exp(x / T), one launch, each row split over a cluster of CTAs.
//
// One pass over the row, bound by bandwidth.  A CTA streams its span in batches of kTopVec
// 16-byte vectors per thread, the next batch loading while this one is reduced:
//   - the sum of 2^((x - m) log2(e)/T) per thread, m its running maximum, rescaled at most once
//     per batch;
//   - keys (value, id) of the logits that reach a threshold go to shared memory.  The first
//     threshold is the n-th largest of the 256 threads' maxima over the first batch: n distinct
//     logits reach it, so every one of the span's n largest does.  A batch whose keys do not
//     fit is taken again vector by vector, the buffer cut down to its n largest keys whenever the
//     next vectors might not fit and the threshold set above the n-th: spans are read in id
//     order, so a later equal logit loses to those kept.  Any input is exact; rows of equal
//     values take this path.
// Each CTA cuts its keys to n by a radix selection over (value, id); the cluster's first CTA
// gathers the CTAs' keys and sums through distributed shared memory, selects and ranks the row's n
// and writes the record.
#include "block_utils.cuh"
#include "vocab_rows.cuh"

namespace dspark {

namespace {

constexpr int kTopVec = 4;
constexpr int kTopBatch = kTopVec * kRowThreads;             // vectors per batch
constexpr int kTopCap = 2560;                                // keys a CTA holds
constexpr int kTopStep = kRowThreads * 8;                    // keys one vector per thread adds at most
static_assert(kTopCap >= DSPARK_MAX_TOP_LOGITS + kTopStep, "a cut buffer must take one step");
static_assert(kTopCap >= kMaxCluster * DSPARK_MAX_TOP_LOGITS, "the merge must take every CTA's keys");
static_assert(DSPARK_MAX_TOP_LOGITS <= kRowThreads, "the first threshold ranks one maximum per thread");

// (order-preserving value key, id reversed): 32 + 24 bits.
constexpr int kIdBits = 24;
constexpr unsigned kIdMask = (1u << kIdBits) - 1;
__device__ __forceinline__ unsigned long long top_key(float v, int id) {
    return (static_cast<unsigned long long>(fkey(v)) << kIdBits) | (kIdMask - static_cast<unsigned>(id));
}
__device__ __forceinline__ float top_key_v(unsigned long long k) { return key_to_f(static_cast<uint32_t>(k >> kIdBits)); }
__device__ __forceinline__ int top_key_id(unsigned long long k) { return static_cast<int>(kIdMask - (static_cast<unsigned>(k) & kIdMask)); }

struct TopArgs {
    int V, n, cluster;
    float c;                                                 // log2(e) / T
    double inv_t;                                            // 1 / T
    long long stride;
    const void* x;
    float* values;
    int* ids;
    float* lse;
    int* row_status;
};

struct __align__(16) TopSmem {
    unsigned long long keys[kTopCap];
    int hist[256];
    alignas(16) float tmax[kRowThreads];
    ExpSum es[kRowWarps];
    ExpSum part;                                             // this CTA's sum
    int n;                                                   // keys held (passes kTopCap when a batch overflows)
    int bcast[2];
    float th;
    int wtot[kRowWarps];
};

// Smallest key of the n largest of keys[0, m), 0 < n <= m: radix selection from the top byte,
// left as soon as the digit's keys are all wanted.  The value's 32 bits, then the id's 24; a
// bf16 value's key has its low 16 bits fixed by the sign (all ones below zero): they are not searched.
template <int SX>
__device__ unsigned long long select_nth(TopSmem& s, int m, int n) {
    const int tid = threadIdx.x;
    unsigned long long prefix = 0, pmask = 0;
    int want = n;
    for (int shift = 48; shift >= 0; shift -= 8) {
        if (SX == 2 && shift == 32) {
            if (!(prefix >> 55)) prefix |= 0xFFFFull << kIdBits;
            pmask |= 0xFFFFull << kIdBits;
        }
        if (SX == 2 && (shift == 32 || shift == 24)) continue;
        s.hist[tid] = 0;
        __syncthreads();
        for (int i = tid; i < m; i += kRowThreads) {
            const unsigned long long k = s.keys[i];
            if ((k & pmask) == prefix) atomicAdd(&s.hist[static_cast<unsigned>(k >> shift) & 255u], 1);
        }
        __syncthreads();
        if (tid < 32) {                                      // lane l: digits 255-8l .. 248-8l
            int c[8], t = 0;
#pragma unroll
            for (int q = 0; q < 8; ++q) { c[q] = s.hist[255 - 8 * tid - q]; t += c[q]; }
            int incl = t;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (tid >= o) incl += y;
            }
            int run = incl - t;
            if (run < want && incl >= want) {
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    if (run < want && run + c[q] >= want) {
                        s.bcast[0] = 255 - 8 * tid - q;
                        s.bcast[1] = (want - run) | (run + c[q] == want ? 1 << 30 : 0);
                    }
                    run += c[q];
                }
            }
        }
        __syncthreads();
        prefix |= static_cast<unsigned long long>(s.bcast[0]) << shift;
        pmask |= 255ull << shift;
        const int w = s.bcast[1];
        want = w & ~(1 << 30);
        if (w >> 30) break;
    }
    return prefix;
}

// Keep the n largest of keys[0, m) (m > n) in keys[0, n), in no particular order.
template <int SX>
__device__ void cut_to(TopSmem& s, int m, int n) {
    const int tid = threadIdx.x;
    __syncthreads();
    const unsigned long long least = select_nth<SX>(s, m, n);
    unsigned long long mine[(kTopCap + kRowThreads - 1) / kRowThreads];
    int cnt = 0;
#pragma unroll
    for (int q = 0; q < (kTopCap + kRowThreads - 1) / kRowThreads; ++q) {
        const int i = q * kRowThreads + tid;
        mine[q] = i < m ? s.keys[i] : 0ull;
        if (mine[q] < least) mine[q] = 0ull;                 // no key is 0: fkey of a number is not
        cnt += mine[q] != 0ull;
    }
    int incl = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if ((tid & 31) >= o) incl += y;
    }
    if ((tid & 31) == 31) s.wtot[tid >> 5] = incl;
    __syncthreads();
    int at = incl - cnt;
    for (int w = 0; w < (tid >> 5); ++w) at += s.wtot[w];
#pragma unroll
    for (int q = 0; q < (kTopCap + kRowThreads - 1) / kRowThreads; ++q)
        if (mine[q] != 0ull) s.keys[at++] = mine[q];
    if (tid == 0) s.n = n;
    __syncthreads();
}

// Hand the vector's logits that reach th to the buffer; *cnt counts them.  True when one found
// the buffer full.
template <int SX>
__device__ __forceinline__ bool offer(TopSmem& s, const uint4& w, int i0, float th, int* cnt) {
    constexpr int VE = VocabRow<SX>::VE;
    bool full = false;
#pragma unroll
    for (int q = 0; q < VE; ++q) {
        const float v = elem<SX>(w, q);
        if (v >= th) {
            const int at = atomicAdd(&s.n, 1);
            ++*cnt;
            if (at < kTopCap) s.keys[at] = top_key(v, i0 + q);
            else full = true;
        }
    }
    return full;
}

// The least value above the n-th largest key kept (keys[0, n)): what a later logit must reach.
__device__ float above_least(TopSmem& s, int n) {
    const int tid = threadIdx.x;
    unsigned long long k = tid < n ? s.keys[tid] : ~0ull;    // n <= kRowThreads
    for (int o = 16; o; o >>= 1) {
        const unsigned long long y = __shfl_xor_sync(0xffffffffu, k, o);
        k = y < k ? y : k;
    }
    unsigned long long* const part = reinterpret_cast<unsigned long long*>(s.tmax);   // tmax is free by now
    if ((tid & 31) == 0) part[tid >> 5] = k;
    __syncthreads();
    for (int w = 0; w < kRowWarps; ++w) k = part[w] < k ? part[w] : k;
    __syncthreads();
    return key_to_f(static_cast<uint32_t>(k >> kIdBits) + 1u);
}

template <int SX>
__global__ void __launch_bounds__(kRowThreads) top_logits_kernel(TopArgs a) {
    constexpr int VE = VocabRow<SX>::VE;
    __shared__ TopSmem s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = a.cluster, rank = static_cast<int>(blockIdx.x % C);
    const long long row = blockIdx.x / C;
    const VocabRow<SX> x(a.x, row, a.stride, a.V);
    const int k0 = static_cast<int>(static_cast<long long>(x.nvec) * rank / C);
    const int k1 = static_cast<int>(static_cast<long long>(x.nvec) * (rank + 1) / C);
    if (tid == 0) s.n = 0;

    uint4 cur[kTopVec], nxt[kTopVec];
#pragma unroll
    for (int u = 0; u < kTopVec; ++u) nxt[u] = load_vec<SX>(x, k0 + u * kRowThreads + tid, k1);

    ExpSum es{-INFINITY, 0.f};
    float th = -INFINITY;
    for (int base = k0; base < k1; base += kTopBatch) {
#pragma unroll
        for (int u = 0; u < kTopVec; ++u) cur[u] = nxt[u];
        if (base + kTopBatch < k1) {
#pragma unroll
            for (int u = 0; u < kTopVec; ++u) nxt[u] = load_vec<SX>(x, base + kTopBatch + u * kRowThreads + tid, k1);
        }
        float vm[kTopVec], bm = -INFINITY;
#pragma unroll
        for (int u = 0; u < kTopVec; ++u) {
            vm[u] = vec_max<SX>(cur[u]);
            bm = fmaxf(bm, vm[u]);
        }
        if (base == k0) {
            // the n-th largest thread maximum, ties counted by thread order
            s.tmax[tid] = bm;
            __syncthreads();
            int above = 0;
            for (int i = 0; i < kRowThreads; i += 4) {
                const float4 o = *reinterpret_cast<const float4*>(&s.tmax[i]);
                above += (o.x > bm || (o.x == bm && i < tid)) + (o.y > bm || (o.y == bm && i + 1 < tid)) +
                         (o.z > bm || (o.z == bm && i + 2 < tid)) + (o.w > bm || (o.w == bm && i + 3 < tid));
            }
            if (above == a.n - 1) s.th = bm;
            __syncthreads();
            th = fmaxf(s.th, -3.402823466e38f);              // -inf logits have no place in the record
        }
        if (bm > es.m) {
            es.sum *= rebase(es.m, bm, a.c);
            es.m = bm;
        }
        const float m = es.m > -INFINITY ? es.m : 0.f;
#pragma unroll
        for (int u = 0; u < kTopVec; ++u)
#pragma unroll
            for (int q = 0; q < VE; ++q) es.sum += exp_of(elem<SX>(cur[u], q), m, a.c);
        int mine = 0;
        bool full = false;
#pragma unroll
        for (int u = 0; u < kTopVec; ++u)
            if (vm[u] >= th) full |= offer<SX>(s, cur[u], x.first(base + u * kRowThreads + tid), th, &mine);
        if (__syncthreads_or(full)) {                        // take the batch back, then again in steps
            if (mine) atomicSub(&s.n, mine);
            __syncthreads();
            int held = s.n;
            __syncthreads();
            for (int u = 0; u < kTopVec; ++u) {
                if (held + kTopStep > kTopCap) {             // then more than n are held
                    cut_to<SX>(s, held, a.n);
                    th = above_least(s, a.n);
                }
                uint4 w = cur[0];
#pragma unroll
                for (int t = 1; t < kTopVec; ++t) if (u == t) w = cur[t];
                if (vec_max<SX>(w) >= th) offer<SX>(s, w, x.first(base + u * kRowThreads + tid), th, &mine);
                __syncthreads();
                held = s.n;
                __syncthreads();
            }
        }
    }
    __syncthreads();
    int held = s.n;
    __syncthreads();
    if (held > a.n) { cut_to<SX>(s, held, a.n); held = a.n; }

    // the block's sum of exponentials, warps in order
    for (int o = 16; o; o >>= 1) {
        const ExpSum other{__shfl_xor_sync(0xffffffffu, es.m, o), __shfl_xor_sync(0xffffffffu, es.sum, o)};
        es = merge(es, other, a.c);
    }
    if (lane == 0) s.es[warp] = es;
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kRowWarps; ++w) es = merge(es, s.es[w], a.c);
        s.part = es;
    }
    if (C > 1) {
        __syncthreads();
        cluster_arrive();
        cluster_wait();
    }
    if (rank == 0) {
        int total = held;
        if (C > 1) {
            for (int p = 1; p < C; ++p) {
                const int np = static_cast<int>(peer_ld32(peer_addr(&s.n, p)));
                const unsigned from = peer_addr(s.keys, p);
                for (int i = tid; i < np; i += kRowThreads) s.keys[total + i] = peer_ld64(from + 8u * i);
                total += np;
            }
            if (tid == 0)
                for (int p = 1; p < C; ++p) {
                    const unsigned from = peer_addr(&s.part, p);
                    es = merge(es, ExpSum{__uint_as_float(peer_ld32(from)), __uint_as_float(peer_ld32(from + 4))}, a.c);
                }
            __syncthreads();
            if (total > a.n) { cut_to<SX>(s, total, a.n); total = a.n; }
        }
        if (tid == 0) s.part = es;
        __syncthreads();
        es = s.part;
        // a row with NaN or +inf has a NaN sum, one with nothing above -inf a maximum of -inf
        const bool ok = es.sum == es.sum && es.m > -INFINITY;
        if (tid == 0) {
            a.row_status[row] = ok ? 0 : DSPARK_ROW_NONFINITE;
            if (a.lse) a.lse[row] = ok ? static_cast<float>(es.m * a.inv_t + log(static_cast<double>(es.sum))) : NAN;
        }
        if (tid < a.n) {                                     // n <= kRowThreads: rank one key per thread
            const long long o = row * a.n;
            if (ok && tid < total) {
                const unsigned long long k = s.keys[tid];
                int at = 0;
                for (int i = 0; i < total; ++i) at += s.keys[i] > k;
                a.values[o + at] = top_key_v(k);
                a.ids[o + at] = top_key_id(k);
            } else {
                a.values[o + tid] = -INFINITY;
                a.ids[o + tid] = -1;
            }
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
    // CTAs per row: one batch of vectors each at least
    a.cluster = 1;
    while (a.cluster < kMaxCluster && max_vectors(p->V, sx) >= 2 * a.cluster * kTopBatch) a.cluster *= 2;
    const unsigned grid = static_cast<unsigned>(p->n_rows) * static_cast<unsigned>(a.cluster);
    cudaStream_t s = static_cast<cudaStream_t>(p->stream);
    const cudaError_t e = sx == 2 ? launch_cluster(top_logits_kernel<2>, grid, a.cluster, 0, s, a)
                                  : launch_cluster(top_logits_kernel<4>, grid, a.cluster, 0, s, a);
    return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}
