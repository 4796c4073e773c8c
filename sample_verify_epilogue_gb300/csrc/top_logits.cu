// top_logits_kernel: the n largest logits of every row (value descending, id ascending among
// equals) and log sum exp(x / T), one launch, each row split over a cluster of C CTAs.
//
// One pass over the row, bound by bandwidth: a CTA streams its span through three 16 KB buffers filled
// by bulk copies, a batch of four 16-byte vectors per thread at a time, and each thread keeps the sum of
// its exponentials and its four largest batch maxima (where they were, and the fifth), nothing
// else.  512 of the row's largest such maxima then give a threshold: their n-th largest is reached by
// at least n logits, and by few more (of 512 groups about -512 ln(1 - n/512) logits: 69 for n = 64), so
//   1. maxima go to shared memory; every CTA reads the row's 512 through distributed shared memory
//      and finds their n-th largest by bisection on the upper 16 bits of its key;
//   2. a thread whose maximum reaches it reads that batch again (L2), or up to four, or all of its
//      vectors where the fifth maximum reaches it too, and lists the logits that do (576 rows of 262144,
//      n = 256: 90 us with three noted, 76 with four; n = 64: 57 both ways);
//   3. every CTA reads the row's whole list, sorts it into 256 buckets by value and ranks its own entries in
//      theirs: the rank is the place in the record (against the whole list: 96 us where buckets take 90,
//      same rows, three noted; 333 rows of 50001 fp32, n = 256: 36 and 29).
// Rows whose list would be too long (equal values, few distinct values, values bunched in one
// group, more than a tenth of a row of 1000 to 2500 wanted) take an exact path: bisection on the value over counts of the whole row, from that
// threshold up to the maximum; then the logits above the n-th value, and in id order as many equal
// to it as are wanted.
#include "vocab_rows.cuh"

namespace dspark {

namespace {

constexpr int kTopVec = 4;
constexpr int kTopBatch = kTopVec * kRowThreads;             // vectors per piece: a batch per thread
constexpr int kTopSlots = 3;                                 // buffers
constexpr int kTopGroups = 512;                              // of a row, whatever its cluster
constexpr int kTopOwn = 1024;                                // entries a CTA lists at most
constexpr int kTopAll = 1024;                                // entries of a row on the short path
constexpr int kTopBuf = DSPARK_MAX_TOP_LOGITS * (kMaxCluster + 1);   // ... on the exact path: < n above, n equal per CTA
constexpr size_t kTopSmem = sizeof(uint4) * kTopSlots * kTopBatch;
constexpr unsigned kTopBuckets = kRowThreads;                // a thread to a bucket
static_assert(kTopBuckets == 256, "the bucket is 8 bits of the key");
constexpr size_t kTopLists = sizeof(unsigned long long) * (kTopOwn + 2 * kTopBuf);
static_assert(kTopLists <= kTopSmem, "the lists take the buffers' place");

struct TopArgs {
    int V, n, log_c;                                         // log_c: of the cluster's size
    int keep;                                                // the span stays in its buffers
    float c;                                                 // log2(e) / T
    float inv_t, inv_t_low;                                  // 1 / T in two parts
    long long stride;
    const void* x;
    float* values;
    int* ids;
    float* lse;
    int* row_status;
};

struct __align__(16) TopSmem {
    unsigned short gmax[kTopGroups];                         // this CTA's 512/C group maxima: upper halves of their keys
    uint64_t full[kTopSlots], empty[kTopSlots];
    ExpSum es[kRowWarps];
    int late, issued;                                        // a copy did not come in time; copies asked for until then
    int todo[kRowWarps][4 * 32];                             // a warp's (batch << 5 | lane) to look at again
    int n;                                                   // entries listed (passes kTopOwn when they do not fit)
    int cnt;                                                 // exact path: this CTA's count
    int wcnt[kRowWarps];
    int bucket[kTopBuckets];                                 // entries of a bucket, then where it ends
    uint2 range[kRowWarps];                                  // smallest and largest maxima of a warp's
    alignas(16) int reach[2][kRowWarps];                     // a warp's maxima that reach a step's key
    unsigned th;                                             // threshold key
    ExpSum row;
    int row_late;
};

__device__ __forceinline__ float key_floor(unsigned k) {     // value of a key, never -inf
    return fmaxf(key_to_f(k), -3.402823466e38f);
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
    extern __shared__ uint4 s_ring[];                        // [kTopSlots][kTopBatch]; after the stream, or behind it, the lists:
    unsigned long long* const own = reinterpret_cast<unsigned long long*>(s_ring + (a.keep ? kTopSlots * kTopBatch : 0));   // this CTA's entries
    unsigned long long* const all = own + kTopOwn;           // the row's
    unsigned long long* const sorted = all + kTopBuf;        // the row's by buckets
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = 1 << a.log_c, rank = static_cast<int>(blockIdx.x & (C - 1));
    const long long row = blockIdx.x >> a.log_c;
    const VocabRow<SX> x(a.x, row, a.stride, a.V);
    const int k0 = x.nvec * rank >> a.log_c, k1 = x.nvec * (rank + 1) >> a.log_c;   // nvec * C < 2^31
    const int np = (k1 - k0 + kTopBatch - 1) / kTopBatch;
    if (tid == 0) {
        for (int k = 0; k < kTopSlots; ++k) {
            mbar_init(&s.full[k], 1);
            mbar_init(&s.empty[k], kRowWarps);
        }
        fence_mbar_init();
        s.n = 0;
        s.late = 0;
        s.issued = np;
    }
    s.bucket[tid] = 0;
    __syncthreads();
    pdl_wait();                                              // what came before in the stream

    // ---- the stream
    RunSum run;
    float m1 = -INFINITY, m2 = -INFINITY, m3 = -INFINITY, m4 = -INFINITY, m5 = -INFINITY;   // the thread's largest batch maxima
    int b1 = 0, b2 = 0, b3 = 0, b4 = 0;                              // where the first four were
    auto note = [&](float bm, int j) {
        const bool first = bm > m1, second = bm > m2, third = bm > m3, fourth = bm > m4;
        m5 = fmaxf(m5, fminf(m4, bm));
        m4 = third ? m3 : fmaxf(m4, bm);
        b4 = third ? b3 : fourth ? j : b4;
        m3 = second ? m2 : fmaxf(m3, bm);
        b3 = second ? b2 : third ? j : b3;
        m2 = first ? m1 : fmaxf(m2, bm);
        b2 = first ? b1 : second ? j : b2;
        m1 = fmaxf(m1, bm);
        b1 = first ? j : b1;
    };
    {
        bool late = false;
        if (warp == 0)
            for (int j = 0; j < min(np, kTopSlots); ++j)
                fetch_piece<SX>(x, k0 + j * kTopBatch, min(k1, k0 + (j + 1) * kTopBatch), s_ring + j * kTopBatch, &s.full[j]);
        int slot = 0, before = kTopSlots - 1;                // of piece j and of piece j - 1
        unsigned parity = 0, parity_before = 0;
        for (int j = 0; j < np; ++j) {
            if (warp == 0 && j > 0 && j + kTopSlots - 1 < np) {   // the piece before this one leaves its buffer
                const int f = j + kTopSlots - 1;
                late = late || !copy_wait(&s.empty[before], parity_before);
                if (__any_sync(0xffffffffu, late)) s.issued = min(s.issued, f);
                else fetch_piece<SX>(x, k0 + f * kTopBatch, min(k1, k0 + (f + 1) * kTopBatch), s_ring + before * kTopBatch, &s.full[before]);
            }
            late = late || !copy_wait(&s.full[slot], parity);
            const uint4* const q0 = s_ring + slot * kTopBatch;
            const int cnt = min(kTopBatch, k1 - k0 - j * kTopBatch);
            uint4 v[kTopVec];
#pragma unroll
            for (int u = 0; u < kTopVec; ++u) v[u] = u * kRowThreads + tid < cnt ? q0[u * kRowThreads + tid] : ninf_vec<SX>();
            const float bm = vecs_max<SX>(v);
            add_exps<SX>(run, v, bm, a.c);
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.empty[slot]);
            note(bm, j);
            before = slot;
            parity_before = parity;
            if (++slot == kTopSlots) { slot = 0; parity ^= 1u; }
        }
        if (late) s.late = 1;
    }
    // a span of one piece: every vector is a batch of its own, or a short row had no more batches than a long
    // record has entries (333 rows of 4096, n = 256: 44 us with batches of four, on the exact path, 12 so;
    // n = 20: 7.9 and 8.2)
    const bool fine = np == 1;
    if (fine) {
        m1 = m2 = m3 = m4 = m5 = -INFINITY;
#pragma unroll
        for (int u = 0; u < kTopVec; ++u) {
            const int k = u * kRowThreads + tid;
            note(k < k1 - k0 ? vec_max<SX>(s_ring[k]) : -INFINITY, u);
        }
    }

    // ---- group maxima: 512/C of this CTA; a group is a batch, a thread, or 2 or 4 threads
    {
        float gm = m1;
        if (C == 1) {
            s.gmax[tid] = static_cast<unsigned short>(fkey(m1) >> 16);
            s.gmax[tid + kRowThreads] = static_cast<unsigned short>(fkey(m2) >> 16);
        } else {
            if (C >= 4) gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, 1));
            if (C >= 8) gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, 2));
            const int per = C / 2;                           // threads of a group, a power of two
            if ((tid & (per - 1)) == 0) s.gmax[tid >> (a.log_c - 1)] = static_cast<unsigned short>(fkey(gm) >> 16);
        }
        const ExpSum es = warp_merge(run.get(), a.c);
        if (lane == 0) s.es[warp] = es;
    }
    row_sync(C);

    // ---- threshold, and the row's sum
    {
        // two of the row's 512 maxima to a thread; CTA p has 256/C words of two
        const int log_per = 8 - a.log_c;
        const unsigned* const word = reinterpret_cast<const unsigned*>(s.gmax) + (tid & ((1 << log_per) - 1));
        const unsigned two = C > 1 ? peer_ld32(peer_addr(word, tid >> log_per)) : *word;
        const unsigned x0 = two & 0xFFFFu, x1 = two >> 16;
        ExpSum es{-INFINITY, 0.f};                           // (warp 1: the row's warps' sums, joined below)
        int late = 0;
        if (warp == 1) {
            auto sum_of = [&](int w) {                       // of warp w mod 8 of CTA w / 8
                if (w >= kRowWarps * C) return ExpSum{-INFINITY, 0.f};
                const unsigned from = peer_addr(&s.es[w % kRowWarps], w / kRowWarps);
                return ExpSum{__uint_as_float(peer_ld32(from)), __uint_as_float(peer_ld32(from + 4))};
            };
            static_assert(kRowWarps * kMaxCluster == 64, "two sums to a lane");
            es = merge(sum_of(lane), sum_of(lane + 32), a.c);
            if (lane < C) late = static_cast<int>(peer_ld32(peer_addr(&s.late, lane)));
        }
        // the largest key that n maxima reach, or a smaller one that exactly n do
        unsigned lo = __reduce_min_sync(0xffffffffu, min(x0, x1)), hi = __reduce_max_sync(0xffffffffu, max(x0, x1));
        if (lane == 0) s.range[warp] = make_uint2(lo, hi);
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) {
            lo = min(lo, s.range[w].x);
            hi = max(hi, s.range[w].y);
        }
        for (int step = 0; lo < hi; ++step) {
            const unsigned mid = (lo + hi + 1) >> 1;
            const int c = __popc(__ballot_sync(0xffffffffu, x0 >= mid)) + __popc(__ballot_sync(0xffffffffu, x1 >= mid));
            if (lane == 0) s.reach[step & 1][warp] = c;
            __syncthreads();
            int all_c = 0;
#pragma unroll
            for (int w = 0; w < kRowWarps; ++w) all_c += s.reach[step & 1][w];
            if (all_c >= a.n) lo = mid; else hi = mid - 1;
            if (all_c == a.n) break;
        }
        if (tid == 0) s.th = lo << 16;
        if (warp == 1) {
            es = warp_merge(es, a.c);
            late = __any_sync(0xffffffffu, late);
            if (lane == 0) {
                s.row = es;
                s.row_late = late;
            }
        }
    }
    __syncthreads();
    const float top = s.row.m;
    // a row with NaN or +inf has a NaN sum, one with nothing above -inf a maximum of -inf
    const bool ok = s.row.sum == s.row.sum && top > -INFINITY && !s.row_late;

    // ---- list the logits that reach the threshold
    const float th = key_floor(s.th);
    // A warp's vectors, one per lane (k, or nothing for a vector of -inf): one place for all of it.
    auto offer = [&](const uint4& w, int k) {
        unsigned hits = 0u;
#pragma unroll
        for (int q = 0; q < VE; ++q) hits |= static_cast<unsigned>(elem<SX>(w, q) >= th) << q;
        if (!__any_sync(0xffffffffu, hits != 0u)) return;
        const int c = __popc(hits);
        int incl = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        int at = 0;
        if (lane == 31) at = atomicAdd(&s.n, incl);
        at = __shfl_sync(0xffffffffu, at, 31) + incl - c;
#pragma unroll
        for (int q = 0; q < VE; ++q)
            if (hits >> q & 1u) {
                if (at < kTopOwn) own[at] = ckey(elem<SX>(w, q), x.first(k) + q);
                ++at;
            }
    };
    auto again = [&](int k) { return !a.keep ? load_vec<SX>(x, k, k1) : k < k1 ? s_ring[k - k0] : ninf_vec<SX>(); };
    if (ok) {
        // the batches to look at again, a lane to a vector: (lane, batch) pairs of the warp's threads
        const bool whole = m5 >= th;                         // or all its vectors
        const unsigned f1 = __ballot_sync(0xffffffffu, m1 >= th && !whole), f2 = __ballot_sync(0xffffffffu, m2 >= th && !whole);
        const unsigned f3 = __ballot_sync(0xffffffffu, m3 >= th && !whole), f4 = __ballot_sync(0xffffffffu, m4 >= th && !whole), below = (1u << lane) - 1u;
        const int n1 = __popc(f1), n2 = n1 + __popc(f2), n3 = n2 + __popc(f3), n4 = n3 + __popc(f4);
        int* const todo = s.todo[warp];
        if (f1 >> lane & 1u) todo[__popc(f1 & below)] = b1 << 5 | lane;
        if (f2 >> lane & 1u) todo[n1 + __popc(f2 & below)] = b2 << 5 | lane;
        if (f3 >> lane & 1u) todo[n2 + __popc(f3 & below)] = b3 << 5 | lane;
        if (f4 >> lane & 1u) todo[n3 + __popc(f4 & below)] = b4 << 5 | lane;
        __syncwarp();
        const int log_vec = fine ? 0 : 2;                    // vectors of a batch
        static_assert(kTopVec == 4, "log_vec");
        for (int i0 = 0; i0 < n4; i0 += 32 >> log_vec) {
            const int i = i0 + (lane >> log_vec), what = i < n4 ? todo[i] : 0;
            const int k = k0 + ((what >> 5 << log_vec) + (lane & ((1 << log_vec) - 1))) * kRowThreads + warp * 32 + (what & 31);
            offer(i < n4 ? again(k) : ninf_vec<SX>(), k);
        }
        unsigned many = __ballot_sync(0xffffffffu, whole);
        while (many) {
            const int t = warp * 32 + __ffs(many) - 1;
            many &= many - 1;
            for (int base = k0 + t; base < k1; base += 32 * kRowThreads) {
                const int k = base + lane * kRowThreads;
                offer(again(k), k);
            }
            // the exact path counts anew (a lane's view of the count is as good as another's)
            if (__any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&s.n) > kTopOwn)) break;
        }
    }
    row_sync(C);

    // ---- the row's list, counted by buckets of the value's key between the maximum (bucket 0) and the threshold
    const long long out = row * a.n;
    const unsigned key_lo = fkey(th), key_hi = fkey(top);
    const int shift = max(0, 32 - __clz(key_hi - key_lo) - 8);
    auto bucket = [&](unsigned long long k) {
        const unsigned key = static_cast<unsigned>(k >> 32);
        return min(kTopBuckets - 1u, (key_hi - min(key, key_hi)) >> shift);
    };
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
            if (i < total) {
                const unsigned long long k = C > 1 ? peer_ld64(peer_addr(&own[i - start], p)) : own[i];
                all[i] = k;
                atomicAdd(&s.bucket[bucket(k)], 1);
            }
        }
        return true;
    };
    if (ok && !gather(kTopAll)) {
        // exact path (the same for every CTA of the row): v, the n-th largest value, is the largest
        // with at least n logits at or above it
        row_sync(C);                                         // the counts have been read
        unsigned lo = fkey(th), hi = fkey(top);
        while (lo < hi) {
            const unsigned mid = lo + ((hi - lo) >> 1) + 1;
            const float v = key_to_f(mid);
            int c = 0;
            for (int k = k0 + tid; k < k1; k += kRowThreads) {
                const uint4 w = again(k);
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
            int count = 0;
            for (int p = 0; p < C; ++p) count += C > 1 ? static_cast<int>(peer_ld32(peer_addr(&s.cnt, p))) : s.cnt;
            row_sync(C);
            if (count >= a.n) lo = mid; else hi = mid - 1;
        }
        const float v = key_to_f(lo);
        if (tid == 0) s.n = 0;
        __syncthreads();
        // above v: fewer than n in the row.  Equal: the span's first n in id order
        for (int k = k0 + tid; k < k1; k += kRowThreads) {
            const uint4 w = again(k);
#pragma unroll
            for (int q = 0; q < VE; ++q) {
                const float e = elem<SX>(w, q);
                if (e > v) own[atomicAdd(&s.n, 1)] = ckey(e, x.first(k) + q);
            }
        }
        __syncthreads();
        const int above = s.n;
        int equal = 0;
        for (int base = k0; base < k1 && equal < a.n; base += kRowThreads) {
            const int k = base + tid;
            const uint4 w = again(k);
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
                    if (at < a.n) own[above + at] = ckey(v, x.first(k) + q);
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

    // ---- places: an entry's rank in the row's list
    if (ok) {
        int incl = s.bucket[tid];
        const int c = incl;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) s.wcnt[warp] = incl;
        __syncthreads();
        incl -= c;
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) incl += w < warp ? s.wcnt[w] : 0;
        s.bucket[tid] = incl;                                // where a bucket begins; then, entry by entry, where it ends
        __syncthreads();
        for (int i = tid; i < total; i += kRowThreads) {
            const unsigned long long k = all[i];
            sorted[atomicAdd(&s.bucket[bucket(k)], 1)] = k;
        }
        __syncthreads();
        const int sub = tid & 3;                             // four lanes to an entry, a quarter of its bucket each
        for (int i0 = 0; i0 < mine; i0 += kRowThreads / 4) {
            const int i = i0 + (tid >> 2);
            int at = 0, begin = 0;
            unsigned long long k = 0;
            if (i < mine) {
                k = all[before + i];
                const unsigned b = bucket(k);
                begin = b ? s.bucket[b - 1] : 0;
                const int end = begin < a.n ? s.bucket[b] : begin;   // (past the record)
                for (int e = begin + sub; e < end; e += 4) at += sorted[e] > k;
            }
            at += __shfl_xor_sync(0xffffffffu, at, 1);
            at += __shfl_xor_sync(0xffffffffu, at, 2);
            at += begin;
            if (sub == 0 && i < mine && at < a.n) {
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
        if (tid == kRowThreads - 1) {                        // (a warp that ranks little)
            a.row_status[row] = s.row_late ? DSPARK_ROW_INTERNAL : ok ? 0 : DSPARK_ROW_NONFINITE;
            if (a.lse) {
                const ExpRef ref(top, a.c);
                const TwoFloat unit = ref.whole ? TwoFloat{ref.r, 0.f} * ln2_two() : TwoFloat{top, 0.f} * TwoFloat{a.inv_t, a.inv_t_low};
                const TwoFloat l = unit + log_two(s.row.sum);
                a.lse[row] = !ok ? NAN : fabsf(unit.hi) < INFINITY ? l.hi + l.lo : unit.hi;
            }
        }
    }
    if (!ok && warp == 0 && s.late)                          // the last copies in flight
        for (int f = max(0, s.issued - kTopSlots); f < s.issued; ++f) bar_wait(&s.full[f % kTopSlots], f / kTopSlots & 1);
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
    a.V = p->V; a.n = p->n; a.c = c; a.stride = p->logits_stride;
    a.inv_t = static_cast<float>(1.0 / p->temperature);
    a.inv_t_low = static_cast<float>(1.0 / p->temperature - static_cast<double>(a.inv_t));
    a.x = logits; a.values = out_values; a.ids = out_ids; a.lse = out_lse; a.row_status = p->row_status;
    // CTAs per row: one, or more, down to three quarters of a piece of the row each, while that makes no more
    // than two CTAs per SM or so: what follows the stream costs a CTA about what 100 KB do, and more
    // CTAs only stand in line.  Rows of 304 KB: 250 of them 25.0 us whole, 24.5 in halves, 31.5 in
    // quarters; 80 of them 20.3, 15.5, 13.5 us and 18.6 in eighths; 16 of them 19.3, 13.8, 10.3, 9.6 (before
    // a row's end was shortened by 1 us).
    const int nvec = max_vectors(p->V, sx);
    int cluster = 1;
    while (cluster < kMaxCluster && nvec >= 2 * cluster * (kTopBatch * 3 / 4) && static_cast<long long>(p->n_rows) * 2 * cluster <= 330)
        cluster *= 2;
    while ((1 << a.log_c) < cluster) ++a.log_c;
    const unsigned grid = static_cast<unsigned>(p->n_rows) << a.log_c;
    // A span that fits the buffers stays there where two CTAs to an SM are enough, and is looked at again there
    // instead of in L2, with the lists behind it (200 rows of 20000, n = 256: 14.5 us, 13.2 so; 9 of 151936:
    // 9.0, 8.8).
    a.keep = (nvec + cluster - 1) / cluster <= kTopSlots * kTopBatch && grid <= 300;
    const size_t smem = kTopSmem + (a.keep ? kTopLists : 0);
    cudaStream_t s = static_cast<cudaStream_t>(p->stream);
    auto kern = sx == 2 ? top_logits_kernel<2> : top_logits_kernel<4>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kTopSmem + kTopLists)) != cudaSuccess)
        return DSPARK_ERR_CUDA;
    const cudaError_t e = launch_cluster(kern, grid, kRowThreads, cluster, smem, s, a);
    return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}
