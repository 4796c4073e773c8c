// What the one-launch kernels around the epilogue (logit processing, top-logit records, drafter
// distillation) share: a vocabulary row seen as 16-byte vectors whatever its alignment, packed
// maxima, and thread-block clusters that split one row.
#pragma once

#include <cuda_bf16.h>

#include "dspark_internal.cuh"

namespace dspark {

constexpr int kRowThreads = 256;                 // threads of a row CTA
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kMaxCluster = 8;                   // CTAs that share a row at most (the portable limit)
constexpr float kLog2E = 1.4426950408889634f;

// A row of V logits of SX bytes at p, cut into 16-byte vectors at the address's own 16-byte
// boundaries: vector k holds the logits k*VE - a0 .. k*VE - a0 + VE - 1, of which the first and
// last vector may lack some.
template <int SX>
struct VocabRow {
    static constexpr int VE = 16 / SX;           // logits per vector
    const unsigned char* p;
    int V, a0, nvec;

    __device__ __forceinline__ VocabRow(const void* base, long long row, long long stride, int V_)
        : p(static_cast<const unsigned char*>(base) + row * stride * SX), V(V_) {
        a0 = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / SX);
        nvec = (a0 + V + VE - 1) / VE;
    }
    __device__ __forceinline__ int first(int k) const { return k * VE - a0; }     // logit at lane 0 of vector k
    __device__ __forceinline__ bool whole(int k) const { return first(k) >= 0 && first(k) + VE <= V; }
};

// Vectors a row of V logits can have at most, whatever its alignment.
inline int max_vectors(int V, int sx) { return (V + 16 / sx - 1 + 16 / sx - 1) / (16 / sx); }

__device__ __forceinline__ uint4 ld_vec16(const void* p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void st_vec16(void* p, const uint4& v) {
    asm volatile("st.global.v4.u32 [%0], {%1, %2, %3, %4};"
                 :: "l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ uint32_t word_of(const uint4& w, int k) { return k == 0 ? w.x : k == 1 ? w.y : k == 2 ? w.z : w.w; }

template <int SX>
__device__ __forceinline__ float elem(const uint4& w, int q) {
    if (SX == 2) {
        const uint32_t x = word_of(w, q >> 1);
        return (q & 1) ? bf16_hi(x) : bf16_lo(x);
    }
    return __uint_as_float(word_of(w, q));
}

// Replace lane q (a compile-time constant after unrolling) by the bits of an SX-byte value.
template <int SX>
__device__ __forceinline__ void put_bits(uint4& w, int q, uint32_t bits) {
    const int k = SX == 2 ? q >> 1 : q;
    uint32_t& x = k == 0 ? w.x : k == 1 ? w.y : k == 2 ? w.z : w.w;
    if (SX == 2) x = (q & 1) ? ((x & 0x0000FFFFu) | (bits << 16)) : ((x & 0xFFFF0000u) | bits);
    else x = bits;
}
template <int SX>
__device__ __forceinline__ constexpr uint32_t ninf_bits() { return SX == 2 ? 0xFF80u : 0xFF800000u; }
// A vector of -inf.
template <int SX>
__device__ __forceinline__ uint4 ninf_vec() {
    constexpr uint32_t w = SX == 2 ? 0xFF80FF80u : 0xFF800000u;
    return make_uint4(w, w, w, w);
}

// Round v to the row's type (to nearest even) and return its bits.
template <int SX>
__device__ __forceinline__ uint32_t to_bits(float v) {
    if (SX == 2) return static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(v)));
    return __float_as_uint(v);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}

template <int SX>
__device__ __forceinline__ float load_logit(const VocabRow<SX>& r, int i) {
    if (SX == 2) return __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const unsigned short*>(r.p + 2LL * i)) << 16);
    return *reinterpret_cast<const float*>(r.p + 4LL * i);
}

// Vector k of the row; the lanes it lacks (and all of a k past the row) read as -inf.
template <int SX>
__device__ __forceinline__ uint4 load_vec(const VocabRow<SX>& r, int k, int k_end) {
    constexpr int VE = VocabRow<SX>::VE;
    if (k >= k_end) return ninf_vec<SX>();
    const int i0 = r.first(k);
    if (r.whole(k)) return ld_vec16(r.p + static_cast<long long>(i0) * SX);
    uint4 w = ninf_vec<SX>();
#pragma unroll
    for (int q = 0; q < VE; ++q)
        if (i0 + q >= 0 && i0 + q < r.V) put_bits<SX>(w, q, to_bits<SX>(load_logit<SX>(r, i0 + q)));
    return w;
}

// One warp copies vectors [b, e) of a row to shared memory: whole ones by a bulk copy, the row's
// ragged first and last by two lanes, whose fence puts a later bulk copy into the same buffer behind their
// stores.  The mbarrier takes one arrival per phase.
template <int SX>
__device__ __forceinline__ void fetch_piece(const VocabRow<SX>& r, int b, int e, uint4* dst, uint64_t* bar) {
    const int lane = threadIdx.x & 31;
    const int wb = b + (e > b && !r.whole(b)), we = e - (e > wb && !r.whole(e - 1));
    const bool ragged = wb > b || we < e;
    if (lane == 0) {
        const unsigned bytes = we > wb ? 16u * static_cast<unsigned>(we - wb) : 0u;
        if (ragged) asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" :: "r"(smem_u32(bar)), "r"(bytes) : "memory");
        else mbar_arrive_expect_tx(bar, bytes);
        if (bytes) bulk_g2s(dst + (wb - b), r.p + static_cast<long long>(r.first(wb)) * SX, bytes, bar);
    }
    if (ragged) {
        if (lane == 1 && wb > b) dst[0] = load_vec<SX>(r, b, e);
        if (lane == 2 && we < e && we >= wb) dst[we - b] = load_vec<SX>(r, we, e);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    }
}

// Maximum of a vector's lanes, NaN lanes left out.
template <int SX>
__device__ __forceinline__ float vec_max(const uint4& w) {
    if (SX == 2) {
        const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&w);
        const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        const uint32_t x = *reinterpret_cast<const uint32_t*>(&m);
        return fmaxf(bf16_lo(x), bf16_hi(x));
    }
    return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
}

// The same over U vectors.
template <int SX, int U>
__device__ __forceinline__ float vecs_max(const uint4 (&w)[U]) {
    if (SX == 2) {
        const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(w);
        __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
#pragma unroll
        for (int u = 1; u < U; ++u)
            m = __hmax2(m, __hmax2(__hmax2(h[4 * u], h[4 * u + 1]), __hmax2(h[4 * u + 2], h[4 * u + 3])));
        const uint32_t x = *reinterpret_cast<const uint32_t*>(&m);
        return fmaxf(bf16_lo(x), bf16_hi(x));
    }
    float m = vec_max<SX>(w[0]);
#pragma unroll
    for (int u = 1; u < U; ++u) m = fmaxf(m, vec_max<SX>(w[u]));
    return m;
}

// ---------------------------------------------------------------- packed fp32 pairs
__device__ __forceinline__ unsigned long long pack2(float lo, float hi) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(unsigned long long v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// Pair k (a compile-time constant after unrolling) of a vector, as fp32.
template <int SX>
__device__ __forceinline__ unsigned long long pair_of(const uint4& w, int k) {
    return pack2(elem<SX>(w, 2 * k), elem<SX>(w, 2 * k + 1));
}

// ---------------------------------------------------------------- values as the sum of two floats
// For what meets cancellation at a row's end: some 2^-45 relative, in a few dozen cycles a step (the
// 64-bit unit takes as long for one addition, and a thread's chain of them kept its CTA).  The exact sum is
// Knuth's, the exact product Dekker's with a fused multiply-add for its splitting.
struct TwoFloat {
    float hi, lo;
};
__device__ __forceinline__ TwoFloat two_sum(float a, float b) {   // exact
    const float s = a + b, t = s - a;
    return TwoFloat{s, (a - (s - t)) + (b - t)};
}
__device__ __forceinline__ TwoFloat two_prod(float a, float b) {   // exact, underflow aside
    const float p = a * b;
    return TwoFloat{p, fmaf(a, b, -p)};
}
__device__ __forceinline__ TwoFloat operator+(const TwoFloat& a, const TwoFloat& b) {
    const TwoFloat s = two_sum(a.hi, b.hi);
    return TwoFloat{s.hi, s.lo + (a.lo + b.lo)};
}
__device__ __forceinline__ TwoFloat operator-(const TwoFloat& a) { return TwoFloat{-a.hi, -a.lo}; }
__device__ __forceinline__ TwoFloat operator*(const TwoFloat& a, const TwoFloat& b) {
    const TwoFloat p = two_prod(a.hi, b.hi);
    return TwoFloat{p.hi, p.lo + fmaf(a.hi, b.lo, a.lo * b.hi)};
}
__device__ __forceinline__ TwoFloat operator/(const TwoFloat& a, const TwoFloat& b) {
    const float q = a.hi / b.hi;
    return TwoFloat{q, (fmaf(-q, b.hi, a.hi) + fmaf(-q, b.lo, a.lo)) / b.hi};
}
__device__ __forceinline__ TwoFloat ln2_two() { return TwoFloat{0.693147182464599609375f, -1.90465429995777e-9f}; }
// log(v), v > 0 normal: the exponent's part, and logf of what is left in [0.75, 1.5).
__device__ __forceinline__ TwoFloat log_two(float v) {
    const int e = (__float_as_int(v) - 0x3F400000) >> 23;
    return TwoFloat{static_cast<float>(e), 0.f} * ln2_two() + TwoFloat{logf(__int_as_float(__float_as_int(v) - (e << 23))), 0.f};
}

// ---------------------------------------------------------------- sums of exponentials
// exp(x / T) relative to a row's or thread's maximum m, as 2^(x c - r) with c = log2(e)/T: r is m c
// rounded up to a whole number, so that the one fma rounds nothing but its result and sums of
// different maxima join by powers of two.  Where m c has no such whole number (the type's lowest
// values, infinities) the form is 2^((x - m) c); where sums of both forms meet (logits of 2.9 million T, on
// either side of it) the join is off by up to one power of two.
struct ExpRef {
    float m, c, r;
    bool whole;
    __device__ __forceinline__ ExpRef(float m_, float c_) : m(m_), c(c_), r(ceilf(m_ * c_)), whole(fabsf(m_ * c_) < 4194304.f) {}
    __device__ __forceinline__ float of(float x) const {     // m > -inf
        return ex2_approx(whole ? fmaf(x, c, -r) : (x - m) * c);
    }
};

// A sum of them: m is the largest x seen (-inf while nothing above -inf was).
struct ExpSum {
    float m, sum;
};
__device__ __forceinline__ float rebase(float from, float to, float c) {   // 0 for an empty sum
    if (!(from > -INFINITY)) return 0.f;
    const ExpRef a(from, c), b(to, c);
    return ex2_approx(a.whole && b.whole ? a.r - b.r : (from - to) * c);
}
// NaN sums carry over: a NaN logit leaves m alone and makes its sum NaN, so does +inf.
__device__ __forceinline__ ExpSum merge(const ExpSum& a, const ExpSum& b, float c) {
    ExpSum r;
    r.m = fmaxf(a.m, b.m);
    r.sum = r.m > -INFINITY ? a.sum * rebase(a.m, r.m, c) + b.sum * rebase(b.m, r.m, c) : a.sum + b.sum;
    return r;
}
// The warp's sum, in every lane: one rescaling to the warp's maximum, then plain additions.
__device__ __forceinline__ ExpSum warp_merge(ExpSum a, float c) {
    const float m = key_to_f(__reduce_max_sync(0xffffffffu, fkey(a.m)));
    a.sum = warp_sum(m > -INFINITY ? a.sum * rebase(a.m, m, c) : a.sum);
    a.m = m;
    return a;
}
// A thread's sum while it streams: the maximum, its whole exponent r, the sum.
struct RunSum {
    float m = -INFINITY, r = -INFINITY, sum = 0.f;
    __device__ __forceinline__ ExpSum get() const { return ExpSum{m, sum}; }
};
// Add the exponentials of U vectors whose maximum is bm.
template <int SX, int U>
__device__ __forceinline__ void add_exps(RunSum& es, const uint4 (&v)[U], float bm, float c) {
    constexpr int VE = 16 / SX;
    const float m = fmaxf(es.m, bm), t = m * c, r = ceilf(t);
    if (fabsf(t) < 4194304.f) {
        // what came before scales by a power of two: 0 for nothing (r = -inf) and for the lowest values
        const unsigned long long c2 = pack2(c, c), r2 = pack2(-r, -r);
        unsigned long long acc[2] = {pack2(es.sum * ex2_approx(es.r - r), 0.f), 0ull};
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < VE / 2; ++k) {
                float lo, hi;
                unpack2(fma2(pair_of<SX>(v[u], k), c2, r2), lo, hi);
                acc[k & 1] = add2(acc[k & 1], pack2(ex2_approx(lo), ex2_approx(hi)));
            }
        float lo, hi;
        unpack2(add2(acc[0], acc[1]), lo, hi);
        es.sum = lo + hi;
    } else {
        es.sum = rebase(es.m, m, c) * es.sum;
        const float ref = m > -INFINITY ? m : 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int q = 0; q < VE; ++q) es.sum += ex2_approx((elem<SX>(v[u], q) - ref) * c);
    }
    es.m = m;
    es.r = r;
}

// ---------------------------------------------------------------- clusters
__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ unsigned cluster_id() {
    unsigned r;
    asm("mov.u32 %0, %%clusterid.x;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// Shared-window address of the same variable in CTA `rank` of the cluster.
__device__ __forceinline__ unsigned peer_addr(const void* smem, unsigned rank) {
    unsigned a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(smem)), "r"(rank));
    return a;
}
__device__ __forceinline__ uint32_t peer_ld32(unsigned a) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ unsigned long long peer_ld64(unsigned a) {
    unsigned long long v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
    return v;
}

// Write 16 or 8 bytes into a cluster CTA's shared memory; the bytes count on the mbarrier there.
__device__ __forceinline__ void peer_push128(unsigned a, unsigned bar, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];"
                 :: "r"(a), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar) : "memory");
}
__device__ __forceinline__ void peer_push64(unsigned a, unsigned bar, unsigned long long v) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];"
                 :: "r"(a), "l"(v), "r"(bar) : "memory");
}
__device__ __forceinline__ unsigned global_ms() {            // 2^20 ns to the unit
    unsigned long long t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    return static_cast<unsigned>(t >> 20);
}
// Wait for an mbarrier's phase with a bound, false when it runs out; data pushed by the
// cluster's CTAs is visible afterwards.  The thread sleeps up to 1 ms at a time: without the
// hint a waiting warp polls, and takes issue slots from those that work.  For a peer the bound is longer than what the
// peer may wait for its copies: it pushes late rather than not at all, and to a CTA that is still there.
constexpr unsigned kCopyMs = 2000, kPeerMs = 10 * kCopyMs;
__device__ __forceinline__ bool bar_wait(uint64_t* bar, unsigned parity, unsigned limit = kCopyMs, const volatile int* given_up = nullptr) {
    unsigned t0 = 0;
    for (unsigned i = 0;; ++i) {
        unsigned ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity), "r"(1000000u) : "memory");
        if (ok) return true;
        if (given_up && (*given_up & DSPARK_ROW_INTERNAL)) return false;   // another wait of the CTA has run out
        const unsigned t = global_ms();
        if (i == 0) t0 = t;
        else if (t - t0 > limit) return false;
    }
}
// The same for a copy's arrival, or for a buffer to be free for one.  After an expired one no further copy is
// asked for, and the CTA waits once more, for those in flight, before it ends.
#ifdef DSPARK_TEST_EXPIRED_WAITS
constexpr bool kExpireAtOnce = true;                         // test build: every one of them
#else
constexpr bool kExpireAtOnce = false;
#endif
__device__ __forceinline__ bool copy_wait(uint64_t* bar, unsigned parity, const volatile int* given_up = nullptr) {
    return !kExpireAtOnce && bar_wait(bar, parity, kCopyMs, given_up);
}

// Launch `grid` CTAs of `threads` threads in clusters of `cluster`, as a programmatic dependent of the
// previous kernel in s: the CTAs are placed while that one's last end, and wait for it (0.1 to 0.6 us a
// call).  The kernels do not let their own successors in before they end: its CTAs took the places
// that even out a grid of a few per SM (333 top-logit rows of 50001: 24.7 us, 21.8 without).
// The cluster attribute is left out for single CTAs: each pays for it (4096 token rows of 16000: 33.0 us, 28.3 without).
template <typename... KArgs, typename... Args2>
inline cudaError_t launch_cluster(void (*kern)(KArgs...), unsigned grid, int threads, int cluster, size_t smem, cudaStream_t s,
                                  Args2&&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = cluster == 1 ? attr + 1 : attr;
    cfg.numAttrs = cluster == 1 ? 1 : 2;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Args2>(args)...);
}

}  // namespace dspark
