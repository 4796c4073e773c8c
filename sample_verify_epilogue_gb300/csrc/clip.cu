// The norm of many gradients together, and the gradients scaled to a largest norm.
//
// norm_kernel: every CTA takes an equal share of the list, whatever tensors it belongs to, and leaves one sum of squares;
// scale_kernel adds the shares up in a fixed order, in every CTA, and scales.  The list travels in
// the launches' parameters, so that a call needs no copy to the device and can be captured as it is.
//
// A thread's squares of a few vectors are added in fp32, those sums in pairs of floats.  Squares leave fp32's range
// for elements beyond 2^64 or below 2^-63: a share whose sum is infinite, or next to nothing though not all of it is 0,
// is summed again by a power of two.
//
// Bound by bandwidth: 374 M bf16 into fp32 take 112 us for the norm (6.7 TB/s) and 368 for the scaling (6.1 TB/s of reads and
// writes).  The gradients are read twice, since the factor needs them all; of lists that fit L2 the second read is from there.
// A short list (4 tensors of 1 MB) takes 5.0 us: two launches, and the shares' way through L2.
#include <algorithm>
#include <cmath>

#include "vocab_rows.cuh"

namespace dspark {

namespace {

constexpr int kClipThreads = 256, kClipWarps = kClipThreads / 32;
constexpr int kClipVec = 4;                                  // vectors a thread has on their way (8 in the norm: lists of 5 to 80 MB 1 to 15% slower)
constexpr int kClipCtas = 4;                                 // CTAs to an SM (five in the scaling: lists of 1 to 20 MB 1 to 10% slower)
constexpr int kUnit = kClipThreads;                          // vectors that go to one CTA together
constexpr int kMaxShares = 2048;                             // shares of a group of tensors
constexpr int kLargeList = 1000, kSmallList = 100;           // tensors of a launch: 32,000 bytes of parameters hold 1000

struct ClipItem {
    const unsigned char* grad;
    unsigned char* out;
    long long numel;
    int first;                                               // its first unit
    unsigned short bf16, wide;                               // the gradient is bf16; out is fp32 all the same
};

// A share's sum of squares: (hi + lo) 2^(180 kind) for kind 0 and 1, 2^-160 for -1.
struct __align__(16) Share {
    float hi, lo;
    int kind, pad;
};

template <int N>
struct ClipList {
    Share* shares;                                           // [all shares]
    float* norm;
    int* status;
    float max_norm;
    int n, units, n_shares, write_norm;                      // of this group; of all groups (scale); the first group's launch
    ClipItem item[N];
};

// A tensor as 16-byte vectors at its address's own boundaries: vector k holds elements k*VE - a0 .. + VE - 1.
template <int SX>
struct Flat {
    static constexpr int VE = 16 / SX;
    const unsigned char* p;
    long long numel, nvec;
    int a0;
    __device__ __forceinline__ Flat(const void* base, long long n)
        : p(static_cast<const unsigned char*>(base)), numel(n), a0(static_cast<int>((reinterpret_cast<uintptr_t>(base) & 15u) / SX)) {
        nvec = (a0 + n + VE - 1) / VE;
    }
    __device__ __forceinline__ long long first(long long k) const { return k * VE - a0; }
    __device__ __forceinline__ bool whole(long long k) const { return first(k) >= 0 && first(k) + VE <= numel; }
    __device__ __forceinline__ uint4 load(long long k) const {   // elements it lacks read as 0
        const long long i0 = first(k);
        if (whole(k)) return ld_vec16(p + i0 * SX);
        uint4 w = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int q = 0; q < VE; ++q)
            if (i0 + q >= 0 && i0 + q < numel)
                put_bits<SX>(w, q, SX == 2 ? reinterpret_cast<const unsigned short*>(p)[i0 + q] : reinterpret_cast<const unsigned*>(p)[i0 + q]);
        return w;
    }
};

// Calls part(item, first vector, last vector) for what units [j0, j1) of the list hold of each tensor.
template <int N, typename Part>
__device__ __forceinline__ void for_parts(const ClipList<N>& a, Part part) {
    int j = static_cast<int>(static_cast<long long>(a.units) * blockIdx.x / gridDim.x);
    const int j1 = static_cast<int>(static_cast<long long>(a.units) * (blockIdx.x + 1) / gridDim.x);
    if (j >= j1) return;
    int i = 0, hi = a.n - 1;
    while (i < hi) {
        const int mid = (i + hi + 1) >> 1;
        if (a.item[mid].first <= j) i = mid;
        else hi = mid - 1;
    }
    for (; j < j1; ++i) {
        const int next = i + 1 < a.n ? min(a.item[i + 1].first, j1) : j1;
        part(a.item[i], static_cast<long long>(j - a.item[i].first) * kUnit, static_cast<long long>(next - a.item[i].first) * kUnit);
        j = next;
    }
}

struct Squares {
    TwoFloat sum{0.f, 0.f};
    unsigned any = 0u;                                       // not 0: something is not 0

    template <int SX, int U>
    __device__ __forceinline__ void add(const uint4 (&v)[U], float scale) {
        unsigned long long acc[2] = {0ull, 0ull};
        const unsigned long long s2 = pack2(scale, scale);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            any |= (v[u].x | v[u].y | v[u].z | v[u].w) & (SX == 2 ? 0x7fff7fffu : 0x7fffffffu);
#pragma unroll
            for (int k = 0; k < 16 / SX / 2; ++k) {
                unsigned long long x = pair_of<SX>(v[u], k);
                if (scale != 1.f) x = mul2(x, s2);
                acc[k & 1] = fma2(x, x, acc[k & 1]);
            }
        }
        float lo, hi;
        unpack2(add2(acc[0], acc[1]), lo, hi);
        const TwoFloat d = two_sum(sum.hi, lo + hi);
        sum = TwoFloat{d.hi, sum.lo + d.lo};
    }
    template <int SX>
    __device__ __forceinline__ void add_part(const ClipItem& it, long long b, long long e, float scale) {
        const Flat<SX> g(it.grad, it.numel);
        e = min(e, g.nvec);
        // whole vectors go straight through
        const long long w0 = b + (b < e && !g.whole(b)), w1 = e - (e > w0 && !g.whole(e - 1));
        const unsigned char* p = g.p + g.first(w0 + threadIdx.x) * SX;
        const int n = static_cast<int>(w1 - w0);             // a CTA's share of fewer than 2^31 units
        int k = threadIdx.x;
        for (; k + (kClipVec - 1) * kClipThreads < n; k += kClipVec * kClipThreads, p += 16 * kClipVec * kClipThreads) {
            uint4 v[kClipVec];
#pragma unroll
            for (int u = 0; u < kClipVec; ++u) v[u] = ld_vec16(p + 16 * u * kClipThreads);
            add<SX>(v, scale);
        }
        for (; k < n; k += kClipThreads, p += 16 * kClipThreads) {
            const uint4 v[1] = {ld_vec16(p)};
            add<SX>(v, scale);
        }
        if (threadIdx.x < 2) {                               // the ragged ends
            if (threadIdx.x ? w1 < e : b < w0) {
                const uint4 v[1] = {g.load(threadIdx.x ? w1 : b)};
                add<SX>(v, scale);
            }
        }
    }
    __device__ __forceinline__ void join(const TwoFloat& o) {
        const TwoFloat d = two_sum(sum.hi, o.hi);
        sum = TwoFloat{d.hi, d.lo + (sum.lo + o.lo)};
    }
};

// Sum of the CTA's share by scale, in every thread; *any: something in it is not 0.
template <int N>
__device__ __forceinline__ TwoFloat share_sum(const ClipList<N>& a, float scale, TwoFloat* s_sum, bool* any) {
    Squares q;
    for_parts(a, [&](const ClipItem& it, long long b, long long e) {
        if (it.bf16) q.add_part<2>(it, b, e, scale);
        else q.add_part<4>(it, b, e, scale);
    });
#pragma unroll
    for (int o = 16; o; o >>= 1)
        q.join(TwoFloat{__shfl_xor_sync(0xffffffffu, q.sum.hi, o), __shfl_xor_sync(0xffffffffu, q.sum.lo, o)});
    if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = q.sum;
    *any = __syncthreads_or(q.any != 0u);
    q.sum = s_sum[0];
    for (int w = 1; w < kClipWarps; ++w) q.join(s_sum[w]);
    __syncthreads();
    return q.sum;
}

template <int N>
__global__ void __launch_bounds__(kClipThreads, kClipCtas) norm_kernel(const __grid_constant__ ClipList<N> a) {
    __shared__ TwoFloat s_sum[kClipWarps];
    pdl_wait();
    TwoFloat sum{0.f, 0.f};
    int kind = 0;
    float scale = 1.f;
#pragma unroll 1
    for (;;) {
        bool any;
        sum = share_sum(a, scale, s_sum, &any);              // the same in every thread
        if (kind != 0) break;
        if (!(sum.hi < INFINITY)) {
            scale = 0x1p-90f;
            kind = 1;
        } else if (any && sum.hi < 0x1p-90f) {
            scale = 0x1p80f;
            kind = -1;
        } else {
            break;
        }
    }
    if (threadIdx.x == 0) a.shares[blockIdx.x] = Share{sum.hi, sum.hi < INFINITY ? sum.lo : 0.f, kind, 0};
}

// v 2^e, |e| below 250, rounded once
__device__ __forceinline__ float times_2(float v, int e) {
    const int half = e >> 1;
    return v * __int_as_float((127 + half) << 23) * __int_as_float((127 + e - half) << 23);
}
// m 2^e, m in [1, 2] as a pair of floats, or what is 0 or not finite with e = 0.
struct Norm {
    TwoFloat m;
    int e;
    __device__ __forceinline__ float value() const { return times_2(m.hi, e); }
};
// sqrt(sum 2^e), e even, by a float's root and a step of Newton's: relative 2^-46
__device__ __forceinline__ Norm norm_of(TwoFloat sum, int e) {
    if (!(sum.hi > 0.f && sum.hi < INFINITY)) return Norm{TwoFloat{sum.hi, 0.f}, 0};
    if (sum.hi < 0x1p-64f) {
        sum = TwoFloat{sum.hi * 0x1p64f, sum.lo * 0x1p64f};
        e -= 64;
    }
    const int x = ((__float_as_int(sum.hi) >> 23) - 127) & ~1;
    const float by = __int_as_float((127 - x) << 23), hi = sum.hi * by, lo = sum.lo * by, r = sqrtf(hi);   // hi in [1, 4)
    return Norm{two_sum(r, __fdividef(0.5f, r) * (fmaf(-r, r, hi) + lo)), (x + e) / 2};
}
// v / m, rounded once (and a hundredth of that)
__device__ __forceinline__ float over(float v, const TwoFloat& m) {
    const float inv = __fdividef(1.f, m.hi), q = v * inv;
    return fmaf(fmaf(-q, m.hi, v) - q * m.lo, inv, q);
}

// The norm from all shares, the same in every thread of every CTA.  In pairs of floats: 64-bit sums, of which an SM adds some
// two a cycle, took 0.7 us of a list of 1 MB and 2 us of one of 12 MB.
struct ShareSum {
    TwoFloat sum;
    unsigned kinds;                                          // bits: some are of kind 1, -1, 0 and not 0
};
__device__ __forceinline__ Norm norm_of_shares(const Share* shares, int n, ShareSum* s_part) {
    const int tid = threadIdx.x;
    for (int unit = 0;;) {                                   // the sum by this kind's power of two
        Squares q;
        unsigned kinds = 0u;
        for (int k = tid; k < n; k += kClipThreads) {
            const Share s = shares[k];
            kinds |= s.kind > 0 ? 1u : s.kind < 0 ? 2u : s.hi > 0.f ? 4u : 0u;
            // (a share far below the unit's: its root twice, as a float holds no 2^-160)
            const float f = s.kind >= unit ? 1.f : unit == 0 ? 0x1p-80f : s.kind == 0 ? 0x1p-90f : 0.f;
            q.join(TwoFloat{s.hi * f * f, s.lo * f * f});
        }
#pragma unroll
        for (int o = 16; o; o >>= 1)
            q.join(TwoFloat{__shfl_xor_sync(0xffffffffu, q.sum.hi, o), __shfl_xor_sync(0xffffffffu, q.sum.lo, o)});
        kinds = __reduce_or_sync(0xffffffffu, kinds);
        if ((tid & 31) == 0) s_part[tid >> 5] = ShareSum{q.sum, kinds};
        __syncthreads();
        q.sum = s_part[0].sum;
        kinds = s_part[0].kinds;
#pragma unroll
        for (int w = 1; w < kClipWarps; ++w) {
            q.join(s_part[w].sum);
            kinds |= s_part[w].kinds;
        }
        const bool large = (kinds & 1u) || !(q.sum.hi < INFINITY), small = kinds == 2u;
        if (unit != 0 || !(large || small)) return norm_of(q.sum, unit > 0 ? 180 : unit < 0 ? -160 : 0);
        unit = large ? 1 : -1;
        __syncthreads();
    }
}

__device__ __forceinline__ void st_vec32(void* p, const float (&f)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 :: "l"(p), "r"(__float_as_uint(f[0])), "r"(__float_as_uint(f[1])), "r"(__float_as_uint(f[2])), "r"(__float_as_uint(f[3])),
                    "r"(__float_as_uint(f[4])), "r"(__float_as_uint(f[5])), "r"(__float_as_uint(f[6])), "r"(__float_as_uint(f[7])) : "memory");
}

template <int SX, bool WIDE>
__device__ __forceinline__ void scale_one(const Flat<SX>& g, unsigned char* out, long long k, const uint4& v, float c, bool alike) {
    constexpr int VE = 16 / SX;
    const long long i0 = g.first(k);
    float f[VE];
    uint4 w = v;                                             // c = 1: as they are (a NaN keeps its bits)
    if (c == 1.f) {
#pragma unroll
        for (int q = 0; q < VE; ++q) f[q] = elem<SX>(v, q);
    } else {
        const unsigned long long c2 = pack2(c, c);
#pragma unroll
        for (int h = 0; h < VE / 2; ++h) unpack2(mul2(pair_of<SX>(v, h), c2), f[2 * h], f[2 * h + 1]);
        if (SX == 2) w = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4 % VE], f[5 % VE]), pack_bf16(f[6 % VE], f[7 % VE]));
        else w = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
    const bool whole = alike && g.whole(k);
    if (WIDE) {
        float* o = reinterpret_cast<float*>(out);
        if (whole) {
            float f8[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) f8[q] = f[q % VE];
            st_vec32(o + i0, f8);                            // whole sectors: two stores of 16 bytes took 427 us for 368
        } else {
#pragma unroll
            for (int q = 0; q < VE; ++q)
                if (i0 + q >= 0 && i0 + q < g.numel) o[i0 + q] = f[q];
        }
    } else if (whole) {
        st_vec16(out + i0 * SX, w);
    } else {
#pragma unroll
        for (int q = 0; q < VE; ++q) {
            if (i0 + q < 0 || i0 + q >= g.numel) continue;
            if (SX == 2) reinterpret_cast<unsigned short*>(out)[i0 + q] = static_cast<unsigned short>(word_of(w, q >> 1) >> (16 * (q & 1)));
            else reinterpret_cast<unsigned*>(out)[i0 + q] = word_of(w, q);
        }
    }
}
template <int SX, bool WIDE>
__device__ __forceinline__ void scale_part(const ClipItem& it, long long b, long long e, float c) {
    const Flat<SX> g(it.grad, it.numel);
    e = min(e, g.nvec);
    // the output's vectors lie as the gradient's do
    const bool alike = ((reinterpret_cast<uintptr_t>(it.out) - static_cast<uintptr_t>(g.a0) * (WIDE ? 4 : SX)) & (WIDE ? 31u : 15u)) == 0;
    long long k = b + threadIdx.x;
    for (; k + (kClipVec - 1) * kClipThreads < e; k += kClipVec * kClipThreads) {
        uint4 v[kClipVec];
#pragma unroll
        for (int u = 0; u < kClipVec; ++u) v[u] = g.load(k + u * kClipThreads);
#pragma unroll
        for (int u = 0; u < kClipVec; ++u) scale_one<SX, WIDE>(g, it.out, k + u * kClipThreads, v[u], c, alike);
    }
    for (; k < e; k += kClipThreads) scale_one<SX, WIDE>(g, it.out, k, g.load(k), c, alike);
}

// The same by a factor below 2^-126, which fp32 holds with fewer bits or as 0: first by a power of two that brings the norm
// into [0.5, 1], then by the rest.  Element by element, as the other calls share its registers and code (by vectors: a list of 12 MB
// 9.9 us for 9.6).
template <int N>
__device__ __forceinline__ void scale_tiny(const ClipList<N>& a, float first, float c) {
    for_parts(a, [&](const ClipItem& it, long long b, long long e) {
        const int sx = it.bf16 ? 2 : 4, ve = 16 / sx, a0 = static_cast<int>((reinterpret_cast<uintptr_t>(it.grad) & 15u) / sx);
        const long long i1 = min(it.numel, e * ve - a0);
#pragma unroll 1
        for (long long i = max(0LL, b * ve - a0) + threadIdx.x; i < i1; i += kClipThreads) {
            const float g = it.bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(it.grad)[i]) : reinterpret_cast<const float*>(it.grad)[i];
            const float v = g * first * c;
            if (it.bf16 && !it.wide) reinterpret_cast<__nv_bfloat16*>(it.out)[i] = __float2bfloat16_rn(v);
            else reinterpret_cast<float*>(it.out)[i] = v;
        }
    });
}

template <int N>
__global__ void __launch_bounds__(kClipThreads, kClipCtas) scale_kernel(const __grid_constant__ ClipList<N> a) {
    __shared__ ShareSum s_part[kClipWarps];
    pdl_wait();
    const Norm n = norm_of_shares(a.shares, a.n_shares, s_part);
    const float norm = n.value();
    const bool finite = norm < INFINITY;
    // by the norm before its rounding (by the rounded one up to 1.7 u off for 1)
    // (a small max_norm by 2^64: what its quotient leaves would lie below fp32's numbers)
    const bool small = a.max_norm < 0x1p-64f;
    const float c = finite && norm > a.max_norm ? times_2(over(small ? a.max_norm * 0x1p64f : a.max_norm, n.m), small ? -n.e - 64 : -n.e) : 1.f;
    if (a.write_norm && blockIdx.x == 0 && threadIdx.x == 0) {
        *a.norm = norm;
        *a.status = finite ? 0 : DSPARK_ROW_NONFINITE;
    }
    if (__builtin_expect(!(c < 0x1p-126f), 1)) {
        for_parts(a, [&](const ClipItem& it, long long b, long long e) {
            if (c == 1.f && it.out == it.grad) return;
            if (!it.bf16) scale_part<4, false>(it, b, e, c);
            else if (it.wide) scale_part<2, true>(it, b, e, c);
            else scale_part<2, false>(it, b, e, c);
        });
    } else {
        scale_tiny(a, ldexpf(1.f, -n.e - 1), over(2.f * a.max_norm, n.m));
    }
}

int groups_of(int n) { return (n + kLargeList - 1) / kLargeList; }

dspark_status_t check_list(const dspark_grad_t* grads, int n) {
    for (int i = 0; i < n; ++i) {
        const dspark_grad_t& g = grads[i];
        if (g.numel < 0 || (g.dtype != DSPARK_BF16 && g.dtype != DSPARK_FP32)) return DSPARK_ERR_INVALID_ARG;
        if (g.out_dtype != g.dtype && g.out_dtype != DSPARK_FP32) return DSPARK_ERR_INVALID_ARG;
        if (g.numel == 0) continue;
        if (g.numel > (1LL << 43)) return DSPARK_ERR_UNSUPPORTED;   // (2^31 units are checked for where they are counted)
        const size_t sx = g.dtype == DSPARK_BF16 ? 2 : 4, so = g.out_dtype == DSPARK_BF16 ? 2 : 4;
        if (!g.grad || !g.out || reinterpret_cast<uintptr_t>(g.grad) % sx || reinterpret_cast<uintptr_t>(g.out) % so)
            return DSPARK_ERR_INVALID_ARG;
        if (g.grad == g.out && g.dtype != g.out_dtype) return DSPARK_ERR_INVALID_ARG;
    }
    return DSPARK_OK;
}

// Fill the list with the group's tensors; false when it has too many units.
template <int N>
bool fill(ClipList<N>& a, const dspark_grad_t* grads, int n) {
    long long units = 0;
    a.n = 0;
    for (int i = 0; i < n; ++i) {
        const dspark_grad_t& g = grads[i];
        if (g.numel == 0) continue;
        const int sx = g.dtype == DSPARK_BF16 ? 2 : 4;
        const long long a0 = static_cast<long long>(reinterpret_cast<uintptr_t>(g.grad) & 15u) / sx;
        const long long nvec = (a0 + g.numel + 16 / sx - 1) / (16 / sx);
        a.item[a.n++] = ClipItem{static_cast<const unsigned char*>(g.grad), static_cast<unsigned char*>(g.out), g.numel,
                                 static_cast<int>(units), g.dtype == DSPARK_BF16, g.out_dtype != g.dtype};
        units += (nvec + kUnit - 1) / kUnit;
        if (units > 0x7fffffffLL) return false;
    }
    a.units = static_cast<int>(units);
    return true;
}

template <int N>
dspark_status_t clip(const dspark_grad_t* grads, int n, float max_norm, float* norm, int* status, Share* shares, int sms, cudaStream_t s) {
    ClipList<N> a;
    a.max_norm = max_norm;
    a.norm = norm;
    a.status = status;
    const int groups = groups_of(n);
    int total = 0;
    for (int pass = 0; pass < 2; ++pass) {
        int done = 0;
        for (int k = 0; k < groups; ++k) {
            if (!fill(a, grads + k * kLargeList, std::min(kLargeList, n - k * kLargeList))) return DSPARK_ERR_UNSUPPORTED;
            // a unit to a CTA, or two where there are more than two for every SM (a list of 3 MB by one and two: 7.3 and 6.5 us;
            // one of 1 MB by two: 5.8 for 5.2)
            const int grid = std::max(1, std::min({a.units <= 2 * sms ? a.units : a.units / 2, kMaxShares, sms * kClipCtas}));
            a.shares = pass == 0 ? shares + done : shares;
            a.n_shares = total;
            a.write_norm = k == 0;
            if (pass == 0) done += grid;
            const bool skip = pass == 1 && k > 0 && a.units == 0;
            if (!skip && launch_k(pass == 0 ? norm_kernel<N> : scale_kernel<N>, dim3(static_cast<unsigned>(grid)), dim3(kClipThreads), 0, s,
                                  true, a) != cudaSuccess)
                return DSPARK_ERR_CUDA;
        }
        if (pass == 0) total = done;
    }
    return DSPARK_OK;
}

}  // namespace
}  // namespace dspark

using namespace dspark;

extern "C" {

size_t dspark_clip_workspace_bytes(int32_t n_grads) {
    if (n_grads < 1 || n_grads > DSPARK_MAX_GRADS) return 0;
    return static_cast<size_t>(groups_of(n_grads)) * kMaxShares * sizeof(Share);
}

dspark_status_t dspark_clip_grads(const dspark_grad_t* grads, int32_t n_grads, float max_norm, float* out_norm, int32_t* out_status,
                                  void* workspace, size_t workspace_bytes, void* stream) {
    if (!grads || n_grads < 1 || n_grads > DSPARK_MAX_GRADS || !(max_norm >= 0.f) || !out_norm || !out_status) return DSPARK_ERR_INVALID_ARG;
    if (const dspark_status_t st = check_list(grads, n_grads); st != DSPARK_OK) return st;
    if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 || workspace_bytes < dspark_clip_workspace_bytes(n_grads))
        return DSPARK_ERR_WORKSPACE;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return DSPARK_ERR_CUDA;
    Share* const shares = static_cast<Share*>(workspace);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return n_grads <= kSmallList ? clip<kSmallList>(grads, n_grads, max_norm, out_norm, out_status, shares, sms, s)
                                 : clip<kLargeList>(grads, n_grads, max_norm, out_norm, out_status, shares, sms, s);
}

}  // extern "C"
