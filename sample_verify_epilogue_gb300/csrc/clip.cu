// The norm of many gradients together, and the gradients scaled to a largest norm.
//
// norm_kernel: every CTA takes an equal share of the list's 16 KB chunks, whatever tensors they belong to, and leaves
// one sum of squares; scale_kernel adds the shares up in a fixed order, in every CTA, and scales.  The list travels in
// the launches' parameters, so that a call needs no copy to the device and can be captured as it is.
//
// A thread's squares of one chunk are added in fp32, the chunks' sums in pairs of floats.  Squares leave fp32's range
// for elements beyond 2^64 or below 2^-63: a share whose sum is infinite, or next to nothing though not all of it is 0,
// is summed again by a power of two.
#include <algorithm>
#include <cmath>

#include "vocab_rows.cuh"

namespace dspark {

namespace {

constexpr int kClipThreads = 256, kClipWarps = kClipThreads / 32;
constexpr int kClipVec = 4;                                  // vectors a thread holds at a time
constexpr int kChunk = kClipThreads * kClipVec;              // vectors of a chunk: 16 KB of the gradient
constexpr int kClipCtas = 8;                                 // CTAs to an SM
constexpr int kMaxShares = 2048;                             // shares of a group of tensors
constexpr int kLargeList = 1000, kSmallList = 100;           // tensors of a launch: 32,000 bytes of parameters hold 1000

struct ClipItem {
    const unsigned char* grad;
    unsigned char* out;
    long long numel;
    int first;                                               // its first chunk
    unsigned short bf16, wide;                               // the gradient is bf16; out is fp32 all the same
};

template <int N>
struct ClipList {
    double* shares;                                          // [all shares]
    float* norm;
    int* status;
    float max_norm;
    int n, chunks, n_shares, write_norm;                     // of this group; of all groups (scale); the first group's launch
    ClipItem item[N];
};

// A tensor as 16-byte vectors at its address's own boundaries: vector k holds elements k*VE - a0 .. + VE - 1.
template <int SX>
struct Flat {
    static constexpr int VE = 16 / SX;
    const unsigned char* p;
    long long numel;
    int a0;
    __device__ __forceinline__ Flat(const void* base, long long n)
        : p(static_cast<const unsigned char*>(base)), numel(n), a0(static_cast<int>((reinterpret_cast<uintptr_t>(base) & 15u) / SX)) {}
    __device__ __forceinline__ long long first(long long k) const { return k * VE - a0; }
    __device__ __forceinline__ uint4 load(long long k) const {   // elements it lacks read as 0
        const long long i0 = first(k);
        if (i0 >= 0 && i0 + VE <= numel) return ld_vec16(p + i0 * SX);
        uint4 w = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int q = 0; q < VE; ++q)
            if (i0 + q >= 0 && i0 + q < numel)
                put_bits<SX>(w, q, SX == 2 ? reinterpret_cast<const unsigned short*>(p)[i0 + q] : reinterpret_cast<const unsigned*>(p)[i0 + q]);
        return w;
    }
};

// The item that chunk j belongs to.
template <int N>
__device__ __forceinline__ int item_of(const ClipList<N>& a, int j) {
    int lo = 0, hi = a.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.item[mid].first <= j) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

template <int SX>
__device__ __forceinline__ void add_squares(const ClipItem& it, int j, float scale, TwoFloat& sum, unsigned& any) {
    const Flat<SX> g(it.grad, it.numel);
    uint4 v[kClipVec];
#pragma unroll
    for (int u = 0; u < kClipVec; ++u) v[u] = g.load(static_cast<long long>(j) * kChunk + u * kClipThreads + threadIdx.x);
    unsigned long long acc[2] = {0ull, 0ull};
    const unsigned long long s2 = pack2(scale, scale);
#pragma unroll
    for (int u = 0; u < kClipVec; ++u) {
        any |= (v[u].x | v[u].y | v[u].z | v[u].w) & (SX == 2 ? 0x7fff7fffu : 0x7fffffffu);
#pragma unroll
        for (int k = 0; k < 16 / SX / 2; ++k) {
            const unsigned long long x = mul2(pair_of<SX>(v[u], k), s2);
            acc[k & 1] = fma2(x, x, acc[k & 1]);
        }
    }
    float lo, hi;
    unpack2(add2(acc[0], acc[1]), lo, hi);
    const TwoFloat d = two_sum(sum.hi, lo + hi);
    sum = TwoFloat{d.hi, sum.lo + d.lo};
}

// Sum of the CTA's share by scale, in thread 0; *any: something in it is not 0.
template <int N>
__device__ __forceinline__ TwoFloat share_sum(const ClipList<N>& a, int j0, int j1, float scale, TwoFloat* s_sum, bool* any) {
    TwoFloat sum{0.f, 0.f};
    unsigned bits = 0u;
    if (j0 < j1) {
        int i = item_of(a, j0);
        for (int j = j0; j < j1; ++j) {
            while (i + 1 < a.n && a.item[i + 1].first <= j) ++i;
            const ClipItem& it = a.item[i];
            if (it.bf16) add_squares<2>(it, j - it.first, scale, sum, bits);
            else add_squares<4>(it, j - it.first, scale, sum, bits);
        }
    }
    auto join = [&](const TwoFloat& o) {
        const TwoFloat d = two_sum(sum.hi, o.hi);
        sum = TwoFloat{d.hi, d.lo + (sum.lo + o.lo)};
    };
#pragma unroll
    for (int o = 16; o; o >>= 1) join(TwoFloat{__shfl_xor_sync(0xffffffffu, sum.hi, o), __shfl_xor_sync(0xffffffffu, sum.lo, o)});
    if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = sum;
    *any = __syncthreads_or(bits != 0u);
    sum = s_sum[0];
    for (int w = 1; w < kClipWarps; ++w) join(s_sum[w]);
    __syncthreads();
    return sum;
}

template <int N>
__global__ void __launch_bounds__(kClipThreads, kClipCtas) norm_kernel(const __grid_constant__ ClipList<N> a) {
    __shared__ TwoFloat s_sum[kClipWarps];
    pdl_wait();
    const int j0 = static_cast<int>(static_cast<long long>(a.chunks) * blockIdx.x / gridDim.x);
    const int j1 = static_cast<int>(static_cast<long long>(a.chunks) * (blockIdx.x + 1) / gridDim.x);
    bool any;
    TwoFloat sum = share_sum(a, j0, j1, 1.f, s_sum, &any);
    double scale = 1.0;
    if (!(sum.hi < INFINITY)) {                              // the same in every thread
        sum = share_sum(a, j0, j1, 0x1p-90f, s_sum, &any);
        scale = 0x1p180;
    } else if (any && sum.hi < 0x1p-90f) {
        sum = share_sum(a, j0, j1, 0x1p80f, s_sum, &any);
        scale = 0x1p-160;
    }
    if (threadIdx.x == 0) a.shares[blockIdx.x] = (static_cast<double>(sum.hi) + static_cast<double>(sum.hi < INFINITY ? sum.lo : 0.f)) * scale;
}

template <int SX>
__device__ __forceinline__ void scale_chunk(const ClipItem& it, int j, float c) {
    constexpr int VE = 16 / SX;
    const Flat<SX> g(it.grad, it.numel);
    const long long k0 = static_cast<long long>(j) * kChunk + threadIdx.x;
    uint4 v[kClipVec];
#pragma unroll
    for (int u = 0; u < kClipVec; ++u) v[u] = g.load(k0 + u * kClipThreads);
    const bool wide = SX == 2 && it.wide;
    // the output's vectors lie as the gradient's do
    const bool alike = ((reinterpret_cast<uintptr_t>(it.out) - static_cast<uintptr_t>(g.a0) * (wide ? 4 : SX)) & 15u) == 0;
    const unsigned long long c2 = pack2(c, c);
#pragma unroll
    for (int u = 0; u < kClipVec; ++u) {
        const long long i0 = g.first(k0 + u * kClipThreads);
        if (i0 >= it.numel) break;
        float f[VE];
        if (c == 1.f) {                                      // as they are (a NaN keeps its bits)
#pragma unroll
            for (int q = 0; q < VE; ++q) f[q] = elem<SX>(v[u], q);
        } else {
#pragma unroll
            for (int h = 0; h < VE / 2; ++h) unpack2(mul2(pair_of<SX>(v[u], h), c2), f[2 * h], f[2 * h + 1]);
            if (SX == 2 && !wide) v[u] = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4 % VE], f[5 % VE]), pack_bf16(f[6 % VE], f[7 % VE]));
            if (SX == 4) v[u] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
        }
        const bool whole = alike && i0 >= 0 && i0 + VE <= it.numel;
        if (wide) {
            float* o = reinterpret_cast<float*>(it.out);
            if (whole) {
                st_vec16(o + i0, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])));
                st_vec16(o + i0 + 4, make_uint4(__float_as_uint(f[4 % VE]), __float_as_uint(f[5 % VE]), __float_as_uint(f[6 % VE]), __float_as_uint(f[7 % VE])));
            } else {
#pragma unroll
                for (int q = 0; q < VE; ++q)
                    if (i0 + q >= 0 && i0 + q < it.numel) o[i0 + q] = f[q];
            }
        } else if (whole) {
            st_vec16(it.out + i0 * SX, v[u]);
        } else {
#pragma unroll
            for (int q = 0; q < VE; ++q) {
                if (i0 + q < 0 || i0 + q >= it.numel) continue;
                if (SX == 2) reinterpret_cast<unsigned short*>(it.out)[i0 + q] = static_cast<unsigned short>(word_of(v[u], q >> 1) >> (16 * (q & 1)));
                else reinterpret_cast<unsigned*>(it.out)[i0 + q] = word_of(v[u], q);
            }
        }
    }
}

template <int N>
__global__ void __launch_bounds__(kClipThreads, kClipCtas) scale_kernel(const __grid_constant__ ClipList<N> a) {
    __shared__ double s_part[kClipWarps];
    __shared__ float s_c;
    const int tid = threadIdx.x;
    pdl_wait();
    double sum = 0.0;
    for (int k = tid; k < a.n_shares; k += kClipThreads) sum += a.shares[k];
    sum = warp_sum_d(sum);
    if ((tid & 31) == 0) s_part[tid >> 5] = sum;
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kClipWarps; ++w) sum += s_part[w];
        const double n = sqrt(sum);
        const float norm = static_cast<float>(n);
        const bool finite = norm < INFINITY;
        s_c = finite && n > static_cast<double>(a.max_norm) ? static_cast<float>(static_cast<double>(a.max_norm) / n) : 1.f;
        if (a.write_norm && blockIdx.x == 0) {
            *a.norm = norm;
            *a.status = finite ? 0 : DSPARK_ROW_NONFINITE;
        }
    }
    __syncthreads();
    const float c = s_c;
    const int j0 = static_cast<int>(static_cast<long long>(a.chunks) * blockIdx.x / gridDim.x);
    const int j1 = static_cast<int>(static_cast<long long>(a.chunks) * (blockIdx.x + 1) / gridDim.x);
    if (j0 >= j1) return;
    int i = item_of(a, j0);
    for (int j = j0; j < j1; ++j) {
        while (i + 1 < a.n && a.item[i + 1].first <= j) ++i;
        const ClipItem& it = a.item[i];
        if (c == 1.f && it.out == it.grad) continue;
        if (it.bf16) scale_chunk<2>(it, j - it.first, c);
        else scale_chunk<4>(it, j - it.first, c);
    }
}

int groups_of(int n) { return (n + kLargeList - 1) / kLargeList; }

dspark_status_t check_list(const dspark_grad_t* grads, int n) {
    for (int i = 0; i < n; ++i) {
        const dspark_grad_t& g = grads[i];
        if (g.numel < 0 || (g.dtype != DSPARK_BF16 && g.dtype != DSPARK_FP32)) return DSPARK_ERR_INVALID_ARG;
        if (g.out_dtype != g.dtype && g.out_dtype != DSPARK_FP32) return DSPARK_ERR_INVALID_ARG;
        if (g.numel == 0) continue;
        if (g.numel > (1LL << 43)) return DSPARK_ERR_UNSUPPORTED;   // 2^31 chunks of an fp32 list
        const size_t sx = g.dtype == DSPARK_BF16 ? 2 : 4, so = g.out_dtype == DSPARK_BF16 ? 2 : 4;
        if (!g.grad || !g.out || reinterpret_cast<uintptr_t>(g.grad) % sx || reinterpret_cast<uintptr_t>(g.out) % so)
            return DSPARK_ERR_INVALID_ARG;
        if (g.grad == g.out && g.dtype != g.out_dtype) return DSPARK_ERR_INVALID_ARG;
    }
    return DSPARK_OK;
}

// Fill the list with the group's tensors; false when it has too many chunks.
template <int N>
bool fill(ClipList<N>& a, const dspark_grad_t* grads, int n) {
    long long chunks = 0;
    a.n = 0;
    for (int i = 0; i < n; ++i) {
        const dspark_grad_t& g = grads[i];
        if (g.numel == 0) continue;
        const int sx = g.dtype == DSPARK_BF16 ? 2 : 4;
        const long long a0 = static_cast<long long>(reinterpret_cast<uintptr_t>(g.grad) & 15u) / sx;
        const long long nvec = (a0 + g.numel + 16 / sx - 1) / (16 / sx);
        a.item[a.n++] = ClipItem{static_cast<const unsigned char*>(g.grad), static_cast<unsigned char*>(g.out), g.numel,
                                 static_cast<int>(chunks), g.dtype == DSPARK_BF16, g.out_dtype != g.dtype};
        chunks += (nvec + kChunk - 1) / kChunk;
        if (chunks > 0x7fffffffLL) return false;
    }
    a.chunks = static_cast<int>(chunks);
    return true;
}

template <int N>
dspark_status_t clip(const dspark_grad_t* grads, int n, float max_norm, float* norm, int* status, double* shares, int most, cudaStream_t s) {
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
            const int grid = std::max(1, std::min(a.chunks, most));
            a.shares = pass == 0 ? shares + done : shares;
            a.n_shares = total;
            a.write_norm = k == 0;
            done += grid;
            const bool skip = pass == 1 && k > 0 && a.chunks == 0;
            if (!skip && launch_k(pass == 0 ? norm_kernel<N> : scale_kernel<N>, dim3(static_cast<unsigned>(grid)), dim3(kClipThreads), 0, s,
                                  true, a) != cudaSuccess)
                return DSPARK_ERR_CUDA;
        }
        total = done;
    }
    return DSPARK_OK;
}

}  // namespace
}  // namespace dspark

using namespace dspark;

extern "C" {

size_t dspark_clip_workspace_bytes(int32_t n_grads) {
    if (n_grads < 1 || n_grads > DSPARK_MAX_GRADS) return 0;
    return static_cast<size_t>(groups_of(n_grads)) * kMaxShares * sizeof(double);
}

dspark_status_t dspark_clip_grads(const dspark_grad_t* grads, int32_t n_grads, float max_norm, float* out_norm, int32_t* out_status,
                                  void* workspace, size_t workspace_bytes, void* stream) {
    if (!grads || n_grads < 1 || n_grads > DSPARK_MAX_GRADS || !(max_norm >= 0.f) || !out_norm || !out_status) return DSPARK_ERR_INVALID_ARG;
    if (const dspark_status_t st = check_list(grads, n_grads); st != DSPARK_OK) return st;
    if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 || workspace_bytes < dspark_clip_workspace_bytes(n_grads))
        return DSPARK_ERR_WORKSPACE;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return DSPARK_ERR_CUDA;
    const int most = std::min(kMaxShares, sms * kClipCtas);
    double* const shares = static_cast<double*>(workspace);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return n_grads <= kSmallList ? clip<kSmallList>(grads, n_grads, max_norm, out_norm, out_status, shares, most, s)
                                 : clip<kLargeList>(grads, n_grads, max_norm, out_norm, out_status, shares, most, s);
}

}  // extern "C"
