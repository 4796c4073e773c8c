// process_kernel: repetition, presence and frequency penalties, biases and grammar masks on the
// logits of every verify position, one launch.
//
// y = rule(x) is an elementwise copy with a mask (bandwidth) plus, for the few tokens of the
// request's lists, an exact value of its own.  A CTA takes kProcVec 16-byte vectors per thread
// of one row: it copies them under the mask's bits, then its threads write the listed tokens of
// that span, found by a 32-way search in the sorted lists.  A listed token is written by
// exactly one list (history before drafts before biases), with what the other lists say about it
// looked up, so that it is rounded once.  A vector that the mask empties is not read; in place, a
// vector that the mask leaves whole is neither read nor written.
//
// The first B CTAs check one request each (parameters, list order and ranges, draft ids, mask
// rows) and write its status; they run beside the copying CTAs, whose own range checks keep every
// access in bounds whatever the lists hold.
#include "vocab_rows.cuh"

namespace dspark {

namespace {

constexpr int kProcVec = 4;                                  // vectors per thread
constexpr int kProcSpan = kProcVec * kRowThreads;            // vectors per CTA

struct ProcArgs {
    int B, Km, V, tiles;
    long long x_stride, y_stride, mask_stride;
    const void* x;
    void* y;
    const dspark_process_row_t* rows;
    const int* d;
    const int *h_off, *h_ids, *h_cnt;
    const int *b_off, *b_ids;
    const float* b_val;
    const unsigned* mask;
    const int* mask_rows;
    int n_mask;
    int in_place;
    int* row_status;
};

// First index in [lo, hi) whose id is at least key; the whole warp searches.  Each step keeps one
// of 33 parts, so the range shrinks whatever the ids hold.
__device__ int warp_lower_bound(const int* ids, int lo, int hi, int key) {
    const int lane = threadIdx.x & 31;
    while (hi - lo > 32) {
        const long long len = hi - lo;
        const int mine = lo + static_cast<int>(len * (lane + 1) / 33);
        const int n = __popc(__ballot_sync(0xffffffffu, ids[mine] < key));
        const int below = lo + static_cast<int>(len * n / 33);
        const int above = lo + static_cast<int>(len * (n + 1) / 33);
        if (n < 32) hi = above;
        if (n > 0) lo = below + 1;
    }
    const bool less = lo + lane < hi && ids[lo + lane] < key;
    return lo + __popc(__ballot_sync(0xffffffffu, less));
}

// Index of key in ids[lo, hi), or -1.
__device__ __forceinline__ int find(const int* ids, int lo, int hi, int key) {
    const int end = hi;
    while (lo < hi) {
        const int m = lo + ((hi - lo) >> 1);
        if (ids[m] < key) lo = m + 1; else hi = m;
    }
    return lo < end && ids[lo] == key ? lo : -1;
}

__device__ __forceinline__ bool proc_row_ok(const dspark_process_row_t& r, int Km) {
    return r.repetition_penalty > 0.f && isfinite(r.repetition_penalty) && isfinite(r.presence_penalty) &&
           isfinite(r.frequency_penalty) && r.num_drafts >= 0 && r.num_drafts <= Km;
}

// Status of request b: the whole block looks through its lists.
__device__ void check_request(const ProcArgs& a, int b) {
    const int tid = threadIdx.x;
    const dspark_process_row_t r = a.rows[b];
    const bool ok = proc_row_ok(r, a.Km);
    int st = ok ? 0 : DSPARK_ROW_BAD_PARAMS;
    if (a.h_off) {
        const int lo = a.h_off[b], hi = a.h_off[b + 1];
        if (lo < 0 || hi < lo) st |= DSPARK_ROW_BAD_HISTORY;
        else
            for (int e = lo + tid; e < hi; e += kRowThreads) {
                const int t = a.h_ids[e];
                if (t < 0 || t >= a.V || (e > lo && a.h_ids[e - 1] >= t) || a.h_cnt[e] < 0) st |= DSPARK_ROW_BAD_HISTORY;
            }
    }
    if (a.b_off) {
        const int lo = a.b_off[b], hi = a.b_off[b + 1];
        if (lo < 0 || hi < lo) st |= DSPARK_ROW_BAD_BIAS;
        else
            for (int e = lo + tid; e < hi; e += kRowThreads) {
                const int t = a.b_ids[e];
                if (t < 0 || t >= a.V || (e > lo && a.b_ids[e - 1] >= t) || !(a.b_val[e] < INFINITY)) st |= DSPARK_ROW_BAD_BIAS;
            }
    }
    if (ok) {
        if (a.d)
            for (int i = tid; i < r.num_drafts; i += kRowThreads) {
                const int t = a.d[static_cast<long long>(b) * a.Km + i];
                if (t < 0 || t >= a.V) st |= DSPARK_ROW_BAD_DRAFT;
            }
        if (a.mask)
            for (int j = tid; j <= r.num_drafts; j += kRowThreads) {
                const int row = b * (a.Km + 1) + j, k = a.mask_rows ? a.mask_rows[row] : row;
                if (k < -1 || k >= a.n_mask) st |= DSPARK_ROW_BAD_MASK;
            }
    }
    st = __reduce_or_sync(0xffffffffu, static_cast<unsigned>(st));
    __shared__ int s_st[kRowWarps];
    if ((tid & 31) == 0) s_st[tid >> 5] = st;
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kRowWarps; ++w) st |= s_st[w];
        a.row_status[b] = st;
    }
}

// Mask bits of the VE tokens from i0 on (i0 may be negative; bits outside the row are junk).
template <int VE>
__device__ __forceinline__ unsigned mask_bits(const unsigned* m, int words, int i0) {
    const int w = i0 >> 5, sh = i0 & 31;                     // arithmetic shift: floor
    unsigned lo = w >= 0 && w < words ? __ldg(m + w) : 0u;
    unsigned bits = lo >> sh;
    if (sh + VE > 32 && w + 1 < words) bits |= __ldg(m + w + 1) << (32 - sh);
    return bits & ((1u << VE) - 1u);
}

template <int SX>
__global__ void __launch_bounds__(kRowThreads) process_kernel(ProcArgs a) {
    constexpr int VE = VocabRow<SX>::VE;
    if (blockIdx.x < static_cast<unsigned>(a.B)) {
        check_request(a, static_cast<int>(blockIdx.x));
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5;
    const unsigned item = blockIdx.x - static_cast<unsigned>(a.B);
    const int row = static_cast<int>(item / a.tiles), tile = static_cast<int>(item % a.tiles);
    const int W = a.Km + 1, b = row / W, j = row - b * W;
    const dspark_process_row_t r = a.rows[b];
    if (!proc_row_ok(r, a.Km) || j > r.num_drafts) return;

    const VocabRow<SX> x(a.x, row, a.x_stride, a.V);
    const VocabRow<SX> y(a.y, row, a.y_stride, a.V);
    const int k0 = tile * kProcSpan, k1 = min(x.nvec, k0 + kProcSpan);
    if (k0 >= k1) return;
    const int i_lo = max(0, x.first(k0)), i_hi = min(a.V, x.first(k1));
    const int words = (a.V + 31) >> 5;
    const unsigned* m = nullptr;
    if (a.mask) {
        const int k = a.mask_rows ? a.mask_rows[row] : row;
        if (k >= 0 && k < a.n_mask) m = a.mask + k * a.mask_stride;
    }
    const bool penal = r.repetition_penalty != 1.f || r.presence_penalty != 0.f || r.frequency_penalty != 0.f;

    __shared__ int s_at[4];                                  // list ranges of this span: history, biases
    __shared__ int s_d[DSPARK_MAX_K];
    const int nd = penal && a.d ? j : 0;
    if (tid >= 4 * 32 && tid - 4 * 32 < nd) s_d[tid - 4 * 32] = a.d[static_cast<long long>(b) * a.Km + tid - 4 * 32];
    if (warp < 4) {
        const int* off = warp < 2 ? (penal ? a.h_off : nullptr) : a.b_off;
        const int* ids = warp < 2 ? a.h_ids : a.b_ids;
        int at = 0;
        if (off) {
            const int lo = off[b], hi = off[b + 1];
            if (lo >= 0 && hi > lo) at = warp_lower_bound(ids, lo, hi, (warp & 1) ? i_hi : i_lo);
        }
        if ((tid & 31) == 0) s_at[warp] = at;
    }

    // the copy under the mask, every load before the first store
    const bool same_phase = x.a0 == y.a0;
    unsigned char* const yp = const_cast<unsigned char*>(y.p);
    constexpr unsigned kAll = (1u << VE) - 1u;
    unsigned bits[kProcVec];
    uint4 w[kProcVec];
#pragma unroll
    for (int u = 0; u < kProcVec; ++u) {
        const int k = k0 + u * kRowThreads + tid;
        bits[u] = m && k < k1 ? mask_bits<VE>(m, words, x.first(k)) : kAll;
    }
#pragma unroll
    for (int u = 0; u < kProcVec; ++u) {
        const int k = k0 + u * kRowThreads + tid;
        const bool keep = a.in_place && bits[u] == kAll;
        w[u] = bits[u] && !keep ? load_vec<SX>(x, k, k1) : ninf_vec<SX>();
    }
#pragma unroll
    for (int u = 0; u < kProcVec; ++u) {
        const int k = k0 + u * kRowThreads + tid;
        if (k >= k1 || (a.in_place && bits[u] == kAll)) continue;
        if (bits[u] != kAll && bits[u]) {
            if (SX == 2) {
                // two bits to a word's halves: 0xFFFF where the token is kept
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    uint32_t& x2 = h == 0 ? w[u].x : h == 1 ? w[u].y : h == 2 ? w[u].z : w[u].w;
                    const unsigned two = bits[u] >> (2 * h);
                    const unsigned sel = ((two & 1u) * 0xFFFFu) | ((two & 2u) * 0x7FFF8000u);
                    x2 = (x2 & sel) | (0xFF80FF80u & ~sel);
                }
            } else {
#pragma unroll
                for (int q = 0; q < VE; ++q)
                    if (!((bits[u] >> q) & 1u)) put_bits<SX>(w[u], q, ninf_bits<SX>());
            }
        }
        const int i0 = x.first(k);
        if (x.whole(k) && same_phase) {
            st_stream(yp + static_cast<long long>(i0) * SX, w[u]);
        } else {
#pragma unroll
            for (int q = 0; q < VE; ++q) {
                const int i = i0 + q;
                if (i < 0 || i >= a.V) continue;
                if (SX == 2) reinterpret_cast<unsigned short*>(yp)[i] = static_cast<unsigned short>(word_of(w[u], q >> 1) >> (16 * (q & 1)));
                else reinterpret_cast<unsigned*>(yp)[i] = word_of(w[u], q);
            }
        }
    }
    __syncthreads();

    // the listed tokens of this span (in place their logit still stands: the copy above wrote the
    // same value or -inf)
    const int hs = s_at[0], nh = max(0, s_at[1] - hs), bs = s_at[2], nb = max(0, s_at[3] - bs);
    for (int e = tid; e < nh + nb + nd; e += kRowThreads) {
        int tok, cnt = 0, bi = -1;
        bool seen = true;
        if (e < nh) {
            tok = a.h_ids[hs + e];
            cnt = a.h_cnt[hs + e];
        } else if (e < nh + nb) {
            bi = bs + (e - nh);
            tok = a.b_ids[bi];
            seen = false;
            if (find(a.h_ids, hs, hs + nh, tok) >= 0) continue;
        } else {
            tok = s_d[e - nh - nb];
        }
        if (tok < i_lo || tok >= i_hi) continue;
        int n = 0, first = nd;
        for (int i = nd - 1; i >= 0; --i)
            if (s_d[i] == tok) { ++n; first = i; }
        if (e >= nh + nb) {
            if (first != e - nh - nb || find(a.h_ids, hs, hs + nh, tok) >= 0) continue;
        } else if (e >= nh && n) {
            continue;
        }
        if (m && !((m[tok >> 5] >> (tok & 31)) & 1u)) continue;
        float v = load_logit<SX>(x, tok);
        if (seen) {
            v = v > 0.f ? __fdiv_rn(v, r.repetition_penalty) : __fmul_rn(v, r.repetition_penalty);
            v = penalise(v, cnt + n, r.frequency_penalty, r.presence_penalty);
            if (nb) bi = find(a.b_ids, bs, bs + nb, tok);
        }
        if (bi >= 0) v = __fadd_rn(v, a.b_val[bi]);
        if (SX == 2) reinterpret_cast<unsigned short*>(yp)[tok] = static_cast<unsigned short>(to_bits<SX>(v));
        else reinterpret_cast<float*>(yp)[tok] = v;
    }
}

}  // namespace
}  // namespace dspark

using namespace dspark;

extern "C" dspark_status_t dspark_process_logits(const void* logits, void* out, const int32_t* draft_ids,
                                                 const dspark_counts_t* history, const dspark_bias_t* bias,
                                                 const dspark_mask_t* mask, const dspark_process_params_t* p) {
    if (!p || !logits || !out || !p->rows || !p->row_status) return DSPARK_ERR_INVALID_ARG;
    if (p->B < 1 || p->B > DSPARK_MAX_B || p->K_max < 0 || p->K_max > DSPARK_MAX_K) return DSPARK_ERR_INVALID_ARG;
    if (p->V < 1 || p->V > DSPARK_MAX_V) return DSPARK_ERR_INVALID_ARG;
    if (p->logits_dtype != DSPARK_BF16 && p->logits_dtype != DSPARK_FP32) return DSPARK_ERR_INVALID_ARG;
    const int sx = p->logits_dtype == DSPARK_BF16 ? 2 : 4;
    if (p->logits_stride < p->V || p->out_stride < p->V) return DSPARK_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(logits) % sx || reinterpret_cast<uintptr_t>(out) % sx) return DSPARK_ERR_INVALID_ARG;
    if (out == logits && p->out_stride != p->logits_stride) return DSPARK_ERR_INVALID_ARG;
    if (history && history->row_offsets && (!history->token_ids || !history->counts)) return DSPARK_ERR_INVALID_ARG;
    if (bias && bias->row_offsets && (!bias->token_ids || !bias->biases)) return DSPARK_ERR_INVALID_ARG;
    if (mask && mask->words) {
        if (mask->n_rows < 1 || mask->words_stride < (p->V + 31) / 32) return DSPARK_ERR_INVALID_ARG;
        if (reinterpret_cast<uintptr_t>(mask->words) % 4) return DSPARK_ERR_INVALID_ARG;
        if (!mask->rows && mask->n_rows < p->B * (p->K_max + 1)) return DSPARK_ERR_INVALID_ARG;
    }

    ProcArgs a{};
    a.B = p->B; a.Km = p->K_max; a.V = p->V;
    a.x_stride = p->logits_stride; a.y_stride = p->out_stride;
    a.x = logits; a.y = out; a.rows = p->rows; a.d = draft_ids;
    if (history && history->row_offsets) { a.h_off = history->row_offsets; a.h_ids = history->token_ids; a.h_cnt = history->counts; }
    if (bias && bias->row_offsets) { a.b_off = bias->row_offsets; a.b_ids = bias->token_ids; a.b_val = bias->biases; }
    if (mask && mask->words) {
        a.mask = mask->words; a.mask_stride = mask->words_stride; a.mask_rows = mask->rows; a.n_mask = mask->n_rows;
    }
    a.in_place = out == logits;
    a.row_status = p->row_status;
    a.tiles = (max_vectors(p->V, sx) + kProcSpan - 1) / kProcSpan;
    const long long grid = p->B + static_cast<long long>(p->B) * (p->K_max + 1) * a.tiles;
    if (grid > 0x7fffffffLL) return DSPARK_ERR_UNSUPPORTED;
    cudaStream_t s = static_cast<cudaStream_t>(p->stream);
    const dim3 g(static_cast<unsigned>(grid)), t(kRowThreads);
    const cudaError_t e = sx == 2 ? launch_k(process_kernel<2>, g, t, 0, s, false, a)
                                  : launch_k(process_kernel<4>, g, t, 0, s, false, a);
    return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}
