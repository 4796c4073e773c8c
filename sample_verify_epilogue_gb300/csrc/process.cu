// process_kernel: repetition, presence and frequency penalties, biases and grammar masks on the
// logits of every verify position, one launch.
//
// y = rule(x) is an elementwise copy with a mask (bandwidth) plus, for the few tokens of the
// request's lists, an exact value of its own.  A CTA takes one or more tiles of kProcVec 16-byte vectors per
// thread of one row: it copies them under the mask's bits, then its threads write the listed tokens
// of that span, found by a 32-way search in the sorted lists while the first tile was on its way.
// A listed token is written by exactly one list (history before drafts before biases), with what
// the other lists say about it looked up, so that it is rounded once.  A vector that the mask
// empties is not read; in place, a vector that the mask leaves whole is neither read nor written.
//
// Without lists the copy runs at 0.99 of the measured bandwidth (64x9 rows of 262144 bf16, no
// masks: 90 us); the 1700 listed tokens of a row add 10 us of scattered two-byte stores, 13 us where masks
// shorten the copy (30 with loads and stores that pass the L1 cache by).  Taking the tokens through shared
// memory into the vectors before they are stored costs more than that, in barriers for every tile or in what
// the first store waits for (104 to 130 us where this takes 89), and so does a warp to a span without
// barriers (117 us).
//
// The first B CTAs check one request each (parameters, list order and ranges, draft ids, mask
// rows) and write its status; they run beside the copying CTAs, whose own range checks keep every
// access in bounds whatever the offsets and lists hold.
#include "vocab_rows.cuh"

namespace dspark {

namespace {

constexpr int kProcVec = 4;                                  // vectors per thread
constexpr int kProcHist = 512, kProcBias = kRowThreads;      // listed tokens of a span held in shared memory
constexpr int kProcTile = kProcVec * kRowThreads;            // vectors of a tile

struct ProcArgs {
    int B, Km, V, spans, span;                               // CTAs to a row, their vectors
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
    int n_mask, h_nnz, b_nnz;
    int in_place;
    int* row_status;
};

// First index in [lo, hi) whose id is at least key; the whole warp searches.  Each step keeps one
// of 33 parts, so the range shrinks whatever the ids hold.
__device__ int warp_lower_bound(const int* ids, int lo, int hi, int key) {
    const int lane = threadIdx.x & 31;
    while (hi - lo > 32) {
        const int part = static_cast<int>(static_cast<unsigned>(hi - lo) / 33u);
        const int n = __popc(__ballot_sync(0xffffffffu, ids[lo + part * (lane + 1)] < key));
        if (n < 32) hi = lo + part * (n + 1);
        if (n > 0) lo += part * n + 1;
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
        if (lo < 0 || hi < lo || hi > a.h_nnz) st |= DSPARK_ROW_BAD_HISTORY;
        else
            for (int e = lo + tid; e < hi; e += kRowThreads) {
                const int t = a.h_ids[e];
                if (t < 0 || t >= a.V || (e > lo && a.h_ids[e - 1] >= t) || a.h_cnt[e] < 0) st |= DSPARK_ROW_BAD_HISTORY;
            }
    }
    if (a.b_off) {
        const int lo = a.b_off[b], hi = a.b_off[b + 1];
        if (lo < 0 || hi < lo || hi > a.b_nnz) st |= DSPARK_ROW_BAD_BIAS;
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
        if (a.mask || a.mask_rows)                           // (mask rows of no mask: all have to be -1)
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

// -inf in the lanes whose bit is 0.
template <int SX>
__device__ __forceinline__ void mask_vec(uint4& w, unsigned bits) {
    if (SX == 2) {
#pragma unroll
        for (int h = 0; h < 4; ++h) {                        // two bits to a word's halves
            uint32_t& x = h == 0 ? w.x : h == 1 ? w.y : h == 2 ? w.z : w.w;
            const uint32_t keep = ((bits >> (2 * h)) * 0x8001u & 0x00010001u) * 0xFFFFu;
            x = (x & keep) | (0xFF80FF80u & ~keep);
        }
    } else {
        if (!(bits & 1u)) w.x = ninf_bits<SX>();
        if (!(bits & 2u)) w.y = ninf_bits<SX>();
        if (!(bits & 4u)) w.z = ninf_bits<SX>();
        if (!(bits & 8u)) w.w = ninf_bits<SX>();
    }
}

template <int SX>
__global__ void __launch_bounds__(kRowThreads, 6) process_kernel(ProcArgs a) {
    constexpr int VE = VocabRow<SX>::VE;
    pdl_wait();                                              // what came before in the stream
    if (blockIdx.x < static_cast<unsigned>(a.B)) {
        check_request(a, static_cast<int>(blockIdx.x));
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5;
    const unsigned item = blockIdx.x - static_cast<unsigned>(a.B);
    const int row = static_cast<int>(item / a.spans), part = static_cast<int>(item % a.spans);
    const int W = a.Km + 1, b = row / W, j = row - b * W;
    const dspark_process_row_t r = a.rows[b];
    if (!proc_row_ok(r, a.Km) || j > r.num_drafts) return;

    const VocabRow<SX> x(a.x, row, a.x_stride, a.V);
    const VocabRow<SX> y(a.y, row, a.y_stride, a.V);
    const int k0 = part * a.span, k1 = min(x.nvec, k0 + a.span);
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
    __shared__ int s_hid[kProcHist], s_bid[kProcBias];       // the lists' part in this span, where it fits
    __shared__ float s_bval[kProcBias];
    const int nd = penal && a.d ? j : 0;
    // The list ranges, by four warps; called while a warp's first tile is on its way.
    auto search = [&]() {
        if (warp >= 4) {
            if (tid - 4 * 32 < nd) s_d[tid - 4 * 32] = a.d[static_cast<long long>(b) * a.Km + tid - 4 * 32];
            return;
        }
        const int* off = warp < 2 ? (penal ? a.h_off : nullptr) : a.b_off;
        const int* ids = warp < 2 ? a.h_ids : a.b_ids;
        int at = 0;
        if (off) {
            const int lo = off[b], hi = off[b + 1];
            if (lo >= 0 && hi > lo && hi <= (warp < 2 ? a.h_nnz : a.b_nnz)) at = warp_lower_bound(ids, lo, hi, (warp & 1) ? i_hi : i_lo);
        }
        if ((tid & 31) == 0) s_at[warp] = at;
    };

    // the copy under the mask
    const bool same_phase = x.a0 == y.a0;
    unsigned char* const yp = const_cast<unsigned char*>(y.p);
    constexpr unsigned kAll = (1u << VE) - 1u;
    auto one = [&](int k) {
        const int i0 = x.first(k);
        const unsigned bits = m ? mask_bits<VE>(m, words, i0) : kAll;
        if (a.in_place && bits == kAll) return;
        uint4 w = ninf_vec<SX>();
        if (bits) {
            w = load_vec<SX>(x, k, k1);
            if (bits != kAll) mask_vec<SX>(w, bits);
        }
        if (x.whole(k) && same_phase) {
            st_vec16(yp + static_cast<long long>(i0) * SX, w);
            return;
        }
#pragma unroll
        for (int q = 0; q < VE; ++q) {
            const int i = i0 + q;
            if (i < 0 || i >= a.V) continue;
            if (SX == 2) reinterpret_cast<unsigned short*>(yp)[i] = static_cast<unsigned short>(word_of(w, q >> 1) >> (16 * (q & 1)));
            else reinterpret_cast<unsigned*>(yp)[i] = word_of(w, q);
        }
    };
    if (same_phase) {
        // whole vectors, a tile's loads before its stores.  From one of a thread's vectors to the next the
        // mask's bits stand at one place of a word (or of two), 8 VE words on.
        const int w0 = k0 + !x.whole(k0), w1 = max(w0, k1 - !x.whole(k1 - 1));
        const int i0 = x.first(w0 + tid), sh = i0 & 31;
        const unsigned* mp = m ? m + (i0 >> 5) : nullptr;
        const int over = sh + VE > 32 ? 1 : 0;
        const long long at = static_cast<long long>(i0) * SX;
        const unsigned char* xp = x.p + at;
        unsigned char* dp = yp + at;
        const bool in_place = a.in_place != 0;
        bool searched = false;
        // (a warp goes on together: search() is its work as a whole)
        for (int left = w1 - w0 - tid; left + (tid & 31) > 0; left -= kProcTile) {
            unsigned bits[kProcVec], more[kProcVec];
            uint4 w[kProcVec];
#pragma unroll
            for (int u = 0; u < kProcVec; ++u) {
                const bool here = u * kRowThreads < left;
                const unsigned* q = mp + u * (kRowThreads * VE / 32);
                bits[u] = here ? (m ? __ldg(q) : ~0u) : 0u;
                more[u] = here && over ? (m ? __ldg(q + 1) : ~0u) : 0u;
            }
#pragma unroll
            for (int u = 0; u < kProcVec; ++u) bits[u] = __funnelshift_r(bits[u], more[u], sh) & kAll;
#pragma unroll
            for (int u = 0; u < kProcVec; ++u) {
                w[u] = ninf_vec<SX>();
                if (bits[u] && !(in_place && bits[u] == kAll)) w[u] = ld_vec16(xp + u * (16 * kRowThreads));
            }
            if (!searched) search();
            searched = true;
#pragma unroll
            for (int u = 0; u < kProcVec; ++u) {
                if (u * kRowThreads >= left || (in_place && bits[u] == kAll)) continue;
                if (bits[u] != kAll) mask_vec<SX>(w[u], bits[u]);
                st_vec16(dp + u * (16 * kRowThreads), w[u]);
            }
            xp += 16 * kProcTile;
            dp += 16 * kProcTile;
            mp += kProcTile * VE / 32;
        }
        if (!searched) search();
        if (tid == 0 && w0 > k0) one(k0);                    // the row's ragged first and last
        if (tid == 32 && w1 < k1 && w1 >= w0 && k1 - 1 >= w0) one(k1 - 1);
    } else {
        search();
        for (int k = k0 + tid; k < k1; k += kRowThreads) one(k);
    }
    __syncthreads();

    // the listed tokens of this span (in place their logit still stands: the copy above wrote the
    // same value or -inf): history entries, then biases, then drafts.  The loads of a thread's first
    // token do not wait for the look-ups in the other lists.
    const int hs = s_at[0], nh = max(0, s_at[1] - hs), bs = s_at[2], nb = max(0, s_at[3] - bs);
    const int count = nh + nb + nd;
    if (count == 0) return;
    const bool staged = nh <= kProcHist && nb <= kProcBias;
    auto find_h = [&](int tok) { return staged ? find(s_hid, 0, nh, tok) : find(a.h_ids, hs, hs + nh, tok); };
    struct Item {
        int tok, cnt;
        unsigned allowed;
        float raw;
    };
    auto load = [&](int e) {
        Item t{-1, 0, ~0u, 0.f};
        if (e < nh) {
            t.tok = a.h_ids[hs + e];
            t.cnt = a.h_cnt[hs + e];
        } else if (e < nh + nb) {
            t.tok = a.b_ids[bs + e - nh];
        } else if (e < count) {
            t.tok = s_d[e - nh - nb];
        }
        if (t.tok >= i_lo && t.tok < i_hi) {
            if (m) t.allowed = m[t.tok >> 5] >> (t.tok & 31);
            t.raw = load_logit<SX>(x, t.tok);
        } else {
            t.allowed = 0u;
        }
        return t;
    };
    auto finish = [&](int e, const Item& t) {
        if (!(t.allowed & 1u)) return;
        int n = 0, first = nd;
        for (int i = nd - 1; i >= 0; --i)
            if (s_d[i] == t.tok) { ++n; first = i; }
        float v = t.raw, bias = 0.f;
        bool biased = false;
        if (e < nh || e >= nh + nb) {
            if (e >= nh && (first != e - nh - nb || find_h(t.tok) >= 0)) return;
            v = v > 0.f ? __fdiv_rn(v, r.repetition_penalty) : __fmul_rn(v, r.repetition_penalty);
            v = penalise(v, t.cnt + n, r.frequency_penalty, r.presence_penalty);
            if (nb) {
                const int k = staged ? find(s_bid, 0, nb, t.tok) : find(a.b_ids, bs, bs + nb, t.tok);
                biased = k >= 0;
                if (biased) bias = staged ? s_bval[k] : a.b_val[k];
            }
        } else {
            if (n || find_h(t.tok) >= 0) return;
            biased = true;
            bias = staged ? s_bval[e - nh] : a.b_val[bs + e - nh];
        }
        if (biased) v = __fadd_rn(v, bias);
        if (SX == 2) reinterpret_cast<unsigned short*>(yp)[t.tok] = static_cast<unsigned short>(to_bits<SX>(v));
        else reinterpret_cast<float*>(yp)[t.tok] = v;
    };
    const Item mine = load(tid);
    if (staged) {
        for (int i = tid; i < nh; i += kRowThreads) s_hid[i] = i == tid ? mine.tok : a.h_ids[hs + i];
        if (tid < nb) {
            s_bid[tid] = a.b_ids[bs + tid];
            s_bval[tid] = a.b_val[bs + tid];
        }
        __syncthreads();
    }
    finish(tid, mine);
    for (int e = tid + kRowThreads; e < count; e += kRowThreads) finish(e, load(e));
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
    if (reinterpret_cast<uintptr_t>(p->rows) % 4) return DSPARK_ERR_INVALID_ARG;   // (bytes, in the binding)
    if (out == logits && p->out_stride != p->logits_stride) return DSPARK_ERR_INVALID_ARG;
    if (history && history->row_offsets && (!history->token_ids || !history->counts)) return DSPARK_ERR_INVALID_ARG;
    if (bias && bias->row_offsets && (!bias->token_ids || !bias->biases)) return DSPARK_ERR_INVALID_ARG;
    if (p->history_nnz < 0 || p->bias_nnz < 0) return DSPARK_ERR_INVALID_ARG;
    if (mask && mask->words) {
        if (mask->n_rows < 1 || mask->words_stride < (p->V + 31) / 32) return DSPARK_ERR_INVALID_ARG;
        if (reinterpret_cast<uintptr_t>(mask->words) % 4) return DSPARK_ERR_INVALID_ARG;
        if (!mask->rows && mask->n_rows < p->B * (p->K_max + 1)) return DSPARK_ERR_INVALID_ARG;
    } else if (mask && mask->n_rows != 0) {
        return DSPARK_ERR_INVALID_ARG;
    }

    ProcArgs a{};
    a.B = p->B; a.Km = p->K_max; a.V = p->V;
    a.x_stride = p->logits_stride; a.y_stride = p->out_stride;
    a.x = logits; a.y = out; a.rows = p->rows; a.d = draft_ids;
    a.h_nnz = p->history_nnz; a.b_nnz = p->bias_nnz;
    if (history && history->row_offsets) { a.h_off = history->row_offsets; a.h_ids = history->token_ids; a.h_cnt = history->counts; }
    if (bias && bias->row_offsets) { a.b_off = bias->row_offsets; a.b_ids = bias->token_ids; a.b_val = bias->biases; }
    if (mask) { a.mask = mask->words; a.mask_stride = mask->words_stride; a.mask_rows = mask->rows; a.n_mask = mask->n_rows; }
    a.in_place = out == logits;
    a.row_status = p->row_status;
    // Tiles per CTA: a CTA's chain of list and mask look-ups is worth a few tiles, so more than one where
    // that leaves CTAs enough.  18432 tiles: 94 us in twos, 89 in fours, 94 in sixes; 1520 tiles:
    // 12.4 us one by one, 11.2 in twos, 12.6 in fours; 684 tiles: 7.1, 7.7, 8.0 us.
    const bool aligned = reinterpret_cast<uintptr_t>(logits) % 16 == 0 && p->logits_stride * sx % 16 == 0;
    const int nvec = aligned ? (p->V + 16 / sx - 1) / (16 / sx) : max_vectors(p->V, sx);
    const int tiles = (nvec + kProcTile - 1) / kProcTile;
    const long long rows = static_cast<long long>(p->B) * (p->K_max + 1);
    const int per = rows * tiles >= 8000 ? 4 : rows * tiles >= 1200 ? 2 : 1;
    a.spans = (tiles + per - 1) / per;
    a.span = per * kProcTile;
    const long long grid = p->B + rows * a.spans;
    if (grid > 0x7fffffffLL) return DSPARK_ERR_UNSUPPORTED;
    cudaStream_t s = static_cast<cudaStream_t>(p->stream);
    const dim3 g(static_cast<unsigned>(grid)), t(kRowThreads);
    const cudaError_t e = sx == 2 ? launch_k(process_kernel<2>, g, t, 0, s, true, a)
                                  : launch_k(process_kernel<4>, g, t, 0, s, true, a);
    return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}
