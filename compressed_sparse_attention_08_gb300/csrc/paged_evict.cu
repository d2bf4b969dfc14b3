// Eviction from the paged cache by accumulated attention weight.
//
// A sequence of n > budget rows keeps its last `recent` rows and, of the ones before, the
// budget - recent of greatest weight (equal: the lower row; the rule of topk.cu, which selects
// them). The kept rows move, in order, to rows 0 .. budget - 1 of the output table's pages. The
// pages have no counterpart.
//
// Three steps: the lengths are clamped and copied (kv_len_out may be kv_len), the top-k gives
// the kept old rows in ascending order, and the move kernel carries rows, weights and the list.
// HBM bound: the kept rows are read and written once. In place, row i comes from a row >= i, so
// going through the rows upwards and reading each block of rows before writing it never reads
// a row that was overwritten; a CTA therefore takes a slice of every row's channels (their
// copies are independent) and walks all rows. Into other pages there is no such order, and
// the rows are spread over CTAs too.
// Measured, into other pages: 4 sequences of up to 64K rows x 512 cut to 32K in 70 us (the move 50
// us, 5.4 TB/s); 3 of up to 1.5K rows 12 us, three dependent launches. In place: 4 sequences of 64K
// rows 366 us (slices of 16 bytes, half a sector each), 16 of 16K rows cut to 8K 130 us (slices of
// 64 bytes), 3 of 1.5K 20 us: the walk over all rows is serial in each CTA.
#include "internal.h"
#include "paged.cuh"

namespace dsv4 {
namespace {

constexpr int kT = 256, kU = 8;

struct EvictParams {
    uint4 *k, *v;
    const int32_t *table, *out_table, *len, *n_old, *idx;
    const float* acc;
    float* acc_out;
    int32_t *keep, *kv_len_out;
    int batch, max_pages, out_pages, page_size, num_pages, acc_rows, budget, recent;
    int row16;                           // 16-byte pieces per row
    int slice;                           // pieces per CTA (in place: a slice of each row)
    int rows_cta;                        // rows per CTA
    int same;                            // the rows stay on their pages
    uint32_t* eword;
};

__global__ void __launch_bounds__(kT)
evict_plan_kernel(const int32_t* kv_len, int32_t* len, int32_t* n_old, int32_t* kv_len_out, int batch, int cap, int budget,
                  int recent, uint32_t* eword, uint4* zero, size_t zero16) {
    __shared__ uint32_t err;
    pdl_trigger();
    pdl_wait();
    if (blockIdx.x > 0) {                // the top-k's counts
        for (size_t i = (blockIdx.x - 1) * kT + threadIdx.x; i < zero16; i += static_cast<size_t>(gridDim.x - 1) * kT)
            zero[i] = make_uint4(0, 0, 0, 0);
        return;
    }
    if (threadIdx.x == 0) err = 0;
    __syncthreads();
    for (int s = threadIdx.x; s < batch; s += kT) {
        const int n = kv_len[s], m = min(max(n, 0), cap);
        if (m != n) atomicOr(&err, DSV4_EWORD_BAD_INDEX);
        len[s] = m;
        n_old[s] = max(m - recent, 0);
        kv_len_out[s] = min(m, budget);
    }
    __syncthreads();
    if (threadIdx.x == 0) *eword = err;
}

// Grid: (slices x pools, row blocks, batch). A CTA takes kRows rows at a time: the places of the
// rows first (their pages are looked up once per row, by a thread of its own), then every load of
// the block, then its stores. Few registers, so that many CTAs' loads are in flight (with the
// places worked out by every thread the copy ran at 3 TB/s).
// In place a CTA goes through all rows of its slice of the channels, a larger block at a time.
template <bool IN_PLACE> constexpr int kRows = IN_PLACE ? 512 : 64;
template <bool IN_PLACE>
__global__ void __launch_bounds__(kT)
evict_move_kernel(const __grid_constant__ EvictParams p) {
    constexpr int R = kRows<IN_PLACE>, RT = (R + kT - 1) / kT;      // rows of a block, per thread
    __shared__ long long s_src[R], s_dst[R];
    const int tid = threadIdx.x, b = blockIdx.z;
    const int slices = (p.row16 + p.slice - 1) / p.slice;
    const int pool = blockIdx.x / slices, sl = blockIdx.x - pool * slices;
    pdl_trigger();
    pdl_wait();
    const int len = p.len[b], n_old = p.n_old[b], k_old = p.budget - p.recent;
    const int kept_old = min(n_old, k_old), kept = kept_old + (len - n_old);
    const int r0 = static_cast<int>(blockIdx.y) * p.rows_cta, r1 = min(r0 + p.rows_cta, kept);
    const bool lists = pool == 0 && sl == 0;            // this CTA also moves the weights and writes the list
    uint4* rows = pool ? p.v : p.k;
    const int per = kT / p.slice;                       // rows per step
    const int sub = tid / p.slice, col = sl * p.slice + tid % p.slice;
    const bool mine = sub < per && col < p.row16;
    for (int base = r0; base < r1; base += R) {
        int src[RT];
        float w[RT];
#pragma unroll
        for (int k = 0; k < RT; ++k) {
            const int j = tid + k * kT, i = base + j;
            src[k] = -1;
            if (j >= R) continue;
            long long from = -1, to = -1;
            if (i < r1) {
                const int s = i < kept_old ? p.idx[static_cast<size_t>(b) * (k_old > 0 ? k_old : 1) + i] : n_old + i - kept_old;
                if (static_cast<unsigned>(s) >= static_cast<unsigned>(len)) {   // (a NaN weight: no choice of rows)
                    flag_error(p.eword, DSV4_EWORD_BAD_INDEX);
                    s_src[j] = s_dst[j] = -1;
                    if (lists) p.keep[static_cast<size_t>(b) * p.budget + i] = -1;
                    continue;
                }
                src[k] = s;
                if (lists) w[k] = p.acc[static_cast<size_t>(b) * p.acc_rows + s];
                if (!(IN_PLACE && p.same && s == i)) {
                    const int pi = s / p.page_size, po = i / p.page_size;
                    const int a = p.table[static_cast<size_t>(b) * p.max_pages + pi];
                    const int c = p.out_table[static_cast<size_t>(b) * p.out_pages + po];
                    if (a < 0 || a >= p.num_pages || c < 0 || c >= p.num_pages) {
                        flag_error(p.eword, DSV4_EWORD_BAD_INDEX);
                    } else {
                        from = (static_cast<long long>(a) * p.page_size + s - pi * p.page_size) * p.row16;
                        to = (static_cast<long long>(c) * p.page_size + i - po * p.page_size) * p.row16;
                    }
                }
            }
            s_src[j] = from;
            s_dst[j] = to;
        }
        __syncthreads();
        for (int j0 = 0; j0 < R; j0 += per * kU) {
            uint4 x[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int j = j0 + u * per + sub;
                if (mine && j < R && s_src[j] >= 0) x[u] = rows[s_src[j] + col];
            }
            if (IN_PLACE) __syncthreads();              // these rows are read (the ones after lie further up)
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int j = j0 + u * per + sub;
                if (mine && j < R && s_src[j] >= 0) rows[s_dst[j] + col] = x[u];
            }
        }
        if (lists) {                                    // (in place: every weight of the block is read by now)
#pragma unroll
            for (int k = 0; k < RT; ++k) {
                const int i = base + tid + k * kT;
                if (src[k] < 0) continue;
                p.acc_out[static_cast<size_t>(b) * p.acc_rows + i] = w[k];
                p.keep[static_cast<size_t>(b) * p.budget + i] = src[k];
            }
        }
        __syncthreads();
    }
    if (lists) {
        const int e = min(r0 + p.rows_cta, p.budget);
        for (int i = max(r0, kept) + tid; i < e; i += kT) p.keep[static_cast<size_t>(b) * p.budget + i] = -1;
    }
}

struct Layout { size_t len, n_old, idx, topk, end; };
Layout layout(const dsv4_paged_evict_args& a) {
    Layout l{};
    size_t o = 0;
    l.len = o;
    o = align_up(o + static_cast<size_t>(a.batch) * 4, 256);
    l.n_old = o;
    o = align_up(o + static_cast<size_t>(a.batch) * 4, 256);
    l.idx = o;
    const int k = a.budget - a.recent;
    o = align_up(o + static_cast<size_t>(a.batch) * (k > 0 ? k : 1) * 4, 256);
    l.topk = o;
    if (k > 0) o += topk_ws_bytes(a.batch, a.acc_rows, k);
    l.end = o;
    return l;
}

}  // namespace

size_t paged_evict_ws_bytes(const dsv4_paged_evict_args& a) { return layout(a).end; }

int launch_paged_evict(const dsv4_paged_evict_args& a, uint8_t* ws, uint32_t* eword, cudaStream_t st) {
    if (a.batch == 0) return cudaMemsetAsync(eword, 0, 4, st) == cudaSuccess ? DSV4_OK : DSV4_ERR_LAUNCH;
    const Layout l = layout(a);
    const int k = a.budget - a.recent;
    const long long rows_in = static_cast<long long>(a.max_pages) * a.page_size;
    EvictParams p{};
    p.k = static_cast<uint4*>(a.k_pages);
    p.v = static_cast<uint4*>(a.v_pages);
    p.table = a.block_table;
    p.out_table = a.out_table;
    int32_t* len = reinterpret_cast<int32_t*>(ws + l.len);
    int32_t* n_old = reinterpret_cast<int32_t*>(ws + l.n_old);
    int32_t* idx = reinterpret_cast<int32_t*>(ws + l.idx);
    p.len = len;
    p.n_old = n_old;
    p.idx = idx;
    p.acc = a.acc;
    p.acc_out = a.acc_out;
    p.keep = a.keep;
    p.batch = a.batch;
    p.max_pages = a.max_pages;
    p.out_pages = a.out_pages;
    p.page_size = a.page_size;
    p.num_pages = a.num_pages;
    p.acc_rows = a.acc_rows;
    p.budget = a.budget;
    p.recent = a.recent;
    p.eword = eword;
    const bool hist = k > 0 && topk_uses_hist(a.acc_rows);
    const size_t zero16 = hist ? topk_hist_bytes(a.batch) / 16 : 0;
    count_launch();
    if (launch_k(evict_plan_kernel, dim3(hist ? 1 + 64 : 1), dim3(kT), 0, st, true, a.kv_len, len, n_old, a.kv_len_out, a.batch,
                 static_cast<int>(rows_in < a.acc_rows ? rows_in : a.acc_rows), a.budget, a.recent, eword,
                 hist ? reinterpret_cast<uint4*>(topk_hist_buffer(ws + l.topk)) : nullptr, zero16) != cudaSuccess)
        return DSV4_ERR_LAUNCH;
    if (k > 0) {
        TopkRows t{};
        t.scores = a.acc;
        t.n_vis = n_old;
        t.n_q = 1;
        t.ratio = 1;
        t.idx_out = idx;
        t.rows = a.batch;
        t.max_comp = a.acc_rows;
        t.top_k = k;
        t.hist_zeroed = hist;
        t.hist_built = false;
        t.pdl = true;
        if (int rc = launch_topk(t, ws + l.topk, eword, st)) return rc;
    }
    p.same = a.out_table == a.block_table;
    const bool in_place = p.same || a.acc_out == a.acc;
    const int pools = a.v_pages ? 2 : 1;
    p.row16 = a.kv_heads * a.dim / 8;
    const int sms = sm_count() > 0 ? sm_count() : 152;
    if (in_place) {
        // slices of 64 bytes; thinner ones, down to 16 bytes, while that leaves SMs without work
        p.slice = 4;
        while (p.slice > 1 && static_cast<long long>(a.batch) * pools * (p.row16 / p.slice) < sms) p.slice /= 2;
        p.rows_cta = a.budget;
    } else {
        p.slice = p.row16 < 64 ? p.row16 : 64;
        p.rows_cta = kRows<false>;
        while ((a.budget + p.rows_cta - 1) / p.rows_cta > 65535) p.rows_cta *= 2;
    }
    const unsigned slices = static_cast<unsigned>((p.row16 + p.slice - 1) / p.slice);
    const dim3 grid(slices * pools, static_cast<unsigned>((a.budget + p.rows_cta - 1) / p.rows_cta), a.batch);
    count_launch();
    return launch_k(in_place ? evict_move_kernel<true> : evict_move_kernel<false>, grid, dim3(kT), 0, st, true, p) == cudaSuccess
               ? DSV4_OK : DSV4_ERR_LAUNCH;
}

}  // namespace dsv4
