// Geometry of the paged KV cache and the division of its attention work.
//
// A cache is a pool of pages [num_pages, page_size, kv_heads, dim]; row r of sequence s lies in
// page table[s, r / page_size] at slot r % page_size. The n_s newest rows of a sequence belong
// to the n_s tokens whose queries are given (tokens cu_q[s] .. cu_q[s + 1] - 1), so token t of
// the sequence stands at row p = kv_len[s] - n_s + t and sees the rows [max(0, p + 1 - window),
// p + 1) (window 0: from row 0).
//
// Work is cut into units of kUnit = 128 cache rows x one row tile: a row tile is `tpt` tokens times
// `hb` query heads of one KV head (at most N rows, the tensor-core tile). All units of a call
// form one line, in the order (sequence, token tile, KV head and head block, rows), and CTA c
// of g takes the units [T c / g, T (c + 1) / g): every CTA has the same amount of work whatever
// the lengths are, a row tile that crosses a border is finished by a merge of the partial
// results, and no CTA leaves more than two of those. The lengths live on the device, so each
// CTA forms the line itself from cu_q and kv_len.
#pragma once

#include "common.cuh"

namespace dsv4 {

// 2^x by the hardware's approximation (relative error about 2^-22, results below 2^-126 are 0).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The inverse of float_to_key.
__device__ __forceinline__ float key_to_float(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}

constexpr int kUnit = 128;               // cache rows per unit

struct PagedGeom {
    const int32_t* table;                // [batch, max_pages]
    const int32_t* cu_q;                 // [batch + 1]
    const int32_t* kv_len;               // [batch]
    int batch, total_q, max_pages, page_size, num_pages;
    int H, KV, G;                        // query heads, KV heads, query heads per KV head
    int hb, nhb, tpt;                    // heads per row tile, head blocks per KV head, tokens per row tile
    int window;                          // 0: none
    int br, br_log2;                     // cache rows per TMA box: a power of two that divides page_size, <= kUnit
};

// Row tiles of at most N rows for groups of G heads: whole groups, or the split of a group into
// equal blocks that fills the tiles best (64 heads in tiles of 96: three tokens of 32).
inline void paged_tile(PagedGeom& g, int N) {
    double best = -1.0;
    const int least = (g.G + N - 1) / N;
    for (int k = least; k < least + 4 && k <= g.G; ++k) {
        const int hb = (g.G + k - 1) / k, nhb = (g.G + hb - 1) / hb, tpt = N / hb;
        const double fill = static_cast<double>(g.G) * tpt / (static_cast<double>(nhb) * N);
        if (fill > best + 0.05) {
            best = fill;
            g.hb = hb;
            g.nhb = nhb;
            g.tpt = tpt;
        }
    }
}

inline int paged_box_rows(int page_size) {
    const int low = page_size & -page_size;
    return low < kUnit ? low : kUnit;
}

struct PagedSeq { int q0, n, L; };       // first token, tokens, cache rows

// Counts outside their arrays are clamped, and `bad` is set.
__device__ __forceinline__ PagedSeq paged_seq(const PagedGeom& g, int s, bool& bad) {
    const int a = g.cu_q[s], b = g.cu_q[s + 1], len = g.kv_len[s];
    const int cap = g.max_pages * g.page_size;
    PagedSeq q;
    q.q0 = min(max(a, 0), g.total_q);
    const int e = min(max(b, q.q0), g.total_q);
    q.n = e - q.q0;
    q.L = min(max(len, 0), cap);
    bad |= q.q0 != a || e != b || q.L != len;
    return q;
}

__device__ __forceinline__ int paged_hi(const PagedSeq& q, int t) { return max(q.L - q.n + t + 1, 0); }
__device__ __forceinline__ int paged_lo(const PagedGeom& g, const PagedSeq& q, int t) {
    return g.window > 0 ? max(q.L - q.n + t + 1 - g.window, 0) : 0;
}

// Units of token tile tt: the blocks of kUnit rows that some token of it sees (at least one, so that
// tokens that see nothing are still answered).
__device__ __forceinline__ int paged_tile_units(const PagedGeom& g, const PagedSeq& q, int tt) {
    const int t0 = tt * g.tpt, t1 = min(t0 + g.tpt, q.n) - 1;
    return max((paged_hi(q, t1) + kUnit - 1) / kUnit - paged_lo(g, q, t0) / kUnit, 1);
}

struct PagedSched {
    long long total, u0, u1;             // all units, this CTA's [u0, u1)
    int ge;                              // CTAs with work
    int s, tt, inner, k;                 // where u0 lies
    PagedSeq q;                          // sequence s
};

// The share of worker `self` of `count`. Whole block of NT threads; `pref` is scratch for `batch` counts in shared memory. At least
// `min_units` units go to each worker with work. Returns with the result visible to the block.
template <int NT>
__device__ void paged_schedule(const PagedGeom& g, int self, int count, int min_units, long long* pref, PagedSched* out,
                               uint32_t* err) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int mult = g.KV * g.nhb;
    bool bad = false;
    // (up to 32 sequences per warp at a time, a lane each; the whole warp goes over a long one's tiles)
    const int step = min((g.batch + NT / 32 - 1) / (NT / 32), 32);
    for (int s0 = warp * step; s0 < g.batch; s0 += NT / 32 * step) {
        const int s = s0 + lane;
        const bool here = lane < step && s < g.batch;
        PagedSeq q{0, 0, 0};
        if (here) q = paged_seq(g, s, bad);
        const int nt = (q.n + g.tpt - 1) / g.tpt;
        long long units = 0;
        if (nt <= 4)
            for (int tt = 0; tt < nt; ++tt) units += paged_tile_units(g, q, tt);
        for (unsigned big = __ballot_sync(~0u, nt > 4); big; big &= big - 1) {
            const int src = __ffs(big) - 1;
            const PagedSeq b{0, __shfl_sync(~0u, q.n, src), __shfl_sync(~0u, q.L, src)};
            const int bnt = (b.n + g.tpt - 1) / g.tpt;
            long long u = 0;
            for (int tt = lane; tt < bnt; tt += 32) u += paged_tile_units(g, b, tt);
#pragma unroll
            for (int w = 16; w; w >>= 1) u += __shfl_xor_sync(~0u, u, w);
            if (lane == src) units = u;
        }
        if (here) pref[s] = units * mult;
    }
    if (bad) atomicOr(err, DSV4_EWORD_BAD_INDEX);
    __syncthreads();
    if (warp == 0) {
        long long carry = 0;
        for (int s0 = 0; s0 < g.batch; s0 += 32) {
            const int s = s0 + lane;
            long long v = s < g.batch ? pref[s] : 0;
#pragma unroll
            for (int w = 1; w < 32; w <<= 1) {
                const long long o = __shfl_up_sync(~0u, v, w);
                if (lane >= w) v += o;
            }
            v += carry;
            if (s < g.batch) pref[s] = v;
            carry = __shfl_sync(~0u, v, 31);
        }
    }
    __syncthreads();
    // Warp 0 finds where this CTA's units start, warp 1 where the next CTA's do. A border inside a
    // tile of few units moves to the tile's end: a partial result costs about a unit's time on
    // either side, more than the imbalance of at most 2 units or 1/32 of a share.
    if (warp < 2) {
        const long long T = g.batch > 0 ? pref[g.batch - 1] : 0;
        const long long most = T / min_units < 1 ? 1 : T / min_units;
        const int ge = most < count ? static_cast<int>(most) : count;
        const long long share32 = T / ge / 32, small = share32 > 2 ? share32 : 2;
        const int c = self + warp;
        long long u = c < ge ? T * c / ge : T;
        int s = 0, tt = 0, inner = 0, k = 0;
        PagedSeq q{0, 0, 0};
        bool dummy = false;
        if (u == 0 && T > 0) q = paged_seq(g, 0, dummy);
        if (u < T && u > 0) {
            int hi = g.batch - 1;                    // the first sequence whose units end past u
            while (s < hi) {
                const int mid = (s + hi) >> 1;
                if (pref[mid] > u) hi = mid; else s = mid + 1;
            }
            const long long rem = u - (s ? pref[s - 1] : 0);
            q = paged_seq(g, s, dummy);
            const int nt = (q.n + g.tpt - 1) / g.tpt;
            long long cum = 0;
            for (int tt0 = 0; tt0 < nt; tt0 += 32) {
                const int n = tt0 + lane < nt ? paged_tile_units(g, q, tt0 + lane) : 0;
                long long v = static_cast<long long>(n) * mult;
#pragma unroll
                for (int w = 1; w < 32; w <<= 1) {
                    const long long o = __shfl_up_sync(~0u, v, w);
                    if (lane >= w) v += o;
                }
                const unsigned past = __ballot_sync(~0u, cum + v > rem);
                if (past) {
                    const int f = __ffs(past) - 1;
                    const int nf = __shfl_sync(~0u, n, f);
                    const long long r = rem - cum - (__shfl_sync(~0u, v, f) - static_cast<long long>(nf) * mult);
                    tt = tt0 + f;
                    inner = static_cast<int>(r / nf);
                    k = static_cast<int>(r - static_cast<long long>(inner) * nf);
                    if (k > 0 && nf <= small) {      // the next tile's start
                        u += nf - k;
                        k = 0;
                        if (++inner == mult) { inner = 0; ++tt; }
                    }
                    break;
                }
                cum += __shfl_sync(~0u, v, 31);
            }
        }
        if (lane == 0) {
            if (warp == 0) {
                out->total = T;
                out->u0 = u;
                out->ge = ge;
                out->s = s;
                out->tt = tt;
                out->inner = inner;
                out->k = k;
                out->q = q;
            } else {
                out->u1 = u;
            }
        }
    }
    __syncthreads();
}

// The row tile a CTA works on and its part of that tile's units.
struct PagedSeg {
    PagedSeq q;
    int s, t0, tok0, tn;                 // sequence, first token in it and in the batch, tokens
    int kvh, head0, hv;                  // KV head, first query head, query heads
    int lo_u, hi_u;                      // rows that some token sees
    int lo_max, hi_min;                  // rows that every token sees
    int row0;                            // first row of unit 0 (a multiple of kUnit)
    int n, kb, ke;                       // the tile's units, this CTA's [kb, ke)
};

struct PagedWalk {
    const PagedGeom& g;
    int s, tt, inner, k;
    long long left;
    PagedSeq q;
    __device__ PagedWalk(const PagedGeom& geom, const PagedSched& sc)
        : g(geom), s(sc.s), tt(sc.tt), inner(sc.inner), k(sc.k), left(sc.u1 - sc.u0), q(sc.q) {}
    __device__ bool next(PagedSeg& o) {
        if (left <= 0) return false;
        while (tt * g.tpt >= q.n) {      // the next sequence with tokens
            if (++s >= g.batch) return false;
            tt = 0;
            bool dummy = false;
            q = paged_seq(g, s, dummy);
        }
        const int t0 = tt * g.tpt;
        o.q = q;
        o.s = s;
        o.t0 = t0;
        o.tok0 = q.q0 + t0;
        o.tn = min(g.tpt, q.n - t0);
        o.kvh = inner / g.nhb;
        const int blk = inner - o.kvh * g.nhb;
        o.head0 = o.kvh * g.G + blk * g.hb;
        o.hv = min(g.hb, g.G - blk * g.hb);
        o.lo_u = paged_lo(g, q, t0);
        o.hi_u = paged_hi(q, t0 + o.tn - 1);
        o.lo_max = paged_lo(g, q, t0 + o.tn - 1);
        o.hi_min = paged_hi(q, t0);
        o.row0 = o.lo_u / kUnit * kUnit;
        o.n = max((o.hi_u + kUnit - 1) / kUnit - o.lo_u / kUnit, 1);
        o.kb = k;
        const long long take = left < o.n - k ? left : o.n - k;
        o.ke = k + static_cast<int>(take);
        left -= take;
        k = 0;
        if (++inner == g.KV * g.nhb) { inner = 0; ++tt; }
        return true;
    }
};

// One tile of kUnit cache rows as boxes of `br` rows: lanes 2i and 2i + 1 answer for box i (the
// two 64-channel halves of a slot). The page is only looked up here; paged_boxes uses it.
struct PagedLook { int page, slot; bool need; };
__device__ __forceinline__ PagedLook paged_look(const PagedGeom& g, const PagedSeg& sg, int row, int lane) {
    PagedLook t{0, 0, false};
    const int i = lane >> 1, r = row + i * g.br;
    t.need = i < (kUnit >> g.br_log2) && r < sg.hi_u && r + g.br > sg.lo_u;   // holds rows that some token sees
    if (t.need) {
        const int pg = r / g.page_size;
        t.slot = r - pg * g.page_size;
        t.page = g.table[static_cast<size_t>(sg.s) * g.max_pages + pg];
    }
    return t;
}
// Whole warp: the lanes with something to load, and (bits 2i) the boxes on pages that are not in
// the pool: their rows are hidden.
struct PagedBoxes { unsigned ok, bad; };
__device__ __forceinline__ PagedBoxes paged_boxes(const PagedGeom& g, const PagedLook& t) {
    const bool in = t.page >= 0 && t.page < g.num_pages;
    return PagedBoxes{__ballot_sync(~0u, t.need && in), __ballot_sync(~0u, t.need && !in) & 0x55555555u};
}
__device__ __forceinline__ bool paged_bad_row(const PagedGeom& g, unsigned bad, int row) { return (bad >> (2 * (row >> g.br_log2))) & 1; }

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z,
                                            int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];"
        :: "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w),
           "r"(smem_u32(bar)) : "memory");
}

// Waits (bounded) for the copies in flight into a ring of ST slots that kLoadWarps warps fill in
// turn: slot r % ST by warp r % kLoadWarps, of which `end[w]` says where it stopped.
constexpr int kLoadWarps = 3;
constexpr unsigned long long kDrainNs = 100000000ull;
template <int ST>
__device__ __forceinline__ void ring_drain(uint64_t* full, const uint32_t (&end)[kLoadWarps]) {
    const uint32_t last = max(max(end[0], end[1]), end[2]);
    for (uint32_t i = last > ST ? last - ST : 0; i < last; ++i) {
        uint32_t r = i;
        if (r >= end[r % kLoadWarps]) {              // not issued: the slot's copy before it is the last
            if (r < ST) continue;
            r -= ST;
        }
        mbar_wait(&full[r % ST], (r / ST) & 1, nullptr, kDrainNs);
    }
}

}  // namespace dsv4
