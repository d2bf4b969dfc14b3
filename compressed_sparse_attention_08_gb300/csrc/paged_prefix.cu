// Attention over a paged cache for groups of sequences that share their first rows.
//
//   s_j = scale q . k_j over the rows j the token sees,   m = max_j s_j (and the sink)
//   o = sum_j e^(s_j - m) v_j / (sum_j e^(s_j - m) + e^(sink - m)),   lse = m + log(that sum)
// as paged_attn.cu, whose sources hold here too; sharing a prefix is this library's own. The softmax
// splits over any partition of the rows: with (m, l, o) of each part, l = sum e^(s - m) and o = sum e^(s - m) v,
// the whole is sum_p e^(m_p - M) o_p / sum_p e^(m_p - M) l_p. So the prefix's rows meet all the group's tokens
// together (the tokens of 32 sequences with 4 heads per KV head fill a tile of the tensor core, of which one
// sequence's fill 4 rows of 128), each sequence's own rows meet its own tokens, and a merge joins them.
//
// The work is the line of units of paged.cuh over `groups + batch` sequences: first the groups' prefixes (rows
// [0, P), all visible), then the sequences' own rows [P, ..). Every CTA takes an equal piece of the line.
// A row of the tensor core's 128 lanes is a query (a token's head), its columns are cache rows:
// S = Q K^T (128 queries x 128 rows, one step), O += P V with P in tensor memory, so a thread has one whole
// row of scores: its maximum and sum need no other thread. Two steps are in flight, each with a buffer of
// scores and a group of four softmax warps: while one group works on its scores, the tensor core does
// the other's products. At 128 channels the steps are two tiles of queries over the same unit (when there
// are that many queries), else two units; then both groups add to one O and hand each other the reference maximum.
// Of 512 channels tensor memory holds 256 beside the scores, so a tile is taken twice, each time
// with the scores over all channels and the product with half of V's (1.5 times the products' time).
// What bounds it: at 128 channels the chain of a unit of two tiles, 3,030 cycles against 2,048 of products (issue, the scores'
// arrival 370, the softmax 1,128, P's arrival 450); at 512 shared memory, which gives 128 bytes a cycle: 4,096 cycles of a unit's 4,550 (Q
// and K for the scores 2,048, V 512, the copies 1,536; products 3,070); with short own rows the segments' starts and ends; in
// small calls, cold (L2 flushed), the schedule's loads (10,000 cycles) and those until the first scores (14,000). Measured, merge included: 16
// chunks of up to 256 tokens behind 32,768 shared rows, 32 heads over 8 of 128, K and V apart, 583 us (1,310 TFLOP/s, tensor pipe 62 %
// active); 64 single tokens behind them 73; 48 tokens behind 65,536 rows, 16 heads of 512, one row as K and V, 153 (48 %
// active); 45 tokens in three groups behind 12,345 rows, 16 heads over 2 of 256, 42; 2 tokens behind 1,000, 8 heads, 14.3.
// Roles: warps 0, 2 and 3 move pages by TMA into a ring of slots of 128 rows x 128 channels, warp 1 issues tcgen05.mma,
// warps 4-11 do the softmax, write the parts and, once a segment's last scores have come, ask for the next one's queries.
#include <cfloat>
#include <cmath>

#include "internal.h"
#include "paged.cuh"

namespace dsv4 {
namespace {

constexpr int kThreads = 384;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// A query's reference maximum moves only when a score exceeds it by more than kSpan (base-2 units): P =
// 2^(s - m) then stays far inside the fp32 and bf16 range, and o does not depend on which m was used.
constexpr float kSpan = 24.f;
// The reference of a query that has seen nothing yet: finite, so that a score of -inf gives P = 0 beside it.
constexpr float kUnset = -3.0e38f;

// Sequence v of the line: the prefix of group v, or the rows of sequence v - groups behind its prefix.
struct PrefixSeq {
    int q0, n, L, lo;                    // first token, tokens, rows [lo, L)
    int row;                             // of the block table
    int own;                             // 1: a sequence's own rows (token t sees those below L - n + t + 1)
};

struct PrefixGeom {
    PagedGeom p;
    const int32_t* prefix_len;           // [groups]
    const int32_t* group_start;          // [groups + 1] or null: one group of all
    int groups, tiles, halves;           // tiles of queries per segment, passes over V's channels
};

// The geometry with the prefix lengths as they are used (by this CTA: each forms its own copy). While the schedule is made,
// lengths, groups and sequences lie in shared memory; afterwards they are read again where they are needed.
struct PrefixLine {
    using Seq = PrefixSeq;
    const PrefixGeom& g;
    const int32_t* plen;
    const int32_t* start;                // group_start, or null
    const PagedSeq* seqs;                // or null
};

__device__ __forceinline__ int group_first(const PrefixLine& l, int i) {
    const int b = l.start ? l.start[i] : (i ? l.g.p.batch : 0);
    return min(max(b, 0), l.g.p.batch);
}
// The group of sequence s, or -1.
__device__ __forceinline__ int group_of(const PrefixLine& l, int s) {
    if (!l.start) return 0;
    int lo = 0, hi = l.g.groups;         // the last group that starts at or before s
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (l.start[mid] <= s) lo = mid; else hi = mid;
    }
    return group_first(l, lo) <= s && s < group_first(l, lo + 1) ? lo : -1;
}

__device__ __forceinline__ PrefixSeq paged_seq(const PrefixLine& l, int v, bool& bad) {
    const PrefixGeom& g = l.g;
    PrefixSeq q;
    if (v < g.groups) {
        const int a = group_first(l, v), b = group_first(l, v + 1), P = l.plen[v];
        q.q0 = min(max(g.p.cu_q[a], 0), g.p.total_q);
        q.n = P > 0 ? max(min(max(g.p.cu_q[b], 0), g.p.total_q) - q.q0, 0) : 0;
        q.L = P;
        q.lo = 0;
        q.row = a;
        q.own = 0;
        return q;
    }
    const int s = v - g.groups;
    const PagedSeq o = l.seqs ? l.seqs[s] : paged_seq(g.p, s, bad);
    const int grp = group_of(l, s);
    q.q0 = o.q0;
    q.n = o.n;
    q.L = o.L;
    q.lo = grp >= 0 && o.n > 0 ? l.plen[grp] : 0;
    q.row = s;
    q.own = 1;
    return q;
}
__device__ __forceinline__ int paged_count(const PrefixLine& l) { return l.g.groups + l.g.p.batch; }
__device__ __forceinline__ int paged_tokens(const PrefixLine& l) { return l.g.p.tpt * l.g.tiles; }
__device__ __forceinline__ int paged_mult(const PrefixLine& l) { return l.g.p.KV * l.g.p.nhb * l.g.halves; }
__device__ __forceinline__ PrefixSeq paged_shfl(const PrefixSeq& q, int src) {
    return PrefixSeq{0, __shfl_sync(~0u, q.n, src), __shfl_sync(~0u, q.L, src), __shfl_sync(~0u, q.lo, src), 0,
                     __shfl_sync(~0u, q.own, src)};
}
__device__ __forceinline__ int seen(const PrefixSeq& q, int t) { return q.own ? max(q.L - q.n + t + 1, 0) : q.L; }
__device__ __forceinline__ int unit_row0(const PrefixGeom& g, const PrefixSeq& q) { return q.lo & ~(g.p.br - 1); }
__device__ __forceinline__ int segment_units(const PrefixGeom& g, const PrefixSeq& q, int t_last) {
    return max((seen(q, t_last) - unit_row0(g, q) + kUnit - 1) / kUnit, 1);
}
// The line counts time, in 600 cycles or so: a unit of two tiles takes 5, of one tile 3 (at 256 and 512 channels all
// have one, and take longer: only ratios count), a segment's start and end 25 and 11 (4 of longer units).
// Measured at 16 sequences of 256 tokens of 32 heads behind 32,768 shared rows: 590 us; with 21, 11 and 6 596, with 30 657, with 18 and 9 640.
// On 20 other batches at 128 channels (2 to 63 sequences of 1 to 168 tokens in 1 to 4 groups) 17 to 30 in the first place and 8 to 14
// in the second come to the same within 1 % on average (single ones within 7 %): what they decide is how a batch falls on the
// CTAs. On 20 at 256 and 512, with 2 in place of 4 3 to 5 % slower, with 3 0 to 2 %, with 6 and 8 1 to 2 % faster.
__device__ __forceinline__ bool two_tiles(const PrefixLine& l, const PrefixSeq& q, int tt) {
    return l.g.tiles == 2 && q.n - tt * paged_tokens(l) > l.g.p.tpt;
}
__device__ __forceinline__ int paged_weight(const PrefixLine& l, const PrefixSeq& q, int tt) { return two_tiles(l, q, tt) ? 5 : 3; }
__device__ __forceinline__ int paged_over(const PrefixLine& l, const PrefixSeq& q, int tt) {
    return l.g.tiles == 1 ? 4 : two_tiles(l, q, tt) ? 25 : 11;
}
__device__ __forceinline__ int paged_tile_units(const PrefixLine& l, const PrefixSeq& q, int tt) {
    return segment_units(l.g, q, min((tt + 1) * paged_tokens(l), q.n) - 1) * paged_weight(l, q, tt) + paged_over(l, q, tt);
}

// A segment of the line: up to `tiles` tiles of queries of one KV head, and this CTA's part of their units.
struct PrefixSeg {
    PrefixSeq q;
    int t0, tok0, tn, nt;                // first token in the sequence and in the batch, tokens, tiles
    int kvh, head0, hv, half;            // KV head, first query head, query heads, half of V's channels
    int hi_u, hi_min;                    // rows below which some token sees, and every token
    int row0, n, kb, ke;                 // first row of unit 0, the segment's units, this CTA's [kb, ke)
    int weight, cost;                    // of a unit, and of this CTA's part, on the line
};

struct PrefixWalk {
    const PrefixLine& l;
    int s, tt, inner, k;
    long long left;
    PrefixSeq q;
    __device__ PrefixWalk(const PrefixLine& line, const PagedSchedOf<PrefixLine>& sc)
        : l(line), s(sc.s), tt(sc.tt), inner(sc.inner), k(sc.k), left(sc.u1 - sc.u0), q(sc.q) {}
    __device__ bool next(PrefixSeg& o) {
        if (left <= 0) return false;
        const PrefixGeom& g = l.g;
        const int tps = paged_tokens(l);
        while (tt * tps >= q.n) {        // the next sequence with tokens
            if (++s >= paged_count(l)) return false;
            tt = 0;
            bool dummy = false;
            q = paged_seq(l, s, dummy);
        }
        o.q = q;
        o.t0 = tt * tps;
        o.tok0 = q.q0 + o.t0;
        o.tn = min(tps, q.n - o.t0);
        o.nt = o.tn > g.p.tpt ? 2 : 1;
        const int hb = inner / g.halves;
        o.half = inner - hb * g.halves;
        o.kvh = hb / g.p.nhb;
        const int blk = hb - o.kvh * g.p.nhb;
        o.head0 = o.kvh * g.p.G + blk * g.p.hb;
        o.hv = min(g.p.hb, g.p.G - blk * g.p.hb);
        o.hi_u = seen(q, o.t0 + o.tn - 1);
        o.hi_min = seen(q, o.t0);
        o.row0 = unit_row0(g, q);
        o.n = segment_units(g, q, o.t0 + o.tn - 1);
        o.weight = paged_weight(l, q, tt);
        o.kb = k / o.weight;
        o.ke = left >= static_cast<long long>(o.n - o.kb) * o.weight ? o.n : o.kb + static_cast<int>(left) / o.weight;
        o.cost = (o.ke - o.kb) * o.weight + (o.ke == o.n ? paged_over(l, q, tt) : 0);
        left -= o.cost;
        k = 0;
        if (++inner == paged_mult(l)) { inner = 0; ++tt; }
        return true;
    }
};

struct PrefixParams {
    PrefixGeom g;
    const float* sink;                   // [H] or null
    __nv_bfloat16* out;                  // [total_q, H, D]
    float* lse;                          // [total_q, H] or null
    // Parts: of a segment's first units, by kind (0 prefix, 1 own rows), token and head; of a
    // segment that goes on from another CTA, by CTA (each has one at most).
    float4* home_ml;                     // [2][halves][total_q][H]: m, l, (CTA | CTAs << 8 | row << 16), whether there is a prefix
    float2* cont_ml;                     // [CTAs][tiles * 128]
    float* home_o;                       // [2][total_q][H][D]
    float* cont_o;                       // [CTAs][tiles * 128][DV]
    int32_t* plen;                       // [CTAs][groups]
    uint32_t* err;                       // [CTAs]
    float scale2;                        // scale * log2(e)
    const int64_t* orp;                  // [total_q] or null
    int or_pairs;
    int shared, min_units;
    int negate;                          // a negative scale: Q is negated (bit 13 of the products' descriptor)
    int fault;                           // test control: a CTA's first query tile is never copied
    unsigned long long wait_ns;
    double or_freq[64];                  // theta^(-2j / out_rope_dim)
};

constexpr int kMaxSlots = 8, kSegs = 10; // (see the static_assert beside the roles)
struct PrefixCtl {
    uint64_t q_full, empty[kMaxSlots];
    // A slot's copies, counted apart for K (and tiles that are both) and for V.
    uint64_t full[2][kMaxSlots];
    uint8_t last[kMaxSlots];             // a slot's last copy: 4 | parity << 1 | V
    uint64_t seg_full[kSegs], s_full[2], p_full[2], pv_done[2], o_done[2], ref_done[2][4], l_ready[2][4], o_empty;
    uint64_t drained;                    // products in flight when a wait ran out
    uint32_t seg_end;                    // query tiles that were copied
    PagedSchedOf<PrefixLine> sched;
    PrefixSeg segs[kSegs];               // written by a load warp
    float ref[128];                      // reference maxima (base-2 units), where two groups share a tile
    float l[2][128];
    unsigned bad[8];
    uint32_t tmem, err;
    int abort;
};

template <int D_>
struct XCfg {
    static constexpr int D = D_;
    static constexpr int TILES = D == 128 ? 2 : 1, HALVES = D == 512 ? 2 : 1;
    static constexpr int DV = D == 512 ? 256 : D;            // V's channels of a pass
    static constexpr int KS = D / 128, VS = DV / 128;        // slots of a K and a V tile
    static constexpr int BOX = kUnit * 128, SLOT = 2 * BOX;  // 128 rows x 64 channels; x 128
    static constexpr int QBOX = 128 * 128, QTILE = 2 * KS * QBOX, QB = TILES * QTILE;
    static constexpr int ST_FIT = (232448 - static_cast<int>(sizeof(PrefixCtl)) - QB) / SLOT;
    static constexpr int ST = ST_FIT > kMaxSlots ? kMaxSlots : ST_FIT;
    static constexpr int OFF_Q = ST * SLOT, OFF_C = OFF_Q + QB, SMEM = OFF_C + static_cast<int>(sizeof(PrefixCtl));
    // A shared K/V tile stays for both products where the ring then still holds five units. At 256 channels it would hold two
    // and a half, and the next K waits for the product with V (45 tokens of 16 heads over 12,345 rows 44.5 us, loaded twice 42;
    // 64 tokens over 32,768 67.6 and 63.5; 16 chunks of 128 over 8,192 369 and 379).
    static constexpr bool KEEP = D == 128;
    static constexpr int OCOL = 256;                         // scores: columns 0 and 128; P over their first 64
    static_assert(ST == (D == 512 ? 3 : 5), "slots");
    static_assert(SMEM <= 232448 && (!KEEP || ST > 2 * KS) && OCOL + TILES * DV <= 512, "fits");
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// D[tmem] (+)= A[tmem] * B[smem desc], kind::f16 (bf16 inputs, fp32 accumulate): A's rows are lanes, a column holds two k.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        :: "r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}

// The largest of three (a NaN loses), in one instruction.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// 32 bytes, a sector of its own for every lane.
__device__ __forceinline__ void store32(float* p, const uint32_t* r) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]),
                 "r"(r[5]), "r"(r[6]), "r"(r[7]) : "memory");
}

__device__ __noinline__ float2 out_rope_angle(double a) {
    float sn, cs;
    sincosf(reduced_angle(a), &sn, &cs);
    return make_float2(cs, sn);
}

// A bounded wait whose first look is all that stands in the way of a barrier that is there already.
__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, const volatile int* abort, unsigned long long ns) {
    return mbar_wait(bar, parity, abort, ns);
}
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, const volatile int* abort, unsigned long long ns) {
    return mbar_try_wait(bar, parity) || wait_on(bar, parity, abort, ns);
}

// A reader's place in the ring of ST slots, and for each slot the parity of its next copy for this reader.
template <uint32_t ST>
struct RingAt {
    uint32_t slot, turns;
    template <uint32_t N>
    __device__ __forceinline__ void skip() {
        slot += N % ST;
        if (slot >= ST) slot -= ST;
    }
    __device__ __forceinline__ uint32_t parity() const { return turns >> slot & 1; }
    __device__ __forceinline__ void next() {             // this slot's copy is used
        turns ^= 1u << slot;
        skip<1>();
    }
};

// The pages of a tile of kUnit rows, as paged_look.
__device__ __forceinline__ PagedLook prefix_look(const PagedGeom& g, const PrefixSeg& sg, int row, int lane) {
    PagedLook t{0, 0, false};
    const int i = lane >> 1, r = row + i * g.br;
    t.need = i < (kUnit >> g.br_log2) && r < sg.hi_u && r + g.br > sg.q.lo;
    if (t.need) {
        const int pg = r / g.page_size;
        t.slot = r - pg * g.page_size;
        t.page = g.table[static_cast<size_t>(sg.q.row) * g.max_pages + pg];
    }
    return t;
}

// Scratch of the schedule, in the ring's place.
struct PrefixScratch {
    long long pref[4096];
    PagedSeq seqs[2048];
    int32_t plen[2048], start[2052];
};

// The prefix lengths that the groups use: no row that some token of the group does not see.
__device__ void prefix_lengths(const PrefixGeom& g, PrefixScratch& z, int32_t* out, uint32_t* err) {
    bool bad = false;
    const int cap = g.p.max_pages * g.p.page_size;
    for (int i = threadIdx.x; i < g.groups; i += kThreads) {
        const int x = g.prefix_len[i];
        z.plen[i] = min(max(x, 0), cap);
        bad |= x != z.plen[i];
        if (g.group_start) {
            const int a = g.group_start[i], b = g.group_start[i + 1];
            bad |= a < 0 || b < a || b > g.p.batch;
            z.start[i] = a;
            if (i + 1 == g.groups) z.start[i + 1] = b;
        }
    }
    for (int s = threadIdx.x; s < g.p.batch; s += kThreads) z.seqs[s] = paged_seq(g.p, s, bad);
    __syncthreads();
    const PrefixLine l{g, z.plen, g.group_start ? z.start : nullptr, z.seqs};
    for (int s = threadIdx.x; s < g.p.batch; s += kThreads) {
        const PagedSeq q = z.seqs[s];
        const int grp = group_of(l, s);
        if (grp >= 0 && q.n > 0 && q.L - q.n < z.plen[grp]) atomicMin(&z.plen[grp], max(q.L - q.n, 0));
    }
    if (bad) atomicOr(err, DSV4_EWORD_BAD_INDEX);
    __syncthreads();
    for (int i = threadIdx.x; i < g.groups; i += kThreads) out[i] = z.plen[i];
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
paged_prefix_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap vmap, const __grid_constant__ PrefixParams p) {
    using C = XCfg<D>;
    constexpr int ST = C::ST, KS = C::KS, VS = C::VS;
    extern __shared__ __align__(1024) uint8_t sm[];
    PrefixCtl& ctl = *reinterpret_cast<PrefixCtl*>(sm + C::OFF_C);
    uint8_t* sQ = sm + C::OFF_Q;
    volatile int* abort_flag = &ctl.abort;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int worker = blockIdx.x, workers = gridDim.x;
    if (tid == 0) {
        tma_prefetch_desc(&qmap);
        tma_prefetch_desc(&kmap);
        tma_prefetch_desc(&vmap);
        mbar_init(&ctl.q_full, 1);
        for (int i = 0; i < ST; ++i) {
            mbar_init(&ctl.full[0][i], 1);
            mbar_init(&ctl.full[1][i], 1);
            mbar_init(&ctl.empty[i], 1);
            ctl.last[i] = 0;
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl.s_full[i], 1);
            mbar_init(&ctl.p_full[i], 4);
            mbar_init(&ctl.pv_done[i], 1);
            mbar_init(&ctl.o_done[i], 1);
            for (int j = 0; j < 4; ++j) { mbar_init(&ctl.ref_done[i][j], 1); mbar_init(&ctl.l_ready[i][j], 1); }
        }
        for (int i = 0; i < kSegs; ++i) mbar_init(&ctl.seg_full[i], 1);
        mbar_init(&ctl.o_empty, 8);
        mbar_init(&ctl.drained, 1);
        ctl.abort = 0;
        ctl.err = 0;
        ctl.seg_end = 0;
        fence_barrier_init();
    }
    if (warp == 2) tmem_alloc(&ctl.tmem, 512);
    pdl_trigger();
    pdl_wait();                          // lengths, queries and rows may come from the kernel before
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem;
    int32_t* plen = p.plen + static_cast<size_t>(worker) * p.g.groups;
    PrefixScratch& scratch = *reinterpret_cast<PrefixScratch*>(sm);
    static_assert(sizeof(PrefixScratch) <= static_cast<size_t>(C::OFF_Q), "in the ring's place");
    prefix_lengths(p.g, scratch, plen, &ctl.err);
    paged_schedule<kThreads>(PrefixLine{p.g, scratch.plen, p.g.group_start ? scratch.start : nullptr, scratch.seqs}, worker, workers,
                             p.min_units, scratch.pref, &ctl.sched, &ctl.err);
    const PrefixLine line{p.g, plen, p.g.group_start, nullptr};
    // the schedule's scratch is overwritten by TMA next
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();

    const PagedGeom& g = p.g.p;
    const PagedSchedOf<PrefixLine>& sched = ctl.sched;
    // Descriptions in use at once: those of the segments from s on, of which some warp still writes outputs, to the newest. No
    // slot of s + 1 becomes free before all warps have arrived at o_empty for s. If every segment is one slot, place s + 1 +
    // ST waits for that; the load warp that describes passes up to kLoadWarps - 1 places of the other warps before its
    // own stops it, and has described the segment behind that place by then.
    static_assert(kSegs >= ST + kLoadWarps + 2, "descriptions");
    const bool keep = C::KEEP && p.shared;               // K rows stay in place as V
    const uint32_t share = static_cast<uint32_t>(sched.u1 - sched.u0);
    if (warp == 0 || warp == 2 || warp == 3) {
        // ---------------------------------------------------------------- pages and queries
        // Three warps walk the same slots and take them in turn. Order: as the products need them, K0 V0 K1
        // V1 .. with two tiles of queries, K0 K1 V0 K2 V1 .. with one, K0 K1 .. where a tile is both. They go on into the next
        // segment as far as the ring lets them; its description is formed a segment ahead (it takes a few dependent loads).
        const int mine = warp == 0 ? 0 : warp - 1;
        PrefixWalk w(line, sched);
        PrefixSeg sg, after;
        const int piece = lane >> 1, box = lane & 1;
        uint32_t ring = 0, seg = 0, turn[2] = {0, 0};    // (a bit per slot: the parity of its next copy)
        bool dead = false, more = w.next(sg), then = false, known = false;   // (whether `then` and `after` are)
        auto describe = [&] {                            // a new segment, for the other roles
            if (lane == 0 && mine == 0) {
                ctl.segs[seg % kSegs] = sg;
                mbar_arrive(&ctl.seg_full[seg % kSegs]);
            }
            ++seg;
        };
        if (more) describe();
        PagedLook cur{0, 0, false}, prev{0, 0, false};
        if (more) cur = prefix_look(g, sg, sg.row0 + sg.kb * kUnit, lane);
        int k = more ? sg.kb : 0;
        auto load = [&](const CUtensorMap* map, const PagedLook& t, int slots, int ch0, int kvh, int unit) {
            const int kind = unit < 0;                   // K (with its unit), or V
            const PagedBoxes bx = paged_boxes(g, t);
            const uint32_t bytes = static_cast<uint32_t>(__popc(bx.ok)) * g.br * 128;
#pragma unroll 1
            for (int mt = 0; mt < slots; ++mt, ++ring) {
                const uint32_t slot = ring % ST, parity = turn[kind] >> slot & 1;
                turn[kind] ^= 1u << slot;
                if (ring % kLoadWarps != static_cast<uint32_t>(mine)) continue;
                if (ring >= ST)
                    dead = __any_sync(~0u, !wait_for(&ctl.empty[slot], (ring / ST - 1) & 1, abort_flag, p.wait_ns));
                if (dead) return;
                if (lane == 0) {
                    if (mt == 0 && unit >= 0) {
                        ctl.bad[unit & 7] = bx.bad;
                        if (bx.bad) atomicOr(&ctl.err, DSV4_EWORD_BAD_INDEX);
                    }
                    ctl.last[slot] = static_cast<uint8_t>(4 | parity << 1 | kind);
                    if (bytes) mbar_arrive_expect_tx(&ctl.full[kind][slot], bytes);
                    else mbar_arrive(&ctl.full[kind][slot]);
                }
                __syncwarp();
                if ((bx.ok >> lane) & 1)
                    tma_load_4d(sm + slot * C::SLOT + box * C::BOX + piece * g.br * 128, map, &ctl.full[kind][slot],
                                ch0 + mt * 128 + box * 64, kvh, t.slot, t.page);
            }
        };
        for (int u = 0; !dead && more; ++u) {
            // the pages of the next unit are looked up while this one's copies wait
            const int kvh = sg.kvh, v0 = sg.half * 256;
            const bool first = k == sg.kb, last = k + 1 == sg.ke, two = sg.nt == 2;
            PagedLook next{0, 0, false};
            if (++k >= sg.ke) {
                if (!known) then = w.next(after);
                known = false;
                more = then;
                sg = after;
                k = more ? sg.kb : 0;
                if (more) describe();
            }
            if (more) next = prefix_look(g, sg, sg.row0 + k * kUnit, lane);
            load(&kmap, cur, KS, 0, kvh, u);
            if (!keep) {
                if (two) {
                    if (!dead) load(&vmap, cur, VS, v0, kvh, -1);
                } else {
                    if (!dead && !first) load(&vmap, prev, VS, v0, kvh, -1);
                    if (!dead && last) load(&vmap, cur, VS, v0, kvh, -1);
                }
            }
            if (!known && more) {
                then = w.next(after);
                known = true;
            }
            prev = cur;
            cur = next;
        }
        if (dead && lane == 0) {
            atomicOr(&ctl.err, DSV4_EWORD_TIMEOUT);
            ctl.abort = 1;
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- tensor core
        // Steps (unit, tile) in order; the product with V of step i - 2 comes before the scores of step i, whose
        // buffer holds that step's P (the tensor core does a thread's products in the order of their issue; a commit
        // speaks for all before it, so scores that have come say that the product two steps before is done).
        // A product takes the core 64 cycles and the warp 23; but anything else costs the warp about 10 cycles an
        // instruction, 60 a commit and 100 to 150 a look at a barrier, and with a general loop over steps that was 1,400 a
        // step, more than the products' 1,024. So the two forms of a segment have loops of their own with little in
        // them, P, V and K are looked at together, a lane each, and what can wait is done behind issued products.
        // (One warp for S and one for O: the two tiles' products mixed, both tiles' softmax ran at the same time, and then
        // the core idled.) Votes and exchanges tell the compiler that the warp stays together.
        // (Every wait of the kernel is for a phase whose predecessor the waiter has seen, itself or through what it waited for
        // before, and whose successor cannot end before it goes on: parity tells no more.)
        struct { int row0, kb, ke, lo, hi_u; } sg{};
        uint32_t at = 0, u = 0, seg = 0, i0 = 0, ends = 0;   // place on the line; units, segments, steps, steps with pv_done before this segment
        bool dead = false;
        const bool one = elect_one();
        // (a wait that runs out does so for all lanes)
        auto look = [&](uint64_t* bar, uint32_t parity, bool on) {
            return !__any_sync(~0u, on && !wait_for(bar, parity & 1, abort_flag, p.wait_ns));
        };
        auto wait = [&](uint64_t* bar, uint32_t parity) { return look(bar, parity, true); };
        RingAt<ST> kat{0, 0}, vat{0, 0};                 // the next K and V slots, in the order of the loads
        const uint32_t tm = __shfl_sync(~0u, tmem, 0);
        const uint32_t idS = idesc_bf16_f32(128, kUnit) | (p.negate ? 1u << 13 : 0u), idO = idesc_bf16_f32(128, 128) | (1u << 16);
        const uint64_t qdesc = sdesc_kmajor_sw128(smem_u32(sQ)), kdesc = sdesc_kmajor_sw128(smem_u32(sm)),
                       vdesc = sdesc_mnmajor_sw128(smem_u32(sm), C::BOX, 1024u);
        // (one lane) S of buffer `buf` (+)= Q's channels 128 s .. of a tile x K's in a slot
        auto mul_k = [&](uint32_t buf, uint32_t tile, int s, uint32_t slot) {
            const uint64_t a = qdesc + tile * (C::QTILE / 16) + s * (2 * C::QBOX / 16), b = kdesc + slot * (C::SLOT / 16);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
                umma_bf16(tm + buf * 128, a + (kk >> 2) * (C::QBOX / 16) + (kk & 3) * 2, b + (kk >> 2) * (C::BOX / 16) + (kk & 3) * 2, idS,
                          kk > 0 ? 1u : s);
        };
        // (one lane) O's columns at `d` (+)= P of buffer `buf` x V in a slot
        auto mul_v = [&](uint32_t d, uint32_t buf, uint32_t slot, uint32_t more) {
            const uint64_t b = vdesc + slot * (C::SLOT / 16);
#pragma unroll
            for (int kk = 0; kk < kUnit / 16; ++kk)
                umma_bf16_ts(tm + C::OCOL + d, tm + buf * 128 + kk * 8, b + kk * 128, idO, kk > 0 ? 1u : more);
        };
        // Whether unit x of the segment, whose K has come, holds rows that no token sees.
        auto edge = [&](uint32_t x) {
            const int j0 = sg.row0 + (sg.kb + static_cast<int>(x)) * kUnit;
            const unsigned bad = *reinterpret_cast<volatile unsigned*>(&ctl.bad[(u + x) & 7]);
            return __any_sync(~0u, j0 < sg.lo || j0 + kUnit > sg.hi_u || bad);
        };
        // Such rows hold anything: as V they must not meet P = 0.
        auto clear_rows = [&](uint32_t x) {
            const int j0 = sg.row0 + (sg.kb + static_cast<int>(x)) * kUnit;
            const unsigned bad = *reinterpret_cast<volatile unsigned*>(&ctl.bad[(u + x) & 7]);
            constexpr int per = VS * 16;                 // 16-byte pieces of a row, a lane each (two rows at a time of 128 channels)
            const int x16 = lane % per;
            uint32_t slot = vat.slot + (x16 >> 4);
            if (slot >= ST) slot -= ST;
            uint8_t* z = sm + slot * C::SLOT + ((x16 >> 3) & 1) * C::BOX + (x16 & 7) * 16;
            auto clear = [&](int row, int end) {
#pragma unroll 4
                for (row += lane / per; row < end; row += 32 / per) *reinterpret_cast<uint4*>(z + row * 128) = make_uint4(0, 0, 0, 0);
            };
            const int z0 = min(max(sg.lo - j0, 0), kUnit), z1 = min(max(sg.hi_u - j0, z0), kUnit);
            clear(0, z0);
            clear(z1, kUnit);
            for (int r = 0; bad && r < (kUnit >> g.br_log2); ++r)
                if (bad >> (2 * r) & 1) clear(r << g.br_log2, (r + 1) << g.br_log2);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
        };
        // Two tiles: K0 V0 K1 V1 .. (one slot each), or K0 K1 ..
        auto two_tiles = [&]() {
            const uint32_t n = __shfl_sync(~0u, sg.ke - sg.kb, 0), b0 = i0 & 1, b1 = b0 ^ 1;
            uint32_t pp0 = i0 >> 1, pp1 = (i0 + 1) >> 1; // phases of P
            if (!keep) vat.template skip<1>();
            if (!wait(&ctl.full[0][kat.slot], kat.parity())) return false;
            tc_fence_after();
            bool edgy = edge(0);
            if (one) {
                mul_k(b0, 0, 0, kat.slot);
                umma_commit(&ctl.s_full[b0]);
                mul_k(b1, 1, 0, kat.slot);
                umma_commit(&ctl.s_full[b1]);
                if (!keep) umma_commit(&ctl.empty[kat.slot]);
            }
            __syncwarp();
            kat.next();
            if (!keep) kat.template skip<1>();
            for (uint32_t x = 0; x < n; ++x, ++pp0, ++pp1) {
                const bool more = x + 1 < n;
                if (edgy) {                              // (before P is waited for)
                    if (!keep && !wait(&ctl.full[1][vat.slot], vat.parity())) return false;
                    clear_rows(x);
                }
                // lane 0: the first tile's P; 1: the next K; others: V
                if (!look(lane == 0 ? &ctl.p_full[b0] : lane == 1 ? &ctl.full[0][kat.slot] : &ctl.full[1][vat.slot],
                          lane == 0 ? pp0 : lane == 1 ? kat.parity() : vat.parity(), lane == 0 || (lane == 1 ? more : !keep)))
                    return false;
                tc_fence_after();
                if (x == 0 && seg > 0 && !wait(&ctl.o_empty, seg - 1)) return false;
                if (one) {
                    mul_v(0, b0, vat.slot, x);
                    if (more) {
                        mul_k(b0, 0, 0, kat.slot);
                        umma_commit(&ctl.s_full[b0]);
                    } else {
                        umma_commit(&ctl.o_done[b0]);
                    }
                }
                __syncwarp();
                if (more) edgy = edge(x + 1);
                if (!wait(&ctl.p_full[b1], pp1)) return false;
                tc_fence_after();
                if (one) {
                    mul_v(C::DV, b1, vat.slot, x);
                    if (more) {
                        mul_k(b1, 1, 0, kat.slot);
                        umma_commit(&ctl.s_full[b1]);
                        if (!keep) umma_commit(&ctl.empty[kat.slot]);
                    } else {
                        umma_commit(&ctl.o_done[b1]);
                    }
                    umma_commit(&ctl.empty[vat.slot]);
                }
                __syncwarp();
                vat.next();
                if (more) {
                    kat.next();
                    if (!keep) {
                        vat.template skip<1>();
                        kat.template skip<1>();
                    }
                }
            }
            return true;
        };
        // One tile: K0 K1 V0 K2 V1 .., or K0 K1 ..
        auto one_tile = [&]() {
            const uint32_t n = __shfl_sync(~0u, sg.ke - sg.kb, 0);
            uint32_t edges = 0;                          // a bit per unit, the newest lowest
            auto scores = [&](uint32_t x) {
                const uint32_t buf = (i0 + x) & 1;
#pragma unroll 1
                for (int s = 0; s < KS; ++s) {
                    if (!wait(&ctl.full[0][kat.slot], kat.parity())) return false;
                    tc_fence_after();
                    if (one) {
                        mul_k(buf, 0, s, kat.slot);
                        if (!keep) umma_commit(&ctl.empty[kat.slot]);
                        if (s + 1 == KS) umma_commit(&ctl.s_full[buf]);
                    }
                    __syncwarp();
                    kat.next();
                }
                if (!keep && x > 0) kat.template skip<VS>();
                edges = edges << 1 | (edge(x) ? 1u : 0u);
                return true;
            };
            if (!keep) {
                vat.template skip<KS>();
                if (n > 1) vat.template skip<KS>();
            }
            if (!scores(0) || (n > 1 && !scores(1))) return false;
            for (uint32_t x = 0; x < n; ++x) {
                const uint32_t i = i0 + x, buf = i & 1;
                RingAt<ST> v1 = vat;
                if (VS == 2) v1.template skip<1>();
                const bool odd = VS == 2 && (lane & 1);
                if (edges >> (x + 1 < n ? 1 : 0) & 1) {  // (before P is waited for)
                    if (!look(&ctl.full[1][odd ? v1.slot : vat.slot], odd ? v1.parity() : vat.parity(), !keep)) return false;
                    clear_rows(x);
                }
                // lane 0: P; others: V
                if (!look(lane == 0 ? &ctl.p_full[buf] : &ctl.full[1][odd ? v1.slot : vat.slot],
                          lane == 0 ? i >> 1 : odd ? v1.parity() : vat.parity(), lane == 0 || !keep))
                    return false;
                tc_fence_after();
                if (x == 0 && seg > 0 && !wait(&ctl.o_empty, seg - 1)) return false;
                if (one) {
                    mul_v(0, buf, vat.slot, x);
                    umma_commit(&ctl.empty[vat.slot]);
                    if (VS == 2) {
                        mul_v(128, buf, v1.slot, x);
                        umma_commit(&ctl.empty[v1.slot]);
                    }
                    umma_commit(&ctl.pv_done[(ends + x) & 1]);
                }
                __syncwarp();
                vat.next();
                if (VS == 2) vat.next();
                if (x + 2 < n) {
                    if (!keep) vat.template skip<KS>();
                    if (!scores(x + 2)) return false;
                }
            }
            if (!keep) kat.template skip<VS>();          // (the segment's last V)
            ends += n;
            return true;
        };
        for (; at < share; ++seg) {
            // the segment's description and its queries
            dead = !look(lane == 0 ? &ctl.seg_full[seg % kSegs] : &ctl.q_full, lane == 0 ? seg / kSegs : seg, true);
            if (dead) break;
            const PrefixSeg& d = ctl.segs[seg % kSegs];
            sg = {d.row0, d.kb, d.ke, d.q.lo, d.hi_u};
            const uint32_t nt = d.nt, units = d.ke - d.kb, cost = d.cost;
            const bool two = C::TILES == 2 && __any_sync(~0u, nt == 2);
            if constexpr (C::TILES == 2) {
                if (two) dead = !two_tiles();
            }
            if (!two) dead = !one_tile();
            if (dead) break;
            at += __shfl_sync(~0u, cost, 0);
            u += units;
            i0 += __shfl_sync(~0u, units * nt, 0);
        }
        if (dead && lane == 0) {
            atomicOr(&ctl.err, DSV4_EWORD_TIMEOUT);
            ctl.abort = 1;
        }
    } else {
        // ---------------------------------------------------------------- softmax and parts
        const int q4 = warp & 3, grp = (warp - 4) >> 2;
        const int row = q4 * 32 + lane;                              // of a tile
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(q4 * 32) << 16);
        const uint32_t sbuf = lane_base + grp * 128;
        const uint64_t scale22 = pack_f32x2(p.scale2, p.scale2);
        const int rt = row / g.hb, rh = row - rt * g.hb;             // this row's token in a tile, and head
        // Queries of segment `next` (one warp, when the products with the ones before are done).
        const uint32_t qtile = static_cast<uint32_t>(g.hb) * g.tpt * D * 2;
        auto fetch_queries = [&](uint32_t next) {
            if (__any_sync(~0u, !wait_for(&ctl.seg_full[next % kSegs], (next / kSegs) & 1, abort_flag, p.wait_ns))) return;
            if (p.fault && next == 0) return;
            const PrefixSeg& d = ctl.segs[next % kSegs];
            if (lane == 0) {
                ctl.seg_end = next + 1;
                mbar_arrive_expect_tx(&ctl.q_full, qtile * d.nt);
            }
            __syncwarp();
            if (lane < 2 * KS * d.nt) {                              // 64 channels of a tile each
                const int tile = lane >= 2 * KS ? 1 : 0, c = lane - tile * 2 * KS;
                tma_load_3d(sQ + lane * C::QBOX, &qmap, &ctl.q_full, c * 64, d.head0, d.tok0 + tile * g.tpt);
            }
        };
        if (share > 0 && warp == 4) fetch_queries(0);
        uint32_t at = 0, u = 0, i0 = 0, ends = 0, twos = 0;          // place on the line; units, steps, steps with pv_done, segments of two tiles
        bool dead = false;
        for (uint32_t seg = 0; at < share; ++seg) {
            dead = !wait_for(&ctl.seg_full[seg % kSegs], (seg / kSegs) & 1, abort_flag, p.wait_ns);
            dead = __any_sync(~0u, dead);
            if (dead) break;
            const PrefixSeg& sg = ctl.segs[seg % kSegs];
            const uint32_t nt = sg.nt, n = sg.ke - sg.kb, steps = n * nt, cost = sg.cost;
            const uint32_t tile = nt == 2 ? (grp ^ i0) & 1 : 0;
            const int tok = static_cast<int>(tile) * g.tpt + rt;     // in the segment
            const bool valid = rt < g.tpt && tok < sg.tn && rh < sg.hv;
            const int lo = sg.q.lo, hi = valid ? seen(sg.q, sg.t0 + tok) : 0;
            const bool any = __any_sync(~0u, valid);
            const uint32_t ocol = lane_base + C::OCOL + tile * C::DV;
            float ref = kUnset, l = 0.f;
            for (uint32_t j = (grp ^ i0) & 1; j < steps; j += 2) {
                const uint32_t i = i0 + j, x = nt == 2 ? j >> 1 : j;
                if (!dead) dead = !wait_for(&ctl.s_full[grp], (i >> 1) & 1, abort_flag, p.wait_ns);
                if (nt == 1 && j > 0) {                              // the other group's reference
                    if (!dead) dead = !wait_for(&ctl.ref_done[grp ^ 1][q4], ((i - 1) >> 1) & 1, abort_flag, p.wait_ns);
                    const float r = ctl.ref[row];
                    if (r != ref) {
                        l *= ex2(ref - r);
                        ref = r;
                    }
                }
                dead = __any_sync(~0u, dead);
                if (dead) break;
                tc_fence_after();
                if (!any) {                                          // (P of rows without a query: their outputs are not written)
                    if (lane == 0) {
                        mbar_arrive(&ctl.ref_done[grp][q4]);
                        mbar_arrive(&ctl.p_full[grp]);
                    }
                    __syncwarp();
                    continue;
                }
                const int j0 = sg.row0 + (sg.kb + static_cast<int>(x)) * kUnit;
                const unsigned bad = *reinterpret_cast<volatile unsigned*>(&ctl.bad[(u + x) & 7]);
                if (j0 < lo || j0 + kUnit > sg.hi_min || bad) {      // hidden scores become -inf in tensor memory
#pragma unroll 1
                    for (int c = 0; c < 128; c += 32) {
                        const int a = lo - j0 - c, b = hi - j0 - c;  // columns [a, b) of these are seen
                        uint32_t on = b <= 0 || a >= 32 ? 0u : (b >= 32 ? ~0u : (1u << b) - 1) & (a <= 0 ? ~0u : ~0u << a);
                        for (int i = 0; bad && i < 32; i += 8)
                            if (paged_bad_row(g, bad, c + i)) on &= ~(255u << i);
                        if (__all_sync(~0u, on == ~0u || !valid)) continue;
                        uint32_t v[32];
                        DSV4_TMEM_LD_32x32b_X32(sbuf + c, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!(on & 1u << i)) v[i] = 0xFF800000u;
                        DSV4_TMEM_ST_32x32b_X32(sbuf + c, v);
                    }
                    DSV4_TMEM_WAIT_ST();
                }
                // The row's largest score, then its exponentials: the scores are read twice (a row's 128 in registers
                // throughout would leave none for the rest), the second time a quarter ahead of the exponentials.
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int h = 0; h < 128; h += 64) {
                    uint32_t v[64];
                    DSV4_TMEM_LD_32x32b_X64(sbuf + h, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 64; c += 2)
                        mx[(c >> 1) & 3] = max3(__uint_as_float(v[c]), __uint_as_float(v[c + 1]), mx[(c >> 1) & 3]);
                }
                uint32_t v[2][32];
                DSV4_TMEM_LD_32x32b_X32(sbuf, v[0]);
                mx[0] = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                const bool unset = ref == kUnset;
                const float top = fmaf(mx[0], p.scale2, unset ? 0.f : -ref);
                // A row that outruns its reference moves it (its first scores always do).
                const bool move = valid && (unset ? top > -INFINITY : top > kSpan);
                if (__any_sync(~0u, move)) {
                    const float f = move && !unset ? ex2(-top) : 1.f;
                    if (move) ref = unset ? top : ref + top;
                    l *= f;
                    if (x > 0 && __any_sync(~0u, f != 1.f)) {
                        // O by the factors, once the product before is done (of two tiles, this one's is: see above)
                        const uint32_t e = ends + j - 1;
                        if (!dead && nt == 1) dead = !wait_for(&ctl.pv_done[e & 1], (e >> 1) & 1, abort_flag, p.wait_ns);
                        dead = __any_sync(~0u, dead);
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < C::DV; c += 8) {
                            uint32_t r[8];
                            DSV4_TMEM_LD_32x32b_X8(ocol + c, r);
                            tmem_wait_ld();
#pragma unroll
                            for (int b = 0; b < 8; ++b) r[b] = __float_as_uint(__uint_as_float(r[b]) * f);
                            DSV4_TMEM_ST_32x32b_X8(ocol + c, r);
                        }
                        DSV4_TMEM_WAIT_ST();
                    }
                }
                if (nt == 1) ctl.ref[row] = ref;
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.ref_done[grp][q4]);
                // P = 2^(s - m) in bf16, over the scores (rounded: the tensor core takes bf16 beside bf16 V; the sum stays
                // in fp32)
                const float nref = ref == kUnset ? 0.f : -ref;
                const uint64_t nref2 = pack_f32x2(nref, nref);
                uint64_t sum[2] = {0ull, 0ull};
                auto exps = [&](int h) {
                    uint32_t o[16];
                    uint32_t (&now)[32] = v[h & 1], (&next)[32] = v[~h & 1];
                    tmem_wait_ld();
                    if (h < 3) DSV4_TMEM_LD_32x32b_X32(sbuf + 32 * h + 32, next);
#pragma unroll
                    for (int c = 0; c < 32; c += 2) {
                        uint64_t y = nref2;
                        fma_f32x2(y, pack_f32x2(__uint_as_float(now[c]), __uint_as_float(now[c + 1])), scale22);
                        float a, b;
                        unpack_f32x2(y, a, b);
                        a = ex2(a);
                        b = ex2(b);
                        add_f32x2(sum[(c >> 1) & 1], pack_f32x2(a, b));
                        o[c >> 1] = pack2(a, b);
                    }
                    DSV4_TMEM_ST_32x32b_X16(sbuf + 16 * h, o);
                };
                exps(0);
                exps(1);
                exps(2);
                exps(3);
                DSV4_TMEM_WAIT_ST();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.p_full[grp]);
                add_f32x2(sum[0], sum[1]);
                float sa, sb;
                unpack_f32x2(sum[0], sa, sb);
                l += sa + sb;
            }
            dead = __any_sync(~0u, dead);
            if (dead) break;
            // ---------------------------------------------------------------- the segment's part
            // (The segment's last scores have come to the warps of this group: its queries are read.)
            // The end of the last product, once the last step is known to have come to its softmax (the phase before is over
            // then). The warps of the same rows in both groups meet here: all that either waits for in the next segment comes
            // after all of this one.
            const uint32_t il = i0 + steps - 1 - (nt == 2 ? 1 - tile : 0);
            if (q4 == 0 && ((i0 + steps - 1) & 1) == static_cast<uint32_t>(grp) && at + cost < share) fetch_queries(seg + 1);
            if ((il & 1) != static_cast<uint32_t>(grp))
                dead = !wait_for(&ctl.ref_done[grp ^ 1][q4], (il >> 1) & 1, abort_flag, p.wait_ns);
            const uint32_t e = ends + steps - 1;
            if (!dead)
                dead = nt == 2 ? !wait_for(&ctl.o_done[grp], twos & 1, abort_flag, p.wait_ns)
                               : !wait_for(&ctl.pv_done[e & 1], (e >> 1) & 1, abort_flag, p.wait_ns);
            if (nt == 2) ++twos;
            else ends += steps;
            int ch0 = 0, chn = C::DV;                                // this warp's channels
            if (nt == 1) {                                           // both have the same rows: the last reference, both sums
                const float r = ctl.ref[row];
                ctl.l[grp][row] = r == ref ? l : l * ex2(ref - r);
                ref = r;
                ch0 = grp * (C::DV / 2);
                chn = C::DV / 2;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.l_ready[grp][q4]);
            if (!dead) dead = !wait_for(&ctl.l_ready[grp ^ 1][q4], seg & 1, abort_flag, p.wait_ns);
            if (nt == 1) l = ctl.l[0][row] + ctl.l[1][row];
            dead = __any_sync(~0u, dead);
            if (dead) break;
            tc_fence_after();
            const bool home = sg.kb == 0;
            const size_t qh = (static_cast<size_t>(sg.tok0 + (valid ? tok : 0)) * g.H + sg.head0 + (valid ? rh : 0));
            const int crow = static_cast<int>(tile) * 128 + row;
            float* dst;
            if (home) dst = p.home_o + (static_cast<size_t>(sg.q.own) * g.total_q * g.H + qh) * D + sg.half * 256 + ch0;
            else dst = p.cont_o + (static_cast<size_t>(worker) * C::TILES * 128 + crow) * C::DV + ch0;
            if (any) {
#pragma unroll 1
                for (int c = 0; c < chn; c += 32) {
                    uint32_t r[32];
                    DSV4_TMEM_LD_32x32b_X32(ocol + ch0 + c, r);
                    tmem_wait_ld();
                    if (valid) {
#pragma unroll
                        for (int b = 0; b < 32; b += 8) store32(dst + c + b, r + b);
                    }
                }
                if (valid && (nt == 2 || grp == 0)) {
                    // No row of this part is the query's, by its bounds or because their pages are not in the pool (then the
                    // sum is 0).
                    const bool none = min(hi, sg.row0 + sg.ke * kUnit) <= max(lo, sg.row0 + sg.kb * kUnit) ||
                                      (l == 0.f && (*reinterpret_cast<volatile uint32_t*>(&ctl.err) & DSV4_EWORD_BAD_INDEX));
                    const float m = none ? -INFINITY : ref;
                    if (home) {
                        int np = 1;
                        if (sg.ke < sg.n) {                          // the CTAs that go on with the segment
                            const long long end = sched.u0 + at + static_cast<long long>(sg.n) * sg.weight, T = sched.total;   // (home: the segment starts here)
                            int last = static_cast<int>((end * sched.ge - 1) / T);
                            while (last + 1 < sched.ge && T * (last + 1) / sched.ge < end) ++last;
                            while (T * last / sched.ge >= end) --last;
                            np = last - worker + 1;
                        }
                        const int info = worker | np << 8 | crow << 16;
                        p.home_ml[static_cast<size_t>(sg.q.own * C::HALVES + sg.half) * g.total_q * g.H + qh] =
                            make_float4(m, l, __int_as_float(info), __int_as_float(sg.q.own && lo > 0 ? 1 : 0));
                    } else {
                        p.cont_ml[static_cast<size_t>(worker) * C::TILES * 128 + crow] = make_float2(m, l);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.o_empty);        // (sg is not read any more)
            at += cost;
            u += n;
            i0 += steps;
        }
        dead = __any_sync(~0u, dead);
        if (dead && lane == 0) {
            atomicOr(&ctl.err, DSV4_EWORD_TIMEOUT);
            ctl.abort = 1;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (ctl.abort) {
        // A wait ran out in some role, and the others may have finished before it: the copies and
        // products still in flight end (each wait bounded) before memory is given up.
        if (warp == 1) {
            if (elect_one()) umma_commit(&ctl.drained);
            __syncwarp();
            mbar_wait(&ctl.drained, 0, nullptr, kDrainNs);
        }
        if (tid == 0) {
            const uint32_t seg = ctl.seg_end;
            if (seg && !p.fault) mbar_wait(&ctl.q_full, (seg - 1) & 1, nullptr, kDrainNs);
            for (int i = 0; i < ST; ++i)
                if (ctl.last[i]) mbar_wait(&ctl.full[ctl.last[i] & 1][i], ctl.last[i] >> 1 & 1, nullptr, kDrainNs);
        }
        __syncthreads();
    }
    if (warp == 2) tmem_dealloc(tmem, 512);
    if (tid == 0) p.err[blockIdx.x] = ctl.err;
}

// Joins each query's parts, and gathers the error bits. An item is 128 channels of one query: one warp, four
// channels per lane. Up to 16 parts of the prefix's rows and 16 of the query's own take one look: a lane each has a part's maximum
// and sum, and the first parts' outputs are on their way meanwhile. (Looking at up to 160 parts of either, as for a few
// queries over a long prefix, issued 300 instructions an item: 54 us for 1,415 tokens of 32 heads, now 33.)
constexpr int kMergeThreads = 256;

// One query's joined channels: rotated back, rounded, stored.
template <int D>
__device__ __forceinline__ void merge_store(const PrefixParams& p, size_t at, int tok, int ch, float (&o)[4]) {
    const int r0 = D - 2 * p.or_pairs;
    if (p.orp && ch + 3 >= r0) {
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            if (ch + i < r0) continue;
            const float2 cs = out_rope_angle(static_cast<double>(p.orp[tok]) * p.or_freq[(ch + i - r0) >> 1]);
            const float e = o[i], b = o[i + 1];
            o[i] = e * cs.x + b * cs.y;
            o[i + 1] = -e * cs.y + b * cs.x;
        }
    }
    *reinterpret_cast<uint2*>(p.out + at * D + ch) = make_uint2(pack2(o[0], o[1]), pack2(o[2], o[3]));
}

template <int D, bool MANY>
__global__ void __launch_bounds__(kMergeThreads, MANY ? 3 : 2)
prefix_merge_kernel(const __grid_constant__ PrefixParams p, int ctas, uint32_t* eword) {
    using C = XCfg<D>;
    constexpr int CH = D / 128, PL = 5;  // chunks of a query; parts of a segment per lane (at most 160)
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    if (blockIdx.x == 0 && warp == 0) {
        uint32_t err = 0;
        for (int c = lane; c < ctas; c += 32) err |= p.err[c];
        err = __reduce_or_sync(~0u, err);
        if (lane == 0) *eword = err;
    }
    const PagedGeom& g = p.g.p;
    const int first = min(max(g.cu_q[0], 0), g.total_q), end = min(max(g.cu_q[g.batch], 0), g.total_q);
    constexpr int WB = kMergeThreads / 32;
    const long long items = static_cast<long long>(max(end - first, 0)) * g.H * CH, step = static_cast<long long>(gridDim.x) * WB;
    const size_t kind = static_cast<size_t>(g.total_q) * g.H, row0 = static_cast<size_t>(first) * g.H;
    // an item's two records (the prefix's may be anything where the query has none)
    auto records = [&](long long it, float4& mp, float4& mo) {
        if (it >= items) return;
        const long long qh = it / CH;
        const int half = C::HALVES == 2 ? static_cast<int>(it - qh * CH) >> 1 : 0;
        mp = p.home_ml[half * kind + row0 + qh];
        mo = p.home_ml[(C::HALVES + half) * kind + row0 + qh];
    };
    long long it = static_cast<long long>(blockIdx.x) * WB + warp;
    float4 mp_next, mo_next;
    records(it, mp_next, mo_next);
    for (; it < items; it += step) {
        const float4 mp = mp_next, mo = mo_next;
        records(it + step, mp_next, mo_next);
        const long long qh = it / CH;
        const int chunk = static_cast<int>(it - qh * CH), half = C::HALVES == 2 ? chunk >> 1 : 0, ch = chunk * 128 + lane * 4;
        const size_t at = row0 + qh;
        const int tok = static_cast<int>(at / g.H), h = static_cast<int>(at - static_cast<size_t>(tok) * g.H);
        const bool two = __float_as_int(mo.w) == 1;
        const float snk = p.sink ? p.sink[h] * kLog2e : -INFINITY;
        int c0[2], np[2], row[2];
        const float* home[2], *cont[2];
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            const int info = __float_as_int(a ? mo.z : mp.z);
            c0[a] = info & 255;
            row[a] = min((info >> 16) & 0x7FFF, C::TILES * 128 - 1);
            np[a] = a || two ? min((info >> 8) & 255, ctas - c0[a]) : 0;
            home[a] = p.home_o + (a * kind + at) * D + ch;
            cont[a] = p.cont_o + (static_cast<size_t>(c0[a]) * C::TILES * 128 + row[a]) * C::DV + (ch - half * 256);
        }
        auto part = [&](int a, int i) {
            return *reinterpret_cast<const float4*>(i ? cont[a] + static_cast<size_t>(i) * C::TILES * 128 * C::DV : home[a]);
        };
        float o[4] = {0.f, 0.f, 0.f, 0.f}, f;
        auto add = [&](float e, const float4& v) {       // (a part that saw nothing may hold anything)
            if (e == 0.f) return;
            o[0] = fmaf(e, v.x, o[0]); o[1] = fmaf(e, v.y, o[1]);
            o[2] = fmaf(e, v.z, o[2]); o[3] = fmaf(e, v.w, o[3]);
        };
        auto finish = [&](float M, float top, float sum) {
            const float den = sum + (snk == -INFINITY ? 0.f : exp2f(snk - top));
            if (chunk == 0 && lane == 0 && p.lse)
                p.lse[at] = M == -INFINITY ? (p.sink ? p.sink[h] : -INFINITY) : top * kLn2 + logf(den);
            f = M == -INFINITY ? 0.f : 1.f / den;        // (-inf: no part had a row of the query's)
        };
        if (np[0] <= 16 && np[1] <= 16) {
            const int a = lane >> 4, i = lane & 15;
            float2 ml = make_float2(-INFINITY, 0.f);
            if (i < (a ? np[1] : np[0])) {
                if (i == 0) ml = a ? make_float2(mo.x, mo.y) : make_float2(mp.x, mp.y);
                else ml = p.cont_ml[static_cast<size_t>((a ? c0[1] : c0[0]) + i) * C::TILES * 128 + (a ? row[1] : row[0])];
            }
            float4 v0[2], v1[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (k < np[0]) v0[k] = part(0, k);
                if (k < np[1]) v1[k] = part(1, k);
            }
            float M = ml.x;
#pragma unroll
            for (int s = 16; s; s >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, s));
            const float top = fmaxf(M, snk), w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - top);
            float sum = ml.y * w;                        // (a part that holds NaN keeps it, also beside a weight of 0)
#pragma unroll
            for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(~0u, sum, s);
            finish(M, top, sum);
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll 1
                for (int k = 0; k < np[b]; k += 2) {
                    if (k) {
                        v0[0] = part(b, k);
                        if (k + 1 < np[b]) v0[1] = part(b, k + 1);
                    }
                    const float e0 = __shfl_sync(~0u, w, 16 * b + k), e1 = __shfl_sync(~0u, w, 16 * b + ((k + 1) & 15));
                    add(e0, b && !k ? v1[0] : v0[0]);
                    if (k + 1 < np[b]) add(e1, b && !k ? v1[1] : v0[1]);
                }
        } else if (MANY) {
            auto load = [&](int a, int i) {
                if (i == 0 && np[a] > 0) return a ? make_float2(mo.x, mo.y) : make_float2(mp.x, mp.y);
                return i < np[a] ? p.cont_ml[static_cast<size_t>(c0[a] + i) * C::TILES * 128 + row[a]] : make_float2(-INFINITY, 0.f);
            };
            float M = -INFINITY;
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll 1
                for (int i = lane; i < np[a]; i += 32) M = fmaxf(M, load(a, i).x);
#pragma unroll
            for (int s = 16; s; s >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, s));
            const float top = fmaxf(M, snk);
            float sum = 0.f;
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll 1
                for (int i0 = 0; i0 < np[a]; i0 += 32) {
                    const float2 ml = load(a, i0 + lane);
                    const float w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - top);
                    sum += ml.y * w;
#pragma unroll 1
                    for (int k = 0; k < 32 && i0 + k < np[a]; k += 2) {
                        const float4 v0 = part(a, i0 + k), v1 = i0 + k + 1 < np[a] ? part(a, i0 + k + 1) : v0;
                        const float e0 = __shfl_sync(~0u, w, k), e1 = __shfl_sync(~0u, w, k + 1);
                        add(e0, v0);
                        add(e1, v1);                     // (past the last part: a weight of 0)
                    }
                }
#pragma unroll
            for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(~0u, sum, s);
            finish(M, top, sum);
        } else {
            float w[2][PL], l[2][PL], M = -INFINITY;
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int k = 0; k < PL; ++k) {
                    const int i = lane + 32 * k;
                    float2 x = make_float2(-INFINITY, 0.f);
                    if (i == 0 && np[a] > 0) x = a ? make_float2(mo.x, mo.y) : make_float2(mp.x, mp.y);
                    else if (i < np[a]) x = p.cont_ml[static_cast<size_t>(c0[a] + i) * C::TILES * 128 + row[a]];
                    w[a][k] = x.x;
                    l[a][k] = x.y;
                    M = fmaxf(M, x.x);
                }
            float4 v[8];
            auto fetch = [&](int a, int i0) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i0 + i < np[a]) v[i] = part(a, i0 + i);
            };
            fetch(0, 0);
#pragma unroll
            for (int s = 16; s; s >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, s));
            const float top = fmaxf(M, snk);
            float sum = 0.f;
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int k = 0; k < PL; ++k) {
                    w[a][k] = w[a][k] == -INFINITY ? 0.f : exp2f(w[a][k] - top);
                    sum += l[a][k] * w[a][k];
                }
#pragma unroll
            for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(~0u, sum, s);
            finish(M, top, sum);
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                if (a) fetch(1, 0);
                for (int i0 = 0; i0 < np[a]; i0 += 8) {
                    float wk = w[a][0];
#pragma unroll
                    for (int k = 1; k < PL; ++k)
                        if (i0 >= 32 * k) wk = w[a][k];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float e = __shfl_sync(~0u, wk, (i0 + i) & 31);
                        if (i0 + i < np[a]) add(e, v[i]);
                    }
                    fetch(a, i0 + 8);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = f == 0.f ? 0.f : o[i] * f;
        merge_store<D>(p, at, tok, ch, o);
    }
}

int prefix_ctas() {
    const int n = sm_count();
    return n > 0 && n <= 160 ? n : 160;
}

struct PrefixWs {
    size_t home_ml, cont_ml, home_o, cont_o, plen, err, total;
};
PrefixWs prefix_ws(const dsv4_paged_prefix_args& a) {
    const size_t ctas = prefix_ctas(), th = static_cast<size_t>(a.total_q) * a.heads;
    const int tiles = a.dim == 128 ? 2 : 1, halves = a.dim == 512 ? 2 : 1, dv = a.dim == 512 ? 256 : a.dim;
    PrefixWs w{};
    size_t at = 0;
    auto take = [&](size_t bytes) { const size_t r = at; at += align_up(bytes, 256); return r; };
    w.home_ml = take(2 * halves * th * 16);
    w.cont_ml = take(ctas * tiles * 128 * 8);
    w.home_o = take(2 * th * a.dim * 4);
    w.cont_o = take(ctas * tiles * 128 * dv * 4);
    w.plen = take(ctas * a.groups * 4);
    w.err = take(ctas * 4);
    w.total = at + 256;                  // (the parts start at a multiple of 256, wherever the workspace does)
    return w;
}

template <int D>
int run(const dsv4_paged_prefix_args& a, uint8_t* ws, uint32_t* eword, cudaStream_t st) {
    using C = XCfg<D>;
    PrefixParams p{};
    p.g.p = paged_geom(a.block_table, a.cu_q, a.kv_len, a.batch, a.total_q, a.max_pages, a.page_size, a.num_pages, a.heads,
                       a.kv_heads, 0);
    paged_tile(p.g.p, 128);
    p.g.prefix_len = a.prefix_len;
    p.g.group_start = a.group_start;
    p.g.groups = a.groups;
    p.g.tiles = C::TILES;
    p.g.halves = C::HALVES;
    CUtensorMap qmap, kmap, vmap;
    if (!paged_query_map(&qmap, a.q, D, a.heads, a.total_q, a.q_stride, p.g.p.hb, p.g.p.tpt) ||
        !paged_pool_map(&kmap, a.k_pages, D, a.kv_heads, a.page_size, a.num_pages, p.g.p.br))
        return DSV4_ERR_LAUNCH;
    if (!a.v_pages) vmap = kmap;
    else if (!paged_pool_map(&vmap, a.v_pages, D, a.kv_heads, a.page_size, a.num_pages, p.g.p.br)) return DSV4_ERR_LAUNCH;
    auto kern = paged_prefix_kernel<D>;
    if (once_per_device(reinterpret_cast<const void*>(kern), kAttrLaunch, [kern] {
            return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        }) != cudaSuccess)
        return DSV4_ERR_LAUNCH;
    const int ctas = prefix_ctas();
    const PrefixWs w = prefix_ws(a);
    ws = reinterpret_cast<uint8_t*>(align_up(reinterpret_cast<uintptr_t>(ws), 256));
    p.home_ml = reinterpret_cast<float4*>(ws + w.home_ml);
    p.cont_ml = reinterpret_cast<float2*>(ws + w.cont_ml);
    p.home_o = reinterpret_cast<float*>(ws + w.home_o);
    p.cont_o = reinterpret_cast<float*>(ws + w.cont_o);
    p.plen = reinterpret_cast<int32_t*>(ws + w.plen);
    p.err = reinterpret_cast<uint32_t*>(ws + w.err);
    p.sink = a.sink;
    p.out = static_cast<__nv_bfloat16*>(a.out);
    p.lse = a.lse;
    p.scale2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
    p.negate = p.scale2 < 0.f;
    p.scale2 = std::fabs(p.scale2);
    if (p.scale2 == 0.f) p.scale2 = FLT_MIN;             // (a hidden row's -inf stays -inf, and any score is 0 beside a reference)
    p.orp = a.out_rope_pos;
    p.or_pairs = a.out_rope_pos ? a.out_rope_dim / 2 : 0;
    for (int j = 0; j < p.or_pairs; ++j) p.or_freq[j] = std::pow(a.out_rope_theta, -2.0 * j / a.out_rope_dim);
    p.shared = a.v_pages == nullptr;
    p.min_units = 6;                     // two units of one tile
    const WaitCtl wc = wait_ctl(DSV4_WAIT_FAULT_PAGED_PREFIX);
    p.fault = wc.fault;
    p.wait_ns = wc.wait_ns;
    count_launch();
    if (launch_k(kern, dim3(ctas), dim3(kThreads), C::SMEM, st, true, qmap, kmap, vmap, p) != cudaSuccess) return DSV4_ERR_LAUNCH;
    // With more items than two CTAs per SM have warps the merge takes three with fewer registers and two loads in flight per
    // item, else two with eight. Whole call: 1,415 tokens of 32 heads 580 us (584 in the other form), 48 of 16 heads x 512 154
    // (157). Left to itself the compiler takes 136 registers for the second form, and one CTA: 64 of 32 heads 76 us, not 73.
    const long long items = static_cast<long long>(a.total_q) * a.heads * (D / 128), wb = kMergeThreads / 32;
    const bool many = items > 2 * wb * ctas;
    const long long blocks = (items + wb - 1) / wb, most = 6 * ctas;
    auto merge = many ? prefix_merge_kernel<D, true> : prefix_merge_kernel<D, false>;
    count_launch();
    if (launch_k(merge, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), dim3(kMergeThreads), 0, st, true, p, ctas, eword) !=
        cudaSuccess)
        return DSV4_ERR_LAUNCH;
    return DSV4_OK;
}

}  // namespace

size_t paged_prefix_ws_bytes(const dsv4_paged_prefix_args& a) { return prefix_ws(a).total; }

int launch_paged_prefix(const dsv4_paged_prefix_args& a, uint8_t* ws, uint32_t* eword, cudaStream_t st) {
    if (a.batch == 0 || a.total_q == 0) return cudaMemsetAsync(eword, 0, 4, st) == cudaSuccess ? DSV4_OK : DSV4_ERR_LAUNCH;
    if (a.dim == 512) return run<512>(a, ws, eword, st);
    if (a.dim == 256) return run<256>(a, ws, eword, st);
    return run<128>(a, ws, eword, st);
}

}  // namespace dsv4
