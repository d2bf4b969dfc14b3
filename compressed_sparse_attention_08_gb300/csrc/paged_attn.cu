// Attention of a ragged batch of new tokens (one per sequence, or a chunk) over a paged cache.
//
//   s_j = scale q . k_j over the rows j the token sees,   m = max_j s_j (and the sink)
//   o = sum_j e^(s_j - m) v_j / (sum_j e^(s_j - m) + e^(sink - m)),   lse = m + log(that sum)
// Sources: "nvfp4-megamoe-kernel: compare v0.1-e2e-working...v-c1-c2-c3-20260602",
// fmha_6warp_tma_multirow_multitile.cuh "Sink bias correction" (the sink adds to the denominator
// only) and PERFORMANCE_AUDIT.md "P4" (V is the K row itself); "nvfp4-megamoe-kernel: compare
// master..pure-nvfp4", single_shot_inference.py eager_attention (sliding-window rows, inverse
// RoPE of the output). The pages keep dense per-sequence buffers; the paged form is this
// library's own.
//
// Persistent CTAs walk their shares of the work line (paged.cuh). Both products have the cache
// rows or the channels on the tensor core's 128 lanes and the queries on its columns: S^T = K Q^T
// (128 rows x N queries, one unit) and O^T += V^T P^T (128 channels per tile x N). So the number of
// query columns N is free (64 or 128), a single token's 64 heads fill a tile, and one
// shared-memory copy of a shared KV row serves as K (K-major) and as V (MN-major).
// Roles: warps 0, 2 and 3 move pages by TMA into a ring, a slot in turn each (a warp needs 300
// cycles for a slot and 70 to 120 for each box in it, however small), warp 1 issues tcgen05.mma, warps 4-19 do the
// softmax (a thread holds one cache row and a quarter of the queries; with 8 warps its chain of
// steps, not the tensor core, set the pace). The scores have two TMEM buffers, so S^T of unit
// u + 1 runs under the softmax of unit u.
//
// 512 channels: a tile is 128 KB and the ring holds no second one beside it. Kept for both products,
// it made loads, products and softmax take turns (7000 cycles per unit, of which the tensor core
// worked 3300). So the rows come in twice, as K and as V, in the order of use K0 K1 V0 K2 V1 ..:
// L2 has them the second time, and nothing waits for a whole tile (5100 cycles per unit: shared
// memory moves 640 KB per unit at the 128 bytes a cycle that it has). Slower were
// units of 64 rows, of which two fit the ring (S^T with M = 64 costs as much as with M = 128),
// and two CTAs with 256 channels each that exchange scores and P through distributed shared memory
// (which moved about 12 bytes a cycle).
//
// Measured (64 heads x 512, K = V): 2,048 tokens behind 14K rows 3.98 ms, 1,030 TFLOP/s, bound by
// shared memory; 16 single tokens over up to 8K rows 47 us (15 us of it HBM, the rest the start of cold
// CTAs and the merge); 4 over up to 256K rows 176 us, 5.05 TB/s. 32 heads over 8 of 128, tokens and
// chunks mixed: 228 us, 565 TFLOP/s, bound by a unit's chain of softmax steps.
#include <cmath>

#include "internal.h"
#include "paged.cuh"

namespace dsv4 {
namespace {

constexpr int kThreads = 640;
constexpr int kGroups = 4;                       // softmax: groups of 4 warps, one per quarter of the columns
constexpr int kSoftWarps = 16, kSoftThreads = 512, kSoftBar = 1;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// A query's reference maximum moves only when a score exceeds it by more than kSpan (base-2
// units): P = 2^(s - m) then stays far inside the fp32 and bf16 range, and o does not depend on
// which m was used.
constexpr float kSpan = 24.f;
// A query's reference until a score moves it: lower than any score but finite, so that a score of
// -inf gives P = 0 beside it, and not NaN. What a query sees is told by the bounds of its rows: a
// reference that never moved may also stand for scores that are all NaN or -inf.
constexpr float kUnset = -3.0e38f;

struct PagedAttnParams {
    PagedGeom g;
    const float* sink;                   // [H] or null
    __nv_bfloat16* out;                  // [total_q, H, D]
    float* lse;                          // [total_q, H] or null
    float* part_ml;                      // [2 * workers, N, 2]
    float* part_o;                       // [2 * workers, N, D]
    int* desc;                           // [workers, 8]
    uint32_t* err;                       // [CTAs] error bits
    float scale2;                        // scale * log2(e)
    const int64_t* orp;                  // [total_q] or null
    int or_pairs;
    int shared, min_units;
    int fault;                           // test control: a CTA's first query tile is never copied
    unsigned long long wait_ns;
    double or_freq[64];                  // theta^(-2j / out_rope_dim)
};

constexpr int kMaxSlots = 8;
constexpr int kSegs = 8;                 // tiles described at a time (the loads run at most three ahead of the outputs)
constexpr int kPT = kUnit;               // cache rows per unit
template <int N>
struct PagedCtl {
    uint64_t q_full, q_empty, full[kMaxSlots], empty[kMaxSlots], s_full[2], s_empty[2], p_full[2], pv_done[2];
    uint64_t v_ready, v_clean;           // V apart from K: an edge unit's rows have come, and are cleared
    uint64_t drained;                    // products in flight when a wait ran out
    uint32_t ring_end[kLoadWarps], seg_end[kLoadWarps];              // slots and query tiles that a load warp issued
    PagedSched sched;
    PagedSeg segs[kSegs];                // the tiles, written by the load warps for the softmax
    alignas(16) float nm[N];             // reference maxima (base-2 units), negated
    alignas(16) float f[N];              // factors
    uint32_t top[N];                     // a unit's maxima as ordered keys
    unsigned char tok[N];                // the column's token in the tile, 255: no query
    unsigned bad[8];
    uint32_t tmem, err;
    int abort;
};

// Shared memory: a ring of slots of 128 cache rows x 128 channels (two swizzled boxes), in which a
// K or V tile takes MT slots, so a slot is loaded again as soon as the product that reads it is
// done; the queries; P; and a few arrays per query.
template <int D_, int N_>
struct PCfg {
    static constexpr int D = D_, N = N_;
    static constexpr int MT = D / 128;
    static constexpr int BOX = kPT * 128;                    // 128 rows x 64 channels
    static constexpr int SLOT = 2 * BOX;
    static constexpr int QBOX = N * 128, QB = 2 * MT * QBOX;
    static constexpr int PB = kPT * N * 2, PN = D == 512 ? 2 : 1;    // P, and how many (two where the products are long)
    static constexpr int ST_FIT = (232448 - sizeof(PagedCtl<N>) - QB - PN * PB) / SLOT;
    static constexpr int ST = ST_FIT > kMaxSlots ? kMaxSlots : ST_FIT;
    static constexpr int OFF_Q = ST * SLOT, OFF_P = OFF_Q + QB, OFF_C = OFF_P + PN * PB;
    static constexpr int SMEM = OFF_C + sizeof(PagedCtl<N>);
    static constexpr int TCOLS = 512;
    static constexpr int OCOL = 2 * N;
    static_assert(ST >= MT && SMEM <= 232448 && OCOL + MT * N <= 512, "one tile, and all accumulators in TMEM");
    static constexpr bool KEEP = ST >= 2 * MT;               // a shared K/V tile stays for both products
};

// Whether the unit that starts at row j0 holds rows that no token of the tile sees.
__device__ __forceinline__ bool unit_edge(const PagedGeom& g, const PagedSeg& sg, int j0, unsigned bad) {
    return j0 < sg.lo_u || j0 + kUnit > sg.hi_u || bad != 0;
}

// Places of unit u's tiles in the order of loading, in tiles: K0 K1 V0 K2 V1 .. V_last for each
// query tile, or one tile for both. (V_last before the next query tile's K0: its product ends this tile.)
__device__ __forceinline__ uint32_t k_place(bool keep, uint32_t u, bool first) { return keep ? u : 2 * u - (first ? 0 : 1); }
__device__ __forceinline__ uint32_t v_place(bool keep, uint32_t u, bool last) { return keep ? u : 2 * u + (last ? 1 : 2); }

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// K values per lane, reduced over the warp's lanes: lane i returns the reduction of value i mod K
// (K: 8, 16 or 32).
template <bool kMax, int K>
__device__ __forceinline__ float lanes_reduce(float (&v)[K], int lane) {
#pragma unroll
    for (int w = 16; w >= K; w >>= 1)
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const float got = __shfl_xor_sync(0xffffffffu, v[i], w);
            v[i] = kMax ? fmaxf(v[i], got) : v[i] + got;
        }
#pragma unroll
    for (int w = K / 2; w >= 1; w >>= 1) {
        const bool upper = (lane & w) != 0;
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float keep = upper ? v[i + w] : v[i];
            const float send = upper ? v[i] : v[i + w];
            const float got = __shfl_xor_sync(0xffffffffu, send, w);
            v[i] = kMax ? fmaxf(keep, got) : keep + got;
        }
    }
    return v[0];
}

__device__ __forceinline__ bool soft_sync_or(bool x) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
                 "barrier.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r) : "r"(static_cast<uint32_t>(x)), "n"(kSoftBar), "n"(kSoftThreads) : "memory");
    return r != 0;
}
__device__ __forceinline__ void soft_sync() { named_bar_sync(kSoftBar, kSoftThreads); }

// (cos, sin) of the inverse rotation of pair j of token tok. Not inlined: sixteen copies of it in
// the output loops pushed the code around them out of the instruction cache.
__device__ __noinline__ float2 out_rope_angle(double a) {
    float sn, cs;
    sincosf(reduced_angle(a), &sn, &cs);
    return make_float2(cs, sn);
}
__device__ __forceinline__ float2 out_rope_cs(const PagedAttnParams& p, int tok, int j) {
    return out_rope_angle(static_cast<double>(p.orp[tok]) * p.or_freq[j]);
}

// The lse of a query that sees nothing: its sink, as given (in base-2 units the type's lowest
// values would leave the range).
__device__ __forceinline__ float own_sink(const PagedAttnParams& p, int h) { return p.sink ? p.sink[h] : -INFINITY; }

// NT TMEM columns of this thread's lane.
template <int NT>
__device__ __forceinline__ void tmem_cols(uint32_t addr, uint32_t (&r)[NT]) {
    if constexpr (NT == 32) {
        DSV4_TMEM_LD_32x32b_X32(addr, r);
    } else {
        static_assert(NT == 16, "columns per thread");
        DSV4_TMEM_LD_32x32b_X16(addr, r);
    }
}

template <int D, int N>
__global__ void __launch_bounds__(kThreads, 1)
paged_attn_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap, const __grid_constant__ PagedAttnParams p) {
    using C = PCfg<D, N>;
    constexpr int ST = C::ST, MT = C::MT;
    constexpr int NE = N / kGroups;                                  // scores of a unit per softmax thread: one row
    constexpr bool LATE = NE <= 16;
    extern __shared__ __align__(1024) uint8_t sm[];
    PagedCtl<N>& ctl = *reinterpret_cast<PagedCtl<N>*>(sm + C::OFF_C);
    uint8_t* sQ = sm + C::OFF_Q;
    uint8_t* sP = sm + C::OFF_P;
    float *s_nm = ctl.nm, *s_f = ctl.f;
    volatile int* abort_flag = &ctl.abort;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int worker = blockIdx.x, workers = gridDim.x;
    if (tid == 0) {
        tma_prefetch_desc(&qmap);
        tma_prefetch_desc(&kmap);
        tma_prefetch_desc(&vmap);
        mbar_init(&ctl.q_full, kLoadWarps);
        mbar_init(&ctl.q_empty, 1);
        for (int i = 0; i < ST; ++i) { mbar_init(&ctl.full[i], 1); mbar_init(&ctl.empty[i], 1); }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl.s_full[i], 1);
            mbar_init(&ctl.s_empty[i], kSoftWarps);
            mbar_init(&ctl.p_full[i], kSoftWarps);
            mbar_init(&ctl.pv_done[i], 1);
        }
        mbar_init(&ctl.v_ready, 1);
        mbar_init(&ctl.v_clean, kSoftWarps);
        mbar_init(&ctl.drained, 1);
        ctl.abort = 0;
        ctl.err = 0;
        fence_barrier_init();
    }
    if (tid < N) ctl.top[tid] = 0;
    if (warp == 2) tmem_alloc(&ctl.tmem, C::TCOLS);
    pdl_trigger();
    pdl_wait();                          // lengths, queries and rows may come from the kernel before
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem;
    paged_schedule<kThreads>(p.g, worker, workers, p.min_units, reinterpret_cast<long long*>(sm), &ctl.sched, &ctl.err);
    // the schedule's scratch is overwritten by TMA next
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();

    const PagedGeom& g = p.g;
    const PagedSched& sched = ctl.sched;
    const bool keep = C::KEEP && p.shared;               // K rows stay in place as V
    const uint32_t units = static_cast<uint32_t>(sched.u1 - sched.u0);
    if (warp == 0 || warp == 2 || warp == 3) {
        // ---------------------------------------------------------------- pages and queries
        // Three warps walk the same slots and take them in turn.
        const int mine = warp == 0 ? 0 : warp - 1;
        PagedWalk w(g, sched);
        PagedSeg sg;
        const uint32_t qbytes = static_cast<uint32_t>(g.hb) * g.tpt * D * 2;
        const int piece = lane >> 1, box = lane & 1;
        uint32_t ring = 0, seg = 0;
        bool dead = false, more = w.next(sg);
        PagedLook cur{0, 0, false}, prev{0, 0, false};
        if (more) cur = paged_look(g, sg, sg.row0 + sg.kb * kPT, lane);
        int k = more ? sg.kb : 0;
        // one tile (K, or V of the unit before) into the next MT slots
        auto load = [&](const CUtensorMap* map, const PagedLook& t, int kvh, int unit) {
            const PagedBoxes bx = paged_boxes(g, t);
            const uint32_t bytes = static_cast<uint32_t>(__popc(bx.ok)) * g.br * 128;
#pragma unroll 1
            for (int mt = 0; mt < MT; ++mt, ++ring) {
                if (ring % kLoadWarps != static_cast<uint32_t>(mine)) continue;
                const uint32_t slot = ring % ST;
                if (ring >= ST)
                    dead = __any_sync(~0u, !mbar_wait(&ctl.empty[slot], (ring / ST - 1) & 1, abort_flag, p.wait_ns));
                if (dead) return;
                if (lane == 0) {
                    if (mt == 0 && unit >= 0) {
                        ctl.bad[unit & 7] = bx.bad;
                        if (bx.bad) atomicOr(&ctl.err, DSV4_EWORD_BAD_INDEX);
                    }
                    if (bytes) mbar_arrive_expect_tx(&ctl.full[slot], bytes);
                    else mbar_arrive(&ctl.full[slot]);
                }
                __syncwarp();
                if ((bx.ok >> lane) & 1)
                    tma_load_4d(sm + slot * C::SLOT + box * C::BOX + piece * g.br * 128, map, &ctl.full[slot], mt * 128 + box * 64,
                                kvh, t.slot, t.page);
            }
        };
        for (int u = 0; !dead && more; ++u) {
            if (k == sg.kb) {                        // a new row tile
                if (seg > 0) dead = __any_sync(~0u, !mbar_wait(&ctl.q_empty, (seg - 1) & 1, abort_flag, p.wait_ns));
                if (dead) break;
                if (lane == 0) {
                    if (mine == 0) ctl.segs[seg % kSegs] = sg;
                    const bool skip = p.fault && seg == 0;
                    if (!skip && mine == 0) mbar_arrive_expect_tx(&ctl.q_full, qbytes);
                    else if (!skip) mbar_arrive(&ctl.q_full);
#pragma unroll 1
                    for (int b = skip ? 2 * MT : mine; b < 2 * MT; b += kLoadWarps)
                        tma_load_3d(sQ + b * C::QBOX, &qmap, &ctl.q_full, b * 64, sg.head0, sg.tok0);
                }
                ++seg;
            }
            // the pages of the next unit are looked up while this one's copies wait
            const int kvh = sg.kvh;
            const bool first = k == sg.kb, last = k + 1 == sg.ke;
            PagedLook next{0, 0, false};
            if (++k >= sg.ke) {
                more = w.next(sg);
                k = more ? sg.kb : 0;
            }
            if (more) next = paged_look(g, sg, sg.row0 + k * kPT, lane);
            load(&kmap, cur, kvh, u);
            if (!keep && !dead && !first) load(&vmap, prev, kvh, -1);
            if (!keep && !dead && last) load(&vmap, cur, kvh, -1);
            prev = cur;
            cur = next;
        }
        if (lane == 0) {
            ctl.ring_end[mine] = ring;
            ctl.seg_end[mine] = seg;
            if (dead) {
                atomicOr(&ctl.err, DSV4_EWORD_TIMEOUT);
                ctl.abort = 1;
            }
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- tensor core
        PagedWalk w(g, sched);
        PagedSeg sg;
        uint32_t u = 0, seg = 0, pend_u = 0, pend_place = 0;
        uint32_t edges = 0;
        bool dead = false, pend = false, pend_first = false, pend_edge = false;
        const bool one = elect_one();
        // (the warp stays together: a wait that runs out does so for all lanes)
        auto wait = [&](uint64_t* bar, uint32_t parity) { return !__any_sync(~0u, !mbar_wait(bar, parity & 1, abort_flag, p.wait_ns)); };
        const uint32_t q0 = smem_u32(sQ), t0 = smem_u32(sm);
        const uint32_t idS = idesc_bf16_f32(kPT, N), idO = idesc_bf16_f32(128, N) | (1u << 15) | (1u << 16);
        const uint64_t pdesc0 = sdesc_mnmajor_sw128(smem_u32(sP), kPT * 128, 1024u);
        // (descriptors advance by 16-byte units)
        auto pv = [&](uint32_t x, uint32_t place, bool first, bool edge) {   // O^T += V^T P^T of unit x
            if (!wait(&ctl.p_full[x & 1], x >> 1)) return false;
            uint32_t r = place * MT;
            if (!keep && edge) {                     // its rows come, and those that nobody sees are cleared
                for (int mt = 0; mt < MT; ++mt)
                    if (!wait(&ctl.full[(r + mt) % ST], (r + mt) / ST)) return false;
                if (lane == 0) mbar_arrive(&ctl.v_ready);
                if (!wait(&ctl.v_clean, edges)) return false;
                ++edges;
            }
            const uint64_t pdesc = pdesc0 + (x % C::PN) * (C::PB / 16);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt, ++r) {
                const uint32_t slot = r % ST;
                if (!keep && !wait(&ctl.full[slot], r / ST)) return false;
                tc_fence_after();
                const uint64_t a = sdesc_mnmajor_sw128(t0 + slot * C::SLOT, C::BOX, 1024u);
                const uint32_t d = tmem + static_cast<uint32_t>(C::OCOL + mt * N);
                if (one) {
#pragma unroll
                    for (int kk = 0; kk < kPT / 16; ++kk)
                        umma_bf16(d, a + kk * 128, pdesc + kk * 128, idO, kk > 0 ? 1u : (first ? 0u : 1u));
                    umma_commit(&ctl.empty[slot]);
                }
                __syncwarp();
            }
            if (one) umma_commit(&ctl.pv_done[x & 1]);
            __syncwarp();
            return true;
        };
        while (!dead && w.next(sg)) {
            dead = !wait(&ctl.q_full, seg);
            ++seg;
            for (int k = sg.kb; k < sg.ke && !dead; ++k, ++u) {
                uint32_t r = k_place(keep, u, k == sg.kb) * MT;
                if (pend && keep) {
                    // Whichever can start: this unit's scores (first, if both), or the product with V
                    // of the unit before, whose slots this unit's rows may be waiting for. (Rows that
                    // come in twice have their order.)
                    const uint32_t last = r + MT - 1;
                    const uint64_t t_start = global_timer_ns();
                    for (uint32_t it = 1;; ++it) {
                        if (__all_sync(~0u, mbar_test(&ctl.full[last % ST], (last / ST) & 1))) break;
                        if (__all_sync(~0u, mbar_test(&ctl.p_full[pend_u & 1], (pend_u >> 1) & 1))) {
                            dead = !pv(pend_u, pend_place, pend_first, pend_edge);
                            pend = false;
                            break;
                        }
                        if ((it & 255u) == 0u &&
                            __any_sync(~0u, *abort_flag != 0 || global_timer_ns() - t_start > p.wait_ns)) { dead = true; break; }
                    }
                }
                if (!dead && u >= 2) dead = !wait(&ctl.s_empty[u & 1], (u >> 1) - 1);
                const uint32_t d = tmem + (u & 1) * N;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt, ++r) {           // S^T = K Q^T
                    const uint32_t slot = r % ST;
                    dead = dead || !wait(&ctl.full[slot], r / ST);
                    if (dead) break;
                    tc_fence_after();
                    const uint64_t a = sdesc_kmajor_sw128(t0 + slot * C::SLOT), b = sdesc_kmajor_sw128(q0 + mt * 2 * C::QBOX);
                    if (one) {
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            umma_bf16(d, a + (kk >> 2) * (C::BOX / 16) + (kk & 3) * 2, b + (kk >> 2) * (C::QBOX / 16) + (kk & 3) * 2,
                                      idS, mt > 0 || kk > 0 ? 1u : 0u);
                        if (!keep) umma_commit(&ctl.empty[slot]);
                    }
                    __syncwarp();
                }
                if (dead) break;
                if (one) {
                    umma_commit(&ctl.s_full[u & 1]);
                    if (k + 1 == sg.ke) umma_commit(&ctl.q_empty);
                }
                __syncwarp();
                if (pend) dead = !pv(pend_u, pend_place, pend_first, pend_edge);
                pend = true;
                pend_u = u;
                pend_place = v_place(keep, u, k + 1 == sg.ke);
                pend_first = k == sg.kb;
                pend_edge = unit_edge(g, sg, sg.row0 + k * kPT, ctl.bad[u & 7]);
            }
            // the tile's last product first: its outputs are waited for, the next tile's scores are not
            if (!dead && pend) dead = !pv(pend_u, pend_place, pend_first, pend_edge);
            pend = false;
        }
        if (dead && lane == 0) {
            atomicOr(&ctl.err, DSV4_EWORD_TIMEOUT);
            ctl.abort = 1;
        }
    } else {
        // ---------------------------------------------------------------- softmax and output
        const int st = tid - 128, q4 = warp & 3, grp = (warp - 4) >> 2;
        const int c0 = grp * (N / kGroups);                          // columns of this thread's group
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(q4 * 32) << 16);
        const int row = q4 * 32 + lane;                              // cache row of the unit, channel of an O tile
        const uint64_t scale22 = pack_f32x2(p.scale2, p.scale2);
        auto pv_over = [&](uint32_t x) { return mbar_wait(&ctl.pv_done[x & 1], (x >> 1) & 1, abort_flag, p.wait_ns); };
        uint32_t u = 0, edges = 0;
        bool dead = false;
        const int ct = st / g.hb;                                    // column st's token in a tile
        int* desc = p.desc + worker * 8;
        if (st == 0) desc[0] = 0;
        for (uint32_t tile = 0; u < units; ++tile) {
            // The tile's description stays in shared memory (walked here it took the registers that the
            // scores need): its first scores come after it. All warps go on, or none.
            if (!dead) dead = !mbar_wait(&ctl.s_full[u & 1], (u >> 1) & 1, abort_flag, p.wait_ns);
            if (soft_sync_or(dead)) break;                           // (and the tile before is written out)
            const PagedSeg& sg = ctl.segs[tile % kSegs];
            if (st < N) {
                const int h = st - ct * g.hb;
                const bool ok = ct < sg.tn && h < sg.hv;
                s_nm[st] = ok ? -kUnset : -INFINITY;                 // (a column without a query gets P = 0)
                ctl.tok[st] = ok ? ct : 255;
            }
            soft_sync();
            const int base = sg.q.L - sg.q.n + sg.t0;                // row of the tile's first token
            float sink = -INFINITY;                                  // of column st (read now, needed at the end)
            if (p.sink && st < N && ctl.tok[st] != 255) sink = p.sink[sg.head0 + st - ctl.tok[st] * g.hb] * kLog2e;
            uint64_t lacc[NE / 2];                                   // this row's P per query (pairs), summed over the units
#pragma unroll
            for (int i = 0; i < NE / 2; ++i) lacc[i] = 0ull;
            for (int k = sg.kb; k < sg.ke; ++k, ++u) {
                if (!dead) dead = !mbar_wait(&ctl.s_full[u & 1], (u >> 1) & 1, abort_flag, p.wait_ns);
                tc_fence_after();
                const int j0 = sg.row0 + k * kPT;
                const unsigned bad = *reinterpret_cast<volatile unsigned*>(&ctl.bad[u & 7]);
                const bool edge = unit_edge(g, sg, j0, bad);
                const bool masked = edge || j0 < sg.lo_max || j0 + kPT > sg.hi_min;
                auto live = [&](int r) { return j0 + r >= sg.lo_u && j0 + r < sg.hi_u && !paged_bad_row(g, bad, r); };
                const uint32_t scol = lane_base + (u & 1) * N + c0;
                float x[NE];
                auto scores = [&] {
                    uint32_t raw[NE];
                    tmem_cols<NE>(scol, raw);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < NE; ++i) x[i] = __uint_as_float(raw[i]);
                };
                auto hide = [&] {
                    // this row is seen by the tile's tokens t_lo .. t_hi
                    const bool on = live(row);
                    const int t_lo = on ? j0 + row - base : 1;
                    const int t_hi = on ? (g.window > 0 ? j0 + row - base + g.window - 1 : 254) : 0;
#pragma unroll
                    for (int i = 0; i < NE; i += 4) {
                        const uint32_t t4 = *reinterpret_cast<const uint32_t*>(ctl.tok + c0 + i);
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            const int t = (t4 >> (8 * b)) & 255;
                            if (t < t_lo || t > t_hi) x[i + b] = -INFINITY;
                        }
                    }
                };
                auto less_ref = [&] {                // base-2 scores relative to the references
#pragma unroll
                    for (int i = 0; i < NE; i += 4) {
                        ulonglong2 y = *reinterpret_cast<const ulonglong2*>(s_nm + c0 + i);
                        uint64_t y0 = y.x, y1 = y.y;
                        fma_f32x2(y0, pack_f32x2(x[i], x[i + 1]), scale22);
                        fma_f32x2(y1, pack_f32x2(x[i + 2], x[i + 3]), scale22);
                        unpack_f32x2(y0, x[i], x[i + 1]);
                        unpack_f32x2(y1, x[i + 2], x[i + 3]);
                    }
                    if (masked) hide();
                };
                // P = 2^(s - m) in bf16 (rounded: the tensor core takes bf16 beside bf16 V; the sum stays in
                // fp32. The outputs' error against 64 bits, relative to their size, is 0.0019 to 0.0023
                // with it and 0.0017, their own rounding, without),
                // the MN-major operand: a cache row's 64 queries are one 128-byte line
                uint8_t* pbuf = sP + (u % C::PN) * C::PB;
                auto put = [&] {
                    // its place is free once the product that read it is done
                    if (!dead && u >= C::PN) dead = !pv_over(u - C::PN);
#pragma unroll
                    for (int i = 0; i < NE; ++i) x[i] = ex2(x[i]);
                    uint8_t* line = pbuf + (c0 >> 6) * (kPT * 128) + (row >> 3) * 1024 + (row & 7) * 128;
#pragma unroll
                    for (int i = 0; i < NE / 8; ++i)
                        *reinterpret_cast<uint4*>(line + (((((c0 & 63) >> 3) + i) ^ (row & 7)) << 4)) =
                            make_uint4(pack2(x[8 * i], x[8 * i + 1]), pack2(x[8 * i + 2], x[8 * i + 3]),
                                       pack2(x[8 * i + 4], x[8 * i + 5]), pack2(x[8 * i + 6], x[8 * i + 7]));
                };
                auto add_up = [&] {
#pragma unroll
                    for (int i = 0; i < NE; i += 2) add_f32x2(lacc[i / 2], pack_f32x2(x[i], x[i + 1]));
                };
                auto outrun = [&] {
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < NE; i += 2) mx[(i >> 1) & 3] = fmaxf(fmaxf(x[i], x[i + 1]), mx[(i >> 1) & 3]);
                    return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) > kSpan;
                };
                // A unit that outruns the references (the warps vote; a tile's first unit always) moves them.
                // With few scores per thread the vote comes after P, so that the warps need not wait for
                // one another between their steps, and P is formed again where it was too soon; with many,
                // what is held across the vote would not fit.
                bool rescale = false, over = k == sg.kb;
                if (!over) {
                    scores();
                    less_ref();
                    const bool mine = outrun();
                    if (LATE) put();
                    over = soft_sync_or(mine);
                }
                if (over) {                          // the unit's maxima, and the references above theirs
                    scores();
#pragma unroll
                    for (int i = 0; i < NE; ++i) x[i] *= p.scale2;
                    if (masked) hide();
                    const float top = lanes_reduce<true>(x, lane);
                    atomicMax(&ctl.top[c0 + (lane & (NE - 1))], float_to_key(top));
                    soft_sync();
                    if (st < N) {
                        const float cm = key_to_float(ctl.top[st]);
                        const float mo = -s_nm[st];
                        float f = 1.f;
                        if (cm > mo) {
                            f = mo == kUnset ? 0.f : ex2(mo - cm);
                            s_nm[st] = -cm;
                            rescale = k > sg.kb;
                        }
                        s_f[st] = f;
                        ctl.top[st] = 0;
                    }
                    rescale = soft_sync_or(rescale);
                    if (rescale) {
#pragma unroll
                        for (int i = 0; i < NE; i += 2)
                            lacc[i / 2] = mul_f32x2(lacc[i / 2], *reinterpret_cast<const uint64_t*>(s_f + c0 + i));
                    }
                    scores();
                    less_ref();
                }
                if (!LATE || over) put();
                add_up();
                if (rescale) {                       // O^T by the factors of the references that moved
                    if (!dead) dead = !pv_over(u - 1);
                    tc_fence_after();
#pragma unroll 1
                    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll 1
                        for (int c = c0; c < c0 + N / kGroups; c += 8) {
                            uint32_t r[8];
                            const uint32_t ta = lane_base + C::OCOL + mt * N + c;
                            DSV4_TMEM_LD_32x32b_X8(ta, r);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 8; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * s_f[c + i]);
                            DSV4_TMEM_ST_32x32b_X8(ta, r);
                        }
                    }
                    DSV4_TMEM_WAIT_ST();
                }
                // Rows of the tile that nobody may see (past the cache, before the window, of a page that was
                // not loaded) hold anything: as V they must not meet P = 0.
                auto clear_rows = [&] {
                    const int zr = st & (kPT - 1);
                    if (live(zr)) return;
#pragma unroll 1
                    for (int b = st / kPT; b < 2 * MT; b += kSoftThreads / kPT) {
                        const uint32_t slot = (v_place(keep, u, k + 1 == sg.ke) * MT + (b >> 1)) % ST;
                        uint4* z = reinterpret_cast<uint4*>(sm + slot * C::SLOT + (b & 1) * C::BOX + zr * 128);
#pragma unroll
                        for (int i = 0; i < 8; ++i) z[i ^ (zr & 7)] = make_uint4(0, 0, 0, 0);    // (eight rows, eight banks)
                    }
                };
                if (edge && keep) clear_rows();
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&ctl.s_empty[u & 1]);
                    mbar_arrive(&ctl.p_full[u & 1]);
                }
                if (edge && !keep) {
                    if (!dead) dead = !mbar_wait(&ctl.v_ready, edges & 1, abort_flag, p.wait_ns);
                    ++edges;
                    clear_rows();
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl.v_clean);
                }
            }
            // ---------------------------------------------------------------- the tile's results
            if (!dead) dead = !pv_over(u - 1);
            tc_fence_after();
            float* red = reinterpret_cast<float*>(sP);               // [4][N] (P is read)
            {
                float l[NE];
#pragma unroll
                for (int i = 0; i < NE; i += 2) unpack_f32x2(lacc[i / 2], l[i], l[i + 1]);
                const float sum = lanes_reduce<false>(l, lane);
                if (lane < NE) red[q4 * N + c0 + lane] = sum;
            }
            soft_sync();
            const bool whole = sg.kb == 0 && sg.ke == sg.n;
            const int slot2 = worker * 2 + (sg.kb > 0 ? 0 : 1);
            if (st < N) {
                const int c = st;
                const float l = (red[c] + red[N + c]) + (red[2 * N + c] + red[3 * N + c]);
                const float m = -s_nm[c];
                const int t = ctl.tok[c];
                // No row of this part is the query's, by its bounds or because their pages are not in
                // the pool (then the sum is 0).
                const bool none = t == 255 || (l == 0.f && (ctl.err & DSV4_EWORD_BAD_INDEX)) ||
                                  min(paged_hi(sg.q, sg.t0 + t), sg.row0 + sg.ke * kPT) <=
                                      max(paged_lo(g, sg.q, sg.t0 + t), sg.row0 + sg.kb * kPT);
                if (whole) {
                    float f = 0.f;
                    if (t != 255) {
                        const int h = sg.head0 + c - t * g.hb;
                        const float snk = sink;
                        const float M = fmaxf(m, snk);
                        const float e = exp2f(m - M);
                        const float den = l * e + (snk == -INFINITY ? 0.f : exp2f(snk - M));
                        if (!none) f = e / den;      // (0/0 where every score is -inf)
                        if (p.lse)
                            p.lse[static_cast<size_t>(sg.tok0 + t) * g.H + h] = none ? own_sink(p, h) : M * kLn2 + logf(den);
                    }
                    s_f[c] = f;
                } else {
                    float* ml = p.part_ml + (static_cast<size_t>(slot2) * N + c) * 2;
                    ml[0] = none ? -INFINITY : m;
                    ml[1] = l;
                }
            }
            soft_sync();
            const int cols = (sg.tn - 1) * g.hb + sg.hv;             // (no query behind them)
            float* po = p.part_o + static_cast<size_t>(slot2) * N * D;
            __nv_bfloat16* ob = p.out + (static_cast<size_t>(sg.tok0) * g.H + sg.head0) * D;
            const int r0 = D - 2 * p.or_pairs;
#pragma unroll 1
            for (int cb = c0; cb < c0 + NE && cb < cols; cb += 16) {
                // Two columns at a time: even lanes write the first, odd lanes the second, each a pair
                // of neighbouring channels.
                int off[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int c = cb + 2 * i + (lane & 1), t = ctl.tok[c];
                    off[i] = t == 255 ? -1 : (t * g.H + c - t * g.hb) * D;
                }
#pragma unroll 1
                for (int mt = 0; mt < MT; ++mt) {
                    uint32_t r[16];
                    DSV4_TMEM_LD_32x32b_X16(lane_base + C::OCOL + mt * N + cb, r);
                    tmem_wait_ld();
                    if (!whole) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) po[(cb + i) * D + mt * 128 + row] = __uint_as_float(r[i]);
                        continue;
                    }
                    const int d = mt * 128 + (row & ~1);             // this lane's pair of channels
                    float e[8], o[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        // (a factor of 0 stands for a query that sees nothing: O may hold anything)
                        const float2 f = *reinterpret_cast<const float2*>(s_f + cb + 2 * i);
                        const float a = f.x == 0.f ? 0.f : __uint_as_float(r[2 * i]) * f.x;
                        const float b = f.y == 0.f ? 0.f : __uint_as_float(r[2 * i + 1]) * f.y;
                        const float got = __shfl_xor_sync(~0u, (lane & 1) ? a : b, 1);
                        e[i] = (lane & 1) ? got : a;
                        o[i] = (lane & 1) ? b : got;
                    }
                    if (p.orp && mt * 128 + q4 * 32 + 31 >= r0) {    // (a warp's 32 channels: apart, or the branches below cost all)
                        int rt = 255;
                        float2 cs = make_float2(1.f, 0.f);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int t = ctl.tok[cb + 2 * i + (lane & 1)];
                            if (d < r0 || t == 255) continue;
                            if (t != rt) { cs = out_rope_cs(p, sg.tok0 + t, (d - r0) >> 1); rt = t; }
                            const float e0 = e[i];
                            e[i] = e0 * cs.x + o[i] * cs.y;
                            o[i] = -e0 * cs.y + o[i] * cs.x;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (off[i] >= 0) *reinterpret_cast<uint32_t*>(ob + off[i] + d) = pack2(e[i], o[i]);
                }
            }
            if (st == 0 && !whole && sg.kb == 0) {                   // this worker starts the tile: it is merged under its number
                const long long end = sched.u0 + u - sg.ke + sg.n, T = sched.total;
                int last = static_cast<int>((end * sched.ge - 1) / T);
                while (last + 1 < sched.ge && T * (last + 1) / sched.ge < end) ++last;
                while (T * last / sched.ge >= end) --last;
                desc[0] = last - worker + 1;
                desc[1] = sg.tok0;
                desc[2] = sg.tn;
                desc[3] = sg.head0;
                desc[4] = sg.hv;
            }
        }
        dead = __any_sync(~0u, dead);                                // (each lane waits for itself: any of them may run out)
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
            const uint32_t seg = max(max(ctl.seg_end[0], ctl.seg_end[1]), ctl.seg_end[2]);
            if (seg && !p.fault) mbar_wait(&ctl.q_full, (seg - 1) & 1, nullptr, kDrainNs);
            ring_drain<ST>(ctl.full, ctl.ring_end);
        }
        __syncthreads();
    }
    if (warp == 2) tmem_dealloc(tmem, C::TCOLS);
    if (tid == 0) p.err[blockIdx.x] = ctl.err;
}

// Merges the partial results of the row tiles that several CTAs worked on, and gathers the error
// bits. An item is 128 channels of one query of such a tile: one warp, four channels per lane, so
// that one sequence's 64 queries over all CTAs and many short tiles alike spread over the device,
// and eight parts' loads are in flight at once. (A block per query took three times as long.)
constexpr int kMergeThreads = 256;

__device__ __forceinline__ size_t part_slot(int first, int i, int N, int c) {
    return static_cast<size_t>(i ? (first + i) * 2 : first * 2 + 1) * N + c;
}

template <int D, int N>
__global__ void __launch_bounds__(kMergeThreads)
paged_merge_kernel(const __grid_constant__ PagedAttnParams p, int ctas, uint32_t* eword) {
    constexpr int CH = D / 128, PL = 5;  // chunks of a query; parts per lane (at most 160)
    __shared__ int starts[160], d_s[160][5], n_starts;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    // the tiles to merge, by the CTA that starts each
    if (warp == 0) {
        int n = 0;
        uint32_t err = 0;
        for (int c0 = 0; c0 < ctas; c0 += 32) {
            const int c = c0 + lane;
            const int np = c < ctas ? p.desc[c * 8] : 0;
            if (c < ctas) err |= p.err[c];
            const unsigned m = __ballot_sync(~0u, np > 0);
            if (np > 0) starts[n + __popc(m & ((1u << lane) - 1))] = c;
            n += __popc(m);
        }
        err = __reduce_or_sync(~0u, err);
        if (lane == 0) {
            n_starts = n;
            if (blockIdx.x == 0) *eword = err;
        }
    } else if (tid - 32 < ctas) {
        for (int c = tid - 32; c < ctas; c += kMergeThreads - 32)
            for (int i = 0; i < 5; ++i) d_s[c][i] = p.desc[c * 8 + i];
    }
    __syncthreads();
    constexpr int WB = kMergeThreads / 32;
    for (int x = blockIdx.x * WB + warp; x < n_starts * N * CH; x += gridDim.x * WB) {
        const int first = starts[x / (N * CH)], rest = x % (N * CH), c = rest / CH, ch = (rest % CH) * 128 + lane * 4;
        const int* d = d_s[first];
        const int np = d[0], t = c / p.g.hb, hh = c - t * p.g.hb;
        if (t >= d[2] || hh >= d[4]) continue;
        const int h = d[3] + hh, tok = d[1] + t;
        float w[PL], l[PL], M = -INFINITY;
#pragma unroll
        for (int k = 0; k < PL; ++k) {
            const int i = lane + 32 * k;
            float2 ml = make_float2(-INFINITY, 0.f);
            if (i < np) ml = *reinterpret_cast<const float2*>(p.part_ml + part_slot(first, i, N, c) * 2);
            w[k] = ml.x;
            l[k] = ml.y;
            M = fmaxf(M, ml.x);
        }
        const float snk = p.sink ? p.sink[h] * kLog2e : -INFINITY;
        float4 v[8];                     // (the first parts' loads do not wait for the factors)
        const float* po = p.part_o + ch;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < np) v[i] = *reinterpret_cast<const float4*>(po + part_slot(first, i, N, c) * D);
#pragma unroll
        for (int s = 16; s; s >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, s));
        const float top = fmaxf(M, snk);
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < PL; ++k) {
            w[k] = w[k] == -INFINITY ? 0.f : exp2f(w[k] - top);
            sum += w[k] * l[k];
        }
#pragma unroll
        for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(~0u, sum, s);
        const float den = sum + (snk == -INFINITY ? 0.f : exp2f(snk - top));
        if (ch == 0 && p.lse)
            p.lse[static_cast<size_t>(tok) * p.g.H + h] = M == -INFINITY ? own_sink(p, h) : top * kLn2 + logf(den);
        const float f = M == -INFINITY ? 0.f : 1.f / den;            // (-inf: no part had a row of the query's)
        float o[4] = {0.f, 0.f, 0.f, 0.f};
        for (int i0 = 0; i0 < np; i0 += 8) {
            float wk = w[0];
#pragma unroll
            for (int k = 1; k < PL; ++k)
                if (i0 >= 32 * k) wk = w[k];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float e = __shfl_sync(~0u, wk, (i0 + i) & 31);
                if (i0 + i < np && e != 0.f) {       // (a part that saw nothing may hold anything)
                    o[0] = fmaf(e, v[i].x, o[0]); o[1] = fmaf(e, v[i].y, o[1]);
                    o[2] = fmaf(e, v[i].z, o[2]); o[3] = fmaf(e, v[i].w, o[3]);
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i0 + 8 + i < np) v[i] = *reinterpret_cast<const float4*>(po + part_slot(first, i0 + 8 + i, N, c) * D);
        }
        const int r0 = D - 2 * p.or_pairs;
#pragma unroll 1
        for (int i = 0; i < 4; i += 2) {
            float e = (i ? o[2] : o[0]) * f, b = (i ? o[3] : o[1]) * f;
            if (p.orp && ch + i >= r0) {
                const float2 cs = out_rope_cs(p, tok, (ch + i - r0) >> 1);
                const float e0 = e;
                e = e0 * cs.x + b * cs.y;
                b = -e0 * cs.y + b * cs.x;
            }
            *reinterpret_cast<uint32_t*>(p.out + (static_cast<size_t>(tok) * p.g.H + h) * D + ch + i) = pack2(e, b);
        }
    }
}

// Query columns per row tile: 64 for single tokens and small groups; else as many as the
// accumulators and two K/V tiles leave room for.
int tile_queries(const dsv4_paged_attn_args& a) {
    const long long rows = static_cast<long long>(a.max_q) * (a.heads / a.kv_heads);
    return a.dim == 512 || rows <= 64 ? 64 : 128;
}

int attn_ctas() {
    const int n = sm_count();
    return n > 0 && n <= 160 ? n : 160;
}

template <int D, int N>
int run(const dsv4_paged_attn_args& a, uint8_t* ws, uint32_t* eword, cudaStream_t st) {
    using C = PCfg<D, N>;
    PagedAttnParams p{};
    p.g = paged_geom(a.block_table, a.cu_q, a.kv_len, a.batch, a.total_q, a.max_pages, a.page_size, a.num_pages, a.heads,
                     a.kv_heads, a.window);
    paged_tile(p.g, N);
    CUtensorMap qmap, kmap, vmap;
    if (!paged_query_map(&qmap, a.q, D, a.heads, a.total_q, a.q_stride, p.g.hb, p.g.tpt) ||
        !paged_pool_map(&kmap, a.k_pages, D, a.kv_heads, a.page_size, a.num_pages, p.g.br))
        return DSV4_ERR_LAUNCH;
    if (!a.v_pages) vmap = kmap;
    else if (!paged_pool_map(&vmap, a.v_pages, D, a.kv_heads, a.page_size, a.num_pages, p.g.br)) return DSV4_ERR_LAUNCH;
    auto kern = paged_attn_kernel<D, N>;
    if (once_per_device(reinterpret_cast<const void*>(kern), kAttrLaunch, [kern] {
            return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        }) != cudaSuccess)
        return DSV4_ERR_LAUNCH;
    const int ctas = attn_ctas();
    const size_t ml = align_up(static_cast<size_t>(ctas) * 2 * N * 2 * 4, 256);
    const size_t po = static_cast<size_t>(ctas) * 2 * N * D * 4;
    p.part_ml = reinterpret_cast<float*>(ws);
    p.part_o = reinterpret_cast<float*>(ws + ml);
    p.desc = reinterpret_cast<int*>(ws + ml + po);
    p.err = reinterpret_cast<uint32_t*>(p.desc + ctas * 8);
    p.sink = a.sink;
    p.out = static_cast<__nv_bfloat16*>(a.out);
    p.lse = a.lse;
    p.scale2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
    p.orp = a.out_rope_pos;
    p.or_pairs = a.out_rope_pos ? a.out_rope_dim / 2 : 0;
    for (int j = 0; j < p.or_pairs; ++j) p.or_freq[j] = std::pow(a.out_rope_theta, -2.0 * j / a.out_rope_dim);
    p.shared = a.v_pages == nullptr;
    p.min_units = 2;
    const WaitCtl wc = wait_ctl(DSV4_WAIT_FAULT_PAGED_ATTN);
    p.fault = wc.fault;
    p.wait_ns = wc.wait_ns;
    count_launch();
    if (launch_k(kern, dim3(ctas), dim3(kThreads), C::SMEM, st, true, qmap, kmap, vmap, p) != cudaSuccess) return DSV4_ERR_LAUNCH;
    count_launch();
    if (launch_k(paged_merge_kernel<D, N>, dim3(ctas * 4), dim3(kMergeThreads), 0, st, true, p, ctas, eword) !=
        cudaSuccess)
        return DSV4_ERR_LAUNCH;
    return DSV4_OK;
}

}  // namespace

PagedGeom paged_geom(const int32_t* table, const int32_t* cu_q, const int32_t* kv_len, int batch, int total_q, int max_pages,
                     int page_size, int num_pages, int heads, int kv_heads, int window) {
    PagedGeom g{};
    g.table = table;
    g.cu_q = cu_q;
    g.kv_len = kv_len;
    g.batch = batch;
    g.total_q = total_q;
    g.max_pages = max_pages;
    g.page_size = page_size;
    g.num_pages = num_pages;
    g.H = heads;
    g.KV = kv_heads;
    g.G = heads / kv_heads;
    g.window = static_cast<long long>(max_pages) * page_size <= window ? 0 : window;   // (no effect: none)
    g.br = paged_box_rows(page_size);
    while ((1 << g.br_log2) < g.br) ++g.br_log2;
    return g;
}

bool paged_query_map(CUtensorMap* map, const void* q, int D, int heads, int total_q, long long stride, int hb, int tpt) {
    const uint64_t dims[3] = {static_cast<uint64_t>(D), static_cast<uint64_t>(heads), static_cast<uint64_t>(total_q)};
    const uint64_t strides[2] = {static_cast<uint64_t>(D) * 2, static_cast<uint64_t>(stride) * 2};
    const uint32_t box[3] = {64, static_cast<uint32_t>(hb), static_cast<uint32_t>(tpt)};
    return encode_nd_bf16(map, q, 3, dims, strides, box);
}

bool paged_pool_map(CUtensorMap* map, const void* pages, int D, int kv_heads, int page_size, int num_pages, int br) {
    const uint64_t row = static_cast<uint64_t>(D) * 2;
    const uint64_t dims[4] = {static_cast<uint64_t>(D), static_cast<uint64_t>(kv_heads), static_cast<uint64_t>(page_size),
                              static_cast<uint64_t>(num_pages)};
    const uint64_t strides[3] = {row, row * kv_heads, row * kv_heads * page_size};
    const uint32_t box[4] = {64, 1, static_cast<uint32_t>(br), 1};
    return encode_nd_bf16(map, pages, 4, dims, strides, box);
}

size_t paged_attn_ws_bytes(const dsv4_paged_attn_args& a) {
    const size_t ctas = attn_ctas(), n = ctas * 2 * tile_queries(a);
    return align_up(n * 2 * 4, 256) + n * a.dim * 4 + ctas * 9 * 4;
}

int launch_paged_attn(const dsv4_paged_attn_args& a, uint8_t* ws, uint32_t* eword, cudaStream_t st) {
    if (a.batch == 0 || a.total_q == 0) return cudaMemsetAsync(eword, 0, 4, st) == cudaSuccess ? DSV4_OK : DSV4_ERR_LAUNCH;
    const int n = tile_queries(a);
    if (a.dim == 512) return run<512, 64>(a, ws, eword, st);
    if (a.dim == 256) return n == 64 ? run<256, 64>(a, ws, eword, st) : run<256, 128>(a, ws, eword, st);
    return n == 64 ? run<128, 64>(a, ws, eword, st) : run<128, 128>(a, ws, eword, st);
}

}  // namespace dsv4
