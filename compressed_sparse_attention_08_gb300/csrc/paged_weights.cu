// The attention weight every cached row received from a call's tokens:
//   acc[s, j] += sum over tokens t that see j, and heads h, of exp(scale q[t, h] . k_j - lse[t, h])
// with the log-sum-exp that the attention before wrote (the pages have no counterpart: it is
// what an eviction by accumulated weight needs).
//
// The scores are formed as in paged_attn.cu: S^T = K Q^T on the tensor core, 128 cache rows on
// the lanes and up to 128 queries on the columns, so a thread of the epilogue owns one cache row
// and its sum over a quarter of the queries stays in registers: no reduction over threads but the
// last one over the four quarters, and a fixed order of addition. One of the operands stays in
// shared memory while the other streams through a ring of 16 KB boxes (64 channels of 128 rows):
// with one row tile of queries per sequence (single tokens) the queries stay and the rows stream,
// each read once; otherwise the rows of a tile stay and the queries of every token that sees them
// stream. A unit is a tile of 128 cache rows x one row tile of queries; as in the attention all
// units form one line, (sequence, rows, KV head, row tile), and each CTA takes an equal piece of
// it. A tile that crosses a border leaves partial sums in the workspace, at most two per CTA, which
// the second kernel adds in order. Roles as in paged_attn.cu.
//
// Measured (64 heads x 512): 16 single tokens over up to 8K rows 28.5 us, 3.5 TB/s, bound by HBM
// latency behind the ring and the start; 1,023 tokens behind 7K rows 445 us, 1,150 TFLOP/s,
// bound by shared memory (two operands read, one written: 3,100 of the 3,700 cycles a unit takes).
#include <cmath>

#include "internal.h"
#include "paged.cuh"

namespace dsv4 {
namespace {

constexpr int kThreads = 640, kGroups = 4;
constexpr int kSoftWarps = 16, kSoftThreads = 512, kSoftBar = 1;
constexpr int kN = 128;                  // query columns
constexpr int kPT = kUnit;               // cache rows per tile
constexpr int kSB = 4;                   // accumulators (TMEM)
constexpr float kLog2e = 1.4426950408889634f;

struct PagedWeightsParams {
    PagedGeom g;
    const float* lse;
    const float* acc_in;                 // or null
    float* acc;
    float* part;                         // [2 * grid, 128]
    int* desc;                           // [grid, 4]: of the tile that a CTA starts and others finish
    uint32_t* err;
    int acc_rows, keep_q;                // keep_q: the queries stay in shared memory
    int fault;                           // test control: a CTA's first resident operand is never copied
    float scale2;
    unsigned long long wait_ns;
};

template <int D_>
struct WCfg {
    static constexpr int D = D_, NB = D / 64;
    static constexpr int BOX = kPT * 128;                    // 128 rows (or queries) x 64 channels
    static constexpr int RES = NB * BOX;                     // the operand that stays
    // and how many: with several KV heads it changes every unit, and the next one comes while this one
    // is used (16 single tokens over 8,192 rows each, 32 heads over 8, pages of 16: D = 128 127 -> 82 us,
    // D = 256 156 -> 116; a 300-token chunk alike with one or two, 59 and 63 us). At 512 two do not fit.
    static constexpr int RB = D <= 256 ? 2 : 1;
    static constexpr int RS = D == 128 ? 8 : 5;              // ring boxes
    // The tensor core's running fp32 sum is cut, not rounded, at every step, which pulls scores
    // towards 0. At scores of about 3 a weight is then off by 1.1e-6 on average (relative) with 512
    // channels in one sum, and by 5.0e-7 with two sums of 256 that are added in fp32 (one sum of 256:
    // 5.1e-7, of 128: 2.9e-7).
    static constexpr int SUMS = D == 512 ? 2 : 1;
    static constexpr int SB = kSB / SUMS;                    // score buffers
    static constexpr int OFF_R = RB * RES, OFF_S = OFF_R + RS * BOX;
    static constexpr int SMALL = 2 * kN * 8 + kGroups * kPT * 4;
    static constexpr int SMEM = OFF_S + SMALL + 1024;
    static_assert(SMEM <= 232448, "shared memory");
};

__device__ __forceinline__ void soft_sync() { named_bar_sync(kSoftBar, kSoftThreads); }

// Rows of a sequence that are accumulated: its length, at most acc_rows.
__device__ __forceinline__ int weight_rows(const PagedWeightsParams& p, const PagedSeq& q) { return min(q.L, p.acc_rows); }
__device__ __forceinline__ int weight_tiles(const PagedWeightsParams& p, const PagedSeq& q) {
    return (weight_rows(p, q) + kPT - 1) / kPT;
}

// Token tiles [tt0, tt1) with a token that sees a row of the tile from row0: hi(t) > row0 and
// lo(t) < row0 + 128.
struct WSpan { int tt0, tt1; };
__device__ __forceinline__ WSpan weight_span(const PagedGeom& g, const PagedSeq& q, int row0) {
    const int base = q.L - q.n, a = max(row0 - base, 0);
    int b = q.n;
    if (g.window > 0) b = static_cast<int>(min(static_cast<long long>(b), static_cast<long long>(row0) + kPT - 1 + g.window - base));
    if (a >= b) return WSpan{0, 0};
    return WSpan{a / g.tpt, (b + g.tpt - 1) / g.tpt};
}
// Units of a tile (at least one, so that its rows are written).
__device__ __forceinline__ int weight_units(const PagedGeom& g, const PagedSeq& q, int tile) {
    const WSpan w = weight_span(g, q, tile * kPT);
    return max((w.tt1 - w.tt0) * g.nhb * g.KV, 1);
}

struct WSched {
    long long total, u0, u1;             // all units, this CTA's [u0, u1)
    int s, tile, k;                      // where u0 lies
    PagedSeq q;                          // sequence s
};

// Whole block; `pref` is scratch for `batch` counts.
__device__ void weight_schedule(const PagedWeightsParams& p, long long* pref, WSched* out, uint32_t* err) {
    const PagedGeom& g = p.g;
    constexpr int NW = kThreads / 32;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int mult = g.nhb * g.KV;
    bool bad = false;
    const int step = min((g.batch + NW - 1) / NW, 32);
    for (int s0 = warp * step; s0 < g.batch; s0 += NW * step) {
        const int s = s0 + lane;
        const bool here = lane < step && s < g.batch;
        PagedSeq q{0, 0, 0};
        if (here) {
            q = paged_seq(g, s, bad);
            bad |= q.L > p.acc_rows;
        }
        const int nt = weight_tiles(p, q);
        long long units = 0;
        const bool one = q.n > 0 && q.n <= g.tpt;    // one row tile: every tile from the first seen one
        if (one) {
            const int f = min(paged_lo(g, q, 0) / kPT, nt);
            units = static_cast<long long>(nt - f) * mult + f;
        } else if (nt <= 4) {
            for (int t = 0; t < nt; ++t) units += weight_units(g, q, t);
        }
        for (unsigned big = __ballot_sync(~0u, !one && nt > 4); big; big &= big - 1) {
            const int src = __ffs(big) - 1;
            const PagedSeq b{0, __shfl_sync(~0u, q.n, src), __shfl_sync(~0u, q.L, src)};
            const int bnt = weight_tiles(p, b);
            long long u = 0;
            for (int t = lane; t < bnt; t += 32) u += weight_units(g, b, t);
#pragma unroll
            for (int w = 16; w; w >>= 1) u += __shfl_xor_sync(~0u, u, w);
            if (lane == src) units = u;
        }
        if (here) pref[s] = units;
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
        __syncwarp();
        const long long T = carry, c = blockIdx.x, ge = min(T, static_cast<long long>(gridDim.x));
        const long long u0 = c < ge ? T * c / ge : T, u1 = c < ge ? T * (c + 1) / ge : T;
        int s = 0, tile = 0, k = 0;
        PagedSeq q{0, 0, 0};
        if (u1 > u0) {
            int hi = g.batch - 1;                    // the first sequence whose units end past u0
            while (s < hi) {
                const int mid = (s + hi) >> 1;
                if (pref[mid] > u0) hi = mid; else s = mid + 1;
            }
            long long rem = u0 - (s ? pref[s - 1] : 0);
            bool dummy = false;
            q = paged_seq(g, s, dummy);
            const int nt = weight_tiles(p, q);
            const int f = q.n > 0 && q.n <= g.tpt ? min(paged_lo(g, q, 0) / kPT, nt) : 0;
            if (q.n > 0 && q.n <= g.tpt) {
                tile = rem < f ? static_cast<int>(rem) : f + static_cast<int>((rem - f) / mult);
                k = rem < f ? 0 : static_cast<int>((rem - f) % mult);
                rem = -1;
            }
            long long cum = 0;
            for (int t0 = 0; t0 < nt && rem >= 0; t0 += 32) {
                long long v = t0 + lane < nt ? weight_units(g, q, t0 + lane) : 0;
                const long long own = v;
#pragma unroll
                for (int w = 1; w < 32; w <<= 1) {
                    const long long o = __shfl_up_sync(~0u, v, w);
                    if (lane >= w) v += o;
                }
                const unsigned past = __ballot_sync(~0u, cum + v > rem);
                if (past) {
                    const int f = __ffs(past) - 1;
                    tile = t0 + f;
                    k = static_cast<int>(rem - cum - __shfl_sync(~0u, v - own, f));
                    break;
                }
                cum += __shfl_sync(~0u, v, 31);
            }
        }
        if (lane == 0) *out = WSched{T, u0, u1, s, tile, k, q};
    }
    __syncthreads();
}

// A CTA's part [kb, ke) of a tile's n units: KV head by KV head, token tile by token tile, head
// block by head block (nx = 0: nobody sees the rows, and the one unit has no work).
struct WItem {
    PagedSeq q;
    int s, row0, n, kb, ke, nx;
    int tt0, tt1;                        // token tiles that see the rows
    int lo_u, hi_u;                      // rows that some token of the tile sees
};

struct WWalk {
    const PagedWeightsParams& p;
    int s, tile, k;
    long long left;
    PagedSeq q;
    __device__ WWalk(const PagedWeightsParams& par, const WSched& sc)
        : p(par), s(sc.s), tile(sc.tile), k(sc.k), left(sc.u1 - sc.u0), q(sc.q) {}
    __device__ bool next(WItem& o) {
        if (left <= 0) return false;
        const PagedGeom& g = p.g;
        while (tile >= weight_tiles(p, q)) {         // the next sequence with rows
            if (++s >= g.batch) return false;
            tile = 0;
            bool dummy = false;
            q = paged_seq(g, s, dummy);
        }
        o.q = q;
        o.s = s;
        o.row0 = tile * kPT;
        const WSpan w = weight_span(g, q, o.row0);
        o.nx = (w.tt1 - w.tt0) * g.nhb;
        o.tt0 = w.tt0;
        o.tt1 = w.tt1;
        o.n = max(o.nx * g.KV, 1);
        o.lo_u = o.nx ? paged_lo(g, q, w.tt0 * g.tpt) : 0;
        o.hi_u = o.nx ? min(paged_hi(q, min(w.tt1 * g.tpt, q.n) - 1), weight_rows(p, q)) : 0;
        o.kb = k;
        const long long take = left < o.n - k ? left : o.n - k;
        o.ke = k + static_cast<int>(take);
        left -= take;
        k = 0;
        ++tile;
        return true;
    }
};

// A unit of an item, counted on without divisions.
struct WUnit {
    int kvh, tt, blk;
    __device__ WUnit(const PagedGeom& g, const WItem& it) {
        const int nx = max(it.nx, 1);
        kvh = it.kb / nx;
        const int x = it.kb - kvh * nx;
        tt = x / g.nhb;
        blk = x - tt * g.nhb;
        tt += it.tt0;
    }
    __device__ void step(const PagedGeom& g, const WItem& it) {
        if (++blk < g.nhb) return;
        blk = 0;
        if (++tt < it.tt1) return;
        tt = it.tt0;
        ++kvh;
    }
};

// What the resident operand holds: the queries of one row tile, or the rows of a tile's KV head.
struct WStay {
    int a = -1, h = -1, b = -1;
    __device__ bool moved(bool keep_q, const PagedGeom& g, const WItem& it, const WUnit& c) {
        const int nb = keep_q ? c.tt * g.nhb + c.blk : it.row0;
        if (a == it.s && h == c.kvh && b == nb) return false;
        a = it.s;
        h = c.kvh;
        b = nb;
        return true;
    }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
paged_weights_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ PagedWeightsParams p) {
    using C = WCfg<D>;
    constexpr int NB = C::NB, RS = C::RS, RB = C::RB, SB = C::SB, SUMS = C::SUMS;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t tmem_slot, s_err;
    __shared__ volatile int abort_flag;
    __shared__ WSched sched;
    __shared__ uint64_t res_full[RB], res_empty[RB], full[RS], empty[RS], s_full[SB], s_empty[SB];
    __shared__ unsigned s_bad[16];
    __shared__ uint64_t drained;                     // products in flight when a wait ran out
    __shared__ uint32_t ring_end[kLoadWarps], res_end[kLoadWarps];   // boxes and resident operands that a load warp issued
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* sR = sm + C::OFF_R;
    float* s_nl = reinterpret_cast<float*>(sm + C::OFF_S);           // [2][N] lse in base-2 units, negated
    int* s_tok = reinterpret_cast<int*>(s_nl + 2 * kN);              // [2][N] the column's token in the tile, -1: no query
    float* red = reinterpret_cast<float*>(s_tok + 2 * kN);           // [4][128]

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        tma_prefetch_desc(&qmap);
        tma_prefetch_desc(&kmap);
        for (int i = 0; i < RB; ++i) { mbar_init(&res_full[i], kLoadWarps); mbar_init(&res_empty[i], 1); }
        for (int i = 0; i < RS; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
        for (int i = 0; i < SB; ++i) { mbar_init(&s_full[i], 1); mbar_init(&s_empty[i], kSoftWarps); }
        mbar_init(&drained, 1);
        abort_flag = 0;
        s_err = 0;
        fence_barrier_init();
    }
    if (warp == 2) tmem_alloc(&tmem_slot, kSB * kN);
    pdl_trigger();
    pdl_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    weight_schedule(p, reinterpret_cast<long long*>(sm), &sched, &s_err);
    // the schedule's scratch is overwritten by TMA next
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();

    const PagedGeom& g = p.g;
    const bool keep_q = p.keep_q != 0;
    if (warp == 0 || warp == 2 || warp == 3) {
        // ---------------------------------------------------------------- copies
        // Three warps walk the same boxes and take them in turn.
        const int mine = warp == 0 ? 0 : warp - 1;
        WWalk w(p, sched);
        WItem it;
        PagedSeg sg{};
        WStay stays;
        const int piece = lane >> 1;
        const uint32_t qbox = static_cast<uint32_t>(g.hb) * g.tpt * 128;
        uint32_t ring = 0, res = 0, unit = 0;
        bool dead = false;
        while (!dead && w.next(it)) {
            if (it.nx == 0) continue;
            sg.s = it.s;
            sg.lo_u = it.lo_u;
            sg.hi_u = it.hi_u;
            const PagedLook t = paged_look(g, sg, it.row0, lane);
            const PagedBoxes bx = paged_boxes(g, t);
            const uint32_t kbox = static_cast<uint32_t>(__popc(bx.ok)) * g.br * 64;
            const bool piece_ok = (lane & 1) == 0 && ((bx.ok >> lane) & 1);
            // 64 channels of the item's rows, or of a row tile's queries
            auto load_k = [&](uint8_t* dst, uint64_t* bar, int kvh, int b) {
                if (piece_ok) tma_load_4d(dst + piece * g.br * 128, &kmap, bar, b * 64, kvh, t.slot, t.page);
            };
            auto load_q = [&](uint8_t* dst, uint64_t* bar, int kvh, int b, int tt, int blk) {
                if (lane == 0) tma_load_3d(dst, &qmap, bar, b * 64, kvh * g.G + blk * g.hb, it.q.q0 + tt * g.tpt);
            };
            WUnit c(g, it);
            for (int i = it.kb; i < it.ke && !dead; ++i, ++unit, c.step(g, it)) {
                const int kvh = c.kvh, tt = c.tt, blk = c.blk;
                if (stays.moved(keep_q, g, it, c)) {
                    const uint32_t rb = res % RB;
                    if (res >= RB) dead = __any_sync(~0u, !mbar_wait(&res_empty[rb], (res / RB - 1) & 1, &abort_flag, p.wait_ns));
                    if (dead) break;
                    const bool skip = p.fault && res == 0;
                    if (lane == 0 && !skip) {
                        const uint32_t bytes = NB * (keep_q ? qbox : kbox);
                        if (mine == 0 && bytes) mbar_arrive_expect_tx(&res_full[rb], bytes);
                        else mbar_arrive(&res_full[rb]);
                    }
                    __syncwarp();
#pragma unroll 1
                    for (int b = skip ? NB : mine; b < NB; b += kLoadWarps) {
                        if (keep_q) load_q(sm + rb * C::RES + b * C::BOX, &res_full[rb], kvh, b, tt, blk);
                        else load_k(sm + rb * C::RES + b * C::BOX, &res_full[rb], kvh, b);
                    }
                    ++res;
                }
#pragma unroll 1
                for (int b = 0; b < NB; ++b, ++ring) {
                    if (ring % kLoadWarps != static_cast<uint32_t>(mine)) continue;
                    const uint32_t slot = ring % RS;
                    if (ring >= RS)
                        dead = __any_sync(~0u, !mbar_wait(&empty[slot], (ring / RS - 1) & 1, &abort_flag, p.wait_ns));
                    if (dead) break;
                    const uint32_t bytes = keep_q ? kbox : qbox;
                    if (lane == 0) {
                        if (b < kLoadWarps) {    // (the first of the unit's boxes that this warp takes)
                            s_bad[unit & 15] = bx.bad;
                            if (bx.bad) atomicOr(&s_err, DSV4_EWORD_BAD_INDEX);
                        }
                        if (bytes) mbar_arrive_expect_tx(&full[slot], bytes);
                        else mbar_arrive(&full[slot]);
                    }
                    __syncwarp();
                    if (keep_q) load_k(sR + slot * C::BOX, &full[slot], kvh, b);
                    else load_q(sR + slot * C::BOX, &full[slot], kvh, b, tt, blk);
                }
            }
        }
        if (lane == 0) {
            ring_end[mine] = ring;
            res_end[mine] = res;
            if (dead) {
                atomicOr(&s_err, DSV4_EWORD_TIMEOUT);
                abort_flag = 1;
            }
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- tensor core
        WWalk w(p, sched);
        WItem it;
        WStay stays;
        uint32_t ring = 0, res = 0, u = 0;
        bool dead = false;
        const bool one = elect_one();
        auto wait = [&](uint64_t* bar, uint32_t parity) { return !__any_sync(~0u, !mbar_wait(bar, parity & 1, &abort_flag, p.wait_ns)); };
        const uint32_t r0 = smem_u32(sm), g0 = smem_u32(sR);
        const uint32_t id = idesc_bf16_f32(kPT, kN);
        while (!dead && w.next(it)) {
            if (it.nx == 0) continue;
            WUnit c(g, it);
            for (int i = it.kb; i < it.ke && !dead; ++i, ++u, c.step(g, it)) {
                if (stays.moved(keep_q, g, it, c)) {
                    if (res > 0 && one) umma_commit(&res_empty[(res - 1) % RB]);
                    __syncwarp();
                    dead = !wait(&res_full[res % RB], res / RB);
                    ++res;
                    if (dead) break;
                }
                const uint32_t sb = u % SB;
                if (u >= SB) dead = !wait(&s_empty[sb], u / SB - 1);
#pragma unroll
                for (int b = 0; b < NB; ++b, ++ring) {
                    const uint32_t slot = ring % RS;
                    dead = dead || !wait(&full[slot], ring / RS);
                    if (dead) break;
                    tc_fence_after();
                    const uint64_t stay = sdesc_kmajor_sw128(r0 + (res - 1) % RB * C::RES + b * C::BOX), strm = sdesc_kmajor_sw128(g0 + slot * C::BOX);
                    const uint64_t a0 = keep_q ? strm : stay, b0 = keep_q ? stay : strm;
                    const uint32_t d = tmem + (sb * SUMS + b / (NB / SUMS)) * kN;
                    if (one) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_bf16(d, a0 + kk * 2, b0 + kk * 2, id, (b % (NB / SUMS) > 0 || kk > 0) ? 1u : 0u);
                        umma_commit(&empty[slot]);
                    }
                    __syncwarp();
                }
                if (!dead && one) umma_commit(&s_full[sb]);
                __syncwarp();
            }
        }
        if (dead && lane == 0) {
            atomicOr(&s_err, DSV4_EWORD_TIMEOUT);
            abort_flag = 1;
        }
    } else {
        // ---------------------------------------------------------------- weights
        WWalk w(p, sched);
        WItem it;
        const int st = tid - 128, q4 = warp & 3, grp = (warp - 4) >> 2;
        const int row = q4 * 32 + lane, c0 = grp * (kN / kGroups);
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(q4 * 32) << 16);
        const uint64_t scale22 = pack_f32x2(p.scale2, p.scale2);
        const int ct = st / g.hb, ch = st - ct * g.hb;               // column st: token and head in the tile
        uint32_t u = 0;
        bool dead = false;
        int d_parts = 0, d_s = 0, d_row = 0;
        long long at = sched.u0;                                     // first unit of the item on the line
        while (w.next(it)) {
            uint64_t sums[4] = {0ull, 0ull, 0ull, 0ull};
            const int rows = weight_rows(p, it.q), j = it.row0 + row;
            const int ke = it.nx ? it.ke : it.kb;                    // (nobody sees the rows: no unit)
            // column st of unit i (its lse is read a unit ahead)
            float nl = 0.f;
            int tok = -1;
            auto fetch = [&](const WUnit& c, int i) {
                tok = -1;
                if (st >= kN || i >= ke) return;
                const int t = c.tt * g.tpt + ct, h = c.blk * g.hb + ch;
                if (ct < g.tpt && t < it.q.n && h < g.G) {
                    nl = p.lse[static_cast<size_t>(it.q.q0 + t) * g.H + c.kvh * g.G + h];
                    tok = ct;
                }
            };
            WUnit c(g, it);
            fetch(c, it.kb);
            for (int i = it.kb; i < ke; ++i, ++u) {
                const uint32_t sb = u % SB;
                float* unl = s_nl + (u & 1) * kN;
                int* utok = s_tok + (u & 1) * kN;
                if (st < kN) {
                    // (a query that saw nothing, lse -inf, has no weight to give)
                    if (tok >= 0 && nl == -INFINITY) tok = -1;
                    unl[st] = tok >= 0 ? -nl * kLog2e : -INFINITY;
                    utok[st] = tok;
                }
                soft_sync();
                const int t0 = c.tt * g.tpt, tn = min(g.tpt, it.q.n - t0), hv = min(g.hb, g.G - c.blk * g.hb);
                c.step(g, it);
                fetch(c, i + 1);
                const int cols = (tn - 1) * g.hb + hv;       // (no query behind them)
                // every token of the tile sees every row of the unit, and every column has a query
                const bool open = it.row0 + kPT <= paged_hi(it.q, t0) && it.row0 >= paged_lo(g, it.q, t0 + tn - 1) &&
                                  (hv == g.hb || tn == 1) && c0 + 32 <= cols;
                // else, of the tile's tokens, those that see row j
                const int from = j - (it.q.L - it.q.n) - t0, seen0 = max(from, 0);
                const int seen1 = g.window > 0 && g.window - 1 < g.tpt - from ? from + g.window - 1 : g.tpt;
                if (!dead) dead = !mbar_wait(&s_full[sb], (u / SB) & 1, &abort_flag, p.wait_ns);
                tc_fence_after();
                if (c0 < cols) {
                    uint32_t r[32];
                    const uint32_t scol = lane_base + sb * SUMS * kN + c0;
                    DSV4_TMEM_LD_32x32b_X32(scol, r);
                    uint64_t x2[16];
                    if constexpr (SUMS == 2) {
                        uint32_t r2[32];
                        DSV4_TMEM_LD_32x32b_X32(scol + kN, r2);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            x2[i] = pack_f32x2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
                            add_f32x2(x2[i], pack_f32x2(__uint_as_float(r2[2 * i]), __uint_as_float(r2[2 * i + 1])));
                        }
                    } else {
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            x2[i] = pack_f32x2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
                    }
#pragma unroll
                    for (int c = 0; c < 16; c += 2) {
                        const ulonglong2 m = *reinterpret_cast<const ulonglong2*>(unl + c0 + 2 * c);
                        uint64_t a = m.x, b = m.y;
                        fma_f32x2(a, x2[c], scale22);
                        fma_f32x2(b, x2[c + 1], scale22);
                        float e[4];
                        unpack_f32x2(a, e[0], e[1]);
                        unpack_f32x2(b, e[2], e[3]);
                        if (!open) {
                            const int4 t = *reinterpret_cast<const int4*>(utok + c0 + 2 * c);
                            if (t.x < seen0 || t.x > seen1) e[0] = -INFINITY;
                            if (t.y < seen0 || t.y > seen1) e[1] = -INFINITY;
                            if (t.z < seen0 || t.z > seen1) e[2] = -INFINITY;
                            if (t.w < seen0 || t.w > seen1) e[3] = -INFINITY;
                        }
                        add_f32x2(sums[c & 3], pack_f32x2(ex2(e[0]), ex2(e[1])));
                        add_f32x2(sums[(c & 3) + 1], pack_f32x2(ex2(e[2]), ex2(e[3])));
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_empty[sb]);
            }
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float a, b;
                unpack_f32x2(sums[i], a, b);
                sum += a + b;
            }
            red[grp * kPT + row] = sum;
            soft_sync();
            if (st < kPT) {
                float v = (red[st] + red[kPT + st]) + (red[2 * kPT + st] + red[3 * kPT + st]);
                const int jj = it.row0 + st;
                // (a row on a page outside the pool: hidden)
                if (it.nx && paged_bad_row(g, *reinterpret_cast<volatile unsigned*>(&s_bad[(u - 1) & 15]), st)) v = 0.f;
                if (it.kb > 0 || it.ke < it.n) {
                    p.part[static_cast<size_t>(blockIdx.x * 2 + (it.kb > 0 ? 0 : 1)) * kPT + st] = v;
                } else if (jj < rows) {
                    const size_t o = static_cast<size_t>(it.s) * p.acc_rows + jj;
                    p.acc[o] = (p.acc_in ? p.acc_in[o] : 0.f) + v;
                }
            }
            if (it.kb == 0 && it.ke < it.n) {        // this CTA starts the tile: its parts are added under its number
                const long long end = at + it.n, T = sched.total, n = min(T, static_cast<long long>(gridDim.x));
                int last = static_cast<int>((end * n - 1) / T);
                while (last + 1 < n && T * (last + 1) / n < end) ++last;
                while (T * last / n >= end) --last;
                d_parts = last - static_cast<int>(blockIdx.x) + 1;
                d_s = it.s;
                d_row = it.row0;
            }
            at += it.ke - it.kb;
            soft_sync();
        }
        if (st == 0) {
            int* d = p.desc + blockIdx.x * 4;
            d[0] = d_parts; d[1] = d_s; d[2] = d_row;
        }
        dead = __any_sync(~0u, dead);                                // (each lane waits for itself: any of them may run out)
        if (dead && lane == 0) {
            atomicOr(&s_err, DSV4_EWORD_TIMEOUT);
            abort_flag = 1;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (abort_flag) {
        // A wait ran out in some role, and the others may have finished before it: the copies and
        // products still in flight end (each wait bounded) before memory is given up.
        if (warp == 1) {
            if (elect_one()) umma_commit(&drained);
            __syncwarp();
            mbar_wait(&drained, 0, nullptr, kDrainNs);
        }
        if (tid == 0) {
            const uint32_t res = max(max(res_end[0], res_end[1]), res_end[2]);
            for (uint32_t r = res > RB ? res - RB : p.fault; r < res; ++r)     // (the test control's copy never comes)
                mbar_wait(&res_full[r % RB], (r / RB) & 1, nullptr, kDrainNs);
            ring_drain<RS>(full, ring_end);
        }
        __syncthreads();
    }
    if (warp == 2) tmem_dealloc(tmem, kSB * kN);
    if (tid == 0) p.err[blockIdx.x] = s_err;
}

// Adds the partial sums of the tiles that several CTAs worked on, in order, one block per CTA that
// starts one, and gathers the error bits.
__global__ void __launch_bounds__(kPT)
paged_weights_sum_kernel(const __grid_constant__ PagedWeightsParams p, uint32_t* eword) {
    pdl_wait();
    const int tid = threadIdx.x, c = blockIdx.x;
    if (c == 0 && tid < 32) {
        uint32_t e = 0;
        for (int i = tid; i < static_cast<int>(gridDim.x); i += 32) e |= p.err[i];
        e = __reduce_or_sync(~0u, e);
        if (tid == 0) *eword = e;
    }
    const int parts = p.desc[c * 4], s = p.desc[c * 4 + 1], j = p.desc[c * 4 + 2] + tid;
    if (parts == 0) return;
    bool dummy = false;
    if (j >= weight_rows(p, paged_seq(p.g, s, dummy))) return;
    float v = p.part[static_cast<size_t>(c * 2 + 1) * kPT + tid];
#pragma unroll 8
    for (int i = 1; i < parts; ++i) v += p.part[static_cast<size_t>((c + i) * 2) * kPT + tid];
    const size_t o = static_cast<size_t>(s) * p.acc_rows + j;
    p.acc[o] = (p.acc_in ? p.acc_in[o] : 0.f) + v;
}

int weight_ctas() {
    const int n = sm_count();
    return n > 0 && n <= 160 ? n : 160;
}

template <int D>
int run(const dsv4_paged_weights_args& a, uint8_t* ws, uint32_t* eword, cudaStream_t st) {
    using C = WCfg<D>;
    PagedWeightsParams p{};
    p.g = paged_geom(a.block_table, a.cu_q, a.kv_len, a.batch, a.total_q, a.max_pages, a.page_size, a.num_pages, a.heads,
                     a.kv_heads, a.window);
    paged_tile(p.g, kN);
    CUtensorMap qmap, kmap;
    if (!paged_pool_map(&kmap, a.k_pages, D, a.kv_heads, a.page_size, a.num_pages, p.g.br)) return DSV4_ERR_LAUNCH;
    qmap = kmap;                         // (no tokens: never used)
    if (a.total_q > 0 && !paged_query_map(&qmap, a.q, D, a.heads, a.total_q, a.q_stride, p.g.hb, p.g.tpt)) return DSV4_ERR_LAUNCH;
    const int ctas = weight_ctas();
    p.lse = a.lse;
    p.acc_in = a.acc_in;
    p.acc = a.acc;
    p.acc_rows = a.acc_rows;
    p.part = reinterpret_cast<float*>(ws);
    p.desc = reinterpret_cast<int*>(ws + static_cast<size_t>(2 * ctas) * kPT * 4);
    p.err = reinterpret_cast<uint32_t*>(p.desc + 4 * ctas);
    // one row tile per sequence: the queries stay
    p.keep_q = p.g.nhb == 1 && a.max_q <= p.g.tpt;
    p.scale2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
    const WaitCtl wc = wait_ctl(DSV4_WAIT_FAULT_PAGED_WEIGHTS);
    p.fault = wc.fault;
    p.wait_ns = wc.wait_ns;
    auto kern = paged_weights_kernel<D>;
    if (once_per_device(reinterpret_cast<const void*>(kern), kAttrLaunch, [kern] {
            return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        }) != cudaSuccess)
        return DSV4_ERR_LAUNCH;
    count_launch();
    if (launch_k(kern, dim3(ctas), dim3(kThreads), C::SMEM, st, true, qmap, kmap, p) != cudaSuccess) return DSV4_ERR_LAUNCH;
    count_launch();
    return launch_k(paged_weights_sum_kernel, dim3(ctas), dim3(kPT), 0, st, true, p, eword) == cudaSuccess
               ? DSV4_OK : DSV4_ERR_LAUNCH;
}

}  // namespace

size_t paged_weights_ws_bytes(const dsv4_paged_weights_args& a) {
    (void)a;
    const size_t n = static_cast<size_t>(weight_ctas());
    return 2 * n * kPT * 4 + 5 * n * 4;
}

int launch_paged_weights(const dsv4_paged_weights_args& a, uint8_t* ws, uint32_t* eword, cudaStream_t st) {
    if (a.batch == 0) return cudaMemsetAsync(eword, 0, 4, st) == cudaSuccess ? DSV4_OK : DSV4_ERR_LAUNCH;
    if (a.dim == 512) return run<512>(a, ws, eword, st);
    if (a.dim == 256) return run<256>(a, ws, eword, st);
    return run<128>(a, ws, eword, st);
}

}  // namespace dsv4
