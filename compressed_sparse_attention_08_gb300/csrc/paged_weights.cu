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
// each read once; otherwise the rows of an item stay and the queries of every token that sees
// them stream. An item is a tile of 128 cache rows, or, where whole tiles would leave CTAs waiting
// for others, a share of the tokens that see it; those partial sums lie in the workspace and the
// second kernel adds them in order. Roles as in paged_attn.cu.
#include <cmath>

#include "internal.h"
#include "paged.cuh"

namespace dsv4 {
namespace {

constexpr int kThreads = 640, kLoadWarps = 3, kGroups = 4;
constexpr int kSoftWarps = 16, kSoftThreads = 512, kSoftBar = 1;
constexpr int kN = 128;                  // query columns
constexpr int kPT = 128;                 // cache rows per tile
constexpr int kSB = 4;                   // accumulators (TMEM)
constexpr int kMaxSplit = 64, kMaxShares = 8;    // shares per tile, and per CTA in all
constexpr float kLog2e = 1.4426950408889634f;

struct PagedWeightsParams {
    PagedGeom g;
    const float* lse;
    const float* acc_in;                 // or null
    float* acc;
    float* part;                         // [kMaxShares * grid, 128]
    int* head;                           // [0] tiles, [1] split, then per tile (sequence, first row)
    uint32_t* err;
    int acc_rows, keep_q;                // keep_q: the queries stay in shared memory
    float scale2;
    unsigned long long wait_ns;
};

template <int D_>
struct WCfg {
    static constexpr int D = D_, NB = D / 64;
    static constexpr int BOX = kPT * 128;                    // 128 rows (or queries) x 64 channels
    static constexpr int RES = NB * BOX;                     // the operand that stays
    static constexpr int RS = D == 512 ? 5 : 8;              // ring boxes
    // The tensor core's running fp32 sum is cut, not rounded, at every step, which pulls scores
    // towards 0: by 1.1e-6 on average at scores of 3 with 512 channels in one sum (measured), which
    // the weights show in full. Two sums of 256 channels, added in fp32, leave half of it.
    static constexpr int SUMS = D == 512 ? 2 : 1;
    static constexpr int SB = kSB / SUMS;                    // score buffers
    static constexpr int OFF_R = RES, OFF_S = RES + RS * BOX;
    static constexpr int OFF_PF = OFF_S + 2 * kN * 8 + kGroups * kPT * 4;   // tiles before each sequence
    static constexpr int SMALL = OFF_PF - OFF_S + kPagedMaxBatch * 4;
    static constexpr int SMEM = OFF_S + SMALL + 1024;
    static_assert(SMEM <= 232448, "shared memory");
};

__device__ __forceinline__ void soft_sync() { named_bar_sync(kSoftBar, kSoftThreads); }

// An item: a tile of cache rows of one sequence and a share of the token tiles that see it.
struct WItem {
    PagedSeq q;
    int s, row0, tt0, tt1;               // token tiles [tt0, tt1)
    int tile, part;
};

// Rows of a sequence that are accumulated: its length, at most acc_rows.
__device__ __forceinline__ int weight_rows(const PagedWeightsParams& p, const PagedSeq& q) { return min(q.L, p.acc_rows); }

struct WSched { int tiles, split; };

// Tiles before each sequence, and the split. Whole block.
__device__ void weight_schedule(const PagedWeightsParams& p, int* pref, WSched* out, uint32_t* err) {
    const PagedGeom& g = p.g;
    const int tid = threadIdx.x, lane = tid & 31;
    bool bad = false;
    for (int s = tid; s < g.batch; s += kThreads) {
        const PagedSeq q = paged_seq(g, s, bad);
        bad |= q.L > p.acc_rows;
        pref[s] = (weight_rows(p, q) + kPT - 1) / kPT;
    }
    if (bad) atomicOr(err, DSV4_EWORD_BAD_INDEX);
    __syncthreads();
    if (tid < 32) {
        int carry = 0;                   // (batch * rows / 128 fits: the host checks it)
        for (int s0 = 0; s0 < g.batch; s0 += 32) {
            const int s = s0 + lane;
            int v = s < g.batch ? pref[s] : 0;
#pragma unroll
            for (int w = 1; w < 32; w <<= 1) {
                const int o = __shfl_up_sync(~0u, v, w);
                if (lane >= w) v += o;
            }
            v += carry;
            if (s < g.batch) pref[s] = v;
            carry = __shfl_sync(~0u, v, 31);
        }
        // The split with the shortest longest CTA: rounds of items, each a share of a tile and a
        // fiftieth of one for loading its rows again. One split per lane.
        float best = 1e30f;
        int split = 1;
        for (int n = lane + 1; n <= kMaxSplit; n += 32) {
            const bool may = n == 1 || (!p.keep_q && static_cast<long long>(carry) * n <= kMaxShares * static_cast<int>(gridDim.x));
            if (!may) continue;
            const int rounds = (carry * n + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
            const float cost = n == 1 ? static_cast<float>(rounds) : rounds * (1.f / n + 0.02f);
            if (cost < best) {
                best = cost;
                split = n;
            }
        }
#pragma unroll
        for (int w = 16; w; w >>= 1) {
            const float ob = __shfl_xor_sync(~0u, best, w);
            const int os = __shfl_xor_sync(~0u, split, w);
            if (ob < best || (ob == best && os < split)) {
                best = ob;
                split = os;
            }
        }
        if (lane == 0) *out = WSched{carry, split};
    }
    __syncthreads();
}

struct WWalk {
    const PagedWeightsParams& p;
    const int* pref;
    WSched sc;
    long long i;                         // item
    int s;                               // the sequence of the item before
    __device__ WWalk(const PagedWeightsParams& par, const int* pr, const WSched& sched)
        : p(par), pref(pr), sc(sched), i(blockIdx.x), s(0) {}
    // Items go round over the CTAs, so neighbours read the same queries at about the same time.
    __device__ bool next(WItem& o) {
        if (i >= static_cast<long long>(sc.tiles) * sc.split) return false;
        const PagedGeom& g = p.g;
        o.tile = static_cast<int>(i / sc.split);
        o.part = static_cast<int>(i - static_cast<long long>(o.tile) * sc.split);
        int lo = s, hi = g.batch - 1;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (pref[mid] > o.tile) hi = mid; else lo = mid + 1;
        }
        s = lo;
        bool dummy = false;
        o.s = s;
        o.q = paged_seq(g, s, dummy);
        o.row0 = (o.tile - (s ? pref[s - 1] : 0)) * kPT;
        // tokens t with hi(t) > row0 and lo(t) < row0 + 128
        const long long base = static_cast<long long>(o.q.L) - o.q.n;
        long long a = o.row0 - base, b = o.q.n;
        if (a < 0) a = 0;
        if (g.window > 0) {
            const long long e = o.row0 + kPT - 1 + g.window - base;
            if (e < b) b = e;
        }
        int t0 = static_cast<int>(a / g.tpt), t1 = b > a ? static_cast<int>((b + g.tpt - 1) / g.tpt) : t0;
        if (a >= b) t1 = t0;
        const int n = t1 - t0;
        o.tt0 = t0 + static_cast<int>(static_cast<long long>(n) * o.part / sc.split);
        o.tt1 = t0 + static_cast<int>(static_cast<long long>(n) * (o.part + 1) / sc.split);
        i += gridDim.x;
        return true;
    }
    // the rows that some token of the item sees
    __device__ void bounds(const WItem& o, PagedSeg& sg) const {
        const int ta = o.tt0 * p.g.tpt, tb = min(o.tt1 * p.g.tpt, o.q.n) - 1;
        sg.s = o.s;
        sg.lo_u = paged_lo(p.g, o.q, ta);
        sg.hi_u = min(paged_hi(o.q, tb), weight_rows(p, o.q));
    }
};

// What the resident operand holds: the queries of one row tile, or the rows of an item's KV head.
struct WStay {
    int a = -1, h = -1, b = -1;
    __device__ bool moved(bool keep_q, const WItem& it, int kvh, int x) {
        const int na = keep_q ? it.s : it.tile, nb = keep_q ? x : it.part;
        if (a == na && h == kvh && b == nb) return false;
        a = na;
        h = kvh;
        b = nb;
        return true;
    }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
paged_weights_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ PagedWeightsParams p) {
    using C = WCfg<D>;
    constexpr int NB = C::NB, RS = C::RS, SB = C::SB, SUMS = C::SUMS;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t tmem_slot, s_err;
    __shared__ volatile int abort_flag;
    __shared__ WSched sched;
    __shared__ uint64_t res_full, res_empty, full[RS], empty[RS], s_full[SB], s_empty[SB];
    __shared__ unsigned s_bad[16];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* sR = sm + C::OFF_R;
    float* s_nl = reinterpret_cast<float*>(sm + C::OFF_S);           // [2][N] lse in base-2 units, negated
    int* s_tok = reinterpret_cast<int*>(s_nl + 2 * kN);              // [2][N] the column's token in the tile, -1: no query
    float* red = reinterpret_cast<float*>(s_tok + 2 * kN);           // [4][128]
    int* pref = reinterpret_cast<int*>(sm + C::OFF_PF);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        tma_prefetch_desc(&qmap);
        tma_prefetch_desc(&kmap);
        mbar_init(&res_full, kLoadWarps);
        mbar_init(&res_empty, 1);
        for (int i = 0; i < RS; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
        for (int i = 0; i < SB; ++i) { mbar_init(&s_full[i], 1); mbar_init(&s_empty[i], kSoftWarps); }
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
    weight_schedule(p, pref, &sched, &s_err);

    const PagedGeom& g = p.g;
    const bool keep_q = p.keep_q != 0;
    if (warp == 0 || warp == 2 || warp == 3) {
        // ---------------------------------------------------------------- copies
        // Three warps walk the same boxes and take them in turn.
        const int mine = warp == 0 ? 0 : warp - 1;
        WWalk w(p, pref, sched);
        WItem it;
        PagedSeg sg{};
        WStay stays;
        const int piece = lane >> 1;
        const uint32_t qbox = static_cast<uint32_t>(g.hb) * g.tpt * 128;
        uint32_t ring = 0, res = 0, unit = 0;
        bool dead = false;
        while (!dead && w.next(it)) {
            if (it.tt1 <= it.tt0) continue;
            w.bounds(it, sg);
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
            for (int kvh = 0; kvh < g.KV && !dead; ++kvh) {
                for (int x = it.tt0 * g.nhb; x < it.tt1 * g.nhb && !dead; ++x, ++unit) {
                    const int tt = x / g.nhb, blk = x - tt * g.nhb;
                    if (stays.moved(keep_q, it, kvh, x)) {
                        if (res > 0) dead = __any_sync(~0u, !mbar_wait(&res_empty, (res - 1) & 1, &abort_flag, p.wait_ns));
                        if (dead) break;
                        if (lane == 0) {
                            const uint32_t bytes = NB * (keep_q ? qbox : kbox);
                            if (mine == 0 && bytes) mbar_arrive_expect_tx(&res_full, bytes);
                            else mbar_arrive(&res_full);
                        }
                        __syncwarp();
#pragma unroll 1
                        for (int b = mine; b < NB; b += kLoadWarps) {
                            if (keep_q) load_q(sm + b * C::BOX, &res_full, kvh, b, tt, blk);
                            else load_k(sm + b * C::BOX, &res_full, kvh, b);
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
        }
        if (dead && lane == 0) {                     // a wait ran out: let the copies in flight land
            atomicOr(&s_err, DSV4_EWORD_TIMEOUT);
            abort_flag = 1;
            if (res) mbar_wait(&res_full, (res - 1) & 1, nullptr, 100000000ull);
            for (uint32_t r = ring > RS ? ring - RS : 0; r < ring; ++r)
                if (r % kLoadWarps == static_cast<uint32_t>(mine)) mbar_wait(&full[r % RS], (r / RS) & 1, nullptr, 100000000ull);
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- tensor core
        WWalk w(p, pref, sched);
        WItem it;
        WStay stays;
        uint32_t ring = 0, res = 0, u = 0;
        bool dead = false;
        const bool one = elect_one();
        auto wait = [&](uint64_t* bar, uint32_t parity) { return !__any_sync(~0u, !mbar_wait(bar, parity & 1, &abort_flag, p.wait_ns)); };
        const uint32_t r0 = smem_u32(sm), g0 = smem_u32(sR);
        const uint32_t id = idesc_bf16_f32(kPT, kN);
        while (!dead && w.next(it)) {
            if (it.tt1 <= it.tt0) continue;
            for (int kvh = 0; kvh < g.KV && !dead; ++kvh) {
                for (int x = it.tt0 * g.nhb; x < it.tt1 * g.nhb && !dead; ++x, ++u) {
                    if (stays.moved(keep_q, it, kvh, x)) {
                        if (res > 0 && one) umma_commit(&res_empty);
                        __syncwarp();
                        dead = !wait(&res_full, res);
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
                        const uint64_t stay = sdesc_kmajor_sw128(r0 + b * C::BOX), strm = sdesc_kmajor_sw128(g0 + slot * C::BOX);
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
        }
        if (dead && lane == 0) {
            atomicOr(&s_err, DSV4_EWORD_TIMEOUT);
            abort_flag = 1;
        }
    } else {
        // ---------------------------------------------------------------- weights
        WWalk w(p, pref, sched);
        WItem it;
        const int st = tid - 128, q4 = warp & 3, grp = (warp - 4) >> 2;
        const int row = q4 * 32 + lane, c0 = grp * (kN / kGroups);
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(q4 * 32) << 16);
        const uint64_t scale22 = pack_f32x2(p.scale2, p.scale2);
        const int ct = st / g.hb, ch = st - ct * g.hb;               // column st: token and head in the tile
        uint32_t u = 0;
        bool dead = false;
        while (w.next(it)) {
            uint64_t sums[4] = {0ull, 0ull, 0ull, 0ull};
            const int n = (it.tt1 - it.tt0) * g.nhb, rows = weight_rows(p, it.q), j = it.row0 + row;
            if (n > 0) {
                for (int kvh = 0; kvh < g.KV; ++kvh) {
                    // column st of unit x (its lse is read a unit ahead)
                    float nl = 0.f;
                    int tok = -1;
                    auto fetch = [&](int x) {
                        tok = -1;
                        if (st >= kN || x >= n) return;
                        const int tt = it.tt0 + x / g.nhb, blk = x - x / g.nhb * g.nhb;
                        const int t = tt * g.tpt + ct, h = blk * g.hb + ch;
                        if (ct < g.tpt && t < it.q.n && h < g.G) {
                            nl = p.lse[static_cast<size_t>(it.q.q0 + t) * g.H + kvh * g.G + h];
                            tok = ct;
                        }
                    };
                    fetch(0);
                    for (int x = 0; x < n; ++x, ++u) {
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
                        fetch(x + 1);
                        const int tt = it.tt0 + x / g.nhb, blk = x - x / g.nhb * g.nhb;
                        const int t0 = tt * g.tpt, tn = min(g.tpt, it.q.n - t0), hv = min(g.hb, g.G - blk * g.hb);
                        const int cols = (tn - 1) * g.hb + hv;       // (no query behind them)
                        // every token of the tile sees every row of the unit, and every column has a query
                        const bool open = it.row0 + kPT <= paged_hi(it.q, t0) && it.row0 >= paged_lo(g, it.q, t0 + tn - 1) &&
                                          (hv == g.hb || tn == 1) && c0 + 32 <= cols;
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
                            for (int i = 0; i < 16; i += 2) {
                                const ulonglong2 m = *reinterpret_cast<const ulonglong2*>(unl + c0 + 2 * i);
                                uint64_t a = m.x, b = m.y;
                                fma_f32x2(a, x2[i], scale22);
                                fma_f32x2(b, x2[i + 1], scale22);
                                float e[4];
                                unpack_f32x2(a, e[0], e[1]);
                                unpack_f32x2(b, e[2], e[3]);
                                if (!open) {
                                    const unsigned bad = *reinterpret_cast<volatile unsigned*>(&s_bad[u & 15]);
                                    const bool live = j < rows && !paged_bad_row(g, bad, row);
#pragma unroll
                                    for (int k = 0; k < 4; ++k) {
                                        const int t = utok[c0 + 2 * i + k];
                                        if (!live || t < 0 || j >= paged_hi(it.q, t0 + t) || j < paged_lo(g, it.q, t0 + t)) e[k] = -INFINITY;
                                    }
                                }
                                add_f32x2(sums[i & 3], pack_f32x2(ex2(e[0]), ex2(e[1])));
                                add_f32x2(sums[(i & 3) + 1], pack_f32x2(ex2(e[2]), ex2(e[3])));
                            }
                        }
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&s_empty[sb]);
                    }
                }
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
                // (a row on a page outside the pool: hidden; the units that all tokens see do not ask)
                if (n > 0 && paged_bad_row(g, *reinterpret_cast<volatile unsigned*>(&s_bad[(u - 1) & 15]), st)) v = 0.f;
                if (sched.split > 1) {
                    p.part[(static_cast<size_t>(it.tile) * sched.split + it.part) * kPT + st] = v;
                } else if (jj < rows) {
                    const size_t o = static_cast<size_t>(it.s) * p.acc_rows + jj;
                    p.acc[o] = (p.acc_in ? p.acc_in[o] : 0.f) + v;
                }
            }
            if (st == 0 && sched.split > 1 && it.part == 0) {
                p.head[2 + it.tile * 2] = it.s;
                p.head[3 + it.tile * 2] = it.row0;
            }
            soft_sync();
        }
        if (dead && lane == 0) {
            atomicOr(&s_err, DSV4_EWORD_TIMEOUT);
            abort_flag = 1;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 2) tmem_dealloc(tmem, kSB * kN);
    if (tid == 0) {
        p.err[blockIdx.x] = s_err;
        if (blockIdx.x == 0) {
            p.head[0] = sched.split > 1 ? sched.tiles : 0;
            p.head[1] = sched.split;
        }
    }
}

// Adds the partial sums of split items in order, and gathers the error bits.
__global__ void __launch_bounds__(kPT)
paged_weights_sum_kernel(const __grid_constant__ PagedWeightsParams p, int ctas, uint32_t* eword) {
    pdl_wait();
    const int tid = threadIdx.x;
    if (blockIdx.x == 0 && tid < 32) {
        uint32_t e = 0;
        for (int c = tid; c < ctas; c += 32) e |= p.err[c];
        e = __reduce_or_sync(~0u, e);
        if (tid == 0) *eword = e;
    }
    if (static_cast<int>(blockIdx.x) >= p.head[0]) return;
    const int split = p.head[1], s = p.head[2 + blockIdx.x * 2], j = p.head[3 + blockIdx.x * 2] + tid;
    bool dummy = false;
    if (j >= weight_rows(p, paged_seq(p.g, s, dummy))) return;
    const float* src = p.part + static_cast<size_t>(blockIdx.x) * split * kPT + tid;
    float v = 0.f;
#pragma unroll 8
    for (int i = 0; i < split; ++i) v += src[i * kPT];
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
                     a.kv_heads, a.window, kPT);
    paged_tile(p.g, kN);
    CUtensorMap qmap, kmap;
    if (!paged_query_map(&qmap, a.q, D, a.heads, a.total_q, a.q_stride, p.g.hb, p.g.tpt) ||
        !paged_pool_map(&kmap, a.k_pages, D, a.kv_heads, a.page_size, a.num_pages, p.g.br))
        return DSV4_ERR_LAUNCH;
    const int ctas = weight_ctas();
    p.lse = a.lse;
    p.acc_in = a.acc_in;
    p.acc = a.acc;
    p.acc_rows = a.acc_rows;
    p.part = reinterpret_cast<float*>(ws);
    p.head = reinterpret_cast<int*>(ws + static_cast<size_t>(kMaxShares * ctas) * kPT * 4);
    p.err = reinterpret_cast<uint32_t*>(p.head + 2 + kMaxShares * ctas);
    // one row tile per sequence: the queries stay
    p.keep_q = p.g.nhb == 1 && a.max_q <= p.g.tpt;
    p.scale2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
    p.wait_ns = kDefaultWaitNs;
    auto kern = paged_weights_kernel<D>;
    if (once_per_device(reinterpret_cast<const void*>(kern), kAttrLaunch, [kern] {
            return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        }) != cudaSuccess)
        return DSV4_ERR_LAUNCH;
    count_launch();
    if (launch_k(kern, dim3(ctas), dim3(kThreads), C::SMEM, st, true, qmap, kmap, p) != cudaSuccess) return DSV4_ERR_LAUNCH;
    count_launch();
    return launch_k(paged_weights_sum_kernel, dim3(kMaxShares / 2 * ctas), dim3(kPT), 0, st, true, p, ctas, eword) == cudaSuccess
               ? DSV4_OK : DSV4_ERR_LAUNCH;
}

}  // namespace

size_t paged_weights_ws_bytes(const dsv4_paged_weights_args& a) {
    (void)a;
    const size_t n = static_cast<size_t>(weight_ctas());
    return kMaxShares * n * kPT * 4 + (2 + (kMaxShares + 1) * n) * 4;
}

int launch_paged_weights(const dsv4_paged_weights_args& a, uint8_t* ws, uint32_t* eword, cudaStream_t st) {
    if (a.batch == 0) return cudaMemsetAsync(eword, 0, 4, st) == cudaSuccess ? DSV4_OK : DSV4_ERR_LAUNCH;
    if (a.dim == 512) return run<512>(a, ws, eword, st);
    if (a.dim == 256) return run<256>(a, ws, eword, st);
    return run<128>(a, ws, eword, st);
}

}  // namespace dsv4
