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
// One persistent CTA per SM walks its share of the work line (paged.cuh). Both products have the
// cache rows or the channels on the tensor core's 128 lanes and the queries on its columns:
// S^T = K Q^T (128 rows x N queries, one unit) and O^T += V^T P^T (128 channels per tile x N).
// So the number of query columns N is free (64 or 128), a single token's 64 heads fill a tile,
// and one shared-memory copy of a shared KV row serves as K (K-major) and as V (MN-major).
// Roles: warp 0 moves pages by TMA into a ring of 128-row tiles, warp 1 issues tcgen05.mma,
// warps 4-11 do the softmax (a thread holds one cache row and half of the queries). The scores
// have two TMEM buffers, so S^T of unit u + 1 runs under the softmax of unit u.
#include <cmath>

#include "internal.h"
#include "paged.cuh"

namespace dsv4 {
namespace {

constexpr int kThreads = 384;
constexpr int kSoftWarps = 8, kSoftThreads = 256, kSoftBar = 1;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// A query's reference maximum moves only when a score exceeds it by more than kSpan (base-2
// units): P = 2^(s - m) then stays far inside the fp32 and bf16 range, and o does not depend on
// which m was used.
constexpr float kSpan = 24.f;

struct PagedAttnParams {
    PagedGeom g;
    const float* sink;                   // [H] or null
    __nv_bfloat16* out;                  // [total_q, H, D]
    float* lse;                          // [total_q, H] or null
    float* part_ml;                      // [2 * grid, N, 2]
    float* part_o;                       // [2 * grid, N, D]
    int* desc;                           // [grid, 8]
    uint32_t* err;                       // [grid] error bits
    float scale2;                        // scale * log2(e)
    const int64_t* orp;                  // [total_q] or null
    int or_pairs;
    int shared, min_units;
    unsigned long long wait_ns;
    double or_freq[64];                  // theta^(-2j / out_rope_dim)
};

template <int D_, int N_>
struct PCfg {
    static constexpr int D = D_, N = N_;
    static constexpr int NB = D / 64, MT = D / 128;
    static constexpr int BOX = kPT * 128;                    // 128 rows x 64 channels
    static constexpr int TILE = NB * BOX;
    static constexpr int QBOX = N * 128, QB = NB * QBOX;
    static constexpr int PB = kPT * N * 2;
    // after the tiles: reference maxima, factors, row bounds and offsets per query, partial sums
    static constexpr int SMALL = N * 4 * 5 + 4 * N * 4 + 512;
    static constexpr int ST_FIT = (232448 - 1024 - QB - PB - SMALL) / TILE;
    static constexpr int ST = ST_FIT > 6 ? 6 : ST_FIT;       // ring of K / V tiles
    static constexpr int OFF_Q = ST * TILE, OFF_P = OFF_Q + QB, OFF_S = OFF_P + PB;
    static constexpr int SMEM = OFF_S + SMALL + 1024;
    static constexpr int TCOLS = 512;
    static constexpr int OCOL = 2 * N;
    static_assert(ST >= 1 && OCOL + MT * N <= 512, "one tile, and both accumulators in TMEM");
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// 32 values per lane, reduced over the warp's lanes: lane i returns the reduction of value i.
template <bool kMax>
__device__ __forceinline__ float lanes_reduce(float (&v)[32], int lane) {
#pragma unroll
    for (int w = 16; w >= 1; w >>= 1) {
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

// (cos, sin) of the inverse rotation of pair j of token tok.
__device__ __forceinline__ float2 out_rope_cs(const PagedAttnParams& p, int tok, int j) {
    float sn, cs;
    sincosf(reduced_angle(static_cast<double>(p.orp[tok]) * p.or_freq[j]), &sn, &cs);
    return make_float2(cs, sn);
}

template <int D, int N>
__global__ void __launch_bounds__(kThreads, 1)
paged_attn_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap, const __grid_constant__ PagedAttnParams p) {
    using C = PCfg<D, N>;
    constexpr int ST = C::ST, NB = C::NB, MT = C::MT, NC = N / 64;   // NC: 32-column pieces per thread
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t tmem_slot, s_err;
    __shared__ volatile int abort_flag;
    __shared__ PagedSched sched;
    __shared__ uint64_t q_full, q_empty, full[ST], empty[ST], s_full[2], s_empty[2], p_full, pv_done;
    __shared__ unsigned s_bad[8];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* sQ = sm + C::OFF_Q;
    uint8_t* sP = sm + C::OFF_P;
    float* s_m = reinterpret_cast<float*>(sm + C::OFF_S);            // reference maxima (base-2 units)
    float* s_f = s_m + N;
    int* s_hi = reinterpret_cast<int*>(s_f + N);
    int* s_lo = s_hi + N;
    int* s_off = s_lo + N;                                           // output offsets, -1: no query
    float* red = reinterpret_cast<float*>(s_off + N);                // [4][N]

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        mbar_init(&q_full, 1);
        mbar_init(&q_empty, 1);
        for (int i = 0; i < ST; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
        for (int i = 0; i < 2; ++i) { mbar_init(&s_full[i], 1); mbar_init(&s_empty[i], kSoftWarps); }
        mbar_init(&p_full, kSoftWarps);
        mbar_init(&pv_done, 1);
        abort_flag = 0;
        s_err = 0;
        fence_barrier_init();
    }
    if (warp == 2) tmem_alloc(&tmem_slot, C::TCOLS);
    pdl_trigger();
    pdl_wait();                          // lengths, queries and rows may come from the kernel before
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    paged_schedule<kThreads>(p.g, p.min_units, reinterpret_cast<long long*>(sm), &sched, &s_err);
    // the schedule's scratch is overwritten by TMA next
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();

    const PagedGeom& g = p.g;
    const int parts = p.shared ? 1 : 2;
    if (warp == 0) {
        // ---------------------------------------------------------------- pages and queries
        PagedWalk w(g, sched);
        PagedSeg sg;
        const int pieces = kPT / g.br;
        const uint32_t qbytes = static_cast<uint32_t>(g.hb) * g.tpt * D * 2;
        uint32_t ring = 0, u = 0, seg = 0;
        bool dead = false;
        while (!dead && w.next(sg)) {
            if (seg > 0) dead = __any_sync(~0u, !mbar_wait(&q_empty, (seg - 1) & 1, &abort_flag, p.wait_ns));
            if (dead) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(&q_full, qbytes);
                for (int b = 0; b < NB; ++b)
                    tma_load_3d(sQ + b * C::QBOX, &qmap, &q_full, b * 64, sg.head0, sg.tok0);
            }
            ++seg;
            for (int k = sg.kb; k < sg.ke && !dead; ++k, ++u) {
                const PagedTile t = paged_tile_boxes(g, sg, sg.row0 + k * kPT, lane);
                for (int part = 0; part < parts; ++part, ++ring) {
                    const uint32_t slot = ring % ST;
                    if (ring >= ST) dead = !mbar_wait(&empty[slot], (ring / ST - 1) & 1, &abort_flag, p.wait_ns);
                    dead = __any_sync(~0u, dead);
                    if (dead) break;
                    if (lane == 0) {
                        if (part == 0) {
                            s_bad[u & 7] = t.bad;
                            if (t.bad) atomicOr(&s_err, DSV4_EWORD_BAD_INDEX);
                        }
                        const uint32_t bytes = static_cast<uint32_t>(__popc(t.ok)) * g.br * D * 2;
                        if (bytes) mbar_arrive_expect_tx(&full[slot], bytes);
                        else mbar_arrive(&full[slot]);
                    }
                    __syncwarp();
                    const CUtensorMap* map = part ? &vmap : &kmap;
                    uint8_t* tile = sm + slot * C::TILE;
                    for (int i0 = 0; i0 < NB * pieces; i0 += 32) {
                        const int i = i0 + lane, piece = i & (pieces - 1), box = i / pieces;
                        const int page = __shfl_sync(~0u, t.page, piece), at = __shfl_sync(~0u, t.slot, piece);
                        if (box < NB && ((t.ok >> piece) & 1))
                            tma_load_4d(tile + box * C::BOX + piece * g.br * 128, map, &full[slot], box * 64, sg.kvh, at,
                                        page);
                    }
                }
            }
        }
        if (dead && lane == 0) {                     // a wait ran out: let the copies in flight land
            atomicOr(&s_err, DSV4_EWORD_TIMEOUT);
            abort_flag = 1;
            if (seg) mbar_wait(&q_full, (seg - 1) & 1, nullptr, 100000000ull);
            for (uint32_t r = ring > ST ? ring - ST : 0; r < ring; ++r)
                mbar_wait(&full[r % ST], (r / ST) & 1, nullptr, 100000000ull);
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- tensor core
        if (lane == 0) {
            PagedWalk w(g, sched);
            PagedSeg sg;
            uint32_t u = 0, seg = 0;
            bool dead = false, pend = false, pend_first = false;
            uint32_t pend_u = 0;
            const uint32_t q0 = smem_u32(sQ), p0 = smem_u32(sP), t0 = smem_u32(sm);
            const uint32_t idS = idesc_bf16_f32(kPT, N), idO = idS | (1u << 15) | (1u << 16);
            auto pv = [&](uint32_t x, bool first) {
                const uint32_t r = p.shared ? x : 2 * x + 1, slot = r % ST;
                if (!mbar_wait(&p_full, x & 1, &abort_flag, p.wait_ns)) return false;
                if (!p.shared && !mbar_wait(&full[slot], (r / ST) & 1, &abort_flag, p.wait_ns)) return false;
                tc_fence_after();
                const uint32_t a0 = t0 + slot * C::TILE;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                    for (int kk = 0; kk < kPT / 16; ++kk)
                        umma_bf16(tmem + static_cast<uint32_t>(C::OCOL + mt * N),
                                  sdesc_mnmajor_sw128(a0 + 2 * mt * C::BOX + kk * 2048, C::BOX, 1024u),
                                  sdesc_mnmajor_sw128(p0 + kk * 2048, kPT * 128, 1024u), idO,
                                  (!first || kk > 0) ? 1u : 0u);
                }
                umma_commit(&empty[slot]);
                umma_commit(&pv_done);
                return true;
            };
            while (!dead && w.next(sg)) {
                dead = !mbar_wait(&q_full, seg & 1, &abort_flag, p.wait_ns);
                ++seg;
                for (int k = sg.kb; k < sg.ke && !dead; ++k, ++u) {
                    const uint32_t r = p.shared ? u : 2 * u, slot = r % ST;
                    dead = !mbar_wait(&full[slot], (r / ST) & 1, &abort_flag, p.wait_ns);
                    if (!dead && u >= 2) dead = !mbar_wait(&s_empty[u & 1], ((u >> 1) - 1) & 1, &abort_flag, p.wait_ns);
                    if (dead) break;
                    tc_fence_after();
                    const uint32_t a0 = t0 + slot * C::TILE;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        umma_bf16(tmem + (u & 1) * N, sdesc_kmajor_sw128(a0 + (kk >> 2) * C::BOX + (kk & 3) * 32),
                                  sdesc_kmajor_sw128(q0 + (kk >> 2) * C::QBOX + (kk & 3) * 32), idS, kk > 0 ? 1u : 0u);
                    umma_commit(&s_full[u & 1]);
                    if (!p.shared) umma_commit(&empty[slot]);
                    if (k + 1 == sg.ke) umma_commit(&q_empty);
                    if constexpr (ST == 1) {
                        dead = !pv(u, k == sg.kb);
                    } else {
                        if (pend) dead = !pv(pend_u, pend_first);
                        pend = true;
                        pend_u = u;
                        pend_first = k == sg.kb;
                    }
                }
            }
            if (!dead && pend) dead = !pv(pend_u, pend_first);
            if (dead) {
                atomicOr(&s_err, DSV4_EWORD_TIMEOUT);
                abort_flag = 1;
            }
        }
    } else if (warp >= 4) {
        // ---------------------------------------------------------------- softmax and output
        PagedWalk w(g, sched);
        PagedSeg sg;
        const int st = tid - 128, q4 = warp & 3, half = (warp - 4) >> 2;
        const int row = q4 * 32 + lane;                              // cache row of the unit, channel of an O tile
        const int c0 = half * (N / 2);                               // first query column of this thread
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(q4 * 32) << 16);
        uint32_t u = 0;
        bool dead = false;
        int d_parts = 0, d_tok = 0, d_tn = 0, d_head = 0, d_hv = 0;
        long long at = sched.u0;                                     // first unit of the segment on the line
        while (w.next(sg)) {
            soft_sync();                                             // the tile before is written out
            for (int c = st; c < N; c += kSoftThreads) {
                const int t = c / g.hb, h = c - t * g.hb;
                const bool ok = t < sg.tn && h < sg.hv;
                s_m[c] = ok ? -INFINITY : INFINITY;                  // (a column without a query gets P = 0)
                s_hi[c] = ok ? paged_hi(sg.q, sg.t0 + t) : 0;
                s_lo[c] = ok ? paged_lo(g, sg.q, sg.t0 + t) : 0;
                s_off[c] = ok ? (t * g.H + h) * D : -1;
            }
            soft_sync();
            float lacc[NC][32];                                      // this row's P per query, summed over the units
#pragma unroll
            for (int n = 0; n < NC; ++n)
#pragma unroll
                for (int i = 0; i < 32; ++i) lacc[n][i] = 0.f;
            for (int k = sg.kb; k < sg.ke; ++k, ++u) {
                if (!dead) dead = !mbar_wait(&s_full[u & 1], (u >> 1) & 1, &abort_flag, p.wait_ns);
                tc_fence_after();
                const int j0 = sg.row0 + k * kPT, j = j0 + row;
                const unsigned bad = *reinterpret_cast<volatile unsigned*>(&s_bad[u & 7]);
                const bool edge = j0 < sg.lo_u || j0 + kPT > sg.hi_u || bad != 0;
                const bool masked = edge || j0 < sg.lo_max || j0 + kPT > sg.hi_min;
                const bool live = j >= sg.lo_u && j < sg.hi_u && !((bad >> (row / g.br)) & 1);
                const uint32_t scol = lane_base + (u & 1) * N + c0;
                float x[NC][32];
                float mx = -INFINITY;
                auto load_scores = [&](int n) {
                    uint32_t r[32];
                    DSV4_TMEM_LD_32x32b_X32(scol + n * 32, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[n][i] = __uint_as_float(r[i]);
                };
                auto hide = [&](int n) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const int c = c0 + n * 32 + i;
                        if (!live || j >= s_hi[c] || j < s_lo[c]) x[n][i] = -INFINITY;
                    }
                };
#pragma unroll
                for (int n = 0; n < NC; ++n) {
                    load_scores(n);
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const float4 m4 = *reinterpret_cast<const float4*>(s_m + c0 + n * 32 + i);
                        x[n][i] = fmaf(x[n][i], p.scale2, -m4.x);
                        x[n][i + 1] = fmaf(x[n][i + 1], p.scale2, -m4.y);
                        x[n][i + 2] = fmaf(x[n][i + 2], p.scale2, -m4.z);
                        x[n][i + 3] = fmaf(x[n][i + 3], p.scale2, -m4.w);
                    }
                    if (masked) hide(n);
#pragma unroll
                    for (int i = 0; i < 32; ++i) mx = fmaxf(mx, x[n][i]);
                }
                bool rescale = false;
                if (soft_sync_or(mx > kSpan)) {
                    // some score outruns its reference: reduce the unit's maxima and move the references
#pragma unroll
                    for (int n = 0; n < NC; ++n) {
                        load_scores(n);
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[n][i] *= p.scale2;
                        if (masked) hide(n);
                        red[q4 * N + c0 + n * 32 + lane] = lanes_reduce<true>(x[n], lane);
                    }
                    soft_sync();
                    for (int c = st; c < N; c += kSoftThreads) {
                        const float cm = fmaxf(fmaxf(red[c], red[N + c]), fmaxf(red[2 * N + c], red[3 * N + c]));
                        const float mo = s_m[c];
                        float f = 1.f;
                        if (cm > mo) {
                            f = mo == -INFINITY ? 0.f : ex2(mo - cm);
                            s_m[c] = cm;
                            rescale = k > sg.kb;
                        }
                        s_f[c] = f;
                    }
                    rescale = soft_sync_or(rescale);
#pragma unroll
                    for (int n = 0; n < NC; ++n) {
                        load_scores(n);
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const int c = c0 + n * 32 + i;
                            lacc[n][i] *= s_f[c];
                            x[n][i] = fmaf(x[n][i], p.scale2, -s_m[c]);
                        }
                        if (masked) hide(n);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_empty[u & 1]);
                // P and O are free once the product before is done
                if (!dead && u > 0) dead = !mbar_wait(&pv_done, (u - 1) & 1, &abort_flag, p.wait_ns);
                if (rescale) {
                    tc_fence_after();
#pragma unroll
                    for (int n = 0; n < NC; ++n) {
                        for (int mt = 0; mt < MT; ++mt) {
                            uint32_t r[32];
                            const uint32_t ta = lane_base + C::OCOL + mt * N + c0 + n * 32;
                            DSV4_TMEM_LD_32x32b_X32(ta, r);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                r[i] = __float_as_uint(__uint_as_float(r[i]) * s_f[c0 + n * 32 + i]);
                            DSV4_TMEM_ST_32x32b_X32(ta, r);
                        }
                    }
                    DSV4_TMEM_WAIT_ST();
                }
                // P = 2^(s - m) in bf16 (rounded: the tensor core takes bf16; the sum below stays
                // in fp32), the MN-major operand: row j's 64 queries are one 128-byte line
#pragma unroll
                for (int n = 0; n < NC; ++n) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        x[n][i] = ex2(x[n][i]);
                        lacc[n][i] += x[n][i];
                    }
                    const int cb = c0 + n * 32;                      // first column of the piece
                    uint8_t* prow = sP + (cb >> 6) * (kPT * 128) + (row >> 3) * 1024 + (row & 7) * 128;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int c16 = ((cb & 63) >> 3) + i;
                        *reinterpret_cast<uint4*>(prow + ((c16 ^ (row & 7)) << 4)) =
                            make_uint4(pack2(x[n][8 * i], x[n][8 * i + 1]), pack2(x[n][8 * i + 2], x[n][8 * i + 3]),
                                       pack2(x[n][8 * i + 4], x[n][8 * i + 5]), pack2(x[n][8 * i + 6], x[n][8 * i + 7]));
                    }
                }
                if (edge) {
                    // rows of the tile that nobody may see (past the cache, before the window, of a
                    // page that was not loaded) hold anything: as V they must not meet P = 0
                    const uint32_t r = p.shared ? u : 2 * u + 1, slot = r % ST;
                    if (!p.shared && !dead) dead = !mbar_wait(&full[slot], (r / ST) & 1, &abort_flag, p.wait_ns);
                    if (!live) {
                        for (int b = half * (NB / 2); b < (half + 1) * (NB / 2); ++b) {
                            uint4* z = reinterpret_cast<uint4*>(sm + slot * C::TILE + b * C::BOX + row * 128);
#pragma unroll
                            for (int i = 0; i < 8; ++i) z[i] = make_uint4(0, 0, 0, 0);
                        }
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full);
            }
            // ---------------------------------------------------------------- the tile's results
            if (!dead) dead = !mbar_wait(&pv_done, (u - 1) & 1, &abort_flag, p.wait_ns);
            tc_fence_after();
#pragma unroll
            for (int n = 0; n < NC; ++n) red[q4 * N + c0 + n * 32 + lane] = lanes_reduce<false>(lacc[n], lane);
            soft_sync();
            const bool whole = sg.kb == 0 && sg.ke == sg.n;
            const int slot2 = blockIdx.x * 2 + (sg.kb > 0 ? 0 : 1);
            for (int c = st; c < N; c += kSoftThreads) {
                const float l = (red[c] + red[N + c]) + (red[2 * N + c] + red[3 * N + c]);
                const float m = s_m[c];
                const int off = s_off[c];
                if (whole) {
                    float f = 0.f;
                    if (off >= 0) {
                        const int t = c / g.hb, h = sg.head0 + c - t * g.hb;
                        const float snk = p.sink ? p.sink[h] * kLog2e : -INFINITY;
                        const float M = fmaxf(m, snk);
                        const float e = m == -INFINITY ? 0.f : exp2f(m - M);
                        const float den = l * e + (snk == -INFINITY ? 0.f : exp2f(snk - M));
                        f = m == -INFINITY ? 0.f : e / den;
                        if (p.lse)
                            p.lse[static_cast<size_t>(sg.tok0 + t) * g.H + h] =
                                M == -INFINITY ? -INFINITY : M * kLn2 + logf(den);
                    }
                    s_f[c] = f;
                } else {
                    float* ml = p.part_ml + (static_cast<size_t>(slot2) * N + c) * 2;
                    ml[0] = off >= 0 ? m : -INFINITY;
                    ml[1] = l;
                    s_f[c] = 1.f;
                }
            }
            soft_sync();
            float* po = p.part_o + static_cast<size_t>(slot2) * N * D;
            __nv_bfloat16* ob = p.out + (static_cast<size_t>(sg.tok0) * g.H + sg.head0) * D;
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                const int cb = c0 + n * 32;
                for (int mt = 0; mt < MT; ++mt) {
                    uint32_t r[32];
                    DSV4_TMEM_LD_32x32b_X32(lane_base + C::OCOL + mt * N + cb, r);
                    tmem_wait_ld();
                    if (!whole) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (s_off[cb + i] >= 0) po[(cb + i) * D + mt * 128 + row] = __uint_as_float(r[i]);
                        continue;
                    }
                    // two columns at a time: even lanes write the first, odd lanes the second, each
                    // a pair of neighbouring channels
                    const int d = mt * 128 + (row & ~1), pair = (d - (D - 2 * p.or_pairs)) >> 1;
                    const bool rot = p.orp && d >= D - 2 * p.or_pairs;
                    int rtok = -1;
                    float2 cs = make_float2(1.f, 0.f);
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        // (a factor of 0 stands for a query that sees nothing: O may hold anything)
                        const float f0 = s_f[cb + i], f1 = s_f[cb + i + 1];
                        const float a = f0 == 0.f ? 0.f : __uint_as_float(r[i]) * f0;
                        const float b = f1 == 0.f ? 0.f : __uint_as_float(r[i + 1]) * f1;
                        const float got = __shfl_xor_sync(~0u, (lane & 1) ? a : b, 1);
                        float e = (lane & 1) ? got : a, o = (lane & 1) ? b : got;
                        const int c = cb + i + (lane & 1), off = s_off[c];
                        if (off < 0) continue;
                        if (rot) {
                            const int tok = sg.tok0 + c / g.hb;
                            if (tok != rtok) { cs = out_rope_cs(p, tok, pair); rtok = tok; }
                            const float e0 = e;
                            e = e0 * cs.x + o * cs.y;
                            o = -e0 * cs.y + o * cs.x;
                        }
                        *reinterpret_cast<uint32_t*>(ob + off + d) = pack2(e, o);
                    }
                }
            }
            if (!whole && sg.kb == 0) {                              // this CTA starts the tile: it is merged under its number
                const long long end = at + sg.n, T = sched.total;
                int last = static_cast<int>((end * sched.ge - 1) / T);
                while (last + 1 < sched.ge && T * (last + 1) / sched.ge < end) ++last;
                while (T * last / sched.ge >= end) --last;
                d_parts = last - static_cast<int>(blockIdx.x) + 1;
                d_tok = sg.tok0;
                d_tn = sg.tn;
                d_head = sg.head0;
                d_hv = sg.hv;
            }
            at += sg.ke - sg.kb;
        }
        if (dead && lane == 0) {
            atomicOr(&s_err, DSV4_EWORD_TIMEOUT);
            abort_flag = 1;
        }
        if (st == 0) {
            int* d = p.desc + blockIdx.x * 8;
            d[0] = d_parts; d[1] = d_tok; d[2] = d_tn; d[3] = d_head; d[4] = d_hv;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 2) tmem_dealloc(tmem, C::TCOLS);
    if (tid == 0) p.err[blockIdx.x] = s_err;
}

// Merges the partial results of the row tiles that several CTAs worked on: one block per (tile,
// query), its threads over channels x groups of partials. Also gathers the error bits.
constexpr int kMergeThreads = 512;
template <int D, int N>
__global__ void __launch_bounds__(kMergeThreads)
paged_merge_kernel(const __grid_constant__ PagedAttnParams p, int ctas, uint32_t* eword) {
    constexpr int LD = D / 4, GR = kMergeThreads / LD;
    __shared__ int starts[160 + 8];
    __shared__ float wgt[512];
    __shared__ float4 acc[GR][LD];
    __shared__ float bc[2];
    __shared__ int n_starts;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    if (warp == 0) {                     // the tiles to merge, by the CTA that starts each
        int n = 0;
        uint32_t err = 0;
        for (int c0 = 0; c0 < ctas; c0 += 32) {
            const int c = c0 + lane;
            const bool is = c < ctas && p.desc[c * 8] > 0;
            if (c < ctas) err |= p.err[c];
            const unsigned b = __ballot_sync(~0u, is);
            if (is) starts[n + __popc(b & ((1u << lane) - 1))] = c;
            n += __popc(b);
        }
        err = __reduce_or_sync(~0u, err);
        if (lane == 0) n_starts = n;
        if (lane == 0 && blockIdx.x == 0) *eword = err;
    }
    __syncthreads();
    const PagedGeom& g = p.g;
    for (int item = blockIdx.x; item < n_starts * N; item += gridDim.x) {
        const int first = starts[item / N], c = item % N;
        const int* d = p.desc + first * 8;
        const int np = d[0], t = c / g.hb, hh = c - t * g.hb;
        if (t >= d[2] || hh >= d[4]) continue;
        const int h = d[3] + hh, tok = d[1] + t;
        auto slot = [&](int i) { return static_cast<size_t>(i ? (first + i) * 2 : first * 2 + 1) * N + c; };
        if (warp == 0) {
            float M = -INFINITY;
            for (int i = lane; i < np; i += 32) M = fmaxf(M, p.part_ml[slot(i) * 2]);
            for (int w = 16; w; w >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, w));
            const float snk = p.sink ? p.sink[h] * kLog2e : -INFINITY;
            const float top = fmaxf(M, snk);
            float l = 0.f;
            for (int i = lane; i < np; i += 32) {
                const float m = p.part_ml[slot(i) * 2];
                const float e = m == -INFINITY ? 0.f : exp2f(m - top);
                wgt[i] = e;
                l += e * p.part_ml[slot(i) * 2 + 1];
            }
            for (int w = 16; w; w >>= 1) l += __shfl_xor_sync(~0u, l, w);
            if (lane == 0) {
                const float den = l + (snk == -INFINITY ? 0.f : exp2f(snk - top));
                bc[0] = M == -INFINITY ? 0.f : 1.f / den;
                if (p.lse)
                    p.lse[static_cast<size_t>(tok) * g.H + h] = top == -INFINITY ? -INFINITY : top * kLn2 + logf(den);
            }
        }
        __syncthreads();
        const int dl = tid % LD, gr = tid / LD;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int i = gr; i < np; i += GR) {
            const float e = wgt[i];
            const float4 v = *reinterpret_cast<const float4*>(p.part_o + slot(i) * D + dl * 4);
            if (e != 0.f) {
                a.x = fmaf(e, v.x, a.x); a.y = fmaf(e, v.y, a.y);
                a.z = fmaf(e, v.z, a.z); a.w = fmaf(e, v.w, a.w);
            }
        }
        acc[gr][dl] = a;
        __syncthreads();
        if (gr == 0) {
            float o[4] = {a.x, a.y, a.z, a.w};
            for (int i = 1; i < GR; ++i) {
                const float4 v = acc[i][dl];
                o[0] += v.x; o[1] += v.y; o[2] += v.z; o[3] += v.w;
            }
            const float f = bc[0];
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] *= f;
            if (p.orp) {
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    const int ch = dl * 4 + i, pair = (ch - (D - 2 * p.or_pairs)) >> 1;
                    if (ch >= D - 2 * p.or_pairs) {
                        const float2 cs = out_rope_cs(p, tok, pair);
                        const float e0 = o[i], o0 = o[i + 1];
                        o[i] = e0 * cs.x + o0 * cs.y;
                        o[i + 1] = -e0 * cs.y + o0 * cs.x;
                    }
                }
            }
            *reinterpret_cast<uint2*>(p.out + (static_cast<size_t>(tok) * g.H + h) * D + dl * 4) =
                make_uint2(pack2(o[0], o[1]), pack2(o[2], o[3]));
        }
        __syncthreads();
    }
}

// Query columns per row tile: 128 where chunks fill them and the accumulators fit.
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
        !paged_pool_map(&kmap, a.k_pages, D, a.kv_heads, a.page_size, a.num_pages, p.g.br) ||
        !paged_pool_map(&vmap, a.v_pages ? a.v_pages : a.k_pages, D, a.kv_heads, a.page_size, a.num_pages, p.g.br))
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
    p.scale2 = a.scale * kLog2e;
    p.orp = a.out_rope_pos;
    p.or_pairs = a.out_rope_pos ? a.out_rope_dim / 2 : 0;
    for (int j = 0; j < p.or_pairs; ++j) p.or_freq[j] = std::pow(a.out_rope_theta, -2.0 * j / a.out_rope_dim);
    p.shared = a.v_pages == nullptr;
    p.min_units = 2;
    p.wait_ns = kDefaultWaitNs;
    auto kern = paged_attn_kernel<D, N>;
    if (once_per_device(reinterpret_cast<const void*>(kern), kAttrLaunch, [kern] {
            return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        }) != cudaSuccess)
        return DSV4_ERR_LAUNCH;
    count_launch();
    if (launch_k(kern, dim3(ctas), dim3(kThreads), C::SMEM, st, true, qmap, kmap, vmap, p) != cudaSuccess) return DSV4_ERR_LAUNCH;
    count_launch();
    if (launch_k(paged_merge_kernel<D, N>, dim3(ctas * 2), dim3(kMergeThreads), 0, st, true, p, ctas, eword) != cudaSuccess)
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
    g.window = window;
    g.br = paged_box_rows(page_size);
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
    const size_t n = static_cast<size_t>(attn_ctas()) * 2 * tile_queries(a);
    return align_up(n * 2 * 4, 256) + n * a.dim * 4 + static_cast<size_t>(attn_ctas()) * 9 * 4;
}

int launch_paged_attn(const dsv4_paged_attn_args& a, uint8_t* ws, uint32_t* eword, cudaStream_t st) {
    if (a.batch == 0 || a.total_q == 0) return cudaMemsetAsync(eword, 0, 4, st) == cudaSuccess ? DSV4_OK : DSV4_ERR_LAUNCH;
    const int n = tile_queries(a);
    if (a.dim == 512) return run<512, 64>(a, ws, eword, st);
    if (a.dim == 256) return n == 64 ? run<256, 64>(a, ws, eword, st) : run<256, 128>(a, ws, eword, st);
    return n == 64 ? run<128, 64>(a, ws, eword, st) : run<128, 128>(a, ws, eword, st);
}

}  // namespace dsv4
