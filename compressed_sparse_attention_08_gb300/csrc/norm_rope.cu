// RMSNorm of queries and keys per head, RoPE, and the append of the rows to the paged cache.
//
//   y = x / sqrt(mean(x^2) + eps) * gamma, pairs (2j, 2j + 1) of the last rope_dim channels
//   turned by pos * theta^(-2j / rope_dim), one rounding to bf16
// Sources: "nvfp4-megamoe-kernel: compare master..pure-nvfp4", single_shot_inference.py
// (RMSNorm of q per head, kv_norm, RoPE, append to the sliding-window cache);
// "nvfp4-megamoe-kernel: compare v0.1-e2e-working...v-c1-c2-c3-20260602", compressor_reduce.cu
// apply_kv_norm_kernel.
//
// HBM bound: every element is read and written once. One launch serves query heads, keys and
// values, so a fused projection's output is read where it lies. A CTA takes one token (or, with
// few tokens, a share of one token's heads): the token's angles are formed once (fp64, Cody-
// Waite reduced) into shared memory while the first rows are already on their way; a row lies
// in 16 or 32 lanes, 8 channels (one 16-byte load) per lane and vector, so its pairs stay inside
// a thread and the sum of squares takes four or five shuffles. Six such loads per thread are in
// flight at once.
#include <cmath>

#include "internal.h"
#include "common.cuh"

namespace dsv4 {
namespace {

constexpr int kT = 256, kMaxPairs = 64;
constexpr int kLoads = 6;                // 16-byte loads of a thread in flight

struct NormRopeParams {
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16 *q_out, *k_pages, *v_pages;
    const int64_t *slots, *pos;
    const float *gamma_q, *gamma_k;
    long long q_stride, k_stride, v_stride, q_out_stride, n_slots;
    int tokens, heads, kv_heads, rows, split, pairs;
    float eps;
    double freq[kMaxPairs];              // theta^(-2j / rope_dim)
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

template <int D>
__global__ void __launch_bounds__(kT)
norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
    constexpr int LR = D >= 256 ? 32 : 16;               // lanes per row
    constexpr int VL = D / (8 * LR);                     // 16-byte vectors per lane
    constexpr int RP = kT / LR;                          // rows per pass
    constexpr int U = kLoads / VL;                       // passes whose loads are in flight together
    __shared__ float2 cs[kMaxPairs];
    const int tid = threadIdx.x, sub = tid / LR, l = tid % LR;
    const int tok = blockIdx.x / p.split, part = blockIdx.x - tok * p.split;
    const int r0 = static_cast<int>(static_cast<long long>(p.rows) * part / p.split);
    const int r1 = static_cast<int>(static_cast<long long>(p.rows) * (part + 1) / p.split);
    pdl_trigger();
    pdl_wait();
    // a weight's 8 channels from c as pairs, or ones
    auto gamma_of = [](const float* gamma, int c, uint64_t (&g)[4]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) g[j] = gamma ? *reinterpret_cast<const uint64_t*>(gamma + c + 2 * j) : pack_f32x2(1.f, 1.f);
    };
    uint4 x[U][VL];
    // rows of a token: its query heads, its keys, its values
    auto load = [&](int base) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = base + u * RP;
            if (r >= r1) continue;
            const __nv_bfloat16* src;
            if (r < p.heads) src = p.q + tok * p.q_stride + static_cast<long long>(r) * D;
            else if (r < p.heads + p.kv_heads) src = p.k + tok * p.k_stride + static_cast<long long>(r - p.heads) * D;
            else src = p.v + tok * p.v_stride + static_cast<long long>(r - p.heads - p.kv_heads) * D;
#pragma unroll
            for (int i = 0; i < VL; ++i) x[u][i] = *reinterpret_cast<const uint4*>(src + (i * LR + l) * 8);
        }
    };
    load(r0 + sub);
    const long long slot = p.slots ? p.slots[tok] : -1;
    if (tid < p.pairs) {
        float sn, c;
        sincosf(reduced_angle(static_cast<double>(p.pos[tok]) * p.freq[tid]), &sn, &c);
        cs[tid] = make_float2(c, sn);
    }
    __syncthreads();
    const int rope0 = D - 2 * p.pairs;
    uint64_t gq[VL][4];
#pragma unroll
    for (int i = 0; i < VL; ++i) gamma_of(p.gamma_q, (i * LR + l) * 8, gq[i]);
    for (int base = r0 + sub; __any_sync(~0u, base < r1); base += U * RP) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = base + u * RP;
            const bool on = r < r1, is_q = r < p.heads, is_v = r >= p.heads + p.kv_heads;
            if (!__any_sync(~0u, on)) break;
            uint64_t f[VL][4], ss2 = 0ull;               // channel pairs
#pragma unroll
            for (int i = 0; i < VL; ++i) {
                const uint32_t w[4] = {x[u][i].x, x[u][i].y, x[u][i].z, x[u][i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    f[i][j] = pack_f32x2(bf16_lo(w[j]), bf16_hi(w[j]));
                    fma_f32x2(ss2, f[i][j], f[i][j]);
                }
            }
            float sa, sb;
            unpack_f32x2(ss2, sa, sb);
            float ss = sa + sb;
#pragma unroll
            for (int w = LR / 2; w; w >>= 1) ss += __shfl_xor_sync(~0u, ss, w);
            // (the hardware's reciprocal root: within 2 units of the last place, the output has 16 fewer bits)
            const float inv = rsqrtf(ss * (1.f / D) + p.eps);
            const uint64_t inv2 = pack_f32x2(inv, inv);
            __nv_bfloat16* dst = nullptr;
            if (on) {
                if (is_q) {
                    dst = p.q_out + tok * p.q_out_stride + static_cast<long long>(r) * D;
                } else if (slot >= 0 && slot < p.n_slots) {
                    const int h = r - p.heads - (is_v ? p.kv_heads : 0);
                    dst = (is_v ? p.v_pages : p.k_pages) + (slot * p.kv_heads + h) * D;
                }
            }
            if (!dst) continue;
#pragma unroll
            for (int i = 0; i < VL; ++i) {
                const int c0 = (i * LR + l) * 8;
                uint4 y = x[u][i];
                if (!is_v) {
                    uint64_t g[4];
                    if (is_q) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) g[j] = gq[i][j];
                    } else {
                        gamma_of(p.gamma_k, c0, g);
                    }
                    uint32_t o[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float e, d;
                        unpack_f32x2(mul_f32x2(mul_f32x2(f[i][j], inv2), g[j]), e, d);
                        const int pr = (c0 + 2 * j - rope0) >> 1;
                        if (pr >= 0) {
                            const float2 t = cs[pr];
                            const float e0 = e;
                            e = e0 * t.x - d * t.y;
                            d = e0 * t.y + d * t.x;
                        }
                        o[j] = pack2(e, d);
                    }
                    y = make_uint4(o[0], o[1], o[2], o[3]);
                }
                *reinterpret_cast<uint4*>(dst + c0) = y;
            }
        }
        load(base + U * RP);
    }
}

template <int D>
int run(const dsv4_norm_rope_args& a, cudaStream_t st) {
    NormRopeParams p{};
    p.q = static_cast<const __nv_bfloat16*>(a.q);
    p.k = static_cast<const __nv_bfloat16*>(a.k);
    p.v = static_cast<const __nv_bfloat16*>(a.v);
    p.q_out = static_cast<__nv_bfloat16*>(a.q_out);
    p.k_pages = static_cast<__nv_bfloat16*>(a.k_pages);
    p.v_pages = static_cast<__nv_bfloat16*>(a.v_pages);
    p.slots = a.kv_heads ? a.slots : nullptr;
    p.pos = a.pos;
    p.gamma_q = a.gamma_q;
    p.gamma_k = a.gamma_k;
    p.q_stride = a.q_stride;
    p.k_stride = a.k_stride;
    p.v_stride = a.v_stride;
    p.q_out_stride = a.q_out_stride;
    p.n_slots = static_cast<long long>(a.num_pages) * a.page_size;
    p.tokens = a.tokens;
    p.heads = a.heads;
    p.kv_heads = a.kv_heads;
    p.rows = a.heads + a.kv_heads * (a.v ? 2 : 1);
    p.pairs = a.rope_dim / 2;
    p.eps = a.eps;
    for (int j = 0; j < p.pairs; ++j) p.freq[j] = std::pow(a.rope_theta, -2.0 * j / a.rope_dim);
    // With few tokens a token's heads are spread over CTAs of one pass each; with many, one CTA
    // per token forms the angles once.
    constexpr int RP = kT / (D >= 256 ? 32 : 16);
    const int sms = sm_count() > 0 ? sm_count() : 152;
    p.split = a.tokens < 4 * sms ? (p.rows + RP - 1) / RP : 1;
    count_launch();
    return launch_k(norm_rope_kernel<D>, dim3(static_cast<unsigned>(a.tokens) * p.split), dim3(kT), 0, st, true, p) == cudaSuccess
               ? DSV4_OK : DSV4_ERR_LAUNCH;
}

}  // namespace

int launch_norm_rope(const dsv4_norm_rope_args& a, cudaStream_t st) {
    if (a.tokens == 0 || a.heads + a.kv_heads == 0) return DSV4_OK;
    if (a.dim == 512) return run<512>(a, st);
    if (a.dim == 256) return run<256>(a, st);
    return run<128>(a, st);
}

}  // namespace dsv4
