// RMSNorm of queries and keys per head, RoPE, and the append of the rows to the paged cache.
//
//   y = x / sqrt(mean(x^2) + eps) * gamma, pairs (2j, 2j + 1) of the last rope_dim channels
//   turned by pos * theta^(-2j / rope_dim), one rounding to bf16
// Sources: "nvfp4-megamoe-kernel: compare master..pure-nvfp4", single_shot_inference.py
// (RMSNorm of q per head, kv_norm, RoPE, append to the sliding-window cache);
// "nvfp4-megamoe-kernel: compare v0.1-e2e-working...v-c1-c2-c3-20260602", compressor_reduce.cu
// apply_kv_norm_kernel.
//
// Every element is read and written once (the floor is HBM). One launch serves query heads, keys and
// values, so a fused projection's output is read where it lies. A CTA takes one token (or, with
// few tokens, a share of one token's heads): the token's angles are formed once (fp64, Cody-
// Waite reduced) into shared memory while its rows are already on their way; a row lies in 16 or
// 32 lanes, 8 channels (one 16-byte load) per lane and vector, so its pairs stay inside a thread
// and the sum of squares takes four or five shuffles. A lane has the same channels of every row:
// weight, cosine and sine become four factors per pair, held in registers for all rows, and a
// pair costs three paired operations (with each row working out its own, the kernel issued 205
// instructions per 16 bytes and was bound by that).
// Measured: 2,039 tokens of 64 + 8 + 8 heads x 128 19.5 us, 4.3 TB/s: latency of loads, shuffles and
// barriers at eight CTAs per SM (64 registers a thread) in 1.7 waves, with 28 % of the issue slots
// used; 16 tokens of 64 + 1 x 512 3.7 us, a launch and one chain of latencies.
#include <cmath>

#include "internal.h"
#include "common.cuh"

namespace dsv4 {
namespace {

constexpr int kT = 128, kMaxPairs = 64;
struct NormRopeParams {
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16 *q_out, *k_pages, *v_pages;
    const int64_t *slots, *pos;
    const float *gamma_q, *gamma_k;
    long long q_stride, k_stride, v_stride, q_out_stride, n_slots;
    int tokens, heads, kv_heads, split, pairs;
    float eps;
    double freq[kMaxPairs];              // theta^(-2j / rope_dim)
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// A lane's factors for its pairs of channels: the pair (e, o) of a normed row becomes
// (e, o) * a + (o, e) * b with a = (w_e cos, w_o cos), b = (-w_o sin, w_e sin).
template <int VL>
struct Factors { uint64_t a[VL][4], b[VL][4]; };

template <int D>
__global__ void __launch_bounds__(kT)
norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
    constexpr int LR = D >= 256 ? 32 : 16;               // lanes per row
    constexpr int VL = D / (8 * LR);                     // 16-byte vectors per lane
    constexpr int RP = kT / LR;                          // rows per pass
    constexpr int U = 4;                                 // passes whose loads are in flight together
    __shared__ float4 fac[2][D / 2];                     // of queries and keys, per pair
    const int tid = threadIdx.x, sub = tid / LR, l = tid % LR;
    const int tok = blockIdx.x / p.split, part = blockIdx.x - tok * p.split;
    // with few tokens: the parts but the last share the query heads, the last has the keys and values
    const int qn = p.split > 1 ? p.split - 1 : 1;
    const int qa = part < qn ? p.heads * part / qn : p.heads, qb = part < qn ? p.heads * (part + 1) / qn : p.heads;
    const bool kv = part == p.split - 1 && p.kv_heads > 0;
    pdl_trigger();
    pdl_wait();
    auto load = [&](const __nv_bfloat16* src, int r, int n, uint4 (&x)[VL]) {
        if (r >= n) return;
#pragma unroll
        for (int i = 0; i < VL; ++i) x[i] = *reinterpret_cast<const uint4*>(src + static_cast<long long>(r) * D + (i * LR + l) * 8);
    };
    const __nv_bfloat16* q = p.q + tok * p.q_stride;
    const __nv_bfloat16* k = p.k + tok * p.k_stride;
    const __nv_bfloat16* v = p.v + tok * p.v_stride;
    uint4 x[U][VL], xk[VL], xv[VL];
#pragma unroll
    for (int u = 0; u < U; ++u) load(q, qa + sub + u * RP, qb, x[u]);
    if (kv) {
        load(k, sub, p.kv_heads, xk);
        if (p.v) load(v, sub, p.kv_heads, xv);
    }
    const long long slot = kv ? p.slots[tok] : -1;
    const int rope0 = D - 2 * p.pairs;
    for (int i = tid; i < D / 2; i += kT) {
        float sn = 0.f, c = 1.f;
        if (2 * i >= rope0) sincosf(reduced_angle(static_cast<double>(p.pos[tok]) * p.freq[i - rope0 / 2]), &sn, &c);
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {
            const float* gamma = kind ? p.gamma_k : p.gamma_q;
            float2 w = make_float2(1.f, 1.f);
            if (gamma) w = *reinterpret_cast<const float2*>(gamma + 2 * i);
            fac[kind][i] = make_float4(w.x * c, w.y * c, -w.y * sn, w.x * sn);
        }
    }
    __syncthreads();
    auto factors = [&](int kind, Factors<VL>& f) {
#pragma unroll
        for (int i = 0; i < VL; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const ulonglong2 t = *reinterpret_cast<const ulonglong2*>(&fac[kind][(i * LR + l) * 4 + j]);
                f.a[i][j] = t.x;
                f.b[i][j] = t.y;
            }
    };
    auto row = [&](const uint4 (&xr)[VL], const Factors<VL>& f, __nv_bfloat16* dst, bool on) {
        uint64_t ss2 = 0ull;
#pragma unroll
        for (int i = 0; i < VL; ++i) {
            const uint32_t w[4] = {xr[i].x, xr[i].y, xr[i].z, xr[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint64_t eo = pack_f32x2(bf16_lo(w[j]), bf16_hi(w[j]));
                fma_f32x2(ss2, eo, eo);
            }
        }
        float sa, sb;
        unpack_f32x2(ss2, sa, sb);
        float ss = sa + sb;
#pragma unroll
        for (int w = LR / 2; w; w >>= 1) ss += __shfl_xor_sync(~0u, ss, w);
        // (the hardware's reciprocal root: within 2 units of the last place, the output has 16 bits fewer)
        const float inv = rsqrtf(ss * (1.f / D) + p.eps);
        const uint64_t inv2 = pack_f32x2(inv, inv);
        if (!on) return;
#pragma unroll
        for (int i = 0; i < VL; ++i) {
            const uint32_t w[4] = {xr[i].x, xr[i].y, xr[i].z, xr[i].w};
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float e = bf16_lo(w[j]), d = bf16_hi(w[j]);
                uint64_t y = mul_f32x2(pack_f32x2(e, d), f.a[i][j]);
                fma_f32x2(y, pack_f32x2(d, e), f.b[i][j]);
                float y0, y1;
                unpack_f32x2(mul_f32x2(y, inv2), y0, y1);
                o[j] = pack2(y0, y1);
            }
            *reinterpret_cast<uint4*>(dst + (i * LR + l) * 8) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    };
    Factors<VL> f;
    if (qa < qb) {
        factors(0, f);
        __nv_bfloat16* out = p.q_out + tok * p.q_out_stride;
        for (int base = qa; base < qb; base += U * RP) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = base + sub + u * RP;
                row(x[u], f, out + static_cast<long long>(r) * D, r < qb);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) load(q, base + sub + (U + u) * RP, qb, x[u]);
        }
    }
    if (kv && slot >= 0 && slot < p.n_slots) {
        factors(1, f);
        const long long at = slot * p.kv_heads;
        for (int base = 0; base < p.kv_heads; base += RP) {
            const int r = base + sub;
            row(xk, f, p.k_pages + (at + r) * D, r < p.kv_heads);
            if (p.v && r < p.kv_heads) {
#pragma unroll
                for (int i = 0; i < VL; ++i) *reinterpret_cast<uint4*>(p.v_pages + (at + r) * D + (i * LR + l) * 8) = xv[i];
            }
            load(k, r + RP, p.kv_heads, xk);
            if (p.v) load(v, r + RP, p.kv_heads, xv);
        }
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
    p.pairs = a.rope_dim / 2;
    p.eps = a.eps;
    for (int j = 0; j < p.pairs; ++j) p.freq[j] = std::pow(a.rope_theta, -2.0 * j / a.rope_dim);
    // With few tokens a token's heads are spread over CTAs of one pass each, and its keys and values
    // have one; with many, one CTA per token forms the angles and the factors once.
    constexpr int RP = kT / (D >= 256 ? 32 : 16);
    const int sms = sm_count() > 0 ? sm_count() : 152;
    p.split = a.tokens < 4 * sms ? (a.heads + RP - 1) / RP + 1 : 1;
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
