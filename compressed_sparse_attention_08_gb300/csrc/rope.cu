// Rotary positions of queries and keys, and the append of the rows to the paged cache.
//
//   (a, b) -> m (a cos t - b sin t, a sin t + b cos t),  t = +-pos f_j, for the pairs (2j, 2j + 1) or
//   (j, j + rope_dim / 2) of a part of each head; the other channels are copied
// f_j: theta^(-2j / rope_dim), or scaled for a longer context (B. Peng, J. Quesnelle, H. Fan, E.
// Shippole, "YaRN: Efficient Context Window Extension of Large Language Models", 2023). The sources'
// pages rotate interleaved pairs of the last 64 channels ("nvfp4-megamoe-kernel: compare
// master..pure-nvfp4", single_shot_inference.py _apply_rope); the second layout, the scaled
// frequencies and the other types are this library's own.
//
// Every element is read and written once (the floor is HBM). A CTA takes one token, or, with few
// tokens, a share of one token's heads. A thread has one column of the heads (16 bytes, or two times 16
// bytes half a part apart) and goes down the heads with it, so that the cosines and sines of its pairs
// are read from shared memory once and stay in registers. They are formed once per CTA, in fp64 (Cody-
// Waite reduced), while the first rows are already on their way.
// What matters is how many such CTAs an SM holds (each waits for a position, then for its loads and angles): 128
// threads held to 72 registers where a column is two vectors and to 48 where it is one. Measured: 2,039 tokens of 64 + 8 + 8
// heads x 128 with the append 17.0 us, 4.9 TB/s (with 256 threads 19.2); 1,023 tokens of 64 + 1 x 512, 64 channels
// turning, 27.8 us, 4.9 TB/s; 8,192 tokens of 32 + 8 x 128 in fp32 59.9 us, 5.6 TB/s of 6.8; 16 tokens 4.3 us. CTAs that walk
// the tokens with the next one's loads in registers were slower (23, 37 and 83 us): fewer fit, and a barrier a token
// ties their threads together.
#include <cmath>
#include <cuda_fp16.h>
#include <type_traits>

#include "internal.h"
#include "common.cuh"

namespace dsv4 {
namespace {

constexpr int kT = 128, kMaxPairs = 256;
constexpr int kInFlight = 4;             // heads per thread whose loads are in flight together

struct RopePart {                        // queries, keys or values
    const uint8_t* src;
    uint8_t* dst;
    long long src_stride, dst_stride;    // bytes from token to token (dst: from slot to slot with slots)
    int heads;
};
struct RopeParams {
    RopePart part[3];
    const int64_t *slots, *pos;
    long long n_slots;
    int tokens, split;
    int row;                             // bytes of a head
    int cols, rot0, rot;                 // columns a head is cut into; those that rotate: [rot0, rot0 + rot)
    int half;                            // bytes from a pair's first channel to its second (layout 1)
    int first, pairs;
    float magnitude, sign;
    double freq[kMaxPairs];
};

// 16 bytes of a type as floats, and back.
template <class E>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void get(const uint4& x, float (&f)[N]) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) { f[2 * i] = bf16_lo(w[i]); f[2 * i + 1] = bf16_hi(w[i]); }
    }
    static __device__ __forceinline__ uint4 put(const float (&f)[N]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&v);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ float one(const void* p) { return __bfloat162float(*static_cast<const __nv_bfloat16*>(p)); }
    static __device__ __forceinline__ void one(void* p, float f) { *static_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(f); }
};
template <>
struct Vec<__half> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void get(const uint4& x, float (&f)[N]) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
        }
    }
    static __device__ __forceinline__ uint4 put(const float (&f)[N]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 v = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&v);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ float one(const void* p) { return __half2float(*static_cast<const __half*>(p)); }
    static __device__ __forceinline__ void one(void* p, float f) { *static_cast<__half*>(p) = __float2half_rn(f); }
};
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void get(const uint4& x, float (&f)[N]) {
        f[0] = __uint_as_float(x.x); f[1] = __uint_as_float(x.y); f[2] = __uint_as_float(x.z); f[3] = __uint_as_float(x.w);
    }
    static __device__ __forceinline__ uint4 put(const float (&f)[N]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
    static __device__ __forceinline__ float one(const void* p) { return *static_cast<const float*>(p); }
    static __device__ __forceinline__ void one(void* p, float f) { *static_cast<float*>(p) = f; }
};

// How a head is cut into columns: pairs side by side, 16 bytes each; halves of a part whose vectors
// are aligned, 2 x 16 bytes where they rotate and 16 where not; any other halves, single channels.
enum { kPairs = 0, kHalves = 1, kScalar = 2 };

template <class E, int MODE>
__global__ void __launch_bounds__(kT, MODE == kHalves ? 7 : 10)
rope_kernel(const __grid_constant__ RopeParams p) {
    using V = Vec<E>;
    constexpr int N = V::N, U = kInFlight;
    constexpr int NF = MODE == kPairs ? N / 2 : MODE == kHalves ? N : 1;
    using Data = typename std::conditional<MODE == kScalar, E, uint4>::type;
    __shared__ float2 cs[kMaxPairs];
    const int tid = threadIdx.x;
    const int tok = blockIdx.x / p.split, part = blockIdx.x - tok * p.split;
    pdl_trigger();
    pdl_wait();
    const int64_t pos = p.pos[tok];
    const long long slot = p.slots ? p.slots[tok] : tok;
    const int most = p.part[0].heads + p.part[1].heads + p.part[2].heads;
    const int h0 = most * part / p.split, hn = most * (part + 1) / p.split;
    const int rp = p.cols < kT ? kT / p.cols : 1;        // heads per pass
    const int sub = tid / p.cols;
    for (int c0 = 0; c0 < p.cols; c0 += kT) {            // (more than kT columns: in laps)
        const int col = c0 + tid - sub * p.cols;
        const bool here = sub < rp && col < p.cols;
        const bool rot = here && col >= p.rot0 && col < p.rot0 + p.rot;
        constexpr int width = MODE == kScalar ? static_cast<int>(sizeof(E)) : 16;
        const int at = MODE == kPairs || col < p.rot0 + p.rot ? col * width : col * width + p.half;   // place in a head
        // where a head's column comes from and goes to; nothing in place where it does not turn
        auto place = [&](int h, const uint8_t*& src, uint8_t*& dst) {
            int w = 0;
            if (h >= p.part[0].heads) { h -= p.part[0].heads; w = 1; }
            if (w && h >= p.part[1].heads) { h -= p.part[1].heads; w = 2; }
            const RopePart& r = p.part[w];
            src = r.src + tok * r.src_stride + static_cast<long long>(h) * p.row + at;
            dst = r.dst + (w ? slot : tok) * r.dst_stride + static_cast<long long>(h) * p.row + at;
            return rot && w < 2;
        };
        Data a[U], b[U];
        auto load = [&](int base) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = base + u * rp;
                if (!here || h >= hn) continue;
                const uint8_t* src;
                uint8_t* dst;
                place(h, src, dst);
                a[u] = *reinterpret_cast<const Data*>(src);
                if (MODE != kPairs && rot) b[u] = *reinterpret_cast<const Data*>(src + p.half);
            }
        };
        load(h0 + sub);                                  // (on their way while the angles are formed)
        if (c0 == 0) {
            for (int i = tid; i < p.pairs; i += kT) {
                float sn, c;
                sincosf(reduced_angle(static_cast<double>(pos) * p.freq[i]), &sn, &c);
                cs[i] = make_float2(c * p.magnitude, sn * p.magnitude * p.sign);
            }
            __syncthreads();
        }
        if (!here) continue;
        // a token without a slot stores no keys and values
        const int h1 = p.slots && !(slot >= 0 && slot < p.n_slots) ? min(hn, p.part[0].heads) : hn;
        float2 f[NF];
        unsigned in = ~0u;                               // pairs of the column that belong to the part
        if constexpr (MODE == kPairs) {
            in = 0;
#pragma unroll
            for (int i = 0; i < NF; ++i) {
                const int j = (col * N - p.first) / 2 + i;
                const bool on = j >= 0 && j < p.pairs;
                in |= on ? 1u << i : 0u;
                f[i] = on ? cs[j] : make_float2(1.f, 0.f);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NF; ++i) f[i] = rot ? cs[(col - p.rot0) * NF + i] : make_float2(1.f, 0.f);
        }
        for (int base = h0 + sub; base < h1; base += U * rp) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = base + u * rp;
                if (h >= h1) continue;
                const uint8_t* src;
                uint8_t* dst;
                const bool turn = place(h, src, dst);
                if (!turn && src == dst) continue;       // (in place: the copy is there)
                if (turn) {
                    if constexpr (MODE == kScalar) {
                        const float x = V::one(&a[u]), y = V::one(&b[u]);
                        V::one(&a[u], x * f[0].x - y * f[0].y);
                        V::one(&b[u], x * f[0].y + y * f[0].x);
                    } else {
                        float x[N];
                        V::get(a[u], x);
                        if constexpr (MODE == kPairs) {
#pragma unroll
                            for (int i = 0; i < NF; ++i) {
                                const float e = x[2 * i], o = x[2 * i + 1];
                                if (!(in >> i & 1)) continue;    // (a copy, also of what has no product with 0)
                                x[2 * i] = e * f[i].x - o * f[i].y;
                                x[2 * i + 1] = e * f[i].y + o * f[i].x;
                            }
                        } else {
                            float y[N];
                            V::get(b[u], y);
#pragma unroll
                            for (int i = 0; i < NF; ++i) {
                                const float e = x[i], o = y[i];
                                x[i] = e * f[i].x - o * f[i].y;
                                y[i] = e * f[i].y + o * f[i].x;
                            }
                            b[u] = V::put(y);
                        }
                        a[u] = V::put(x);
                    }
                }
                *reinterpret_cast<Data*>(dst) = a[u];
                if (MODE != kPairs && rot) *reinterpret_cast<Data*>(dst + p.half) = b[u];
            }
            if (base + U * rp < h1) load(base + U * rp);
        }
    }
}

template <class E>
int run(const dsv4_rope_args& a, RopeParams& p, cudaStream_t st) {
    constexpr int size = sizeof(E), N = 16 / size;
    p.row = a.dim * size;
    const long long pool = static_cast<long long>(a.kv_heads) * p.row;
    p.part[0] = {static_cast<const uint8_t*>(a.q), static_cast<uint8_t*>(a.q_out), a.q_stride * size, a.q_out_stride * size, a.heads};
    p.part[1] = {static_cast<const uint8_t*>(a.k), static_cast<uint8_t*>(a.k_out), a.k_stride * size,
                 a.slots ? pool : a.k_out_stride * size, a.kv_heads};
    p.part[2] = {static_cast<const uint8_t*>(a.v), static_cast<uint8_t*>(a.v_out), a.v_stride * size, pool, a.v ? a.kv_heads : 0};
    const int hd = a.rope_dim / 2;
    int mode = kPairs;
    if (a.layout == 0) {
        p.cols = a.dim / N;
        p.rot0 = a.first / N;
        p.rot = (a.first + a.rope_dim + N - 1) / N - p.rot0;
    } else {
        mode = a.first % N == 0 && hd % N == 0 ? kHalves : kScalar;
        const int w = mode == kHalves ? N : 1;
        p.half = hd * size;
        p.cols = (a.dim - hd) / w;
        p.rot0 = a.first / w;
        p.rot = hd / w;
    }
    // With few tokens a token's heads are spread over CTAs of one pass each, with many over CTAs of at most eight passes: each
    // forms the angles anew, but the tail is short.
    const int rp = p.cols < kT ? kT / p.cols : 1, heads = p.part[0].heads + p.part[1].heads + p.part[2].heads;
    const int sms = sm_count() > 0 ? sm_count() : 152, each = a.tokens < 4 * sms ? rp : 2 * kInFlight * rp;
    p.split = (heads + each - 1) / each;
    auto kern = mode == kPairs ? rope_kernel<E, kPairs> : mode == kHalves ? rope_kernel<E, kHalves> : rope_kernel<E, kScalar>;
    count_launch();
    return launch_k(kern, dim3(static_cast<unsigned>(a.tokens) * p.split), dim3(kT), 0, st, true, p) == cudaSuccess ? DSV4_OK
                                                                                                                    : DSV4_ERR_LAUNCH;
}

// f_j of the header's definition.
void frequencies(const dsv4_rope_args& a, double* freq) {
    constexpr double kPi2 = 6.283185307179586;
    const int n = a.rope_dim / 2;
    double lo = 0.0, hi = 0.0;
    if (a.scaling == DSV4_ROPE_BY_INDEX) {
        auto at = [&](double beta) { return a.rope_dim * std::log(a.original_len / (beta * kPi2)) / (2.0 * std::log(a.rope_theta)); };
        lo = std::fmax(std::floor(at(a.beta_fast)), 0.0);
        hi = std::fmin(std::ceil(at(a.beta_slow)), a.rope_dim - 1.0);
    }
    for (int j = 0; j < n; ++j) {
        const double f = std::pow(a.rope_theta, -2.0 * j / a.rope_dim);
        double keep = 1.0;
        if (a.scaling == DSV4_ROPE_LINEAR) keep = 0.0;
        if (a.scaling == DSV4_ROPE_BY_TURNS) keep = (a.original_len * f / kPi2 - a.beta_slow) / (a.beta_fast - a.beta_slow);
        if (a.scaling == DSV4_ROPE_BY_INDEX) keep = 1.0 - (j - lo) / (hi > lo ? hi - lo : 0.001);
        keep = std::fmin(std::fmax(keep, 0.0), 1.0);
        freq[j] = a.scaling == DSV4_ROPE_PLAIN ? f : f / a.factor * (1.0 - keep) + f * keep;
    }
}

}  // namespace

int launch_rope(const dsv4_rope_args& a, cudaStream_t st) {
    if (a.tokens == 0 || a.heads + a.kv_heads == 0) return DSV4_OK;
    RopeParams p{};
    p.slots = a.kv_heads ? a.slots : nullptr;
    p.pos = a.pos;
    p.n_slots = static_cast<long long>(a.num_pages) * a.page_size;
    p.tokens = a.tokens;
    p.first = a.first;
    p.pairs = a.rope_dim / 2;
    p.magnitude = static_cast<float>(a.magnitude);
    p.sign = a.inverse ? -1.f : 1.f;
    frequencies(a, p.freq);
    if (a.dtype == DSV4_FP32) return run<float>(a, p, st);
    if (a.dtype == DSV4_FP16) return run<__half>(a, p, st);
    return run<__nv_bfloat16>(a, p, st);
}

}  // namespace dsv4
