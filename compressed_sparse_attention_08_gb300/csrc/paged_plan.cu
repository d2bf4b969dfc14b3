// The bookkeeping of a serving step over the paged cache: offsets, positions and slots of the new
// tokens, pages taken from and given back to a stack, the tables' new entries (include/dsv4.h has the
// rules). The sources keep dense per-sequence buffers; the paged form is this library's own.
//
// All of it follows from three sums over the sequences: of tokens, of pages given back, of pages taken.
// Each CTA forms the sums of the whole batch itself (at most 2,048 sequences, four per thread), so the
// CTAs need nothing from one another, and then takes its share of three flat lists: tokens, pages
// given back, pages taken. An entry finds its sequence by bisection in the sums. A page that is given back and
// taken again is read where it stands in its table, so the lists need no order among them. The state
// (lengths, pages held, the stack's height) may be updated in place: the CTAs form one cluster, and its
// first writes the state after all have met at the cluster's barrier.
#include "internal.h"
#include "common.cuh"

namespace dsv4 {
namespace {

constexpr int kT = 512, kPer = 4, kMaxBatch = kT * kPer, kCluster = 8;

__device__ __forceinline__ void red_cluster_or(uint32_t addr, uint32_t v) {
    asm volatile("red.shared::cluster.or.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Inclusive sum over the block of a thread's four numbers; v becomes the sums, the total is returned.
__device__ __forceinline__ long long block_sum(long long (&v)[kPer], long long* part) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int i = 1; i < kPer; ++i) v[i] += v[i - 1];
    long long x = v[kPer - 1];
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) {
        const long long o = __shfl_up_sync(~0u, x, w);
        if (lane >= w) x += o;
    }
    __syncthreads();                                     // (part may still be read by the sum before)
    if (lane == 31) part[warp] = x;
    __syncthreads();
    long long before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kT / 32; ++w) {
        const long long p = part[w];
        before += w < warp ? p : 0;
        total += p;
    }
    const long long base = before + x - v[kPer - 1];
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] += base;
    return total;
}

// The first sequence whose sum ends past x (x is below the last sum).
__device__ __forceinline__ int find(const int* ends, int n, int x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (ends[mid] > x) hi = mid; else lo = mid + 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kT)
paged_plan_kernel(const __grid_constant__ dsv4_paged_plan_args p, uint32_t* eword) {
    __shared__ int s_tok[kMaxBatch], s_back[kMaxBatch], s_take[kMaxBatch];   // inclusive sums
    __shared__ uint32_t s_off[kMaxBatch / 32];                               // sequences that are not served
    __shared__ long long s_part[kT / 32];
    __shared__ int s_taken;
    __shared__ uint32_t s_err;
    const int tid = threadIdx.x, lane = tid & 31;
    const int rank = blockIdx.x, ctas = gridDim.x, B = p.batch;
    pdl_trigger();
    pdl_wait();
    if (tid == 0) { s_err = 0; s_taken = 0; }
    if (tid < kMaxBatch / 32) s_off[tid] = 0;
    if (ctas > 1) cluster_arrive();
    const int cap = p.free_cap;
    uint32_t err = 0;
    const int count0 = *p.free_count, count = min(max(count0, 0), cap);
    if (count != count0) err |= DSV4_EWORD_BAD_INDEX;
    // this thread's sequences
    int n[kPer], L[kPer], h[kPer], keep[kPer], take[kPer];
    long long sum[kPer];
    bool off[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int s = tid * kPer + i;
        n[i] = L[i] = h[i] = keep[i] = take[i] = 0;
        off[i] = false;
        if (s < B) {
            const int n0 = p.new_len ? p.new_len[s] : 0, L0 = p.kv_len[s], h0 = p.held[s], sh = p.shared ? p.shared[s] : 0;
            n[i] = max(n0, 0);
            L[i] = min(max(L0, 0), p.max_pages * p.page_size);
            h[i] = min(max(h0, 0), p.max_pages);
            keep[i] = min(max(sh, 0), h[i]);
            if (n0 < 0 || L[i] != L0 || h[i] != h0 || sh < 0) err |= DSV4_EWORD_BAD_INDEX;
        }
        sum[i] = n[i];
    }
    block_sum(sum, s_part);
    long long back[kPer], want[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int s = tid * kPer + i;
        want[i] = (static_cast<long long>(L[i]) + n[i] + p.page_size - 1) / p.page_size;
        off[i] = (n[i] > 0 && sum[i] > p.total_q) || want[i] > p.max_pages;
        if (off[i]) err |= DSV4_EWORD_BAD_INDEX;
        keep[i] = off[i] ? h[i] : static_cast<int>(min(max(want[i], static_cast<long long>(keep[i])), static_cast<long long>(h[i])));
        back[i] = h[i] - keep[i];
        take[i] = off[i] ? 0 : static_cast<int>(max(want[i] - h[i], 0ll));
        if (s < B) s_tok[s] = static_cast<int>(min(sum[i], static_cast<long long>(p.total_q)));
    }
    // (at most 2,048 x 2^26 pages: the sums of counts that cannot be are cut to the stack's size)
    long long ends[kPer];
    const long long all_back = block_sum(back, s_part);
#pragma unroll
    for (int i = 0; i < kPer; ++i) ends[i] = take[i];
    block_sum(ends, s_part);
    const int room = cap - count, n_back = static_cast<int>(min(all_back, static_cast<long long>(room)));
    if (all_back > room) err |= DSV4_EWORD_BAD_INDEX;
    const int stack = count + n_back;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int s = tid * kPer + i;
        if (s >= B) continue;
        if (take[i] > 0 && ends[i] > stack) {
            off[i] = true;
            err |= DSV4_EWORD_NO_PAGES;
        }
        s_back[s] = static_cast<int>(min(back[i], static_cast<long long>(n_back)));
        s_take[s] = static_cast<int>(min(ends[i], static_cast<long long>(cap) + 1));
        if (off[i]) atomicOr(&s_off[s >> 5], 1u << (s & 31));
    }
    // Pages taken in all: the sum at the last sequence that is served and takes some. (Behind the first that is not
    // served no one takes any, and the sums of those before do not exceed the stack.)
    int top = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if (take[i] > 0 && !off[i]) top = static_cast<int>(ends[i]);
    top = __reduce_max_sync(~0u, top);
    if (lane == 0 && top) atomicMax(&s_taken, top);
    __syncthreads();
    const int taken = s_taken;
    const long long mp = p.max_pages;
    const int g0 = rank * kT + tid, step = ctas * kT;
    // Pages given back. (Where the stack has no room for all, the sums are cut and the first n_back are kept: from a
    // sequence's first on, so its place is counted from what it keeps.)
    auto back_page = [&](int i) {
        const int s = find(s_back, B, i);
        const int first = s ? s_back[s - 1] : 0;
        const int hs = min(max(p.held[s], 0), p.max_pages);
        const int sh = min(max(p.shared ? p.shared[s] : 0, 0), hs);
        const int Ls = min(max(p.kv_len[s], 0), p.max_pages * p.page_size), ns = max(p.new_len ? p.new_len[s] : 0, 0);
        const long long w = (static_cast<long long>(Ls) + ns + p.page_size - 1) / p.page_size;
        const int from = static_cast<int>(max(w, static_cast<long long>(sh)));
        return p.block_table[s * mp + from + (i - first)];
    };
    for (int i = g0; i < n_back; i += step) p.free_pages[count + i] = back_page(i);
    auto taken_page = [&](int k) {                       // the k-th page taken
        const int x = stack - 1 - k;
        return x < count ? p.free_pages[x] : back_page(x - count);
    };
    for (int k = g0; k < taken; k += step) {
        const int s = find(s_take, B, k);
        const int first = s ? s_take[s - 1] : 0;
        p.block_table[s * mp + min(max(p.held[s], 0), p.max_pages) + (k - first)] = taken_page(k);
    }
    const int tokens = B > 0 ? s_tok[B - 1] : 0;
    for (int t = g0; t < p.total_q; t += step) {
        long long slot = -1, pos = 0;
        int s = -1;
        if (t < tokens) {
            s = find(s_tok, B, t);
            const int i = t - (s ? s_tok[s - 1] : 0);
            const int Ls = min(max(p.kv_len[s], 0), p.max_pages * p.page_size);
            pos = (p.next_pos ? p.next_pos[s] : Ls) + i;
            if (!(s_off[s >> 5] >> (s & 31) & 1)) {
                const int row = Ls + i, j = row / p.page_size;
                const int hs = min(max(p.held[s], 0), p.max_pages);
                const int page = j < hs ? p.block_table[s * mp + j] : taken_page((s ? s_take[s - 1] : 0) + j - hs);
                if (page >= 0 && page < p.num_pages) slot = static_cast<long long>(page) * p.page_size + (row - j * p.page_size);
                else err |= DSV4_EWORD_BAD_INDEX;
            }
        }
        p.slots[t] = slot;
        if (p.pos) p.pos[t] = pos;
        if (p.seq) p.seq[t] = s;
    }
    __syncwarp();
    if (ctas > 1) cluster_wait();                        // (the first CTA's error bits are cleared)
    err = __reduce_or_sync(~0u, err);
    if (lane == 0 && err) {
        if (ctas > 1) red_cluster_or(cluster_map(&s_err, 0), err);
        else atomicOr(&s_err, err);
    }
    __syncwarp();
    // the state, once every CTA has read it
    if (ctas > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    if (rank != 0) return;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int s = tid * kPer + i;
        if (s >= B) continue;
        p.cu_q[s + 1] = s_tok[s];
        p.kv_len_out[s] = off[i] ? L[i] : L[i] + n[i];
        p.held_out[s] = off[i] ? h[i] : keep[i] + take[i];
        if (p.next_pos_out) p.next_pos_out[s] = p.next_pos[s] + (off[i] ? 0 : n[i]);
    }
    if (tid == 0) {
        p.cu_q[0] = 0;
        *p.free_count_out = stack - taken;
        *eword = s_err;
    }
}

}  // namespace

int launch_paged_plan(const dsv4_paged_plan_args& a, uint32_t* eword, cudaStream_t st) {
    // One CTA while its threads have a few tokens each; eight with more (the cluster's barriers cost
    // about as much as the tokens of one CTA then).
    const long long work = a.total_q;
    const unsigned ctas = work <= 4 * kT ? 1 : kCluster;
    count_launch();
    return launch_cluster_k(paged_plan_kernel, dim3(ctas), dim3(kT), 0, st, true, ctas, a, eword) == cudaSuccess ? DSV4_OK
                                                                                                                  : DSV4_ERR_LAUNCH;
}

}  // namespace dsv4
