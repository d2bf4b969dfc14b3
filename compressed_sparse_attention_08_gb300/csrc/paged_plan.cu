// The bookkeeping of a serving step over the paged cache: offsets, positions and slots of the new
// tokens, pages taken from and given back to a stack, the tables' new entries (include/dsv4.h has the
// rules). The sources keep dense per-sequence buffers; the paged form is this library's own.
//
// All of it follows from three sums over the sequences: of tokens, of pages given back, of pages taken.
// One CTA forms them for the whole batch (at most 2,048 sequences, two per thread) and writes the state (lengths,
// pages held, the stack's height; in place too: it has read them all by then). What is left are three flat lists,
// tokens, pages given back and pages taken, whose entries find their sequence by bisection in the sums. A page
// that is given back and taken again is read where it stands in its table, so the lists need no order among
// them. Where they must be short the same CTA goes through them; else a second launch does, from the sums in the
// workspace, on the whole device.
// Latency bounds both: a launch, the lengths' loads, three sums, then a token's search, its sequence's numbers, its page and its
// slot, one after the other. Measured: 16 sequences of one token 3.9 us, 2,000 sequences with 44,483 tokens 11.3.
#include "internal.h"
#include "common.cuh"

namespace dsv4 {
namespace {

constexpr int kMaxBatch = 2048, kListT = 256;
constexpr int kFewTokens = 256, kFewPages = 4096;    // up to these one launch (see launch_paged_plan)

// What the lists need of a batch: sums (inclusive) and numbers per sequence.
struct PlanSums {
    int64_t next[kMaxBatch];             // position of the first new token
    int tok[kMaxBatch], back[kMaxBatch], take[kMaxBatch];
    int rows[kMaxBatch], held[kMaxBatch], from[kMaxBatch];   // before the step; the first page given back
    uint32_t off[kMaxBatch / 32];        // sequences that are not served
    int stack, count, taken, n_back;     // the stack's height with what is given back, and before; pages taken, given back
};

// Inclusive sums over a thread's numbers v[i] of places i * T + tid; v becomes the sums, the total is returned.
// `part`: scratch for PER * T / 32 numbers, not in use by another sum.
template <int T, int PER>
__device__ __forceinline__ long long block_sum(long long (&v)[PER], long long* part) {
    constexpr int W = T / 32, NP = PER * W, PL = (NP + 31) / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
#pragma unroll
        for (int w = 1; w < 32; w <<= 1) {
            const long long o = __shfl_up_sync(~0u, v[i], w);
            if (lane >= w) v[i] += o;
        }
        if (lane == 31) part[i * W + warp] = v[i];
    }
    __syncthreads();
    if (warp == 0) {                                     // the warps' totals, PL neighbours a lane
        long long x[PL], sum = 0;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            x[i] = lane * PL + i < NP ? part[lane * PL + i] : 0;
            sum += x[i];
        }
        long long incl = sum;
#pragma unroll
        for (int w = 1; w < 32; w <<= 1) {
            const long long o = __shfl_up_sync(~0u, incl, w);
            if (lane >= w) incl += o;
        }
        incl -= sum;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            incl += x[i];
            if (lane * PL + i < NP) part[lane * PL + i] = incl;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (i * W + warp > 0) v[i] += part[i * W + warp - 1];
    return part[NP - 1];
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

// The three lists, by threads `self`, `self` + `step`, ..; returns error bits. The sums tok, back and take are passed apart.
__device__ uint32_t plan_lists(const dsv4_paged_plan_args& p, const PlanSums& q, const int* tok, const int* back, const int* take, int self,
                               int step) {
    const int B = p.batch;
    const long long mp = p.max_pages;
    uint32_t err = 0;
    auto given_page = [&](int i) {                       // the i-th page given back
        const int s = find(back, B, i);
        return p.block_table[s * mp + q.from[s] + (i - (s ? back[s - 1] : 0))];
    };
    auto taken_page = [&](int k) {                       // the k-th page taken
        const int x = q.stack - 1 - k;
        return x < q.count ? p.free_pages[x] : given_page(x - q.count);
    };
    auto known = [&](int page) { return page >= 0 && page < p.num_pages; };
    const int tokens = B > 0 ? tok[B - 1] : 0, n_back = q.n_back, taken = q.taken;
    const long long all = static_cast<long long>(p.total_q) + taken + n_back;   // (one behind the other, so that no thread has all three)
    for (long long at = self; at < all; at += step) {
        if (at >= p.total_q) {
            const int k = static_cast<int>(at - p.total_q), i = k - taken;
            // (a page that is none moves as it stands, and is told of when it enters the stack, not only when a row meets it)
            const int page = i >= 0 ? given_page(i) : taken_page(k);
            if (!known(page)) err |= DSV4_EWORD_BAD_INDEX;
            if (i >= 0) {
                p.free_pages[q.count + i] = page;
            } else {
                const int s = find(take, B, k);
                p.block_table[s * mp + q.held[s] + (k - (s ? take[s - 1] : 0))] = page;
            }
            continue;
        }
        const int t = static_cast<int>(at);
        long long slot = -1, pos = 0;
        int s = -1;
        if (t < tokens) {
            s = find(tok, B, t);
            const int i = t - (s ? tok[s - 1] : 0), row = q.rows[s] + i, held = q.held[s];
            pos = q.next[s] + i;
            if (!(q.off[s >> 5] >> (s & 31) & 1)) {
                const int j = row / p.page_size;
                const int page = j < held ? p.block_table[s * mp + j] : taken_page((s ? take[s - 1] : 0) + j - held);
                if (known(page)) slot = static_cast<long long>(page) * p.page_size + (row - j * p.page_size);
                else err |= DSV4_EWORD_BAD_INDEX;
            }
        }
        p.slots[t] = slot;
        if (p.pos) p.pos[t] = pos;
        if (p.seq) p.seq[t] = s;
    }
    return err;
}

// Sums and state; with `lists`, the lists too. q: in the workspace.
template <int T, int PER>
__global__ void __launch_bounds__(T)
plan_kernel(const __grid_constant__ dsv4_paged_plan_args p, PlanSums* out, int lists, uint32_t* eword) {
    constexpr int MOST = T * PER;
    __shared__ int s_tok[MOST], s_back[MOST], s_take[MOST];
    __shared__ long long s_part[3][MOST / 32];
    __shared__ int s_taken;
    __shared__ uint32_t s_err;
    const int tid = threadIdx.x, lane = tid & 31, B = p.batch;
    pdl_trigger();
    pdl_wait();
    PlanSums& q = *out;
    if (tid == 0) { s_err = 0; s_taken = 0; }
    const int cap = p.free_cap, count0 = *p.free_count, count = min(max(count0, 0), cap);
    uint32_t err = count != count0 ? DSV4_EWORD_BAD_INDEX : 0;
    // this thread's sequences
    int n[PER], L[PER], h[PER], keep[PER], take[PER];
    long long sum[PER], next[PER];
    bool off[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int s = i * T + tid;
        n[i] = L[i] = h[i] = keep[i] = take[i] = 0;
        off[i] = false;
        next[i] = 0;
        if (s < B) {
            const int n0 = p.new_len ? p.new_len[s] : 0, L0 = p.kv_len[s], h0 = p.held[s], sh = p.shared ? p.shared[s] : 0;
            n[i] = min(max(n0, 0), p.total_q + 1);       // (more than fit is more than fit)
            L[i] = min(max(L0, 0), p.max_pages * p.page_size);
            h[i] = min(max(h0, 0), p.max_pages);
            keep[i] = min(max(sh, 0), h[i]);
            next[i] = p.next_pos ? p.next_pos[s] : L[i];
            if (n0 < 0 || L[i] != L0 || h[i] != h0 || sh < 0) err |= DSV4_EWORD_BAD_INDEX;
        }
        sum[i] = n[i];
    }
    block_sum<T, PER>(sum, s_part[0]);
    long long back[PER], ends[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int s = i * T + tid;
        const int want = static_cast<int>(static_cast<unsigned>(L[i] + n[i] + p.page_size - 1) / static_cast<unsigned>(p.page_size));
        off[i] = (n[i] > 0 && sum[i] > p.total_q) || want > p.max_pages;
        if (off[i]) err |= DSV4_EWORD_BAD_INDEX;
        keep[i] = off[i] ? h[i] : min(max(want, keep[i]), h[i]);
        back[i] = h[i] - keep[i];
        take[i] = off[i] ? 0 : max(want - h[i], 0);
        ends[i] = take[i];
        if (s < B) s_tok[s] = static_cast<int>(min(sum[i], static_cast<long long>(p.total_q)));
    }
    // (at most 2,048 x 2^26 pages: sums of counts that cannot be are cut to the stack's size)
    const long long all_back = block_sum<T, PER>(back, s_part[1]);
    block_sum<T, PER>(ends, s_part[2]);
    const int room = cap - count, n_back = static_cast<int>(min(all_back, static_cast<long long>(room)));
    if (all_back > room) err |= DSV4_EWORD_BAD_INDEX;
    const int stack = count + n_back;
    // Pages taken in all: the sum at the last sequence that is served and takes some. (Behind the first that is not
    // served no one takes any, and the sums of those before do not exceed the stack.)
    int top = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int s = i * T + tid;
        if (take[i] > 0 && ends[i] > stack) {
            off[i] = true;
            err |= DSV4_EWORD_NO_PAGES;
        }
        if (take[i] > 0 && !off[i]) top = static_cast<int>(ends[i]);
        if (s >= B) continue;
        s_back[s] = static_cast<int>(min(back[i], static_cast<long long>(n_back)));
        s_take[s] = static_cast<int>(min(ends[i], static_cast<long long>(cap) + 1));
        q.rows[s] = L[i];
        q.held[s] = h[i];
        q.from[s] = keep[i];
        q.next[s] = next[i];
    }
    top = __reduce_max_sync(~0u, top);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const uint32_t word = __ballot_sync(~0u, off[i]);
        if (lane == 0) q.off[(i * T + tid) / 32] = word;
        if (off[i]) n[i] = 0;                            // what is added to the state
    }
    if (lane == 0 && top) atomicMax(&s_taken, top);
    __syncthreads();
    const int taken = s_taken;
    if (tid == 0) {
        q.stack = stack;
        q.count = count;
        q.taken = taken;
        q.n_back = n_back;
    }
    if (lists) {
        __syncthreads();                                 // (the numbers in the workspace)
        err |= plan_lists(p, q, s_tok, s_back, s_take, tid, T);
    }
    err = __reduce_or_sync(~0u, err);
    if (lane == 0 && err) atomicOr(&s_err, err);
    __syncthreads();
    // the state (every thread has read it)
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int s = i * T + tid;
        if (s >= B) continue;
        p.cu_q[s + 1] = s_tok[s];
        p.kv_len_out[s] = L[i] + n[i];
        p.held_out[s] = off[i] ? h[i] : keep[i] + take[i];
        if (p.next_pos_out) p.next_pos_out[s] = next[i] + n[i];
        if (!lists) {
            q.tok[s] = s_tok[s];
            q.back[s] = s_back[s];
            q.take[s] = s_take[s];
        }
    }
    if (tid == 0) {
        p.cu_q[0] = 0;
        *p.free_count_out = stack - taken;
        *eword = s_err;
    }
}

__global__ void __launch_bounds__(kListT)
plan_lists_kernel(const __grid_constant__ dsv4_paged_plan_args p, const PlanSums* in, uint32_t* eword) {
    __shared__ int s_tok[kMaxBatch], s_back[kMaxBatch], s_take[kMaxBatch];
    const PlanSums& q = *in;
    pdl_trigger();
    pdl_wait();
    for (int s = threadIdx.x; s < p.batch; s += kListT) {
        s_tok[s] = q.tok[s];
        s_back[s] = q.back[s];
        s_take[s] = q.take[s];
    }
    __syncthreads();
    uint32_t err = plan_lists(p, q, s_tok, s_back, s_take, blockIdx.x * kListT + threadIdx.x, gridDim.x * kListT);
    err = __reduce_or_sync(~0u, err);
    if ((threadIdx.x & 31) == 0 && err) atomicOr(eword, err);
}

}  // namespace

size_t paged_plan_ws_bytes() { return sizeof(PlanSums); }

int launch_paged_plan(const dsv4_paged_plan_args& a, uint8_t* ws, uint32_t* eword, cudaStream_t st) {
    PlanSums* q = reinterpret_cast<PlanSums*>(ws);
    // One CTA goes through the lists in passes of its threads, 0.4 us each with tables in L2 and 0.7 without (a search, a table
    // entry, a store); a second launch costs 1.2 us whatever they hold. 16 sequences (back to back, one launch and two): 16
    // tokens 3.0 and 4.2 us, 256 4.3 and 4.5, 1,024 8.5 and 4.9. How many pages go back and forth only the device knows: as many
    // as the tables and the stack have room for, as when all requests end at once. One request of 8,192 pages took 53 us in one
    // CTA, 128 of them 6.9 ms; in two launches 10 and 22. So one launch is for what is short at its most (4,096 pages: 22 us).
    const long long tables = static_cast<long long>(a.batch) * a.max_pages, pages = tables < a.free_cap ? tables : a.free_cap;
    const int lists = a.total_q <= kFewTokens && pages <= kFewPages;
    count_launch();
    const cudaError_t e = a.batch <= 128 ? launch_k(plan_kernel<128, 1>, dim3(1), dim3(128), 0, st, true, a, q, lists, eword)
                                         : launch_k(plan_kernel<1024, 2>, dim3(1), dim3(1024), 0, st, true, a, q, lists, eword);
    if (e != cudaSuccess) return DSV4_ERR_LAUNCH;
    if (lists) return DSV4_OK;
    // (each CTA copies the sums first: 2,000 sequences of 44,483 tokens warm 11.1 us with four CTAs per SM, 10.5 with two, 10.8 with one)
    const int sms = sm_count() > 0 ? sm_count() : 152, most = 2 * sms;
    const long long need = (a.total_q + pages + kListT - 1) / kListT;
    count_launch();
    return launch_k(plan_lists_kernel, dim3(need < most ? static_cast<unsigned>(need) : most), dim3(kListT), 0, st, true, a, q, eword) == cudaSuccess
               ? DSV4_OK : DSV4_ERR_LAUNCH;
}

}  // namespace dsv4
