// Block tables and slot maps from the requests' lengths (ft_kv_plan).
//
// Three prefix sums over the requests: token rows, pages that are lacked, pages
// that come back.  With them every table entry, slot and free-list entry is found
// on its own: the stack V = free list ++ returned pages is never built, its i-th
// entry is read where it stands, so all workgroups work from the call's inputs.  Each
// workgroup computes the sums for itself (some 4096 lengths, L2-resident) and
// takes a share of the rows; the one that arrives last writes what may alias an
// input (kv_len, counts), when nobody reads those any more.  Latency bounds it.
#include "kv.h"
#include "resident.h"

namespace ftmoe {
namespace {

constexpr int kThreads = 1024;
constexpr int kPer = kv::kMaxRequests / kThreads;      // requests of a thread
constexpr int kRowsPerGroup = 4096;                    // token rows or page moves of a workgroup

// Exclusive prefix sums over the workgroup of each thread's own sum.
__device__ __forceinline__ int block_scan(int v, int* lds, int* total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int x = v;
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
        const int y = __shfl_up(x, m);
        if (lane >= m) x += y;
    }
    __syncthreads();                                   // (lds may still be read from the scan before)
    if (lane == 63) lds[wave] = x;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) {
        const int s = lds[w];
        if (w < wave) before += s;
        all += s;
    }
    *total = all;
    return before + x - v;
}

// Last index i of the non-decreasing p[0..n-1] with p[i] <= v (p[0] <= v).
__device__ __forceinline__ int last_at_most(const int* p, int n, int v) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p[mid] <= v) lo = mid;
        else hi = mid;
    }
    return lo;
}

struct PlanArgs {
    ft_kv_batch b;
    uint32_t* counter;
    int page_shift;
};

__global__ void __launch_bounds__(kThreads) plan_kernel(PlanArgs a) {
    const ft_kv_batch& c = a.b;
    __shared__ int first[kv::kMaxRequests + 1];        // token row of each request
    __shared__ int lack[kv::kMaxRequests + 1];         // pages lacked before it
    __shared__ int back[kv::kMaxRequests + 1];         // pages returned before it
    __shared__ uint8_t served[kv::kMaxRequests];
    __shared__ int scan_lds[kThreads / 64];
    __shared__ uint32_t flag;
    const int B = c.requests, tid = threadIdx.x, P = 1 << a.page_shift, room = c.width << a.page_shift;
    const int b0 = tid * kPer;
    auto context = [&](int b) { const int v = c.context[b]; return v < 0 ? 0 : v > room ? room : v; };
    auto pages_of = [&](int n) { return (n + P - 1) >> a.page_shift; };
    const int free_in = *c.free_count, F = free_in < 0 ? 0 : free_in > c.pages ? c.pages : free_in;

    int ctx[kPer], n[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const bool on = b0 + i < B;
        ctx[i] = on ? context(b0 + i) : 0;
        n[i] = on ? c.add[b0 + i] : 0;
        n[i] = n[i] > c.tokens ? c.tokens + 1 : n[i];  // (one more than fits: the sums stay within 32 bits)
        sum += n[i] > 0 ? n[i] : 0;
    }
    int all, at = block_scan(sum, scan_lds, &all);
    int want[kPer], returned[kPer], wants = 0, returns = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int m = n[i] > 0 ? n[i] : 0;
        const bool fits = (c.row_tokens ? m <= c.row_tokens : at + m <= c.tokens) && m <= room - ctx[i];
        const int have = pages_of(ctx[i]);
        want[i] = !fits || n[i] < 0 ? -1 : pages_of(ctx[i] + m) - have;     // -1: not to be served
        returned[i] = n[i] < 0 ? have : 0;
        wants += want[i] > 0 ? want[i] : 0;
        returns += returned[i];
        if (b0 + i <= B) first[b0 + i] = c.row_tokens ? (b0 + i) * c.row_tokens : at < c.tokens ? at : c.tokens;
        at += m;
    }
    int R, unused;
    int w = block_scan(wants, scan_lds, &unused), r = block_scan(returns, scan_lds, &R);
    int taken = 0, placed = 0, refused = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (b0 + i <= B) {
            lack[b0 + i] = w;
            back[b0 + i] = r;
        }
        if (b0 + i < B) {
            const bool ok = want[i] == 0 || (want[i] > 0 && w + want[i] <= F + R);
            served[b0 + i] = ok;
            taken += ok ? want[i] : 0;
            placed += ok ? n[i] : 0;
            refused += !ok && n[i] > 0;
        }
        w += want[i] > 0 ? want[i] : 0;
        r += returned[i];
    }
    if (B == kv::kMaxRequests && tid == kThreads - 1) {
        first[B] = c.row_tokens ? B * c.row_tokens : at < c.tokens ? at : c.tokens;
        lack[B] = w;
        back[B] = r;
    }
    int total_taken, total_placed, total_refused;
    block_scan(taken, scan_lds, &total_taken);
    block_scan(placed, scan_lds, &total_placed);
    block_scan(refused, scan_lds, &total_refused);
    __syncthreads();

    // entry i of the stack; i < F + R
    auto returned_page = [&](int i) {
        const int b = last_at_most(back, B, i);
        return c.table[(int64_t)b * c.width + (i - back[b])];
    };
    auto stack = [&](int i) { return i < F ? c.free_pages[i] : returned_page(i - F); };
    const int top = F + R - 1, stride = gridDim.x * kThreads, self = blockIdx.x * kThreads + tid;

    for (int t = self; t < c.tokens; t += stride) {
        int b = c.row_tokens ? t / c.row_tokens : t < first[B] ? last_at_most(first, B + 1, t) : B;
        int pos = -1, slot = -1;
        if (b < B && served[b]) {
            const int k = t - first[b], cb = context(b);
            if (k < c.add[b]) {
                pos = cb + k;
                const int j = pos >> a.page_shift, have = pages_of(cb);
                const int page = j < have ? c.table[(int64_t)b * c.width + j] : stack(top - (lack[b] + j - have));
                if (page >= 0 && page < c.pages) slot = (page << a.page_shift) | (pos & (P - 1));
            }
        }
        c.pos[t] = pos;
        c.slot[t] = slot;
    }
    for (int i = self; i < total_taken; i += stride) {
        const int b = last_at_most(lack, B, i);
        c.table[(int64_t)b * c.width + pages_of(context(b)) + (i - lack[b])] = stack(top - i);
    }
    // returned pages that nobody took: the free list grows (never past its `pages` entries, whatever a
    // table that names pages twice returns)
    const int left = min(F + R - total_taken, c.pages);
    for (int i = F + self; i < left; i += stride) c.free_pages[i] = returned_page(i - F);

    if (gridDim.x > 1 && !rs::last_arrival(a.counter, gridDim.x, &flag)) return;
    __syncthreads();
    for (int b = tid; b < B; b += kThreads) {
        const int cb = context(b), m = c.add[b];
        c.kv_len[b] = m < 0 ? 0 : served[b] ? cb + m : cb;
    }
    for (int b = tid; b <= B; b += kThreads) c.start[b] = first[b];
    if (tid == 0) {
        c.counts[0] = total_placed;
        c.counts[1] = total_taken;
        c.counts[2] = left;
        c.counts[3] = total_refused;
    }
}

}  // namespace

hipError_t launch_kv_plan(const ft_kv_batch& b, ft_workspace* ws, hipStream_t st) {
    PlanArgs a;
    a.b = b;
    a.counter = reinterpret_cast<uint32_t*>(ws->mem);
    a.page_shift = __builtin_ctz(b.page_tokens);
    const int groups = (b.tokens + b.requests + kRowsPerGroup - 1) / kRowsPerGroup;
    return launch(plan_kernel, dim3(groups), dim3(kThreads), 0, st, a);
}

}  // namespace ftmoe
