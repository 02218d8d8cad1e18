// Block tables and slot maps from the requests' lengths (ft_kv_plan).
//
// Three prefix sums over the requests: token rows, pages that are lacked, pages
// that come back.  With them every table entry, slot and free-list entry is found
// on its own: the stack V = free list ++ returned pages is never built, its i-th
// entry is read where it stands, so all workgroups work from the call's inputs.  Each
// workgroup computes the sums for itself (some 4096 lengths, L2-resident) and
// takes a share of the rows; the one that arrives last writes what may alias an
// input (kv_len, counts), when nobody reads those any more.  Latency bounds it: 64
// requests of a decode step 4.4 us, 1,000 of 16,384 rows 7.8 us, 4,096 13.3; in
// place 0.5 to 0.7 us more.
#include "kv_device.h"
#include "resident.h"

namespace ftmoe {
namespace {

// N exclusive prefix sums over the workgroup, of each thread's own sums v; total: the workgroup's.
template <int THREADS, int N>
__device__ __forceinline__ void block_scan(int (&v)[N], int (&total)[N], int (*lds)[THREADS / 64]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i] = kv::wave_scan(v[i]);
        if constexpr (THREADS == 64) {
            total[i] = __builtin_amdgcn_readlane(x[i], 63);
            v[i] = x[i] - v[i];
        }
    }
    if constexpr (THREADS > 64) {
        __syncthreads();                               // (lds may still be read from the scan before)
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (lane == 63) lds[i][wave] = x[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            int before = 0, all = 0;
#pragma unroll
            for (int w = 0; w < THREADS / 64; ++w) {
                const int s = lds[i][w];
                if (w < wave) before += s;
                all += s;
            }
            total[i] = all;
            v[i] = before + x[i] - v[i];
        }
    }
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
    bool shared;                                       // kv_len or counts lies over an input
};

template <int THREADS, int PER>
__global__ void __launch_bounds__(THREADS) plan_kernel(PlanArgs a) {
    const ft_kv_batch& c = a.b;
    constexpr int kPer = PER, kMost = THREADS * kPer;  // requests of a thread, and of all
    constexpr bool kKept = PER < 4;                    // (LDS holds no more; 2 to 3% by fewer trips to the L2)
    __shared__ int first[kMost + 1];                   // token row of each request
    __shared__ int lack[kMost + 1];                    // pages lacked before it
    __shared__ int back[kMost + 1];                    // pages returned before it
    __shared__ uint8_t served[kMost];
    __shared__ int held[kKept ? kMost : 1], added[kKept ? kMost : 1];     // the clamped context, and add
    __shared__ int scan_lds[3][THREADS / 64];
    __shared__ uint32_t flag;
    const int B = c.requests, tid = threadIdx.x, P = 1 << a.page_shift, room = c.width << a.page_shift;
    const int b0 = tid * kPer;
    auto context = [&](int b) { const int v = c.context[b]; return v < 0 ? 0 : v > room ? room : v; };
    auto pages_of = [&](int n) { return (n + P - 1) >> a.page_shift; };
    const int free_in = *c.free_count, F = free_in < 0 ? 0 : free_in > c.pages ? c.pages : free_in;

    int ctx[kPer], n[kPer], sum[1] = {0}, all[1];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const bool on = b0 + i < B;
        ctx[i] = on ? context(b0 + i) : 0;
        n[i] = on ? c.add[b0 + i] : 0;
        if constexpr (kKept) {
            held[b0 + i] = ctx[i];
            added[b0 + i] = n[i];
        }
        n[i] = n[i] > c.tokens ? c.tokens + 1 : n[i];  // (one more than fits: the sums stay within 32 bits)
        sum[0] += n[i] > 0 ? n[i] : 0;
    }
    block_scan<THREADS>(sum, all, scan_lds);
    int at = sum[0], want[kPer], returned[kPer], pages[2] = {0, 0}, pages_all[2];     // lacked and returned
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int m = n[i] > 0 ? n[i] : 0;
        const bool fits = (c.row_tokens ? m <= c.row_tokens : at + m <= c.tokens) && m <= room - ctx[i];
        const int have = pages_of(ctx[i]);
        want[i] = !fits || n[i] < 0 ? -1 : pages_of(ctx[i] + m) - have;     // -1: not to be served
        returned[i] = n[i] < 0 ? have : 0;
        pages[0] += want[i] > 0 ? want[i] : 0;
        pages[1] += returned[i];
        if (b0 + i <= B) first[b0 + i] = c.row_tokens ? (b0 + i) * c.row_tokens : at < c.tokens ? at : c.tokens;
        at += m;
    }
    block_scan<THREADS>(pages, pages_all, scan_lds);
    const int R = pages_all[1];
    int w = pages[0], r = pages[1], count[3] = {0, 0, 0}, total[3];    // pages taken, tokens served, requests refused
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (b0 + i <= B) {
            lack[b0 + i] = w;
            back[b0 + i] = r;
        }
        if (b0 + i < B) {
            const bool ok = want[i] == 0 || (want[i] > 0 && w + want[i] <= F + R);
            served[b0 + i] = ok;
            count[0] += ok ? want[i] : 0;
            count[1] += ok ? n[i] : 0;
            count[2] += !ok && n[i] > 0;
        }
        w += want[i] > 0 ? want[i] : 0;
        r += returned[i];
    }
    if (B == kMost && tid == THREADS - 1) {
        first[B] = c.row_tokens ? B * c.row_tokens : at < c.tokens ? at : c.tokens;
        lack[B] = w;
        back[B] = r;
    }
    block_scan<THREADS>(count, total, scan_lds);
    __syncthreads();

    auto held_by = [&](int b) { return kKept ? held[b] : context(b); };
    auto added_to = [&](int b) { return kKept ? added[b] : c.add[b]; };
    // entry i of the stack; i < F + R
    auto returned_page = [&](int i) {
        const int b = last_at_most(back, B, i);
        return c.table[(int64_t)b * c.width + (i - back[b])];
    };
    auto stack = [&](int i) { return i < F ? c.free_pages[i] : returned_page(i - F); };
    const int top = F + R - 1, stride = gridDim.x * THREADS, self = blockIdx.x * THREADS + tid;

    for (int t = self; t < c.tokens; t += stride) {
        int b = c.row_tokens ? t / c.row_tokens : t < first[B] ? last_at_most(first, B + 1, t) : B;
        int pos = -1, slot = -1;
        if (b < B && served[b]) {
            const int k = t - first[b], cb = held_by(b);
            if (k < added_to(b)) {
                pos = cb + k;
                const int j = pos >> a.page_shift, have = pages_of(cb);
                const int page = j < have ? c.table[(int64_t)b * c.width + j] : stack(top - (lack[b] + j - have));
                if (page >= 0 && page < c.pages) slot = (page << a.page_shift) | (pos & (P - 1));
            }
        }
        c.pos[t] = pos;
        c.slot[t] = slot;
    }
    for (int i = self; i < total[0]; i += stride) {
        const int b = last_at_most(lack, B, i);
        c.table[(int64_t)b * c.width + pages_of(held_by(b)) + (i - lack[b])] = stack(top - i);
    }
    // returned pages that nobody took: the free list grows (never past its `pages` entries, whatever a
    // table that names pages twice returns)
    const int left = min(F + R - total[0], c.pages);
    for (int i = F + self; i < left; i += stride) c.free_pages[i] = returned_page(i - F);

    // What may lie over an input is written when nobody reads those any more: by the last workgroup to arrive.
    if (gridDim.x > 1 && (a.shared ? !rs::last_arrival(a.counter, gridDim.x, &flag) : blockIdx.x != 0)) return;
    __syncthreads();
    for (int b = tid; b < B; b += THREADS) {
        const int cb = held_by(b), m = added_to(b);
        c.kv_len[b] = m < 0 ? 0 : served[b] ? cb + m : cb;
    }
    for (int b = tid; b <= B; b += THREADS) c.start[b] = first[b];
    if (tid == 0) {
        c.counts[0] = total[1];
        c.counts[1] = total[0];
        c.counts[2] = left;
        c.counts[3] = total[2];
    }
}

template <int THREADS, int PER>
hipError_t go(const PlanArgs& a, hipStream_t st) {
    const int rows = a.b.tokens + a.b.requests;
    return launch(plan_kernel<THREADS, PER>, dim3((rows + THREADS - 1) / THREADS), dim3(THREADS), 0, st, a);
}

}  // namespace

// The smallest workgroup with a thread a request, for scans of few waves and rows over many compute units (with four
// requests a thread, in 1,024 threads: 1,000 requests of 16,384 rows 10.0 us, 8.5 so; 16 of 8,000 rows 7.2, 4.9; a wave
// of four each for 64 decode requests 6.4, 5.2; 2,000 requests take two each: 10.3, 11.7 with four; calls in a captured graph).  Of small ones at most
// 64, since arrivals at one counter queue: 20 requests of 60,000 rows in place 5.4 us, 14 in 938 workgroups of a wave.
constexpr int kMostGroups = 64;

hipError_t launch_kv_plan(const ft_kv_batch& b, ft_workspace* ws, hipStream_t st) {
    PlanArgs a;
    a.b = b;
    a.counter = reinterpret_cast<uint32_t*>(ws->mem);
    a.page_shift = __builtin_ctz(b.page_tokens);
    auto over = [](const int32_t* p, int64_t n, const int32_t* q, int64_t m) { return p < q + m && q < p + n; };
    a.shared = false;
    for (const int32_t* in : {b.context, b.add})
        a.shared |= over(b.kv_len, b.requests, in, b.requests) || over(b.counts, 4, in, b.requests);
    a.shared |= over(b.kv_len, b.requests, b.free_count, 1) || over(b.counts, 4, b.free_count, 1);
    const int rows = b.tokens + b.requests;
    if (b.requests <= 64 && rows <= 64 * kMostGroups) return go<64, 1>(a, st);
    if (b.requests <= 256 && rows <= 256 * kMostGroups) return go<256, 1>(a, st);
    if (b.requests <= 512) return go<512, 1>(a, st);
    if (b.requests <= 1024) return go<1024, 1>(a, st);
    if (b.requests <= 2048) return go<1024, 2>(a, st);
    return go<1024, kv::kMaxRequests / 1024>(a, st);
}

}  // namespace ftmoe
