// A whole mixture-of-experts layer for a few tokens over resident records:
//
//   z = x Wr (fp64), ids = top-k of z, w = softmax over the chosen k,
//   y[t] = base[t] + sum_j w[t, j] FFN_{ids[t, j]}(x[t]),
//   FFN(x) = (silu(x Wg) * (x Wu)) Wd.
//
// The experts' records are read once each from where they lie (E records,
// `stride` bytes apart); no control step, no planner and no host branch takes
// part.  The router picks k of the layer's experts per token ("Making Large
// MoE Models Practical on a Single Machine", section 1); the expert FFN reads
// a complete layer-expert record ("The Expert Cache That Follows the Router",
// section "One logical expert, two physical levels of memory").
#include "resident.h"

namespace ftmoe {
namespace {

using namespace rs;

// ---- routing ----------------------------------------------------------------------

constexpr int kRouteThreads = 256;
constexpr int kRouteTokens = 8;           // tokens of one routing workgroup
constexpr int kRouteRows = 64;            // router rows of one slice
constexpr int kRouteMaxSlices = 64;

// Slices of the hidden size: each is kRouteRows rows or more, so that the
// partial logits (one fp64 per slice, token and expert) stay small.
inline int route_slices(int d) {
    const int s = (d + kRouteRows - 1) / kRouteRows;
    return s < kRouteMaxSlices ? s : kRouteMaxSlices;
}

struct RouteArgs {
    const uint16_t* x;
    const uint16_t* wr;
    int T, d, E, k, slices;
    double* part;          // [slices][T][E]
    uint32_t* counters;    // one per token group
    int32_t* ids;
    float* w;
};

__device__ __forceinline__ double bf16_f64(uint32_t u) { return (double)__uint_as_float(u << 16); }

// Workgroup (slice, group of 8 tokens): the slice's part of every logit of its
// tokens, products exact and sums in fp64.  A thread takes VE experts of the
// rows rs, rs + RPI, ... of the slice; the row groups are added in order.  The
// group's last workgroup adds the slices in order, takes each token's k
// largest logits by rank (an expert's rank is the number of experts before
// it: a larger logit, or an equal one of a lower index) and their softmax.
// A NaN logit counts as minus infinity in the order, so every rank is taken
// exactly once and every id is a valid expert.
template <int VE>
__global__ void __launch_bounds__(kRouteThreads) layer_route_kernel(RouteArgs a) {
    __shared__ double red[kRouteThreads * VE];
    __shared__ double z[kMaxRouteExperts];
    __shared__ double zsel[kMaxTopK];
    __shared__ int esel[kMaxTopK];
    __shared__ uint32_t flag;
    const int tid = threadIdx.x;
    const int slice = blockIdx.x, t0 = blockIdx.y * kRouteTokens;
    const int nt = min(kRouteTokens, a.T - t0);
    const int ncg = (a.E + VE - 1) / VE;          // expert groups (VE divides E)
    const int rpi = kRouteThreads / ncg;
    const int cg = tid % ncg, rsub = tid / ncg;
    const int span = (a.d + a.slices - 1) / a.slices;
    const int r0 = slice * span, r1 = min(a.d, r0 + span);

    double acc[kRouteTokens][VE];
#pragma unroll
    for (int t = 0; t < kRouteTokens; ++t)
#pragma unroll
        for (int j = 0; j < VE; ++j) acc[t][j] = 0.0;
    if (rsub < rpi) {
#pragma unroll 2
        for (int r = r0 + rsub; r < r1; r += rpi) {
            double wv[VE];
            if constexpr (VE == 8) {
                const u32x4_t v = *reinterpret_cast<const u32x4_t*>(a.wr + (int64_t)r * a.E + cg * 8);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    wv[2 * j] = (double)bf16lo(v[j]);
                    wv[2 * j + 1] = (double)bf16hi(v[j]);
                }
            } else {
                wv[0] = bf16_f64(a.wr[(int64_t)r * a.E + cg]);
            }
#pragma unroll
            for (int t = 0; t < kRouteTokens; ++t)
                if (t < nt) {
                    const double xv = bf16_f64(a.x[(int64_t)(t0 + t) * a.d + r]);
#pragma unroll
                    for (int j = 0; j < VE; ++j) acc[t][j] = fma(xv, wv[j], acc[t][j]);
                }
        }
    }
    for (int t = 0; t < nt; ++t) {
        __syncthreads();
        double mine[VE];
#pragma unroll
        for (int tt = 0; tt < kRouteTokens; ++tt)
            if (tt == t)
#pragma unroll
                for (int j = 0; j < VE; ++j) mine[j] = acc[tt][j];
        if (rsub < rpi)
#pragma unroll
            for (int j = 0; j < VE; ++j) red[rsub * a.E + cg * VE + j] = mine[j];
        __syncthreads();
        for (int e = tid; e < a.E; e += kRouteThreads) {
            double s = 0.0;
            for (int q = 0; q < rpi; ++q) s += red[q * a.E + e];
            put_agent(a.part + ((int64_t)slice * a.T + t0 + t) * a.E + e, s);
        }
    }
    if (!last_arrival(a.counters + blockIdx.y, a.slices, &flag)) return;

    for (int t = 0; t < nt; ++t) {
        if (tid < a.E) {
            double s = 0.0;
            const double* p = a.part + (int64_t)(t0 + t) * a.E + tid;
#pragma unroll 16
            for (int q = 0; q < a.slices; ++q) s += get_agent(p + (int64_t)q * a.T * a.E);
            z[tid] = s == s ? s : -INFINITY;
            red[tid] = s;
        }
        __syncthreads();
        if (tid < a.E) {
            const double mz = z[tid];
            int rank = 0;
            for (int e = 0; e < a.E; ++e) {
                const double o = z[e];
                rank += (o > mz || (o == mz && e < tid)) ? 1 : 0;
            }
            if (rank < a.k) {
                esel[rank] = tid;
                zsel[rank] = red[tid];
            }
        }
        __syncthreads();
        if (tid < a.k) {
            double s = 0.0;
            for (int r = 0; r < a.k; ++r) s += exp(zsel[r] - zsel[0]);
            a.ids[(int64_t)(t0 + t) * a.k + tid] = esel[tid];
            a.w[(int64_t)(t0 + t) * a.k + tid] = (float)(exp(zsel[tid] - zsel[0]) / s);
        }
        __syncthreads();
    }
}

// ---- the routed experts --------------------------------------------------------------

constexpr int kMaxRoutes = kMaxLayerTokens * kMaxTopK;       // 1024

struct ExpertArgs {
    const uint16_t* x;
    const uint8_t* rec;
    int64_t stride, off_gate, off_up, off_down, off_sg, off_su, off_sd;
    const int32_t* ids;
    const float* w;
    const uint16_t* base;
    uint16_t* y;
    uint16_t* hhi;         // [T k][f] h as two bf16 planes
    uint16_t* hlo;
    float* part;           // [splits][T][d] (splits > 1)
    uint32_t* counters;    // one per row panel of WdT
    int T, E, k, d, f, splits;
};

// The call's routes grouped by expert, in LDS.  A token names an expert at most
// once, so an expert's tokens are a 64-bit mask, and its routes lie in token
// order: every workgroup finds the same tiles.
struct Groups {
    unsigned long long mask[kMaxRouteExperts];   // tokens routed to the expert
    int start[kMaxRouteExperts];                 // first of its routes in `route`
    int active[kMaxRouteExperts];                // active experts, ascending
    int tile0[kMaxRouteExperts + 1];             // first tile of an active expert
    int n_active, n_tiles;
    uint16_t route[kMaxRoutes];                  // routes t k + j by expert
};

// Every thread of the workgroup calls it.
__device__ __forceinline__ void group_routes(Groups& g, const int32_t* ids, int R, int E, int k) {
    constexpr int PT = kMaxRoutes / kThreads;
    const int tid = threadIdx.x, lane = tid & 63;
    for (int e = tid; e < E; e += kThreads) g.mask[e] = 0;
    __syncthreads();
    int id[PT], tok[PT];
#pragma unroll
    for (int i = 0; i < PT; ++i) {
        const int r = tid + i * kThreads;
        id[i] = tok[i] = 0;
        if (r < R) {
            id[i] = ids[r];
            tok[i] = r / k;
            atomicOr(&g.mask[id[i]], 1ull << tok[i]);
        }
    }
    __syncthreads();
    if (tid < 64) {
        int base = 0, act = 0, tiles = 0;
        for (int e0 = 0; e0 < E; e0 += 64) {
            const int e = e0 + lane;
            const int c = e < E ? __popcll(g.mask[e]) : 0;
            const int tl = (c + kTile - 1) / kTile;
            int sc = c, st = tl;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int a0 = __shfl_up(sc, o, 64), b0 = __shfl_up(st, o, 64);
                if (lane >= o) {
                    sc += a0;
                    st += b0;
                }
            }
            const uint64_t m = __ballot(c > 0);
            if (c > 0) {
                const int r = act + __popcll(m & ((1ull << lane) - 1));
                g.start[e] = base + sc - c;
                g.active[r] = e;
                g.tile0[r] = tiles + st - tl;
            }
            base += __shfl(sc, 63, 64);
            tiles += __shfl(st, 63, 64);
            act += __popcll(m);
        }
        if (lane == 0) {
            g.n_active = act;
            g.n_tiles = tiles;
            g.tile0[act] = tiles;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PT; ++i) {
        const int r = tid + i * kThreads;
        if (r < R) g.route[g.start[id[i]] + __popcll(g.mask[id[i]] & ((1ull << tok[i]) - 1))] = (uint16_t)r;
    }
    __syncthreads();
}

// Gate/up and SwiGLU: workgroups take items (tile of at most 32 routes of one
// expert, 32 neurons); the waves split K = d.
template <int FMT>
__global__ void __launch_bounds__(kThreads, 2) layer_gateup_kernel(ExpertArgs a) {
    extern __shared__ __attribute__((aligned(16))) float red[];
    __shared__ Groups g;
    const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
    group_routes(g, a.ids, a.T * a.k, a.E, a.k);
    const int panels = a.f >> 5, items = g.n_tiles * panels;
    const int units = a.d / kUnit;
    const int u0 = wid * units / kWaves, u1 = (wid + 1) * units / kWaves;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int tile = item / panels, p = item - tile * panels;
        // the tile's expert: the last active one whose first tile is not past it
        int lo = 0, hi = g.n_active;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (g.tile0[mid] <= tile) lo = mid;
            else hi = mid;
        }
        const int e = g.active[lo];
        const int first = g.start[e] + (tile - g.tile0[lo]) * kTile;
        const int nt = min(kTile, g.start[e] + (int)__popcll(g.mask[e]) - first);
        const uint8_t* rec = a.rec + (int64_t)e * a.stride;
        const PanelRef pg = panel_ref<FMT>(rec + a.off_gate, rec + a.off_sg, a.d, p);
        const PanelRef pu = panel_ref<FMT>(rec + a.off_up, rec + a.off_su, a.d, p);
        // lanes past the tile's routes repeat its last one: their columns are not stored
        const uint16_t* xrow = a.x + (int64_t)(g.route[first + min(lane & 31, nt - 1)] / a.k) * a.d;

        f32x16_t ag[1] = {zero16()}, au[1] = {zero16()};
        WUnit<FMT> wg[2], wu[2];
        XUnit xu[2];
        auto load = [&](int b, int u) {
            load_unit<FMT>(wg[b], pg, u, lane);
            load_unit<FMT>(wu[b], pu, u, lane);
            load_x<FMT>(xu[b], xrow, u, lane);
        };
        auto mma = [&](int b) {
            const XUnit* const xs[1] = {&xu[b]};
            mma_unit<FMT, 1>(ag, wg[b], xs);
            mma_unit<FMT, 1>(au, wu[b], xs);
        };
        if (u0 < u1) load(0, u0);
        for (int u = u0; u < u1; u += 2) {
            if (u + 1 < u1) load(1, u + 1);
            mma(0);
            if (u + 1 < u1) {
                if (u + 2 < u1) load(0, u + 2);
                mma(1);
            }
        }
        // gate, then up, through the same LDS: a thread sums the waves of its (token, neuron) places
        constexpr int PT = kTile * 32 / kThreads;
        float gs[PT], us[PT];
        put_acc(red, ag[0], wid, nt, lane);
        __syncthreads();
        sum_waves(gs, red, nt, tid);
        __syncthreads();
        put_acc(red, au[0], wid, nt, lane);
        __syncthreads();
        sum_waves(us, red, nt, tid);
#pragma unroll
        for (int i = 0; i < PT; ++i) {
            const int t = (tid + i * kThreads) >> 5, n = tid & 31;
            if (t >= nt) break;
            // h in 16 significant bits: its rounding stays far below that of y
            uint16_t h, l;
            split_bf16(silu(gs[i]) * us[i], h, l);
            const int64_t o = (int64_t)g.route[first + t] * a.f + p * 32 + n;
            a.hhi[o] = h;
            a.hlo[o] = l;
        }
        __syncthreads();
    }
}

// Down and combine: workgroup (row panel of WdT, split).  The active experts'
// K = f units form one axis, divided evenly over the splits and their waves;
// a wave sums an expert's units for every token at once (lane = token; a lane
// whose token is not routed to the expert computes on another route's h and
// drops the result), then adds w times the sum to the tokens routed there.  The
// waves' sums are added in order, and with several splits the panel's last
// workgroup adds the splits in order, so y does not depend on timing.
template <int FMT, int NT>
__global__ void __launch_bounds__(kThreads, 2) layer_down_kernel(ExpertArgs a) {
    extern __shared__ __attribute__((aligned(16))) float red[];
    __shared__ Groups g;
    __shared__ uint32_t flag;
    const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
    group_routes(g, a.ids, a.T * a.k, a.E, a.k);
    const int na = g.n_active;

    const int p = blockIdx.x, split = blockIdx.y;
    const int uf = a.f / kUnit, units = na * uf;
    const int part = split * kWaves + wid, parts = a.splits * kWaves;
    const int u0 = (int)((int64_t)part * units / parts), u1 = (int)((int64_t)(part + 1) * units / parts);

    f32x16_t acc[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i] = zero16();
    for (int u = u0; u < u1;) {
        const int ai = u / uf, ue = min(u1, (ai + 1) * uf);
        const int e = g.active[ai];
        const uint8_t* rec = a.rec + (int64_t)e * a.stride;
        const PanelRef pd = panel_ref<FMT>(rec + a.off_down, rec + a.off_sd, a.f, p);
        const uint16_t *hrow[NT], *lrow[NT];
        float wt[NT];
        bool on[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int t = i * kTile + (lane & 31);
            const unsigned long long m = g.mask[e];
            on[i] = (m >> t) & 1;
            const int r = g.route[g.start[e] + (on[i] ? __popcll(m & ((1ull << t) - 1)) : 0)];
            wt[i] = on[i] ? a.w[r] : 0.0f;
            hrow[i] = a.hhi + (int64_t)r * a.f;
            lrow[i] = a.hlo + (int64_t)r * a.f;
        }
        f32x16_t sum[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) sum[i] = zero16();
        // two weight buffers; h in two as well where the registers hold them
        constexpr int HB = NT == 1 && FMT != FT_FMT_FP8_B128 ? 2 : 1;
        WUnit<FMT> wd[2];
        XUnit hu[HB][NT], lu[HB][NT];
        auto load_h = [&](int b, int uu) {
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                load_x<FMT>(hu[b][i], hrow[i], uu - ai * uf, lane);
                load_x<FMT>(lu[b][i], lrow[i], uu - ai * uf, lane);
            }
        };
        auto load = [&](int b, int uu) {
            load_unit<FMT>(wd[b], pd, uu - ai * uf, lane);
            if constexpr (HB == 2) load_h(b, uu);
        };
        auto mma = [&](int b, int uu) {
            if constexpr (HB == 1) load_h(0, uu);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                f32x16_t s2[1] = {sum[i]};
                const XUnit* const x0[1] = {&hu[b % HB][i]};
                const XUnit* const x1[1] = {&lu[b % HB][i]};
                mma_unit<FMT, 1>(s2, wd[b], x0);
                mma_unit<FMT, 1>(s2, wd[b], x1);
                sum[i] = s2[0];
            }
        };
        load(0, u);
        for (; u < ue; u += 2) {
            if (u + 1 < ue) load(1, u + 1);
            mma(0, u);
            if (u + 1 < ue) {
                if (u + 2 < ue) load(0, u + 2);
                mma(1, u + 1);
            }
        }
        u = ue;
        // the product of an unrouted token may be anything, infinities among it: selected away
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][v] = on[i] ? fmaf(wt[i], sum[i][v], acc[i][v]) : acc[i][v];
    }
    auto emit = [&](int t, int n, float v) {
        const int64_t o = (int64_t)t * a.d + p * 32 + n;
        if (a.base) v += __uint_as_float((uint32_t)a.base[o] << 16);
        a.y[o] = f32_to_bf16_rne(v);
    };
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int nt = min(kTile, a.T - i * kTile);
        float s[kTile * 32 / kThreads];
        if (i > 0) __syncthreads();
        put_acc(red, acc[i], wid, nt, lane);
        __syncthreads();
        sum_waves(s, red, nt, tid);
#pragma unroll
        for (int q = 0; q < kTile * 32 / kThreads; ++q) {
            const int t = (tid + q * kThreads) >> 5, n = tid & 31;
            if (t >= nt) break;
            if (a.splits == 1) emit(i * kTile + t, n, s[q]);
            else put_agent(a.part + ((int64_t)split * a.T + i * kTile + t) * a.d + p * 32 + n, s[q]);
        }
    }
    if (a.splits == 1 || !last_arrival(a.counters + p, a.splits, &flag)) return;
    for (int i = tid; i < a.T * 32; i += kThreads) {
        const int t = i >> 5, n = i & 31;
        float s = 0.0f;
        for (int q = 0; q < a.splits; ++q) s += get_agent(a.part + ((int64_t)q * a.T + t) * a.d + p * 32 + n);
        emit(t, n, s);
    }
}

// Workgroups over a row panel of WdT: enough for the card, and no more than
// leaves each wave a unit when every route has an expert of its own.
int down_splits(const ft_shape& s, int T) {
    const int panels = s.d_model / 32;
    const int64_t units = (int64_t)(T * s.top_k < s.experts ? T * s.top_k : s.experts) * (s.d_ff / kUnit);
    int64_t n = (256 + panels - 1) / panels;
    const int64_t most = (units + kWaves - 1) / kWaves;
    if (n > most) n = most;
    return n < 1 ? 1 : (int)n;
}

constexpr size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

struct LayerBuffers {
    size_t part, hhi, hlo, logits, total;
};
LayerBuffers layer_buffers(const ft_shape& s, int T) {
    LayerBuffers b;
    const size_t R = (size_t)T * s.top_k;
    b.logits = 0;
    b.hhi = align256((size_t)route_slices(s.d_model) * T * s.experts * sizeof(double));
    b.hlo = b.hhi + align256(R * s.d_ff * 2);
    b.part = b.hlo + align256(R * s.d_ff * 2);
    b.total = b.part + align256((size_t)down_splits(s, T) * T * s.d_model * sizeof(float));
    return b;
}

template <int FMT>
hipError_t launch_fmt(const ft_shape& s, const RouteArgs& r, const ExpertArgs& a, hipStream_t st) {
    const dim3 rg(r.slices, (r.T + kRouteTokens - 1) / kRouteTokens);
    if (r.E % 8 == 0) hipLaunchKernelGGL(layer_route_kernel<8>, rg, dim3(kRouteThreads), 0, st, r);
    else hipLaunchKernelGGL(layer_route_kernel<1>, rg, dim3(kRouteThreads), 0, st, r);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;

    const int R = a.T * a.k;
    const int tiles = (R < a.E ? R : a.E) + R / (kTile + 1);
    const int64_t items = (int64_t)tiles * (a.f / 32);
    const int nt = a.T < kTile ? a.T : kTile;
    const size_t lds = (size_t)kWaves * nt * kRedRow * sizeof(float);
    hipLaunchKernelGGL(layer_gateup_kernel<FMT>, dim3((unsigned)(items < 512 ? items : 512)), dim3(kThreads), lds, st, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;

    const dim3 dg(a.d / 32, a.splits);
    if (a.T <= kTile)
        hipLaunchKernelGGL((layer_down_kernel<FMT, 1>), dg, dim3(kThreads), lds, st, a);
    else
        hipLaunchKernelGGL((layer_down_kernel<FMT, 2>), dg, dim3(kThreads), lds, st, a);
    return hipGetLastError();
}

}  // namespace

size_t layer_workspace(const ft_shape& s, int T) { return layer_buffers(s, T).total; }

hipError_t launch_layer(const ft_shape& s, const LayerArgs& la, ft_workspace* ws, hipStream_t st) {
    const LayerBuffers b = layer_buffers(s, la.T);
    if (b.total > ws->bytes) return hipErrorInvalidValue;
    uint8_t* m = ws->mem + kCounterBytes;
    uint32_t* counters = reinterpret_cast<uint32_t*>(ws->mem);
    RouteArgs r;
    r.x = la.x;
    r.wr = la.wr;
    r.T = la.T;
    r.d = s.d_model;
    r.E = s.experts;
    r.k = s.top_k;
    r.slices = route_slices(s.d_model);
    r.part = reinterpret_cast<double*>(m + b.logits);
    r.counters = counters;
    r.ids = la.ids;
    r.w = la.w;
    ExpertArgs a;
    a.x = la.x;
    a.rec = la.rec;
    a.stride = la.stride;
    a.off_gate = la.rl.off_gate;
    a.off_up = la.rl.off_up;
    a.off_down = la.rl.off_down;
    a.off_sg = la.rl.off_sg;
    a.off_su = la.rl.off_su;
    a.off_sd = la.rl.off_sd;
    a.ids = la.ids;
    a.w = la.w;
    a.base = la.base;
    a.y = la.y;
    a.hhi = reinterpret_cast<uint16_t*>(m + b.hhi);
    a.hlo = reinterpret_cast<uint16_t*>(m + b.hlo);
    a.part = reinterpret_cast<float*>(m + b.part);
    a.counters = counters + kMaxLayerTokens;
    a.T = la.T;
    a.E = s.experts;
    a.k = s.top_k;
    a.d = s.d_model;
    a.f = s.d_ff;
    a.splits = down_splits(s, la.T);
    switch (s.fmt) {
        case FT_FMT_BF16: return launch_fmt<FT_FMT_BF16>(s, r, a, st);
        case FT_FMT_FP8_B128: return launch_fmt<FT_FMT_FP8_B128>(s, r, a, st);
        case FT_FMT_MXFP4_B32: return launch_fmt<FT_FMT_MXFP4_B32>(s, r, a, st);
    }
    return hipErrorInvalidValue;
}

}  // namespace ftmoe
