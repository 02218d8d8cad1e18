// Projections with the low-rank adapters of many requests beside them:
//
//   y[t] = base[t] + x[t] W^T + s_a (x[t] A_a^T) B_a^T,   a = adapter[t],
//
// and a SwiGLU expert whose three projections carry adapters.  W is read
// once for all requests; an adapter's A [r x K] and B [n x r] are read once
// per 32 tokens that name it.  The first launch computes v = s_a x A_a^T
// (r <= 128 values per token), the second streams W and adds v B_a^T to its
// accumulators.  The expert FFN reads one complete record ("The Expert Cache
// That Follows the Router", section "One logical expert, two physical levels
// of memory").
#include "resident.h"

namespace ftmoe {
namespace {

using namespace rs;

// ---- the adapters of a tile of 32 tokens ------------------------------------------

// Calls body(i, a) for the distinct adapters a of a tile, in the order of
// their first token; `id` is the lane's token's adapter, -1 for none (lanes l
// and l + 32 hold the same token).  The loop is the same in every lane.
template <typename F>
__device__ __forceinline__ void each_adapter(int id, F&& body) {
    uint32_t left = (uint32_t)__ballot(id >= 0);
    for (int i = 0; left; ++i) {
        const int a = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
        body(i, a);
        left &= ~(uint32_t)__ballot(id == a);
    }
}

// The lane's token's adapter; ids outside the pool name none.
__device__ __forceinline__ int tile_adapter(const int32_t* adapter, int t0, int T, int count, int lane) {
    const int t = t0 + (lane & 31);
    const int id = t < T ? adapter[t] : -1;
    return (uint32_t)id < (uint32_t)count ? id : -1;
}

struct ShrinkArgs {
    LoraView lora[2];
    uint16_t* vhi[2];      // [T][R] v as two bf16 planes
    uint16_t* vlo[2];
    const int32_t* adapter;
    const uint16_t* xhi;
    const uint16_t* xlo;   // second plane of x (PL = 2)
    int T, K, panels;      // rank panels of 16 per projection
};

// Workgroup (tile of 32 tokens, stride over the tile's adapters, projection
// and 16 ranks): v for every token of the adapter; the waves split K.  Both
// operands are row-major: of 128 K a lane takes 32 consecutive ones, so the
// four lanes of a row use its 256 bytes.
template <int PL>
__global__ void __launch_bounds__(kThreads, 2) lora_shrink_kernel(ShrinkArgs s) {
    extern __shared__ __attribute__((aligned(16))) float red[];
    const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
    const int t0 = blockIdx.x * kTile, nt = min(kTile, s.T - t0);
    const int proj = blockIdx.z / s.panels, r0 = (blockIdx.z - proj * s.panels) * 16;
    const LoraView lo = s.lora[proj];
    const int R = lo.max_rank;
    if (r0 >= R) return;
    const int id = tile_adapter(s.adapter, t0, s.T, lo.count, lane);
    const int units = s.K / kUnit;
    const int u0 = wid * units / kWaves, u1 = (wid + 1) * units / kWaves;
    int64_t xo[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) xo[i] = (int64_t)(t0 + min(i * kCols + (lane & 15), nt - 1)) * s.K;
    const int nx = nt > kCols ? 2 : 1;
    each_adapter(id, [&](int i, int a) {
        if (i % (int)gridDim.y != (int)blockIdx.y) return;
        const int rank = min(max(lo.rank[a], 0), R);
        if (r0 >= rank) return;           // the expand reads v in steps of 16 up to the rank
        const uint16_t* arow = lo.a + ((int64_t)a * R + min(r0 + (lane & 15), rank - 1)) * s.K;
        f32x4_t acc[2] = {f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}, f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}};
        XUnit au[2], x[2][2][PL];
        auto load = [&](int b, int u) {
            load_x<FT_FMT_MXFP4_B32>(au[b], arow, u, lane);
#pragma unroll
            for (int q = 0; q < 2; ++q)
                if (q < nx) {
                    load_x<FT_FMT_MXFP4_B32>(x[b][q][0], s.xhi + xo[q], u, lane);
                    if constexpr (PL == 2) load_x<FT_FMT_MXFP4_B32>(x[b][q][PL - 1], s.xlo + xo[q], u, lane);
                }
        };
        auto step = [&](int b) {
#pragma unroll
            for (int v = 0; v < 4; ++v)
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    if (q < nx)
#pragma unroll
                        for (int p = 0; p < PL; ++p)
                            acc[q] = mma(__builtin_bit_cast(bf16x8_t, au[b].v[v]), x[b][q][p].v[v], acc[q]);
        };
        if (u0 < u1) load(0, u0);
        for (int u = u0; u < u1; u += 2) {
            if (u + 1 < u1) load(1, u + 1);
            step(0);
            if (u + 1 < u1) {
                if (u + 2 < u1) load(0, u + 2);
                step(1);
            }
        }
        // 16 ranks of up to 32 tokens: one place per thread
        __syncthreads();
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int m = q * kCols + (lane & 15);
            if (m < nt) *reinterpret_cast<f32x4_t*>(red + (wid * nt + m) * 20 + 4 * (lane >> 4)) = acc[q];
        }
        __syncthreads();
        const int t = tid >> 4, n = r0 + (tid & 15);
        if (t < nt && s.adapter[t0 + t] == a) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) v += red[(w * nt + t) * 20 + (tid & 15)];
            // v in 16 significant bits; zero past the adapter's rank
            uint16_t h, l;
            split_bf16(n < rank ? lo.scale[a] * v : 0.0f, h, l);
            const int64_t o = (int64_t)(t0 + t) * R + n;
            s.vhi[proj][o] = h;
            s.vlo[proj][o] = l;
        }
    });
}

// acc += v B_a^T for row panel p of B [n x R] and the 16 tokens `id` (the
// lane's column's adapter) and `t` (its token); the other tokens' products
// are selected away (an adapter's infinities and NaN stay with its own
// requests), and ranks past the adapter's own are masked out of B, whatever
// the pool holds there.
__device__ __forceinline__ void expand(Acc& acc, const LoraView& lo, const uint16_t* vhi, const uint16_t* vlo, int n,
                                       int p, int a, int id, int t, int lane) {
    if (__ballot(id == a) == 0) return;
    const int R = lo.max_rank, g = lane >> 4;
    const int rank = min(max(lo.rank[a], 0), R);
    const uint16_t* brow = lo.b + ((int64_t)a * n + p * 32 + (lane & 15)) * R + g * 8;
    const int64_t vo = (int64_t)t * R + g * 8;
    const u32x4_t none = u32x4_t{0u, 0u, 0u, 0u};
    Acc sum = zero_acc();
    for (int k0 = 0; k0 < rank; k0 += 32) {
        u32x4_t b[2] = {none, none}, h = none, l = none;
        const int left = rank - k0 - g * 8;          // ranks of this lane's eight that exist
        if (left > 0) {
            b[0] = *reinterpret_cast<const u32x4_t*>(brow + k0);
            b[1] = *reinterpret_cast<const u32x4_t*>(brow + 16 * R + k0);
            if (id == a) {
                h = *reinterpret_cast<const u32x4_t*>(vhi + vo + k0);
                l = *reinterpret_cast<const u32x4_t*>(vlo + vo + k0);
            }
        }
        if (left < 8) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t keep = left >= 2 * j + 2 ? 0xFFFFFFFFu : left == 2 * j + 1 ? 0xFFFFu : 0u;
                b[0][j] &= keep;
                b[1][j] &= keep;
            }
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const bf16x8_t bf = __builtin_bit_cast(bf16x8_t, b[q]);
            sum.h[q] = mma(bf, h, sum.h[q]);
            sum.h[q] = mma(bf, l, sum.h[q]);
        }
    }
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc.h[q][v] = id == a ? acc.h[q][v] + sum.h[q][v] : acc.h[q][v];
}

// ---- the projections -----------------------------------------------------------------

struct ProjectArgs {
    const uint8_t* codes[2];
    const uint8_t* scales[2];
    LoraView lora[2];          // count 0: no adapters
    const uint16_t* vhi[2];
    const uint16_t* vlo[2];
    const int32_t* adapter;
    const uint16_t* xhi;
    const uint16_t* xlo;       // second plane of x (PL = 2)
    int T, n, K, splits;
    float* part;               // [splits][NM][T][n]
    uint32_t* counters;        // one per (panel, tile) with several splits
    const uint16_t* base;      // NM = 1
    uint16_t* y;               // NM = 1: [T][n] bf16
    uint16_t* hhi;             // NM = 2: h = silu(first) * second as two planes [T][n]
    uint16_t* hlo;
};

// Workgroup (row panel, split of K, tile of 32 tokens): the waves and splits
// divide K evenly and the tile's adapters in turn; sums in wave order, then
// in split order by the last workgroup of the (panel, tile).  NM matrices
// share x; PL planes of x add up.
template <int FMT, int NM, int PL, int NX>
__global__ void __launch_bounds__(kThreads, 2) lora_project_kernel(ProjectArgs a) {
    extern __shared__ __attribute__((aligned(16))) float red[];
    __shared__ uint32_t flag;
    const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
    const int p = blockIdx.x, split = blockIdx.y, t0 = blockIdx.z * kTile;
    const int nt = min(kTile, a.T - t0), nx = nt > kCols ? 2 : 1;
    const int units = a.K / kUnit, parts = a.splits * kWaves, me = split * kWaves + wid;
    const int u0 = me * units / parts, u1 = (me + 1) * units / parts;
    int t[NX];
#pragma unroll
    for (int i = 0; i < NX; ++i) t[i] = t0 + min(i * kCols + (lane & 15), nt - 1);

    PanelRef pr[NM];
    Acc acc[NM][NX];
#pragma unroll
    for (int m = 0; m < NM; ++m) {
        pr[m] = panel_ref<FMT>(a.codes[m], a.scales[m], a.K, p);
#pragma unroll
        for (int i = 0; i < NX; ++i) acc[m][i] = zero_acc();
    }
    WUnit<FMT> w[2][NM];
    XUnit x[2][NX][PL];
    auto load = [&](int b, int u) {
#pragma unroll
        for (int m = 0; m < NM; ++m) load_unit<FMT>(w[b][m], pr[m], u, lane);
#pragma unroll
        for (int i = 0; i < NX; ++i)
            if (i < nx) {
                load_x<FMT>(x[b][i][0], a.xhi + (int64_t)t[i] * a.K, u, lane);
                if constexpr (PL == 2) load_x<FMT>(x[b][i][PL - 1], a.xlo + (int64_t)t[i] * a.K, u, lane);
            }
    };
    auto step = [&](int b) {
#pragma unroll
        for (int m = 0; m < NM; ++m) mma_unit<FMT, NX, PL>(acc[m], w[b][m], x[b], nx);
    };
    if (u0 < u1) load(0, u0);
    for (int u = u0; u < u1; u += 2) {
        if (u + 1 < u1) load(1, u + 1);
        step(0);
        if (u + 1 < u1) {
            if (u + 2 < u1) load(0, u + 2);
            step(1);
        }
    }
#pragma unroll
    for (int m = 0; m < NM; ++m)
        if (a.lora[m].count > 0) {
            const int id = tile_adapter(a.adapter, t0, a.T, a.lora[m].count, lane);
            int col[NX];                 // the columns' adapters
#pragma unroll
            for (int i = 0; i < NX; ++i) col[i] = __shfl(id, i * kCols + (lane & 15), 64);
            each_adapter(id, [&](int i, int ad) {
                if (i % parts != me) return;
#pragma unroll
                for (int q = 0; q < NX; ++q)
                    expand(acc[m][q], a.lora[m], a.vhi[m], a.vlo[m], a.n, p, ad, col[q], t[q], lane);
            });
        }

    constexpr int PT = kPlaces;
    float s[NM][PT];
#pragma unroll
    for (int m = 0; m < NM; ++m) {
        if (m > 0) __syncthreads();
#pragma unroll
        for (int i = 0; i < NX; ++i) put_acc(red, acc[m][i], i, wid, nt, lane);
        __syncthreads();
        sum_waves(s[m], red, nt, tid);
    }
    auto place = [&](int q) { return (int64_t)(t0 + ((tid + q * kThreads) >> 5)) * a.n + p * 32 + (tid & 31); };
    auto valid = [&](int q) { return ((tid + q * kThreads) >> 5) < nt; };
    if (a.splits > 1) {
        const int64_t plane = (int64_t)a.T * a.n;
#pragma unroll
        for (int q = 0; q < PT; ++q)
            if (valid(q))
#pragma unroll
                for (int m = 0; m < NM; ++m) put_agent(a.part + (split * NM + m) * plane + place(q), s[m][q]);
        if (!last_arrival(a.counters + blockIdx.z * gridDim.x + p, a.splits, &flag)) return;
#pragma unroll
        for (int q = 0; q < PT; ++q)
            if (valid(q))
#pragma unroll
                for (int m = 0; m < NM; ++m) {
                    float v = 0.0f;
                    for (int i = 0; i < a.splits; ++i) v += get_agent(a.part + (i * NM + m) * plane + place(q));
                    s[m][q] = v;
                }
    }
#pragma unroll
    for (int q = 0; q < PT; ++q) {
        if (!valid(q)) continue;
        const int64_t o = place(q);
        if constexpr (NM == 2) {
            // h in 16 significant bits: its rounding stays far below that of y
            uint16_t h, l;
            split_bf16(silu(s[0][q]) * s[NM - 1][q], h, l);
            a.hhi[o] = h;
            a.hlo[o] = l;
        } else {
            float v = s[0][q];
            if (a.base) v += __uint_as_float((uint32_t)a.base[o] << 16);
            a.y[o] = f32_to_bf16_rne(v);
        }
    }
}

// ---- launches ---------------------------------------------------------------------------

constexpr size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// Splits of K: enough workgroups for the card's 256 compute units, and no
// more than leaves every wave a unit.
int project_splits(int n, int K, int T) {
    const int64_t wgs = (int64_t)(n / 32) * ((T + kTile - 1) / kTile);
    int64_t s = 256 / wgs;
    const int64_t most = (K / kUnit + kWaves - 1) / kWaves;
    if (s > most) s = most;
    return s < 1 ? 1 : (int)s;
}

size_t part_bytes(int nm, int n, int K, int T) {
    const int s = project_splits(n, K, T);
    return s > 1 ? align256((size_t)s * nm * T * n * sizeof(float)) : 0;
}

size_t lds_bytes(int T) { return (size_t)kWaves * (T < kTile ? T : kTile) * kRedRow * sizeof(float); }

hipError_t launch_shrink(const ShrinkArgs& s, int projections, hipStream_t st) {
    const int tiles = (s.T + kTile - 1) / kTile;
    int most = 0;
    for (int i = 0; i < projections; ++i) most = s.lora[i].count > most ? s.lora[i].count : most;
    // a workgroup per adapter of a tile while tiles are few; prompts have few adapters per tile
    int gy = most < kTile ? most : kTile;
    if (gy > s.T) gy = s.T;
    if (tiles >= 32 && gy > 4) gy = 4;
    const dim3 grid(tiles, gy, projections * s.panels);
    if (s.xlo) hipLaunchKernelGGL(lora_shrink_kernel<2>, grid, dim3(kThreads), lds_bytes(s.T), st, s);
    else hipLaunchKernelGGL(lora_shrink_kernel<1>, grid, dim3(kThreads), lds_bytes(s.T), st, s);
    return hipGetLastError();
}

template <int FMT, int NM, int PL>
void launch_project_nx(const ProjectArgs& a, hipStream_t st) {
    const dim3 grid(a.n / 32, a.splits, (a.T + kTile - 1) / kTile);
    if (a.T <= kCols)
        hipLaunchKernelGGL((lora_project_kernel<FMT, NM, PL, 1>), grid, dim3(kThreads), lds_bytes(a.T), st, a);
    else
        hipLaunchKernelGGL((lora_project_kernel<FMT, NM, PL, 2>), grid, dim3(kThreads), lds_bytes(a.T), st, a);
}

// Prompts: from this many tokens on the 128-row GEMM tiles are faster than
// streaming the weights once per 32 tokens.  They reach rows by 32-bit
// offsets and move outputs in 16-byte pieces; other calls stream.
constexpr int kGemmTokens = 256;
bool gemm_fits(int T, int K, const void* y, const void* base) {
    return T >= kGemmTokens && (int64_t)T * K * 2 < (1ll << 32) && (reinterpret_cast<uintptr_t>(y) & 15) == 0 &&
           (reinterpret_cast<uintptr_t>(base) & 15) == 0;
}

template <int NM, int PL>
hipError_t launch_project(int fmt, const ProjectArgs& a, hipStream_t st) {
    switch (fmt) {
        case FT_FMT_BF16: launch_project_nx<FT_FMT_BF16, NM, PL>(a, st); break;
        case FT_FMT_FP8_B128: launch_project_nx<FT_FMT_FP8_B128, NM, PL>(a, st); break;
        case FT_FMT_MXFP4_B32: launch_project_nx<FT_FMT_MXFP4_B32, NM, PL>(a, st); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

struct ExpertBuffers {
    size_t v[3], h, part, total;
};
// v of a projection: two planes [T][R]; h: two planes [T][f]
ExpertBuffers expert_buffers(const ft_shape& s, int max_rank, int T) {
    ExpertBuffers b;
    size_t o = 0;
    for (int i = 0; i < 3; ++i) {
        b.v[i] = o;
        o += 2 * align256((size_t)T * max_rank * 2);
    }
    b.h = o;
    o += 2 * align256((size_t)T * s.d_ff * 2);
    b.part = o;
    const size_t p1 = part_bytes(2, s.d_ff, s.d_model, T), p2 = part_bytes(1, s.d_model, s.d_ff, T);
    b.total = o + (p1 > p2 ? p1 : p2);
    return b;
}

}  // namespace

size_t lora_project_call_bytes(int n, int K, int max_rank, int T) {
    return part_bytes(1, n, K, T) + 2 * align256((size_t)T * max_rank * 2);
}
size_t lora_expert_call_bytes(const ft_shape& s, int max_rank, int T) { return expert_buffers(s, max_rank, T).total; }

// The largest need of any call of up to max_tokens tokens: the partial sums
// shrink when a call's tiles alone fill the card, so every tile count up to
// that point is looked at.
size_t lora_project_workspace(int n, int K, int max_rank, int max_tokens) {
    size_t most = 0;
    for (int T = 1;; T = T + kTile < max_tokens ? (T / kTile + 1) * kTile : max_tokens) {
        const size_t b = lora_project_call_bytes(n, K, max_rank, T);
        most = b > most ? b : most;
        if (T >= max_tokens) break;
    }
    return most;
}

size_t lora_expert_workspace(const ft_shape& s, int max_rank, int max_tokens) {
    size_t most = 0;
    for (int T = 1;; T = T + kTile < max_tokens ? (T / kTile + 1) * kTile : max_tokens) {
        const size_t b = lora_expert_call_bytes(s, max_rank, T);
        most = b > most ? b : most;
        if (T >= max_tokens) break;
    }
    return most;
}

hipError_t launch_lora_project(const MatrixView& m, const LoraView* lora, const int32_t* adapter, const uint16_t* x,
                               int T, const uint16_t* base, uint16_t* y, ft_workspace* ws, hipStream_t st) {
    uint8_t* mem = ws->mem + kCounterBytes;
    ProjectArgs a = {};
    a.codes[0] = m.codes;
    a.scales[0] = m.scales;
    a.lora[0] = lora ? *lora : LoraView();
    a.lora[1] = LoraView();
    a.adapter = adapter;
    a.xhi = x;
    a.T = T;
    a.n = m.n;
    a.K = m.K;
    a.splits = project_splits(m.n, m.K, T);
    a.counters = reinterpret_cast<uint32_t*>(ws->mem);
    a.base = base;
    a.y = y;
    size_t o = 0;
    if (a.lora[0].count > 0) {
        const size_t plane = align256((size_t)T * lora->max_rank * 2);
        ShrinkArgs s = {};
        s.lora[0] = *lora;
        s.lora[1] = LoraView();
        s.vhi[0] = reinterpret_cast<uint16_t*>(mem);
        s.vlo[0] = reinterpret_cast<uint16_t*>(mem + plane);
        s.adapter = adapter;
        s.xhi = x;
        s.T = T;
        s.K = m.K;
        s.panels = lora->max_rank / 16;
        hipError_t e = launch_shrink(s, 1, st);
        if (e != hipSuccess) return e;
        a.vhi[0] = s.vhi[0];
        a.vlo[0] = s.vlo[0];
        o = 2 * plane;
    }
    if (gemm_fits(T, m.K, y, base)) {
        LoraGemmArgs g = {};
        g.Hin = x;
        g.Y = y;
        g.T = T;
        g.d = m.n;
        g.f = m.K;
        g.h_bytes = (uint32_t)((int64_t)T * m.K * 2);
        g.codes[0] = m.codes;
        g.scales[0] = m.scales;
        g.lora[0] = a.lora[0];
        g.vhi[0] = a.vhi[0];
        g.vlo[0] = a.vlo[0];
        g.adapter = adapter;
        g.base = base;
        return launch_lora_gemm(m.fmt, false, g, st);
    }
    a.part = reinterpret_cast<float*>(mem + o);
    return launch_project<1, 1>(m.fmt, a, st);
}

hipError_t launch_lora_expert(const ft_shape& sh, const RecordLayout& rl, const uint8_t* rec, const LoraView* gate,
                              const LoraView* up, const LoraView* down, const int32_t* adapter, const uint16_t* x,
                              int T, const uint16_t* base, uint16_t* y, ft_workspace* ws, hipStream_t st) {
    uint8_t* mem = ws->mem + kCounterBytes;
    int R = 0;
    for (const LoraView* l : {gate, up, down})
        if (l && l->max_rank > R) R = l->max_rank;
    const ExpertBuffers b = expert_buffers(sh, R, T);
    auto v_hi = [&](int i) { return reinterpret_cast<uint16_t*>(mem + b.v[i]); };
    auto v_lo = [&](int i) { return reinterpret_cast<uint16_t*>(mem + b.v[i] + align256((size_t)T * R * 2)); };
    uint16_t* hhi = reinterpret_cast<uint16_t*>(mem + b.h);
    uint16_t* hlo = reinterpret_cast<uint16_t*>(mem + b.h + align256((size_t)T * sh.d_ff * 2));

    // one launch for the adapters of gate and up, where either has any
    ShrinkArgs s = {};
    int n = 0;
    s.adapter = adapter;
    s.xhi = x;
    s.T = T;
    s.K = sh.d_model;
    s.lora[0] = s.lora[1] = LoraView();
    const LoraView* gu[2] = {gate, up};
    for (int i = 0; i < 2; ++i)
        if (gu[i] && gu[i]->count > 0) {
            s.lora[n] = *gu[i];
            s.vhi[n] = v_hi(i);
            s.vlo[n] = v_lo(i);
            const int p = gu[i]->max_rank / 16;
            s.panels = p > s.panels ? p : s.panels;
            ++n;
        }
    hipError_t e;
    if (n > 0 && (e = launch_shrink(s, n, st)) != hipSuccess) return e;

    const bool gemm = gemm_fits(T, sh.d_model > sh.d_ff ? sh.d_model : sh.d_ff, y, base);
    LoraGemmArgs gm = {};
    if (gemm) {
        gm.x = x;
        gm.Hin = gm.Hout = hhi;
        gm.Y = y;
        gm.T = T;
        gm.d = sh.d_model;
        gm.f = sh.d_ff;
        gm.x_bytes = (uint32_t)((int64_t)T * sh.d_model * 2);
        gm.h_bytes = (uint32_t)((int64_t)T * sh.d_ff * 2);
        gm.codes[0] = rec + rl.off_gate;
        gm.codes[1] = rec + rl.off_up;
        gm.scales[0] = rec + rl.off_sg;
        gm.scales[1] = rec + rl.off_su;
        for (int i = 0; i < 2; ++i) {
            gm.lora[i] = gu[i] ? *gu[i] : LoraView();
            gm.vhi[i] = v_hi(i);
            gm.vlo[i] = v_lo(i);
        }
        gm.adapter = adapter;
        if ((e = launch_lora_gemm(sh.fmt, true, gm, st)) != hipSuccess) return e;
    }

    ProjectArgs a = {};
    a.codes[0] = rec + rl.off_gate;
    a.codes[1] = rec + rl.off_up;
    a.scales[0] = rec + rl.off_sg;
    a.scales[1] = rec + rl.off_su;
    for (int i = 0; i < 2; ++i) {
        a.lora[i] = gu[i] ? *gu[i] : LoraView();
        a.vhi[i] = v_hi(i);
        a.vlo[i] = v_lo(i);
    }
    a.adapter = adapter;
    a.xhi = x;
    a.T = T;
    a.n = sh.d_ff;
    a.K = sh.d_model;
    a.splits = project_splits(a.n, a.K, T);
    a.part = reinterpret_cast<float*>(mem + b.part);
    a.counters = reinterpret_cast<uint32_t*>(ws->mem);
    a.hhi = hhi;
    a.hlo = hlo;
    if (!gemm && (e = launch_project<2, 1>(sh.fmt, a, st)) != hipSuccess) return e;

    if (down && down->count > 0) {
        ShrinkArgs d = {};
        d.lora[0] = *down;
        d.lora[1] = LoraView();
        d.vhi[0] = v_hi(2);
        d.vlo[0] = v_lo(2);
        d.adapter = adapter;
        d.xhi = hhi;
        d.xlo = gemm ? nullptr : hlo;
        d.T = T;
        d.K = sh.d_ff;
        d.panels = down->max_rank / 16;
        if ((e = launch_shrink(d, 1, st)) != hipSuccess) return e;
    }
    if (gemm) {
        gm.codes[0] = rec + rl.off_down;
        gm.scales[0] = rec + rl.off_sd;
        gm.lora[0] = down ? *down : LoraView();
        gm.vhi[0] = v_hi(2);
        gm.vlo[0] = v_lo(2);
        gm.base = base;
        return launch_lora_gemm(sh.fmt, false, gm, st);
    }
    ProjectArgs c = {};
    c.codes[0] = rec + rl.off_down;
    c.scales[0] = rec + rl.off_sd;
    c.lora[0] = down ? *down : LoraView();
    c.lora[1] = LoraView();
    c.vhi[0] = v_hi(2);
    c.vlo[0] = v_lo(2);
    c.adapter = adapter;
    c.xhi = hhi;
    c.xlo = hlo;
    c.T = T;
    c.n = sh.d_model;
    c.K = sh.d_ff;
    c.splits = project_splits(c.n, c.K, T);
    c.part = a.part;
    c.counters = a.counters;
    c.base = base;
    c.y = y;
    return launch_project<1, 2>(sh.fmt, c, st);
}

}  // namespace ftmoe
