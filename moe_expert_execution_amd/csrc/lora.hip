// Projections with the low-rank adapters of many requests beside them:
//
//   y[t] = base[t] + x[t] W^T + s_a (x[t] A_a^T) B_a^T,   a = adapter[t],
//
// and a SwiGLU expert whose three projections carry adapters.  Up to 32 tokens
// read W once for all requests, longer calls once per tile of 32 tokens (the
// prompts' GEMM: of 64 or 128); an adapter's A [r x K] and B [n x r] are read
// once per tile, or span of up to 64 tokens, that names it.  The first launch
// computes v = s_a x A_a^T (r <= 128 values per token), the second streams W
// and adds v B_a^T to its accumulators.  With few adapters one launch does
// both, and each panel of 32 rows of W reads their A again.  The expert FFN
// reads one complete record ("The Expert Cache That Follows the Router",
// section "One logical expert, two physical levels of memory").
#include "lora_rules.h"
#include "resident.h"

namespace ftmoe {
namespace {

using namespace rs;

// ---- the adapters of a tile -----------------------------------------------------------

// The adapter of token t0 + lane % N; ids outside the pool name none (-1).
template <int N>
__device__ __forceinline__ int tile_adapter(const int32_t* adapter, int t0, int T, int count, int lane) {
    const int t = t0 + (lane & (N - 1));
    const int id = t < T ? adapter[t] : -1;
    return (uint32_t)id < (uint32_t)count ? id : -1;
}

// A tile's adapters as steps of RS ranks, in the order of their first token.
struct Step {
    int a, r0, rank;
    float scale;
};
constexpr int kMaxSteps = kTile * kMaxRank / 16;

// One wave writes the steps of the pool for the tile's 32 tokens; returns
// their number in *n.
template <int RS>
__device__ __forceinline__ void list_steps(Step* steps, int* n, const LoraView& lo, int id, int lane) {
    int rank = 0;
    float scale = 0.0f;
    if (lo.count > 0 && lo.count <= 64) {      // the whole pool's ranks and scales at once, not behind the ids
        const int c = min(lane, lo.count - 1);
        const int r = lo.rank[c];
        const float sc = lo.scale[c];
        rank = __shfl(r, id & 63, 64);
        scale = __shfl(sc, id & 63, 64);
    } else if (id >= 0) {
        rank = lo.rank[id];
        scale = lo.scale[id];
    }
    rank = id >= 0 ? min(max(rank, 0), lo.max_rank) : 0;
    bool first = id >= 0 && lane < kTile;
#pragma unroll
    for (int o = 1; o < kTile; ++o) {
        const int other = __shfl(id, lane - o, 64);
        first = first && (o > lane || other != id);
    }
    const int mine = first ? (rank + RS - 1) / RS : 0;
    int at = mine;
#pragma unroll
    for (int o = 1; o < kTile; o <<= 1) {
        const int v = __shfl_up(at, o, 64);
        if (lane >= o) at += v;
    }
    if (lane == kTile - 1) *n = at;
    at -= mine;
    for (int q = 0; q < mine; ++q) steps[at + q] = Step{id, q * RS, rank, scale};
}

struct ShrinkArgs {
    LoraView lora[2];
    uint16_t* vhi[2];      // [parts][T][R] v over the parts of K, as two bf16 planes (prompts), or
    uint16_t* vlo[2];
    float* vpart[2];       // in fp32, with
    Step* steps[2];        // the steps of 32 ranks of each tile of 32 tokens [tiles][kMaxSteps / 2]
    int* n_steps[2];       // and their number
    const int32_t* adapter;
    const uint16_t* xhi;
    const uint16_t* xlo;   // second plane of x (PL = 2)
    int T, K, panels;      // rank panels of 16 per projection
    int slots;             // projections times panels
    int parts;             // parts of K
};

// Workgroup (span of SPAN tokens, stride over the span's adapters, S slots and
// part of K), a slot being 16 ranks of a projection: v for every token of the
// adapter, gathered from the span as columns that the slots share; the waves
// split the part.  The later adapters of a span go first: most spans of a prompt
// have one adapter, so those workgroups mostly end at once, and the others' work
// should not start behind it.
//
// Latency and the gathered reads bound it: 64 tokens of 32 adapters of up to 64
// ranks, K = 4,096 (17 MB of A) take 8.4 us, 777 tokens of K = 2,048 6.4, 8,192
// tokens of two slots 15 (33 MB of x, read twice).
template <int PL, int NX, int SPAN, int S>
__global__ void __launch_bounds__(kThreads, 2) lora_shrink_kernel(ShrinkArgs s) {
    extern __shared__ __attribute__((aligned(16))) float red[];
    __shared__ uint8_t cols[kWaves][SPAN];          // (a copy per wave: no barrier)
    constexpr int CW = NX * kCols;                  // columns of a pass
    const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
    const int t0 = blockIdx.x * SPAN, stride = gridDim.z, first = stride - 1 - (int)blockIdx.z;
    const int part = blockIdx.y % s.parts, slot0 = blockIdx.y / s.parts * S;
    int proj[S], r0[S], ranks[S], id = -1;          // the lane's token's adapter, and its ranks in each slot's pool
    float scales[S];
    const int raw = lane < SPAN && t0 + lane < s.T ? s.adapter[t0 + lane] : -1;
#pragma unroll
    for (int m = 0; m < S; ++m) {
        const int slot = slot0 + m, q = slot / s.panels;
        const bool live = slot < s.slots && (slot - q * s.panels) * 16 < s.lora[min(q, 1)].max_rank;
        proj[m] = live ? q : 0;
        r0[m] = live ? (slot - q * s.panels) * 16 : kMaxRank;
        const LoraView& lo = s.lora[proj[m]];
        ranks[m] = 0;
        scales[m] = 0.0f;
        if (live && (uint32_t)raw < (uint32_t)lo.count) {
            id = raw;
            ranks[m] = min(max(lo.rank[raw], 0), lo.max_rank);
            scales[m] = lo.scale[raw];
        }
    }
    const int units = s.K / kUnit;
    const int me = part * kWaves + wid, all = s.parts * kWaves;
    const int u0 = me * units / all, u1 = (me + 1) * units / all;
    if constexpr (S == 1) {
        if (s.steps[proj[0]] && first == 0 && r0[0] == 0 && part == 0 && wid < SPAN / kTile) {
            const int tile = t0 / kTile + wid;
            if (tile * kTile < s.T)
                list_steps<32>(s.steps[proj[0]] + (int64_t)tile * (kMaxSteps / 2), s.n_steps[proj[0]] + tile, s.lora[proj[0]],
                               __shfl(id, wid * kTile + (lane & (kTile - 1)), 64), lane);
        }
    }
    uint64_t left = __ballot(id >= 0);
    for (int i = 0; left; ++i) {
        const int src = __builtin_ctzll(left);
        const int a = __builtin_amdgcn_readlane(id, src);
        const uint64_t hit = __ballot(id == a);
        left &= ~hit;
        if (i % stride != first) continue;
        int rank[S];
        bool on[S], any = false;          // the expand reads v in steps of 16 up to the rank
#pragma unroll
        for (int m = 0; m < S; ++m) {
            rank[m] = __builtin_amdgcn_readlane(ranks[m], src);
            on[m] = r0[m] < rank[m];
            any = any || on[m];
        }
        if (!any) continue;
        if (id == a) cols[wid][__popcll(hit & ((1ull << lane) - 1))] = (uint8_t)lane;
        const int nc = __popcll(hit);
        const uint16_t* arow[S];
#pragma unroll
        for (int m = 0; m < S; ++m)
            arow[m] = s.lora[proj[m]].a +
                      ((int64_t)a * s.lora[proj[m]].max_rank + min(r0[m] + (lane & 15), max(rank[m] - 1, 0))) * s.K;
        for (int c0 = 0; c0 < nc; c0 += CW) {
            const int n = min(CW, nc - c0);
            int64_t xo[NX];
#pragma unroll
            for (int q = 0; q < NX; ++q)
                xo[q] = (int64_t)(t0 + cols[wid][c0 + min(q * kCols + (lane & 15), n - 1)]) * s.K;
            f32x4_t acc[S][NX];
#pragma unroll
            for (int m = 0; m < S; ++m)
#pragma unroll
                for (int q = 0; q < NX; ++q) acc[m][q] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
            XUnit au[2][S], x[2][NX][PL];
            pipelined<2>(
                u1 - u0,
                [&](int b, int u) {
#pragma unroll
                    for (int m = 0; m < S; ++m)
                        if (S == 1 || on[m]) load_x<FT_FMT_BF16>(au[b][m], arow[m], u0 + u, lane);
#pragma unroll
                    for (int q = 0; q < NX; ++q)
                        if (q == 0 || q * kCols < n) {
                            load_x<FT_FMT_BF16>(x[b][q][0], s.xhi + xo[q], u0 + u, lane);
                            if constexpr (PL == 2) load_x<FT_FMT_BF16>(x[b][q][PL - 1], s.xlo + xo[q], u0 + u, lane);
                        }
                },
                [&](int b, int) {
#pragma unroll
                    for (int m = 0; m < S; ++m)
                        if (S == 1 || on[m])
#pragma unroll
                            for (int v = 0; v < 4; ++v)
#pragma unroll
                                for (int q = 0; q < NX; ++q)
                                    if (q == 0 || q * kCols < n)
#pragma unroll
                                        for (int p = 0; p < PL; ++p)
                                            acc[m][q] = mma(__builtin_bit_cast(bf16x8_t, au[b][m].v[v]), x[b][q][p].v[v], acc[m][q]);
                });
            constexpr int RR = 20;                   // floats of a column's ranks in LDS, padded
            __syncthreads();
#pragma unroll
            for (int q = 0; q < NX; ++q) {
                const int c = q * kCols + (lane & 15);
#pragma unroll
                for (int m = 0; m < S; ++m)
                    if (c < n) *reinterpret_cast<f32x4_t*>(red + ((m * kWaves + wid) * n + c) * RR + 4 * (lane >> 4)) = acc[m][q];
            }
            __syncthreads();
#pragma unroll
            for (int m = 0; m < S; ++m) {
                if (!on[m]) continue;
                const float scale = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(scales[m]), src));
                const int R = s.lora[proj[m]].max_rank;
                for (int q = tid; q < n * 16; q += kThreads) {
                    const int c = q >> 4, k = q & 15, r = r0[m] + k;
                    float v = 0.0f;
#pragma unroll
                    for (int w = 0; w < kWaves; ++w) v += red[((m * kWaves + w) * n + c) * RR + k];
                    v = r < rank[m] ? scale * v : 0.0f;
                    const int64_t at = ((int64_t)part * s.T + t0 + cols[wid][c0 + c]) * R + r;
                    if (s.vpart[proj[m]]) {
                        s.vpart[proj[m]][at] = v;
                    } else {
                        uint16_t h, l;
                        split_bf16(v, h, l);              // 16 significant bits
                        s.vhi[proj[m]][at] = h;
                        s.vlo[proj[m]][at] = l;
                    }
                }
            }
        }
    }
}

// ---- the projections -----------------------------------------------------------------

struct ProjectArgs {
    const uint8_t* codes[2];
    const uint8_t* scales[2];
    LoraView lora[2];          // count 0: no adapters
    const float* v[2];         // of the shrink launch: v [vparts][T][R],
    const Step* steps[2];      // and each tile's steps of 32 ranks (unless FUSED)
    const int* n_steps[2];
    int vparts;
    const int32_t* adapter;
    const uint16_t* xhi;
    const uint16_t* xlo;       // second plane of x (PL = 2)
    int T, n, K;
    int splits;                // workgroups of a (panel, tile) that split K
    int lsplits;               // and, per matrix, that take its adapters (FUSED)
    float* part;               // [splits + lsplits][NM][T][n] (more than one workgroup in all)
    uint32_t* counters;        // one per (panel, tile)
    const uint16_t* base;      // NM = 1
    uint16_t* y;               // NM = 1: [T][n] bf16
    uint16_t* hhi;             // NM = 2: h = silu(first) * second as two planes [T][n]
    uint16_t* hlo;
};

// The lane's 16-bit pieces of `w` (two per dword) from position `left` on are cleared.
template <typename V>
__device__ __forceinline__ void keep_ranks(V& w, int left) {
    constexpr int N = sizeof(V) / 4;
#pragma unroll
    for (int j = 0; j < N; ++j) w[j] &= left >= 2 * j + 2 ? 0xFFFFFFFFu : left == 2 * j + 1 ? 0xFFFFu : 0u;
}

// v of a tile's tokens in LDS, as two bf16 planes of rows R + 8 apart: the sum
// of the shrink launch's parts, in 16 significant bits.  Tokens without an
// adapter and ranks that no step reaches hold anything.
__device__ __forceinline__ int v_row(int R) { return R + 8; }
__device__ __forceinline__ void stage_v(uint16_t* vs, const float* v, int vparts, int T, int R, int t0, int nt, int tid) {
    typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
    const int64_t plane = (int64_t)T * R;
    for (int i = tid; i < nt * (R / 4); i += kThreads) {
        const int m = i / (R / 4), k = (i - m * (R / 4)) * 4;
        const float* src = v + (int64_t)(t0 + m) * R + k;
        f32x4_t part[kMaxParts], z = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < kMaxParts; ++j)
            if (j < vparts) part[j] = *reinterpret_cast<const f32x4_t*>(src + j * plane);
#pragma unroll
        for (int j = 0; j < kMaxParts; ++j)
            if (j < vparts)
#pragma unroll
                for (int e = 0; e < 4; ++e) z[e] += part[j][e];
        uint16_t h[4], l[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split_bf16(z[e], h[e], l[e]);
        uint16_t* d = vs + m * v_row(R) + k;
        *reinterpret_cast<u32x2_t*>(d) = u32x2_t{h[0] | ((uint32_t)h[1] << 16), h[2] | ((uint32_t)h[3] << 16)};
        *reinterpret_cast<u32x2_t*>(d + kTile * v_row(R)) = u32x2_t{l[0] | ((uint32_t)l[1] << 16), l[2] | ((uint32_t)l[3] << 16)};
    }
}

// The B operand pairs of the steps me, me + parts, ... of 32 ranks for row
// panel p of B [n x R].
struct BStep {
    u32x4_t b[2];
};
__device__ __forceinline__ void load_b(BStep& o, const LoraView& lo, int n, int p, const Step st, int lane) {
    const int k = st.r0 + (lane >> 4) * 8;
    o.b[0] = o.b[1] = u32x4_t{0u, 0u, 0u, 0u};
    if (k < st.rank) {
        const uint16_t* row = lo.b + ((int64_t)st.a * n + p * 32 + (lane & 15)) * lo.max_rank + k;
        o.b[0] = *reinterpret_cast<const u32x4_t*>(row);
        o.b[1] = *reinterpret_cast<const u32x4_t*>(row + 16 * lo.max_rank);
    }
}

// acc += v B_a^T for one step.  `col` is the lane's columns' adapters; the
// other tokens' products are selected away (an adapter's infinities and NaN
// stay with its own requests), and ranks past the adapter's own are masked
// out of B, whatever the pool holds there.
template <int NX>
__device__ __forceinline__ void expand(Acc (&acc)[NX], const BStep& bs, const Step st, const uint16_t* vs, int R,
                                       const int (&col)[NX], int lane) {
    const u32x4_t none = u32x4_t{0u, 0u, 0u, 0u};
    const int k = st.r0 + (lane >> 4) * 8, left = st.rank - k;      // ranks of this lane's eight that exist
    u32x4_t w[2] = {bs.b[0], bs.b[1]};
    keep_ranks(w[0], left);
    keep_ranks(w[1], left);
#pragma unroll
    for (int x = 0; x < NX; ++x) {
        if (__ballot(col[x] == st.a) == 0) continue;
        u32x4_t h = none, l = none;
        if (left > 0 && col[x] == st.a) {
            const uint16_t* r = vs + (x * kCols + (lane & 15)) * v_row(R) + k;
            h = *reinterpret_cast<const u32x4_t*>(r);
            l = *reinterpret_cast<const u32x4_t*>(r + kTile * v_row(R));
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const bf16x8_t bf = __builtin_bit_cast(bf16x8_t, w[e]);
            f32x4_t s = mma(bf, h, f32x4_t{0.0f, 0.0f, 0.0f, 0.0f});
            s = mma(bf, l, s);
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[x].h[e][c] = col[x] == st.a ? acc[x].h[e][c] + s[c] : acc[x].h[e][c];
        }
    }
}

// The adapters without a launch of their own: v B_a^T is linear in v and v in
// the parts of K, so the pairs (16 ranks, unit of K) of a tile go round the
// waves, which multiply their part of v by B at once; the sums of the waves
// and workgroups are those of the projection itself.  The 16 x 16 sums of
// x A_a^T (rows: ranks, columns: tokens) are the B operand of the 16 x 16 x 16
// product as they stand.
template <int PL, int NX>
__device__ __forceinline__ void adapt(Acc (&acc)[NX], const LoraView& lo, const uint16_t* xhi, const uint16_t* xlo, int K,
                                      int n, int p, const Step* steps, int ns, int me, int parts, const int (&col)[NX],
                                      const int (&t)[NX], int lane) {
    typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
    typedef short s16x4_t __attribute__((ext_vector_type(4)));
    const int units = K / kUnit, R = lo.max_rank, g = lane >> 4;
    const int pairs = ns * units, mine = pairs > me ? (pairs - me - 1) / parts + 1 : 0;
    constexpr int D = NX * PL == 1 ? 4 : NX == 1 ? 3 : 2;
    XUnit au[D], xu[D][NX][PL];
    u32x2_t b[D][2];
    pipelined<D>(
        mine,
        [&](int q, int i) {
            const int j = me + i * parts, u = j % units;
            const Step st = steps[j / units];
            load_x<FT_FMT_BF16>(au[q], lo.a + ((int64_t)st.a * R + min(st.r0 + (lane & 15), st.rank - 1)) * K, u, lane);
#pragma unroll
            for (int x = 0; x < NX; ++x) {
                load_x<FT_FMT_BF16>(xu[q][x][0], xhi + (int64_t)t[x] * K, u, lane);
                if constexpr (PL == 2) load_x<FT_FMT_BF16>(xu[q][x][PL - 1], xlo + (int64_t)t[x] * K, u, lane);
            }
            const uint16_t* row = lo.b + ((int64_t)st.a * n + p * 32 + (lane & 15)) * R + st.r0 + 4 * g;
            b[q][0] = *reinterpret_cast<const u32x2_t*>(row);
            b[q][1] = *reinterpret_cast<const u32x2_t*>(row + 16 * R);
        },
        [&](int q, int i) {
            const Step st = steps[(me + i * parts) / units];
            const int left = st.rank - st.r0 - 4 * g;      // ranks of this lane's four that exist
            u32x2_t w[2] = {b[q][0], b[q][1]};
            keep_ranks(w[0], left);
            keep_ranks(w[1], left);
#pragma unroll
            for (int x = 0; x < NX; ++x) {
                f32x4_t v = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int pl = 0; pl < PL; ++pl) v = mma(__builtin_bit_cast(bf16x8_t, au[q].v[e]), xu[q][x][pl].v[e], v);
                // v in 16 significant bits; zero past the adapter's rank
                f32x4_t z, r;
#pragma unroll
                for (int e = 0; e < 4; ++e) z[e] = e < left ? st.scale * v[e] : 0.0f;
                const bf16x4_t h = __builtin_convertvector(z, bf16x4_t);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float hf = (float)h[e];
                    r[e] = fabsf(hf) < INFINITY ? z[e] - hf : 0.0f;
                }
                const bf16x4_t l = __builtin_convertvector(r, bf16x4_t);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    f32x4_t s = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
                    const s16x4_t bw = __builtin_bit_cast(s16x4_t, w[e]);
                    s = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(bw, __builtin_bit_cast(s16x4_t, h), s, 0, 0, 0);
                    s = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(bw, __builtin_bit_cast(s16x4_t, l), s, 0, 0, 0);
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[x].h[e][c] = col[x] == st.a ? acc[x].h[e][c] + s[c] : acc[x].h[e][c];
                }
            }
        });
}

// Workgroups of a row panel and tile of 32 tokens: `splits` that stream the
// panel, their waves dividing K.  The adapters, FUSED: lsplits workgroups more
// per matrix take them; they run beside the stream, not in
// its way (listing a tile's adapters and following their addresses takes
// several dependent loads).  Otherwise the streaming waves divide the steps of
// 32 ranks, the first of them loaded before the stream is multiplied.  Sums in
// wave order, then in workgroup order by the last workgroup of the (panel,
// tile).  NM matrices share x; PL planes of x add up.
//
// One token through [2,048 x 2,048] bf16 takes 6.5 us, 2.4 of them the launch (8.4 MB;
// latency); 64 tokens with 32 FP8 adapters of [4,096 x 4,096] 16 to 17.3: each workgroup
// brings 0.13 MB of weights, 0.26 of x and some 0.1 of B to its compute unit, at
// the 40 to 80 GB/s that one draws from L2: 6.4 us until the first two units, v and
// the list are in, 4.5 for the stream's other two, 3.4 for the adapters and 1.4 for
// the sum over waves, measured with two units in flight (three, which fit where one
// matrix and one plane of x take part, took 0.4 us off the call on one box).  v and
// the list loaded before the stream took 1 us more, four steps of B before it changed nothing.  The bf16 pair of matrices over
// two operands behind a shrink launch (an expert's gate and up for more than 16
// tokens of many adapters) spills 43 registers.
template <int FMT, int NM, int PL, int NX, bool FUSED>
__global__ void __launch_bounds__(kThreads, 2) lora_project_kernel(ProjectArgs a) {
    extern __shared__ __attribute__((aligned(16))) float red[];
    __shared__ uint32_t flag;
    __shared__ Step steps[FUSED ? 1 : NM][FUSED ? kMaxFusedSteps : kMaxSteps / 2];
    __shared__ int n_steps[NM];
    const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
    const int p = blockIdx.x, split = blockIdx.y, t0 = blockIdx.z * kTile;
    const int nt = min(kTile, a.T - t0), nx = nt > kCols ? 2 : 1;
    const int units = a.K / kUnit;
    int t[NX];
#pragma unroll
    for (int i = 0; i < NX; ++i) t[i] = t0 + min(i * kCols + (lane & 15), nt - 1);

    Acc acc[NM][NX];
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int i = 0; i < NX; ++i) acc[m][i] = zero_acc();
    const bool adapters = FUSED && split >= a.splits;
    const int am = adapters ? (split - a.splits) % NM : 0;      // the matrix of an adapter workgroup
    if (!adapters) {
        const int parts = a.splits * kWaves, me = split * kWaves + wid;
        const int u0 = me * units / parts, nu = (me + 1) * units / parts - u0;
        PanelRef pr[NM];
#pragma unroll
        for (int m = 0; m < NM; ++m) pr[m] = panel_ref<FMT>(a.codes[m], a.scales[m], a.K, p);
        constexpr int D = NM * PL == 1 ? 3 : 2;        // units in flight
        WUnit<FMT> w[D][NM];
        XUnit x[D][NX][PL];
        auto load = [&](int b, int u) {
#pragma unroll
            for (int m = 0; m < NM; ++m) load_unit<FMT>(w[b][m], pr[m], u0 + u, lane);
#pragma unroll
            for (int i = 0; i < NX; ++i)
                if (i < nx) {
                    load_x<FMT>(x[b][i][0], a.xhi + (int64_t)t[i] * a.K, u0 + u, lane);
                    if constexpr (PL == 2) load_x<FMT>(x[b][i][PL - 1], a.xlo + (int64_t)t[i] * a.K, u0 + u, lane);
                }
        };
        auto work = [&](int b) {
#pragma unroll
            for (int m = 0; m < NM; ++m) mma_unit<FMT, NX, PL>(acc[m], w[b][m], x[b], nx);
        };
#pragma unroll
        for (int b = 0; b < D; ++b)
            if (b < nu) load(b, b);
        uint16_t* vs[NM];
        int col[NM][NX], mine[NM];       // the columns' adapters; the wave's steps
        BStep first[NM];
        if constexpr (!FUSED) {
            uint16_t* at = reinterpret_cast<uint16_t*>(red + kWaves * min(a.T, kTile) * kRedRow);
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                vs[m] = at;
                mine[m] = 0;
                const LoraView& lo = a.lora[m];
                if (lo.count == 0) continue;
                at += 2 * kTile * v_row(lo.max_rank);
                const int id = tile_adapter<kTile>(a.adapter, t0, a.T, lo.count, lane);
                if (tid < kMaxSteps / 2) steps[m][tid] = a.steps[m][(int64_t)blockIdx.z * (kMaxSteps / 2) + tid];
                if (tid == 0) n_steps[m] = a.n_steps[m][blockIdx.z];
                stage_v(vs[m], a.v[m], a.vparts, a.T, lo.max_rank, t0, nt, tid);
#pragma unroll
                for (int i = 0; i < NX; ++i) col[m][i] = __shfl(id, i * kCols + (lane & 15), 64);
            }
            if (a.lora[0].count > 0 || a.lora[NM - 1].count > 0) {
                __syncthreads();
#pragma unroll
                for (int m = 0; m < NM; ++m)
                    if (a.lora[m].count > 0) {
                        const int ns = n_steps[m];
                        mine[m] = ns > me ? (ns - me - 1) / parts + 1 : 0;
                        if (mine[m] > 0) load_b(first[m], a.lora[m], a.n, p, steps[m][me], lane);
                    }
            }
        }
        for (int u = 0; u < nu; u += D)
#pragma unroll
            for (int b = 0; b < D; ++b)
                if (u + b < nu) {
                    work(b);
                    if (u + b + D < nu) load(b, u + b + D);
                }
        if constexpr (!FUSED) {
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                if (mine[m] == 0) continue;
                const LoraView& lo = a.lora[m];
                constexpr int BD = 4;
                BStep bs[BD];
                expand<NX>(acc[m], first[m], steps[m][me], vs[m], lo.max_rank, col[m], lane);
                pipelined<BD>(
                    mine[m] - 1,
                    [&](int q, int i) { load_b(bs[q], lo, a.n, p, steps[m][me + (i + 1) * parts], lane); },
                    [&](int q, int i) {
                        expand<NX>(acc[m], bs[q], steps[m][me + (i + 1) * parts], vs[m], lo.max_rank, col[m], lane);
                    });
            }
        }
    } else {
        const LoraView& lo = a.lora[am];
        const int sub = (split - a.splits) / NM, parts = a.lsplits * kWaves, me = sub * kWaves + wid;
        const int id = tile_adapter<kTile>(a.adapter, t0, a.T, lo.count, lane);
        if (wid == 0) list_steps<16>(steps[0], n_steps, lo, id, lane);
        int col[NX];
#pragma unroll
        for (int i = 0; i < NX; ++i) col[i] = __shfl(id, i * kCols + (lane & 15), 64);
        __syncthreads();
        Acc la[NX];
#pragma unroll
        for (int i = 0; i < NX; ++i) la[i] = zero_acc();
        adapt<PL, NX>(la, lo, a.xhi, a.xlo, a.K, a.n, p, steps[0], n_steps[0], me, parts, col, t, lane);
#pragma unroll
        for (int i = 0; i < NX; ++i) acc[0][i] = la[i];
    }

    // an adapter workgroup's sums are those of its matrix alone, in place 0
    constexpr int PT = kPlaces;
    float s[NM][PT];
#pragma unroll
    for (int m = 0; m < NM; ++m) {
        if (m > 0) {
            if (adapters) break;
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < NX; ++i) put_acc(red, acc[m][i], i, wid, nt, lane);
        __syncthreads();
        sum_waves(s[m], red, nt, tid);
    }
    auto place = [&](int q) { return (int64_t)(t0 + ((tid + q * kThreads) >> 5)) * a.n + p * 32 + (tid & 31); };
    auto valid = [&](int q) { return ((tid + q * kThreads) >> 5) < nt; };
    if (gridDim.y > 1) {
        const int64_t plane = (int64_t)a.T * a.n;
        const int row = adapters ? a.splits + (split - a.splits) / NM : split;
#pragma unroll
        for (int q = 0; q < PT; ++q)
            if (valid(q))
#pragma unroll
                for (int m = 0; m < NM; ++m)
                    if (m == 0 || !adapters) put_agent(a.part + (row * NM + (adapters ? am : m)) * plane + place(q), s[m][q]);
        if (!last_arrival(a.counters + blockIdx.z * gridDim.x + p, gridDim.y, &flag)) return;
        const int rows = a.splits + a.lsplits;
#pragma unroll
        for (int q = 0; q < PT; ++q)
            if (valid(q))
#pragma unroll
                for (int m = 0; m < NM; ++m) {
                    float v = 0.0f;
#pragma unroll 4
                    for (int i = 0; i < rows; ++i) v += get_agent(a.part + (i * NM + m) * plane + place(q));
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

size_t part_bytes(int nm, int n, int T, const Split& s) {
    const int rows = s.splits + s.lsplits;
    return rows > 1 ? align256((size_t)rows * nm * T * n * sizeof(float)) : 0;
}

// the waves' sums, and v of the matrices' adapters where the product expands them
template <bool FUSED>
size_t lds_bytes(const ProjectArgs& a) {
    size_t n = (size_t)kWaves * (a.T < kTile ? a.T : kTile) * kRedRow * sizeof(float);
    for (const LoraView& l : a.lora)
        if (!FUSED && l.count > 0) n += (size_t)2 * kTile * (l.max_rank + 8) * sizeof(uint16_t);
    return n;
}

hipError_t launch_shrink(const ShrinkArgs& s, const Shrink& sh, hipStream_t st) {
    const int spans = (s.T + sh.span - 1) / sh.span;
    const int most = s.lora[0].count > s.lora[1].count ? s.lora[0].count : s.lora[1].count;
    // a workgroup per adapter of a span while spans are few; prompts have few adapters per span
    int gy = most < kTile ? most : kTile;
    if (gy > s.T) gy = s.T;
    if (spans >= 16 && gy > 2) gy = 2;
    const dim3 grid(spans, (s.slots + sh.per - 1) / sh.per * s.parts, gy);
    const int cols = s.xlo || sh.span == kTile ? 2 * kCols : 4 * kCols;
    const size_t lds = (size_t)sh.per * kWaves * (s.T < cols ? s.T : cols) * 20 * sizeof(float);
    const auto f = s.xlo             ? lora_shrink_kernel<2, 2, 2 * kTile, 1>
                   : sh.span > kTile ? lora_shrink_kernel<1, 4, 2 * kTile, 1>
                   : sh.per == 1     ? lora_shrink_kernel<1, 2, kTile, 1>
                                     : lora_shrink_kernel<1, 2, kTile, 2>;
    return launch(f, grid, dim3(kThreads), lds, st, s);
}

template <int FMT, int NM, int PL, bool FUSED>
hipError_t launch_project_nx(const ProjectArgs& a, hipStream_t st) {
    const dim3 grid(a.n / 32, a.splits + a.lsplits * NM, (a.T + kTile - 1) / kTile);
    const auto f = a.T <= kCols ? lora_project_kernel<FMT, NM, PL, 1, FUSED> : lora_project_kernel<FMT, NM, PL, 2, FUSED>;
    return launch(f, grid, dim3(kThreads), lds_bytes<FUSED>(a), st, a);
}

// The GEMM's tiles move outputs in 16-byte pieces; other calls stream.
bool tiles_reach(const void* y, const void* base) {
    return (reinterpret_cast<uintptr_t>(y) & 15) == 0 && (reinterpret_cast<uintptr_t>(base) & 15) == 0;
}

template <int NM, int PL, bool FUSED>
hipError_t launch_project_as(int fmt, const ProjectArgs& a, hipStream_t st) {
    switch (fmt) {
        case FT_FMT_BF16: return launch_project_nx<FT_FMT_BF16, NM, PL, FUSED>(a, st);
        case FT_FMT_FP8_B128: return launch_project_nx<FT_FMT_FP8_B128, NM, PL, FUSED>(a, st);
        case FT_FMT_MXFP4_B32: return launch_project_nx<FT_FMT_MXFP4_B32, NM, PL, FUSED>(a, st);
    }
    return hipErrorInvalidValue;
}
template <int NM, int PL>
hipError_t launch_project(int fmt, const ProjectArgs& a, bool fuse, hipStream_t st) {
    return fuse ? launch_project_as<NM, PL, true>(fmt, a, st) : launch_project_as<NM, PL, false>(fmt, a, st);
}

int pool_adapters(const LoraView* l) { return l && l->count > 0 ? l->count : 0; }
int pool_rank(const LoraView* l) { return l && l->count > 0 ? l->max_rank : 0; }

// v of one projection over the parts of K: bf16 planes for the GEMM, else fp32
size_t rank_tiles(int T) { return ((size_t)T + kTile - 1) / kTile; }
// and the tiles' steps
size_t list_bytes(int T) {
    return rank_tiles(T) * (kMaxSteps / 2) * sizeof(Step) + align256(rank_tiles(T) * sizeof(int));
}
size_t v_bytes(int T, int rank, int parts) {
    if (rank == 0) return 0;
    const size_t two = 2 * align256((size_t)parts * T * rank * 2), f32 = align256((size_t)parts * T * rank * sizeof(float)) + list_bytes(T);
    return two > f32 ? two : f32;
}

// Workspace of a call: v of its projections, h, the partial sums.  The sizes
// are those of the most adapters a tile can name, so they hold for any pools
// of up to max_rank.
struct ExpertBuffers {
    size_t v[3], h, part, total;
};
ExpertBuffers expert_buffers(const ft_shape& s, int max_rank, int T) {
    ExpertBuffers b;
    size_t o = 0;
    for (int i = 0; i < 3; ++i) {
        b.v[i] = o;
        o += v_bytes(T, max_rank, kMaxParts);
    }
    b.h = o;
    o += 2 * align256((size_t)T * s.d_ff * 2);
    b.part = o;
    Split gu = split_of(2, s.d_ff, s.d_model, T, 0, 0), dn = split_of(1, s.d_model, s.d_ff, T, 0, 0);
    gu.lsplits = dn.lsplits = max_rank > 0 ? 4 : 0;
    const size_t p1 = part_bytes(2, s.d_ff, T, gu), p2 = part_bytes(1, s.d_model, T, dn);
    b.total = o + (p1 > p2 ? p1 : p2);
    return b;
}

}  // namespace

size_t lora_project_call_bytes(int n, int K, int max_rank, int T) {
    Split s = split_of(1, n, K, T, 0, 0);
    s.lsplits = max_rank > 0 ? 4 : 0;
    return part_bytes(1, n, T, s) + v_bytes(T, max_rank, kMaxParts);
}
size_t lora_expert_call_bytes(const ft_shape& s, int max_rank, int T) { return expert_buffers(s, max_rank, T).total; }

// The largest need of any call of up to max_tokens tokens.  A call's need grows
// with its tokens while the number of tiles stays, and may shrink from one number
// to the next, as the partial sums do when the tiles alone fill the card: so the
// last token count of each number is looked at.
template <typename F>
size_t largest_need(int max_tokens, F&& call_bytes) {
    size_t most = call_bytes(max_tokens);
    for (int T = kTile; T < max_tokens; T += kTile) {
        const size_t b = call_bytes(T);
        most = b > most ? b : most;
    }
    return most;
}

size_t lora_project_workspace(int n, int K, int max_rank, int max_tokens) {
    return largest_need(max_tokens, [&](int T) { return lora_project_call_bytes(n, K, max_rank, T); });
}

size_t lora_expert_workspace(const ft_shape& s, int max_rank, int max_tokens) {
    return largest_need(max_tokens, [&](int T) { return lora_expert_call_bytes(s, max_rank, T); });
}

namespace {

// The shrink launch of up to two projections that read the same x, into
// `planes` (two bf16 planes, for the GEMM) or fp32 parts at v[i].
hipError_t shrink(const LoraView* const* pools, uint8_t* const* v, int n, const int32_t* adapter, const uint16_t* xhi,
                  const uint16_t* xlo, int T, int K, bool planes, const Shrink& sh, hipStream_t st) {
    ShrinkArgs s = {};
    s.adapter = adapter;
    s.xhi = xhi;
    s.xlo = xlo;
    s.T = T;
    s.K = K;
    s.parts = sh.parts;
    int m = 0;
    for (int i = 0; i < n; ++i) {
        if (pool_adapters(pools[i]) == 0) continue;
        s.lora[m] = *pools[i];
        if (planes) {
            s.vhi[m] = reinterpret_cast<uint16_t*>(v[i]);
            s.vlo[m] = reinterpret_cast<uint16_t*>(v[i] + align256((size_t)kMaxParts * T * pools[i]->max_rank * 2));
        } else {
            s.vpart[m] = reinterpret_cast<float*>(v[i]);
            uint8_t* list = v[i] + align256((size_t)kMaxParts * T * pools[i]->max_rank * sizeof(float));
            s.steps[m] = reinterpret_cast<Step*>(list);
            s.n_steps[m] = reinterpret_cast<int*>(list + rank_tiles(T) * (kMaxSteps / 2) * sizeof(Step));
        }
        s.panels = pools[i]->max_rank / 16 > s.panels ? pools[i]->max_rank / 16 : s.panels;
        ++m;
    }
    s.slots = m * s.panels;
    return m > 0 ? launch_shrink(s, sh, st) : hipSuccess;
}

// The shrink launch before a GEMM over K.
Shrink gemm_shrink(const LoraView* const* pools, int n, int K, int T) {
    int m = 0, rank = 16;
    for (int i = 0; i < n; ++i) {
        if (pool_adapters(pools[i]) == 0) continue;
        rank = pools[i]->max_rank > rank ? pools[i]->max_rank : rank;
        ++m;
    }
    return shrink_of(T, K, (m > 0 ? m : 1) * (rank / 16), 1, true);
}

// The pools, planes and adapters of a GEMM's matrices
void gemm_pools(LoraGemmArgs& g, const LoraView* const* pools, uint8_t* const* v, int n, int parts) {
    g.vparts = parts;
    for (int i = 0; i < n; ++i) {
        g.lora[i] = pool_adapters(pools[i]) > 0 ? *pools[i] : LoraView();
        g.vhi[i] = reinterpret_cast<const uint16_t*>(v[i]);
        g.vlo[i] = reinterpret_cast<const uint16_t*>(v[i] + align256((size_t)kMaxParts * g.T * g.lora[i].max_rank * 2));
    }
}

// NM matrices [n x K] on T tokens with their pools: the shrink launch where it
// is needed, then the product.  `a` holds the matrices, x, outputs, part.
template <int NM, int PL>
hipError_t product(int fmt, ProjectArgs& a, const LoraView* const* pools, uint8_t* const* v, hipStream_t st) {
    int adapters = 0, rank = 0;
    for (int i = 0; i < NM; ++i) {
        if (pool_adapters(pools[i]) > adapters) adapters = pool_adapters(pools[i]);
        if (pool_rank(pools[i]) > rank) rank = pool_rank(pools[i]);
        if (pool_adapters(pools[i]) > 0) a.lora[i] = *pools[i];
        a.v[i] = reinterpret_cast<const float*>(v[i]);
        const uint8_t* list = v[i] + align256((size_t)kMaxParts * a.T * pool_rank(pools[i]) * sizeof(float));
        a.steps[i] = reinterpret_cast<const Step*>(list);
        a.n_steps[i] = reinterpret_cast<const int*>(list + rank_tiles(a.T) * (kMaxSteps / 2) * sizeof(Step));
    }
    const Split s = split_of(NM, a.n, a.K, a.T, adapters, rank);
    a.splits = s.splits;
    a.lsplits = s.lsplits;
    a.vparts = s.shrink.parts;
    if (s.adapted && !s.fused) {
        const hipError_t e = shrink(pools, v, NM, a.adapter, a.xhi, a.xlo, a.T, a.K, false, s.shrink, st);
        if (e != hipSuccess) return e;
    }
    return launch_project<NM, PL>(fmt, a, s.fused, st);
}

}  // namespace

hipError_t launch_lora_project(const MatrixView& m, const LoraView* lora, const int32_t* adapter, const uint16_t* x,
                               int T, const uint16_t* base, uint16_t* y, ft_workspace* ws, hipStream_t st) {
    uint8_t* mem = ws->mem + kCounterBytes;
    const LoraView* pools[1] = {lora};
    uint8_t* v[1] = {mem};
    if (project_tiles(m.n, m.K, T) && tiles_reach(y, base)) {
        LoraGemmArgs g = {};
        g.Hin = x;
        g.Y = y;
        g.T = T;
        g.d = m.n;
        g.f = m.K;
        g.h_bytes = (uint32_t)((int64_t)T * m.K * 2);
        g.codes[0] = m.codes;
        g.scales[0] = m.scales;
        g.adapter = adapter;
        g.base = base;
        const Shrink sk = gemm_shrink(pools, 1, m.K, T);
        gemm_pools(g, pools, v, 1, sk.parts);
        const hipError_t e = shrink(pools, v, 1, adapter, x, nullptr, T, m.K, true, sk, st);
        return e != hipSuccess ? e : launch_lora_gemm(m.fmt, false, g, st);
    }
    ProjectArgs a = {};
    a.codes[0] = m.codes;
    a.scales[0] = m.scales;
    a.adapter = adapter;
    a.xhi = x;
    a.T = T;
    a.n = m.n;
    a.K = m.K;
    a.part = reinterpret_cast<float*>(mem + v_bytes(T, pool_rank(lora), kMaxParts));
    a.counters = reinterpret_cast<uint32_t*>(ws->mem);
    a.base = base;
    a.y = y;
    return product<1, 1>(m.fmt, a, pools, v, st);
}

hipError_t launch_lora_expert(const ft_shape& sh, const RecordLayout& rl, const uint8_t* rec, const LoraView* gate,
                              const LoraView* up, const LoraView* down, const int32_t* adapter, const uint16_t* x,
                              int T, const uint16_t* base, uint16_t* y, ft_workspace* ws, hipStream_t st) {
    uint8_t* mem = ws->mem + kCounterBytes;
    const LoraView* pools[3] = {gate, up, down};
    int R = 0;
    for (const LoraView* l : pools) R = pool_rank(l) > R ? pool_rank(l) : R;
    const ExpertBuffers b = expert_buffers(sh, R, T);
    uint8_t* v[3] = {mem + b.v[0], mem + b.v[1], mem + b.v[2]};
    uint16_t* hhi = reinterpret_cast<uint16_t*>(mem + b.h);
    uint16_t* hlo = reinterpret_cast<uint16_t*>(mem + b.h + align256((size_t)T * sh.d_ff * 2));
    hipError_t e;
    if (expert_tiles(sh.d_model, sh.d_ff, T) && tiles_reach(y, base)) {
        LoraGemmArgs g = {};
        g.x = x;
        g.Hin = g.Hout = hhi;
        g.Y = y;
        g.T = T;
        g.d = sh.d_model;
        g.f = sh.d_ff;
        g.x_bytes = (uint32_t)((int64_t)T * sh.d_model * 2);
        g.h_bytes = (uint32_t)((int64_t)T * sh.d_ff * 2);
        g.codes[0] = rec + rl.off_gate;
        g.codes[1] = rec + rl.off_up;
        g.scales[0] = rec + rl.off_sg;
        g.scales[1] = rec + rl.off_su;
        g.adapter = adapter;
        const Shrink gs = gemm_shrink(pools, 2, sh.d_model, T), ds = gemm_shrink(pools + 2, 1, sh.d_ff, T);
        gemm_pools(g, pools, v, 2, gs.parts);
        if ((e = shrink(pools, v, 2, adapter, x, nullptr, T, sh.d_model, true, gs, st)) != hipSuccess) return e;
        if ((e = launch_lora_gemm(sh.fmt, true, g, st)) != hipSuccess) return e;
        g.codes[0] = rec + rl.off_down;
        g.scales[0] = rec + rl.off_sd;
        g.base = base;
        gemm_pools(g, pools + 2, v + 2, 1, ds.parts);
        if ((e = shrink(pools + 2, v + 2, 1, adapter, hhi, nullptr, T, sh.d_ff, true, ds, st)) != hipSuccess) return e;
        return launch_lora_gemm(sh.fmt, false, g, st);
    }
    ProjectArgs a = {};
    a.codes[0] = rec + rl.off_gate;
    a.codes[1] = rec + rl.off_up;
    a.scales[0] = rec + rl.off_sg;
    a.scales[1] = rec + rl.off_su;
    a.adapter = adapter;
    a.xhi = x;
    a.T = T;
    a.n = sh.d_ff;
    a.K = sh.d_model;
    a.part = reinterpret_cast<float*>(mem + b.part);
    a.counters = reinterpret_cast<uint32_t*>(ws->mem);
    a.hhi = hhi;
    a.hlo = hlo;
    if ((e = product<2, 1>(sh.fmt, a, pools, v, st)) != hipSuccess) return e;
    ProjectArgs c = {};
    c.codes[0] = rec + rl.off_down;
    c.scales[0] = rec + rl.off_sd;
    c.adapter = adapter;
    c.xhi = hhi;
    c.xlo = hlo;
    c.T = T;
    c.n = sh.d_model;
    c.K = sh.d_ff;
    c.part = a.part;
    c.counters = a.counters;
    c.base = base;
    c.y = y;
    return product<1, 2>(sh.fmt, c, pools + 2, v + 2, st);
}

}  // namespace ftmoe
