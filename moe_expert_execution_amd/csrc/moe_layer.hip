// A whole mixture-of-experts layer for a few tokens over resident records:
//
//   z = x Wr (fp64), ids = top-k of z, w = softmax over the chosen k,
//   y[t] = base[t] + sum_j w[t, j] FFN_{ids[t, j]}(x[t]),
//   FFN(x) = (silu(x Wg) * (x Wu)) Wd.
//
// The experts' records are read from where they lie (E records, `stride` bytes
// apart), once per tile of 16 or 32 of their routes; no control step, no planner
// and no host branch takes part.  The router picks k of the layer's experts per token ("Making Large
// MoE Models Practical on a Single Machine", section 1); the expert FFN reads
// a complete layer-expert record ("The Expert Cache That Follows the Router",
// section "One logical expert, two physical levels of memory").
#include "resident.h"

namespace ftmoe {
namespace {

using namespace rs;

// The hand-over counters of the experts' launch (below); the routing launch
// before it clears them.
constexpr int kShards = 8, kShardStep = 32;
constexpr int kDrawn = 0, kDone = kShards * kShardStep;              // words of `hand`
constexpr int kHandWords = 2 * kShards * kShardStep;
constexpr int kHandAt = 4096;                 // their place among the workspace's counters (after one per row panel)

// ---- routing ----------------------------------------------------------------------

constexpr int kRouteTokens = 8;           // tokens of one routing workgroup
constexpr int kRouteExperts = 64;         // experts of one routing workgroup

// Rows of the router one wave takes: short slices while the workgroups fit the
// card twice over, so that the loads are all in flight at once.  Groups of 8
// tokens, not the 16 of a matrix-core tile: a group's last workgroup sums and
// selects for all its tokens, one a wave (with 16 that took longer than the
// product); groups of 4 double the product, which bounds 64 tokens.
inline int route_rows(int d, int E, int T) {
    const int64_t groups = (int64_t)((E + kRouteExperts - 1) / kRouteExperts) * ((T + kRouteTokens - 1) / kRouteTokens);
    int rows = 32;
    while (rows < 128 && groups * (d / (kWaves * rows)) > 512) rows *= 2;
    return rows;
}
inline int route_slices(int d, int E, int T) {
    const int per = kWaves * route_rows(d, E, T);
    return (d + per - 1) / per;
}

struct RouteArgs {
    const uint16_t* x;
    const uint16_t* wr;
    int T, d, E, k, rows, slices;
    double* part;          // [slices][T][E]
    uint32_t* counters;    // one per token group
    uint32_t* hand;        // the next launch's hand-over counters
    int32_t* ids;
    float* w;
};

// The largest of the 64 lanes' values.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xF, 0xF, false);
    return o > v ? o : v;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = dpp_max<0x111>(v);        // row_shr 1, 2, 4, 8: the largest of each 16 lanes in its last
    v = dpp_max<0x112>(v);
    v = dpp_max<0x114>(v);
    v = dpp_max<0x118>(v);
    v = dpp_max<0x142>(v);        // row_bcast 15, 31: across the four rows, in lane 63
    v = dpp_max<0x143>(v);
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// One wave picks the k largest of a token's E <= 64 V logits z (LDS), ties to
// the lower expert, and writes ids and the softmax of the chosen.  The order is
// that of 64-bit keys rising with the logit (-0 equals +0), found by their high
// words first; a NaN ranks as minus infinity, so there are always k experts to
// take.
template <int V>
__device__ __forceinline__ void select_experts(const double* z, int E, int k, int lane, int32_t* ids, float* w) {
    uint32_t hi[V], lo[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int e = lane + 64 * j;
        hi[j] = lo[j] = 0;
        if (e < E) {
            const double v = z[e] == z[e] ? z[e] + 0.0 : -INFINITY;
            uint64_t b = (uint64_t)__double_as_longlong(v);
            b = (b >> 63) ? ~b : b | (1ull << 63);
            hi[j] = (uint32_t)(b >> 32);
            lo[j] = (uint32_t)b;
        }
    }
    int mine = 0;                  // lane r keeps the r-th expert
    for (int r = 0; r < k; ++r) {
        uint32_t m = hi[0];
#pragma unroll
        for (int j = 1; j < V; ++j) m = hi[j] > m ? hi[j] : m;
        m = wave_max(m);
        uint64_t b[V];
        int n = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            b[j] = __ballot(hi[j] == m);
            n += __popcll(b[j]);
        }
        if (n > 1) {               // equal high words: the largest low word, then the lowest expert
            uint32_t l = 0;
#pragma unroll
            for (int j = 0; j < V; ++j) l = hi[j] == m && lo[j] > l ? lo[j] : l;
            l = wave_max(l);
#pragma unroll
            for (int j = 0; j < V; ++j) b[j] = __ballot(hi[j] == m && lo[j] == l);
        }
        int e = -1;
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (e < 0 && b[j]) e = 64 * j + __builtin_ctzll(b[j]);
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (lane + 64 * j == e) hi[j] = lo[j] = 0;
        if (lane == r) mine = e;
    }
    const double ex = exp(z[mine] - z[__builtin_amdgcn_readfirstlane(mine)]);
    const uint64_t eb = (uint64_t)__double_as_longlong(ex);
    double sum = 0.0;
    for (int r = 0; r < k; ++r)
        sum += __longlong_as_double((long long)(((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(eb >> 32), r) << 32) |
                                                (uint32_t)__builtin_amdgcn_readlane((int)eb, r)));
    if (lane < k) {
        ids[lane] = mine;
        w[lane] = (float)(ex / sum);
    }
}

// W = 32: a + its other half's in the lower half of the wave, the same of b in the
// upper; W = 16: in the even and odd rows of 16 lanes.
template <int W>
__device__ __forceinline__ double add_halves(double a, double b) {
    const uint64_t x = (uint64_t)__double_as_longlong(a), y = (uint64_t)__double_as_longlong(b);
    uint32_t p[2], q[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t u = (uint32_t)(x >> (32 * i)), v = (uint32_t)(y >> (32 * i));
        const auto r = W == 32 ? __builtin_amdgcn_permlane32_swap(u, v, false, false)
                               : __builtin_amdgcn_permlane16_swap(u, v, false, false);
        p[i] = r[0];
        q[i] = r[1];
    }
    return __longlong_as_double((long long)(p[0] | ((uint64_t)p[1] << 32))) +
           __longlong_as_double((long long)(q[0] | ((uint64_t)q[1] << 32)));
}

// Workgroup (slice of d, 64 experts, 8 tokens): partial logits on the fp64
// matrix cores (bf16 products are exact in fp64, sums are fp64).  Per 32 rows
// lane group g = l / 16 takes rows 8 g .. 8 g + 7, so MFMA step s contracts
// rows 8 g + s; column c = l % 16 of tile n is expert 4 c + n, so one 8-byte
// load gives a lane its four tiles' weights of a row, and one 16-byte load its
// token's 8 activations.  The waves' sums are added in order, and the group's
// last workgroup adds the slices in order and selects, one wave per token
// (a single token's slices are added by the experts' launch: sending them on is
// quicker than waiting for them here).
//
// NT: up to 8 tokens by vector FMAs instead (0: the matrix cores).  A lane sums its
// rows and four experts for each token, and the four lane groups' sums are added
// by exchanging halves.  An fp64 matrix product takes the time of 16 tokens, 2,048
// cycles for 32 rows and 64 experts, whatever there are: one token on 128 experts
// takes 4.1 us and 4.9 with it, on 8 experts 2.9 and 4.7; 5 tokens on 256 experts
// of d = 4,096 12.3 and 12.6.
//
// Latency decides those; of the 5 tokens' time more than half is the last
// workgroup's: the slices (164 KB to one compute unit) and the selection.  16
// tokens on 128 experts take 9.8 us, 64 on 256 experts of d = 7,168 28 to 33 (0.23
// GFLOP: 8 TFLOP/s in fp64, half of each product's rows unused).
template <int NT>
__global__ void __launch_bounds__(kThreads, 2) layer_route_kernel(RouteArgs a) {
    extern __shared__ __attribute__((aligned(16))) double zred[];
    __shared__ uint32_t flag;
    typedef double f64x4 __attribute__((ext_vector_type(4)));
    typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
    const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
    const int g = lane >> 4, c = lane & 15;
    const int slice = blockIdx.x, e0 = blockIdx.y * kRouteExperts, t0 = blockIdx.z * kRouteTokens;
    const int nt = min(kRouteTokens, a.T - t0);
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
        for (int i = tid; i < kHandWords; i += kThreads) a.hand[i] = 0;
    const int k0 = (slice * kWaves + wid) * a.rows, k1 = min(a.d, k0 + a.rows);
    const int e4 = e0 + 4 * c;
    const bool vec = (a.E & 3) == 0;      // rows of the router aligned for 8-byte loads
    constexpr int XT = NT ? NT : 1;       // tokens a lane loads
    f64x4 acc[NT ? NT : 4];               // [token] of the four experts, or [tile]
#pragma unroll
    for (f64x4& v : acc) v = f64x4{0.0, 0.0, 0.0, 0.0};
    const uint16_t* xrow = a.x + (int64_t)(t0 + (NT ? 0 : min(c, nt - 1))) * a.d + 8 * g;
    constexpr int D = 2;
    u32x4_t xv[D][XT];
    u32x2_t wv[D][8];
    auto load = [&](int b, int i) {
        const int kk = k0 + 32 * i;
#pragma unroll
        for (int t = 0; t < XT; ++t)
            if (t < nt) xv[b][t] = *reinterpret_cast<const u32x4_t*>(xrow + (int64_t)t * a.d + kk);
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            const uint16_t* p = a.wr + (int64_t)(kk + 8 * g + s) * a.E + e4;
            wv[b][s] = u32x2_t{0u, 0u};
            if (vec) {
                if (e4 < a.E) wv[b][s] = *reinterpret_cast<const u32x2_t*>(p);
            } else {
                uint32_t h[4];
#pragma unroll
                for (int n = 0; n < 4; ++n) h[n] = e4 + n < a.E ? p[n] : 0u;
                wv[b][s] = u32x2_t{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
            }
        }
    };
    auto work = [&](int b, int) {
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            double wd[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const uint32_t u = wv[b][s][n >> 1];
                wd[n] = (double)((n & 1) ? bf16hi(u) : bf16lo(u));
            }
#pragma unroll
            for (int t = 0; t < XT; ++t) {
                if (t >= nt) break;
                const uint32_t xw = xv[b][t][s >> 1];
                const double xd = (double)((s & 1) ? bf16hi(xw) : bf16lo(xw));
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    if constexpr (NT) acc[t][n] = fma(xd, wd[n], acc[t][n]);
                    else acc[n] = __builtin_amdgcn_mfma_f64_16x16x4f64(xd, wd[n], acc[n], 0, 0, 0);
                }
            }
        }
    };
    pipelined<D>(max(k1 - k0, 0) / 32, load, work);
    if constexpr (NT) {
        // value i = 4 t + n: the halves of the wave keep i and i + 2 NT, then the rows i and i + NT
        double v[4 * NT];
#pragma unroll
        for (int i = 0; i < 4 * NT; ++i) v[i] = acc[i / 4][i % 4];
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i) v[i] = add_halves<32>(v[i], v[i + 2 * NT]);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const double z = add_halves<16>(v[i], v[i + NT]);
            const int at = i + (g & 1) * NT + (g >> 1) * 2 * NT, t = at >> 2;
            if (t < nt) zred[(wid * nt + t) * kRouteExperts + 4 * c + (at & 3)] = z;
        }
    } else {
        // accumulator element v of lane l: token 4 v + l / 16, expert 4 (l % 16) + n
#pragma unroll
        for (int v = 0; v < kRouteTokens / 4; ++v) {
            const int t = 4 * v + g;
            if (t < nt)
#pragma unroll
                for (int n = 0; n < 4; ++n) zred[(wid * nt + t) * kRouteExperts + 4 * c + n] = acc[n][v];
        }
    }
    __syncthreads();
    for (int i = tid; i < nt * kRouteExperts; i += kThreads) {
        const int t = i / kRouteExperts, e = e0 + i % kRouteExperts;
        double s = 0.0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) s += zred[w * nt * kRouteExperts + i];
        if (e < a.E) put_agent(a.part + ((int64_t)slice * a.T + t0 + t) * a.E + e, s);
    }
    if (a.T == 1) return;                 // the experts' launch selects
    if (!last_arrival(a.counters + blockIdx.z, a.slices * gridDim.y, &flag)) return;

    const int n = nt * a.E;
    const double* p = a.part + (int64_t)t0 * a.E;
    const int64_t step = (int64_t)a.T * a.E;
    for (int i = tid; i < n; i += kThreads) {
        double s = 0.0;
#pragma unroll 8
        for (int q = 0; q < a.slices; ++q) s += get_agent(p + q * step + i);
        zred[i] = s;
    }
    __syncthreads();
    static_assert(kRouteTokens <= kWaves, "a token a wave");
    if (wid < nt) {
        const double* z = zred + wid * a.E;
        const int64_t o = (int64_t)(t0 + wid) * a.k;
        if (a.E <= 64) select_experts<1>(z, a.E, a.k, lane, a.ids + o, a.w + o);
        else if (a.E <= 128) select_experts<2>(z, a.E, a.k, lane, a.ids + o, a.w + o);
        else select_experts<4>(z, a.E, a.k, lane, a.ids + o, a.w + o);
    }
}

// ---- the routed experts --------------------------------------------------------------

constexpr int kMaxRoutes = kMaxLayerTokens * kMaxTopK;       // 1024
constexpr int kMaxTiles = kMaxRouteExperts + kMaxRoutes / (kCols + 1);

struct ExpertArgs {
    const double* logits;  // [slices][E] of a single token (ONE)
    int slices;
    const uint16_t* x;
    const uint8_t* rec;
    int64_t stride, off_gate, off_up, off_down, off_sg, off_su, off_sd;
    int32_t* ids;          // (written by the ONE launch)
    float* w;
    const uint16_t* base;
    uint16_t* y;
    uint16_t* hhi;         // [T k][f] h as two bf16 planes
    uint16_t* hlo;
    float* part;           // [splits][T][d] (splits > 1)
    uint32_t* counters;    // one per workgroup of row panels of WdT
    uint32_t* hand;        // the launch's hand-over counters, zero at its start
    uint32_t polls, low_polls;   // bounds of the hand-over's wait (ft_workspace)
    int absent;                  // odd workgroups draw no number when they start (ft_workspace)
    int T, E, k, d, f, splits;
};

// A tile: routes of one expert, as many as its kernel's operands hold.
struct Tile {
    int e, first, nt;      // expert, first place in Groups::route, count
};

// The call's routes grouped by expert, in LDS.  A token names an expert at most
// once, so an expert's tokens are a 64-bit mask, and its routes lie in token
// order: every workgroup finds the same tiles.
struct Groups {
    unsigned long long mask[kMaxRouteExperts];   // tokens routed to the expert
    int start[kMaxRouteExperts];                 // first of its routes in `route`
    int n_tiles;
    uint32_t tile[kMaxTiles];                    // by expert: e | first << 8 | nt << 18
    uint16_t route[kMaxRoutes];                  // routes t k + j by expert

    __device__ __forceinline__ Tile at(int i) const {
        const uint32_t v = __builtin_amdgcn_readfirstlane(tile[i]);
        return Tile{(int)(v & 255), (int)((v >> 8) & 1023), (int)(v >> 18)};
    }
};

// Every thread of the workgroup calls it; tiles of up to W routes.
template <int W>
__device__ __forceinline__ void group_routes(Groups& g, const int32_t* ids, int T, int E, int k) {
    constexpr int PT = kMaxRoutes / kThreads;
    const int tid = threadIdx.x, lane = tid & 63, R = T * k;
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
        int base = 0, tiles = 0;
        for (int e0 = 0; e0 < E; e0 += 64) {
            const int e = e0 + lane;
            const int c = e < E ? __popcll(g.mask[e]) : 0;
            const int tl = (c + W - 1) / W;
            int sc = c, st = tl;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int a0 = __shfl_up(sc, o, 64), b0 = __shfl_up(st, o, 64);
                if (lane >= o) {
                    sc += a0;
                    st += b0;
                }
            }
            if (c > 0) {
                const int first = base + sc - c;
                g.start[e] = first;
                for (int q = 0; q < tl; ++q)
                    g.tile[tiles + st - tl + q] = (uint32_t)e | ((uint32_t)(first + q * W) << 8) |
                                                  ((uint32_t)min(W, c - q * W) << 18);
            }
            base += __shfl(sc, 63, 64);
            tiles += __shfl(st, 63, 64);
        }
        if (lane == 0) g.n_tiles = tiles;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PT; ++i) {
        const int r = tid + i * kThreads;
        if (r < R) g.route[g.start[id[i]] + __popcll(g.mask[id[i]] & ((1ull << tok[i]) - 1))] = (uint16_t)r;
    }
    __syncthreads();
}

// A single token: adds its logits' slices, selects, and makes a tile of each
// route; workgroup 0 writes the outputs.  Every thread of the workgroup calls
// it; `z` is scratch for E logits.
__device__ __forceinline__ void select_one(Groups& g, float* wr, double* z, const ExpertArgs& a) {
    __shared__ int32_t ids[kMaxTopK];
    const int tid = threadIdx.x, lane = tid & 63;
    if (tid < a.E) {
        double s = 0.0;
        for (int q = 0; q < a.slices; q += 16) {
            double v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = a.logits[(int64_t)(q + i < a.slices ? q + i : q) * a.E + tid];
#pragma unroll
            for (int i = 0; i < 16; ++i) s += q + i < a.slices ? v[i] : 0.0;
        }
        z[tid] = s;
    }
    __syncthreads();
    if (tid < 64) {
        if (a.E <= 64) select_experts<1>(z, a.E, a.k, lane, ids, wr);
        else if (a.E <= 128) select_experts<2>(z, a.E, a.k, lane, ids, wr);
        else select_experts<4>(z, a.E, a.k, lane, ids, wr);
        if (lane < a.k) {
            g.tile[lane] = (uint32_t)ids[lane] | ((uint32_t)lane << 8) | (1u << 18);
            g.route[lane] = (uint16_t)lane;
            if (blockIdx.x == 0) {
                a.ids[lane] = ids[lane];
                a.w[lane] = wr[lane];
            }
        }
        if (lane == 0) g.n_tiles = a.k;
    }
    __syncthreads();
}

// ---- the hand-over from gate/up to down inside a launch ---------------------------------
//
// h of every route is needed by every down workgroup, so those wait until all
// gate/up work is done.  The wait always ends, whatever part of the grid is
// running and whatever else runs on the device: gate/up work is bound to
// numbers, not to workgroups.  A workgroup draws the number of its own shard
// when it starts; one that waits also looks for numbers that nobody has drawn
// (their workgroups may not have started, and may not start before this one
// ends) and does their work itself.  So when a workgroup waits with nothing
// left to draw, every number is in the hands of a running workgroup that does
// not wait.  Counters lie 128 bytes apart in kShards shards: 256 arrivals on
// one address take 3 us, on eight of them a third of one.

// Numbers of a shard in a grid of n.
__device__ __forceinline__ uint32_t shard_size(int shard, int n) { return (uint32_t)((n - shard + kShards - 1) / kShards); }

__device__ __forceinline__ uint32_t draw(uint32_t* hand, int shard) {
    return __hip_atomic_fetch_add(hand + kDrawn + shard * kShardStep, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// One wave: waits until all numbers are done (returns -1), or returns a number
// that it has drawn for an absent workgroup (>= 0), or gives up (-2).
__device__ __forceinline__ int wait_done(uint32_t* hand, int n, uint32_t polls, int lane) {
    const int shard = lane & (kShards - 1);
    const uint32_t size = shard_size(shard, n);
    for (uint32_t i = 0; i < polls; ++i) {
        const uint32_t drawn = __hip_atomic_load(hand + kDrawn + shard * kShardStep, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        const uint32_t done = __hip_atomic_load(hand + kDone + shard * kShardStep, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (__ballot(done < size) == 0) return -1;
        const uint64_t open = __ballot(drawn < size);
        if (open) {
            const int s = __builtin_ctzll(open) & (kShards - 1);
            uint32_t v = 0;
            if (lane == 0) v = draw(hand, s);
            v = __builtin_amdgcn_readfirstlane(v);
            if (v < shard_size(s, n)) return (int)v * kShards + s;
        }
        __builtin_amdgcn_s_sleep(1);
    }
    return -2;
}

// The waves' sums of a tile's gate and up panels p, SwiGLU, h.
template <int NX>
__device__ __forceinline__ void store_h(const ExpertArgs& a, const Groups& g, float* red, const Tile& t, int p, Acc (&ag)[NX],
                                        Acc (&au)[NX]) {
    const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
    const int half = kWaves * t.nt * kRedRow;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NX; ++i) {
        put_acc(red, ag[i], i, wid, t.nt, lane);
        put_acc(red + half, au[i], i, wid, t.nt, lane);
        ag[i] = au[i] = zero_acc();
    }
    __syncthreads();
    float gs[kPlaces], us[kPlaces];
    sum_waves(gs, red, t.nt, tid);
    sum_waves(us, red + half, t.nt, tid);
#pragma unroll
    for (int i = 0; i < kPlaces; ++i) {
        const int m = (tid + i * kThreads) >> 5;
        // h in 16 significant bits: its rounding stays far below that of y.  Two
        // neurons a store, past the L2 that other XCDs do not see: the even
        // lane's for the high halves, the odd lane's for the low ones.
        uint16_t h, l;
        split_bf16(silu(gs[i]) * us[i], h, l);
        const uint32_t mine = (uint32_t)h | ((uint32_t)l << 16);
        const uint32_t other = (uint32_t)__shfl_xor((int)mine, 1, 64);
        if (m < t.nt) {
            const bool odd = tid & 1;
            const int64_t o = (int64_t)g.route[t.first + m] * a.f + p * 32 + (tid & 30);
            const uint32_t v = odd ? (other >> 16) | (mine & 0xFFFF0000u) : (mine & 0xFFFFu) | (other << 16);
            __hip_atomic_store(reinterpret_cast<uint32_t*>((odd ? a.hlo : a.hhi) + o), v, __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
        }
    }
}

// Gate/up and SwiGLU: number v does the items (tile, 32 neurons) v, v + grid,
// ...; the waves split K = d.  The next unit's loads are in flight while one is
// multiplied, across items too, so the stream does not stop for an item's
// sums.  64 tokens on 256 MXFP4 experts: 3.5 GB in 580 to 640 us, 5.4 to 6.0 TB/s.
template <int FMT, int NX>
__device__ __forceinline__ void layer_gateup(const ExpertArgs& a, const Groups& g, float* red, const int first_item) {
    const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6, grid = gridDim.x;
    const int panels = a.f >> 5, items = g.n_tiles * panels;
    const int units = a.d / kUnit;
    const int u0 = wid * units / kWaves, nu = (wid + 1) * units / kWaves - u0;
    const int steps = max(nu, 1);     // a wave without units (d < 1024) loads one and leaves it
    struct Cursor {
        int item, step;
        Tile t;
        PanelRef pg, pu;
        const uint16_t* x[NX];
    };
    auto enter = [&](Cursor& c, int item) {
        c.item = item;
        c.step = 0;
        const int tile = item / panels, p = item - tile * panels;
        c.t = g.at(tile);
        const uint8_t* rec = a.rec + (int64_t)c.t.e * a.stride;
        c.pg = panel_ref<FMT>(rec + a.off_gate, rec + a.off_sg, a.d, p);
        c.pu = panel_ref<FMT>(rec + a.off_up, rec + a.off_su, a.d, p);
        // lanes past the tile's routes repeat its last one: their columns are not stored
#pragma unroll
        for (int i = 0; i < NX; ++i)
            c.x[i] = a.x + (int64_t)(g.route[c.t.first + min(i * kCols + (lane & 15), c.t.nt - 1)] / a.k) * a.d;
    };
    WUnit<FMT> wg[2], wu[2];
    XUnit xu[2][NX][1];
    Cursor ld;                        // the next unit to load
    auto load = [&](int b) {
        const int u = min(u0 + ld.step, units - 1);
        load_unit<FMT>(wg[b], ld.pg, u, lane);
        load_unit<FMT>(wu[b], ld.pu, u, lane);
#pragma unroll
        for (int i = 0; i < NX; ++i)
            if (i == 0 || ld.t.nt > i * kCols) load_x<FMT>(xu[b][i][0], ld.x[i], u, lane);
        if (++ld.step == steps && ld.item + grid < items) enter(ld, ld.item + grid);
    };
    Acc ag[NX], au[NX];
    int item = first_item, step = 0;
    if (item >= items) return;
    enter(ld, item);
    load(0);
    Tile t = g.at(item / panels);
#pragma unroll
    for (int i = 0; i < NX; ++i) ag[i] = au[i] = zero_acc();
    // one step: unit `step` of `item`; after the item's last one its sums; true at the end
    auto advance = [&](int b) -> bool {
        if (step < nu) {
            const int nx = t.nt > kCols ? 2 : 1;
            mma_unit<FMT, NX, 1>(ag, wg[b], xu[b], nx);
            mma_unit<FMT, NX, 1>(au, wu[b], xu[b], nx);
        }
        if (++step < steps) return false;
        store_h<NX>(a, g, red, t, item % panels, ag, au);
        item += grid;
        if (item >= items) return true;
        step = 0;
        t = g.at(item / panels);
        return false;
    };
    // whether a step follows the current one
    auto more = [&]() { return step + 1 < steps || item + grid < items; };
    for (;;) {
        if (more()) load(1);
        if (advance(0)) return;
        if (more()) load(0);
        if (advance(1)) return;
    }
}

// The same, one load at a time: the part of an absent workgroup, which is hardly
// ever done, without the registers of a pipeline.  The same sums in the same
// order.
template <int FMT, int NX>
__device__ __forceinline__ void layer_gateup_absent(const ExpertArgs& a, const Groups& g, float* red, const int first_item) {
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
    const int panels = a.f >> 5, items = g.n_tiles * panels, units = a.d / kUnit;
    const int u0 = wid * units / kWaves, u1 = (wid + 1) * units / kWaves;
#pragma unroll 1
    for (int item = first_item; item < items; item += gridDim.x) {
        const int p = item % panels;
        const Tile t = g.at(item / panels);
        const uint8_t* rec = a.rec + (int64_t)t.e * a.stride;
        const PanelRef pg = panel_ref<FMT>(rec + a.off_gate, rec + a.off_sg, a.d, p);
        const PanelRef pu = panel_ref<FMT>(rec + a.off_up, rec + a.off_su, a.d, p);
        Acc ag[NX], au[NX];
#pragma unroll
        for (int i = 0; i < NX; ++i) ag[i] = au[i] = zero_acc();
#pragma unroll 1
        for (int u = u0; u < u1; ++u) {
            WUnit<FMT> w;
            XUnit x[NX][1];
#pragma unroll
            for (int i = 0; i < NX; ++i)
                load_x<FMT>(x[i][0], a.x + (int64_t)(g.route[t.first + min(i * kCols + (lane & 15), t.nt - 1)] / a.k) * a.d, u,
                            lane);
            load_unit<FMT>(w, pg, u, lane);
            mma_unit<FMT, NX, 1>(ag, w, x, NX);
            load_unit<FMT>(w, pu, u, lane);
            mma_unit<FMT, NX, 1>(au, w, x, NX);
        }
        store_h<NX>(a, g, red, t, p, ag, au);
    }
}

// A number's h is on its way past the L2 before the number counts as done.
__device__ __forceinline__ void number_done(uint32_t* hand, int number) {
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (threadIdx.x == 0)
        __hip_atomic_fetch_add(hand + kDone + (number % kShards) * kShardStep, 1u, __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
}

template <int NP>
constexpr int sum_row() { return 32 * NP + 4; }      // floats of a token's sums in LDS, padded

// Down and combine: items (NP row panels of WdT, split) go round the
// workgroups.  The tiles' K = f units form one axis, divided evenly over the
// splits and their waves.  A wave sums a tile's units with the tile's routes as
// columns, then adds w times the sum to its own [token][row] sums in LDS: a
// token's sums see the tiles in order, whatever else the tile holds, and a
// column past the tile's routes goes nowhere.  The waves' sums are added in
// order, and with several splits the panels' last workgroup adds the splits in
// order, so y does not depend on timing.  wait(again) is called once, before h
// is first read, with the first unit of weights on its way; where it has used
// the registers meanwhile it calls again().  It returns whether h is there: where
// it is not, the workgroup's part of y, or its partial sums, are NaN, so that y is
// NaN whichever workgroup adds the splits.
// 64 tokens on 256 MXFP4 experts: 1.7 GB in 323 to 354 us, 4.9 to 5.4 TB/s, the
// rest being the splits' four rounds of grouping, 64 tokens' sums and partial sums.
template <int FMT, int NX, int NP, typename Wait>
__device__ __forceinline__ void layer_down(const ExpertArgs& a, const Groups& g, const float* wr, float* red, uint32_t* flag,
                                           Wait&& wait) {
    constexpr int SR = sum_row<NP>();
    const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6, grid = gridDim.x;
    const int dwg = a.d / 32 / NP, ditems = dwg * a.splits;
    const int uf = a.f / kUnit, units = g.n_tiles * uf;
    bool there = true;
    for (int item = blockIdx.x; item < ditems; item += grid) {
        const int p0 = (item % dwg) * NP, split = item / dwg;
        const int part = split * kWaves + wid, parts = a.splits * kWaves;
        const int u0 = (int)((int64_t)part * units / parts), u1 = (int)((int64_t)(part + 1) * units / parts);
        struct Cursor {
            int tile, kk;
            Tile t;
            PanelRef pd[NP];
            int64_t h[NX];
        };
        auto enter = [&](Cursor& c, int tile) {
            c.tile = tile;
            c.kk = 0;
            c.t = g.at(tile);
            const uint8_t* rec = a.rec + (int64_t)c.t.e * a.stride;
#pragma unroll
            for (int n = 0; n < NP; ++n) c.pd[n] = panel_ref<FMT>(rec + a.off_down, rec + a.off_sd, a.f, p0 + n);
#pragma unroll
            for (int i = 0; i < NX; ++i)
                c.h[i] = (int64_t)g.route[c.t.first + min(i * kCols + (lane & 15), c.t.nt - 1)] * a.f;
        };
        WUnit<FMT> wd[2][NP];
        XUnit hu[2][NX][2];
        Cursor ld;                            // the next unit to load
        auto load_w = [&](int b) {
#pragma unroll
            for (int n = 0; n < NP; ++n) load_unit<FMT>(wd[b][n], ld.pd[n], ld.kk, lane);
        };
        auto load_h = [&](int b) {
#pragma unroll
            for (int i = 0; i < NX; ++i)
                if (i == 0 || ld.t.nt > i * kCols) {
                    load_x<FMT>(hu[b][i][0], a.hhi + ld.h[i], ld.kk, lane);
                    load_x<FMT>(hu[b][i][1], a.hlo + ld.h[i], ld.kk, lane);
                }
            if (++ld.kk == uf && ld.tile + 1 < g.n_tiles) enter(ld, ld.tile + 1);
        };
        auto first_w = [&]() {
            if (u0 < u1) {
                enter(ld, u0 / uf);
                ld.kk = u0 % uf;
                load_w(0);
            }
        };
        first_w();
        if (item == (int)blockIdx.x) there = wait(first_w);
        float* mine = red + wid * a.T * SR;
        for (int i = lane * 4; i < a.T * SR; i += 256) *reinterpret_cast<f32x4_t*>(mine + i) = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        if (u0 < u1) {
            Acc acc[NP][NX];
#pragma unroll
            for (int n = 0; n < NP; ++n)
#pragma unroll
                for (int i = 0; i < NX; ++i) acc[n][i] = zero_acc();
            int u = u0, tile = u0 / uf, kk = u0 - tile * uf;
            load_h(0);
            Tile t = g.at(tile);
            auto advance = [&](int b) -> bool {
                const int nx = t.nt > kCols ? 2 : 1;
#pragma unroll
                for (int n = 0; n < NP; ++n) mma_unit<FMT, NX, 2>(acc[n], wd[b][n], hu[b], nx);
                const bool last = ++u == u1;
                if (++kk < uf && !last) return false;
#pragma unroll
                for (int i = 0; i < NX; ++i) {
                    const int m = i * kCols + (lane & 15);
                    if (m < t.nt) {
                        const int r = g.route[t.first + m];
                        const float w = wr[r];
                        float* s = mine + (r / a.k) * SR + 4 * (lane >> 4);
#pragma unroll
                        for (int n = 0; n < NP; ++n)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                f32x4_t* q = reinterpret_cast<f32x4_t*>(s + 32 * n + 16 * h);
                                f32x4_t v = *q;
#pragma unroll
                                for (int e = 0; e < 4; ++e) v[e] = fmaf(w, acc[n][i].h[h][e], v[e]);
                                *q = v;
                            }
                    }
#pragma unroll
                    for (int n = 0; n < NP; ++n) acc[n][i] = zero_acc();
                }
                if (last) return true;
                kk = 0;
                t = g.at(++tile);
                return false;
            };
            auto next = [&](int b) {
                if (u + 1 < u1) {
                    load_w(b);
                    load_h(b);
                }
            };
            for (;;) {
                next(1);
                if (advance(0)) break;
                next(0);
                if (advance(1)) break;
            }
        }
        __syncthreads();
        auto emit = [&](int t, int n, float v) {
            const int64_t o = (int64_t)t * a.d + p0 * 32 + n;
            if (a.base) v += __uint_as_float((uint32_t)a.base[o] << 16);
            a.y[o] = f32_to_bf16_rne(v);
        };
        constexpr int C = 32 * NP;
        for (int i = tid; i < a.T * C; i += kThreads) {
            const int t = i / C, n = i % C;
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) s += red[(w * a.T + t) * SR + n];
            if (!there) s = __uint_as_float(0x7FC00000u);
            if (a.splits == 1) emit(t, n, s);
            else put_agent(a.part + ((int64_t)split * a.T + t) * a.d + p0 * 32 + n, s);
        }
        if (a.splits > 1 && last_arrival(a.counters + item % dwg, a.splits, flag)) {
            for (int i = tid; i < a.T * C; i += kThreads) {
                const int t = i / C, n = i % C;
                float s = 0.0f;
#pragma unroll 4
                for (int q = 0; q < a.splits; ++q) s += get_agent(a.part + ((int64_t)q * a.T + t) * a.d + p0 * 32 + n);
                emit(t, n, s);
            }
        }
        __syncthreads();
    }
}

// Up to 16 tokens: the routed experts and the combine in one launch.  A launch
// between gate/up and down costs 2.4 us and empties the card twice; here a
// workgroup without gate/up work, or done with it, has its down weights under
// way while it waits (the whole call on 128 bf16 experts of 2,048 x 768: 147 us
// with two launches, 137 in one at 16 tokens; 30.7 and 27.8 at one).
// ONE: a single token, selected here (27.7 and 26.4 us).
//
// Bound by HBM: 779 MB of records and router at 16 tokens in 126 us are 6.2 TB/s,
// what a large read reaches; 947 MB of 40 FP8 experts in 162 us 5.8 TB/s.  At one
// token (75 MB, 21.7 us) and in small layers by latency: grouping or selection,
// the first weights, two sums over waves, the hand-over and the sum over splits.
template <int FMT, int NP, bool ONE>
__global__ void __launch_bounds__(kThreads, 2) layer_experts_kernel(ExpertArgs a) {
    extern __shared__ __attribute__((aligned(16))) float red[];     // the waves' sums of either half
    __shared__ Groups g;
    __shared__ float wr[kMaxRoutes];
    __shared__ uint32_t flag;
    __shared__ int number;
    const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
    const int grid = gridDim.x;
    if (tid == 0) {
        const int shard = blockIdx.x % kShards;
        const uint32_t v = a.absent && (blockIdx.x & 1) ? ~0u : draw(a.hand, shard);
        number = v < shard_size(shard, grid) ? (int)v * kShards + shard : -1;
    }
    if constexpr (ONE) {
        select_one(g, wr, reinterpret_cast<double*>(red), a);
    } else {
        for (int r = tid; r < a.T * a.k; r += kThreads) wr[r] = a.w[r];
        group_routes<kCols>(g, a.ids, a.T, a.E, a.k);
    }
    const int mine = number;
    if (mine >= 0) {
        layer_gateup<FMT, 1>(a, g, red, mine);
        number_done(a.hand, mine);
    }
    layer_down<FMT, 1, NP>(a, g, wr, red, &flag, [&](auto&& again) -> bool {
        auto poll = [&]() -> int {
            __syncthreads();
            if (wid == 0) {
                const int r = wait_done(a.hand, grid, (int)blockIdx.x < grid / 2 ? a.low_polls : a.polls, lane);
                if (lane == 0) number = r;
            }
            __syncthreads();
            return number;
        };
        int r = poll();
        if (r >= 0) {                         // do absent workgroups' parts first, then load again
            do {
                layer_gateup_absent<FMT, 1>(a, g, red, r);
                number_done(a.hand, r);
                r = poll();
            } while (r >= 0);
            again();
        }
        // h is read through the caches from here on: no XCD holds an older copy of it,
        // since a launch starts with its caches invalidated and nothing of it reads h
        // before this.  (An agent-scope fence would invalidate the XCD's L2 once per
        // wave; the down half took 14 us more with one.)
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
        return r == -1;
    });
}

// More tokens: two launches.  (In one, most of these calls gained 0 to 3%, and 64
// tokens on 128 MXFP4 experts of d = 2,048 took 110 us instead of 96: their many
// down items go one after the other through the workgroups that gate/up left.)
template <int FMT, int NX>
__global__ void __launch_bounds__(kThreads, 2) layer_gateup_kernel(ExpertArgs a) {
    extern __shared__ __attribute__((aligned(16))) float red[];
    __shared__ Groups g;
    group_routes<NX * kCols>(g, a.ids, a.T, a.E, a.k);
    layer_gateup<FMT, NX>(a, g, red, blockIdx.x);
}
template <int FMT, int NX, int NP>
__global__ void __launch_bounds__(kThreads, 2) layer_down_kernel(ExpertArgs a) {
    extern __shared__ __attribute__((aligned(16))) float red[];
    __shared__ Groups g;
    __shared__ float wr[kMaxRoutes];
    __shared__ uint32_t flag;
    for (int r = threadIdx.x; r < a.T * a.k; r += kThreads) wr[r] = a.w[r];
    group_routes<NX * kCols>(g, a.ids, a.T, a.E, a.k);
    layer_down<FMT, NX, NP>(a, g, wr, red, &flag, [](auto&&) { return true; });
}

// Tiles of 16 routes instead of 32 (more than 16 tokens).  The second operand
// costs registers (28 spilled in MXFP4's down, 21 in bf16, 6 in FP8) whether a tile fills it
// or not: 64 tokens on 256 MXFP4 experts (2 routes each) take 930 us and 1,085
// with 32, 64 on 128 bf16 experts (4) 199 and 235, 64 on 8 (16) 41 and 43.  An
// expert with more than 16 routes reads its weights again, from L2 at best: with
// 32 routes each, 8 FP8 experts take 116 us and 105 with tiles of 32, 8 MXFP4
// experts at 64 each 188 and 174.
bool narrow_tiles(const ft_shape& s, int T) { return (int64_t)T * s.top_k <= 16ll * s.experts; }

// Row panels per down workgroup.  The h loads beside an MXFP4 panel outweigh its
// codes fourfold, so two panels share them once there are experts enough to
// fill the card all the same (d = 7,168, 256 experts: 170 us and 180 with one at 4
// tokens, 945 and 1,071 at 64; d = 2,048, 128 experts: 29.8 and 28.9 at 2 tokens).
int down_panels(const ft_shape& s, int T) {
    return s.fmt == FT_FMT_MXFP4_B32 && (int64_t)T * s.top_k >= 32 ? 2 : 1;
}

// Splits of the tiles' axis.  A compute unit holds one workgroup, so the launch
// takes ceil(workgroups / 256) rounds of a split's share each; more splits even
// that out (224 panels of d = 7,168 in pairs: 3 splits take 2 rounds of a third
// each, 9 take 4 of a ninth), and each costs its partial sums, written and read
// once.  The times are estimates at 25 GB/s per workgroup and 4 TB/s; no more
// splits than leave each wave a unit when every route has an expert of its own.
int down_splits(const ft_shape& s, int T) {
    const int np = down_panels(s, T), wgs = s.d_model / 32 / np;
    const int64_t R = (int64_t)T * s.top_k, tiles = R < s.experts ? R : s.experts;
    const int64_t units = tiles * (s.d_ff / kUnit);
    const double unit_bytes = s.fmt == FT_FMT_BF16 ? 8192 : s.fmt == FT_FMT_FP8_B128 ? 4096 : 2176;
    const double stream = units * np * unit_bytes / 25e3, join = (double)T * s.d_model * 8 / 4e6;     // us
    int best = 1;
    double least = 1e30;
    for (int n = 1; n <= 16 && (n == 1 || (int64_t)(n - 1) * kWaves < units); ++n) {
        const double t = (double)((wgs * n + 255) / 256) * stream / n + (n > 1 ? 2.0 + n * join : 0.0);
        if (t < least) {
            least = t;
            best = n;
        }
    }
    return best;
}

constexpr size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

struct LayerBuffers {
    size_t part, hhi, hlo, logits, total;
};
LayerBuffers layer_buffers(const ft_shape& s, int T) {
    LayerBuffers b;
    const size_t R = (size_t)T * s.top_k;
    b.logits = 0;
    b.hhi = align256((size_t)route_slices(s.d_model, s.experts, T) * T * s.experts * sizeof(double));
    b.hlo = b.hhi + align256(R * s.d_ff * 2);
    b.part = b.hlo + align256(R * s.d_ff * 2);
    b.total = b.part + align256((size_t)down_splits(s, T) * T * s.d_model * sizeof(float));
    return b;
}

template <int FMT>
hipError_t launch_fmt(const ft_shape& s, const RouteArgs& r, const ExpertArgs& a, hipStream_t st) {
    const dim3 rg(r.slices, (r.E + kRouteExperts - 1) / kRouteExperts, (r.T + kRouteTokens - 1) / kRouteTokens);
    const int rt = r.T < kRouteTokens ? r.T : kRouteTokens;
    // the waves' partial logits, then whole rows
    static_assert(kWaves * kRouteExperts >= kMaxRouteExperts, "a token's logits fit its partial sums' place");
    const auto route = r.T == 1 ? layer_route_kernel<1> : r.T <= kRouteTokens ? layer_route_kernel<kRouteTokens> : layer_route_kernel<0>;
    hipError_t e = launch(route, rg, dim3(kThreads), (size_t)rt * kWaves * kRouteExperts * sizeof(double), st, r);
    if (e != hipSuccess) return e;

    const int R = a.T * a.k;
    const int tiles = (R < a.E ? R : a.E) + R / (kCols + 1);       // at most, whatever the tiles' width
    const int64_t items = (int64_t)tiles * (a.f / 32);
    const int np = down_panels(s, a.T);
    const int64_t ditems = (int64_t)(a.d / 32 / np) * a.splits;
    const int nt = a.T < kTile ? a.T : kTile;
    const size_t glds = (size_t)2 * kWaves * nt * kRedRow * sizeof(float);
    const size_t dlds = (size_t)kWaves * a.T * (32 * np + 4) * sizeof(float);
    auto blocks = [](int64_t n) { return dim3((unsigned)(n < 256 ? n : 256)); };
    if (a.T <= kCols) {                   // every tile fits one operand
        const dim3 grid = blocks(items > ditems ? items : ditems);
        const size_t lds = glds > dlds ? glds : dlds;
        if (a.T == 1) {
            const size_t z = kMaxRouteExperts * sizeof(double);
            return launch(layer_experts_kernel<FMT, 1, true>, grid, dim3(kThreads), lds > z ? lds : z, st, a);
        }
        const auto f = np == 2 ? layer_experts_kernel<FMT, FMT == FT_FMT_MXFP4_B32 ? 2 : 1, false>
                               : layer_experts_kernel<FMT, 1, false>;
        return launch(f, grid, dim3(kThreads), lds, st, a);
    }
    const bool narrow = narrow_tiles(s, a.T);
    const auto gu = narrow ? layer_gateup_kernel<FMT, 1> : layer_gateup_kernel<FMT, 2>;
    e = launch(gu, blocks(items), dim3(kThreads), glds, st, a);
    if (e != hipSuccess) return e;
    constexpr int P2 = FMT == FT_FMT_MXFP4_B32 ? 2 : 1;
    const auto dn = narrow ? (np == 2 ? layer_down_kernel<FMT, 1, P2> : layer_down_kernel<FMT, 1, 1>)
                           : (np == 2 ? layer_down_kernel<FMT, 2, P2> : layer_down_kernel<FMT, 2, 1>);
    return launch(dn, dim3((unsigned)ditems), dim3(kThreads), dlds, st, a);
}

}  // namespace

size_t layer_call_bytes(const ft_shape& s, int T) { return layer_buffers(s, T).total; }

// the largest need of any call of up to T tokens (fewer tokens may take more slices)
size_t layer_workspace(const ft_shape& s, int T) {
    size_t most = 0;
    for (int t = 1; t <= T; ++t) {
        const size_t b = layer_call_bytes(s, t);
        most = b > most ? b : most;
    }
    return most;
}

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
    r.rows = route_rows(s.d_model, s.experts, la.T);
    r.slices = route_slices(s.d_model, s.experts, la.T);
    r.part = reinterpret_cast<double*>(m + b.logits);
    r.counters = counters;
    r.hand = counters + kHandAt;
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
    a.logits = r.part;
    a.slices = r.slices;
    a.base = la.base;
    a.y = la.y;
    a.hhi = reinterpret_cast<uint16_t*>(m + b.hhi);
    a.hlo = reinterpret_cast<uint16_t*>(m + b.hlo);
    a.part = reinterpret_cast<float*>(m + b.part);
    a.counters = counters + kMaxLayerTokens;
    a.hand = counters + kHandAt;
    a.polls = kMaxPolls;
    a.low_polls = ws->low_polls;
    a.absent = ws->absent;
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
