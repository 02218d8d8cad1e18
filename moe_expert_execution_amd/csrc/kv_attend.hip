// Attention of one new token per request over a paged key-value cache
// (ft_kv_attend):  out = sum_t exp(s_t) v_t / sum_t exp(s_t), s_t = scale q . k_t.
//
// The query heads that share a KV head are the columns of one matrix-core operand,
// so a page is read once for all of them.  S^T = K Q^T takes 16 tokens of keys as the
// A operand straight from memory (the cache's unit order is that operand's order) and
// leaves lane l with column l % 16 and tokens 4 (l / 16) .. + 3 of each of two blocks.
// The order of a product's contraction is free, so these very registers are the B
// operand of O^T += V^T P^T if V's lanes take the tokens in the same order: lane l
// loads tokens 4 (l / 16) .. + 3 of both blocks at its own dimensions (whole rows over
// the lanes) and transposes them in registers, one byte permute per pair.  So neither
// keys, values nor probabilities pass through LDS.
//
// Up to 8 query heads the operand's other 8 columns hold the same heads: columns 0 .. 7
// take each probability as bf16, 8 .. 15 its rest, and the two sums add up to
// 16 significant bits at no cost; wider groups take two products.  e4m3 codes become bf16
// exactly; the heads' scales multiply the logits and the result.
//
// Statistics are fp32, one running maximum and sum per column and wave, in base 2.  The
// work is divided as kv_rules.h says; memory bounds long contexts (64 requests of up to 8,192, 64/8 heads of 128, 649
// MB: 110 us, 5.9 TB/s; one of 131,072, 32/4 heads, 268 MB: 50 us, 5.4 TB/s), latency short ones (37 tokens in a table of 4
// pages 4.4 us).  (Times of launches; those in kv_rules.h are of calls in a captured graph.)
#include "kv_device.h"
#include "resident.h"

namespace ftmoe {
namespace {

using rs::last_arrival;
constexpr float kLog2e = 1.44269504088896340736f;

struct AttendArgs {
    CacheView c;
    ft_attend a;
    int g, blocks;            // query heads per KV head, items per KV head
    float* part;              // partial results: two per team
    uint32_t part_bytes;
    uint32_t* counters;       // one per team for its run, one for its item
};

// Agent-scope 16-byte access (sc1): a partial result crosses XCDs, whose L2s do not
// see each other.
constexpr int kAgent = 16;

constexpr uint32_t kRunStats = 2 * kv::kCols * 4;        // a run's statistics, behind its first part's

// A value that all lanes of the wave have, as a scalar.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

template <int D, int FMT>
struct Kv {
    static constexpr int E = FMT == FT_KV_BF16 ? 2 : 1;
    static constexpr int ck = kv::key_unit(E), cv = kv::value_dims(D), tu = kv::value_tokens(D, E);
    static constexpr int BB = 16 * D * E;              // bytes of a block
    static constexpr int L = BB / 1024;                // 16-byte loads of a lane per block
    static constexpr int R = D / (16 * cv);            // rounds of 16 value units
    static constexpr int S = D / 32;                   // matrix-core steps of a block's keys
    typedef u32x4_t Block[L];                          // a block's keys or values in registers, as stored
};

// One step: two blocks.
template <int D, int FMT>
struct Step {
    typename Kv<D, FMT>::Block k[2], v[2];
};

template <int D, int FMT>
__device__ __forceinline__ void load_keys(typename Kv<D, FMT>::Block& k, const uint8_t* p, int lane) {
#pragma unroll
    for (int i = 0; i < Kv<D, FMT>::L; ++i)
        k[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p + i * 1024 + lane * 16));
}

template <int D, int FMT>
__device__ __forceinline__ void load_values(typename Kv<D, FMT>::Block& v, const uint8_t* p, int lane) {
    using T = Kv<D, FMT>;
    constexpr int N = 4 / T::tu;                       // units of a lane's four tokens
#pragma unroll
    for (int r = 0; r < T::R; ++r)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int unit = (N * (lane >> 4) + i) * (D / T::cv) + r * 16 + (lane & 15);
            v[r * N + i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p + unit * 16));
        }
}

__device__ __forceinline__ uint32_t cvt_pair(uint32_t w, bool high) {
    const bf16x2_t p = high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true)
                            : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false);
    return __builtin_bit_cast(uint32_t, p);
}

// The A operand of step j of a block's keys.
template <int D, int FMT>
__device__ __forceinline__ bf16x8_t key_frag(const typename Kv<D, FMT>::Block& k, int j) {
    if constexpr (FMT == FT_KV_BF16) {
        return __builtin_bit_cast(bf16x8_t, k[j]);
    } else {
        return rs::a_frag<FT_FMT_FP8_B128>(k[j >> 1], j & 1, 1.0f);
    }
}

// Two tokens' value at dimension i (of cv) of round r, tokens 2 p and 2 p + 1 of the lane's
// four, as one register of the A operand.
template <int D, int FMT>
__device__ __forceinline__ uint32_t value_pair(const typename Kv<D, FMT>::Block& v, int r, int i, int p) {
    using T = Kv<D, FMT>;
    constexpr int N = 4 / T::tu;
    if constexpr (T::E == 2) {
        // bf16: dimension i is half i % 2 of dword i / 2 of the token's cv / 2
        const u32x4_t u0 = T::tu == 1 ? v[r * N + 2 * p] : v[r * N + p];
        const u32x4_t u1 = T::tu == 1 ? v[r * N + 2 * p + 1] : u0;
        const uint32_t w0 = u0[i >> 1], w1 = T::tu == 1 ? u1[i >> 1] : u1[2 + (i >> 1)];
        return __builtin_amdgcn_perm(w1, w0, i & 1 ? 0x07060302u : 0x05040100u);
    } else {
        // e4m3: byte i % 4 of dword i / 4 of the token's cv / 4; bytes of two tokens side by side, then
        // both converted
        const u32x4_t u = T::tu == 2 ? v[r * N + p] : v[r * N];
        const uint32_t w0 = T::tu == 2 ? u[i >> 2] : u[2 * p], w1 = T::tu == 2 ? u[2 + (i >> 2)] : u[2 * p + 1];
        const uint32_t b = __builtin_amdgcn_perm(w1, w0, i & 2 ? 0x07030602u : 0x05010400u);
        return cvt_pair(b, i & 1);
    }
}

// The running state of a wave: column l % 16, of which the lane has the sums at dimensions
// r 16 cv + (4 (l / 16) + v) cv + i in o[r cv + i][v].
template <int D, int FMT, bool WIDE>
struct State {
    f32x4_t o[D / 16];
    float m, l;          // maximum in base 2; this lane's share of the sum
};

// The query operands of a wave: in registers, or (256 dimensions: with the sums and a step's keys and values they
// pass the 256 registers of two waves) in LDS, one copy for the workgroup.
template <int D, int FMT>
struct Queries {
    static constexpr bool kShared = D == 256;
    bf16x8_t r[kShared ? 1 : Kv<D, FMT>::S];
    const u32x4_t* lds;      // [S][64 lanes]
    __device__ __forceinline__ bf16x8_t operator()(int j, int lane) const {
        if constexpr (kShared) return __builtin_bit_cast(bf16x8_t, lds[j * 64 + lane]);
        else return r[j];
    }
};

// The step's logits in base 2: tokens 16 b + 4 (l / 16) + v of column l % 16.
template <int D, int FMT>
__device__ __forceinline__ void logits(float (&s)[2][4], const Step<D, FMT>& x, const Queries<D, FMT>& q, float scale,
                                       int lane) {
    using T = Kv<D, FMT>;
    f32x4_t acc[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
    for (int j = 0; j < T::S; ++j) {
        const bf16x8_t y = q(j, lane);
#pragma unroll
        for (int b = 0; b < 2; ++b)
            acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(key_frag<D, FMT>(x.k[b], j), y, acc[b], 0, 0, 0);
        if constexpr (D == 256) __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int v = 0; v < 4; ++v) s[b][v] = acc[b][v] * scale;
}

// f over the four lanes of a column, l % 16.
template <typename F>
__device__ __forceinline__ float quarters(float v, F&& f) {
    const uint32_t a = __float_as_uint(v);
    const auto p = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    const uint32_t b = __float_as_uint(f(__uint_as_float(p[0]), __uint_as_float(p[1])));
    const auto r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    return f(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// Two probabilities as bf16 pairs, high + low to 16 significant bits.  Beside values that may be infinite (bf16) the high half is
// cut towards zero and the low one, what is left, not below the least normal number where the probability is not: both products
// of such a value then have its sign, where a rest of zero or below would make their sum NaN.  That adds at most 2^-126 of a
// value, no more than fp32 leaves out of any weight below that.  `down`, the power of two at or below one part of the request's
// tokens, keeps their sum within the largest value, where it would pass fp32.  (e4m3fn has neither: the nearest.)
template <int FMT>
__device__ __forceinline__ void split_pair(float p0, float p1, float down, uint32_t& high, uint32_t& low) {
    if constexpr (FMT == FT_KV_BF16) {
        p0 *= down;
        p1 *= down;
        const uint32_t u0 = __float_as_uint(p0), u1 = __float_as_uint(p1);
        high = __builtin_amdgcn_perm(u1, u0, 0x07060302u);
        const float least = 0x1p-126f;
        const float r0 = fmaxf(p0 - __uint_as_float(u0 & 0xFFFF0000u), fminf(p0, least));
        const float r1 = fmaxf(p1 - __uint_as_float(u1 & 0xFFFF0000u), fminf(p1, least));
        low = __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)r0, (__bf16)r1});
    } else {
        const bf16x2_t h = {(__bf16)p0, (__bf16)p1};
        high = __builtin_bit_cast(uint32_t, h);
        low = __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)(p0 - (float)h[0]), (__bf16)(p1 - (float)h[1])});
    }
}

// A step's probabilities as operands (WIDE: high and low halves; else both in `high`), and which halves of
// value pairs are visible.
struct Probs {
    u32x4_t high, low;
    uint32_t keep[2][2];
    float alpha;             // what the sums so far are multiplied with
};

// Positions t0 + 16 b + 4 (l / 16) + v outside lo .. hi - 1 count for nothing.
template <int D, int FMT, bool WIDE>
__device__ __forceinline__ Probs softmax_step(State<D, FMT, WIDE>& st, float (&s)[2][4], bool masked, int t0, int lo,
                                              int hi, float down, int lane) {
    Probs out;
    uint32_t (&keep)[2][2] = out.keep;
    keep[0][0] = keep[0][1] = keep[1][0] = keep[1][1] = ~0u;
    if (masked) {
        const int t = t0 + 4 * (lane >> 4);
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int at = t + 16 * b + v;
                if (at < lo || at >= hi) {
                    s[b][v] = -INFINITY;
                    keep[b][v >> 1] &= v & 1 ? 0x0000FFFFu : 0xFFFF0000u;
                }
            }
    }
    float mt = fmaxf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3])),
                     fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3])));
    mt = quarters(mt, [](float x, float y) { return fmaxf(x, y); });
    const float m = fmaxf(st.m, mt);
    const float base = m == -INFINITY ? 0.0f : m;      // (nothing visible so far: all terms are 0)
    out.alpha = exp2_of(st.m - base);
    st.m = m;
    float sum = 0.0f;
    uint32_t hi_p[4], lo_p[4];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const float p0 = exp2_of(s[b][2 * p] - base), p1 = exp2_of(s[b][2 * p + 1] - base);
            sum += p0 + p1;
            split_pair<FMT>(p0, p1, down, hi_p[b * 2 + p], lo_p[b * 2 + p]);
        }
    st.l = st.l * out.alpha + sum;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        out.high[i] = WIDE || !(lane & 8) ? hi_p[i] : lo_p[i];
        out.low[i] = lo_p[i];
    }
    return out;
}

template <int D, int FMT, bool WIDE>
__device__ __forceinline__ void add_values(State<D, FMT, WIDE>& st, const Step<D, FMT>& x, const Probs& p) {
    using T = Kv<D, FMT>;
#pragma unroll
    for (int r = 0; r < T::R; ++r)
#pragma unroll
        for (int i = 0; i < T::cv; ++i) {
            u32x4_t a;
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int h = 0; h < 2; ++h) a[b * 2 + h] = value_pair<D, FMT>(x.v[b], r, i, h) & p.keep[b][h];
            f32x4_t& o = st.o[r * T::cv + i];
            o *= p.alpha;
            const bf16x8_t av = __builtin_bit_cast(bf16x8_t, a);
            o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, __builtin_bit_cast(bf16x8_t, p.high), o, 0, 0, 0);
            if constexpr (WIDE)
                o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, __builtin_bit_cast(bf16x8_t, p.low), o, 0, 0, 0);
            // (256 dimensions: operands are made one at a time, not all ahead, which would take their registers)
            if constexpr (D == 256) __builtin_amdgcn_sched_barrier(0);
        }
}

// A row of 16 lanes turned by 8: column n and column n + 8 change places.
__device__ __forceinline__ float other_half(float v) {
    return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x128, 0xF, 0xF, true));
}

// Weight of a part whose maximum is m, beside the whole's maximum (1 for the largest, an infinite one too).
__device__ __forceinline__ float part_weight(float m, float whole) {
    return whole == -INFINITY ? 0.0f : m == whole ? 1.0f : exp2_of(m - whole);
}

// out[0..3] of one head: scale o / l, zeros where nothing was visible.
__device__ __forceinline__ void store_out(uint16_t* to, const f32x4_t o, float l, float scale) {
    const float f = l == 0.0f ? 0.0f : scale / l;
    typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = l == 0.0f ? 0.0f : o[i] * f;
    *reinterpret_cast<u32x2_t*>(to) = u32x2_t{kv::pack_bf16(x[0], x[1]), kv::pack_bf16(x[2], x[3])};
}

// Waves of a SIMD whose registers the kernel fits: a divided launch has at most eight waves to a compute unit (two teams, or
// one where heads have 256 dimensions), whole items as many as can be.
constexpr int waves_of(int D, int fmt, bool direct) { return direct && (D < 256 || fmt == FT_KV_E4M3) ? 3 : 2; }

constexpr int workgroup(int D, int waves) { return 64 * (waves ? waves : kv::team_waves(D)); }

// WAVES: of a workgroup that takes a whole item, or 0: teams of a divided launch.
template <int D, int FMT, bool WIDE, int WAVES>
__global__ void __launch_bounds__(workgroup(D, WAVES), waves_of(D, FMT, WAVES > 0)) attend_kernel(AttendArgs a) {
    using T = Kv<D, FMT>;
    constexpr bool DIRECT = WAVES > 0;
    constexpr int kThreads = workgroup(D, WAVES), kWaves = kThreads / 64;
    constexpr int kUnit = WIDE ? 4 : T::cv, kHalves = T::cv / kUnit;  // dimensions of a value unit that a round takes
    constexpr int kChunk = 16 * kUnit, kRow = kChunk + 4;        // dimensions of a round; padded in LDS
    extern __shared__ __align__(16) int lds[];
    const int B = a.a.requests, tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    int* pre = lds;                                              // [B + 1] length of an item of each request before
    int* lens = pre + B + 1;                                     // [B] visible lengths' ends
    float* wm = reinterpret_cast<float*>(lds + (DIRECT ? 0 : (2 * B + 1 + 3) & ~3));   // [kWaves][16]
    float* wl = wm + kWaves * kv::kCols;
    float* wo = wl + kWaves * kv::kCols;                         // [kWaves][heads][kRow]
    __shared__ uint32_t flag;
    __shared__ int scan[2][kWaves];
    __shared__ u32x4_t wq[Queries<D, FMT>::kShared ? T::S * 64 : 1];
    const int shift = a.c.page_shift, room = a.a.width << shift;

    auto first_of = [&](int hi) { return a.a.window && hi > a.a.window ? hi - a.a.window : 0; };
    auto end_of = [&](int b) {
        const int n = a.a.kv_len[b];
        return n < 0 ? 0 : n > room ? room : n;
    };
    auto steps_of = [&](int hi) {
        return hi ? (hi + kv::kStep - 1) / kv::kStep - first_of(hi) / kv::kStep : 0;
    };
    const int g = a.g, heads_all = a.c.heads * a.blocks;
    // the lengths of the requests' items, summed in slices of the workgroup's width, and how many have any
    int carry = 0, busy = 0;
    for (int b0 = 0; b0 < B && !DIRECT; b0 += kThreads) {
        const int b = b0 + tid;
        const int hi = b < B ? end_of(b) : 0, own = kv::item_length(steps_of(hi));
        const int x = kv::wave_scan(own);
        const int some = __popcll(__ballot(own > 0));
        __syncthreads();
        if (lane == 63) {
            scan[0][wave] = x;
            scan[1][wave] = some;
        }
        __syncthreads();
        int before = carry;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const int sum = uniform(scan[0][w]);
            if (w < wave) before += sum;
            carry += sum;
            busy += uniform(scan[1][w]);
        }
        if (b < B) {
            pre[b] = before + x - own;
            lens[b] = hi;
        }
    }
    kv::Division div = {};
    const int self = DIRECT ? 0 : blockIdx.x;
    int b = 0, item;
    if constexpr (DIRECT) {
        b = blockIdx.x / heads_all;
        item = blockIdx.x % heads_all;
    } else {
        if (tid == 0) pre[B] = carry;
        __syncthreads();
        // requests that see nothing
        for (int r = blockIdx.x; r < B; r += gridDim.x)
            if (pre[r] == pre[r + 1])
                for (int i = tid * 8; i < a.a.q_heads * D; i += kThreads * 8)
                    *reinterpret_cast<u32x4_t*>(a.a.out + r * a.a.out_stride + i) = u32x4_t{0, 0, 0, 0};
        if (carry == 0) return;
        div = kv::divide((uint32_t)busy * heads_all, (uint32_t)carry * heads_all, kv::team_steps(D), gridDim.x,
                         kv::many_items(D * (FMT == FT_KV_BF16 ? 2 : 1)));
        if (self >= div.teams) return;
        // the item that this team's cut falls into, before it moves (64 requests a look); then on from item to
        // item
        const uint32_t at = kv::cut(div, self);
        const int q = at / (uint32_t)heads_all;
        for (int left = B; left > 1;) {
            const int width = (left + 63) >> 6, i = lane * width;
            b += (__popcll(__ballot(i < left && pre[b + (i < left ? i : 0)] <= q)) - 1) * width;
            left = min(width, B - b);
        }
        const uint32_t before = uniform(pre[b]), length = uniform(pre[b + 1]) - before;
        item = (at - before * heads_all) / length;
    }
    const __amdgpu_buffer_rsrc_t parts = __builtin_amdgcn_make_buffer_rsrc(a.part, 0, a.part_bytes, 0x00020000);
    const uint32_t part_stride = (uint32_t)kv::part_floats(g, D) * 4;

    for (;; ++item) {
        int hi, nb, first = 0, n;                                // the request's length, the item's steps, this segment's
        kv::Teams who = {0, 0};
        if constexpr (DIRECT) {
            hi = uniform(end_of(b));
            n = nb = steps_of(hi);
        } else {
            if (item == heads_all) {
                item = 0;
                do ++b;
                while (b < B && uniform(pre[b]) == uniform(pre[b + 1]));
                if (b == B) return;
            }
            hi = uniform(lens[b]);
            const int before = uniform(pre[b]), length = uniform(pre[b + 1]) - before;
            nb = length - kv::kItemCost;
            const uint32_t item_begin = (uint32_t)before * heads_all + (uint32_t)item * length;
            who = kv::teams_of(div, item_begin, nb);
            who.first = uniform(who.first);
            who.last = uniform(who.last);
            if (self > who.last) continue;                       // (the cut has moved to the item's end)
            if (self < who.first) return;
            const kv::Segment seg = kv::segment(div, who, item_begin, nb, self);
            first = seg.from;
            n = seg.to - seg.from;
        }
        const int lo = first_of(hi);
        const int h = item / a.blocks, q0 = h * g + (item % a.blocks) * kv::kCols;
        const int heads = min(kv::kCols, g - (item % a.blocks) * kv::kCols);
        const int step0 = lo / kv::kStep + first;                // in the request's own steps
        const float scale = a.a.scale * kLog2e * (FMT == FT_KV_E4M3 ? a.c.k_scale[h] : 1.0f);
        // bf16: weights meet values as 2^-ceil(log2(tokens)) of themselves, so that the sum is finite where the mean is
        const int halvings = hi - lo > 1 ? 32 - __builtin_clz(hi - lo - 1) : 0;
        const float down = __uint_as_float((uint32_t)(127 - halvings) << 23);
        const float out_scale = FMT == FT_KV_E4M3 ? a.c.v_scale[h] : __uint_as_float((uint32_t)(127 + halvings) << 23);

        Queries<D, FMT> q;
        q.lds = wq;
        {
            const int col = WIDE ? lane & 15 : lane & 7, quarter = lane >> 4;
            const uint16_t* row = a.a.q + b * a.a.q_stride + (int64_t)(q0 + (col < heads ? col : 0)) * D;
#pragma unroll
            for (int j = 0; j < T::S; ++j) {
                if (Queries<D, FMT>::kShared && j % kWaves != wave) continue;
                // the dimensions that key_frag's step j has at this quarter
                const int e = T::E == 2 ? (j * 4 + quarter) * 8 : ((j >> 1) * 4 + quarter) * 16 + (j & 1) * 8;
                u32x4_t v = *reinterpret_cast<const u32x4_t*>(row + e);
                if (col >= heads) v = u32x4_t{0, 0, 0, 0};
                if constexpr (Queries<D, FMT>::kShared) wq[j * 64 + lane] = v;
                else q.r[j] = __builtin_bit_cast(bf16x8_t, v);
            }
            if constexpr (Queries<D, FMT>::kShared) __syncthreads();
        }
        State<D, FMT, WIDE> st;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) st.o[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        st.m = -INFINITY;
        st.l = 0.0f;

        const int64_t head_off = (int64_t)h * ((int64_t)(D * T::E) << shift);
        const int32_t* table = a.a.table + (int64_t)b * a.a.width;
        const int mine = (n - wave + kWaves - 1) / kWaves;       // this wave's steps: wave, wave + kWaves, ...
        // The next step's keys are loaded once this one's have been used, its values likewise, into the same
        // registers: one or the other is always under way.
        Step<D, FMT> x;
        int pages[2] = {-1, -1};
        bool on[2], on_next[2];
        int64_t off[2];
        auto find = [&](int i) {
            if ((i & 63) == 0) {
                // the page ids of this wave's next 64 steps, one step a lane (a block past the request's end is not
                // looked up: it may have no entry)
                const int t = (step0 + wave + (i + lane) * kWaves) * kv::kStep;
                const bool some = i + lane < mine;
                pages[0] = some && t < hi ? table[t >> shift] : -1;
                pages[1] = some && t + 16 < hi ? table[(t + 16) >> shift] : -1;
                // (waited for here: where the branches meet, every step would wait for all its loads)
                asm volatile("" : "+v"(pages[0]), "+v"(pages[1]));
            }
            const int t0 = (step0 + wave + i * kWaves) * kv::kStep;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int id = __builtin_amdgcn_readlane(pages[b], i & 63);
                on_next[b] = id >= 0 && id < a.c.pages;
                off[b] = (on_next[b] ? (int64_t)id * a.c.page_stride : 0) + head_off +
                         (int64_t)(((t0 + 16 * b) & ((1 << shift) - 1)) >> 4) * T::BB;
            }
        };
        auto keys = [&] {
#pragma unroll
            for (int b = 0; b < 2; ++b) load_keys<D, FMT>(x.k[b], a.c.k + off[b], lane);
        };
        auto values = [&] {
#pragma unroll
            for (int b = 0; b < 2; ++b) load_values<D, FMT>(x.v[b], a.c.v + off[b], lane);
        };
        if (mine > 0) {
            find(0);
            keys();
            values();
        }
        for (int i = 0; i < mine; ++i) {
            const int t0 = (step0 + wave + i * kWaves) * kv::kStep;
            on[0] = on_next[0];
            on[1] = on_next[1];
            float s[2][4];
            logits<D, FMT>(s, x, q, scale, lane);
            __builtin_amdgcn_sched_barrier(0);
            // (behind the last step it is the pool's first page, which nothing waits for: were these loads
            // conditional, every step would wait for all loads under way)
            find(i + 1);
            keys();
            // blocks without a page are left out: the visible range shrinks to the other one, or to nothing
            const int from = on[0] ? lo : max(lo, t0 + 16), to = on[1] ? hi : min(hi, t0 + 16);
            const Probs p = softmax_step<D, FMT, WIDE>(st, s, from > t0 || to < t0 + kv::kStep, t0, from, to, down, lane);
            add_values<D, FMT, WIDE>(st, x, p);
            __builtin_amdgcn_sched_barrier(0);
            values();
        }

        // ---- the waves' parts together ----
        const float l = quarters(st.l, [](float x, float y) { return x + y; });
        const int col = lane & 15;
        if (lane < 16) {
            wm[wave * kv::kCols + col] = st.m;
            wl[wave * kv::kCols + col] = l;
        }
        __syncthreads();
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) M = fmaxf(M, wm[w * kv::kCols + col]);
        const float f = part_weight(st.m, M);
        const int waves = min(n, kWaves);                        // those that had steps

        const int tf = who.first, tl = who.last;
        const bool whole = DIRECT || tf == tl;
        const uint32_t slot = kv::part_slot(who, self) * part_stride, stats_at = (uint32_t)(kv::item_heads(g) * D) * 4;
        uint16_t* out = a.a.out + b * a.a.out_stride + (int64_t)q0 * D;

        // The sum of `count` parts, of teams t0, t0 + by, ...: to the output, or in the place of the first, whose
        // threads alone read it (all read its statistics, so the run's have a place of their own).  Threads that have no four
        // dimensions of their own take a share of the parts, and the shares add up in LDS.
        auto join = [&](int t0, int count, int by, bool final) {
            const uint32_t step = (uint32_t)by * part_stride, first_at = kv::part_slot(who, t0) * part_stride;
            const uint32_t stats = stats_at + (by > 1 ? kRunStats : 0);
            const int tasks = heads * (D / 4), groups = max(1, min(kThreads / tasks, count));
            for (int x0 = 0; x0 < tasks; x0 += kThreads) {
                const int group = groups > 1 ? tid / tasks : 0, x = groups > 1 ? tid - group * tasks : x0 + tid;
                const int c = x / (D / 4), e = x % (D / 4) * 4;
                const bool works = x < tasks && group < groups;
                float m = -INFINITY, lt = 0.0f;
                f32x4_t o = {0.0f, 0.0f, 0.0f, 0.0f};
                constexpr int N = 8;                             // parts in flight
                const int p0 = count * group / groups, p1 = works ? count * (group + 1) / groups : p0;
                uint32_t at = first_at + (uint32_t)p0 * step;
                for (int p = p0; p < p1; p += N, at += N * step) {
                    float pm[N], pl[N];
                    f32x4_t po[N];
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        if (p + i >= p1) continue;
                        const uint32_t v = at + stats + c * 4, w = i * step;
                        pm[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(parts, v, w, kAgent));
                        pl[i] = __uint_as_float(
                            __builtin_amdgcn_raw_buffer_load_b32(parts, v + kv::kCols * 4, w, kAgent));
                        po[i] = __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                                parts, at + (uint32_t)(c * D + e) * 4, w, kAgent));
                    }
                    float mn = m;
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        if (p + i < p1) mn = fmaxf(mn, pm[i]);
                    const float f0 = part_weight(m, mn);
                    lt *= f0;
                    o *= f0;
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        if (p + i >= p1) continue;
                        const float f1 = part_weight(pm[i], mn);
                        lt += pl[i] * f1;
                        o += po[i] * f1;
                    }
                    m = mn;
                }
                if (groups > 1) {
                    float* js = wo + kThreads * 4;               // (no wave reads wo any more)
                    if (works) {
                        *reinterpret_cast<f32x4_t*>(wo + tid * 4) = o;
                        js[tid] = m;
                        js[kThreads + tid] = lt;
                    }
                    __syncthreads();
                    if (works && group == 0) {
                        for (int i = 1; i < groups; ++i) m = fmaxf(m, js[i * tasks + x]);
                        lt = 0.0f;
                        o = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
                        for (int i = 0; i < groups; ++i) {
                            const float f1 = part_weight(js[i * tasks + x], m);
                            lt += js[kThreads + i * tasks + x] * f1;
                            o += *reinterpret_cast<const f32x4_t*>(wo + (i * tasks + x) * 4) * f1;
                        }
                    }
                }
                if (works && group == 0) {
                    if (final) {
                        const float sink = a.a.sinks ? a.a.sinks[q0 + c] * kLog2e : -INFINITY, mn = fmaxf(m, sink);
                        const float f1 = part_weight(m, mn);
                        store_out(out + (int64_t)c * D + e, o * f1, lt * f1 + part_weight(sink, mn), out_scale);
                    } else {
                        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, o), parts,
                                                               first_at + (uint32_t)(c * D + e) * 4, 0, kAgent);
                        if (e == 0) {
                            const uint32_t v = first_at + stats_at + kRunStats + c * 4;
                            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(m), parts, v, 0, kAgent);
                            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(lt), parts, v + kv::kCols * 4, 0, kAgent);
                        }
                    }
                }
            }
        };
#pragma unroll
        for (int round = 0; round < T::R * kHalves; ++round) {
            const int r = round / kHalves, half = round % kHalves * kUnit;
            if (round) __syncthreads();
#pragma unroll
            for (int v = 0; v < 4; ++v)
#pragma unroll
                for (int i = 0; i < kUnit; i += 4) {
                    f32x4_t o;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        o[e] = st.o[r * T::cv + half + i + e][v] * f;
                        if constexpr (!WIDE) o[e] += other_half(o[e]);
                    }
                    if (col < heads && wave < waves)
                        *reinterpret_cast<f32x4_t*>(wo + (wave * heads + col) * kRow + (4 * (lane >> 4) + v) * kUnit + i) = o;
                }
            __syncthreads();
            for (int x = tid; x < heads * (kChunk / 4); x += kThreads) {
                const int c = x / (kChunk / 4), e = x % (kChunk / 4) * 4;
                const int dim = r * 16 * T::cv + e / kUnit * T::cv + half + e % kUnit;
                f32x4_t o = {0.0f, 0.0f, 0.0f, 0.0f};
                for (int w = 0; w < waves; ++w) o += *reinterpret_cast<const f32x4_t*>(wo + (w * heads + c) * kRow + e);
                if (whole) {
                    float m = -INFINITY, lt = 0.0f;
#pragma unroll
                    for (int w = 0; w < kWaves; ++w) m = fmaxf(m, wm[w * kv::kCols + c]);
                    const float sink = a.a.sinks ? a.a.sinks[q0 + c] * kLog2e : -INFINITY;
                    const float mm = fmaxf(m, sink);
#pragma unroll
                    for (int w = 0; w < kWaves; ++w)
                        lt += wl[w * kv::kCols + c] * part_weight(wm[w * kv::kCols + c], mm);
                    lt += part_weight(sink, mm);
                    o *= part_weight(m, mm);
                    store_out(out + (int64_t)c * D + dim, o, lt, out_scale);
                } else {
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, o), parts,
                                                           slot + (uint32_t)(c * D + dim) * 4, 0, kAgent);
                }
            }
        }
        if (!DIRECT && !whole) {
            // statistics behind the sums: maxima, then totals
            if (tid < kv::kCols) {
                float m = -INFINITY, lt = 0.0f;
#pragma unroll
                for (int w = 0; w < kWaves; ++w) m = fmaxf(m, wm[w * kv::kCols + tid]);
#pragma unroll
                for (int w = 0; w < kWaves; ++w)
                    lt += wl[w * kv::kCols + tid] * part_weight(wm[w * kv::kCols + tid], m);
                const uint32_t v = slot + stats_at + tid * 4;
#pragma unroll
                for (int i = 0; i < 2; ++i) {                    // (of the part, and of a run that is this part)
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(m), parts, v, i * kRunStats, kAgent);
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(lt), parts, v + kv::kCols * 4, i * kRunStats, kAgent);
                }
            }
            // the run's last team adds its parts up, and the last run's team the runs' sums (a run of one is its
            // part)
            const int run = kv::join_run(who), r0 = tf + (self - tf) / run * run, rn = min(run, tl - r0 + 1);
            const int runs = (tl - tf) / run + 1;
            bool go_on = true;
            if (runs > 1 && rn > 1) {
                go_on = last_arrival(a.counters + r0, (uint32_t)rn, &flag);
                if (go_on) join(r0, rn, 1, false);
            }
            if (go_on && last_arrival(a.counters + kv::kMaxTeams + tf, (uint32_t)(runs > 1 ? runs : rn), &flag))
                join(tf, runs > 1 ? runs : rn, runs > 1 ? run : 1, true);
        }
        if constexpr (DIRECT) return;
        __syncthreads();                                         // the next segment writes wm, wl and wo
    }
}

template <int D, int FMT, bool WIDE, int WAVES>
hipError_t start(const AttendArgs& a, int grid, hipStream_t st) {
    constexpr int kThreads = workgroup(D, WAVES), kWaves = kThreads / 64;
    // (the join's shares take 6 floats a thread)
    const size_t row = 16 * (WIDE ? 4 : Kv<D, FMT>::cv) + 4;
    const size_t waves = (size_t)kWaves * kv::item_heads(a.g) * row * 4, join = kThreads * 6 * 4;
    const size_t list = WAVES ? 0 : ((size_t)2 * a.a.requests + 1 + 3) & ~(size_t)3;
    const size_t lds = list * 4 + 2 * kWaves * kv::kCols * 4 +
                       (waves > join ? waves : join);
    return launch(attend_kernel<D, FMT, WIDE, WAVES>, dim3(grid), dim3(kThreads), lds, st, a);
}

// `steps`: the most that an item can have.
template <int D, int FMT, bool WIDE>
hipError_t go(const AttendArgs& a, int64_t steps, hipStream_t st) {
    const int64_t items = (int64_t)a.a.requests * a.c.heads * a.blocks;
    if (steps > kv::kDirectSteps) return start<D, FMT, WIDE, 0>(a, kv::grid_of(items, items * steps, D, FMT == FT_KV_BF16 ? 2 : 1), st);
    if (kv::direct_waves(items, steps) == 2) return start<D, FMT, WIDE, 2>(a, (int)items, st);
    return start<D, FMT, WIDE, kv::kDirectWaves>(a, (int)items, st);
}

template <int D>
hipError_t pick(const AttendArgs& a, int64_t steps, hipStream_t st) {
    const bool wide = a.g > kv::kCols / 2;
    if (a.c.fmt == FT_KV_BF16)
        return wide ? go<D, FT_KV_BF16, true>(a, steps, st) : go<D, FT_KV_BF16, false>(a, steps, st);
    return wide ? go<D, FT_KV_E4M3, true>(a, steps, st) : go<D, FT_KV_E4M3, false>(a, steps, st);
}

}  // namespace

size_t kv_attend_workspace(int g, int D) { return (size_t)2 * kv::kMaxTeams * kv::part_floats(g, D) * 4; }

hipError_t launch_kv_attend(const CacheView& c, const ft_attend& q, ft_workspace* ws, hipStream_t st) {
    AttendArgs a;
    a.c = c;
    a.a = q;
    a.g = q.q_heads / c.heads;
    a.blocks = kv::head_blocks(a.g);
    a.part = reinterpret_cast<float*>(ws->mem + kCounterBytes);
    a.part_bytes = (uint32_t)kv_attend_workspace(a.g, c.D);
    a.counters = reinterpret_cast<uint32_t*>(ws->mem);
    const int64_t most = (((int64_t)q.width << c.page_shift) + kv::kStep - 1) / kv::kStep + (q.window ? 1 : 0);
    const int64_t seen = q.window ? q.window / kv::kStep + 2 : most;
    const int64_t steps = seen < most ? seen : most;
    if (c.D == 64) return pick<64>(a, steps, st);
    if (c.D == 128) return pick<128>(a, steps, st);
    return pick<256>(a, steps, st);
}

}  // namespace ftmoe
