// New tokens' keys and values into their cache slots, rotated, with the rotated
// queries (ft_kv_append).
//
// A wave takes 8 tokens (16 where heads have 64 dimensions), lane l token l % 8, and
// of each head the two 8-element chunks that rotate together (i and i + rot / 2) of
// its eighth l / 8, so a pair is read once and the angles' cos and sin stay in registers
// over the heads.  8 consecutive tokens of a prompt fill half a block of the cache:
// the lanes' key units are then runs of 128 bytes, and so are value and source rows.  Memory bounds a prompt
// (8,192 tokens of 32 + 8 + 8 heads of 128: 40.5 us, 5.1 TB/s read and written), latency a decode step (16
// tokens 3.8 us).
#include "kv_device.h"

namespace ftmoe {
namespace {

struct AppendArgs {
    CacheView c;
    ft_append a;
    int per;                 // heads of a wave
};

struct Chunk {
    float v[8];
};

__device__ __forceinline__ Chunk chunk_of(const u32x4_t u) {
    Chunk c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        c.v[2 * i] = bf16lo(u[i]);
        c.v[2 * i + 1] = bf16hi(u[i]);
    }
    return c;
}

__device__ __forceinline__ u32x4_t to_bf16(const Chunk& c) {
    u32x4_t u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        u[i] = kv::pack_bf16(c.v[2 * i], c.v[2 * i + 1]);
    return u;
}

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// 8 codes; the comparison keeps a NaN, which min and max would drop.
__device__ __forceinline__ u32x2_t to_e4m3(const Chunk& c, float scale) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float d = c.v[i] / scale;
        x[i] = d > 448.0f ? 448.0f : d < -448.0f ? -448.0f : d;
    }
    u32x2_t u;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i], x[4 * i + 1], 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i + 2], x[4 * i + 3], w, true);
        u[i] = (uint32_t)w;
    }
    return u;
}

// The 8 elements of token r of a block, at dimension e (a multiple of 8), into the head's
// block at `p`: keys as (half of) one unit, values as their share of one unit or more.
template <int D, int FMT, bool KEY>
__device__ __forceinline__ void put(uint8_t* p, int r, int e, const Chunk& c, float scale) {
    constexpr int E = FMT == FT_KV_BF16 ? 2 : 1;
    if constexpr (KEY) {
        constexpr int ck = kv::key_unit(E);
        uint8_t* to = p + ((e / ck) * 16 + r) * 16 + (e % ck) * E;
        if constexpr (E == 2) *reinterpret_cast<u32x4_t*>(to) = to_bf16(c);
        else *reinterpret_cast<u32x2_t*>(to) = to_e4m3(c, scale);
    } else {
        constexpr int cv = kv::value_dims(D), tu = kv::value_tokens(D, E);
        uint8_t* to = p + ((r / tu) * (D / cv) + e / cv) * 16 + (r % tu) * cv * E;
        if constexpr (E == 2) {
            const u32x4_t u = to_bf16(c);
            if constexpr (cv == 8) {
                *reinterpret_cast<u32x4_t*>(to) = u;
            } else {
                *reinterpret_cast<u32x2_t*>(to) = u32x2_t{u[0], u[1]};
                *reinterpret_cast<u32x2_t*>(to + 16) = u32x2_t{u[2], u[3]};
            }
        } else {
            const u32x2_t u = to_e4m3(c, scale);
            if constexpr (cv == 8) {
                *reinterpret_cast<u32x2_t*>(to) = u;
            } else {
                *reinterpret_cast<uint32_t*>(to) = u[0];
                *reinterpret_cast<uint32_t*>(to + 16) = u[1];
            }
        }
    }
}

constexpr int kThreads = 256;
// Lanes of a token: its chunk pairs of a head that a wave takes, whole 128-byte lines on either side.
constexpr int lanes_of(int D) { return D == 64 ? 4 : 8; }
constexpr int kAhead = 2;                 // heads whose loads are under way

template <int D, int FMT, int STREAM>
__global__ void __launch_bounds__(kThreads) append_kernel(AppendArgs a) {
    constexpr int E = FMT == FT_KV_BF16 ? 2 : 1;
    constexpr int kLanes = lanes_of(D), kTokens = 64 / kLanes, kGroups = D / 16 / kLanes;
    const int lane = threadIdx.x & 63;
    const uint32_t wave = blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);      // (below 2^26)
    const int heads = a.a.q_heads + 2 * a.c.heads, parts = (heads + a.per - 1) / a.per;
    const int group = (int)(wave % kGroups), part = (int)(wave / kGroups % parts);
    const int64_t t = (int)(wave / kGroups / parts) * kTokens + lane % kTokens;
    if (t >= a.a.tokens) return;
    const int half = a.a.rot >> 1, pair = group * kLanes + lane / kTokens;
    // the pair's first dimensions: rotating ones come first, the rest are neighbours
    const bool turns = pair < half >> 3;
    const int e0 = turns ? pair * 8 : pair * 16, e1 = turns ? e0 + half : e0 + 8;
    const int h0 = part * a.per, h1 = min(heads, h0 + a.per);
    u32x4_t raw[kAhead][2];
    auto load = [&](int from) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int h = from + i, kh = h - a.a.q_heads, vh = kh - a.c.heads;
            if (h >= h1) continue;
            const uint16_t* src = kh < 0   ? a.a.q + t * a.a.q_stride + h * D
                                  : vh < 0 ? a.a.k + t * a.a.k_stride + kh * D
                                           : a.a.v + t * a.a.v_stride + vh * D;
            raw[i][0] = kv::load16<(STREAM > 1)>(src + e0);
            raw[i][1] = kv::load16<(STREAM > 1)>(src + e1);
        }
    };
    load(h0);                                          // (under way while slot and position come)
    const int slot = a.a.slot[t], p = a.a.rot ? a.a.pos[t] : 0;
    if (slot < 0 || slot >= a.c.pages << a.c.page_shift) return;
    if (a.a.rot && (p < 0 || p >= a.a.positions)) return;
    float cs[8], sn[8];
    if (turns) {
        const float* row = a.a.cos_sin + (int64_t)p * a.a.rot + pair * 8;
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            const f32x4_t c = *reinterpret_cast<const f32x4_t*>(row + i), s = *reinterpret_cast<const f32x4_t*>(row + half + i);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                cs[i + e] = c[e];
                sn[i + e] = s[e];
            }
        }
    }
    const int page = slot >> a.c.page_shift, in = slot & ((1 << a.c.page_shift) - 1), r = in & 15;
    const int64_t head_bytes = (int64_t)(D * E) << a.c.page_shift;
    const int64_t place = (int64_t)page * a.c.page_stride + (in >> 4) * (16 * D * E);
    for (int from = h0; from < h1; from += kAhead) {
        Chunk x[kAhead], y[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            x[i] = chunk_of(raw[i][0]);
            y[i] = chunk_of(raw[i][1]);
        }
        if (from + kAhead < h1) load(from + kAhead);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int h = from + i, kh = h - a.a.q_heads, vh = kh - a.c.heads;
            if (h >= h1) continue;
            if (turns && vh < 0) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float u = x[i].v[j], w = y[i].v[j];
                    x[i].v[j] = u * cs[j] - w * sn[j];
                    y[i].v[j] = w * cs[j] + u * sn[j];
                }
            }
            if (kh < 0) {
                uint16_t* to = a.a.q_out + t * a.a.q_out_stride + h * D;
                kv::store16<(STREAM > 0)>(to + e0, to_bf16(x[i]));
                kv::store16<(STREAM > 0)>(to + e1, to_bf16(y[i]));
            } else if (vh < 0) {
                const float scale = FMT == FT_KV_E4M3 ? a.c.k_scale[kh] : 1.0f;
                uint8_t* to = a.c.k + place + kh * head_bytes;
                put<D, FMT, true>(to, r, e0, x[i], scale);
                put<D, FMT, true>(to, r, e1, y[i], scale);
            } else {
                const float scale = FMT == FT_KV_E4M3 ? a.c.v_scale[vh] : 1.0f;
                uint8_t* to = a.c.v + place + vh * head_bytes;
                put<D, FMT, false>(to, r, e0, x[i], scale);
                put<D, FMT, false>(to, r, e1, y[i], scale);
            }
        }
    }
}

template <int D, int STREAM>
hipError_t go(const AppendArgs& a, int64_t waves, hipStream_t st) {
    const dim3 grid((unsigned)((waves + kThreads / 64 - 1) / (kThreads / 64))), block(kThreads);
    if (a.c.fmt == FT_KV_BF16) return launch(append_kernel<D, FT_KV_BF16, STREAM>, grid, block, 0, st, a);
    return launch(append_kernel<D, FT_KV_E4M3, STREAM>, grid, block, 0, st, a);
}

// Where the rows are more than the L2s hold, queries are written past them, and the rows are read past them if a
// wave's loads take whole lines, that is where heads of 128 or more rotate whole (elsewhere two loads share a
// line): 8,192 tokens of 40 heads and 8 of values 42 us, 50 through the L2s; of 72 heads of 64 and 8 of values 43
// with cached loads, 49 without.  The cache's lines stay: the attention that follows reads them.
template <int D>
hipError_t pick(const AppendArgs& a, int64_t waves, hipStream_t st) {
    const int64_t moved = (int64_t)a.a.tokens * (2 * a.a.q_heads + 2 * a.c.heads) * D * 2;
    if (moved <= kv::kStreamBytes) return go<D, 0>(a, waves, st);
    if (D == 64 || a.a.rot < D) return go<D, 1>(a, waves, st);
    return go<D, 2>(a, waves, st);
}

}  // namespace

// A wave's heads share its slot, angles and start, and keep a step's loads ahead, as long as the waves still cover the
// latency.  Twice the heads where ten waves or more per compute unit are left: 1,000 tokens of 48 heads of 128 9.3 us
// in 3,000 waves, 10.5 in 6,000; 1,500 tokens 13.3 in 2,256, 12.8 in 4,512; 777 e4m3 tokens 7.2 in 1,960, 6.2 in 3,920.
// Eight heads a wave: 8,192 tokens 44, 41 with four.  (Calls in a captured graph.)
hipError_t launch_kv_append(const CacheView& c, const ft_append& a, hipStream_t st) {
    AppendArgs k;
    k.c = c;
    k.a = a;
    const int heads = a.q_heads + 2 * c.heads, lanes = lanes_of(c.D), groups = c.D / 16 / lanes;
    const int64_t blocks = (a.tokens + 64 / lanes - 1) / (64 / lanes);
    k.per = 1;
    while (k.per < 4 && blocks * groups * ((heads + 2 * k.per - 1) / (2 * k.per)) >= 2560) k.per *= 2;
    const int64_t waves = blocks * groups * ((heads + k.per - 1) / k.per);
    if (c.D == 64) return pick<64>(k, waves, st);
    if (c.D == 128) return pick<128>(k, waves, st);
    return pick<256>(k, waves, st);
}

}  // namespace ftmoe
