// New tokens' keys and values into their cache slots, rotated, with the rotated
// queries (ft_kv_append).
//
// A wave takes 16 tokens, lane l token l % 16, and of each head the two 8-element
// chunks that rotate together (i and i + rot / 2) of its quarter l / 16, so a
// pair is read once and the angles' cos and sin stay in registers over the heads.  16
// consecutive tokens of a prompt fill a block of the cache: the lanes' key units
// are then runs of 256 bytes, value rows and source rows of 64.  Memory bounds a prompt,
// latency a decode step.
#include "kv.h"
#include "wfmt.h"

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

__device__ __forceinline__ Chunk load_chunk(const uint16_t* p) {
    const u32x4_t u = *reinterpret_cast<const u32x4_t*>(p);
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
        u[i] = (uint32_t)f32_to_bf16_rne(c.v[2 * i]) | (uint32_t)f32_to_bf16_rne(c.v[2 * i + 1]) << 16;
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

template <int D, int FMT>
__global__ void __launch_bounds__(kThreads) append_kernel(AppendArgs a) {
    constexpr int E = FMT == FT_KV_BF16 ? 2 : 1;
    constexpr int kGroups = D / 64;                    // groups of four chunk pairs of a head
    const int lane = threadIdx.x & 63;
    const int64_t wave = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
    const int heads = a.a.q_heads + 2 * a.c.heads, parts = (heads + a.per - 1) / a.per;
    const int group = (int)(wave % kGroups), part = (int)(wave / kGroups % parts);
    const int64_t t = wave / kGroups / parts * 16 + (lane & 15);
    if (t >= a.a.tokens) return;
    const int slot = a.a.slot[t];
    if (slot < 0 || slot >= a.c.pages << a.c.page_shift) return;
    const int half = a.a.rot >> 1, pair = group * 4 + (lane >> 4);
    // the pair's first dimensions: rotating ones come first, the rest are neighbours
    const bool turns = pair < half >> 3;
    const int e0 = turns ? pair * 8 : pair * 16, e1 = turns ? e0 + half : e0 + 8;
    float cs[8], sn[8];
    if (a.a.rot) {
        const int p = a.a.pos[t];
        if (p < 0 || p >= a.a.positions) return;
        if (turns) {
            const float* row = a.a.cos_sin + (int64_t)p * a.a.rot + pair * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                cs[i] = row[i];
                sn[i] = row[half + i];
            }
        }
    }
    const int page = slot >> a.c.page_shift, in = slot & ((1 << a.c.page_shift) - 1), r = in & 15;
    const int64_t head_bytes = (int64_t)(D * E) << a.c.page_shift;
    const int64_t place = (int64_t)page * a.c.page_stride + (in >> 4) * (16 * D * E);
    const int h1 = min(heads, (part + 1) * a.per);
    for (int h = part * a.per; h < h1; ++h) {
        const int kh = h - a.a.q_heads, vh = kh - a.c.heads;
        const uint16_t* src = kh < 0   ? a.a.q + t * a.a.q_stride + h * D
                              : vh < 0 ? a.a.k + t * a.a.k_stride + kh * D
                                       : a.a.v + t * a.a.v_stride + vh * D;
        Chunk x = load_chunk(src + e0), y = load_chunk(src + e1);
        if (turns && vh < 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float u = x.v[i], w = y.v[i];
                x.v[i] = u * cs[i] - w * sn[i];
                y.v[i] = w * cs[i] + u * sn[i];
            }
        }
        if (kh < 0) {
            uint16_t* to = a.a.q_out + t * a.a.q_out_stride + h * D;
            *reinterpret_cast<u32x4_t*>(to + e0) = to_bf16(x);
            *reinterpret_cast<u32x4_t*>(to + e1) = to_bf16(y);
        } else if (vh < 0) {
            const float scale = FMT == FT_KV_E4M3 ? a.c.k_scale[kh] : 1.0f;
            uint8_t* to = a.c.k + place + kh * head_bytes;
            put<D, FMT, true>(to, r, e0, x, scale);
            put<D, FMT, true>(to, r, e1, y, scale);
        } else {
            const float scale = FMT == FT_KV_E4M3 ? a.c.v_scale[vh] : 1.0f;
            uint8_t* to = a.c.v + place + vh * head_bytes;
            put<D, FMT, false>(to, r, e0, x, scale);
            put<D, FMT, false>(to, r, e1, y, scale);
        }
    }
}

template <int D>
hipError_t go(const AppendArgs& a, int64_t waves, hipStream_t st) {
    const dim3 grid((unsigned)((waves + kThreads / 64 - 1) / (kThreads / 64))), block(kThreads);
    if (a.c.fmt == FT_KV_BF16) return launch(append_kernel<D, FT_KV_BF16>, grid, block, 0, st, a);
    return launch(append_kernel<D, FT_KV_E4M3>, grid, block, 0, st, a);
}

}  // namespace

hipError_t launch_kv_append(const CacheView& c, const ft_append& a, hipStream_t st) {
    AppendArgs k;
    k.c = c;
    k.a = a;
    const int heads = a.q_heads + 2 * c.heads, groups = c.D / 64;
    const int64_t blocks = (a.tokens + 15) / 16;
    k.per = 1;
    while (k.per < 8 && blocks * groups * ((heads + 2 * k.per - 1) / (2 * k.per)) >= 4096) k.per *= 2;
    const int64_t waves = blocks * groups * ((heads + k.per - 1) / k.per);
    if (c.D == 64) return go<64>(k, waves, st);
    if (c.D == 128) return go<128>(k, waves, st);
    return go<256>(k, waves, st);
}

}  // namespace ftmoe
