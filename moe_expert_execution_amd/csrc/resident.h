// Streaming a panel-ordered weight matrix against a few tokens on the matrix
// cores: the device code shared by the operators over resident weights
// (moe_layer.hip, lora.hip).
//
// A 32-row panel is read in units of 128 along K.  Lane l of a wave takes row
// l % 16 of one half of the panel at chunk column l / 16 of four, which is the
// A operand of v_mfma_f32_16x16x32_bf16 as it stands (codes are converted to
// bf16 in registers, exact for e4m3 and for e2m1 times a power of two); a load
// is four runs of 256 bytes.  Up to 16 tokens are the B operand: lane l holds
// token l % 16 at the same K positions, read from memory (L2).  So a panel
// streams from HBM once for the tokens of one tile, of one or two operands (32
// tokens, or an expert's routes in the layer); the next tile of the same rows
// streams it again.  Lane l ends with token l % 16 and rows 4 (l / 16) .. + 3 of
// each half.  16 columns and not 32: a token load returns 1 KiB to the lanes whatever its rows hold, at 64 bytes
// per cycle and CU, so narrower tiles halve what stands beside the weights on
// that path (the layer's down product over MXFP4, 64 tokens on 256 experts,
// ran at a fifth of the card's bandwidth with 32 columns).
#pragma once
#include "lora_rules.h"
#include "resident_api.h"
#include "wfmt.h"

namespace ftmoe {
namespace rs {

constexpr int kThreads = kWaves * 64;

template <int FMT>
struct Panel {
    static constexpr int EPC = WF<FMT>::EPC;
    static constexpr int LPH = kUnit / (4 * EPC);      // loads per half panel and unit: 4, 2, 1
    static constexpr int UB = 32 * kUnit * 16 / EPC;   // bytes of a unit
    static constexpr int64_t row_bytes(int K) { return (int64_t)K * 16 / EPC; }
};

// One unit of one panel in registers: codes and scales as stored.
template <int FMT>
struct WUnit {
    u32x4_t c[2][Panel<FMT>::LPH];
    uint32_t s[FMT == FT_FMT_MXFP4_B32 ? 2 : 1];
};

// A panel's place: its codes and its scales.
struct PanelRef {
    const uint8_t* codes;      // the panel's first byte
    const uint8_t* scales;     // fp8: the fp32 row of block scales; mxfp4: the panel's e8m0 bytes
};

template <int FMT>
__device__ __forceinline__ PanelRef panel_ref(const uint8_t* codes, const uint8_t* scales, int K, int p) {
    PanelRef r;
    r.codes = codes + (int64_t)p * 32 * Panel<FMT>::row_bytes(K);
    r.scales = scales;
    if constexpr (FMT == FT_FMT_FP8_B128) r.scales = scales + (int64_t)(p >> 2) * (K >> 7) * 4;
    if constexpr (FMT == FT_FMT_MXFP4_B32) r.scales = scales + (int64_t)p * K;
    return r;
}

// The lane's unit inside a lane block pair: chunk column l / 16, row l % 16 of the first half.
__device__ __forceinline__ int lane_unit(int lane) {
    const int g = lane >> 4;
    return (g >> 1) * 64 + (g & 1) * 32 + (lane & 15);
}

// Weights are read once per tile of tokens, mostly once per call: non-temporal, so
// that they leave the caches to the tokens and the partial sums.
template <int FMT>
__device__ __forceinline__ void load_unit(WUnit<FMT>& u, const PanelRef& p, int unit, int lane) {
    constexpr int LPH = Panel<FMT>::LPH;
    const int lu = lane_unit(lane);
    const uint8_t* c = p.codes + (int64_t)unit * Panel<FMT>::UB + lu * 16;
#pragma unroll
    for (int b = 0; b < LPH; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            u.c[h][b] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(c + b * 2048 + h * 256));
    if constexpr (FMT == FT_FMT_FP8_B128) {
        u.s[0] = reinterpret_cast<const uint32_t*>(p.scales)[unit];
    } else if constexpr (FMT == FT_FMT_MXFP4_B32) {
#pragma unroll
        for (int h = 0; h < 2; ++h) u.s[h] = p.scales[unit * 128 + lu + h * 16];
    }
}

// The lane's token values of one unit: `row` is the token's bf16 row.
struct XUnit {
    u32x4_t v[4];
};
template <int FMT>
__device__ __forceinline__ void load_x(XUnit& x, const uint16_t* row, int unit, int lane) {
    constexpr int EPC = Panel<FMT>::EPC, V = EPC / 8;
    const uint16_t* p = row + unit * kUnit + (lane >> 4) * EPC;
#pragma unroll
    for (int b = 0; b < 4 / V; ++b)
#pragma unroll
        for (int j = 0; j < V; ++j) x.v[b * V + j] = *reinterpret_cast<const u32x4_t*>(p + b * 4 * EPC + j * 8);
}

// The A operand of MFMA step j of a 16-byte chunk.
template <int FMT>
__device__ __forceinline__ bf16x8_t a_frag(const u32x4_t c, int j, float scale) {
    if constexpr (FMT == FT_FMT_BF16) {
        return __builtin_bit_cast(bf16x8_t, c);
    } else if constexpr (FMT == FT_FMT_FP8_B128) {
        const uint32_t w0 = j ? c[2] : c[0], w1 = j ? c[3] : c[1];
        const bf16x2_t q0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, false);
        const bf16x2_t q1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, true);
        const bf16x2_t q2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, false);
        const bf16x2_t q3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, true);
        return bf16x8_t{q0[0], q0[1], q1[0], q1[1], q2[0], q2[1], q3[0], q3[1]};
    } else {
        const uint32_t w = c[j];
        const bf16x2_t q0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
        const bf16x2_t q1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
        const bf16x2_t q2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
        const bf16x2_t q3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
        return bf16x8_t{q0[0], q0[1], q1[0], q1[1], q2[0], q2[1], q3[0], q3[1]};
    }
}

// A panel's sums for 16 tokens: rows 16 h + 4 (l / 16) + v of token l % 16.
struct Acc {
    f32x4_t h[2];
};
__device__ __forceinline__ Acc zero_acc() {
    Acc a;
    a.h[0] = a.h[1] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    return a;
}

__device__ __forceinline__ f32x4_t mma(const bf16x8_t a, const u32x4_t b, const f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// acc[i] += panel unit x operand set i, for NX sets that share the weights.
// Only the first nx sets are computed.  The PL planes of a set add to the same
// sums (the high and low halves of a value).  An fp8 unit is one scale block: its
// products are summed unscaled and the fp32 scale multiplies the sum, so no
// weight is rounded.
template <int FMT, int NX, int PL>
__device__ __forceinline__ void mma_unit(Acc (&acc)[NX], const WUnit<FMT>& w, const XUnit (&x)[NX][PL], int nx) {
    constexpr int LPH = Panel<FMT>::LPH, V = Panel<FMT>::EPC / 8;
    Acc blk[NX];
    if constexpr (FMT == FT_FMT_FP8_B128) {
#pragma unroll
        for (int i = 0; i < NX; ++i) blk[i] = zero_acc();
    }
    float s[2] = {1.0f, 1.0f};
    if constexpr (FMT == FT_FMT_MXFP4_B32) {
        s[0] = e8m0_to_f32(w.s[0]);
        s[1] = e8m0_to_f32(w.s[FMT == FT_FMT_MXFP4_B32 ? 1 : 0]);
    }
#pragma unroll
    for (int b = 0; b < LPH; ++b)
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bf16x8_t a = a_frag<FMT>(w.c[h][b], j, s[h]);
#pragma unroll
                for (int i = 0; i < NX; ++i)
                    if (i == 0 || i < nx) {
#pragma unroll
                        for (int p = 0; p < PL; ++p) {
                            f32x4_t& d = FMT == FT_FMT_FP8_B128 ? blk[i].h[h] : acc[i].h[h];
                            d = mma(a, x[i][p].v[b * V + j], d);
                        }
                    }
            }
    if constexpr (FMT == FT_FMT_FP8_B128) {
        const float sc = __uint_as_float(w.s[0]);
#pragma unroll
        for (int i = 0; i < NX; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[i].h[h][v] = fmaf(sc, blk[i].h[h][v], acc[i].h[h][v]);
    }
}

// A value as two bf16: the nearest bf16 and the rest's nearest, together 16
// significant bits or more (relative error at most 2^-17).
__device__ __forceinline__ void split_bf16(float v, uint16_t& hi, uint16_t& lo) {
    hi = f32_to_bf16_rne(v);
    const float r = v - __uint_as_float((uint32_t)hi << 16);
    // an infinity (also one that the rounding made) or NaN is whole in the high half
    lo = (hi & 0x7F80u) == 0x7F80u ? 0 : f32_to_bf16_rne(r);
}

__device__ __forceinline__ float silu(float z) { return z * __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }

constexpr int kRedRow = 36;               // floats of a token's 32 panel rows in LDS, padded

// The wave's sums of operand set i into red[wave][token][row] (nt tokens).
__device__ __forceinline__ void put_acc(float* red, const Acc& acc, int i, int wave, int nt, int lane) {
    const int m = i * kCols + (lane & 15);
    if (m < nt) {
        float* p = red + (wave * nt + m) * kRedRow + 4 * (lane >> 4);
        *reinterpret_cast<f32x4_t*>(p) = acc.h[0];
        *reinterpret_cast<f32x4_t*>(p + 16) = acc.h[1];
    }
}

constexpr int kPlaces = kTile * 32 / kThreads;       // (token, row) places of a tile per thread

// out[i] = the waves' sum, in wave order, at place tid + i kThreads of the tile's [nt][32]
__device__ __forceinline__ void sum_waves(float (&out)[kPlaces], const float* red, int nt, int tid) {
#pragma unroll
    for (int i = 0; i < kPlaces; ++i) {
        const int t = (tid + i * kThreads) >> 5, n = tid & 31;
        float s = 0.0f;
        if (t < nt) {
#pragma unroll
            for (int w = 0; w < kWaves; ++w) s += red[(w * nt + t) * kRedRow + n];
        }
        out[i] = s;
    }
}

// DEPTH steps in flight: load(b, i) fills buffer b for step i, work(b, i) uses it.
template <int DEPTH, typename L, typename W>
__device__ __forceinline__ void pipelined(int n, L&& load, W&& work) {
#pragma unroll
    for (int b = 0; b < DEPTH; ++b)
        if (b < n) load(b, b);
    for (int i = 0; i < n; i += DEPTH)
#pragma unroll
        for (int b = 0; b < DEPTH; ++b)
            if (i + b < n) {
                work(b, i + b);
                if (i + b + DEPTH < n) load(b, i + b + DEPTH);
            }
}

// ---- hand-over between workgroups of one launch --------------------------------
// Partial sums that another workgroup of the same launch reads go through
// agent-scope stores and loads: those bypass the XCD's L2, which other XCDs do
// not see, so no cache has to be written back or invalidated.  A workgroup's
// stores are complete (vmcnt 0) before its arrival is counted.
__device__ __forceinline__ void put_agent(float* p, float v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float get_agent(const float* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void put_agent(double* p, double v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ double get_agent(const double* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Counts this workgroup's arrival at `counter` and tells every thread whether
// it was the last of n; the last one puts the counter back to zero for the
// next call.  All threads of the workgroup call it, after their stores.
__device__ __forceinline__ bool last_arrival(uint32_t* counter, uint32_t n, uint32_t* lds_flag) {
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (threadIdx.x == 0) {
        const uint32_t old = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (old == n - 1) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        *lds_flag = old == n - 1;
    }
    __syncthreads();
    return *lds_flag != 0;
}

}  // namespace rs

}  // namespace ftmoe
