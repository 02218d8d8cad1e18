// Streaming a panel-ordered weight matrix against a few tokens on the matrix
// cores: the device code shared by the operators over resident weights
// (moe_layer.hip, lora.hip).
//
// A 32-row panel is read in units of 128 along K, each unit LBU lane blocks
// of 1 KiB: lane l of a wave holds row l % 32 at chunk column l / 32, which is
// the A operand of v_mfma_f32_32x32x16_bf16 as it stands (codes are converted
// to bf16 in registers, which is exact for e4m3 and for e2m1 times a power of
// two).  The tokens are the B operand: lane l holds token l % 32 at the same
// K positions, read from memory (L2) as EPC contiguous bf16.  So a panel
// streams from HBM once whatever the token count up to 32, and lane l ends
// with token l % 32 and, per group q, rows 8 q + 4 (l / 32) .. + 3 of the panel.
// A matrix-core step takes 32 cycles per KiB of bf16 weights (16 KiB of
// e2m1: 128), several times faster than a CU's share of HBM, so the columns
// past the token count cost nothing.
#pragma once
#include "resident_api.h"
#include "wfmt.h"

namespace ftmoe {
namespace rs {

constexpr int kWaves = 8;                 // waves of a streaming workgroup, splitting K
constexpr int kThreads = kWaves * 64;
constexpr int kUnit = 128;                // elements along K per unit (one fp8 scale block)
constexpr int kTile = 32;                 // tokens of one operand tile

template <int FMT>
struct Panel {
    static constexpr int EPC = WF<FMT>::EPC;
    static constexpr int LBU = kUnit / (2 * EPC);      // lane blocks per unit: 8, 4, 2
    static constexpr int64_t row_bytes(int K) { return (int64_t)K * 16 / EPC; }
};

// One unit of one panel in registers: codes and scales as stored.
template <int FMT>
struct WUnit {
    u32x4_t c[Panel<FMT>::LBU];
    uint32_t s[FMT == FT_FMT_MXFP4_B32 ? Panel<FMT>::LBU : 1];
};

// A panel's place: codes of row panel p, its scales, and the matrix's K.
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

// Weights are read once per call: non-temporal, so that they leave the caches
// to the tokens and the partial sums.
template <int FMT>
__device__ __forceinline__ void load_unit(WUnit<FMT>& u, const PanelRef& p, int unit, int lane) {
    constexpr int LBU = Panel<FMT>::LBU;
    const uint8_t* c = p.codes + (int64_t)unit * (LBU * 1024) + lane * 16;
#pragma unroll
    for (int b = 0; b < LBU; ++b) u.c[b] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(c + b * 1024));
    if constexpr (FMT == FT_FMT_FP8_B128) {
        u.s[0] = reinterpret_cast<const uint32_t*>(p.scales)[unit];
    } else if constexpr (FMT == FT_FMT_MXFP4_B32) {
#pragma unroll
        for (int b = 0; b < LBU; ++b) u.s[b] = p.scales[(unit * LBU + b) * 64 + lane];
    }
}

// The lane's token values of one unit: `row` is the token's bf16 row.
struct XUnit {
    u32x4_t v[8];
};
template <int FMT>
__device__ __forceinline__ void load_x(XUnit& x, const uint16_t* row, int unit, int lane) {
    constexpr int EPC = Panel<FMT>::EPC, LBU = Panel<FMT>::LBU, V = EPC / 8;
    const uint16_t* p = row + unit * kUnit + (lane >> 5) * EPC;
#pragma unroll
    for (int b = 0; b < LBU; ++b)
#pragma unroll
        for (int j = 0; j < V; ++j) x.v[b * V + j] = *reinterpret_cast<const u32x4_t*>(p + b * 2 * EPC + j * 8);
}

// The A operand of MFMA step j of a lane block.
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

__device__ __forceinline__ f32x16_t zero16() {
    f32x16_t z;
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = 0.0f;
    return z;
}

// acc += panel unit x tokens, for NX operand sets that share the weights
// (token tiles, or the high and low halves of one).  An fp8 unit is one scale
// block: its products are summed unscaled and the fp32 scale multiplies the
// sum, so no weight is rounded.
template <int FMT, int NX>
__device__ __forceinline__ void mma_unit(f32x16_t (&acc)[NX], const WUnit<FMT>& w, const XUnit* const (&x)[NX]) {
    constexpr int LBU = Panel<FMT>::LBU, V = Panel<FMT>::EPC / 8;
    if constexpr (FMT == FT_FMT_FP8_B128) {
        f32x16_t blk[NX];
#pragma unroll
        for (int i = 0; i < NX; ++i) blk[i] = zero16();
#pragma unroll
        for (int b = 0; b < LBU; ++b)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const bf16x8_t a = a_frag<FMT>(w.c[b], j, 1.0f);
#pragma unroll
                for (int i = 0; i < NX; ++i)
                    blk[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, __builtin_bit_cast(bf16x8_t, x[i]->v[b * V + j]),
                                                                     blk[i], 0, 0, 0);
            }
        const float s = __uint_as_float(w.s[0]);
#pragma unroll
        for (int i = 0; i < NX; ++i)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][v] = fmaf(s, blk[i][v], acc[i][v]);
    } else {
#pragma unroll
        for (int b = 0; b < LBU; ++b) {
            const float s = FMT == FT_FMT_MXFP4_B32 ? e8m0_to_f32(w.s[FMT == FT_FMT_MXFP4_B32 ? b : 0]) : 1.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const bf16x8_t a = a_frag<FMT>(w.c[b], j, s);
#pragma unroll
                for (int i = 0; i < NX; ++i)
                    acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, __builtin_bit_cast(bf16x8_t, x[i]->v[b * V + j]),
                                                                     acc[i], 0, 0, 0);
            }
        }
    }
}

// A value as two bf16: the nearest bf16 and the rest's nearest, together 16
// significant bits or more (relative error at most 2^-17).
__device__ __forceinline__ void split_bf16(float v, uint16_t& hi, uint16_t& lo) {
    hi = f32_to_bf16_rne(v);
    const float r = v - __uint_as_float((uint32_t)hi << 16);
    // an infinity or NaN is whole in the high half (its rest would be NaN)
    lo = (__float_as_uint(v) & 0x7F800000u) == 0x7F800000u ? 0 : f32_to_bf16_rne(r);
}

__device__ __forceinline__ float silu(float z) { return z * __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }

constexpr int kRedRow = 36;               // floats of a token's 32 panel rows in LDS, padded

// Adds the waves' accumulators in wave order: red[wave][token][row].
__device__ __forceinline__ void put_acc(float* red, const f32x16_t& acc, int wave, int tile_tokens, int lane) {
    const int m = lane & 31, g = lane >> 5;
    if (m < tile_tokens) {
        float* p = red + ((int64_t)wave * tile_tokens + m) * kRedRow + 4 * g;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            *reinterpret_cast<f32x4_t*>(p + 8 * q) =
                f32x4_t{acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
    }
}

// out[i] = the waves' sum at place tid + i kThreads of the tile's [nt][32]
__device__ __forceinline__ void sum_waves(float (&out)[kTile * 32 / kThreads], const float* red, int nt, int tid) {
#pragma unroll
    for (int i = 0; i < kTile * 32 / kThreads; ++i) {
        const int t = (tid + i * kThreads) >> 5, n = tid & 31;
        float s = 0.0f;
        if (t < nt) {
#pragma unroll
            for (int w = 0; w < kWaves; ++w) s += red[(w * nt + t) * kRedRow + n];
        }
        out[i] = s;
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
