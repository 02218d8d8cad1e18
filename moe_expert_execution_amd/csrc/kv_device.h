// Device code shared by the kernels of the key-value cache and of the norms.
#pragma once
#include "kv.h"
#include "wfmt.h"

namespace ftmoe {
namespace kv {

// Inclusive prefix sum over the wave: rows of 16 lanes by shifts, then their last lanes into the
// rows behind (vector instructions alone, an eighth of six exchanges' latency).
__device__ __forceinline__ int wave_scan(int x) {
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);    // row_shr 1, 2, 4, 8
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);    // row_bcast 15 into rows 1 and 3
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);    // row_bcast 31 into rows 2 and 3
    return x;
}

// 16 bytes read or written once: where a call moves more than the XCDs' L2s hold (32 MiB), past them.
template <bool STREAM>
__device__ __forceinline__ u32x4_t load16(const void* p) {
    if constexpr (STREAM) return __builtin_nontemporal_load(static_cast<const u32x4_t*>(p));
    else return *static_cast<const u32x4_t*>(p);
}
template <bool STREAM>
__device__ __forceinline__ void store16(void* p, const u32x4_t v) {
    if constexpr (STREAM) __builtin_nontemporal_store(v, static_cast<u32x4_t*>(p));
    else *static_cast<u32x4_t*>(p) = v;
}
constexpr int64_t kStreamBytes = 32ll << 20;

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    return (uint32_t)f32_to_bf16_rne(lo) | (uint32_t)f32_to_bf16_rne(hi) << 16;
}

}  // namespace kv
}  // namespace ftmoe
