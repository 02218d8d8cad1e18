// Host-side declarations of the operators over resident weights: the
// workspace handle and the kernel launchers.
#pragma once
#include "common.h"

namespace ftmoe {

// ---- the workspace handle --------------------------------------------------------
// [0, kCounterBytes): arrival counters, zero between calls; then the calls' buffers.
constexpr size_t kCounterBytes = 64 << 10;
constexpr int kMaxLayerTokens = 64;       // tokens of one ft_moe_layer call
constexpr int kMaxRouteExperts = 256;     // experts of one ft_moe_layer call
// Polls of the wait inside ft_moe_layer's one-launch form before a workgroup gives
// up (its part of y is NaN then): seconds, where a hand-over takes microseconds.
// Only a workspace used by two calls at once gets there.
constexpr uint32_t kMaxPolls = 1u << 22;

}  // namespace ftmoe

struct ft_workspace {
    uint8_t* mem;
    size_t bytes;        // of the buffers after the counters
    int device;
    ft_workspace* next;  // in the list of live workspaces (resident.cpp)
    // for tests: the bound in the lower half of the launch's workgroups (FTMOE_LAYER_WAIT_POLLS)
    uint32_t low_polls;
    // for tests: odd workgroups leave their gate/up numbers to those that wait (FTMOE_LAYER_ABSENT)
    int absent;
};

namespace ftmoe {

// Launches f(a) and returns the launch's own status: hipGetLastError() after it
// would also report, and take away, an error that an earlier call of the
// program left behind, and the launches after this one would be left out.
template <typename A>
hipError_t launch(void (*f)(A), dim3 grid, dim3 block, size_t lds, hipStream_t st, const A& a) {
    void* args[] = {const_cast<A*>(&a)};
    return hipLaunchKernel(reinterpret_cast<const void*>(f), grid, block, args, lds, st);
}

struct LayerArgs {
    const uint16_t* x;
    const uint16_t* wr;
    const uint8_t* rec;
    int64_t stride;
    RecordLayout rl;
    int T;
    const uint16_t* base;
    int32_t* ids;
    float* w;
    uint16_t* y;
};
// ..._call_bytes: what a call of exactly T tokens takes; ..._workspace: the
// largest of any call of up to T.
size_t layer_call_bytes(const ft_shape& s, int T);
size_t layer_workspace(const ft_shape& s, int T);
hipError_t launch_layer(const ft_shape& s, const LayerArgs& a, ft_workspace* ws, hipStream_t st);

constexpr int kMaxRank = 128;             // ranks of an adapter
constexpr int kMaxLoraTokens = 65535;

// The device side of an ft_lora (count 0: no adapters).
struct LoraView {
    int count = 0, max_rank = 0;
    const int32_t* rank = nullptr;
    const float* scale = nullptr;
    const uint16_t* a = nullptr;
    const uint16_t* b = nullptr;
};
struct MatrixView {
    int n, K, fmt;
    const uint8_t* codes;
    const uint8_t* scales;
};
// The prompt-length products (gemm.hip): GU reads x [T x d] and writes h = silu(.) * (.)
// [T x f] in bf16 from the matrices codes[0], codes[1]; otherwise reads Hin [T x f] and
// writes Y [T x d] from codes[0].
struct LoraGemmArgs {
    const uint16_t* x;
    const uint16_t* Hin;
    uint16_t* Hout;
    uint16_t* Y;
    int T, d, f;
    uint32_t x_bytes, h_bytes;         // extents of x and Hin, below 4 GiB
    const uint8_t* codes[2];
    const uint8_t* scales[2];
    LoraView lora[2];
    const uint16_t* vhi[2];            // [vparts][T][R] v over parts of K, two bf16 planes
    const uint16_t* vlo[2];
    int vparts;
    const int32_t* adapter;
    const uint16_t* base;
};
hipError_t launch_lora_gemm(int fmt, bool gu, const LoraGemmArgs& a, hipStream_t st);

size_t lora_project_call_bytes(int n, int K, int max_rank, int T);
size_t lora_expert_call_bytes(const ft_shape& s, int max_rank, int T);
size_t lora_project_workspace(int n, int K, int max_rank, int max_tokens);
size_t lora_expert_workspace(const ft_shape& s, int max_rank, int max_tokens);
hipError_t launch_lora_project(const MatrixView& m, const LoraView* lora, const int32_t* adapter, const uint16_t* x,
                               int T, const uint16_t* base, uint16_t* y, ft_workspace* ws, hipStream_t st);
hipError_t launch_lora_expert(const ft_shape& sh, const RecordLayout& rl, const uint8_t* rec, const LoraView* gate,
                              const LoraView* up, const LoraView* down, const int32_t* adapter, const uint16_t* x,
                              int T, const uint16_t* base, uint16_t* y, ft_workspace* ws, hipStream_t st);

}  // namespace ftmoe
