// Host-side declarations of the paged key-value cache's operators and of the
// norms around a block: checked arguments and the kernel launchers.
#pragma once
#include "kv_rules.h"
#include "resident_api.h"

namespace ftmoe {

// Device-side view of an ft_kv_cache whose arguments were checked.
struct CacheView {
    uint8_t* k;
    uint8_t* v;
    const float* k_scale;
    const float* v_scale;
    int64_t page_stride;
    int pages, page_shift, heads, D, fmt;
};

hipError_t launch_kv_plan(const ft_kv_batch& b, ft_workspace* ws, hipStream_t st);
hipError_t launch_kv_append(const CacheView& c, const ft_append& a, hipStream_t st);
hipError_t launch_kv_attend(const CacheView& c, const ft_attend& a, ft_workspace* ws, hipStream_t st);
size_t kv_attend_workspace(int g, int D);
hipError_t launch_block_norm(const ft_norm& a, hipStream_t st);

// resident.cpp: `stream` is NULL or a created stream of `device` (`owner` words the refusal);
// the workspace is live, large enough and of the current device, which owns the stream.
ft_status check_stream(void* stream, int device, const char* owner);
ft_status check_workspace(const ft_workspace* ws, size_t need, void* stream);

}  // namespace ftmoe
