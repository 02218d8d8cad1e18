// The C ABI of the operators over resident weights (include/ftmoe.h): the
// workspace handle, argument validation and the enqueueing calls.  No C++
// exception crosses the boundary.
#include <new>

#include "resident_api.h"

using namespace ftmoe;

namespace {

constexpr uint64_t kMagic = 0x66746D6F65777331ull;

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The device the workspace lives on has to be current and own the stream.
ft_status check_workspace(const ft_workspace* ws, size_t need, void* stream) {
    FT_REQUIRE(ws, "workspace is null");
    FT_REQUIRE(ws->magic == kMagic, "not a workspace (or a destroyed one)");
    FT_REQUIRE(need <= ws->bytes, "workspace holds %zu bytes; this call needs %zu", ws->bytes, need);
    int dev = -1;
    FT_HIP(hipGetDevice(&dev));
    if (stream) {
        hipDevice_t sd = -1;
        FT_HIP(hipStreamGetDevice((hipStream_t)stream, &sd));
        FT_REQUIRE(sd == ws->device, "the stream belongs to device %d; the workspace was created on device %d", sd,
                   ws->device);
    }
    FT_REQUIRE(dev == ws->device, "device %d is current; the workspace was created on device %d", dev, ws->device);
    return FT_OK;
}

ft_status check_layer_shape(const ft_shape* s) {
    FT_REQUIRE(s, "shape is null");
    FT_REQUIRE(s->experts >= 1 && s->experts <= kMaxRouteExperts, "a layer call supports 1..%d experts",
               kMaxRouteExperts);
    FT_REQUIRE(s->top_k >= 1 && s->top_k <= kMaxTopK && s->top_k <= s->experts, "top_k must be in 1..min(E, %d)",
               kMaxTopK);
    RecordLayout rl;
    FT_REQUIRE(record_layout(*s, &rl), "d_model and d_ff must be positive multiples of 128 and fmt valid");
    return FT_OK;
}

}  // namespace

extern "C" {

ft_status ft_workspace_create(size_t bytes, ft_workspace** out) {
    clear_error();
    FT_REQUIRE(out, "out is null");
    *out = nullptr;
    FT_REQUIRE(bytes > 0 && bytes < ((size_t)1 << 46), "bytes must be positive (and below 2^46)");
    ft_workspace* ws = new (std::nothrow) ft_workspace();
    if (!ws) {
        set_error("out of host memory");
        return FT_ERR_NOMEM;
    }
    hipError_t e = hipGetDevice(&ws->device);
    if (e == hipSuccess) {
        e = hipMalloc(reinterpret_cast<void**>(&ws->mem), kCounterBytes + bytes);
        if (e == hipErrorOutOfMemory || e == hipErrorMemoryAllocation) {
            (void)hipGetLastError();
            delete ws;
            set_error("a workspace of %zu bytes does not fit the device", bytes);
            return FT_ERR_NOMEM;
        }
    }
    if (e == hipSuccess) e = hipMemset(ws->mem, 0, kCounterBytes);
    if (e == hipSuccess) e = hipDeviceSynchronize();
    if (e != hipSuccess) {
        set_error("ft_workspace_create failed: %s", hipGetErrorString(e));
        if (ws->mem) (void)hipFree(ws->mem);
        delete ws;
        return FT_ERR_HIP;
    }
    ws->bytes = bytes;
    ws->magic = kMagic;
    *out = ws;
    return FT_OK;
}

ft_status ft_workspace_destroy(ft_workspace* ws) {
    clear_error();
    if (!ws) return FT_OK;
    FT_REQUIRE(ws->magic == kMagic, "not a workspace (or a destroyed one)");
    ws->magic = 0;
    void* mem = ws->mem;
    delete ws;
    FT_HIP(hipDeviceSynchronize());
    FT_HIP(hipFree(mem));
    return FT_OK;
}

int64_t ft_moe_layer_workspace(const ft_shape* shape, int32_t max_tokens) {
    clear_error();
    if (check_layer_shape(shape) != FT_OK) return 0;
    if (max_tokens < 1 || max_tokens > kMaxLayerTokens) {
        set_error("max_tokens must be in 1..%d", kMaxLayerTokens);
        return 0;
    }
    return (int64_t)layer_workspace(*shape, max_tokens);
}

ft_status ft_moe_layer(const ft_shape* shape, const uint16_t* x, const uint16_t* wr, const void* records,
                       int64_t record_stride, int32_t T, const uint16_t* base, int32_t* ids, float* w, uint16_t* y,
                       ft_workspace* ws, void* stream) {
    clear_error();
    ft_status s = check_layer_shape(shape);
    if (s != FT_OK) return s;
    FT_REQUIRE(T >= 0 && T <= kMaxLayerTokens, "T must be in 0..%d", kMaxLayerTokens);
    if (T == 0) return FT_OK;
    FT_REQUIRE(x && wr && records && ids && w && y, "null pointer");
    LayerArgs a;
    (void)record_layout(*shape, &a.rl);
    FT_REQUIRE(record_stride >= a.rl.S && record_stride % 16 == 0,
               "record_stride must be a multiple of 16 and at least the record's %lld bytes", (long long)a.rl.S);
    FT_REQUIRE(aligned(x, 16) && aligned(wr, 16) && aligned(records, 16), "x, wr and records must be 16-byte aligned");
    FT_REQUIRE(aligned(y, 2) && aligned(base, 2) && aligned(ids, 4) && aligned(w, 4), "misaligned output or base");
    s = check_workspace(ws, layer_workspace(*shape, T), stream);
    if (s != FT_OK) return s;
    a.x = x;
    a.wr = wr;
    a.rec = static_cast<const uint8_t*>(records);
    a.stride = record_stride;
    a.T = T;
    a.base = base;
    a.ids = ids;
    a.w = w;
    a.y = y;
    FT_HIP(launch_layer(*shape, a, ws, (hipStream_t)stream));
    return FT_OK;
}

}  // extern "C"
