// The C ABI of the operators over resident weights (include/ftmoe.h): the
// workspace handle, argument validation and the enqueueing calls.  No C++
// exception crosses the boundary.
#include <stdlib.h>

#include <mutex>
#include <new>

#include "resident_api.h"

using namespace ftmoe;

namespace {

// The live workspaces.  A handle is looked up here before it is read, so that a
// destroyed one is told by its address alone.
std::mutex g_live_mutex;
ft_workspace* g_live = nullptr;

bool is_live(const ft_workspace* ws) {
    std::lock_guard<std::mutex> lock(g_live_mutex);
    const ft_workspace* p = g_live;
    while (p && p != ws) p = p->next;
    return p != nullptr;
}

// Takes a live workspace out of the list; false if it is none.
bool unlink_live(ft_workspace* ws) {
    std::lock_guard<std::mutex> lock(g_live_mutex);
    for (ft_workspace** p = &g_live; *p; p = &(*p)->next)
        if (*p == ws) {
            *p = ws->next;
            return true;
        }
    return false;
}

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

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

ft_status check_rank(int32_t r) {
    FT_REQUIRE(r == 0 || (r >= 16 && r <= kMaxRank && r % 16 == 0), "max_rank must be a multiple of 16 in 16..%d",
               kMaxRank);
    return FT_OK;
}

// *out: the pool's device view, count 0 when there are no adapters
ft_status check_lora(const ft_lora* l, const int32_t* adapter, const char* name, LoraView* out) {
    *out = LoraView();
    if (!l) return FT_OK;
    FT_REQUIRE(l->count >= 0, "%s: count must be >= 0", name);
    if (l->count == 0) return FT_OK;
    FT_REQUIRE(l->max_rank > 0 && check_rank(l->max_rank) == FT_OK,
               "%s: max_rank must be a multiple of 16 in 16..%d", name, kMaxRank);
    FT_REQUIRE(l->rank && l->scale && l->a && l->b, "%s: null pointer", name);
    FT_REQUIRE(aligned(l->a, 16) && aligned(l->b, 16), "%s: a and b must be 16-byte aligned", name);
    FT_REQUIRE(aligned(l->rank, 4) && aligned(l->scale, 4), "%s: rank and scale must be 4-byte aligned", name);
    FT_REQUIRE(adapter, "%s: adapters are given but adapter is null", name);
    FT_REQUIRE(aligned(adapter, 4), "adapter must be 4-byte aligned");
    out->count = l->count;
    out->max_rank = l->max_rank;
    out->rank = l->rank;
    out->scale = l->scale;
    out->a = l->a;
    out->b = l->b;
    return FT_OK;
}

ft_status check_matrix(const ft_matrix* m) {
    FT_REQUIRE(m, "matrix is null");
    FT_REQUIRE(m->n >= 128 && m->K >= 128 && m->n % 128 == 0 && m->K % 128 == 0 && m->n <= 32768 && m->K <= 32768,
               "n and K must be multiples of 128 in 128..32768");
    FT_REQUIRE(m->fmt == FT_FMT_BF16 || m->fmt == FT_FMT_FP8_B128 || m->fmt == FT_FMT_MXFP4_B32, "bad fmt");
    return FT_OK;
}

ft_status check_expert_shape(const ft_shape* s) {
    FT_REQUIRE(s, "shape is null");
    RecordLayout rl;
    FT_REQUIRE(record_layout(*s, &rl), "d_model and d_ff must be positive multiples of 128 and fmt valid");
    return FT_OK;
}

ft_status check_lora_tokens(int32_t T) {
    FT_REQUIRE(T >= 0 && T <= kMaxLoraTokens, "T must be in 0..%d", kMaxLoraTokens);
    return FT_OK;
}

}  // namespace

namespace ftmoe {

ft_status check_stream(void* stream, int device, const char* owner) {
    // The runtime's two handles that are no stream objects: a call with one of them,
    // asked about its device or launched on, has ended the process.
    FT_REQUIRE(stream != hipStreamLegacy && stream != hipStreamPerThread,
               "stream must be NULL or a created stream, not hipStreamLegacy or hipStreamPerThread");
    if (stream) {
        hipDevice_t sd = -1;
        FT_HIP(hipStreamGetDevice((hipStream_t)stream, &sd));
        FT_REQUIRE(sd == device, "the stream belongs to device %d; %s device %d", sd, owner, device);
    }
    return FT_OK;
}

// The device the workspace lives on has to be current and own the stream.
ft_status check_workspace(const ft_workspace* ws, size_t need, void* stream) {
    FT_REQUIRE(ws, "workspace is null");
    FT_REQUIRE(is_live(ws), "not a workspace (or a destroyed one)");
    FT_REQUIRE(need <= ws->bytes, "workspace holds %zu bytes; this call needs %zu", ws->bytes, need);
    const ft_status s = check_stream(stream, ws->device, "the workspace was created on");
    if (s != FT_OK) return s;
    int dev = -1;
    FT_HIP(hipGetDevice(&dev));
    FT_REQUIRE(dev == ws->device, "device %d is current; the workspace was created on device %d", dev, ws->device);
    return FT_OK;
}

}  // namespace ftmoe

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
    ws->low_polls = kMaxPolls;
    if (const char* v = getenv("FTMOE_LAYER_WAIT_POLLS")) ws->low_polls = (uint32_t)strtoul(v, nullptr, 10);
    if (const char* v = getenv("FTMOE_LAYER_ABSENT")) ws->absent = atoi(v) != 0;
    {
        std::lock_guard<std::mutex> lock(g_live_mutex);
        ws->next = g_live;
        g_live = ws;
    }
    *out = ws;
    return FT_OK;
}

ft_status ft_workspace_destroy(ft_workspace* ws) {
    clear_error();
    if (!ws) return FT_OK;
    FT_REQUIRE(is_live(ws), "not a workspace (or a destroyed one)");
    // calls that use it run on its own device, whichever is current
    const int device = ws->device;
    int dev = device;
    hipError_t e = hipGetDevice(&dev);
    if (e == hipSuccess && dev != device) e = hipSetDevice(device);
    if (e == hipSuccess) e = hipDeviceSynchronize();
    if (e == hipSuccess && unlink_live(ws)) {     // (a wait that was refused, as in a capture, leaves it as it was)
        e = hipFree(ws->mem);
        delete ws;
    }
    if (dev != device) {
        const hipError_t back = hipSetDevice(dev);
        if (e == hipSuccess) e = back;
    }
    FT_HIP(e);
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
    s = check_workspace(ws, layer_call_bytes(*shape, T), stream);
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

int64_t ft_lora_project_workspace(const ft_matrix* m, int32_t max_rank, int32_t max_tokens) {
    clear_error();
    if (check_matrix(m) != FT_OK || check_rank(max_rank) != FT_OK) return 0;
    if (max_tokens < 1 || max_tokens > kMaxLoraTokens) {
        set_error("max_tokens must be in 1..%d", kMaxLoraTokens);
        return 0;
    }

    return (int64_t)lora_project_workspace(m->n, m->K, max_rank, max_tokens) + 256;
}

ft_status ft_lora_project(const ft_matrix* m, const ft_lora* lora, const uint16_t* x, const int32_t* adapter,
                          int32_t T, const uint16_t* base, uint16_t* y, ft_workspace* ws, void* stream) {
    clear_error();
    ft_status s = check_matrix(m);
    if (s == FT_OK) s = check_lora_tokens(T);
    if (s != FT_OK) return s;
    if (T == 0) return FT_OK;
    FT_REQUIRE(m->codes && (m->fmt == FT_FMT_BF16 || m->scales) && x && y, "null pointer");
    FT_REQUIRE(aligned(m->codes, 16) && aligned(x, 16), "x and the codes must be 16-byte aligned");
    FT_REQUIRE(aligned(m->scales, m->fmt == FT_FMT_FP8_B128 ? 4 : 1), "the scales must be 4-byte aligned");
    FT_REQUIRE(aligned(y, 2) && aligned(base, 2), "misaligned output or base");
    LoraView l;
    s = check_lora(lora, adapter, "lora", &l);
    if (s != FT_OK) return s;
    s = check_workspace(ws, lora_project_call_bytes(m->n, m->K, l.max_rank, T), stream);
    if (s != FT_OK) return s;
    MatrixView v;
    v.n = m->n;
    v.K = m->K;
    v.fmt = m->fmt;
    v.codes = static_cast<const uint8_t*>(m->codes);
    v.scales = static_cast<const uint8_t*>(m->scales);
    FT_HIP(launch_lora_project(v, l.count > 0 ? &l : nullptr, adapter, x, T, base, y, ws, (hipStream_t)stream));
    return FT_OK;
}

int64_t ft_lora_expert_workspace(const ft_shape* shape, int32_t max_rank, int32_t max_tokens) {
    clear_error();
    if (check_expert_shape(shape) != FT_OK || check_rank(max_rank) != FT_OK) return 0;
    if (max_tokens < 1 || max_tokens > kMaxLoraTokens) {
        set_error("max_tokens must be in 1..%d", kMaxLoraTokens);
        return 0;
    }
    return (int64_t)lora_expert_workspace(*shape, max_rank, max_tokens);
}

ft_status ft_lora_expert(const ft_shape* shape, const void* record, const ft_lora* gate, const ft_lora* up,
                         const ft_lora* down, const uint16_t* x, const int32_t* adapter, int32_t T,
                         const uint16_t* base, uint16_t* y, ft_workspace* ws, void* stream) {
    clear_error();
    ft_status s = check_expert_shape(shape);
    if (s == FT_OK) s = check_lora_tokens(T);
    if (s != FT_OK) return s;
    if (T == 0) return FT_OK;
    FT_REQUIRE(record && x && y, "null pointer");
    FT_REQUIRE(aligned(record, 16) && aligned(x, 16), "x and the record must be 16-byte aligned");
    FT_REQUIRE(aligned(y, 2) && aligned(base, 2), "misaligned output or base");
    const ft_lora* pools[3] = {gate, up, down};
    const char* names[3] = {"gate", "up", "down"};
    LoraView l[3];
    int32_t R = 0;
    for (int i = 0; i < 3; ++i) {
        s = check_lora(pools[i], adapter, names[i], &l[i]);
        if (s != FT_OK) return s;
        if (l[i].max_rank > R) R = l[i].max_rank;
    }
    s = check_workspace(ws, lora_expert_call_bytes(*shape, R, T), stream);
    if (s != FT_OK) return s;
    RecordLayout rl;
    (void)record_layout(*shape, &rl);
    auto view = [&](int i) { return l[i].count > 0 ? &l[i] : nullptr; };
    FT_HIP(launch_lora_expert(*shape, rl, static_cast<const uint8_t*>(record), view(0), view(1), view(2), adapter, x, T,
                              base, y, ws, (hipStream_t)stream));
    return FT_OK;
}

}  // extern "C"
