// The C ABI of the paged key-value cache and of the norms around a block
// (include/ftmoe.h): argument validation and the enqueueing calls.  No C++
// exception crosses the boundary.
#include <math.h>

#include "kv.h"

using namespace ftmoe;

namespace {

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int page_shift(int32_t n) {
    for (int s = 4; s <= 8; ++s)
        if (n == 1 << s) return s;
    return -1;
}

ft_status check_pages(int32_t pages, int32_t page_tokens) {
    FT_REQUIRE(page_shift(page_tokens) >= 0, "page_tokens must be 16, 32, 64, 128 or 256");
    FT_REQUIRE(pages >= 1 && (int64_t)pages * page_tokens <= INT32_MAX, "pages * page_tokens must be in 1..2^31 - 1");
    return FT_OK;
}

ft_status check_geometry(const ft_kv_cache* c) {
    FT_REQUIRE(c, "cache is null");
    const ft_status s = check_pages(c->pages, c->page_tokens);
    if (s != FT_OK) return s;
    FT_REQUIRE(c->kv_heads >= 1 && c->kv_heads <= kv::kMaxHeads, "kv_heads must be in 1..%d", kv::kMaxHeads);
    FT_REQUIRE(c->head_dim == 64 || c->head_dim == 128 || c->head_dim == 256, "head_dim must be 64, 128 or 256");
    FT_REQUIRE(c->fmt == FT_KV_BF16 || c->fmt == FT_KV_E4M3, "fmt must be FT_KV_BF16 or FT_KV_E4M3");
    FT_REQUIRE(c->reserved == 0, "reserved must be 0");
    const int64_t page = (int64_t)c->kv_heads * c->page_tokens * c->head_dim * (c->fmt == FT_KV_BF16 ? 2 : 1);
    FT_REQUIRE(c->page_stride >= page && c->page_stride % 16 == 0 && c->page_stride <= INT64_MAX / c->pages,
               "page_stride must be a multiple of 16 and at least a page's %lld bytes", (long long)page);
    return FT_OK;
}

ft_status check_cache(const ft_kv_cache* c, CacheView* out) {
    const ft_status s = check_geometry(c);
    if (s != FT_OK) return s;
    FT_REQUIRE(c->k && c->v, "null pointer: k or v of the cache");
    FT_REQUIRE(aligned(c->k, 16) && aligned(c->v, 16), "k and v of the cache must be 16-byte aligned");
    if (c->fmt == FT_KV_E4M3) {
        FT_REQUIRE(c->k_scale && c->v_scale, "an e4m3 cache needs k_scale and v_scale");
        FT_REQUIRE(aligned(c->k_scale, 4) && aligned(c->v_scale, 4), "the scales must be 4-byte aligned");
    } else {
        FT_REQUIRE(!c->k_scale && !c->v_scale, "a bf16 cache has no scales");
    }
    *out = CacheView{static_cast<uint8_t*>(c->k), static_cast<uint8_t*>(c->v), c->k_scale, c->v_scale, c->page_stride,
                     c->pages, page_shift(c->page_tokens), c->kv_heads, c->head_dim, c->fmt};
    return FT_OK;
}

// `stream` belongs to the current device.
ft_status check_current_stream(void* stream) {
    int dev = 0;
    if (stream && stream != hipStreamLegacy && stream != hipStreamPerThread) FT_HIP(hipGetDevice(&dev));
    return check_stream(stream, dev, "the current device is");
}

ft_status check_rows(const void* p, int64_t stride, int64_t least, const char* name) {
    FT_REQUIRE(p, "null pointer: %s", name);
    FT_REQUIRE(aligned(p, 16), "%s must be 16-byte aligned", name);
    FT_REQUIRE(stride >= least && stride % 8 == 0 && stride <= ((int64_t)1 << 40),
               "%s: the stride must be a multiple of 8 and at least a row's %lld elements", name, (long long)least);
    return FT_OK;
}

ft_status check_q_heads(int32_t q_heads, int32_t kv_heads) {
    FT_REQUIRE(q_heads >= 1 && q_heads <= kv::kMaxHeads && q_heads % kv_heads == 0,
               "q_heads must be a multiple of kv_heads in 1..%d", kv::kMaxHeads);
    return FT_OK;
}

}  // namespace

extern "C" {

ft_status ft_kv_plan(const ft_kv_batch* b, ft_workspace* ws, void* stream) {
    clear_error();
    FT_REQUIRE(b, "batch is null");
    FT_REQUIRE(b->requests >= 0 && b->requests <= kv::kMaxRequests, "requests must be in 0..%d", kv::kMaxRequests);
    const ft_status s = check_pages(b->pages, b->page_tokens);
    if (s != FT_OK) return s;
    FT_REQUIRE(b->width >= 1 && b->width <= kv::kMaxWidth, "width must be in 1..%d", kv::kMaxWidth);
    FT_REQUIRE(b->tokens >= 0 && b->tokens <= kv::kMaxTokens, "tokens must be in 0..%d", kv::kMaxTokens);
    FT_REQUIRE(b->row_tokens >= 0 && (int64_t)b->row_tokens * b->requests <= b->tokens,
               "row_tokens must be 0, or its product with requests at most tokens");
    if (b->requests == 0) return FT_OK;
    FT_REQUIRE(b->context && b->add && b->table && b->free_pages && b->free_count && b->kv_len && b->start && b->counts,
               "null pointer");
    FT_REQUIRE(b->tokens == 0 || (b->slot && b->pos), "null pointer: slot or pos");
    const void* all[] = {b->context, b->add, b->table, b->free_pages, b->free_count, b->kv_len, b->start, b->counts,
                         b->slot, b->pos};
    for (const void* p : all) FT_REQUIRE(aligned(p, 4), "misaligned pointer");
    const ft_status w = check_workspace(ws, 0, stream);
    if (w != FT_OK) return w;
    FT_HIP(launch_kv_plan(*b, ws, (hipStream_t)stream));
    return FT_OK;
}

ft_status ft_kv_append(const ft_kv_cache* cache, const ft_append* a, void* stream) {
    clear_error();
    CacheView c;
    ft_status s = check_cache(cache, &c);
    if (s != FT_OK) return s;
    FT_REQUIRE(a, "args is null");
    FT_REQUIRE(a->tokens >= 0 && a->tokens <= kv::kMaxTokens, "tokens must be in 0..%d", kv::kMaxTokens);
    FT_REQUIRE(a->q_heads >= 0 && a->q_heads <= kv::kMaxHeads, "q_heads must be in 0..%d", kv::kMaxHeads);
    FT_REQUIRE(a->rot >= 0 && a->rot <= c.D && a->rot % 16 == 0, "rot must be a multiple of 16 in 0..head_dim");
    FT_REQUIRE(a->rot == 0 || a->positions >= 1, "positions must be at least 1 where rot is not 0");
    if (a->tokens == 0) return FT_OK;
    s = check_rows(a->k, a->k_stride, (int64_t)c.heads * c.D, "k");
    if (s == FT_OK) s = check_rows(a->v, a->v_stride, (int64_t)c.heads * c.D, "v");
    if (s != FT_OK) return s;
    if (a->q_heads) {
        s = check_rows(a->q, a->q_stride, (int64_t)a->q_heads * c.D, "q");
        if (s == FT_OK) s = check_rows(a->q_out, a->q_out_stride, (int64_t)a->q_heads * c.D, "q_out");
        if (s != FT_OK) return s;
        FT_REQUIRE(a->q_out != a->q || a->q_out_stride == a->q_stride, "q_out may be q with an equal stride only");
    } else {
        FT_REQUIRE(!a->q && !a->q_out, "q and q_out must be NULL where q_heads is 0");
    }
    FT_REQUIRE(a->slot && aligned(a->slot, 4), "slot is null or misaligned");
    if (a->rot) {
        FT_REQUIRE(a->pos && aligned(a->pos, 4), "pos is null or misaligned");
        FT_REQUIRE(a->cos_sin && aligned(a->cos_sin, 16), "cos_sin is null or not 16-byte aligned");
    }
    s = check_current_stream(stream);
    if (s != FT_OK) return s;
    FT_HIP(launch_kv_append(c, *a, (hipStream_t)stream));
    return FT_OK;
}

int64_t ft_kv_attend_workspace(const ft_kv_cache* cache, int32_t q_heads, int32_t max_requests) {
    clear_error();
    if (check_geometry(cache) != FT_OK || check_q_heads(q_heads, cache->kv_heads) != FT_OK) return 0;
    if (max_requests < 1 || max_requests > kv::kMaxRequests) {
        set_error("max_requests must be in 1..%d", kv::kMaxRequests);
        return 0;
    }
    return (int64_t)kv_attend_workspace(q_heads / cache->kv_heads, cache->head_dim);
}

ft_status ft_kv_attend(const ft_kv_cache* cache, const ft_attend* a, ft_workspace* ws, void* stream) {
    clear_error();
    CacheView c;
    ft_status s = check_cache(cache, &c);
    if (s != FT_OK) return s;
    FT_REQUIRE(a, "args is null");
    FT_REQUIRE(a->requests >= 0 && a->requests <= kv::kMaxRequests, "requests must be in 0..%d", kv::kMaxRequests);
    s = check_q_heads(a->q_heads, c.heads);
    if (s != FT_OK) return s;
    FT_REQUIRE(a->width >= 1 && a->width <= kv::kMaxWidth, "width must be in 1..%d", kv::kMaxWidth);
    const int64_t items = (int64_t)a->requests * c.heads * kv::head_blocks(a->q_heads / c.heads);
    FT_REQUIRE(items * (((int64_t)a->width << c.page_shift) / kv::kBlock) <= 2 * kv::kMaxSteps,
               "requests * kv_heads * ceil(group / 16) * width * page_tokens must be at most 2^35");
    FT_REQUIRE(a->window >= 0, "window must be >= 0");
    FT_REQUIRE(fabsf(a->scale) <= 0x1p127f, "scale must be finite, at most 2^127 in size");   // (times log2 e in fp32)
    FT_REQUIRE(a->reserved == 0, "reserved must be 0");
    if (a->requests == 0) return FT_OK;
    const int64_t row = (int64_t)a->q_heads * c.D;
    s = check_rows(a->q, a->q_stride, row, "q");
    if (s == FT_OK) s = check_rows(a->out, a->out_stride, row, "out");
    if (s != FT_OK) return s;
    FT_REQUIRE(a->out != a->q, "out must not be q");
    FT_REQUIRE(a->table && a->kv_len && aligned(a->table, 4) && aligned(a->kv_len, 4) && aligned(a->sinks, 4),
               "table or kv_len is null, or one of table, kv_len and sinks misaligned");
    s = check_workspace(ws, kv_attend_workspace(a->q_heads / c.heads, c.D), stream);
    if (s != FT_OK) return s;
    FT_HIP(launch_kv_attend(c, *a, ws, (hipStream_t)stream));
    return FT_OK;
}

ft_status ft_block_norm(const ft_norm* a, void* stream) {
    clear_error();
    FT_REQUIRE(a, "args is null");
    FT_REQUIRE(a->T >= 0 && a->T <= 1 << 24, "T must be in 0..2^24");
    FT_REQUIRE(a->d >= 8 && a->d <= 32768 && a->d % 8 == 0, "d must be a multiple of 8 in 8..32768");
    FT_REQUIRE((int64_t)a->T * a->d <= (int64_t)1 << 34, "T * d must be at most 2^34");
    const int kind = a->gate_kind & ~FT_GATE_SIGMOID;
    FT_REQUIRE(a->gate_kind >= 0 && kind <= FT_GATE_FULL && (kind || !a->gate_kind), "bad gate_kind");
    FT_REQUIRE(a->eps >= 0 && isfinite(a->eps) && isfinite(a->residual_scale) && isfinite(a->weight_offset),
               "eps must be >= 0, and eps, residual_scale and weight_offset finite");
    FT_REQUIRE(a->block || (!a->post_w && !kind), "post_w and a gate need block");
    FT_REQUIRE((a->normed != nullptr) == (a->pre_w != nullptr), "normed and pre_w belong together");
    FT_REQUIRE((a->gate != nullptr) == (kind != 0), "gate and gate_kind do not agree");
    if (a->T == 0) return FT_OK;
    FT_REQUIRE(a->block || a->residual, "null pointer: block and residual");
    FT_REQUIRE(a->sum || a->normed, "null pointer: sum and normed");
    FT_REQUIRE(aligned(a->post_w, 16) && aligned(a->pre_w, 16), "post_w and pre_w must be 16-byte aligned");
    FT_REQUIRE(aligned(a->gate, kind == FT_GATE_TOKEN ? 2 : 16), "misaligned gate");
    ft_status s = FT_OK;
    if (a->block) s = check_rows(a->block, a->block_stride, a->d, "block");
    if (s == FT_OK && a->residual) s = check_rows(a->residual, a->residual_stride, a->d, "residual");
    if (s == FT_OK && kind == FT_GATE_FULL) s = check_rows(a->gate, a->gate_stride, a->d, "gate");
    if (s == FT_OK && a->sum) s = check_rows(a->sum, a->sum_stride, a->d, "sum");
    if (s == FT_OK && a->normed) s = check_rows(a->normed, a->normed_stride, a->d, "normed");
    if (s != FT_OK) return s;
    const uint16_t* in[2] = {a->block, a->residual};
    const int64_t in_stride[2] = {a->block_stride, a->residual_stride};
    for (int i = 0; i < 2; ++i)
        FT_REQUIRE((!in[i] || in[i] != a->sum || in_stride[i] == a->sum_stride) &&
                       (!in[i] || in[i] != a->normed || in_stride[i] == a->normed_stride),
                   "an output that is an input needs its stride");
    FT_REQUIRE(!a->sum || a->sum != a->normed, "sum and normed must differ");
    s = check_current_stream(stream);
    if (s != FT_OK) return s;
    FT_HIP(launch_block_norm(*a, (hipStream_t)stream));
    return FT_OK;
}

}  // extern "C"
