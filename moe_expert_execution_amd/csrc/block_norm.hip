// The norms after one block and before the next, with the block's gate and the
// residual between them (ft_block_norm):
//   u = b / sqrt(mean b^2 + eps) * w1,  s = a r + g u,  n = s / sqrt(mean s^2 + eps) * w2.
//
// Every input is read once and every output written once: a row stays in
// registers, 8 elements per 16-byte unit, between its two sums of squares, which
// are the only points where its threads meet.  The second norm uses the fp32
// sum; rounding it first would feed the next block the residual's bf16 error
// twice.  Memory bounds it, or the launch where there are few rows: 4,096 rows of 7,168 with
// both norms and a gate per element 55 us, 5.3 TB/s (a large copy: 5.1 to 5.3), one row of 2,048 3.0 us.
#include <float.h>

#include "kv_device.h"

namespace ftmoe {
namespace {

// Sum over the threads of a row: R lanes of a wave, or the whole workgroup (R > 64).
template <int R>
__device__ __forceinline__ float row_sum(float v, float* lds) {
#pragma unroll
    for (int m = 1; m < (R < 64 ? R : 64); m *= 2) v += __shfl_xor(v, m);
    if constexpr (R > 64) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) lds[wave] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < R / 64; ++w) v += lds[w];
    }
    return v;
}

__device__ __forceinline__ float element(const u32x4_t u, int i) {
    return i & 1 ? bf16hi(u[i >> 1]) : bf16lo(u[i >> 1]);
}

__device__ __forceinline__ float sigmoid_of(float x) { return __builtin_amdgcn_rcpf(1.0f + __expf(-x)); }

// Rows whose squares leave fp32's range (below 2^-50 or above 2^56 in size, where eps does not carry them) are summed again,
// scaled by a power of two; all threads of a row see the same mean, so they go there together.  The first choice makes the
// square of any bf16 below 2^-42 a normal number, the second keeps 32,768 squares of the largest finite.
constexpr float kLeastMean = 0x1p-100f, kUp = 0x1p96f, kDown = 0x1p-72f;
__device__ __forceinline__ bool leaves_range(float mean) {
    return __builtin_expect(mean < kLeastMean || mean > FLT_MAX, false);
}

// R threads per row, U units of 8 elements per thread; a workgroup is one row, or 256 threads where rows are
// a wave's or smaller.
constexpr int threads_of(int R) { return R > 64 ? R : 256; }

template <int R, int U, bool STREAM>
__global__ void __launch_bounds__(threads_of(R)) norm_kernel(ft_norm a) {
    constexpr int kThreads = threads_of(R);
    __shared__ float lds[4][R > 64 ? R / 64 : 1];
    const int64_t t = (int64_t)blockIdx.x * (kThreads / R) + threadIdx.x / R;
    const int lane = threadIdx.x % R, units = a.d >> 3;
    if (t >= a.T) return;                   // (rows of a workgroup-wide reduction have one row a workgroup)
    const int kind = a.gate_kind & ~FT_GATE_SIGMOID;
    const bool sigmoid = a.gate_kind & FT_GATE_SIGMOID;
    const float inv_d = 1.0f / (float)a.d;
    const u32x4_t zero = {0, 0, 0, 0};
    u32x4_t b[U], r[U], g[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int u = lane + i * R;
        const bool on = u < units;
        b[i] = on && a.block ? kv::load16<STREAM>(a.block + t * a.block_stride + u * 8) : zero;
        r[i] = on && a.residual ? kv::load16<STREAM>(a.residual + t * a.residual_stride + u * 8) : zero;
        g[i] = on && kind == FT_GATE_FULL    ? kv::load16<STREAM>(a.gate + t * a.gate_stride + u * 8)
               : on && kind == FT_GATE_CHANNEL ? kv::load16<false>(a.gate + u * 8)
                                               : zero;
    }
    float token_gate = 1.0f;
    if (kind == FT_GATE_TOKEN) {
        token_gate = __uint_as_float((uint32_t)a.gate[t] << 16);
        if (sigmoid) token_gate = sigmoid_of(token_gate);
    }
    float s1 = token_gate;
    if (a.post_w) {
        float q = 0.0f;
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) q = fmaf(element(b[i], e), element(b[i], e), q);
        float mean = row_sum<R>(q, lds[0]) * inv_d + a.eps, one = 1.0f;
        if (leaves_range(mean)) {
            const bool up = mean < kLeastMean;
            const float f = up ? kUp : kDown;
            q = 0.0f;
#pragma unroll
            for (int i = 0; i < U; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float x = bf16lo(b[i][e]) * f, y = bf16hi(b[i][e]) * f;
                    q = fmaf(x, x, fmaf(y, y, q));
                    if (up) b[i][e] = pack_bf16_trunc(x, y);             // (exact: the block stays scaled)
                }
            mean = row_sum<R>(q, lds[1]) * inv_d + a.eps * f * f;
            if (!up) one = f;
        }
        s1 = token_gate * (one / sqrtf(mean));
    }
    float s[U][8];
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int u = lane + i * R;
        const bool on = u < units;
        const u32x4_t w = on && a.post_w ? kv::load16<false>(a.post_w + u * 8) : zero;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float v = element(b[i], e) * s1;
            if (a.post_w) v *= a.weight_offset + element(w, e);
            if (kind == FT_GATE_FULL || kind == FT_GATE_CHANNEL) {
                const float x = element(g[i], e);
                v *= sigmoid ? sigmoid_of(x) : x;
            }
            if (a.residual) v = fmaf(a.residual_scale, element(r[i], e), v);
            s[i][e] = v;
            q = fmaf(v, v, q);
        }
        if (on && a.sum) {
            u32x4_t o;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = kv::pack_bf16(s[i][2 * e], s[i][2 * e + 1]);
            kv::store16<STREAM>(a.sum + t * a.sum_stride + u * 8, o);
        }
    }
    if (!a.normed) return;
    float mean = row_sum<R>(q, lds[2]) * inv_d + a.eps, one = 1.0f;
    if (leaves_range(mean)) {
        const bool up = mean < kLeastMean;
        const float f = up ? kUp : kDown;
        q = 0.0f;
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = s[i][e] * f;
                q = fmaf(x, x, q);
                if (up) s[i][e] = x;
            }
        mean = row_sum<R>(q, lds[3]) * inv_d + a.eps * f * f;
        if (!up) one = f;
    }
    const float s2 = one / sqrtf(mean);
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int u = lane + i * R;
        if (u >= units) continue;
        const u32x4_t w = kv::load16<false>(a.pre_w + u * 8);
        u32x4_t o;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o[e] = kv::pack_bf16(s[i][2 * e] * s2 * (a.weight_offset + element(w, 2 * e)),
                             s[i][2 * e + 1] * s2 * (a.weight_offset + element(w, 2 * e + 1)));
        kv::store16<STREAM>(a.normed + t * a.normed_stride + u * 8, o);
    }
}

template <int R, int U>
hipError_t go(const ft_norm& a, hipStream_t st) {
    constexpr int kThreads = threads_of(R);
    const int64_t rows = kThreads / R;
    const dim3 grid((unsigned)((a.T + rows - 1) / rows));
    // Calls that move more than the L2s hold stream past them (4,096 rows of 7,168, a gate of every element:
    // 56 us, 64 through them).
    const int full = (a.block != nullptr) + (a.residual != nullptr) + ((a.gate_kind & ~FT_GATE_SIGMOID) == FT_GATE_FULL) +
                     (a.sum != nullptr) + (a.normed != nullptr);
    if ((int64_t)a.T * a.d * 2 * full > kv::kStreamBytes) return launch(norm_kernel<R, U, true>, grid, dim3(kThreads), 0, st, a);
    return launch(norm_kernel<R, U, false>, grid, dim3(kThreads), 0, st, a);
}

}  // namespace

// Many rows: few threads a row, two units each, so that a compute unit has several rows under way between
// their sums.  Few rows: a thread a unit (64 rows of 4,096: 4.6 us, 6.0 in the other form; 4,096 of 7,168: 55 us in
// the other, 65 so).
constexpr int kFewRows = 1024;

// A launch stays below 2^32 threads: up to 64 a row of 64 units or fewer (2^24 rows), and below two a unit of longer
// ones (T * d up to 2^34 elements, 2^31 units).
hipError_t launch_block_norm(const ft_norm& a, hipStream_t st) {
    const int units = a.d >> 3;
    if (units <= 8) return go<8, 1>(a, st);
    if (units <= 16) return go<16, 1>(a, st);
    if (units <= 64) return go<64, 1>(a, st);
    if (a.T <= kFewRows) {
        if (units <= 256) return go<256, 1>(a, st);
        if (units <= 512) return go<512, 1>(a, st);
        if (units <= 1024) return go<1024, 1>(a, st);
    } else {
        if (units <= 256) return go<128, 2>(a, st);
        if (units <= 512) return go<256, 2>(a, st);
        if (units <= 1024) return go<512, 2>(a, st);
    }
    return go<1024, 4>(a, st);
}

}  // namespace ftmoe
