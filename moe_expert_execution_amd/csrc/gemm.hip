// Prefill expert FFN: grouped GEMMs over the active slots on MFMA.
//
// Rows are the planner's sorted GPU routes; each tile is 128 rows of one slot.
// Gate/up: C[rows x 2*128] = X[rows x d] * [WgT; WuT]^T for 128 neurons at a
// time, the gate and up halves landing in the same lanes, so the epilogue
// writes h = silu(g) * u (bf16) without a shuffle.  Down: Y[rows x 256 cols] =
// H[rows x f] * WdT^T, accumulated in fp32 and stored as bf16.
//
// Weights are panel-ordered in the slot record: one 16-byte load per lane at
// consecutive addresses delivers a 32-column x (two 16-byte chunk columns)
// operand tile, which is exactly an operand layout of
// v_mfma_f32_32x32x16_bf16 (lane l: row l % 32, chunk column l / 32).  So
// the weights go from memory straight into registers — no LDS staging, no
// shuffles — two K-steps ahead of their use; only the activation tile (shared
// by the four waves) is staged through LDS, loaded straight into a 4-deep
// ring of buffers, one barrier per K-step.  Block-FP8 and MXFP4 weights are
// converted to bf16 in registers right before their MFMA, so every format
// issues the bf16 MFMA.  The expert FFN with its gate/up and down projections
// read from one slot record follows "The Expert Cache That Follows the
// Router", section "One logical expert, two physical levels of memory".
#include <type_traits>

#include "resident_api.h"
#include "wfmt.h"

namespace ftmoe {

constexpr int kBM = 128, kBN = 256, kBK = 64, kStages = 4;
constexpr int kGemmThreads = 256;

int gemm_tile_m() { return kBM; }

struct GemmArgs {
    const uint16_t* x;
    const uint16_t* Hin;   // bf16 [rows x f] (down A)
    uint16_t* Hout;        // bf16 [rows x f] (gate/up C)
    uint16_t* Y;           // bf16 [rows x d]
    int k, d, f;
    uint32_t x_bytes, h_bytes;   // extents of x and H (their rows are reached by 32-bit offsets)
    const int32_t* meta;
    const int32_t* active_slot;
    const int32_t* seg;
    const int32_t* perm;
    const int32_t* tile_active;
    const int32_t* tile_row0;
    const int32_t* tile_first;
    const uint8_t* pool;
    int64_t S;          // slot stride of the pool (bytes)
    int64_t off_gate, off_up, off_down, off_sg, off_su, off_sd;
};

namespace {

// silu with a hardware reciprocal (1 ulp): z / (1 + e^-z)
__device__ __forceinline__ float silu(float z) { return z * __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }

// Per format: lane blocks (1 KiB panel runs) per K-step, and where the lane's
// 8 bf16 of MFMA step ks sit inside the 64-wide K-step (the A side must read
// the same K positions).
template <int FMT>
struct Frag {
    static constexpr int LBK = 64 / (2 * WF<FMT>::EPC);    // lane blocks per K-step: 4, 2, 1
    // a weight scale as stored: fp32 bits (FP8), an e8m0 byte (MXFP4)
    using SRaw = std::conditional_t<FMT == FT_FMT_MXFP4_B32, uint8_t, uint32_t>;
    __device__ static int a_koff(int ks, int g) {
        if constexpr (FMT == FT_FMT_BF16) return ks * 16 + g * 8;
        else if constexpr (FMT == FT_FMT_FP8_B128) return (ks >> 1) * 32 + g * 16 + (ks & 1) * 8;
        else return g * 32 + ks * 8;
    }
};

// B operand of MFMA step ks from the K-step's lane-block registers; `sraw` is
// the scale as loaded (FP8: fp32 bits, MXFP4: the e8m0 byte), decoded here so
// that its load is waited for only where it is used.
template <int FMT>
__device__ __forceinline__ bf16x8_t b_frag(const u32x4_t (&r)[Frag<FMT>::LBK], int ks, typename Frag<FMT>::SRaw sraw) {
    if constexpr (FMT == FT_FMT_BF16) {
        return __builtin_bit_cast(bf16x8_t, r[ks]);
    } else if constexpr (FMT == FT_FMT_FP8_B128) {
        const float scale = __uint_as_float(sraw);
        const u32x4_t w = r[ks >> 1];
        const uint32_t w0 = (ks & 1) ? w[2] : w[0];
        const uint32_t w1 = (ks & 1) ? w[3] : w[1];
        const f32x2_t p0 = __builtin_amdgcn_cvt_pk_f32_fp8((int)w0, false);
        const f32x2_t p1 = __builtin_amdgcn_cvt_pk_f32_fp8((int)w0, true);
        const f32x2_t p2 = __builtin_amdgcn_cvt_pk_f32_fp8((int)w1, false);
        const f32x2_t p3 = __builtin_amdgcn_cvt_pk_f32_fp8((int)w1, true);
        const bf16x2_t q0 = __builtin_convertvector(p0 * scale, bf16x2_t);
        const bf16x2_t q1 = __builtin_convertvector(p1 * scale, bf16x2_t);
        const bf16x2_t q2 = __builtin_convertvector(p2 * scale, bf16x2_t);
        const bf16x2_t q3 = __builtin_convertvector(p3 * scale, bf16x2_t);
        return bf16x8_t{q0[0], q0[1], q1[0], q1[1], q2[0], q2[1], q3[0], q3[1]};
    } else {
        const float scale = e8m0_to_f32(sraw);
        const uint32_t w = r[0][ks];
        const bf16x2_t q0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
        const bf16x2_t q1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
        const bf16x2_t q2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
        const bf16x2_t q3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
        return bf16x8_t{q0[0], q0[1], q1[0], q1[1], q2[0], q2[1], q3[0], q3[1]};
    }
}

// The same of an e4m3 K-step without its scale: the codes' values times the
// power of two `conv`, exact in bf16; all zero where `keep` is 0 (else ~0).
template <int LBK>
__device__ __forceinline__ bf16x8_t b_frag_codes(const u32x4_t (&r)[LBK], int ks, float conv, uint32_t keep) {
    const u32x4_t w = r[(ks >> 1) % LBK];
    const uint32_t w0 = ((ks & 1) ? w[2] : w[0]) & keep;
    const uint32_t w1 = ((ks & 1) ? w[3] : w[1]) & keep;
    const bf16x2_t q0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, conv, false);
    const bf16x2_t q1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, conv, true);
    const bf16x2_t q2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, conv, false);
    const bf16x2_t q3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, conv, true);
    return bf16x8_t{q0[0], q0[1], q1[0], q1[1], q2[0], q2[1], q3[0], q3[1]};
}

// Wait until at most N vector-memory operations of this wave are outstanding
// (they complete in issue order); the other counters are left alone.
template <int N>
__device__ __forceinline__ void vm_wait() {
    static_assert(N >= 0 && N < 64, "vmcnt holds 6 bits");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x70 | 0xF00);
}

// The adapters of a row tile: for each one named in it, acc += v B_a^T on the
// rows that name it (v as two bf16 planes; B_a's rows are the A operand, 16
// ranks at a time, masked past the adapter's own).  Other rows' products are
// selected away, so an adapter's infinities stay with its requests.
template <bool GU, int MI>
__device__ __forceinline__ void lora_rows(f32x16_t (&acc)[MI][2], const LoraGemmArgs& a, int row0, int rows_valid,
                                          const int (&pn)[2], int lane) {
    const int g = lane >> 5, n = GU ? a.f : a.d;
    constexpr int POOLS = GU ? 2 : 1;
#pragma unroll
    for (int pool = 0; pool < POOLS; ++pool) {
        const LoraView& lo = a.lora[pool];
        if (lo.count == 0) continue;
        const int R = lo.max_rank;
        int id[MI];
        uint32_t left[MI];
        int64_t vrow[MI];
#pragma unroll
        for (int mi = 0; mi < MI; ++mi) {
            const int r = mi * 32 + (lane & 31);
            const int v = r < rows_valid ? a.adapter[row0 + r] : -1;
            id[mi] = (uint32_t)v < (uint32_t)lo.count ? v : -1;
            left[mi] = (uint32_t)__ballot(id[mi] >= 0);
            vrow[mi] = (int64_t)(row0 + min(r, rows_valid - 1)) * R + g * 8;
        }
        for (;;) {
            int ad = -1;
#pragma unroll
            for (int mi = 0; mi < MI; ++mi)
                if (ad < 0 && left[mi]) ad = __builtin_amdgcn_readlane(id[mi], __builtin_ctz(left[mi]));
            if (ad < 0) break;
            uint32_t hit[MI];
#pragma unroll
            for (int mi = 0; mi < MI; ++mi) {
                hit[mi] = (uint32_t)__ballot(id[mi] == ad);
                left[mi] &= ~hit[mi];
            }
            const int rank = min(max(lo.rank[ad], 0), R);
            // steps (16 ranks, part of v), the next one's loads under way while one is multiplied
            constexpr int NB = GU ? 1 : 2;
            u32x4_t bw[2][NB], hv[2][MI], lv[2][MI];
            const int steps = (rank + 15) / 16 * a.vparts;
            auto load = [&](int q, int i) {
                const int k0 = i / a.vparts * 16, part = i % a.vparts;
#pragma unroll
                for (int j = 0; j < NB; ++j)
                    bw[q][j] = *reinterpret_cast<const u32x4_t*>(
                        lo.b + ((int64_t)ad * n + pn[GU ? pool : j] * 32 + (lane & 31)) * R + k0 + g * 8);
                const int64_t at = (int64_t)part * a.T * R + k0;
#pragma unroll
                for (int mi = 0; mi < MI; ++mi) {
                    hv[q][mi] = lv[q][mi] = u32x4_t{0u, 0u, 0u, 0u};
                    if (id[mi] == ad) {
                        hv[q][mi] = *reinterpret_cast<const u32x4_t*>(a.vhi[pool] + at + vrow[mi]);
                        lv[q][mi] = *reinterpret_cast<const u32x4_t*>(a.vlo[pool] + at + vrow[mi]);
                    }
                }
            };
            auto work = [&](int q, int i) {
                const int have = rank - i / a.vparts * 16 - g * 8;       // ranks of this lane's eight that exist
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    u32x4_t w = bw[q][j];
                    if (have < 8) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) w[e] &= have >= 2 * e + 2 ? 0xFFFFFFFFu : have == 2 * e + 1 ? 0xFFFFu : 0u;
                    }
                    const bf16x8_t bf = __builtin_bit_cast(bf16x8_t, w);
#pragma unroll
                    for (int mi = 0; mi < MI; ++mi) {
                        if (!hit[mi]) continue;
                        f32x16_t sum;
#pragma unroll
                        for (int v = 0; v < 16; ++v) sum[v] = 0.0f;
                        sum = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf, __builtin_bit_cast(bf16x8_t, hv[q][mi]), sum, 0, 0, 0);
                        sum = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf, __builtin_bit_cast(bf16x8_t, lv[q][mi]), sum, 0, 0, 0);
                        f32x16_t& c = acc[mi][GU ? pool : j];
#pragma unroll
                        for (int v = 0; v < 16; ++v) c[v] = id[mi] == ad ? c[v] + sum[v] : c[v];
                    }
                }
            };
            if (steps > 0) load(0, 0);
            for (int i = 0; i < steps; i += 2) {
                if (i + 1 < steps) load(1, i + 1);
                work(0, i);
                if (i + 1 < steps) {
                    if (i + 2 < steps) load(0, i + 2);
                    work(1, i + 1);
                }
            }
        }
    }
}

// Tile (kBM rows of one slot) x (kBN columns) per workgroup; 4 waves side by
// side along N, each computing 128 x 64 with 4 x 2 v_mfma_f32_32x32x16_bf16
// accumulators.  Gate/up: the kBN columns are 128 gate and the same 128 up
// neurons; wave w owns neurons [32 w, 32 w + 32) of both (B panel 0 gate,
// panel 1 up), so SwiGLU pairs accumulator 0 with 1 in-lane.  Down: wave w
// owns output columns [64 w, 64 w + 64), two panels.
// Workgroups are renumbered so that each XCD (dispatch round-robin over 8)
// receives a contiguous range of blocks, ordered by slot, then N-tile, then
// M-tile: all blocks of an expert run together in one XCD, where its A rows
// and weight panels are read from HBM about once and then hit that XCD's L2.
//
// The activation tile goes from memory straight into LDS (buffer_load_dwordx4
// with the lds modifier: each lane's 16 bytes land at the wave's base + 16 x
// lane) through a ring of kStages K-step buffers, kStages - 1 steps ahead of
// its use.  The buffer form, not global_load_lds: the compiler treats the
// latter as a FLAT access to both memory kinds and then turns every register
// wait into vmcnt(0), draining the weight prefetch.  A buffer is 128 rows x 128 bytes; 16-byte chunk c of row r sits
// at position c ^ f(r), f(r) = (r & 7) ^ ((r >> 3) & 1), so that the 16 (or 8)
// rows one ds_read_b128 serves per cycle fall in distinct banks.  Waits are
// explicit (vmcnt + s_barrier): a __syncthreads would also drain the weight
// loads that are in flight for later steps.
//
// With LoraGemmArgs (LORA): one resident matrix pair (GU) or matrix for T tokens in order, no
// plan: row tile i is tokens 128 i ..; before the epilogue each adapter named
// in the tile adds v B_a^T to its own rows' sums (lora_rows), and the down
// form adds `base` before the rounding.
//
// The full-tile down form with adapters spills 9 or 10 registers, the others none.
//
// WM: waves along M.  1 is the tile above; 2 is half of it each way (64 rows x
// 128 columns, wave (wm, wn) computing 32 x 64), four times the workgroups of
// a batch that would leave most of the card idle.
template <int FMT, bool GU, typename Args, int WM>
__global__ void __launch_bounds__(kGemmThreads, 2) gemm_kernel(Args a) {
    constexpr bool LORA = std::is_same_v<Args, LoraGemmArgs>;
    using FR = Frag<FMT>;
    constexpr int LBK = FR::LBK;
    constexpr int NB = 2 * LBK;                   // weight loads per wave per K-step
    constexpr int BM = kBM / WM, BN = kBN / WM;   // the tile
    constexpr int LA = BM / 32;                   // activation loads per wave per K-step
    constexpr int MMAX = BM / (32 * WM);          // row blocks of a wave
    __shared__ __attribute__((aligned(1024))) uint16_t As[kStages][BM * kBK];
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int w = wave % (4 / WM), wm = wave / (4 / WM);
    // d (a multiple of 128) may end in a half N-tile of the down product: its
    // waves 2 and 3 have no columns, re-read the last panel and store nothing
    const int NT = GU ? a.f / (BN / 2) : (a.d + BN - 1) / BN;
    int V;                                        // valid workgroups
    if constexpr (LORA) V = gridDim.x;
    else V = a.meta[1] * NT;
    const int b = blockIdx.x;
    if (b >= V) return;
    const int q8 = V >> 3, r8 = V & 7, x8 = b & 7;
    const int lb = x8 * q8 + (x8 < r8 ? x8 : r8) + (b >> 3);
    // within one slot's blocks [t0 NT, (t0 + mt) NT): N-tile major, M-tile minor,
    // so the M-tiles sharing a weight panel run side by side
    int nt, row0, rows_valid;
    const uint8_t* rec = nullptr;
    if constexpr (LORA) {
        const int mt = (a.T + BM - 1) / BM;
        nt = lb / mt;
        row0 = (lb - nt * mt) * BM;
        rows_valid = a.T - row0;
    } else {
        const int ai = a.tile_active[lb / NT];
        const int t0 = a.tile_first[ai], mt = a.tile_first[ai + 1] - t0;
        const int local = lb - t0 * NT;
        nt = local / mt;
        const int tile = t0 + (local - nt * mt);
        row0 = a.tile_row0[tile];
        rows_valid = a.seg[ai + 1] - row0;
        rec = a.pool + (int64_t)a.active_slot[ai] * a.S;
    }
    rows_valid = rows_valid > BM ? BM : rows_valid;
    const int K = GU ? a.d : a.f;
    const int64_t rowb = WF<FMT>::row_bytes(K);
    const int64_t panel_bytes = 32 * rowb;

    // this wave's two weight panels (+ lane offset); their scale locations
    const uint8_t* bp[2];
    const uint8_t* sp[2];
    int pn[2];
    if (GU) {
        pn[0] = pn[1] = nt * (BN / 64) + w;
    } else {
        const int last = a.d / 32 - 1;
        pn[0] = min(nt * (BN / 32) + 2 * w, last);
        pn[1] = min(nt * (BN / 32) + 2 * w + 1, last);
    }
    if constexpr (LORA) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            bp[i] = a.codes[GU ? i : 0] + pn[i] * panel_bytes + lane * 16;
            sp[i] = a.scales[GU ? i : 0];
        }
    } else if (GU) {
        bp[0] = rec + a.off_gate + pn[0] * panel_bytes + lane * 16;
        bp[1] = rec + a.off_up + pn[1] * panel_bytes + lane * 16;
        sp[0] = rec + a.off_sg;
        sp[1] = rec + a.off_su;
    } else {
        bp[0] = rec + a.off_down + pn[0] * panel_bytes + lane * 16;
        bp[1] = rec + a.off_down + pn[1] * panel_bytes + lane * 16;
        sp[0] = sp[1] = rec + a.off_sd;
    }
    // per-K-step weight scale of panel i, as stored: FP8 — the 128 x 128
    // block's fp32 (uniform over the panel); MXFP4 — the lane's e8m0 byte for
    // its chunk
    auto scale_of = [&](int i, int kt) -> typename FR::SRaw {
        if constexpr (FMT == FT_FMT_FP8_B128) {
            return reinterpret_cast<const uint32_t*>(sp[i])[(pn[i] >> 2) * (K >> 7) + (kt >> 1)];
        } else if constexpr (FMT == FT_FMT_MXFP4_B32) {
            return sp[i][(int64_t)pn[i] * K + kt * 64 + lane];
        } else {
            return 0;
        }
    };

    // A: wave v fills rows [8 LA v, 8 LA (v + 1)) of a buffer with LA loads, load
    // i covering the 1 KiB of 8 rows from r = 8 (LA v + i): lane l takes row
    // r + l / 8 at physical chunk l % 8, i.e. logical chunk
    // (l % 8) ^ (l / 8) ^ (r / 8 & 1).  Rows past the tile's end repeat its last
    // row: their outputs are never stored.  The loads are buffer loads (byte
    // offsets from x or H, the K-step in the scalar offset); the hardware
    // returns zeros for any offset past the buffer's extent.
    const __amdgpu_buffer_rsrc_t arsrc = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint16_t*>(GU ? a.x : a.Hin), 0, (int)(GU ? a.x_bytes : a.h_bytes), 0x00020000);
    uint32_t avo[4];                              // (LA are used)
#pragma unroll
    for (int i = 0; i < LA; ++i) {
        int r = 8 * (LA * wave + i) + (lane >> 3);
        r = r < rows_valid ? r : rows_valid - 1;
        const int p = row0 + r;
        const int c = (lane & 7) ^ (lane >> 3) ^ ((LA * wave + i) & 1);
        uint32_t row;
        if constexpr (GU && !LORA) row = (uint32_t)(a.perm[p] / a.k) * (uint32_t)a.d;
        else row = (uint32_t)p * (uint32_t)K;
        avo[i] = (row + (uint32_t)c * 8u) * 2u;
    }
    const int KT = K / kBK;        // even: K is a multiple of 128
    auto load_a = [&](int kt, int stage) {
        const int ks = kt < KT ? kt : KT - 1;       // past the end: reload the last step (never read)
#pragma unroll
        for (int i = 0; i < LA; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                arsrc, (__attribute__((address_space(3))) void*)(&As[stage][(LA * wave + i) * 512]), 16, avo[i],
                ks * kBK * 2, 0, 0);
    };

    // The wave's MI = ceil(its valid rows / 32) row blocks are all that is
    // computed: a short last tile of an expert (its few leftover rows) costs
    // MI / 4 of a full tile's MFMAs.
    auto body = [&](auto mi_count) {
        constexpr int MI = decltype(mi_count)::value;
        f32x16_t acc[MI][2];
#pragma unroll
        for (int mi = 0; mi < MI; ++mi)
#pragma unroll
            for (int ni = 0; ni < 2; ++ni)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[mi][ni][v] = 0.0f;

        // Two sets of weight registers, for even and odd K-steps: step kt reads
        // set kt % 2 and then refills it with K-step kt + 2, so every weight load
        // has two K-steps to arrive and lands in the registers its consumer reads.
        u32x4_t br[2][2][LBK];
        typename FR::SRaw bs[2][2];
#pragma unroll
        for (int s2 = 0; s2 < 2; ++s2)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int j = 0; j < LBK; ++j)
                    br[s2][i][j] = *reinterpret_cast<const u32x4_t*>(bp[i] + (int64_t)(s2 * LBK + j) * 1024);
                bs[s2][i] = scale_of(i, s2);
            }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int s = 0; s < kStages - 1; ++s) load_a(s, s);
        __builtin_amdgcn_sched_barrier(0);

        // A operand of MFMA step ks for the MI row blocks, from buffer `stage`
        const int m = lane & 31;
        const int fm = (m & 7) ^ ((m >> 3) & 1);
        const int rm = WM == 1 ? 0 : wm * 32 * MMAX;          // the wave's first row
        auto read_a = [&](bf16x8_t (&af)[MI], int stage, int ks) {
            const int c = FR::a_koff(ks, g) >> 3;
#pragma unroll
            for (int mi = 0; mi < MI; ++mi)
                af[mi] = *reinterpret_cast<const bf16x8_t*>(&As[stage][(rm + mi * 32 + m) * kBK + ((c ^ fm) << 3)]);
        };
        bf16x8_t af[2][MI];
        // A(0) has landed once only A(1) and A(2) may be outstanding
        vm_wait<2 * LA>();
        __builtin_amdgcn_s_barrier();
        read_a(af[0], 0, 0);

        // One K-step.  Vector-memory operations of a wave complete in issue order,
        // so "A of step kt + 1 has landed" is a count of the loads issued after
        // it.  A step issues RP weight refills, then (before its last MFMA
        // group) A(kt + 3), then the last NB - RP refills (scale loads come after
        // them and only make the count conservative); the prologue issued B(0),
        // B(1), A(0), A(1), A(2).  After every wave has seen its own loads land,
        // one barrier publishes buffer kt + 1; it also tells that every wave has
        // finished step kt - 1, the last reader of the buffer A(kt + 3) refills.
        // Putting it before the last MFMA group lets the next step's first LDS
        // reads overlap this step's last MFMAs.  Instruction order is pinned with
        // scheduling barriers: the compiler would otherwise sink every prefetch
        // below the last MFMA.
        constexpr int RP = 2 * (LBK - 1);             // refills issued before A(kt + 3)
        // Block-FP8 beside adapters: the codes are multiplied as they are (exact in
        // bf16) and the accumulators are kept in units of the current block's
        // scale, rescaled when the next 128 K begin; the grouped form rounds code
        // times scale to bf16 instead.  A unit stays within 2^-(kFall + 1) of the
        // largest scale so far, so that rescaling cannot overflow (sums of tokens up
        // to 2^80 fit): a smaller scale keeps a factor 2^-m in the codes, exact in
        // bf16 down to scales 2^-126 of the largest.  Still smaller, subnormal and
        // zero ones leave the unit, and their codes count as zero (the masks take 1
        // to 2 us of a call: 512 tokens through [4,096 x 4,096] 51 us, 4,096 tokens 154).
        constexpr bool UNITS = LORA && FMT == FT_FMT_FP8_B128;
        constexpr int kFall = 16;
        float unit[2] = {1.0f, 1.0f}, conv[2] = {1.0f, 1.0f};
        uint32_t top[2] = {0u, 0u}, keep[2] = {0u, 0u};
        auto begin_block = [&](const typename FR::SRaw (&bss)[2]) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t sb = (uint32_t)__builtin_amdgcn_readfirstlane((int)bss[i]), mag = sb & 0x7FFFFFFFu;
                const int m = max((int)(top[i] >> 23) - (int)(mag >> 23) - kFall, 0);
                if (mag < 0x00800000u || m > 110) {
                    keep[i] = 0u;
                    continue;
                }
                keep[i] = ~0u;
                top[i] = max(top[i], mag);
                conv[i] = __uint_as_float((uint32_t)(127 - m) << 23);
                const float u = __uint_as_float(sb) * __uint_as_float((uint32_t)(127 + m) << 23);
                const float r = unit[i] / u;
                unit[i] = u;
#pragma unroll
                for (int mi = 0; mi < MI; ++mi)
#pragma unroll
                    for (int v = 0; v < 16; ++v) acc[mi][i][v] *= r;
            }
        };
        auto kstep = [&](int kt, int stage, u32x4_t (&brs)[2][LBK], typename FR::SRaw (&bss)[2]) {
            if constexpr (UNITS) {
                if ((kt & 1) == 0) begin_block(bss);
            }
            const int kw = kt + 2 < KT ? kt + 2 : KT - 1;     // weights refilled for two steps ahead
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                if (ks < 3) {
                    read_a(af[(ks + 1) & 1], stage, ks + 1);
                } else {
                    if (kt >= 2) vm_wait<2 * NB + LA>();
                    else if (kt == 1) vm_wait<NB + LA + RP>();
                    else vm_wait<LA + RP>();
                    __builtin_amdgcn_s_barrier();
                    __builtin_amdgcn_sched_barrier(0);
                    load_a(kt + 3, (stage + 3) % kStages);
                    __builtin_amdgcn_sched_barrier(0);
                    read_a(af[0], (stage + 1) % kStages, 0);
                }
                bf16x8_t b0, b1;
                if constexpr (UNITS) {
                    b0 = b_frag_codes(brs[0], ks, conv[0], keep[0]);
                    b1 = b_frag_codes(brs[1], ks, conv[1], keep[1]);
                } else {
                    b0 = b_frag<FMT>(brs[0], ks, bss[0]);
                    b1 = b_frag<FMT>(brs[1], ks, bss[1]);
                }
#pragma unroll
                for (int mi = 0; mi < MI; ++mi) {
                    acc[mi][0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b0, af[ks & 1][mi], acc[mi][0], 0, 0, 0);
                    acc[mi][1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b1, af[ks & 1][mi], acc[mi][1], 0, 0, 0);
                }
                constexpr int kDone = 4 / LBK;                // MFMA steps per lane block
                if ((ks % kDone) == kDone - 1) {
                    const int j = ks / kDone;
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        brs[i][j] = *reinterpret_cast<const u32x4_t*>(bp[i] + (int64_t)(kw * LBK + j) * 1024);
                }
                // order inside the group: the next group's LDS reads interleaved
                // with the first MFMAs, then the rest, then the refill loads
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // MFMA
                    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // LDS read
                }
                __builtin_amdgcn_sched_group_barrier(0x008, MI, 0);
                __builtin_amdgcn_sched_group_barrier(0x020, 2, 0);       // global loads
                __builtin_amdgcn_sched_barrier(0);
            }
            // the refilled set's scales, loaded straight into the registers that
            // step kw reads (a copy would have to wait for the load)
#pragma unroll
            for (int i = 0; i < 2; ++i) bss[i] = scale_of(i, kw);
        };
        static_assert(kStages == 4, "the step unrolling below pairs stages with weight register sets");
        for (int kt = 0; kt < KT; kt += 4) {
            kstep(kt, 0, br[0], bs[0]);
            kstep(kt + 1, 1, br[1], bs[1]);
            if (kt + 2 < KT) {
                kstep(kt + 2, 2, br[0], bs[0]);
                kstep(kt + 3, 3, br[1], bs[1]);
            }
        }
        // the ring's last (unused) loads must land before the buffers are reused
        vm_wait<0>();
        __builtin_amdgcn_s_barrier();

        if constexpr (UNITS) {
#pragma unroll
            for (int mi = 0; mi < MI; ++mi)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int v = 0; v < 16; ++v) acc[mi][i][v] *= unit[i];
        }
        if constexpr (LORA) lora_rows<GU, MI>(acc, a, row0 + rm, max(rows_valid - rm, 0), pn, lane);

        // Epilogue.  The MFMAs compute C^T (weights as the A operand), so lane l
        // holds row mi*32 + l%32 and, per group q, the four consecutive columns
        // 8q + 4(l/32) .. +3 of each 32-column panel.  The tile goes through LDS
        // (free once the ring has drained) so that every global store
        // instruction writes whole contiguous row segments.
        if (GU) {
            // h = silu(g) * u, the whole 128 x 128 bf16 tile, rows padded by 16 bytes.
            // h is rounded to bf16: it is the down product's operand, and a second plane
            // for its lower bits (which calls of few tokens keep, bound by the weights)
            // would double that product's matrix instructions, 133 us of the 340 that 4,096
            // tokens of an MXFP4 expert take.  y's relative error is 0.0023 with it and
            // 0.0016 without, which is y's own rounding.
            constexpr int LDH = BN / 2 + 8;
            uint16_t* Hs = &As[0][0];
            static_assert(BM * LDH <= kStages * BM * kBK, "h tile must fit the A buffers");
#pragma unroll
            for (int mi = 0; mi < MI; ++mi)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float h[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) h[j] = silu(acc[mi][0][4 * q + j]) * acc[mi][1][4 * q + j];
                    uint2 o;
                    o.x = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{h[0], h[1]}, bf16x2_t));
                    o.y = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{h[2], h[3]}, bf16x2_t));
                    *reinterpret_cast<uint2*>(&Hs[(rm + mi * 32 + m) * LDH + 32 * w + 8 * q + 4 * g]) = o;
                }
            __syncthreads();
            // LR lanes per row (16 for 256 bytes), whole rows per pass
            constexpr int LR = BN / 16, RPP = kGemmThreads / LR;
            constexpr int ROWS = WM == 1 ? MI * 32 : BM;
#pragma unroll
            for (int it = 0; it < ROWS / RPP; ++it) {
                const int r = it * RPP + tid / LR, c = (tid % LR) * 8;
                if (r < rows_valid)
                    *reinterpret_cast<u32x4_t*>(a.Hout + (int64_t)(row0 + r) * a.f + nt * (BN / 2) + c) =
                        *reinterpret_cast<const u32x4_t*>(&Hs[r * LDH + c]);
            }
        } else {
            // per wave: 32 rows x 64 bf16 columns at a time, rows padded by 16 bytes
            constexpr int LDY = 64 + 8;
            uint16_t* Ys = &As[0][0] + wave * 32 * LDY;
            const bool col_ok = nt * BN + 64 * w < a.d;
            static_assert(4 * 32 * LDY <= kStages * BM * kBK, "y tiles must fit the A buffers");
#pragma unroll
            for (int mi = 0; mi < MI; ++mi) {
#pragma unroll
                for (int ni = 0; ni < 2; ++ni)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint2 o;
                        if constexpr (LORA) {
                            if (a.base) {
                                const int r = min(rm + mi * 32 + m, rows_valid - 1);
                                const uint2 bv = *reinterpret_cast<const uint2*>(
                                    a.base + (int64_t)(row0 + r) * a.d + pn[ni] * 32 + 8 * q + 4 * g);
                                acc[mi][ni][4 * q] += bf16lo(bv.x);
                                acc[mi][ni][4 * q + 1] += bf16hi(bv.x);
                                acc[mi][ni][4 * q + 2] += bf16lo(bv.y);
                                acc[mi][ni][4 * q + 3] += bf16hi(bv.y);
                            }
                        }
                        o.x = __builtin_bit_cast(uint32_t, __builtin_convertvector(
                                  f32x2_t{acc[mi][ni][4 * q], acc[mi][ni][4 * q + 1]}, bf16x2_t));
                        o.y = __builtin_bit_cast(uint32_t, __builtin_convertvector(
                                  f32x2_t{acc[mi][ni][4 * q + 2], acc[mi][ni][4 * q + 3]}, bf16x2_t));
                        *reinterpret_cast<uint2*>(&Ys[m * LDY + 32 * ni + 8 * q + 4 * g]) = o;
                    }
                // the wave reads back what it wrote (LDS operations of a wave stay in order)
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                __builtin_amdgcn_wave_barrier();
                __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
                // 8 lanes per 128-byte row, 8 rows per pass
#pragma unroll
                for (int it = 0; it < 4; ++it) {
                    const int rr = it * 8 + (lane >> 3), c = (lane & 7) * 8;
                    const int r = rm + mi * 32 + rr;
                    if (r < rows_valid && col_ok)
                        *reinterpret_cast<u32x4_t*>(a.Y + (int64_t)(row0 + r) * a.d + nt * BN + 64 * w + c) =
                            *reinterpret_cast<const u32x4_t*>(&Ys[rr * LDY + c]);
                }
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                __builtin_amdgcn_wave_barrier();
                __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
            }
        }
    };
    if constexpr (WM == 1) {
        const int nmi = (rows_valid + 31) >> 5;
        if (nmi >= 4) body(std::integral_constant<int, 4>{});
        else if (nmi == 3) body(std::integral_constant<int, 3>{});
        else if (nmi == 2) body(std::integral_constant<int, 2>{});
        else body(std::integral_constant<int, 1>{});
    } else {
        body(std::integral_constant<int, MMAX>{});     // (a wave past the rows computes on the last one)
    }
}

template <int FMT>
hipError_t launch_fmt(const GemmArgs& a, int64_t max_tiles, Timing* tm, hipStream_t st) {
    const int64_t g1 = max_tiles * (a.f / (kBN / 2)), g2 = max_tiles * ((a.d + kBN - 1) / kBN);
    TimedLaunch t1 = timing_launch(tm, FT_K_GEMM_GU);
    hipExtLaunchKernelGGL((gemm_kernel<FMT, true, GemmArgs, 1>), dim3((unsigned)g1), dim3(kGemmThreads), 0, st, t1.start, t1.stop,
                          0, a);
    TimedLaunch t2 = timing_launch(tm, FT_K_GEMM_DOWN);
    hipExtLaunchKernelGGL((gemm_kernel<FMT, false, GemmArgs, 1>), dim3((unsigned)g2), dim3(kGemmThreads), 0, st, t2.start,
                          t2.stop, 0, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm(ft_cache* c, const uint16_t* x, int T, hipStream_t st) {
    GemmArgs a;
    a.x = x;
    a.Hin = c->H;
    a.Hout = c->H;
    a.Y = c->Y;
    a.k = c->sh.top_k;
    a.d = c->sh.d_model;
    a.f = c->sh.d_ff;
    // creation keeps both below 4 GiB
    a.x_bytes = (uint32_t)((int64_t)T * a.d * 2);
    a.h_bytes = (uint32_t)((int64_t)c->cap * a.f * 2);
    a.meta = c->plan.meta;
    a.active_slot = c->plan.active_slot;
    a.seg = c->plan.seg;
    a.perm = c->plan.perm;
    a.tile_active = c->plan.tile_active;
    a.tile_row0 = c->plan.tile_row0;
    a.tile_first = c->plan.tile_first;
    a.pool = c->pool;
    a.S = c->rl.P;   // slot stride of the pool
    a.off_gate = c->rl.off_gate;
    a.off_up = c->rl.off_up;
    a.off_down = c->rl.off_down;
    a.off_sg = c->rl.off_sg;
    a.off_su = c->rl.off_su;
    a.off_sd = c->rl.off_sd;
    // tiles possible for T tokens: rows / BM + active slots
    const int64_t R = (int64_t)T * a.k;
    int64_t act = R < c->N ? R : c->N;
    const int64_t max_tiles = (R + kBM - 1) / kBM + act;
    if (max_tiles > c->plan.max_tiles) return hipErrorInvalidValue;
    switch (c->sh.fmt) {
        case FT_FMT_BF16: return launch_fmt<FT_FMT_BF16>(a, max_tiles, c->timing, st);
        case FT_FMT_FP8_B128: return launch_fmt<FT_FMT_FP8_B128>(a, max_tiles, c->timing, st);
        case FT_FMT_MXFP4_B32: return launch_fmt<FT_FMT_MXFP4_B32>(a, max_tiles, c->timing, st);
    }
    return hipErrorInvalidValue;
}

// The half tile while the full one would give the 256 CUs less than a workgroup
// each: 2,048 tokens through [2,048 x 2,048] bf16 take 38 us and 41 with full tiles
// (128 of them), 4,096 tokens 70 and 53 (256 of them); an expert of 2,048 x 768 on
// 777 tokens 42 and 66.  A half tile is bound by its operands from L2, 0.8 MB at
// K = 2,048 in 18 us; full tiles by MFMA: 8,192 tokens through [2,048 x 2,048] in 78 us
// are 890 TFLOP/s, the MXFP4 expert of 7,168 x 2,048 on 4,096 tokens 1,020.
template <int FMT, bool GU>
hipError_t launch_lora_fmt(const LoraGemmArgs& a, hipStream_t st) {
    const int cols = GU ? 2 * a.f : a.d;
    const int64_t full = (int64_t)((a.T + kBM - 1) / kBM) * ((cols + kBN - 1) / kBN);
    const bool half = full < 256;
    const int bm = half ? kBM / 2 : kBM, bn = half ? kBN / 2 : kBN;
    const dim3 grid((unsigned)(((a.T + bm - 1) / bm) * ((cols + bn - 1) / bn)));
    return launch(half ? gemm_kernel<FMT, GU, LoraGemmArgs, 2> : gemm_kernel<FMT, GU, LoraGemmArgs, 1>, grid, dim3(kGemmThreads),
                  0, st, a);
}

template <int FMT>
hipError_t launch_lora_fmt(const LoraGemmArgs& a, bool gu, hipStream_t st) {
    return gu ? launch_lora_fmt<FMT, true>(a, st) : launch_lora_fmt<FMT, false>(a, st);
}

hipError_t launch_lora_gemm(int fmt, bool gu, const LoraGemmArgs& a, hipStream_t st) {
    switch (fmt) {
        case FT_FMT_BF16: return launch_lora_fmt<FT_FMT_BF16>(a, gu, st);
        case FT_FMT_FP8_B128: return launch_lora_fmt<FT_FMT_FP8_B128>(a, gu, st);
        case FT_FMT_MXFP4_B32: return launch_lora_fmt<FT_FMT_MXFP4_B32>(a, gu, st);
    }
    return hipErrorInvalidValue;
}

}  // namespace ftmoe
