// How a call of the adapter operators is divided over launches and workgroups:
// sizes and rules of the host, free of HIP.
#pragma once
#include <stdint.h>

namespace ftmoe {
namespace rs {

constexpr int kWaves = 8;                 // waves of a streaming workgroup, splitting K
constexpr int kUnit = 128;                // elements along K per unit (one fp8 scale block)
constexpr int kCols = 16;                 // tokens of one operand
constexpr int kTile = 2 * kCols;          // tokens of one tile: at most two operands
constexpr int kMaxFusedSteps = 16;        // 16-rank steps per pool that a product's launch takes along
constexpr int kMaxParts = 4;              // parts of K of a shrink launch

// How a shrink launch goes over its tokens and slots.
struct Shrink {
    int span, per;         // tokens, and slots, of a workgroup
    int parts;             // of K
};

// Short calls, whose tokens may all name adapters of their own: spans of 64
// tokens, as the more tokens share an adapter's A the better.  A prompt's spans
// mostly have one adapter: 32 tokens where that still leaves the workgroups one
// round of the 256 compute units (777 tokens of K = 2,048: 6.4 us, 9.1 with 64),
// 64 where it does not (8,192 tokens, two slots: 15.4 us, 19.4 with 32), and where
// x exceeds the XCDs' 32 MiB of L2, so that another slot's workgroups read it from
// beyond them, two slots to a workgroup (4,096 tokens of K = 7,168: 29 us, 40 with
// one; 8,192 of K = 2,048: 17.3).
inline Shrink shrink_of(int T, int K, int slots, int adapters, bool prompt) {
    Shrink s;
    const int64_t narrow = (T + kTile - 1) / kTile;
    s.per = prompt && slots > 1 && narrow * slots >= 256 && (int64_t)T * K * 2 > (32ll << 20) ? 2 : 1;
    s.span = prompt && (s.per == 2 || narrow * slots <= 256) ? kTile : 2 * kTile;
    const int64_t spans = (T + s.span - 1) / s.span;
    const int most = prompt ? K / kUnit / kWaves : (K / kUnit + kWaves - 1) / kWaves;
    int64_t p = 256 / (spans * ((slots + s.per - 1) / s.per) * (prompt ? 1 : adapters));
    p = p > most ? most : p;
    s.parts = p < 1 ? 1 : p > kMaxParts ? kMaxParts : (int)p;
    return s;
}

// How a call's product and its adapters are divided.
struct Split {
    int splits;        // workgroups of a (panel, tile) that stream it
    bool adapted;      // it has adapters:
    bool fused;        // lsplits workgroups per matrix compute v and take them, or
    int lsplits;
    Shrink shrink;     // a launch before it computes v
};

// `nm` matrices [n x K]; `adapters`, `rank`: the most a tile of the call can
// name, and the largest max_rank (0: no adapters).
inline Split split_of(int nm, int n, int K, int T, int adapters, int rank) {
    const int64_t panels = n / 32, tiles = (T + kTile - 1) / kTile;
    const int units = K / kUnit, most = (units + kWaves - 1) / kWaves;
    Split s;
    // enough workgroups for the card's 256 compute units, no more than leaves every wave a unit
    int64_t w = 256 / (panels * tiles);
    w = w > most ? most : w;
    s.splits = w < 1 ? 1 : (int)w;
    s.lsplits = 0;
    s.adapted = s.fused = false;
    s.shrink.parts = 1;
    if (adapters <= 0 || rank <= 0) return s;
    s.adapted = true;
    if (adapters > T) adapters = T;
    if (adapters > kTile) adapters = kTile;
    // Without a launch for v every row panel reads the adapters' A once more (from
    // L2): taken while that is at most 24 MB in all, some 2 us of it, and while the
    // adapters' workgroups fit the card beside the stream's.  [2,048 x 2,048] bf16,
    // rank 16: one adapter 8.3 us and 11.4 with a launch, 8 of them 13.3 and 13.6; the
    // expert of 2,048 x 768 on 7 tokens of 8 adapters 19.0 and 27.6.
    const int64_t steps = (int64_t)adapters * (rank / 16), per = 256 / (panels * tiles);
    s.fused = T <= kTile && steps <= kMaxFusedSteps && panels * steps * 32 * K <= (24ll << 20) && per >= 1 + nm;
    if (s.fused) {
        if (s.splits > per - nm) s.splits = (int)(per - nm);
        const int64_t pairs = steps * units, need = (pairs + kWaves - 1) / kWaves;
        int64_t l = (per - s.splits) / nm;
        l = l > need ? need : l;
        s.lsplits = l < 1 ? 1 : l > 4 ? 4 : (int)l;
    } else {
        s.shrink = shrink_of(T, K, nm * (rank / 16), adapters, false);
    }
    return s;
}

// Prompts go through the GEMM tiles (gemm.hip).  A GEMM workgroup's time is that
// of its K at the rate of one compute unit, however few there are (18 us for
// K = 2,048 in bf16, 37 for 4,096 in fp8); streaming takes rounds of 256
// workgroups of 8 to 16 us.  The most rounds that stream were set where the two
// met: a projection of 384 tokens takes 26 us either way at [768 x 2,048] (2
// rounds), 45 and 44 at [2,048 x 4,096] fp8 (3 rounds); an expert 47 and 46 at 256
// tokens (d = 2,048, f = 768: 3 rounds), 90 and 76 at 192 (fp8, 4,096 and 2,048: 5).
// Up to 64 tokens always stream, and so do calls whose rows the tiles' 32-bit
// offsets do not reach.
inline int64_t stream_rounds(int n, int T) { return ((int64_t)(n / 32) * ((T + kTile - 1) / kTile) + 255) / 256; }
inline bool tiles_fit(int T, int64_t rounds, int64_t most, int K) {
    return T > 64 && rounds > most && (int64_t)T * K * 2 < (1ll << 32);
}
inline bool project_tiles(int n, int K, int T) { return tiles_fit(T, stream_rounds(n, T), 2, K); }
inline bool expert_tiles(int d, int f, int T) {
    return tiles_fit(T, stream_rounds(f, T) + stream_rounds(d, T), 3, d > f ? d : f);
}

}  // namespace rs
}  // namespace ftmoe
