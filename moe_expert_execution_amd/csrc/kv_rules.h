// The paged key-value cache's layout and how an attention call is divided over
// workgroups: arithmetic shared by the host, the kernels and the CPU tests, free
// of HIP.
#pragma once
#include <stdint.h>

#ifdef __HIP__
#define FT_HD __host__ __device__
#else
#define FT_HD
#endif

namespace ftmoe {
namespace kv {

constexpr int kMaxRequests = 4096;
constexpr int kMaxTokens = 65535;
constexpr int kMaxHeads = 1024;
constexpr int kMaxWidth = 131072;          // table entries of a request
constexpr int kBlock = 16;                 // tokens of a layout block
constexpr int kStep = 32;                  // tokens of one attention step: K of a 16x16x32 matrix-core product
constexpr int kCols = 16;                  // query heads of one operand

// Elements of a 16-byte key unit; dimensions and tokens of a value unit.
FT_HD constexpr int key_unit(int esize) { return 16 / esize; }
FT_HD constexpr int value_dims(int D) { return D == 64 ? 4 : 8; }
FT_HD constexpr int value_tokens(int D, int esize) { return 16 / (esize * value_dims(D)); }

// ---- the division of attention ----------------------------------------------------
// A work item is one KV head of one request for up to 16 query heads; its visible
// tokens are steps of 32.  The steps of all items in order (request, then head) are cut
// into `teams` ranges of equal length, one workgroup each, so ragged lengths balance by
// themselves.  An item inside one range is finished there; one that is cut is joined by
// the last of its teams to arrive.
FT_HD inline int64_t team_begin(int64_t total, int teams, int i) { return total * i / teams; }
FT_HD inline int team_of(int64_t total, int teams, int64_t step) {
    return (int)(((step + 1) * teams - 1) / total);
}

constexpr int kWaves = 4;                  // of a team
constexpr int kMaxTeams = 512;
// Steps that are worth a team: one for each of its waves.
constexpr int kTeamSteps = kWaves;

// Teams of a call with `total` > 0 steps, at most `grid`.
FT_HD inline int teams_of(int64_t total, int grid) {
    const int64_t most = (total + kTeamSteps - 1) / kTeamSteps;
    return most < grid ? (int)most : grid;
}

// Query heads of an item and items of a KV head, for a group of g query heads.
FT_HD inline int item_heads(int g) { return g < kCols ? g : kCols; }
FT_HD inline int head_blocks(int g) { return (g + kCols - 1) / kCols; }

// Floats of one partial result: sums, then the heads' maxima and totals.
FT_HD inline int64_t part_floats(int g, int D) { return (int64_t)item_heads(g) * D + 2 * kCols; }

inline int grid_of(int64_t bound_steps) {
    if (bound_steps < 1) return 1;
    return teams_of(bound_steps, kMaxTeams);
}

}  // namespace kv
}  // namespace ftmoe
