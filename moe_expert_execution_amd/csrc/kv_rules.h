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
// themselves.  An item that is cut is joined by the last of its teams to arrive, so a
// cut that falls within `slack` steps of an item's end moves there.
constexpr int kWaves = 4;                  // of a team; they share a segment's steps
constexpr int kMaxTeams = 1024;
constexpr int kSlack = 4;
constexpr int kJoin = 8;                   // parts that one join takes

struct Division {
    int64_t total;                         // steps, > 0
    int64_t per;                           // steps of a team, times 2^16
    float rate;                            // teams per step
    int teams, slack;
};

// `items` that have steps, `total` steps, at most `grid` teams: one for as many steps as it has
// waves, or for an item where items are shorter.
FT_HD inline Division divide(int64_t items, int64_t total, int grid) {
    int64_t t = (total + kWaves - 1) / kWaves;
    if (t < items) t = items;
    if (t > grid) t = grid;
    // (divisions in doubles: exact enough, and a fraction of a 64-bit integer division's latency)
    const double per = (double)(total << 16) / (double)t;
    const double half = (per * (1.0 / 65536) - 1) / 2;           // less than half a range: cuts keep their order
    return Division{total, (int64_t)per, (float)t / (float)total, (int)t, half < kSlack ? (int)half : kSlack};
}
// The cut before team i, and the last team whose cut is at or before a step, before cuts move.
FT_HD inline int64_t cut(const Division& d, int i) { return i == d.teams ? d.total : d.per * i >> 16; }
FT_HD inline int team_at(const Division& d, int64_t step) {
    int i = (int)((float)step * d.rate);               // within one of it
    i = i < d.teams - 1 ? i : d.teams - 1;
    while (cut(d, i) > step) --i;
    while (i < d.teams - 1 && cut(d, i + 1) <= step) ++i;
    return i;
}

// The teams of the item of steps [begin, begin + n): cuts in its first and last steps have moved to its
// ends (the nearer one, the first of two as near).
struct Teams {
    int first, last;
};
FT_HD inline Teams teams_of(const Division& d, int64_t begin, int n) {
    const int after = d.slack < n / 2 ? d.slack : n / 2, before = d.slack < (n - 1) / 2 ? d.slack : (n - 1) / 2;
    return Teams{team_at(d, begin + after), team_at(d, begin + n - 1 - before)};
}
// Steps [from, to) of the item that team i, one of them, works on, counted from the item's begin.
struct Segment {
    int from, to;
};
FT_HD inline Segment segment(const Division& d, const Teams& t, int64_t begin, int n, int i) {
    return Segment{i == t.first ? 0 : (int)(cut(d, i) - begin), i == t.last ? n : (int)(cut(d, i + 1) - begin)};
}

// Parts of an item are joined in runs of kJoin teams, counted from its first, and the runs' sums then:
// runs of more for items of more than kJoin^2 parts.
FT_HD inline int join_run(const Teams& t) {
    int run = kJoin;
    while (run * kJoin < t.last - t.first + 1) run *= 2;
    return run;
}

// Query heads of an item and items of a KV head, for a group of g query heads.
FT_HD inline int item_heads(int g) { return g < kCols ? g : kCols; }
FT_HD inline int head_blocks(int g) { return (g + kCols - 1) / kCols; }

// Floats of one partial result: sums, then the heads' maxima and totals, of the part and of the run
// whose sum takes its place.
FT_HD inline int64_t part_floats(int g, int D) { return (int64_t)item_heads(g) * D + 4 * kCols; }

// Workgroups of a launch whose items and steps are at most these.
inline int grid_of(int64_t items, int64_t steps, int most) { return divide(items, steps, most).teams; }

// Teams of a compute unit, as registers allow: all of a call's teams are resident, since one that starts late
// ends late (64 requests of up to 8,192 tokens, e4m3, 128 dimensions: 73 us with three, 85 with two; bf16, 192
// registers: 122 with the two that fit, 130 with three).
constexpr int teams_per_cu(int D, int esize) { return D == 256 ? 2 : D == 128 ? (esize == 2 ? 2 : 3) : esize == 2 ? 3 : 4; }
constexpr int kComputeUnits = 256;

// Items of at most this many steps are not cut, so they need no division: a workgroup each.
constexpr int kDirectSteps = 4 * kWaves;

}  // namespace kv
}  // namespace ftmoe
