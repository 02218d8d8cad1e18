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
// tokens are steps of 32.  All items in order (request, then head), each as long as its
// steps and kItemCost, are cut into `teams` ranges of equal length, one workgroup each, so
// ragged lengths balance by themselves.  An item that is cut is joined by the last of its teams to
// arrive, so a cut within `slack` steps of an item's end moves there.
constexpr int kMaxTeams = 512;
// Waves of a team, which share a segment's steps, and the most teams of a call: eight waves to each of 256 compute units,
// as registers allow, so all teams are resident (one that starts late ends late).  Heads of 256 have twice the partial
// sums, and one team of eight halves those (13 requests of up to 65,536, e4m3: 56 us, 60 with two of four; bf16, 32 of up to
// 8,192: 34, 39).
FT_HD constexpr int team_waves(int D) { return D == 256 ? 8 : 4; }
FT_HD constexpr int most_teams(int D) { return 8 * 256 / team_waves(D); }
// Steps for which a call takes one more team: more teams read sooner, fewer have fewer parts to join (one request of 8,192
// tokens, 32/4 heads of 128: 14.4 us, 14.8 with 4, 15.2 with 8; heads of 256, whose steps are longer, 16/2 of them: 17.5,
// 19.7 with 6).
FT_HD constexpr int team_steps(int D) { return D == 256 ? 3 : 6; }
// Above one team to a compute unit a call takes two, and no number between (those with two would end last): two where
// its items are many, for their parts are few then, and a token's row of a head, `row` bytes, is so small that four
// waves have too little under way.  Rows of 256 bytes: one team is as fast throughout, with half the parts (131,072
// tokens of one request, 4 KV heads: 50.0 us, 53.0 with two; 64 ragged ones of up to 8,192, 8 KV heads: 108, 112).  128
// bytes: 64 items 21.1 / 19.8 us (e4m3 of 128 / bf16 of 64) with one, 21.9 / 22.0 with two; 256 items 40 / 31.6 and 36 / 30.7;
// 512 items 65.7 / 47.8 and 55.9 / 45.9.  64 bytes: 32 items 19.8 and 17.7, 512 items 28.7 and 23.1.
constexpr uint32_t kUnits = 256;
FT_HD constexpr uint32_t many_items(int row) { return row >= 256 ? UINT32_MAX : row >= 128 ? 192 : 16; }
// Steps that a cut moves, at most (32 ragged requests of up to 2,048 tokens, 16 KV heads: 30.8 us, 32.5 with 16), and what
// an item takes beside its steps, in steps (64 ragged requests of up to 8,192: 108 us, 109 with 12, 115 with 5).
constexpr int kSlack = 8;
constexpr int kItemCost = 8;
// Parts of a run (8,192 tokens of one request in 62 parts an item: 14.3 us, 15.0 with 16).
constexpr int kJoin = 8;

constexpr int64_t kMaxSteps = 1ll << 30;   // of a call: all lengths below are 32-bit

struct Division {
    uint32_t total;                        // of the items' lengths, > 0
    uint32_t base, part;                   // a range's length: base + part / 2^16
    float rate;                            // ranges per length
    int teams, slack;
};

FT_HD inline int item_length(int steps) { return steps ? steps + kItemCost : 0; }

// `items` that have steps, `total` length, at most `grid` teams: one for so many steps, or for an
// item where items are shorter; kUnits where that is more and items fewer than `many`.
FT_HD inline Division divide(uint32_t items, uint32_t total, int steps, int grid, uint32_t many) {
    uint32_t t = (total - items * kItemCost + steps - 1) / steps;
    if (t > kUnits && items >= many) t = kMaxTeams;
    if (t < items) t = items;
    if (t > kUnits && items < many) t = kUnits;
    if (t > (uint32_t)grid) t = grid;
    const uint32_t base = total / t, half = (base - 1) / 2;      // less than half a range: few teams stay idle
    return Division{total, base, ((total - base * t) << 16) / t, (float)t / (float)total, (int)t,
                    (int)(half < kSlack ? half : kSlack)};
}
// The cut before team i, and the last team whose cut is at or before a place, before cuts move.
FT_HD inline uint32_t cut(const Division& d, int i) { return i == d.teams ? d.total : d.base * i + (d.part * i >> 16); }
FT_HD inline int team_at(const Division& d, uint32_t place) {
    int i = (int)((float)place * d.rate);              // within one of it
    i = i < d.teams - 1 ? i : d.teams - 1;
    i -= cut(d, i) > place;
    return i + (i < d.teams - 1 && cut(d, i + 1) <= place);
}

// The teams of the item of n steps at `begin`: cuts near its ends, or in its cost, have moved to them.  (A team
// between two cuts that have moved to one place has no work.)
struct Teams {
    int first, last;
};
FT_HD inline Teams teams_of(const Division& d, uint32_t begin, int n) {
    const int after = d.slack < n / 2 ? d.slack : n / 2, before = d.slack < (n - 1) / 2 ? d.slack : (n - 1) / 2;
    return Teams{team_at(d, begin + kItemCost + after), team_at(d, begin + kItemCost + n - 1 - before)};
}
// Steps [from, to) of the item that team i, one of them, works on.
struct Segment {
    int from, to;
};
FT_HD inline Segment segment(const Division& d, const Teams& t, uint32_t begin, int n, int i) {
    return Segment{i == t.first ? 0 : (int)(cut(d, i) - begin) - kItemCost,
                   i == t.last ? n : (int)(cut(d, i + 1) - begin) - kItemCost};
}

// Where a team's part of an item lies: parts of one item side by side, and no two items' overlap, since the
// next item that is cut begins in this one's last team or later.
FT_HD inline int part_slot(const Teams& t, int i) { return t.first + i; }

// An item of up to 2 kJoin parts is joined at once; one of more in runs of kJoin teams, counted from its first,
// and then the runs' sums (at most kMaxTeams / kJoin).
FT_HD inline int join_run(const Teams& t) {
    const int n = t.last - t.first + 1;
    return n <= 2 * kJoin ? n : kJoin;
}

// Query heads of an item and items of a KV head, for a group of g query heads.
FT_HD inline int item_heads(int g) { return g < kCols ? g : kCols; }
FT_HD inline int head_blocks(int g) { return (g + kCols - 1) / kCols; }

// Floats of one partial result: sums, then the heads' maxima and totals, of the part and of the run
// whose sum takes its place.
FT_HD inline int64_t part_floats(int g, int D) { return (int64_t)item_heads(g) * D + 4 * kCols; }

// Workgroups of a launch of at most so many items and steps (up to kMaxSteps).
inline int grid_of(int64_t items, int64_t steps, int D, int esize) {
    return divide((uint32_t)items, (uint32_t)(steps + items * kItemCost), team_steps(D), most_teams(D),
                  many_items(D * esize)).teams;
}

// Items of at most this many steps are not cut, so they need no division: a workgroup each (64 ragged requests of up to
// 1,000 tokens, 8 KV heads: 16 us, 21 divided; one request of 512 and 4 heads: 7.1, 10.4).  Above, few long items would
// leave compute units idle (2,048 tokens of one request, 4 heads: 22 us, 11.5 divided).
constexpr int kDirectWaves = 4;
constexpr int kDirectSteps = 8 * kDirectWaves;

// Two waves an item where items are short and three or more to each of 256 compute units: a wave's start and the sum over
// waves are most of a short item's cost.  us with two, four waves; a window of 128, heads of 64 / 128 / 256:
//   512 items    7.5, 7.4 / 10.8, 11.1 / 20.4, 20.0    e4m3  7.1, 6.5 /  9.5,  8.8 / 16.1, 14.6
//   640          7.9, 8.7 / 13.1, 13.7 / 23.3, 29.1          7.2, 7.4 / 10.2, 10.3 / 18.2, 17.6
//   768          8.5, 9.5 / 14.3, 14.1 / 26.1, 32.6          7.4, 7.7 / 10.7, 11.1 / 19.1, 18.4
//   800          8.9, 9.7 / 15.0, 16.0 / 28.9, 34.3          7.4, 7.9 / 10.9, 12.1 / 19.6, 21.1
// So the border is where the last form begins to gain.  Above eight steps two waves lose, but for heads of 256: windows of
// 256, 2,000 items 24.6, 23.9 / 46.5, 43.8 / 91.8, 93.2.
constexpr int kShortSteps = 8, kManyItems = 768;
inline int direct_waves(int64_t items, int64_t steps) {
    return steps <= kShortSteps && items >= kManyItems ? kDirectWaves / 2 : kDirectWaves;
}

}  // namespace kv
}  // namespace ftmoe
