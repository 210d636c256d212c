// How layer norm's calls are cut into units, blocks and shared memory: host
// arithmetic, of sizes, formats and places alone.
#pragma once

#include "wgs_sizes.h"

namespace wgs {

namespace {

constexpr int kMaxWidth = 8192;
constexpr int kWarps = 12;          // of a block, at most
constexpr int kThreads = kWarps * 32;
constexpr int kMeet = kWarps / 3 * 4;   // places of their sums: units of three warps have four each
constexpr int kMaxStages = 4;
constexpr int kExchangeBytes = 2 * kMeet * 8;   // of units of several warps
constexpr int kEdgeBytes = kWarps * 8 * 32;     // of ragged rows' ends
constexpr int kEdgeKinds = 3;                   // of chunks that are not full, in the forward
constexpr int kept_edges(int value_bytes) { return kEdgeKinds * (16 + 16 / value_bytes * 4); }

// Shared memory of an SM, and what the device keeps of it for each block.
constexpr int kSmBytes = 228 << 10, kBlockReserve = 1 << 10;
constexpr int kMostOfSm = 216 << 10;   // a block's, at most

// ------------------------------------------------------------------- units --

// A row's unit: chunks that a thread holds, and lanes of a warp, or 0 for several warps.
struct Unit {
    int each, team;
};

// Chunks a thread for units of several warps: those that leave the fewest of a block's
// threads without a part of a row.
inline int chunks_of_units(int chunks, bool six) {
    const int sizes[] = {3, 2, 6};
    int best = 0, best_score = 0;
    for (int c : sizes) {
        const int warps = static_cast<int>(ceil_div(chunks, 32 * c));
        if ((c == 6 && !six) || warps < 2 || warps > kWarps) continue;
        const int score = chunks * 1000 / (warps * 32 * c) * (kWarps / warps * warps) / kWarps;
        if (score > best_score) best = c, best_score = score;
    }
    return best;
}

// Warps of the forward's blocks: two blocks an SM, whose waits fall at different times;
// of fewer warps where a thread's 32 columns need the registers.
constexpr int forward_warps(int each, int value_bytes) { return each * 16 / value_bytes > 24 ? 8 : kWarps; }
// (Six chunks a thread are for rows whose weights leave no room for a second block.)
constexpr int forward_blocks_per_sm(int each) { return each == 6 ? 1 : 2; }

// The narrowest unit that holds a row in three chunks a thread, and the fewest chunks
// that do; four for a whole warp: rows just above its 96 chunks would take a second one
// ([32761, 771] bf16 with residual 45 us, with two warps of two chunks 56).  Four lanes
// for the narrowest ([600000, 24] bf16 15 us, with eight 28).
inline Unit forward_unit(int chunks, int value_bytes, bool whole) {
    if (chunks <= 4) return {1, 4};
    if (chunks <= 8) return {1, 8};
    if (chunks <= 16) return {2, 8};
    if (chunks <= 24) return {3, 8};
    if (chunks <= 32) return {2, 16};
    if (chunks <= 48) return {3, 16};
    if (chunks <= 64) return {2, 32};
    if (chunks <= 96) return {3, 32};
    if (chunks <= 128) return {4, 32};
    const int each = chunks_of_units(chunks, value_bytes == 4 && chunks > 96 * kWarps);
    // Four where that takes fewer than three quarters of the warps ([32768, 4096] bf16 90
    // us, with three chunks 104; [16384, 8192] 103, so 116; but [29127, 4608] 126, so 96),
    // and not for ragged rows ([32760, 4097] 206, so 143), whose ends want more warps.
    if (whole && value_bytes == 2) {
        const int warps = static_cast<int>(ceil_div(chunks, 32 * each)), fewer = static_cast<int>(ceil_div(chunks, 128));
        if (fewer <= forward_warps(4, value_bytes) && 4 * fewer < 3 * warps) return {4, 0};
    }
    return {each, 0};
}

// Units of several warps that forward_unit names: where it has four chunks a thread for
// whole rows of 16 bits, it never has two.
constexpr bool forward_has_warps(int each, int value_bytes, bool whole) {
    if (value_bytes == 4) return each == 2 || each == 3 || each == 6;
    return each == 3 || each == (whole ? 4 : 2);
}

// --------------------------------------------------------------- rows, memory --

// A call's blocks and units: as many units a block as its warps hold, or so few
// that every SM gets some where the rows are few, and at least a block for each
// class of rows (`period` of them).
struct Cut {
    int blocks, units, threads;
};

inline Cut cut_rows(int64_t rows, int period, int team_warps, int rows_per_pass, int most_warps, int most_blocks) {
    const int64_t passes = ceil_div(rows, rows_per_pass);
    int64_t units = most_warps / team_warps;
    if (units > ceil_div(passes, most_blocks)) units = ceil_div(passes, most_blocks);
    int64_t blocks = ceil_div(passes, units);
    if (blocks > most_blocks) blocks = most_blocks;
    const int64_t kinds = rows < period ? rows : period;
    if (blocks < kinds) blocks = kinds;
    return {static_cast<int>(blocks), static_cast<int>(units), static_cast<int>(units) * team_warps * 32};
}

// The forward's static shared memory: sums of units' warps; ragged rows' ends, and what
// of their chunks is the row's.
constexpr int forward_static_bytes(int team, int value_bytes, bool whole) {
    return (team == 0 ? kExchangeBytes : 0) + (whole ? 0 : kEdgeBytes + kept_edges(value_bytes));
}

struct ForwardCut {
    Cut cut;
    int team_warps, kept_bytes, stages, smem;     // kept: before the slots; smem: dynamic
    bool two;                                     // blocks an SM
};

// Two blocks an SM where two stages beside the weights fit twice, with as many as both have
// room for.
inline ForwardCut forward_cut(Unit u, int chunks, int tensors, int value_bytes, bool whole, int64_t rows, int period, int sms) {
    ForwardCut f;
    f.team_warps = u.team == 0 ? static_cast<int>(ceil_div(chunks, 32 * u.each)) : 1;
    f.kept_bytes = u.each * (u.team == 0 ? 32 * f.team_warps : u.team) * 8 * (16 / value_bytes);     // weight and bias
    const int warps = forward_warps(u.each, value_bytes);
    const int most = warps / f.team_warps * f.team_warps * tensors * u.each * 512;
    const int half = kSmBytes / 2 - kBlockReserve - forward_static_bytes(u.team, value_bytes, whole);
    f.two = forward_blocks_per_sm(u.each) == 2 && f.kept_bytes + 2 * most <= half;
    f.cut = cut_rows(rows, period, f.team_warps, u.team == 0 ? 1 : 32 / u.team, warps, (f.two ? 2 : 1) * sms);
    const int stage = f.cut.threads * tensors * u.each * 16, fit = ((f.two ? half : kMostOfSm) - f.kept_bytes) / stage;
    f.stages = fit < kMaxStages ? fit : kMaxStages;
    f.smem = f.kept_bytes + f.stages * stage;
    return f;
}

}  // namespace

}  // namespace wgs
