// Groups of rows (the rows of each expert) as the grouped kernels see them.
//
// A call gets `groups` cumulative end positions in device memory: group e
// holds rows [end(e-1), end(e)), end(-1) = 0.  The positions are a router's
// output that the host never sees, so every workgroup derives what it needs
// from them: the row range of its group, where the group's part of a blob
// starts, and which group the workgroup's tile falls into.  Values outside
// [0, M] are clamped and a value below its predecessor counts as the
// predecessor (an empty group), so no input leads out of the buffers.
//
// A wave reads 64 positions at a time, one per lane, and forms the running
// maximum and the running sums of per-group unit counts with DPP row shifts
// and row broadcasts: 6 steps per 64 groups and quantity, no LDS.
#pragma once

#include "mx_internal.h"

namespace mx {
namespace {

// Inclusive scan over the wave's 64 lanes (values >= 0; identity 0).
// DPP row_shr:1, 2, 4, 8 scan each row of 16 lanes, row_bcast:15 adds row
// 0's and 2's last lane to rows 1 and 3, row_bcast:31 lane 31's to the upper
// half.
template <bool MAX>
__device__ __forceinline__ int wave_scan(int v) {
    const auto op = [](int a, int b) { return MAX ? (a > b ? a : b) : a + b; };
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false));
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false));
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false));
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false));
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false));
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false));
    return v;
}

// Number `b` of `total` in XCD-contiguous order, or -1 (a workgroup past its
// XCD's share).
__device__ __forceinline__ int xcd_position(int b, int total) {
    const int xcd = b % kXcds, local = b / kXcds;
    const int per = total / kXcds, rem = total % kXcds;
    if (local >= per + (xcd < rem ? 1 : 0)) return -1;
    return xcd * per + (xcd < rem ? xcd : rem) + local;
}

// Where a group lies, in rows and in blob units.
struct GroupPos {
    int group;       // its index, or `groups` for the rows behind the last group
    int start, rows; // its rows
    int tile;        // the tile looked for, counted inside the group
    int r16;         // 16-row units of the groups before it (row-wise blob)
    int k128, k512;  // 128-row and 512-row units before it (column-wise blob: data, scales)
};

// One block of 64 groups: lane l holds group base + l.
struct GroupLane {
    int start, rows;
    int tiles, r16, k128, k512;   // inclusive running sums, previous blocks' included
};

__device__ __forceinline__ int units(int n, int per) { return (int)(((uint32_t)n + (uint32_t)per - 1u) / (uint32_t)per); }

// What the blocks before the current one add up to (uniform over the wave).
struct GroupCarry {
    int end = 0, tiles = 0, r16 = 0, k128 = 0, k512 = 0;
};

// UNITS: also the running blob units (otherwise only tiles of TILE rows).
template <int TILE, bool UNITS>
__device__ __forceinline__ GroupLane group_block(const int32_t *__restrict__ ends, int groups, int M, int base,
                                                 int lane, GroupCarry &c) {
    const int e = base + lane;
    int end = e < groups ? ends[e] : 0;
    end = end < 0 ? 0 : (end > M ? M : end);
    end = wave_scan<true>(end > c.end ? end : c.end);
    // the previous lane's end (lane 0: the previous block's)
    int start = __builtin_amdgcn_ds_bpermute(4 * (lane - 1), end);
    start = lane == 0 ? c.end : start;
    GroupLane g;
    g.start = start;
    g.rows = end - start;
    g.tiles = c.tiles + wave_scan<false>(units(g.rows, TILE));
    c.end = __builtin_amdgcn_readlane(end, 63);
    c.tiles = __builtin_amdgcn_readlane(g.tiles, 63);
    g.r16 = g.k128 = g.k512 = 0;
    if constexpr (UNITS) {
        g.r16 = c.r16 + wave_scan<false>(units(g.rows, 16));
        g.k128 = c.k128 + wave_scan<false>(units(g.rows, 128));
        g.k512 = c.k512 + wave_scan<false>(units(g.rows, 512));
        c.r16 = __builtin_amdgcn_readlane(g.r16, 63);
        c.k128 = __builtin_amdgcn_readlane(g.k128, 63);
        c.k512 = __builtin_amdgcn_readlane(g.k512, 63);
    }
    return g;
}

// The group in lane l of a block, as uniform values.
template <int TILE>
__device__ __forceinline__ GroupPos group_at(const GroupLane &g, int base, int l, int tile) {
    GroupPos p;
    p.group = base + l;
    p.start = __builtin_amdgcn_readlane(g.start, l);
    p.rows = __builtin_amdgcn_readlane(g.rows, l);
    p.tile = tile - (__builtin_amdgcn_readlane(g.tiles, l) - units(p.rows, TILE));
    p.r16 = __builtin_amdgcn_readlane(g.r16, l) - units(p.rows, 16);
    p.k128 = __builtin_amdgcn_readlane(g.k128, l) - units(p.rows, 128);
    p.k512 = __builtin_amdgcn_readlane(g.k512, l) - units(p.rows, 512);
    return p;
}

// The group that holds tile `tile` of the sequence of all groups' tiles (TILE
// rows each, a group's last one possibly short), followed by the tiles of the
// rows behind the last group.  False: there is no such tile.  pick(total)
// chooses the tile when the number of tiles (rows behind the last group
// included) is known.
template <int TILE, typename PICK>
__device__ __forceinline__ bool find_tile(const int32_t *__restrict__ ends, int groups, int M, PICK pick,
                                          GroupPos &p) {
    const int lane = threadIdx.x & 63;
    GroupCarry c;
    GroupLane g = group_block<TILE, true>(ends, groups, M, 0, lane, c);
    for (int base = 64; base < groups; base += 64) group_block<TILE, true>(ends, groups, M, base, lane, c);
    const int rest = M - c.end;
    const int tile = pick(c.tiles + units(rest, TILE));
    if (tile < 0 || tile >= c.tiles + units(rest, TILE)) return false;
    if (tile >= c.tiles) {
        p = GroupPos{groups, c.end, rest, tile - c.tiles, c.r16, c.k128, c.k512};
        return true;
    }
    GroupCarry d;
    for (int base = 0; base < groups; base += 64) {
        if (groups > 64) g = group_block<TILE, true>(ends, groups, M, base, lane, d);
        const uint64_t past = __builtin_amdgcn_ballot_w64(tile < g.tiles);
        if (past) {
            p = group_at<TILE>(g, base, __builtin_ctzll(past), tile);
            return true;
        }
    }
    return false;
}

// Group `group`'s position.
__device__ __forceinline__ GroupPos find_group(const int32_t *__restrict__ ends, int groups, int M, int group) {
    const int lane = threadIdx.x & 63;
    GroupCarry c;
    for (int base = 0;; base += 64) {
        const GroupLane g = group_block<128, true>(ends, groups, M, base, lane, c);
        if (group < base + 64) return group_at<128>(g, base, group - base, 0);
    }
}

}  // namespace
}  // namespace mx
