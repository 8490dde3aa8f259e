// Helpers shared by the LDS-tiled GEMMs: operand halves, the workgroup ->
// tile mapping, LDS swizzles, the wait on direct-to-LDS loads and the choice of
// a tile shape.
#pragma once

#include "common.hpp"

namespace fp8q {

constexpr int kCUs = 256;                // compute units of an MI355X

__device__ __forceinline__ v8i cat(const v4i& lo, const v4i& hi)
{
    return v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}

// Workgroups are dispatched round-robin over the 8 XCDs; map the launch index
// so that each XCD receives a contiguous range of logical tile ids.
__device__ __forceinline__ int xcd_remap(int bid, int nb)
{
    const int q = nb >> 3, rem = nb & 7;
    const int xcd = bid & 7, idx = bid >> 3;
    return xcd < rem ? xcd * (q + 1) + idx : rem * (q + 1) + (xcd - rem) * q + idx;
}

// Byte offset of 16-byte unit `u` of row `row` in a tile with 128-byte rows.
__device__ __forceinline__ int swz128(int row, int u) { return row * 128 + ((u ^ (row & 7)) << 4); }
// ... with 64-byte rows (4 units).
__device__ __forceinline__ int swz64(int row, int u) { return row * 64 + ((u ^ ((row >> 1) & 3)) << 4); }

// The compiler does not order LDS reads after asynchronous direct-to-LDS
// loads, so a kernel that uses them waits explicitly (s_waitcnt vmcnt) for
// its own loads and then synchronizes the workgroup before reading.
template <int N_OUTSTANDING>
__device__ __forceinline__ void wait_vm()
{
    // s_waitcnt vmcnt(N) with expcnt and lgkmcnt left at their maxima (gfx9 encoding)
    static_assert(N_OUTSTANDING >= 0 && N_OUTSTANDING < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N_OUTSTANDING & 15) | ((N_OUTSTANDING >> 4) << 14) | (7 << 4) | (15 << 8));
}

// A tile shape, how many of its workgroups a CU holds, and the time of one
// round of them.
struct TileShape { int bm, bn, per_cu; float round_us; };

// The shape of `shapes` whose rounds of workgroups cost least; tiles may not
// be taller than M rounded up to 64 rows.
inline int pick_tile_shape(const TileShape* shapes, int count, int M, int N)
{
    const int64_t mcap = ((int64_t)M + 63) / 64 * 64;
    int best = -1;
    float best_us = 0.f;
    for (int i = 0; i < count; ++i) {
        const TileShape& t = shapes[i];
        if (t.bm > mcap) continue;
        const int64_t tiles = (((int64_t)M + t.bm - 1) / t.bm) * (((int64_t)N + t.bn - 1) / t.bn);
        const int64_t slots = (int64_t)kCUs * t.per_cu;
        const float us = (float)((tiles + slots - 1) / slots) * t.round_us;
        if (best < 0 || us < best_us) { best = i; best_us = us; }
    }
    return best;
}

}  // namespace fp8q
