// etp_groups_of_rows.hpp -- rows in groups of uneven size: how a workgroup
// finds its rows when only the device knows the sizes.
//
// Slots group_ptr[g] .. group_ptr[g + 1] - 1 belong to group g; slot s is row
// order[s] (or s). Groups are cut into tiles of 2^shift slots; tile t of group g
// has the number
//   (group_ptr[g] >> shift) + g + t.
// A group of n slots from p on has at most ((p + n) >> shift) - (p >> shift) + 1
// tiles, so that numbers do not collide, there are (rows >> shift) + n_groups of
// them (at most one a group stands for nothing), and the host can size a grid
// without the sizes; the number's group is the last one that starts at or before
// it, found by 64 probes a step.
#pragma once
#include "etp_dense.hpp"

namespace etp {

struct Groups {
    const int *ptr;    // [n + 1]
    const int *order;  // [rows], or null
    int n, rows;
};

// The start of group i, held to the range of the slots whatever the memory says.
__device__ __forceinline__ int group_start(const Groups &gr, int i)
{
    const int p = gr.ptr[i];
    return p < 0 ? 0 : p < gr.rows ? p : gr.rows;
}

// The last group that starts at or before tile number `tile` (0 where none
// does). Called by whole waves.
__device__ __forceinline__ int group_of_tile(const Groups &gr, int shift, int tile)
{
    const int lane = threadIdx.x & 63;
    int first = 0, count = gr.n;
    for (;;) {
        const int step = (count + 63) >> 6, i = lane * step;
        const bool starts = i < count && (group_start(gr, first + i) >> shift) + first + i <= tile;
        const int found = __builtin_amdgcn_readfirstlane(__popcll(__ballot(starts)));
        const int k = found > 0 ? found - 1 : 0;
        first += k * step;
        if (step == 1)
            return first;
        count = count - k * step < step ? count - k * step : step;
    }
}

// A walk over the tiles from number `tile` to `stop`: the slots slot .. slot + n
// - 1 of group g, n = 0 behind the last one. Called by whole waves.
struct TileWalk {
    int g, begin, end, tile, slot, n;

    __device__ __forceinline__ void start(const Groups &gr, int shift, int from, int stop)
    {
        g = group_of_tile(gr, shift, from);
        begin = group_start(gr, g);
        const int e = group_start(gr, g + 1);
        end = e > begin ? e : begin;
        const int own = (begin >> shift) + g;
        tile = from > own ? from : own;
        n = 0;
        if (tile < stop)
            settle(gr, shift, stop);
    }
    __device__ __forceinline__ void next(const Groups &gr, int shift, int stop)
    {
        n = 0;
        if (++tile < stop)
            settle(gr, shift, stop);
    }
    // the numbers of the group's first and last tile
    __device__ __forceinline__ int first_tile(int shift) const { return (begin >> shift) + g; }
    __device__ __forceinline__ int last_tile(int shift) const { return first_tile(shift) + ((end - begin - 1) >> shift); }

private:
    // From an empty group on to the next one with rows, if one starts before `stop`: 64
    // groups a step. (Taken one by one in the loop below, empty groups cost the others too:
    // 441172 x 64 x 64 float in 4 groups, none empty, 120 us, so 111.)
    __device__ __forceinline__ bool pass_empty(const Groups &gr, int shift, int stop)
    {
        for (; g < gr.n && first_tile(shift) < stop; g += 64) {
            const int i = g + (threadIdx.x & 63);
            const uint64_t some = __ballot(i < gr.n && group_start(gr, i + 1) > group_start(gr, i));
            if (some) {
                g += __builtin_ctzll(some);
                begin = group_start(gr, g);
                end = group_start(gr, g + 1);
                return true;
            }
        }
        return false;
    }
    __device__ __forceinline__ void settle(const Groups &gr, int shift, int stop)
    {
        for (;;) {
            const int64_t at = begin + (static_cast<int64_t>(tile - first_tile(shift)) << shift);
            if (at < end) {
                slot = static_cast<int>(at);
                n = end - slot < (1 << shift) ? end - slot : 1 << shift;
                return;
            }
            if (++g >= gr.n)
                return;
            begin = end;
            const int e = group_start(gr, g + 1);
            end = e > begin ? e : begin;
            if (end == begin && !pass_empty(gr, shift, stop))
                return;
            const int own = first_tile(shift);
            tile = tile > own ? tile : own;
            if (tile >= stop)
                return;
        }
    }
};

// The row of a slot, or -1 for one past the tile (and for an index that is no
// row: what it would have named is left alone).
__device__ __forceinline__ int row_of_slot(const Groups &gr, int slot, bool live)
{
    if (!live)
        return -1;
    const int r = gr.order ? gr.order[slot] : slot;
    return static_cast<unsigned>(r) < static_cast<unsigned>(gr.rows) ? r : -1;
}

}  // namespace etp
