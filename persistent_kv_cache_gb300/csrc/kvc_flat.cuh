// kvc_flat.cuh -- one even share of a ragged batch for every CTA.
//
// The attention over a batch is B x heads independent rows, row (b, h) made
// of n_b equal units of keys; the lengths, and with them n_b, are known on
// the device only.  Laid end to end (b outermost, then h, then the unit) the
// rows are one line of U = heads * sum_b n_b units, cut into G shares of U / G
// units, the first U % G of them one longer: every CTA gets the same work
// whatever the lengths, with no queue, no counters and the same split on every
// run.
// A CTA's share is a tail of one row, whole rows, and a head of another, so
// it leaves at most two partial results (slot 0: its first segment, slot 1:
// its last), and the scratch for them depends on the grid alone.
#pragma once

#include "kvc_common.cuh"

namespace kvc_flat {

struct Shares {
    int each, longer;  // shares [0, longer) are of each + 1 units, the others of each
    __device__ __forceinline__ Shares(int U, int grid) : each(U / grid), longer(U % grid) {}
    __device__ __forceinline__ int begin(int c) const { return c * each + min(c, longer); }
    // the share that holds unit x (0 <= x < U); the shares of a row are
    // consecutive, and none of them is empty
    __device__ __forceinline__ int of(int x) const
    {
        const int head = longer * (each + 1);
        return x < head ? x / (each + 1) : longer + (x - head) / each;
    }
};

// Walks the batch with one warp.  `count(b)` is n_b (>= 0).  Returns U; for
// the unit x (or, when x < 0, for the row b_in) gives the batch row and the
// line position of that row's first unit.
template <typename Count>
__device__ __forceinline__ int locate(int batch, int heads, const Count &count, int b_in, int &b_out,
                                      int &base_out)
{
    const int lane = threadIdx.x & 31;
    int cum = 0;
    b_out = b_in;
    base_out = 0;
    for (int b0 = 0; b0 < batch; b0 += 32) {
        const int n = b0 + lane < batch ? count(b0 + lane) * heads : 0;
        int inc = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d)
                inc += v;
        }
        if (b_in >= b0 && b_in < b0 + 32)
            base_out = cum + __shfl_sync(0xffffffffu, inc - n, b_in - b0);
        cum += __shfl_sync(0xffffffffu, inc, 31);
    }
    return cum;
}

// the batch row that holds unit x (0 <= x < U) and its first unit's position
template <typename Count>
__device__ __forceinline__ void row_of(int batch, int heads, const Count &count, int x, int &b_out,
                                       int &base_out)
{
    const int lane = threadIdx.x & 31;
    int cum = 0;
    b_out = -1;
    base_out = 0;
    for (int b0 = 0; b0 < batch && b_out < 0; b0 += 32) {
        const int n = b0 + lane < batch ? count(b0 + lane) * heads : 0;
        int inc = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d)
                inc += v;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, cum + inc > x);
        if (past) {
            const int at = __ffs(past) - 1;
            b_out = b0 + at;
            base_out = cum + __shfl_sync(0xffffffffu, inc - n, at);
        }
        cum += __shfl_sync(0xffffffffu, inc, 31);
    }
}

// The share [x, x_end) of CTA c of a grid, the batch row of unit x and that
// row's first unit's position (b and base only when the share is not empty).
// Up to 32 batch rows take one pass over their lengths.
template <typename Count>
__device__ __forceinline__ Shares share_of_cta(int batch, int heads, const Count &count, int grid, int c, int &x,
                                               int &x_end, int &b, int &base)
{
    if (batch > 32) {
        const int U = locate(batch, heads, count, -1, b, base);
        const Shares shares(U, grid);
        x = shares.begin(c);
        x_end = shares.begin(c + 1);
        if (x < x_end)
            row_of(batch, heads, count, x, b, base);
        return shares;
    }
    const int lane = threadIdx.x & 31;
    const int n = lane < batch ? count(lane) * heads : 0;
    int inc = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d)
            inc += v;
    }
    const Shares shares(__shfl_sync(0xffffffffu, inc, 31), grid);
    x = shares.begin(c);
    x_end = shares.begin(c + 1);
    b = __ffs(__ballot_sync(0xffffffffu, inc > x)) - 1;
    base = __shfl_sync(0xffffffffu, inc - n, b & 31);
    return shares;
}

} // namespace kvc_flat
