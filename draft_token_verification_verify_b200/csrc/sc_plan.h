// What the host side knows of the attention kernels.
#pragma once

namespace sv {

struct AttendParams;

struct AttendKernel {
    void (*fn)(AttendParams);
    int threads, smem;  // of a CTA
    int block_rows;     // rows a CTA takes at once
    int per_sm;         // CTAs an SM holds
    int tile;           // tokens of a tile
};

constexpr int SC_MOST_ROWS = 80;  // of a block

// The kernel for blocks of up to `rows` rows (at most SC_MOST_ROWS).
template <int DT, int D>
AttendKernel attend_kernel(int rows);

}  // namespace sv
