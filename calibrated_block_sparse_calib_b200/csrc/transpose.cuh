// The skip list by key block: for every (head, key block) the ascending query blocks that keep
// it.  The gradients of K and V sum over the query blocks of a key block, so they walk this list
// where the forward pass and the gradient of Q walk the list by query block.
//
// One CTA per (head, 32 consecutive key blocks), one launch, no counters and no scan over the
// list:
//   - every row's first entry at or past the CTA's columns is found by bisection, since a row is
//     ascending.  The entries before it, summed over the head's rows, are the entries of all
//     earlier columns, and a head has as many entries in either order: the CTA's output starts at
//     row_ptr[h*nq] + that sum.
//   - the row's entries inside the 32 columns become one 32-bit word, and 32 such words are turned
//     over by 32 ballots into one word of rows per column, kept in shared memory;
//   - column counts and their prefix give the new row pointers; one warp per column writes out the
//     set bits' indices.
// Integer work in a fixed order: the result is exact and the same in every run.
// The list is read once per CTA column range only where it has entries, plus about log2(row)
// probes a row; what bounds a call is the latency of those dependent probes (a 40 x 591 x 591 list
// at 25%, 3.5 M entries, 14 MB in and out, is 2.2 us of HBM traffic).
#pragma once
#include "ptx.cuh"
#include "select.cuh"

namespace calib {

constexpr int kTransThreads = 256;
constexpr int kTransCols = 32;

__global__ void __launch_bounds__(kTransThreads)
transpose_csr_kernel(const int32_t* __restrict__ row_ptr, const int16_t* __restrict__ col_idx, int H, int nq, int nk,
                     int32_t* __restrict__ t_row_ptr, int16_t* __restrict__ t_col_idx) {
    extern __shared__ uint32_t colbits[];                 // [kTransCols][words]
    __shared__ int32_t warp_sum[kTransThreads / 32];
    __shared__ int32_t count[kTransCols], first[kTransCols];
    const int tiles = (nk + kTransCols - 1) / kTransCols;
    const int h = blockIdx.x / tiles;
    const int j0 = (blockIdx.x - h * tiles) * kTransCols;
    const int words = (nq + 31) / 32;
    const int warp = static_cast<int>(warp_id()), lane = static_cast<int>(lane_id());
    const int r0 = h * nq;
    int before = 0;
    for (int w = warp; w < words; w += kTransThreads / 32) {
        const int i = w * 32 + lane;
        uint32_t bits = 0;
        if (i < nq) {
            const int beg = row_ptr[r0 + i], end = row_ptr[r0 + i + 1];
            if (beg < 0 || end < beg || end - beg > nk) {
                raise_status(STATUS_BAD_LIST);
            } else {
                int lo = beg, hi = end;
                while (lo < hi) {
                    const int mid = (lo + hi) >> 1;
                    if (col_idx[mid] < j0) lo = mid + 1;
                    else hi = mid;
                }
                before += lo - beg;
                for (; lo < end; ++lo) {
                    const int c = col_idx[lo] - j0;
                    if (c >= kTransCols) break;
                    if (c >= 0) bits |= 1u << c;
                }
            }
        }
        uint32_t mine = 0;
#pragma unroll
        for (int c = 0; c < kTransCols; ++c) {
            const uint32_t rows = __ballot_sync(0xffffffffu, (bits >> c) & 1u);
            if (lane == c) mine = rows;
        }
        colbits[lane * words + w] = mine;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) before += __shfl_xor_sync(0xffffffffu, before, off);
    if (lane == 0) warp_sum[warp] = before;
    __syncthreads();
    for (int c = warp; c < kTransCols; c += kTransThreads / 32) {
        int n = 0;
        for (int w = lane; w < words; w += 32) n += __popc(colbits[c * words + w]);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) n += __shfl_xor_sync(0xffffffffu, n, off);
        if (lane == 0) count[c] = n;
    }
    __syncthreads();
    if (warp == 0) {
        int at = row_ptr[r0];
#pragma unroll
        for (int w = 0; w < kTransThreads / 32; ++w) at += warp_sum[w];
        int incl = count[lane];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += y;
        }
        first[lane] = at + incl - count[lane];
        if (j0 + lane < nk) t_row_ptr[static_cast<size_t>(h) * nk + j0 + lane + 1] = at + incl;
        if (blockIdx.x == 0 && lane == 0) t_row_ptr[0] = at;
    }
    __syncthreads();
    for (int c = warp; c < kTransCols; c += kTransThreads / 32) {
        int out = first[c];
        for (int w0 = 0; w0 < words; w0 += 32) {
            uint32_t bits = w0 + lane < words ? colbits[c * words + w0 + lane] : 0u;
            const int n = __popc(bits);
            int incl = n;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += y;
            }
            int o = out + incl - n;
            while (bits) {
                const int b = __ffs(bits) - 1;
                bits &= bits - 1;
                t_col_idx[o++] = static_cast<int16_t>((w0 + lane) * 32 + b);
            }
            out += __shfl_sync(0xffffffffu, incl, 31);
        }
    }
}

}  // namespace calib
