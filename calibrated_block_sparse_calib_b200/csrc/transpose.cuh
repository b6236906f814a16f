// The skip list by key block: for every (head, key block) the ascending query blocks that keep
// it.  The gradients of K and V sum over the query blocks of a key block, so they walk this list
// where the forward pass and the gradient of Q walk the list by query block.
//
// One CTA per (head, range of key blocks), one launch, no counters and no scan over the list:
//   - a warp reads a row's entries, sets the bit (column, row) in shared memory for those in the
//     CTA's range and counts those before it.  A head has as many entries in either order, so the
//     CTA's output starts at row_ptr[h*nq] + the entries before its range, whatever other CTAs do.
//   - column counts and their prefix give the new row pointers; one warp per column writes out the
//     set bits' indices, a word's 32 rows at a time, side by side.
// Integer work; bits are set in any order and read in one: the result is exact and the same in
// every run.
// A row is ascending, so reading stops behind the range.  Rows longer than 512 entries are first
// narrowed to the 32nd in which the range begins, which costs a dependent probe: up to there reading
// everything before the range is cheaper (40 x 591 x 591 at 25%, 148 entries a row: 105 us with every
// row narrowed, 46 us with a bisection by one thread a row, 16 us as it is).
// What bounds it is the latency of a row's loads, two rows in flight per warp; the 14 MB that a
// 40 x 591 x 591 list at 25% reads and writes would take 2.2 us of HBM time.
#pragma once
#include "ptx.cuh"
#include "select.cuh"

namespace calib {

constexpr int kTransThreads = 1024;
constexpr int kTransWarps = kTransThreads / 32;
constexpr int kTransMaxCols = 128;        // key blocks per CTA, at most
constexpr int kTransNarrow = 512;

__global__ void __launch_bounds__(kTransThreads)
transpose_csr_kernel(const int32_t* __restrict__ row_ptr, const int16_t* __restrict__ col_idx, int H, int nq, int nk,
                     int cols, int32_t* __restrict__ t_row_ptr, int16_t* __restrict__ t_col_idx) {
    extern __shared__ uint32_t bits[];                    // [cols][stride]: bit i of column c's words = row i keeps it
    __shared__ int32_t warp_sum[kTransWarps];
    __shared__ int32_t count[kTransMaxCols], first[kTransMaxCols];
    const int tiles = (nk + cols - 1) / cols;
    const int h = blockIdx.x / tiles;
    const int j0 = (blockIdx.x - h * tiles) * cols, j1 = min(nk, j0 + cols), n_cols = j1 - j0;
    const int words = (nq + 31) / 32, stride = words | 1;   // odd: neighbouring columns on different banks
    const int warp = static_cast<int>(warp_id()), lane = static_cast<int>(lane_id());
    const int r0 = h * nq;
    for (int x = threadIdx.x; x < n_cols * stride; x += kTransThreads) bits[x] = 0u;
    __syncthreads();

    int before = 0;                                       // this lane's entries before the range
    auto visit = [&](int c, int i) {
        if (c < j0) ++before;
        else if (c < j1) atomicOr(&bits[(c - j0) * stride + (i >> 5)], 1u << (i & 31));
    };
    // rows warp, warp + 32, ...: their pointers 32 at a time, one per lane
    for (int b0 = 0; b0 * kTransWarps < nq; b0 += 32) {
        int beg_l = 0, end_l = 0;
        const int il = (b0 + lane) * kTransWarps + warp;
        if (il < nq) {
            beg_l = row_ptr[r0 + il];
            end_l = row_ptr[r0 + il + 1];
            if (beg_l < 0 || end_l < beg_l || end_l - beg_l > nk) {
                raise_status(STATUS_BAD_LIST);
                beg_l = end_l = 0;
            }
        }
        for (int u = 0; u < 32 && (b0 + u) * kTransWarps + warp < nq; u += 2) {
            const int i0 = (b0 + u) * kTransWarps + warp, i1 = i0 + kTransWarps;
            int x0 = __shfl_sync(0xffffffffu, beg_l, u), x1 = __shfl_sync(0xffffffffu, beg_l, u + 1);
            const int e0 = __shfl_sync(0xffffffffu, end_l, u), e1 = __shfl_sync(0xffffffffu, end_l, u + 1);
            // of a long row, skip the whole 32nds that lie before the range
            auto narrow = [&](int& x, int e) {
                while (e - x > kTransNarrow) {
                    const long long len = e - x;
                    const int probe = col_idx[x + static_cast<int>(len * (lane + 1) >> 5) - 1];
                    const int k = __popc(__ballot_sync(0xffffffffu, probe < j0));
                    if (k == 0) break;
                    const int skip = static_cast<int>(len * k >> 5);
                    if (lane == 0) before += skip;
                    x += skip;
                }
            };
            narrow(x0, e0);
            narrow(x1, e1);
            while (x0 < e0 || x1 < e1) {
                int c0[2], c1[2];
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    c0[v] = x0 + v * 32 + lane < e0 ? col_idx[x0 + v * 32 + lane] : 0x7fffffff;
                    c1[v] = x1 + v * 32 + lane < e1 ? col_idx[x1 + v * 32 + lane] : 0x7fffffff;
                }
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    visit(c0[v], i0);
                    visit(c1[v], i1);
                }
                // done with a row once its last entry read is behind the range (or its end was met)
                x0 = __shfl_sync(0xffffffffu, c0[1], 31) >= j1 ? e0 : x0 + 64;
                x1 = __shfl_sync(0xffffffffu, c1[1], 31) >= j1 ? e1 : x1 + 64;
            }
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) before += __shfl_xor_sync(0xffffffffu, before, off);
    if (lane == 0) warp_sum[warp] = before;
    __syncthreads();
    for (int c = warp; c < n_cols; c += kTransWarps) {
        int n = 0;
        for (int w = lane; w < words; w += 32) n += __popc(bits[c * stride + w]);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) n += __shfl_xor_sync(0xffffffffu, n, off);
        if (lane == 0) count[c] = n;
    }
    __syncthreads();
    if (warp == 0) {
        int at = row_ptr[r0] + __reduce_add_sync(0xffffffffu, warp_sum[lane]);
        if (blockIdx.x == 0 && lane == 0) t_row_ptr[0] = at;
        for (int c0 = 0; c0 < n_cols; c0 += 32) {
            const int c = c0 + lane, own = c < n_cols ? count[c] : 0;
            int incl = own;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += y;
            }
            if (c < n_cols) {
                first[c] = at + incl - own;
                t_row_ptr[static_cast<size_t>(h) * nk + j0 + c + 1] = at + incl;
            }
            at += __shfl_sync(0xffffffffu, incl, 31);
        }
    }
    __syncthreads();
    for (int c = warp; c < n_cols; c += kTransWarps) {
        int out = first[c];
        for (int w = 0; w < words; ++w) {
            const uint32_t word = bits[c * stride + w];
            if ((word >> lane) & 1u) t_col_idx[out + __popc(word & lanemask_lt())] = static_cast<int16_t>(w * 32 + lane);
            out += __popc(word);
        }
    }
}

}  // namespace calib
