// Gradients of block-sparse attention.
#pragma once
#include <cuda_bf16.h>
#include "ptx.cuh"
#include "attn_fwd.cuh"

namespace calib {

struct BwdParams {
    const __nv_bfloat16 *q, *k, *v;      // [H, N, D]
    const void *o, *dout;                // [H, N, D] bf16, or fp32 when io_f32
    const float* lse;                    // [H, N] natural log
    void *dq, *dk, *dv;                  // [H, N, D] bf16, or fp32 when grad_f32
    float2* stats;                       // workspace [H, nq * BLK]: (LSE / ln 2, delta)
    __nv_bfloat16* do16;                 // workspace [H, N, D] (io_f32), else dout itself
    __nv_bfloat16 *qa, *doa;             // workspace [H, n_anchor, D] (repeat heads) or nullptr
    const int32_t *row_ptr, *t_row_ptr;
    const int16_t *col_idx, *t_col_idx;
    const int32_t *work, *t_work;
    int n_work, n_t_work;
    AttnParams geo;                      // H, N, nq, nk, scale_log2 and the repeat geometry
    float scale;
    int io_f32, grad_f32;
    uint64_t timeout_ns;
};

__device__ __forceinline__ bool repeats(const AttnParams& p, int h) {
    return (p.repeat_bits[h >> 5] >> (h & 31)) & 1u;
}

// Number of tokens that take anchor a's output, Wl tokens apart from the anchor on.
__device__ __forceinline__ int anchor_copies(const AttnParams& p, int a) {
    if (a >= p.F * p.Ar * p.Wl) return 1;
    return min(p.stride, p.Hl - ((a / p.Wl) % p.Ar) * p.stride);
}

// Row statistics (LSE / ln 2, delta = sum_d dO O), one group of D/8 threads per query row, and the
// operands that the products need as bf16: dO when it came as fp32, and for a repeat head the
// anchors' rows of Q with dO and delta summed over the tokens that take the anchor's output (its O
// and LSE are the same in all of them).  The sum is fp32 and dO enters the products as bf16, so it
// is rounded once (2^-9 relative), as P and dS are.  Rows past the sequence get LSE = +inf, which
// makes their probabilities 0; so do rows with nothing kept (LSE = -inf).
// Reads dO and O once: 2 x 268 MB at 12 x 32760 x 128, bound by memory.
template <int D>
__global__ void __launch_bounds__(256) bwd_prepare_kernel(const BwdParams p, int rows_padded) {
    constexpr int TPR = D / 8;                            // threads per row, 8 values each
    const AttnParams& g = p.geo;
    const long long idx = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) / TPR;
    const int part = threadIdx.x % TPR;
    const int h = static_cast<int>(idx / rows_padded), r = static_cast<int>(idx % rows_padded);
    if (h >= g.H) return;                                 // whole rows: TPR divides 256
    const bool rep = repeats(g, h);
    const int Nq = rep ? g.n_anchor : g.N;
    float acc = 0.f, lse = INFINITY;
    if (r < Nq) {
        const int tok = rep ? anchor_token(g, r) : r;
        const int n = rep ? anchor_copies(g, r) : 1;
        float dsum[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) dsum[e] = 0.f;
        for (int c = 0; c < n; ++c) {
            const size_t at = (static_cast<size_t>(h) * g.N + tok + static_cast<size_t>(c) * g.Wl) * D + part * 8;
            float a[8], b[8];
            if (p.io_f32) {
                const float4* x = reinterpret_cast<const float4*>(static_cast<const float*>(p.dout) + at);
                const float4* y = reinterpret_cast<const float4*>(static_cast<const float*>(p.o) + at);
                const float4 x0 = x[0], x1 = x[1], y0 = y[0], y1 = y[1];
                a[0] = x0.x; a[1] = x0.y; a[2] = x0.z; a[3] = x0.w; a[4] = x1.x; a[5] = x1.y; a[6] = x1.z; a[7] = x1.w;
                b[0] = y0.x; b[1] = y0.y; b[2] = y0.z; b[3] = y0.w; b[4] = y1.x; b[5] = y1.y; b[6] = y1.z; b[7] = y1.w;
            } else {
                const uint4 x = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.dout) + at);
                const uint4 y = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.o) + at);
                const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    a[2 * e] = __uint_as_float(xs[e] << 16);
                    a[2 * e + 1] = __uint_as_float(xs[e] & 0xFFFF0000u);
                    b[2 * e] = __uint_as_float(ys[e] << 16);
                    b[2 * e + 1] = __uint_as_float(ys[e] & 0xFFFF0000u);
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                acc += a[e] * b[e];
                dsum[e] += a[e];
            }
        }
        if (rep || p.io_f32) {
            const uint4 w = make_uint4(pack_bf16x2(dsum[0], dsum[1]), pack_bf16x2(dsum[2], dsum[3]),
                                       pack_bf16x2(dsum[4], dsum[5]), pack_bf16x2(dsum[6], dsum[7]));
            if (rep) {
                const size_t to = (static_cast<size_t>(h) * g.n_anchor + r) * D + part * 8;
                *reinterpret_cast<uint4*>(p.doa + to) = w;
                *reinterpret_cast<uint4*>(p.qa + to) =
                    *reinterpret_cast<const uint4*>(p.q + (static_cast<size_t>(h) * g.N + tok) * D + part * 8);
            } else {
                *reinterpret_cast<uint4*>(p.do16 + (static_cast<size_t>(h) * g.N + r) * D + part * 8) = w;
            }
        }
        const float l = p.lse[static_cast<size_t>(h) * g.N + tok];
        lse = l == -INFINITY ? INFINITY : l * 1.4426950408889634f;
    }
#pragma unroll
    for (int off = TPR / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
    if (part == 0) p.stats[static_cast<size_t>(h) * rows_padded + r] = make_float2(lse, acc);
}

// One warp per row of a block: KV = false, the row is a query and the columns are its kept keys
// (dQ); KV = true, the row is a key and the columns are the queries that keep it (dK, dV).
// s = a.c and dp = b.e for a lane's column, p = 2^(s - LSE), ds = p (dp - delta); then
// out1 += ds c, out2 += p e with the lanes over D.
template <int D, int BLK, bool KV>
__global__ void __launch_bounds__(256) bwd_simple_kernel(const BwdParams p) {
    constexpr int LD = D + 2, SUB = 32;
    __shared__ __nv_bfloat16 sc[SUB * LD], se[SUB * LD];
    __shared__ float sa[8][D], sb[8][D];
    const AttnParams& g = p.geo;
    const int nrow = KV ? g.nk : g.nq;
    const int h = blockIdx.y, i = blockIdx.x / (BLK / 8), sub = blockIdx.x % (BLK / 8);
    const int warp = static_cast<int>(warp_id()), lane = static_cast<int>(lane_id());
    const bool rep = repeats(g, h);
    const int Nq = rep ? g.n_anchor : g.N;
    const __nv_bfloat16* q = rep ? p.qa + static_cast<size_t>(h) * g.n_anchor * D : p.q + static_cast<size_t>(h) * g.N * D;
    const __nv_bfloat16* dO = rep ? p.doa + static_cast<size_t>(h) * g.n_anchor * D : p.do16 + static_cast<size_t>(h) * g.N * D;
    const __nv_bfloat16* k = p.k + static_cast<size_t>(h) * g.N * D;
    const __nv_bfloat16* v = p.v + static_cast<size_t>(h) * g.N * D;
    const __nv_bfloat16 *A = KV ? k : q, *Bm = KV ? v : dO, *C = KV ? q : k, *E = KV ? dO : v;
    const int rows = KV ? g.N : Nq, cols = KV ? Nq : g.N;
    const int r = i * BLK + sub * 8 + warp;
    for (int d = lane; d < D; d += 32) {
        sa[warp][d] = r < rows ? __bfloat162float(A[static_cast<size_t>(r) * D + d]) : 0.f;
        sb[warp][d] = r < rows ? __bfloat162float(Bm[static_cast<size_t>(r) * D + d]) : 0.f;
    }
    const float2* stats = p.stats + static_cast<size_t>(h) * g.nq * BLK;
    const float2 own = !KV && r < rows ? stats[r] : make_float2(INFINITY, 0.f);
    float o1[D / 32], o2[D / 32];
#pragma unroll
    for (int x = 0; x < D / 32; ++x) o1[x] = o2[x] = 0.f;
    const int32_t* rp = KV ? p.t_row_ptr : p.row_ptr;
    const int16_t* ci = KV ? p.t_col_idx : p.col_idx;
    const int beg = rp[h * nrow + i], end = i * BLK < rows ? rp[h * nrow + i + 1] : beg;
    for (int x = beg; x < end; ++x) {
        const int j = ci[x];
        for (int c0 = 0; c0 < BLK; c0 += SUB) {
            __syncthreads();
            for (int y = threadIdx.x; y < SUB * D / 2; y += 256) {
                const int c = y / (D / 2), d = y % (D / 2) * 2;
                const int n = j * BLK + c0 + c;
                uint32_t w0 = 0, w1 = 0;
                if (j >= 0 && n < cols) {
                    w0 = *reinterpret_cast<const uint32_t*>(C + static_cast<size_t>(n) * D + d);
                    w1 = *reinterpret_cast<const uint32_t*>(E + static_cast<size_t>(n) * D + d);
                }
                *reinterpret_cast<uint32_t*>(sc + c * LD + d) = w0;
                *reinterpret_cast<uint32_t*>(se + c * LD + d) = w1;
            }
            __syncthreads();
            float s = 0.f, dp = 0.f;
            for (int d = 0; d < D; ++d) {
                s += sa[warp][d] * __bfloat162float(sc[lane * LD + d]);
                dp += sb[warp][d] * __bfloat162float(se[lane * LD + d]);
            }
            const int n = j * BLK + c0 + lane;
            const bool ok = j >= 0 && n < cols;
            const float2 st = KV ? (ok ? stats[n] : make_float2(INFINITY, 0.f)) : own;
            const float pr = ok ? exp2f(s * g.scale_log2 - st.x) : 0.f;
            const float ds = pr * (dp - st.y);
            for (int c = 0; c < SUB; ++c) {
                const float pc = __shfl_sync(0xffffffffu, pr, c), dc = __shfl_sync(0xffffffffu, ds, c);
#pragma unroll
                for (int y = 0; y < D / 32; ++y) {
                    o1[y] += dc * __bfloat162float(sc[c * LD + y * 32 + lane]);
                    if (KV) o2[y] += pc * __bfloat162float(se[c * LD + y * 32 + lane]);
                }
            }
        }
    }
    auto put = [&](void* base, size_t at, float y) {
        if (p.grad_f32) static_cast<float*>(base)[at] = y;
        else static_cast<__nv_bfloat16*>(base)[at] = __float2bfloat16(y);
    };
    if (r >= rows) return;
    const int tok = !KV && rep ? anchor_token(g, r) : r;
    const int copies = !KV && rep ? anchor_copies(g, r) : 1;
#pragma unroll
    for (int y = 0; y < D / 32; ++y) {
        const size_t at = (static_cast<size_t>(h) * g.N + tok) * D + y * 32 + lane;
        put(KV ? p.dk : p.dq, at, o1[y] * p.scale);
        if (KV) put(p.dv, at, o2[y]);
        // the tokens that only take an anchor's output are no queries of a repeat head
        for (int c = 1; c < copies; ++c) put(p.dq, at + static_cast<size_t>(c) * g.Wl * D, 0.f);
    }
}

}  // namespace calib
