// A paged key/value cache in 8 bits (e4m3) with one scale per block of tokens and head: writing
// new tokens into it, and attention over it.
//
// Cache: k, v [pages, Hkv, B, D] bytes, scales fp32 [pages, Hkv]; a value is its byte times the
// scale of its block and head.  A sequence's block b lives in page table[s, b].
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "ptx.cuh"

namespace calib {

constexpr float kE4m3Max = 448.f;
constexpr float kMinAmax = 7.888609052210118e-31f;        // 2^-100: scale and 1/scale stay normal numbers

// Two packed e4m3 values to half precision (exact: e4m3's values are a subset).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(two));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x2_hi_to_f16x2(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(two));
    return r;
}
// Four floats to e4m3, to nearest even, beyond +-448 to +-448 (NaN stays NaN); `a` in the lowest byte.
__device__ __forceinline__ uint32_t f32x4_to_e4m3(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

// ------------------------------------------------------------------------------------
// writing
// ------------------------------------------------------------------------------------
struct CacheWriteParams {
    const __nv_bfloat16 *k_new, *v_new;   // [S, Hkv, M, D]
    uint8_t *k, *v;                       // [pages, Hkv, B, D]
    float *k_scale, *v_scale;             // [pages, Hkv]
    const int32_t* table;                 // [S, nb]
    const int32_t* lengths;               // [S], the new tokens included
    const int32_t* new_lens;              // [S] or nullptr (M each)
    int S, Hkv, M, nb, pages, T;          // T blocks at most are touched by M tokens
};

constexpr int kWriteThreads = 256;

// One CTA per (sequence, head, touched block, K or V).  The block's new tokens are read once and
// held in registers as bf16; the CTA's largest finite magnitude gives the scale those tokens need,
// max(amax, 2^-100) / 448.  If the block already held tokens its scale only grows, and they are
// then rounded again at the new one (a second rounding, up to half an e4m3 step); if it does not
// grow their bytes stay.  So the largest value of a block is never cut off, and one token costs one
// row, not its block.  Bytes at and behind the sequence's end are left as they were.
// Bound by memory: 2 bytes in and 1 out per value.
template <int D, int B>
__global__ void __launch_bounds__(kWriteThreads) cache_write_kernel(const CacheWriteParams p) {
    constexpr int CPR = D / 8;                             // 8-value chunks per token
    constexpr int PER = B * CPR / kWriteThreads;           // chunks per thread (4 or 8 or 2)
    __shared__ float red[kWriteThreads / 32];
    int x = blockIdx.x;
    const int is_v = x & 1;
    x >>= 1;
    const int t = x % p.T;
    x /= p.T;
    const int h = x % p.Hkv, s = x / p.Hkv;
    const int len = p.lengths[s];
    const int n_new = p.new_lens ? p.new_lens[s] : p.M;
    if (len < 0 || len > static_cast<long long>(p.nb) * B || n_new < 0 || n_new > p.M || n_new > len) {
        if (threadIdx.x == 0) raise_status(STATUS_BAD_CACHE);
        return;
    }
    const int start = len - n_new;                         // first new position
    const int blk = start / B + t;
    if (n_new == 0 || static_cast<long long>(blk) * B >= len) return;
    const int page = p.table[static_cast<size_t>(s) * p.nb + blk];
    if (page < 0 || page >= p.pages) {
        if (threadIdx.x == 0) raise_status(STATUS_BAD_CACHE);
        return;
    }
    const int lo = max(start - blk * B, 0), hi = min(len - blk * B, B);    // new tokens [lo, hi) of the block
    const size_t cell = static_cast<size_t>(page) * p.Hkv + h;
    uint8_t* data = (is_v ? p.v : p.k) + cell * B * D;
    float* scale_at = (is_v ? p.v_scale : p.k_scale) + cell;
    const __nv_bfloat16* src = (is_v ? p.v_new : p.k_new) +
                               (static_cast<size_t>(s) * p.Hkv + h) * p.M * D +
                               (static_cast<long long>(blk) * B - start) * D;   // token 0 of the block, if it were new
    uint4 raw[PER];
    float amax = 0.f;
#pragma unroll
    for (int c = 0; c < PER; ++c) {
        const int idx = static_cast<int>(threadIdx.x) + c * kWriteThreads;
        const int tok = idx / CPR;
        raw[c] = make_uint4(0, 0, 0, 0);
        if (tok >= lo && tok < hi) raw[c] = *reinterpret_cast<const uint4*>(src + static_cast<long long>(tok) * D + idx % CPR * 8);
        const uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float a = fabsf(__uint_as_float(w[e] << 16)), b = fabsf(__uint_as_float(w[e] & 0xFFFF0000u));
            amax = fmaxf(amax, a < INFINITY ? a : 0.f);    // a NaN compares false
            amax = fmaxf(amax, b < INFINITY ? b : 0.f);
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    const float held = lo > 0 ? *scale_at : 0.f;
    if (lane_id() == 0) red[warp_id()] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWriteThreads / 32; ++w) amax = fmaxf(amax, red[w]);
    const float scale = fmaxf(fmaxf(amax, kMinAmax) / kE4m3Max, held);
    const float inv = 1.f / scale;
#pragma unroll
    for (int c = 0; c < PER; ++c) {
        const int idx = static_cast<int>(threadIdx.x) + c * kWriteThreads;
        const int tok = idx / CPR;
        if (tok < lo || tok >= hi) continue;
        const uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
        float f[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f[2 * e] = __uint_as_float(w[e] << 16) * inv;
            f[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u) * inv;
        }
        *reinterpret_cast<uint2*>(data + static_cast<size_t>(tok) * D + idx % CPR * 8) =
            make_uint2(f32x4_to_e4m3(f[0], f[1], f[2], f[3]), f32x4_to_e4m3(f[4], f[5], f[6], f[7]));
    }
    if (scale > held && lo > 0) {
        const float ratio = held * inv;
        for (int idx = threadIdx.x; idx < lo * (D / 16); idx += kWriteThreads) {
            uint4* at = reinterpret_cast<uint4*>(data) + idx;
            const uint4 old = *at;
            const uint32_t w[4] = {old.x, old.y, old.z, old.w};
            uint32_t y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t a = e4m3x2_to_f16x2(w[e]), b = e4m3x2_hi_to_f16x2(w[e]);
                const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&a));
                const float2 fb = __half22float2(*reinterpret_cast<const __half2*>(&b));
                y[e] = f32x4_to_e4m3(fa.x * ratio, fa.y * ratio, fb.x * ratio, fb.y * ratio);
            }
            *at = make_uint4(y[0], y[1], y[2], y[3]);
        }
    }
    // every thread read `held` before the barrier above
    if (threadIdx.x == 0) *scale_at = scale;
}

// ------------------------------------------------------------------------------------
// attention
// ------------------------------------------------------------------------------------
struct CachedParams {
    const __nv_bfloat16* q;               // [S, Hq, M, D]
    const float *k_scale, *v_scale;       // [pages, Hkv]
    const int32_t* table;                 // [S, nb]
    const int32_t* lengths;               // [S]
    const int32_t* new_lens;              // [S] or nullptr
    const int32_t* row_ptr;               // skip list [Hkv * S + 1] or nullptr
    const int16_t* col_idx;
    void* o;                              // [S, Hq, M, D] bf16 or fp32
    float* lse;                           // [S, Hq, M] or nullptr
    float* part_o;                        // workspace [rows][splits][D]
    float2* part_ml;                      // workspace [rows][splits]
    int S, Hq, Hkv, G, M, nb, pages, tiles, splits, causal, out_f32;
    float scale_log2;
    uint64_t timeout_ns;
};

constexpr int kCachedWarps = 8;
constexpr int kCachedThreads = 32 * kCachedWarps;
constexpr int kChunk = 32;                // keys per warp and step
constexpr float kPShift = 15.f;           // P is held as 2^(x - m + 15) <= 2^15

template <int D>
struct CachedSmem {
    static constexpr int STAGES = 3;
    static constexpr uint32_t TILE = kChunk * D;                       // one K or V chunk, bytes
    static constexpr uint32_t RING = kCachedWarps * STAGES * 2 * TILE;
    static constexpr uint32_t OFF_BAR = RING;
    static constexpr uint32_t OFF_ML = OFF_BAR + kCachedWarps * STAGES * 8;   // float2 [warps][16]
    static constexpr uint32_t OFF_MISC = OFF_ML + kCachedWarps * 16 * 8;
    static constexpr uint32_t BYTES = OFF_MISC + 16 + 1024;
    static_assert(RING >= kCachedWarps * 16 * D * 4, "the warps' results are merged in the ring");
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
            "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// Weight of a part with maximum m_part in a row with maximum m.  Parts without keys have m_part =
// -inf and l = 0; a NaN logit leaves l NaN, and it stays NaN here.
__device__ __forceinline__ float merge_weight(float m_part, float m) { return m == -INFINITY ? 1.f : ex2_approx(m_part - m); }
// Natural-log LSE of a row from its maximum and its sum of 2^(x - m + kPShift); -inf without keys.
__device__ __forceinline__ float row_lse(float m, float l) {
    return l == 0.f ? -INFINITY : (m - kPShift + log2f(l)) * 0.69314718055994530942f;
}

// Attention of a few query rows over a sequence's cached keys: the G query heads of a K/V head
// times M query tokens are the rows, 8 * NT of them per CTA.
//
// What bounds it is reading the cache once: 2 D bytes per key and K/V head.  So a CTA's 8 warps
// each stream their own 32-key chunks through a 3-deep ring of TMA tiles (24 chunks, up to 192 KB
// in flight or in use per SM) and meet only at the end.  Rows are few, so they are the N of the
// products and the keys their M: S^T = K Q^T and O^T = V^T P^T as 16x8x16 MMAs, which wastes
// nothing at 8 rows where rows as M would fill half of a tile.  (A tcgen05 tile has 128 rows in
// M; with keys there it would need the 8-bit operands rewritten as 16-bit ones in shared memory
// first.)
//   - e4m3 is exact in half precision.  Q is scaled by a power of two per row so that its largest
//     value is in [2^14, 2^15): bf16's 8 bits fit half's 11, and values down to 2^-30 of the
//     largest stay exact.  P is kept as 2^(x - m + 15), so that half precision holds weights down
//     to 2^-39 of the largest; its rounding (2^-12 relative) is to nearest and has no bias.
//   - A tile row of K is read in an order of d that gives a thread 16 contiguous bytes, the same
//     order for Q; a column of V^T likewise, so a thread ends up with 16 contiguous values of O.
//   - P^T leaves the first product as rows of keys and enters the second as columns: two 8x8
//     transposes in registers.
//   - Each chunk's product goes to its own accumulator, and O = O 2^(m_old - m) + scale_v O_chunk
//     joins it: the softmax's rescaling and the block's scale in one fused multiply-add.
// Shared memory tiles are swizzled by TMA; keys are assigned to MMA rows (a odd: a ^ 4) so that
// both K's and V's reads touch each bank once.
template <int D, int B, int NT>
__global__ void __launch_bounds__(kCachedThreads) cached_attn_kernel(const __grid_constant__ CUtensorMap tm_k,
                                                                     const __grid_constant__ CUtensorMap tm_v,
                                                                     const CachedParams p) {
    using L = CachedSmem<D>;
    constexpr int ST = L::STAGES, KS = D / 16, MT = D / 16, RW = 8 * NT;
    constexpr int CPB = B / kChunk;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC);
    const int warp = static_cast<int>(warp_id()), lane = static_cast<int>(lane_id());
    const int a8 = lane >> 2, t4 = lane & 3;
    const uint32_t ring = smem_u32(smem) + warp * ST * 2 * L::TILE;
    const uint32_t bars = smem_u32(smem + L::OFF_BAR) + warp * ST * 8;

    // ---- the CTA's rows and keys ------------------------------------------------
    int x = blockIdx.x;
    const int split = x % p.splits;
    x /= p.splits;
    const int tile = x % p.tiles;
    x /= p.tiles;
    const int h = x % p.Hkv, s = x / p.Hkv;
    const int rows = p.G * p.M;
    const int row0 = tile * RW;
    int len = p.lengths[s];
    int n_new = p.new_lens ? p.new_lens[s] : p.M;
    if (len < 0 || len > static_cast<long long>(p.nb) * B || n_new < 0 || n_new > p.M || n_new > len) {
        if (threadIdx.x == 0) raise_status(STATUS_BAD_CACHE);
        len = n_new = 0;
    }
    int nblk = (len + B - 1) / B, list0 = 0;
    if (p.row_ptr) {
        const int r = h * p.S + s;
        list0 = p.row_ptr[r];
        const int n = p.row_ptr[r + 1] - list0;
        if (list0 < 0 || n < 0 || n > p.nb) {
            if (threadIdx.x == 0) raise_status(STATUS_BAD_LIST);
            nblk = 0;
        } else if (nblk > 0) {
            nblk = n;
        }
    }
    const int n_chunks = nblk * CPB;
    const int c_beg = static_cast<int>(static_cast<long long>(n_chunks) * split / p.splits);
    const int c_end = static_cast<int>(static_cast<long long>(n_chunks) * (split + 1) / p.splits);

    if (threadIdx.x == 0) *abort_flag = 0;
    if (lane == 0) {
        for (int i = 0; i < ST; ++i) mbar_init(bars + 8 * i, 1);
        fence_barrier_init();
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    __syncthreads();
    const WaitCtl ctl{abort_flag, p.timeout_ns};

    // chunks c_beg + warp, + 8, ...: 32 of them at a time are looked up, one per lane
    const int first = c_beg + warp;
    const int mine = c_end > first ? (c_end - first + kCachedWarps - 1) / kCachedWarps : 0;
    int look_y = -1, look_key = 0;
    float look_ks = 0.f, look_vs = 0.f;
    auto look_up = [&](int n0) {                            // steps n0 .. n0 + 31
        const int n = n0 + lane;
        look_y = -1;
        if (n < mine) {
            const int c = first + n * kCachedWarps;
            int blk = c / CPB;
            if (p.row_ptr) blk = p.col_idx[list0 + blk];
            look_key = blk * B + c % CPB * kChunk;
            if (blk >= 0 && look_key < len) {
                const int page = p.table[static_cast<size_t>(s) * p.nb + blk];
                if (page >= 0 && page < p.pages) {
                    const int cell = page * p.Hkv + h;
                    look_y = cell * B + c % CPB * kChunk;
                    look_ks = p.k_scale[cell];
                    look_vs = p.v_scale[cell];
                } else {
                    raise_status(STATUS_BAD_CACHE);
                }
            }
        }
    };
    // A chunk without keys (past the sequence, or its page unusable) has y = -1: not loaded.
    auto issue = [&](int n, int y) {
        if (y >= 0 && lane == 0) {
            const int st = n % ST;
            mbar_arrive_expect_tx(bars + 8 * st, 2 * L::TILE);
            tma_load_2d(ring + st * 2 * L::TILE, &tm_k, bars + 8 * st, 0, y);
            tma_load_2d(ring + st * 2 * L::TILE + L::TILE, &tm_v, bars + 8 * st, 0, y);
        }
    };
    // each step's place in the cache, first key and scales are passed along as it moves from being
    // issued to being used
    int y_q[ST] = {}, key_q[ST] = {};
    float ks_q[ST] = {}, vs_q[ST] = {};
    uint32_t phase = 0;                                     // bit st: parity of stage st's next wait

    auto fetch = [&](int n, int slot) {                     // look up (from registers) and issue step n
        if ((n & 31) == 0) look_up(n);
        y_q[slot] = __shfl_sync(0xffffffffu, look_y, n & 31);
        key_q[slot] = __shfl_sync(0xffffffffu, look_key, n & 31);
        ks_q[slot] = __shfl_sync(0xffffffffu, look_ks, n & 31);
        vs_q[slot] = __shfl_sync(0xffffffffu, look_vs, n & 31);
        issue(n, y_q[slot]);
    };
#pragma unroll
    for (int n = 0; n < ST - 1; ++n) {
        if (n < mine) fetch(n, n);
    }

    // ---- Q: rows a8 + 8 nt, scaled by a power of two, as the B operand -----------
    uint32_t qf[NT][KS][2];
    float fac[NT][2];                                       // scale_log2 / that power, for rows 2 t4, 2 t4 + 1
    int limit[NT][2];                                       // keys those rows may see
    int lim_min = len;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = row0 + nt * 8 + a8;
        uint4 w[D / 64][2];
        float amax = 0.f;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                w[c][e] = make_uint4(0, 0, 0, 0);
                if (r < rows)
                    w[c][e] = *reinterpret_cast<const uint4*>(
                        p.q + ((static_cast<size_t>(s) * p.Hq + static_cast<size_t>(h) * p.G) * p.M + r) * D + c * 64 +
                        t4 * 16 + e * 8);
                const uint32_t u[4] = {w[c][e].x, w[c][e].y, w[c][e].z, w[c][e].w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(u[i] << 16)), fabsf(__uint_as_float(u[i] & 0xFFFF0000u))));
            }
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // exponent field of the largest: 2^(e - 127) <= amax < 2^(e - 126)
        const int ef = max(15, min(254, static_cast<int>(__float_as_uint(amax) >> 23)));
        const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - (ef - 127)) << 23);   // 2^(14 - (ef - 127))
        const float down = __uint_as_float(static_cast<uint32_t>(max(1, 127 - 14 + (ef - 127))) << 23);
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t u[4] = {w[c][e].x, w[c][e].y, w[c][e].z, w[c][e].w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    qf[nt][c * 4 + e * 2 + i / 2][i & 1] =
                        pack_f16x2(__uint_as_float(u[i] << 16) * up, __uint_as_float(u[i] & 0xFFFF0000u) * up);
            }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            fac[nt][e] = __shfl_sync(0xffffffffu, down, (2 * t4 + e) * 4) * p.scale_log2;
            const int rr = row0 + nt * 8 + 2 * t4 + e;
            const int m = rr % p.M;
            limit[nt][e] = rr < rows && m < n_new ? (p.causal ? len - n_new + m + 1 : len) : 0;
            lim_min = min(lim_min, limit[nt][e]);
        }
    }
    lim_min = __reduce_min_sync(0xffffffffu, lim_min);

    float o[NT][MT][4], m_run[NT][2], l_run[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nt][mt][e] = 0.f;
        m_run[nt][0] = m_run[nt][1] = -INFINITY;
        l_run[nt][0] = l_run[nt][1] = 0.f;
    }

    const int rho = (a8 & 1) ? a8 ^ 4 : a8;                 // key of MMA row a8 (and + 8)
    const int vk0 = 2 * t4, vk1 = (2 * t4 + 1) ^ 4;         // keys of MMA rows 2 t4, 2 t4 + 1
    int slot = 0;
    bool ok = true;
    for (int n = 0; n < mine; ++n) {
        const int y = y_q[0], key0 = key_q[0];
        const float ks = ks_q[0], vs = vs_q[0];
#pragma unroll
        for (int i = 0; i + 1 < ST; ++i) {
            y_q[i] = y_q[i + 1];
            key_q[i] = key_q[i + 1];
            ks_q[i] = ks_q[i + 1];
            vs_q[i] = vs_q[i + 1];
        }
        // the stage read in the previous step is free: every lane has its values in registers
        __syncwarp();
        if (n + ST - 1 < mine) fetch(n + ST - 1, ST - 2);
        const int st = slot;
        slot = slot + 1 == ST ? 0 : slot + 1;
        if (y < 0) continue;
        ok = mbar_wait_warp(bars + 8 * st, (phase >> st) & 1u, ctl);
        if (!ok) break;
        phase ^= 1u << st;
        const uint32_t kt = ring + st * 2 * L::TILE, vt = kt + L::TILE;

        // S^T = K Q^T, two 16-key tiles
        float sc[2][NT][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[i][nt][e] = 0.f;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                const int r0 = i * 16 + rho, r1 = r0 + 8;
                uint4 k0, k1;
                if constexpr (D == 128) {
                    k0 = lds128(kt + r0 * 128 + (((c * 4 + t4) ^ (r0 & 7)) << 4));
                    k1 = lds128(kt + r1 * 128 + (((c * 4 + t4) ^ (r1 & 7)) << 4));
                } else {
                    k0 = lds128(kt + r0 * 64 + ((t4 ^ ((r0 >> 1) & 3)) << 4));
                    k1 = lds128(kt + r1 * 64 + ((t4 ^ ((r1 >> 1) & 3)) << 4));
                }
                const uint32_t u0[4] = {k0.x, k0.y, k0.z, k0.w}, u1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const uint32_t a0 = e4m3x2_to_f16x2(u0[kk]), a2 = e4m3x2_hi_to_f16x2(u0[kk]);
                    const uint32_t a1 = e4m3x2_to_f16x2(u1[kk]), a3 = e4m3x2_hi_to_f16x2(u1[kk]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_f16(sc[i][nt], a0, a1, a2, a3, qf[nt][c * 4 + kk][0], qf[nt][c * 4 + kk][1]);
                }
            }
        }
        // log2-domain logits, masks, running maximum
        uint32_t pf[2][NT][2];
        float alpha[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float f0 = fac[nt][0] * ks, f1 = fac[nt][1] * ks;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                sc[i][nt][0] *= f0;
                sc[i][nt][1] *= f1;
                sc[i][nt][2] *= f0;
                sc[i][nt][3] *= f1;
            }
            if (key0 + kChunk > lim_min) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (key0 + i * 16 + rho + (e >> 1) * 8 >= limit[nt][e & 1]) sc[i][nt][e] = -INFINITY;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mx = fmaxf(fmaxf(sc[0][nt][e], sc[0][nt][e + 2]), fmaxf(sc[1][nt][e], sc[1][nt][e + 2]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                const float m_new = fmaxf(m_run[nt][e], mx);
                const float ref = m_new == -INFINITY ? 0.f : m_new - kPShift;
                alpha[nt][e] = ex2_approx(m_run[nt][e] - (m_new == -INFINITY ? 0.f : m_new));
                m_run[nt][e] = m_new;
                float add = 0.f;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    sc[i][nt][e] = ex2_approx(sc[i][nt][e] - ref);
                    sc[i][nt][e + 2] = ex2_approx(sc[i][nt][e + 2] - ref);
                    add += sc[i][nt][e] + sc[i][nt][e + 2];
                }
                l_run[nt][e] = l_run[nt][e] * alpha[nt][e] + add;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                pf[i][nt][0] = transpose_8x8(pack_f16x2(sc[i][nt][0], sc[i][nt][1]));
                pf[i][nt][1] = transpose_8x8(pack_f16x2(sc[i][nt][2], sc[i][nt][3]));
            }
        }
        // O^T of this chunk = V^T P^T
        float oc[NT][MT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) oc[nt][mt][e] = 0.f;
        const bool tail = key0 + kChunk > len;              // bytes behind the sequence can be anything
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t u[4][D / 32];
#pragma unroll
            for (int kx = 0; kx < 4; ++kx) {
                const int r = i * 16 + (kx & 1 ? vk1 : vk0) + (kx >> 1) * 8;
                if constexpr (D == 128) {
                    const uint4 w = lds128(vt + r * 128 + ((a8 ^ (r & 7)) << 4));
                    u[kx][0] = w.x; u[kx][1] = w.y; u[kx][2] = w.z; u[kx][3] = w.w;
                } else {
                    const uint2 w = lds64(vt + r * 64 + (((a8 >> 1) ^ ((r >> 1) & 3)) << 4) + (a8 & 1) * 8);
                    u[kx][0] = w.x; u[kx][1] = w.y;
                }
                if (tail && key0 + r >= len) {
#pragma unroll
                    for (int e = 0; e < D / 32; ++e) u[kx][e] = 0u;
                }
            }
#pragma unroll
            for (int e = 0; e < D / 32; ++e) {
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const uint32_t x0 = __byte_perm(u[0][e], u[1][e], hf ? 0x7362 : 0x5140);
                    const uint32_t x1 = __byte_perm(u[2][e], u[3][e], hf ? 0x7362 : 0x5140);
                    const uint32_t a0 = e4m3x2_to_f16x2(x0), a1 = e4m3x2_hi_to_f16x2(x0);
                    const uint32_t a2 = e4m3x2_to_f16x2(x1), a3 = e4m3x2_hi_to_f16x2(x1);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_f16(oc[nt][e * 2 + hf], a0, a1, a2, a3, pf[i][nt][0], pf[i][nt][1]);
                }
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nt][mt][e] = o[nt][mt][e] * alpha[nt][e & 1] + oc[nt][mt][e] * vs;
    }

    // ---- the warps' results meet in shared memory -------------------------------
    if (!ok && lane == 0) {                                 // copies still in flight end before the ring is reused
#pragma unroll
        for (int i = 0; i < ST; ++i) mbar_wait_drain(bars + 8 * i, (phase >> i) & 1u, 10000000ull);
    }
    __syncthreads();
    float* so = reinterpret_cast<float*>(smem);             // [warps][RW][D]
    float2* sml = reinterpret_cast<float2*>(smem + L::OFF_ML);   // [warps][16]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float l = l_run[nt][e];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            const int r = nt * 8 + 2 * t4 + e;
            if (a8 == 0) sml[warp * 16 + r] = make_float2(m_run[nt][e], l);
            float* to = so + (static_cast<size_t>(warp) * RW + r) * D + a8 * (D / 8);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
                *reinterpret_cast<float2*>(to + mt * 2) = make_float2(o[nt][mt][e], o[nt][mt][e + 2]);
        }
    }
    __syncthreads();
    if (*abort_flag) return;
    for (int idx = threadIdx.x; idx < RW * (D / 4); idx += kCachedThreads) {
        const int r = idx / (D / 4), d = idx % (D / 4) * 4;
        if (row0 + r >= rows) break;
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < kCachedWarps; ++w) m = fmaxf(m, sml[w * 16 + r].x);
        float l = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kCachedWarps; ++w) {
            const float2 ml = sml[w * 16 + r];
            const float f = merge_weight(ml.x, m);
            l += ml.y * f;
            const float4 y = *reinterpret_cast<const float4*>(so + (static_cast<size_t>(w) * RW + r) * D + d);
            acc.x += y.x * f;
            acc.y += y.y * f;
            acc.z += y.z * f;
            acc.w += y.w * f;
        }
        const size_t row = (static_cast<size_t>(s) * p.Hq + static_cast<size_t>(h) * p.G) * p.M + row0 + r;
        if (p.splits > 1) {
            *reinterpret_cast<float4*>(p.part_o + (row * p.splits + split) * D + d) = acc;
            if (d == 0) p.part_ml[row * p.splits + split] = make_float2(m, l);
            continue;
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        if (p.out_f32)
            *reinterpret_cast<float4*>(static_cast<float*>(p.o) + row * D + d) =
                make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        else
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + row * D + d) =
                make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        if (d == 0 && p.lse) p.lse[row] = row_lse(m, l);
    }
}

// Joins the splits of a row, one warp per row, in split order.
template <int D>
__global__ void __launch_bounds__(128) cached_combine_kernel(const CachedParams p, long long rows) {
    const long long row = static_cast<long long>(blockIdx.x) * 4 + warp_id();
    if (row >= rows) return;
    const int lane = static_cast<int>(lane_id());
    const float2* ml = p.part_ml + row * p.splits;
    float m = -INFINITY;
    for (int i = lane; i < p.splits; i += 32) m = fmaxf(m, ml[i].x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    constexpr int PER = D / 32;
    float acc[PER], l = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] = 0.f;
    for (int i = 0; i < p.splits; ++i) {
        const float2 y = ml[i];
        const float f = merge_weight(y.x, m);
        l += y.y * f;
        const float* src = p.part_o + (row * p.splits + i) * D + lane * PER;
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[e] += src[e] * f;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < PER; e += 2) {
        const size_t at = static_cast<size_t>(row) * D + lane * PER + e;
        if (p.out_f32) *reinterpret_cast<float2*>(static_cast<float*>(p.o) + at) = make_float2(acc[e] * inv, acc[e + 1] * inv);
        else *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.o) + at) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
    }
    if (lane == 0 && p.lse) p.lse[row] = row_lse(m, l);
}

}  // namespace calib
