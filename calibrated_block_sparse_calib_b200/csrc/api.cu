// C ABI of libcalibatt.so (declared in include/calibatt.h): argument validation, TMA
// descriptor encoding, and kernel launches.  The library allocates no device memory;
// its only state is the per-device status word in ptx.cuh and a few host-side caches
// (the driver entry point, per-device capability and shared-memory attributes).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <type_traits>
#include <cstring>
#include <mutex>
#include <set>
#include <utility>
#include <vector>

#include "calibatt.h"
#include "ptx.cuh"
#include "attn_fwd.cuh"
#include "energy.cuh"
#include "select.cuh"
#include "intervals.cuh"
#include "repeat_sim.cuh"
#include "transpose.cuh"
#include "attn_bwd.cuh"
#include "kv_cache.cuh"
#include "kv_cache_wide.cuh"

namespace {

constexpr int kSms = 148;
constexpr uint64_t kDefaultTimeoutNs = 4000000000ull;   // bounded device waits: 4 s

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
int cdiv(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }

cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

// sm_100 check, cached per device.  A thread that has made no CUDA call yet (autograd's, on its first backward pass) has
// no context, which the driver's tensor-map encoder needs: setting the device it is on anyway gives it one.
calib_status check_device() {
    static std::mutex mu;
    static std::set<int> ok_devices;
    static thread_local int bound = -1;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return CALIB_ERR_CUDA;
    if (bound != dev) {
        if (cudaSetDevice(dev) != cudaSuccess) return CALIB_ERR_CUDA;
        bound = dev;
    }
    std::lock_guard<std::mutex> lk(mu);
    if (ok_devices.count(dev)) return CALIB_OK;
    int major = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess)
        return CALIB_ERR_CUDA;
    if (major != 10) return CALIB_ERR_UNSUPPORTED;
    ok_devices.insert(dev);
    return CALIB_OK;
}

// Raise a kernel's dynamic shared-memory limit once per (kernel, device).
calib_status ensure_smem(const void* fn, int bytes) {
    static std::mutex mu;
    static std::set<std::pair<const void*, int>> done;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return CALIB_ERR_CUDA;
    std::lock_guard<std::mutex> lk(mu);
    if (done.count({fn, dev})) return CALIB_OK;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return CALIB_ERR_CUDA;
    done.insert({fn, dev});
    return CALIB_OK;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                   CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                   CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// 3-D bf16 view [H][N][D] of a contiguous tensor; box = 64 elements (128 B, the swizzle
// span) x box_rows x 1, 128-byte swizzle, zero fill out of bounds.
bool make_tmap(CUtensorMap* map, const void* base, int D, int N, int H, int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(N),
                                static_cast<cuuint64_t>(H)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(N) * D * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One launch with what a <<<>>> launch cannot say: a cluster size, or (overlap) that the kernel may begin while
// the stream's previous kernel ends; it then waits itself before it reads that one's results.
template <class... P, class... A>
calib_status launch_with(void (*fn)(P...), int grid, int threads, int smem, cudaStream_t st, int cluster, bool overlap,
                         const A&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = cluster;
        attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (overlap) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, fn, args...) == cudaSuccess ? CALIB_OK : (cudaGetLastError(), CALIB_ERR_CUDA);
}

calib_status launch_status() {
    return cudaGetLastError() == cudaSuccess ? CALIB_OK : CALIB_ERR_CUDA;
}

// ---- attention ---------------------------------------------------------------------
// A validated attention call: parameters and tensor maps (K, V, and Q as whole blocks and
// as single rows for gathered anchor rows), launchable in slices of the work list.
struct AttnCall {
    calib::AttnParams p;
    CUtensorMap tk, tv, tq, tq1;
    int D, B, grid;
};

template <int D, int BLK, bool WITH_LSE>
calib_status launch_attn(const AttnCall& c, const calib::AttnParams& p, int grid, cudaStream_t st) {
    constexpr int KST = 3, VST = 2;   // K / V ring depths (with the Q tile, 200 KB at D = B = 128)
    using L = calib::AttnSmem<D, BLK, KST, VST>;
    static_assert(L::BYTES <= 232448, "shared memory budget");
    auto* fn = calib::attn_fwd_kernel<D, BLK, KST, VST, WITH_LSE>;
    if (calib_status s = ensure_smem(reinterpret_cast<const void*>(fn), L::BYTES)) return s;
    fn<<<grid, calib::kAttnThreads, L::BYTES, st>>>(c.tk, c.tv, c.tq, c.tq1, p);
    return launch_status();
}

template <int D, int BLK>
calib_status launch_attn_lse(const AttnCall& c, const calib::AttnParams& p, int grid, cudaStream_t st) {
    return p.lse ? launch_attn<D, BLK, true>(c, p, grid, st) : launch_attn<D, BLK, false>(c, p, grid, st);
}

calib_status attn_prepare(const void* q, const void* k, const void* v, void* o, float* lse, int H, int N,
                          int D, float scale, const calib_block_list* list, const uint32_t* repeat_bits,
                          int F, int Hl, int Wl, int n_text, int stride, uint32_t flags, AttnCall* c) {
    if (!q || !k || !v || !o || !list || !list->row_ptr || !list->col_idx) return CALIB_ERR_INVALID;
    if (flags & ~CALIB_ATTN_OUT_F32) return CALIB_ERR_INVALID;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return CALIB_ERR_INVALID;
    if (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)) return CALIB_ERR_INVALID;
    if (H < 1 || N < 1 || !(scale > 0.f) || !std::isfinite(scale)) return CALIB_ERR_INVALID;
    if (H > 1024 || static_cast<long long>(H) * N * D >= (1ll << 40)) return CALIB_ERR_INVALID;
    const int B = list->block;
    if (B != 64 && B != 128) return CALIB_ERR_INVALID;
    if (D != 64 && D != 128) return CALIB_ERR_UNSUPPORTED;
    const int nb = cdiv(N, B);
    if (list->H != H || list->nq != nb || list->nk != nb || nb > 32767 || H > 32767) return CALIB_ERR_INVALID;
    if (list->work && list->n_work < 0) return CALIB_ERR_INVALID;
    if (calib_status s = check_device()) return s;

    calib::AttnParams& p = c->p;
    p = calib::AttnParams{};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    p.row_ptr = list->row_ptr;
    p.col_idx = list->col_idx;
    p.work = list->work;
    p.H = H; p.N = N; p.nq = nb; p.nk = nb;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.F = F; p.Hl = Hl; p.Wl = Wl; p.n_text = n_text; p.stride = stride;
    p.Ar = stride > 0 ? (Hl + stride - 1) / stride : 0;
    p.n_anchor = F * p.Ar * Wl + n_text;
    p.nq_anchor = cdiv(p.n_anchor, B);
    for (int w = 0; w < 32; ++w) p.repeat_bits[w] = repeat_bits ? repeat_bits[w] : 0u;
    p.out_f32 = (flags & CALIB_ATTN_OUT_F32) ? 1 : 0;
    p.timeout_ns = kDefaultTimeoutNs;
    c->D = D;
    c->B = B;
    c->grid = list->work ? list->n_work : H * nb;
    if (!make_tmap(&c->tk, k, D, N, H, B) || !make_tmap(&c->tv, v, D, N, H, B) || !make_tmap(&c->tq, q, D, N, H, B))
        return CALIB_ERR_CUDA;
    c->tq1 = c->tq;                 // single rows are gathered for repeat heads only
    if (repeat_bits && !make_tmap(&c->tq1, q, D, N, H, 1)) return CALIB_ERR_CUDA;
    return CALIB_OK;
}

// Launch work items [first, first + count) of a prepared call (items index the work list,
// which must be present unless the slice is the whole grid).
calib_status attn_launch(const AttnCall& c, int first, int count, cudaStream_t st) {
    if (count <= 0) return CALIB_OK;
    calib::AttnParams p = c.p;
    if (p.work) p.work += first;
    else if (first != 0 || count != c.grid) return CALIB_ERR_INVALID;
    if (c.D == 128) return c.B == 128 ? launch_attn_lse<128, 128>(c, p, count, st)
                                      : launch_attn_lse<128, 64>(c, p, count, st);
    return c.B == 128 ? launch_attn_lse<64, 128>(c, p, count, st) : launch_attn_lse<64, 64>(c, p, count, st);
}

calib_status attn_common(const void* q, const void* k, const void* v, void* o, float* lse, int H, int N,
                         int D, float scale, const calib_block_list* list, const uint32_t* repeat_bits,
                         int F, int Hl, int Wl, int n_text, int stride, uint32_t flags, void* stream) {
    AttnCall c;
    if (calib_status s = attn_prepare(q, k, v, o, lse, H, N, D, scale, list, repeat_bits, F, Hl, Wl, n_text,
                                      stride, flags, &c))
        return s;
    return attn_launch(c, 0, c.grid, as_stream(stream));
}

// CUDA events of one call, destroyed on every exit path (a recorded event may be destroyed
// before it completes; its resources are released once it does).
struct EventSet {
    std::vector<cudaEvent_t> ev;
    cudaEvent_t make() {
        cudaEvent_t e = nullptr;
        if (cudaEventCreateWithFlags(&e, cudaEventDisableTiming) != cudaSuccess) return nullptr;
        ev.push_back(e);
        return e;
    }
    ~EventSet() {
        for (cudaEvent_t e : ev) cudaEventDestroy(e);
    }
};

// Host <-> device transfers of a prepared attention call, overlapped with its kernels per
// chunk of heads (see sparse_attn_fwd_host in calibatt.h).
calib_status host_pipeline(const AttnCall& c, const void* q_host, const void* k_host, const void* v_host,
                           void* o_host, void* q_dev, void* k_dev, void* v_dev, const void* o_dev, int H, int N,
                           int D, const calib_block_list* list, uint32_t flags, int heads_per_chunk,
                           void* stream, void* h2d_stream, void* d2h_stream) {
    const int nb = list->nq;
    // Head chunks need the head-major work order (each head's nq items contiguous, as
    // calib_build_schedule writes it); any other list runs as one chunk.
    const bool chunked = list->work && list->n_work == H * nb && heads_per_chunk < H;
    const int hpc = chunked ? heads_per_chunk : H;
    const size_t in_head = static_cast<size_t>(N) * D * 2;
    const size_t out_head = static_cast<size_t>(N) * D * ((flags & CALIB_ATTN_OUT_F32) ? 4 : 2);
    cudaStream_t st = as_stream(stream);
    cudaStream_t sin = h2d_stream ? as_stream(h2d_stream) : st;
    cudaStream_t sout = d2h_stream ? as_stream(d2h_stream) : st;
    EventSet evs;
    cudaEvent_t start = evs.make();
    if (!start || cudaEventRecord(start, st) != cudaSuccess) return CALIB_ERR_CUDA;
    // the copy streams start after the work already queued on the caller's stream
    if (cudaStreamWaitEvent(sin, start, 0) != cudaSuccess || cudaStreamWaitEvent(sout, start, 0) != cudaSuccess)
        return CALIB_ERR_CUDA;
    // The step ends with the last chunk's kernel and copy-back after the last host-to-device
    // copy, so when there are several chunks the last chunk's heads go one per chunk.
    for (int h0 = 0, h1 = 0; h0 < H; h0 = h1) {
        h1 = h0 + hpc < H ? h0 + hpc : H;
        if (h1 == H && h0 > 0) h1 = h0 + 1;
        const size_t off = static_cast<size_t>(h0) * in_head, len = static_cast<size_t>(h1 - h0) * in_head;
        // one copy per tensor and chunk
        if (cudaMemcpyAsync(static_cast<char*>(q_dev) + off, static_cast<const char*>(q_host) + off, len,
                            cudaMemcpyHostToDevice, sin) != cudaSuccess ||
            cudaMemcpyAsync(static_cast<char*>(k_dev) + off, static_cast<const char*>(k_host) + off, len,
                            cudaMemcpyHostToDevice, sin) != cudaSuccess ||
            cudaMemcpyAsync(static_cast<char*>(v_dev) + off, static_cast<const char*>(v_host) + off, len,
                            cudaMemcpyHostToDevice, sin) != cudaSuccess)
            return CALIB_ERR_CUDA;
        cudaEvent_t in_ready = evs.make();
        if (!in_ready || cudaEventRecord(in_ready, sin) != cudaSuccess ||
            cudaStreamWaitEvent(st, in_ready, 0) != cudaSuccess)
            return CALIB_ERR_CUDA;
        const int first = chunked ? h0 * nb : 0, count = chunked ? (h1 - h0) * nb : c.grid;
        if (calib_status s = attn_launch(c, first, count, st)) return s;
        cudaEvent_t out_ready = evs.make();
        if (!out_ready || cudaEventRecord(out_ready, st) != cudaSuccess ||
            cudaStreamWaitEvent(sout, out_ready, 0) != cudaSuccess)
            return CALIB_ERR_CUDA;
        const size_t ooff = static_cast<size_t>(h0) * out_head, olen = static_cast<size_t>(h1 - h0) * out_head;
        if (cudaMemcpyAsync(static_cast<char*>(o_host) + ooff, static_cast<const char*>(o_dev) + ooff, olen,
                            cudaMemcpyDeviceToHost, sout) != cudaSuccess)
            return CALIB_ERR_CUDA;
    }
    // the caller's stream is ordered after the last copy of O
    cudaEvent_t done = evs.make();
    if (!done || cudaEventRecord(done, sout) != cudaSuccess || cudaStreamWaitEvent(st, done, 0) != cudaSuccess)
        return CALIB_ERR_CUDA;
    return CALIB_OK;
}

// Validated repeat geometry: token count N = F*Hl*Wl + n_text and the head bit set.
calib_status repeat_geometry(int H, int F, int Hl, int Wl, int n_text, int stride, const uint8_t* head_repeat,
                             uint32_t* bits, int* N_out) {
    if (!head_repeat || calib_anchor_count(F, Hl, Wl, n_text, stride) < 0 || H < 1 || H > 1024)
        return CALIB_ERR_INVALID;
    const long long N = static_cast<long long>(F) * Hl * Wl + n_text;
    if (N > (1ll << 31) - 1) return CALIB_ERR_INVALID;
    for (int w = 0; w < 32; ++w) bits[w] = 0u;
    for (int h = 0; h < H; ++h)
        if (head_repeat[h]) bits[h >> 5] |= 1u << (h & 31);
    *N_out = static_cast<int>(N);
    return CALIB_OK;
}

// ---- energy ------------------------------------------------------------------------
template <int D, int BLK>
calib_status launch_energy(const CUtensorMap& tk, const calib::EnergyParams& p, int grid, cudaStream_t st) {
    constexpr int KST = 4;
    using L = calib::EnergySmem<D, BLK, KST>;
    static_assert(L::BYTES <= 232448, "shared memory budget");
    auto* fn = calib::block_energy_kernel<D, BLK, KST>;
    if (calib_status s = ensure_smem(reinterpret_cast<const void*>(fn), L::BYTES)) return s;
    fn<<<grid, calib::kEnergyThreads, L::BYTES, st>>>(tk, p);
    return launch_status();
}

// ---- spatial-repetition similarity -----------------------------------------------------
template <int D, int BLK>
calib_status launch_sim(const CUtensorMap& tk, const calib::SimParams& p, int grid, cudaStream_t st) {
    constexpr int KST = 4;
    using L = calib::SimSmem<D, BLK, KST>;
    static_assert(L::BYTES <= 232448, "shared memory budget");
    auto* fn = calib::repeat_sim_kernel<D, BLK, KST>;
    if (calib_status s = ensure_smem(reinterpret_cast<const void*>(fn), L::BYTES)) return s;
    fn<<<grid, calib::kEnergyThreads, L::BYTES, st>>>(tk, p);
    return launch_status();
}

// ---- gradients ---------------------------------------------------------------------
// Workspace of sparse_attn_bwd(_repeat): row statistics over whole blocks, dO as bf16 (fp32 in and
// out only), and the anchors' rows of Q and dO (repeat heads only).
struct BwdSpace {
    size_t ndelta, do16, qa, doa, total;   // nlse is at 0
};
BwdSpace bwd_space(int H, int N, int D, int B, long long n_anchor, bool io_f32) {
    auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
    BwdSpace w{};
    const size_t rows = static_cast<size_t>(cdiv(N, B)) * B;
    w.ndelta = up(H * rows * 4);
    w.do16 = 2 * w.ndelta;
    w.qa = w.do16 + (io_f32 ? up(static_cast<size_t>(H) * N * D * 2) : 0);
    const size_t anchors = n_anchor ? up(static_cast<size_t>(H) * n_anchor * D * 2) : 0;
    w.doa = w.qa + anchors;
    w.total = w.doa + anchors;
    return w;
}

template <int D, int BLK>
calib_status launch_bwd(const calib::BwdMaps& m, const calib::BwdParams& p, cudaStream_t st) {
    // ring depth: what fits beside the two resident tiles (at most 194 KB; 98 KB at D = B = 64, two CTAs an SM)
    constexpr int ST = D == 128 && BLK == 128 ? 2 : 4;
    using L = calib::BwdSmem<D, BLK, ST>;
    static_assert(L::BYTES + 1024 <= 233472 / calib::bwd_ctas(D, BLK), "shared memory budget");
    const int rows = p.geo.nq * BLK;
    const long long threads = static_cast<long long>(p.geo.H) * rows * (D / 8);
    auto* fn = calib::bwd_kernel<D, BLK, ST>;
    if (calib_status s = ensure_smem(reinterpret_cast<const void*>(fn), L::BYTES)) return s;
    calib::bwd_prepare_kernel<D><<<static_cast<int>((threads + 255) / 256), 256, 0, st>>>(p, rows);
    if (calib_status s = launch_status()) return s;
    return launch_with(fn, p.geo.H * (p.geo.nk + p.geo.nq), calib::bwd_threads(BLK), L::BYTES, st, 1, true, m, p);
}

calib_status bwd_common(const void* q, const void* k, const void* v, const void* o, const void* dout,
                        const float* lse, void* dq, void* dk, void* dv, int H, int N, int D, float scale,
                        const calib_block_list* list, const calib_block_list* list_t, const uint32_t* repeat_bits,
                        int F, int Hl, int Wl, int n_text, int stride, uint32_t flags, void* workspace,
                        int64_t workspace_bytes, void* stream) {
    if (!dq || !dk || !dv || !lse || !dout || !workspace || !list_t || !list_t->row_ptr || !list_t->col_idx)
        return CALIB_ERR_INVALID;
    if (flags & ~(CALIB_ATTN_OUT_F32 | CALIB_ATTN_GRAD_F32)) return CALIB_ERR_INVALID;
    for (const void* x : {static_cast<const void*>(dq), static_cast<const void*>(dk), static_cast<const void*>(dv), dout,
                          static_cast<const void*>(workspace)})
        if (!aligned16(x)) return CALIB_ERR_INVALID;
    AttnCall c;
    if (calib_status s = attn_prepare(q, k, v, const_cast<void*>(o), const_cast<float*>(lse), H, N, D, scale, list,
                                      repeat_bits, F, Hl, Wl, n_text, stride, flags & CALIB_ATTN_OUT_F32, &c))
        return s;
    if (list_t->H != H || list_t->nq != list->nk || list_t->nk != list->nq || list_t->block != list->block)
        return CALIB_ERR_INVALID;
    // every row of dq, dk and dv is written: a work order covers all rows
    if ((list->work && list->n_work != H * list->nq) || (list_t->work && list_t->n_work != H * list_t->nq))
        return CALIB_ERR_INVALID;
    const BwdSpace w = bwd_space(H, N, D, c.B, repeat_bits ? c.p.n_anchor : 0, c.p.out_f32);
    if (workspace_bytes < static_cast<int64_t>(w.total)) return CALIB_ERR_INVALID;
    char* base = static_cast<char*>(workspace);
    calib::BwdParams p{};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k = static_cast<const __nv_bfloat16*>(k);
    p.v = static_cast<const __nv_bfloat16*>(v);
    p.o = o;
    p.dout = dout;
    p.lse = lse;
    p.dq = dq; p.dk = dk; p.dv = dv;
    p.nlse = reinterpret_cast<float*>(base);
    p.ndelta = reinterpret_cast<float*>(base + w.ndelta);
    p.io_f32 = c.p.out_f32;
    p.do16 = p.io_f32 ? reinterpret_cast<__nv_bfloat16*>(base + w.do16)
                      : static_cast<__nv_bfloat16*>(const_cast<void*>(dout));
    p.qa = reinterpret_cast<__nv_bfloat16*>(base + w.qa);
    p.doa = reinterpret_cast<__nv_bfloat16*>(base + w.doa);
    p.row_ptr = list->row_ptr; p.col_idx = list->col_idx; p.work = list->work;
    p.t_row_ptr = list_t->row_ptr; p.t_col_idx = list_t->col_idx; p.t_work = list_t->work;
    p.geo = c.p;
    p.scale = scale;
    p.grad_f32 = (flags & CALIB_ATTN_GRAD_F32) ? 1 : 0;
    p.timeout_ns = kDefaultTimeoutNs;
    calib::BwdMaps m;
    m.k = c.tk;
    m.v = c.tv;
    m.q = c.tq;
    if (!make_tmap(&m.dout, p.do16, D, N, H, c.B)) return CALIB_ERR_CUDA;
    m.qa = m.q;
    m.doa = m.dout;
    if (repeat_bits && (!make_tmap(&m.qa, p.qa, D, c.p.n_anchor, H, c.B) ||
                        !make_tmap(&m.doa, p.doa, D, c.p.n_anchor, H, c.B)))
        return CALIB_ERR_CUDA;
    cudaStream_t st = as_stream(stream);
    if (D == 128) return c.B == 128 ? launch_bwd<128, 128>(m, p, st) : launch_bwd<128, 64>(m, p, st);
    return c.B == 128 ? launch_bwd<64, 128>(m, p, st) : launch_bwd<64, 64>(m, p, st);
}

// ---- 8-bit cache -------------------------------------------------------------------
// How a call's work is shared (see cached_attn_kernel): rows per unit (8, 16 or 128), units per K/V head, and `flat`:
// shares per K/V head and row tile, or 0 for a cluster per unit and no second launch.  Clusters where no sequence
// can be longer than 2048 keys (5 to 8 steps for each of a CTA's warps, about what the cut's merge costs), or
// 8192 if the GPU has room for clusters of 8, or where the units fill the GPU 8 times and more; a cluster has one step
// for each of its warps, as far as 8 CTAs and the GPU's places go.  The number of shares is the one that takes the
// fewest steps in all if every sequence is as long as the table allows: rounds of CTAs times a share's steps and 6
// more for its start and end.
//
// cached_wide_kernel takes many query rows.  Its 128 rows cost what 2 tiles of 16 rows (4 at D = 64) cost
// cached_attn_kernel (4 sequences of 65536 keys, 8 K/V heads: 242 against 220 us with 32 rows and 241 against 332 with
// 40 at D = 128; 235 against 236 with 64 at D = 64), and about 10 us more to start and end, which 2^18 keys times tiles
// saved (2^19 at D = 64) make up for: 2 x 1024 keys, 4 heads, 256 rows, 29 against 20 us; 16 x 2048 keys, 8 heads, 40
// rows, 54 against 64.
struct CachedPlan {
    int nt, tiles, flat, cluster;
    long long units, grid;
    int64_t part_o, part_ml, bytes;   // workspace: offsets of the parts and their statistics; `pieces` is at 0
};
CachedPlan cached_plan(int S, int Hq, int Hkv, int M, int D, int B, int nb) {
    CachedPlan c{};
    const long long rows = static_cast<long long>(Hq / Hkv) * M;
    const long long keys = static_cast<long long>(nb) * B;
    const long long saved = cdiv(rows, 16) - (D == 128 ? 2 : 4) * static_cast<long long>(cdiv(rows, calib::kWideRows));
    const bool wide = saved > 0 && static_cast<double>(S) * Hkv * static_cast<double>(keys) * static_cast<double>(saved) >=
                                       (D == 128 ? 262144. : 524288.);
    c.nt = rows <= 8 ? 1 : (wide ? calib::kWideRows / 8 : 2);
    c.tiles = cdiv(rows, 8 * c.nt);
    const long long columns = static_cast<long long>(Hkv) * c.tiles;
    c.units = S * columns;
    c.grid = c.units;
    const long long places = kSms * (D == 128 || wide ? 1 : 2);
    c.cluster = 1;
    if (c.units >= 8 * places || (wide && keys <= 1024)) return c;
    if (!wide && (keys <= 2048 || (keys <= 8192 && c.units * 8 <= places))) {
        const int warps = D == 128 && c.nt == 1 ? 12 : 8;
        while (c.cluster < 8 && c.cluster * warps < keys / calib::kChunk && c.units * c.cluster * 2 <= places) c.cluster *= 2;
        c.grid = c.units * c.cluster;
    } else {
        const long long total = wide ? S * (keys / calib::kWideKeys + calib::kWideCost) : S * (keys / calib::kChunk + calib::kUnitCost);
        const long long warps = wide ? 1 : (D == 128 && c.nt == 1 ? 12 : 8), least = wide ? calib::kWideMinShare : calib::kMinShare;
        double best = 0.;
        for (long long shares = 1; shares <= std::max(1ll, 3 * places / columns) && shares <= std::max(1ll, total / least);
             ++shares) {
            const double cost = static_cast<double>(cdiv(shares * columns, places)) *
                                (static_cast<double>(total) / static_cast<double>(shares * warps) + 6.);
            if (c.flat == 0 || cost < best) {
                c.flat = static_cast<int>(shares);
                best = cost;
            }
        }
        c.grid = c.flat * columns;
        const int64_t slots = 2 * c.grid * 8 * c.nt;
        c.part_o = (c.units * 8 + 15) / 16 * 16;
        c.part_ml = c.part_o + slots * D * 4;
        c.bytes = c.part_ml + slots * 8;
    }
    return c;
}

// Checks shared by the cache calls; S sequences, pages of B tokens, nb entries per row of the table.
calib_status cache_args(const void* k, const void* v, const float* ks, const float* vs, const int32_t* table,
                        const int32_t* lengths, int S, int Hkv, int M, int D, int B, int nb, int64_t pages) {
    if (!k || !v || !ks || !vs || !table || !lengths) return CALIB_ERR_INVALID;
    if (!aligned16(k) || !aligned16(v)) return CALIB_ERR_INVALID;
    for (const void* x : {static_cast<const void*>(ks), static_cast<const void*>(vs), static_cast<const void*>(table),
                          static_cast<const void*>(lengths)})
        if (reinterpret_cast<uintptr_t>(x) & 3u) return CALIB_ERR_INVALID;
    if (S < 1 || Hkv < 1 || M < 1 || nb < 1 || pages < 1) return CALIB_ERR_INVALID;
    if (B != 64 && B != 128) return CALIB_ERR_INVALID;
    if (D != 64 && D != 128) return CALIB_ERR_UNSUPPORTED;
    // token rows of the cache and positions of a sequence are 32-bit numbers
    if (pages > ((1ll << 31) - 1) / B / Hkv || nb > ((1ll << 31) - 1) / B) return CALIB_ERR_UNSUPPORTED;
    if (static_cast<long long>(S) * Hkv * M > (1ll << 31) - 1) return CALIB_ERR_UNSUPPORTED;
    return check_device();
}

// 2-D view [pages * Hkv * B][D] of the cache's bytes; box = 32 tokens, swizzled over a token's row.
bool make_cache_tmap(CUtensorMap* map, const void* base, int D, long long rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(D)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(D), calib::kChunk};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int B, int NT>
calib_status launch_cached(const CUtensorMap& tk, const CUtensorMap& tv, const calib::CachedParams& p,
                           const CachedPlan& c, cudaStream_t st) {
    using L = calib::CachedSmem<D, NT>;
    static_assert(L::BYTES <= 232448 / L::CTAS - (L::CTAS > 1 ? 1024 : 0), "shared memory budget");
    auto* fn = calib::cached_attn_kernel<D, B, NT>;
    if (calib_status s = ensure_smem(reinterpret_cast<const void*>(fn), L::BYTES)) return s;
    if (calib_status s = launch_with(fn, static_cast<int>(c.grid), L::THREADS, L::BYTES, st, p.cluster, false, tk, tv, p))
        return s;
    if (!p.flat) return CALIB_OK;
    return launch_with(calib::cached_combine_kernel<D, NT>, static_cast<int>(c.units) * NT, 256, 0, st, 1, true, p);
}

template <int D, int B>
calib_status launch_wide(const CUtensorMap& tk, const CUtensorMap& tv, const calib::CachedParams& p, const CachedPlan& c,
                         cudaStream_t st) {
    using L = calib::WideSmem<D>;
    static_assert(L::BYTES <= 232448, "shared memory budget");
    auto* fn = calib::cached_wide_kernel<D, B>;
    if (calib_status s = ensure_smem(reinterpret_cast<const void*>(fn), L::BYTES)) return s;
    // the split of the registers waits for ones that the launch does not bring along
    static std::atomic<bool> enough{false};
    if (!enough) {
        cudaFuncAttributes a{};
        if (cudaFuncGetAttributes(&a, fn) != cudaSuccess || a.numRegs != calib::kWideRegs) return CALIB_ERR_CUDA;
        enough = true;
    }
    if (calib_status s = launch_with(fn, static_cast<int>(c.grid), calib::kWideThreads, L::BYTES, st, 1, false, tk, tv, p))
        return s;
    if (!p.flat) return CALIB_OK;
    constexpr int NT = calib::kWideRows / 8;
    return launch_with(calib::cached_combine_kernel<D, NT>, static_cast<int>(c.units) * NT, 256, 0, st, 1, true, p);
}

template <int D, int B>
calib_status launch_cached_nt(const CUtensorMap& tk, const CUtensorMap& tv, const calib::CachedParams& p,
                              const CachedPlan& c, cudaStream_t st) {
    if (c.nt > 2) return launch_wide<D, B>(tk, tv, p, c, st);
    return c.nt == 1 ? launch_cached<D, B, 1>(tk, tv, p, c, st) : launch_cached<D, B, 2>(tk, tv, p, c, st);
}

template <int D, int B>
calib_status launch_write(const calib::CacheWriteParams& p, int grid, cudaStream_t st) {
    calib::cache_write_kernel<D, B><<<grid, calib::kWriteThreads, 0, st>>>(p);
    return launch_status();
}

int rows_grid(long long rows) { return static_cast<int>((rows + 3) / 4); }   // 4 warps per block

}  // namespace

extern "C" {

const char* calib_status_string(calib_status s) {
    switch (s) {
        case CALIB_OK: return "CALIB_OK";
        case CALIB_ERR_INVALID: return "CALIB_ERR_INVALID";
        case CALIB_ERR_UNSUPPORTED: return "CALIB_ERR_UNSUPPORTED";
        case CALIB_ERR_CUDA: return "CALIB_ERR_CUDA";
        case CALIB_ERR_TIMEOUT: return "CALIB_ERR_TIMEOUT";
    }
    return "CALIB_ERR_UNKNOWN";
}

calib_status calib_device_check(void* stream) {
    if (cudaStreamSynchronize(as_stream(stream)) != cudaSuccess) return CALIB_ERR_CUDA;
    uint32_t v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, calib::g_status, sizeof(v)) != cudaSuccess) return CALIB_ERR_CUDA;
    if (v && cudaMemcpyToSymbol(calib::g_status, &zero, sizeof(zero)) != cudaSuccess) return CALIB_ERR_CUDA;
    if (v & calib::STATUS_TIMEOUT) return CALIB_ERR_TIMEOUT;
    if (v & (calib::STATUS_BAD_ENERGY | calib::STATUS_BAD_LIST | calib::STATUS_BAD_CACHE)) return CALIB_ERR_INVALID;
    return CALIB_OK;
}

calib_status calib_block_energy(const void* q, const void* k, const float* lse, int H, int N, int D, int block,
                                float scale, const int32_t* q_rows, int n_q, float* energy, int accumulate,
                                void* stream) {
    if (!q || !k || !energy || !aligned16(q) || !aligned16(k)) return CALIB_ERR_INVALID;
    if ((reinterpret_cast<uintptr_t>(energy) & 3u) || (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)))
        return CALIB_ERR_INVALID;
    if (H < 1 || N < 1 || !(scale > 0.f) || !std::isfinite(scale)) return CALIB_ERR_INVALID;
    if (block != 64 && block != 128) return CALIB_ERR_INVALID;
    if (D != 64 && D != 128) return CALIB_ERR_UNSUPPORTED;
    const int Nq = q_rows ? n_q : N;
    if (q_rows && n_q < 1) return CALIB_ERR_INVALID;
    const int nq = cdiv(Nq, block), nk = cdiv(N, block);
    if (static_cast<long long>(H) * nq > (1ll << 31) - 1) return CALIB_ERR_INVALID;
    if (N > calib::kEnergyMaxTokens) return CALIB_ERR_UNSUPPORTED;
    if (calib_status s = check_device()) return s;
    calib::EnergyParams p{};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.q_rows = q_rows;
    p.lse_in = lse;
    p.energy = energy;
    p.H = H; p.N = N; p.Nq = Nq; p.nq = nq; p.nk = nk;
    p.accumulate = accumulate ? 1 : 0;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.timeout_ns = kDefaultTimeoutNs;
    CUtensorMap tk;
    if (!make_tmap(&tk, k, D, N, H, block)) return CALIB_ERR_CUDA;
    cudaStream_t st = as_stream(stream);
    const int grid = H * nq;
    if (D == 128) return block == 128 ? launch_energy<128, 128>(tk, p, grid, st) : launch_energy<128, 64>(tk, p, grid, st);
    return block == 128 ? launch_energy<64, 128>(tk, p, grid, st) : launch_energy<64, 64>(tk, p, grid, st);
}

calib_status calib_select_mask_batched(const float* energy, int nb, int H, int nq, int nk, const double* tau,
                                       const uint8_t* force_keep, uint8_t* mask_out, int32_t* count_accum,
                                       void* stream) {
    if (!energy || !tau || (!mask_out && !count_accum)) return CALIB_ERR_INVALID;
    if (nb < 1 || nb > calib::kSelMaxBatch || H < 1 || nq < 1 || nk < 1) return CALIB_ERR_INVALID;
    if (nk > 32 * calib::kSelMaxPerLane) return CALIB_ERR_UNSUPPORTED;
    if ((reinterpret_cast<uintptr_t>(energy) & 3u) || (reinterpret_cast<uintptr_t>(count_accum) & 3u))
        return CALIB_ERR_INVALID;
    if (static_cast<long long>(nb) * H * nq * nk > (1ll << 31) - 1) return CALIB_ERR_INVALID;
    for (int b = 0; b < nb; ++b)
        if (!(tau[b] > 0.0) || !(tau[b] <= 1.0)) return CALIB_ERR_INVALID;
    if (calib_status s = check_device()) return s;
    calib::SelectParams p{};
    p.energy = energy;
    p.force = force_keep;
    p.mask_out = mask_out;
    p.count_accum = count_accum;
    p.nb = nb; p.rows = H * nq; p.nq = nq; p.nk = nk;
    for (int b = 0; b < nb; ++b) p.tau[b] = tau[b];
    // one warp per (row, chunk of entries): enough warps to fill every SM a few times over,
    // and each warp walks its chunk of entries so that vote counts accumulate in registers
    const long long target = 148ll * 48;
    int n_chunks = static_cast<int>(std::min<long long>(nb, std::max<long long>(1, (target + p.rows - 1) / p.rows)));
    p.chunk = (nb + n_chunks - 1) / n_chunks;
    p.n_chunks = (nb + p.chunk - 1) / p.chunk;
    p.vec = ((nk & 3) == 0 && (reinterpret_cast<uintptr_t>(energy) & 15u) == 0 &&
             (!mask_out || (reinterpret_cast<uintptr_t>(mask_out) & 3u) == 0)) ? 1 : 0;
    const long long warps = static_cast<long long>(p.rows) * p.n_chunks;
    const int grid = static_cast<int>((warps + calib::kSelWarps - 1) / calib::kSelWarps);
    cudaStream_t st = as_stream(stream);
    // energies per lane: the smallest instantiated count covering the row
    auto launch = [&](auto mpl) {
        calib::select_mask_kernel<decltype(mpl)::value><<<grid, calib::kSelWarps * 32, 0, st>>>(p);
    };
    if (nk <= 64) launch(std::integral_constant<int, 2>{});
    else if (nk <= 128) launch(std::integral_constant<int, 4>{});
    else if (nk <= 256) launch(std::integral_constant<int, 8>{});
    else if (nk <= 512) launch(std::integral_constant<int, 16>{});
    else if (nk <= 640) launch(std::integral_constant<int, 20>{});
    else launch(std::integral_constant<int, 32>{});
    return launch_status();
}

calib_status calib_select_mask(const float* energy, int H, int nq, int nk, double tau, const uint8_t* force_keep,
                               uint8_t* mask_out, int32_t* count_accum, void* stream) {
    if (!mask_out) return CALIB_ERR_INVALID;
    return calib_select_mask_batched(energy, 1, H, nq, nk, &tau, force_keep, mask_out, count_accum, stream);
}

calib_status calib_energy_mean(const float* energy_sum, int64_t count, int n_inputs, float* mean_out,
                               void* stream) {
    if (!energy_sum || !mean_out || count < 1 || n_inputs < 1 || n_inputs > (1 << 24)) return CALIB_ERR_INVALID;
    if ((reinterpret_cast<uintptr_t>(energy_sum) & 3u) || (reinterpret_cast<uintptr_t>(mean_out) & 3u))
        return CALIB_ERR_INVALID;
    if (calib_status s = check_device()) return s;
    const long long want = (count / 4 + 255) / 256;
    const int grid = static_cast<int>(std::max<long long>(1, std::min<long long>(want, 148ll * 8)));
    calib::energy_mean_kernel<<<grid, 256, 0, as_stream(stream)>>>(energy_sum, count, static_cast<float>(n_inputs),
                                                                   mean_out);
    return launch_status();
}

calib_status calib_aggregate_masks(const int32_t* counts, int H, int nq, int nk, int n_inputs, int rho_num,
                                   int rho_den, uint8_t* mask_out, void* stream) {
    if (!counts || !mask_out) return CALIB_ERR_INVALID;
    if (H < 1 || nq < 1 || nk < 1 || n_inputs < 1 || rho_num < 0 || rho_den < 1 || rho_num > rho_den)
        return CALIB_ERR_INVALID;
    if (static_cast<long long>(H) * nq * nk > (1ll << 31) - 1) return CALIB_ERR_INVALID;
    if (calib_status s = check_device()) return s;
    const int rows = H * nq;
    calib::aggregate_kernel<<<rows_grid(rows), 128, 0, as_stream(stream)>>>(counts, rows, nk, n_inputs, rho_num,
                                                                             rho_den, mask_out);
    return launch_status();
}

calib_status calib_mask_to_csr(const uint8_t* mask, int H, int nq, int nk, int32_t* row_ptr_out,
                               int16_t* col_idx_out, void* stream) {
    if (!mask || !row_ptr_out || !col_idx_out) return CALIB_ERR_INVALID;
    if (H < 1 || nq < 1 || nk < 1 || nk > 32767) return CALIB_ERR_INVALID;
    if (static_cast<long long>(H) * nq * nk > (1ll << 31) - 1) return CALIB_ERR_INVALID;
    if (calib_status s = check_device()) return s;
    const int rows = H * nq;
    cudaStream_t st = as_stream(stream);
    calib::csr_count_kernel<<<rows_grid(rows), 128, 0, st>>>(mask, rows, nk, row_ptr_out);
    calib::csr_scan_kernel<<<1, 1024, 0, st>>>(row_ptr_out, rows);
    calib::csr_fill_kernel<<<rows_grid(rows), 128, 0, st>>>(mask, rows, nk, row_ptr_out, col_idx_out);
    return launch_status();
}

calib_status calib_csr_to_intervals(const int32_t* row_ptr, const int16_t* col_idx, int H, int nq,
                                    int32_t* iv_ptr_out, int16_t* iv_start_out, int16_t* iv_len_out, void* stream) {
    if (!row_ptr || !col_idx || !iv_ptr_out || !iv_start_out || !iv_len_out) return CALIB_ERR_INVALID;
    if (H < 1 || nq < 1 || static_cast<long long>(H) * nq > (1ll << 31) - 2) return CALIB_ERR_INVALID;
    if (calib_status s = check_device()) return s;
    const int rows = H * nq;
    cudaStream_t st = as_stream(stream);
    calib::iv_count_kernel<<<rows_grid(rows), 128, 0, st>>>(row_ptr, col_idx, rows, iv_ptr_out);
    calib::csr_scan_kernel<<<1, 1024, 0, st>>>(iv_ptr_out, rows);
    calib::iv_fill_kernel<<<rows_grid(rows), 128, 0, st>>>(row_ptr, col_idx, rows, iv_ptr_out, iv_start_out,
                                                           iv_len_out);
    return launch_status();
}

calib_status calib_intervals_to_csr(const int32_t* iv_ptr, const int16_t* iv_start, const int16_t* iv_len, int H,
                                    int nq, int32_t* row_ptr_out, int16_t* col_idx_out, void* stream) {
    if (!iv_ptr || !iv_start || !iv_len || !row_ptr_out) return CALIB_ERR_INVALID;
    if (H < 1 || nq < 1 || static_cast<long long>(H) * nq > (1ll << 31) - 2) return CALIB_ERR_INVALID;
    if (calib_status s = check_device()) return s;
    const int rows = H * nq;
    cudaStream_t st = as_stream(stream);
    calib::iv_total_kernel<<<rows_grid(rows), 128, 0, st>>>(iv_ptr, iv_len, rows, row_ptr_out);
    calib::csr_scan_kernel<<<1, 1024, 0, st>>>(row_ptr_out, rows);
    if (col_idx_out)
        calib::iv_expand_kernel<<<rows_grid(rows), 128, 0, st>>>(iv_ptr, iv_start, iv_len, rows, row_ptr_out,
                                                                 col_idx_out);
    return launch_status();
}

calib_status calib_transpose_csr(const int32_t* row_ptr, const int16_t* col_idx, int H, int nq, int nk,
                                 int32_t* t_row_ptr_out, int16_t* t_col_idx_out, void* stream) {
    if (!row_ptr || !col_idx || !t_row_ptr_out || !t_col_idx_out) return CALIB_ERR_INVALID;
    if (H < 1 || nq < 1 || nk < 1 || nq > 32767 || nk > 32767) return CALIB_ERR_INVALID;
    if (static_cast<long long>(H) * std::max(nq, nk) > (1ll << 31) - 2) return CALIB_ERR_INVALID;
    if (calib_status s = check_device()) return s;
    // CTAs per head: as many as there are SMs for, at most 8 and one per word of 32 rows.  Each asks for more than
    // half of an SM's shared memory, so that no two share an SM while others idle (40 heads of 591: 39 us with four
    // each and two on some SMs).  Tiles of at most 1024 columns (a thread each), and of 80 KB.
    const int words = cdiv(nq, 32);
    const int cluster = std::max(1, std::min(std::min(kSms / H, calib::kTransMaxCluster), words));
    const int per = cdiv(words, cluster), stride = per | 1;
    const int cols = std::min(std::min(nk, calib::kTransThreads), 80 * 1024 / 4 / stride);
    constexpr int stage = calib::kTransWarps * 4 * calib::kTransStage * 2;
    const int bytes = std::max(116 * 1024, cols * stride * 4 + stage + per * 32 * 2);
    auto* fn = calib::transpose_csr_kernel;
    if (calib_status s = ensure_smem(reinterpret_cast<const void*>(fn), 80 * 1024 + stage + 32768 * 2)) return s;
    return launch_with(fn, H * cluster, calib::kTransThreads, bytes, as_stream(stream), cluster, false, row_ptr, col_idx, nq,
                       nk, cluster, cols, t_row_ptr_out, t_col_idx_out);
}

calib_status calib_cache_write(const void* k_new, const void* v_new, void* k_cache, void* v_cache, float* k_scale,
                               float* v_scale, const int32_t* block_table, const int32_t* lengths,
                               const int32_t* new_lens, int S, int Hkv, int M, int D, int block, int max_blocks,
                               int64_t pages, void* stream) {
    if (!k_new || !v_new || !aligned16(k_new) || !aligned16(v_new)) return CALIB_ERR_INVALID;
    if (reinterpret_cast<uintptr_t>(new_lens) & 3u) return CALIB_ERR_INVALID;
    if (calib_status s = cache_args(k_cache, v_cache, k_scale, v_scale, block_table, lengths, S, Hkv, M, D, block,
                                    max_blocks, pages))
        return s;
    calib::CacheWriteParams p{};
    p.k_new = static_cast<const __nv_bfloat16*>(k_new);
    p.v_new = static_cast<const __nv_bfloat16*>(v_new);
    p.k = static_cast<uint8_t*>(k_cache);
    p.v = static_cast<uint8_t*>(v_cache);
    p.k_scale = k_scale; p.v_scale = v_scale;
    p.table = block_table; p.lengths = lengths; p.new_lens = new_lens;
    p.S = S; p.Hkv = Hkv; p.M = M; p.nb = max_blocks; p.pages = static_cast<int>(pages);
    p.T = std::min(cdiv(M - 1, block) + 1, max_blocks);
    const long long grid = 2ll * S * Hkv * p.T;
    if (grid > (1ll << 31) - 1) return CALIB_ERR_UNSUPPORTED;
    cudaStream_t st = as_stream(stream);
    const int g = static_cast<int>(grid);
    if (D == 128) return block == 128 ? launch_write<128, 128>(p, g, st) : launch_write<128, 64>(p, g, st);
    return block == 128 ? launch_write<64, 128>(p, g, st) : launch_write<64, 64>(p, g, st);
}

int64_t sparse_attn_cached_workspace(int S, int Hq, int Hkv, int M, int D, int block, int max_blocks) {
    if (S < 1 || Hkv < 1 || Hq < Hkv || Hq % Hkv || M < 1 || max_blocks < 1 || (block != 64 && block != 128) ||
        (D != 64 && D != 128) || static_cast<long long>(S) * Hq > (1ll << 31) - 1 ||
        static_cast<long long>(S) * Hq * M > (1ll << 31) - 1)
        return -1;
    return cached_plan(S, Hq, Hkv, M, D, block, max_blocks).bytes;
}

calib_status sparse_attn_cached(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                                const float* v_scale, const int32_t* block_table, const int32_t* lengths,
                                const int32_t* new_lens, void* o, float* lse_opt, int S, int Hq, int Hkv, int M,
                                int D, int block, int max_blocks, int64_t pages, float scale,
                                const calib_block_list* list, uint32_t flags, void* workspace,
                                int64_t workspace_bytes, void* stream) {
    if (!q || !o || !aligned16(q) || !aligned16(o)) return CALIB_ERR_INVALID;
    if (flags & ~(CALIB_ATTN_OUT_F32 | CALIB_ATTN_CAUSAL)) return CALIB_ERR_INVALID;
    if ((reinterpret_cast<uintptr_t>(new_lens) & 3u) || (reinterpret_cast<uintptr_t>(lse_opt) & 3u)) return CALIB_ERR_INVALID;
    if (!(scale > 0.f) || !std::isfinite(scale)) return CALIB_ERR_INVALID;
    if (Hkv < 1 || Hq < Hkv || Hq % Hkv) return CALIB_ERR_INVALID;
    if (calib_status s = cache_args(k_cache, v_cache, k_scale, v_scale, block_table, lengths, S, Hkv, M, D, block,
                                    max_blocks, pages))
        return s;
    if (list && (!list->row_ptr || !list->col_idx || list->H != Hkv || list->nq != S || list->nk != max_blocks ||
                 list->block != block || max_blocks > 32767))
        return CALIB_ERR_INVALID;
    const int64_t need = sparse_attn_cached_workspace(S, Hq, Hkv, M, D, block, max_blocks);
    if (need < 0) return CALIB_ERR_UNSUPPORTED;
    if (need > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < need)) return CALIB_ERR_INVALID;
    const CachedPlan c = cached_plan(S, Hq, Hkv, M, D, block, max_blocks);
    if (c.grid > (1ll << 31) - 1) return CALIB_ERR_UNSUPPORTED;
    calib::CachedParams p{};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k_scale = k_scale; p.v_scale = v_scale;
    p.table = block_table; p.lengths = lengths; p.new_lens = new_lens;
    if (list) {
        p.row_ptr = list->row_ptr;
        p.col_idx = list->col_idx;
    }
    p.o = o;
    p.lse = lse_opt;
    if (c.flat) {
        char* base = static_cast<char*>(workspace);
        p.pieces = reinterpret_cast<int2*>(base);
        p.part_o = reinterpret_cast<float*>(base + c.part_o);
        p.part_ml = reinterpret_cast<float2*>(base + c.part_ml);
    }
    p.S = S; p.Hq = Hq; p.Hkv = Hkv; p.G = Hq / Hkv; p.M = M; p.nb = max_blocks; p.pages = static_cast<int>(pages);
    p.tiles = c.tiles; p.flat = c.flat; p.cluster = c.cluster;
    p.causal = (flags & CALIB_ATTN_CAUSAL) ? 1 : 0;
    p.out_f32 = (flags & CALIB_ATTN_OUT_F32) ? 1 : 0;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.timeout_ns = kDefaultTimeoutNs;
    CUtensorMap tk, tv;
    const long long rows = static_cast<long long>(pages) * Hkv * block;
    if (!make_cache_tmap(&tk, k_cache, D, rows) || !make_cache_tmap(&tv, v_cache, D, rows)) return CALIB_ERR_CUDA;
    cudaStream_t st = as_stream(stream);
    if (D == 128) return block == 128 ? launch_cached_nt<128, 128>(tk, tv, p, c, st) : launch_cached_nt<128, 64>(tk, tv, p, c, st);
    return block == 128 ? launch_cached_nt<64, 128>(tk, tv, p, c, st) : launch_cached_nt<64, 64>(tk, tv, p, c, st);
}

int64_t sparse_attn_bwd_workspace(int H, int N, int D, int block, int n_anchor, uint32_t flags) {
    if (H < 1 || N < 1 || (D != 64 && D != 128) || (block != 64 && block != 128) || n_anchor < 0 || n_anchor > N ||
        static_cast<long long>(H) * N * D >= (1ll << 40) || (flags & ~(CALIB_ATTN_OUT_F32 | CALIB_ATTN_GRAD_F32)))
        return -1;
    return static_cast<int64_t>(bwd_space(H, N, D, block, n_anchor, flags & CALIB_ATTN_OUT_F32).total);
}

calib_status sparse_attn_bwd(const void* q, const void* k, const void* v, const void* o, const void* dout,
                             const float* lse, void* dq, void* dk, void* dv, int H, int N, int D, float scale,
                             const calib_block_list* list, const calib_block_list* list_t, uint32_t flags,
                             void* workspace, int64_t workspace_bytes, void* stream) {
    return bwd_common(q, k, v, o, dout, lse, dq, dk, dv, H, N, D, scale, list, list_t, nullptr, 1, 1, N, 0, 1, flags,
                      workspace, workspace_bytes, stream);
}

calib_status sparse_attn_bwd_repeat(const void* q, const void* k, const void* v, const void* o, const void* dout,
                                    const float* lse, void* dq, void* dk, void* dv, int H, int D, int F, int Hl,
                                    int Wl, int n_text, int stride, const uint8_t* head_repeat, float scale,
                                    const calib_block_list* list, const calib_block_list* list_t, uint32_t flags,
                                    void* workspace, int64_t workspace_bytes, void* stream) {
    uint32_t bits[32];
    int N = 0;
    if (calib_status s = repeat_geometry(H, F, Hl, Wl, n_text, stride, head_repeat, bits, &N)) return s;
    return bwd_common(q, k, v, o, dout, lse, dq, dk, dv, H, N, D, scale, list, list_t, bits, F, Hl, Wl, n_text, stride,
                      flags, workspace, workspace_bytes, stream);
}

calib_status calib_repeat_similarity(const void* q, const void* k, const float* lse, int H, int N, int D, int block,
                                     float scale, int F, int Hl, int Wl, int stride, const int32_t* members, int n,
                                     float* cos_out, void* stream) {
    if (!q || !k || !members || !cos_out || !aligned16(q) || !aligned16(k)) return CALIB_ERR_INVALID;
    if ((reinterpret_cast<uintptr_t>(cos_out) & 3u) || (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)))
        return CALIB_ERR_INVALID;
    if (H < 1 || N < 1 || n < 1 || !(scale > 0.f) || !std::isfinite(scale)) return CALIB_ERR_INVALID;
    if (F < 1 || Hl < 1 || Wl < 1 || stride < 1 || static_cast<long long>(F) * Hl * Wl > N) return CALIB_ERR_INVALID;
    if (block != 64 && block != 128) return CALIB_ERR_INVALID;
    if (D != 64 && D != 128) return CALIB_ERR_UNSUPPORTED;
    const int tiles = cdiv(n, calib::kSimPairs);
    if (static_cast<long long>(H) * tiles > (1ll << 31) - 1) return CALIB_ERR_INVALID;
    if (calib_status s = check_device()) return s;
    calib::SimParams p{};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.members = members;
    p.lse_in = lse;
    p.cos_out = cos_out;
    p.H = H; p.N = N; p.n = n; p.tiles = tiles; p.nk = cdiv(N, block);
    p.F = F; p.Hl = Hl; p.Wl = Wl; p.stride = stride;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.timeout_ns = kDefaultTimeoutNs;
    CUtensorMap tk;
    if (!make_tmap(&tk, k, D, N, H, block)) return CALIB_ERR_CUDA;
    cudaStream_t st = as_stream(stream);
    const int grid = H * tiles;
    if (D == 128) return block == 128 ? launch_sim<128, 128>(tk, p, grid, st) : launch_sim<128, 64>(tk, p, grid, st);
    return block == 128 ? launch_sim<64, 128>(tk, p, grid, st) : launch_sim<64, 64>(tk, p, grid, st);
}

calib_status calib_repeat_flags(const float* cos, const int32_t* members, int H, int n, int F, int Hl, int Wl,
                                int stride, float gamma, float* mean_out, uint8_t* flag_out, void* stream) {
    if (!cos || !members || !mean_out || !flag_out) return CALIB_ERR_INVALID;
    if (H < 1 || n < 1 || F < 1 || Hl < 1 || Wl < 1 || stride < 1 || !std::isfinite(gamma)) return CALIB_ERR_INVALID;
    if (calib_status s = check_device()) return s;
    calib::repeat_flags_kernel<<<H, 256, 0, as_stream(stream)>>>(cos, members, n, F, Hl, Wl, stride, gamma, mean_out,
                                                                  flag_out);
    return launch_status();
}

calib_status calib_build_schedule(const int32_t* row_ptr, int H, int nq, int32_t* work_out, void* stream) {
    if (!row_ptr || !work_out) return CALIB_ERR_INVALID;
    if (H < 1 || nq < 1 || H > 32767 || nq > 65535) return CALIB_ERR_INVALID;
    if (calib_status s = check_device()) return s;
    const int bytes = calib::kSchedBins * 4;
    if (calib_status s = ensure_smem(reinterpret_cast<const void*>(calib::schedule_kernel), bytes)) return s;
    calib::schedule_kernel<<<H, 1024, bytes, as_stream(stream)>>>(row_ptr, nq, work_out);
    return launch_status();
}

int64_t calib_anchor_count(int F, int Hl, int Wl, int n_text, int stride) {
    if (F < 1 || Hl < 1 || Wl < 1 || n_text < 0 || stride < 1) return -1;
    const int64_t Ar = (Hl + stride - 1) / stride;
    return static_cast<int64_t>(F) * Ar * Wl + n_text;
}

calib_status calib_anchor_rows(int F, int Hl, int Wl, int n_text, int stride, int32_t* rows_out, void* stream) {
    const int64_t na = calib_anchor_count(F, Hl, Wl, n_text, stride);
    if (!rows_out || na < 0 || static_cast<int64_t>(F) * Hl * Wl + n_text > (1ll << 31) - 1) return CALIB_ERR_INVALID;
    if (calib_status s = check_device()) return s;
    const int Ar = (Hl + stride - 1) / stride;
    const int n = static_cast<int>(na);
    calib::anchor_rows_kernel<<<cdiv(n, 256), 256, 0, as_stream(stream)>>>(F, Hl, Wl, n_text, stride, Ar, n,
                                                                            rows_out);
    return launch_status();
}

calib_status sparse_attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse_opt, int H, int N,
                             int D, float scale, const calib_block_list* list, uint32_t flags, void* stream) {
    return attn_common(q, k, v, o, lse_opt, H, N, D, scale, list, nullptr, 1, 1, N, 0, 1, flags, stream);
}

calib_status sparse_attn_fwd_host(const void* q_host, const void* k_host, const void* v_host, void* o_host,
                                  void* q_dev, void* k_dev, void* v_dev, void* o_dev, float* lse_opt, int H,
                                  int N, int D, float scale, const calib_block_list* list, uint32_t flags,
                                  int heads_per_chunk, void* stream, void* h2d_stream, void* d2h_stream) {
    if (!q_host || !k_host || !v_host || !o_host || heads_per_chunk < 1) return CALIB_ERR_INVALID;
    AttnCall c;
    if (calib_status s = attn_prepare(q_dev, k_dev, v_dev, o_dev, lse_opt, H, N, D, scale, list, nullptr, 1, 1, N,
                                      0, 1, flags, &c))
        return s;
    return host_pipeline(c, q_host, k_host, v_host, o_host, q_dev, k_dev, v_dev, o_dev, H, N, D, list, flags,
                         heads_per_chunk, stream, h2d_stream, d2h_stream);
}

calib_status sparse_attn_fwd_repeat_host(const void* q_host, const void* k_host, const void* v_host,
                                         void* o_host, void* q_dev, void* k_dev, void* v_dev, void* o_dev,
                                         float* lse_opt, int H, int D, int F, int Hl, int Wl, int n_text,
                                         int stride, const uint8_t* head_repeat, float scale,
                                         const calib_block_list* list, uint32_t flags, int heads_per_chunk,
                                         void* stream, void* h2d_stream, void* d2h_stream) {
    if (!q_host || !k_host || !v_host || !o_host || heads_per_chunk < 1) return CALIB_ERR_INVALID;
    uint32_t bits[32];
    int N = 0;
    if (calib_status s = repeat_geometry(H, F, Hl, Wl, n_text, stride, head_repeat, bits, &N)) return s;
    AttnCall c;
    if (calib_status s = attn_prepare(q_dev, k_dev, v_dev, o_dev, lse_opt, H, N, D, scale, list, bits, F, Hl, Wl,
                                      n_text, stride, flags, &c))
        return s;
    return host_pipeline(c, q_host, k_host, v_host, o_host, q_dev, k_dev, v_dev, o_dev, H, N, D, list, flags,
                         heads_per_chunk, stream, h2d_stream, d2h_stream);
}

calib_status sparse_attn_fwd_repeat(const void* q, const void* k, const void* v, void* o, float* lse_opt, int H,
                                    int D, int F, int Hl, int Wl, int n_text, int stride,
                                    const uint8_t* head_repeat, float scale, const calib_block_list* list,
                                    uint32_t flags, void* stream) {
    uint32_t bits[32];
    int N = 0;
    if (calib_status s = repeat_geometry(H, F, Hl, Wl, n_text, stride, head_repeat, bits, &N)) return s;
    return attn_common(q, k, v, o, lse_opt, H, N, D, scale, list, bits, F, Hl, Wl, n_text, stride, flags, stream);
}

calib_status calib_validate_block_list_host(int H, int nq, int nk, const int32_t* row_ptr, const int16_t* col_idx,
                                            int64_t col_capacity, const int32_t* work, int n_work) {
    if (H < 1 || nq < 1 || nk < 1 || nk > 32767 || !row_ptr || col_capacity < 0) return CALIB_ERR_INVALID;
    const long long rows = static_cast<long long>(H) * nq;
    if (rows > (1ll << 31) - 2 || row_ptr[0] != 0) return CALIB_ERR_INVALID;
    for (long long r = 0; r < rows; ++r) {
        const long long b = row_ptr[r], e = row_ptr[r + 1];
        if (e < b || e - b > nk || e > col_capacity) return CALIB_ERR_INVALID;
        if (e > b && !col_idx) return CALIB_ERR_INVALID;
        for (long long x = b; x < e; ++x) {
            const int j = col_idx[x];
            if (j < 0 || j >= nk || (x > b && j <= col_idx[x - 1])) return CALIB_ERR_INVALID;
        }
    }
    if (work) {
        if (n_work < 0) return CALIB_ERR_INVALID;
        for (int w = 0; w < n_work; ++w) {
            const int32_t item = work[w];
            if (item < 0 || (item >> 16) >= H || (item & 0xFFFF) >= nq) return CALIB_ERR_INVALID;
        }
    }
    return CALIB_OK;
}

calib_status calib_selftest_wait_timeout(uint32_t timeout_us, void* stream) {
    if (calib_status s = check_device()) return s;
    calib::selftest_wait_kernel<<<1, 32, 0, as_stream(stream)>>>(static_cast<uint64_t>(timeout_us) * 1000ull);
    if (cudaGetLastError() != cudaSuccess) return CALIB_ERR_CUDA;
    return calib_device_check(stream);
}

}  // extern "C"
