// pp_api.cu - the C ABI of libpp (declared in include/pp.h): host-side validation, tensor maps, launches, and the
// device error channel. The whole library is this one translation unit; the kernels live in the included headers.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <string>
#include <type_traits>

#include "../../include/pp.h"
#include "pp_ptx.cuh"
#include "pp_meta.cuh"
#include "pp_build.cuh"
#include "pp_rope.cuh"
#include "pp_attn_fwd.cuh"
#include "pp_attn_bwd.cuh"
#include "pp_logprobs.cuh"
#include "pp_pack.cuh"
#include "pp_decode.cuh"
#include "pp_qknorm.cuh"
#include "pp_pages.cuh"
#include "pp_cache.cuh"
#include "pp_paged.cuh"

namespace {

thread_local std::string g_last_error;

pp_status fail(pp_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
pp_status fail(pp_status st, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    g_last_error = buf;
    return st;
}

#define PP_CUDA(call)                                                                                   \
    do {                                                                                                \
        cudaError_t e_ = (call);                                                                        \
        if (e_ != cudaSuccess)                                                                          \
            return fail(PP_ERR_CUDA, "%s failed: %s", #call, cudaGetErrorString(e_));                  \
    } while (0)

inline cudaStream_t as_stream(void *s) { return reinterpret_cast<cudaStream_t>(s); }

constexpr int kMaxDevices = 64;
struct DeviceInfo {
    bool ready = false;
    int sm_count = 0;
    int max_smem_optin = 0;
};
DeviceInfo g_dev[kMaxDevices];
std::mutex g_mu;

pp_status device_info(DeviceInfo **out) {
    int dev = 0;
    PP_CUDA(cudaGetDevice(&dev));
    if (dev < 0 || dev >= kMaxDevices) return fail(PP_ERR_CUDA, "device index %d out of range", dev);
    std::lock_guard<std::mutex> lk(g_mu);
    DeviceInfo &d = g_dev[dev];
    if (!d.ready) {
        PP_CUDA(cudaDeviceGetAttribute(&d.sm_count, cudaDevAttrMultiProcessorCount, dev));
        PP_CUDA(cudaDeviceGetAttribute(&d.max_smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev));
        int major = 0, minor = 0;
        PP_CUDA(cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev));
        PP_CUDA(cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev));
        if (major != 10 || minor != 0)
            return fail(PP_ERR_UNSUPPORTED, "libpp is built for sm_100a (B200); device %d is sm_%d%d", dev, major,
                        minor);
        d.ready = true;
    }
    *out = &d;
    return PP_OK;
}

// cuTensorMapEncodeTiled through the runtime's driver entry point (no link-time dependency on libcuda).
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn g_encode = nullptr;

pp_status get_encoder(EncodeTiledFn *fn) {
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g_encode) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        cudaError_t e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q);
        if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !p)
            return fail(PP_ERR_CUDA, "cuTensorMapEncodeTiled entry point unavailable");
        g_encode = reinterpret_cast<EncodeTiledFn>(p);
    }
    *fn = g_encode;
    return PP_OK;
}

// 3-D map over a [rows, heads, d] bf16 tensor: box = 64 elements x box_heads heads x box_rows rows, 128-byte swizzle.
pp_status make_map_3d_box(CUtensorMap *m, const void *base, int64_t rows, int heads, int d, int box_heads,
                          int box_rows);

pp_status make_map_3d(CUtensorMap *m, const void *base, int64_t rows, int heads, int d, int box_rows) {
    return make_map_3d_box(m, base, rows, heads, d, 1, box_rows);
}

pp_status make_map_3d_box(CUtensorMap *m, const void *base, int64_t rows, int heads, int d, int box_heads,
                          int box_rows) {
    EncodeTiledFn enc;
    pp_status st = get_encoder(&enc);
    if (st != PP_OK) return st;
    if (reinterpret_cast<uintptr_t>(base) % 16) return fail(PP_ERR_INVALID_ARG, "tensor base not 16-byte aligned");
    cuuint64_t dims[3] = {cuuint64_t(d), cuuint64_t(heads), cuuint64_t(rows)};
    cuuint64_t strides[2] = {cuuint64_t(d) * 2, cuuint64_t(heads) * d * 2};
    cuuint32_t box[3] = {64, cuuint32_t(box_heads), cuuint32_t(box_rows)};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(PP_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", int(r));
    return PP_OK;
}

pp_status check_heads(int64_t T, int32_t hq, int32_t hkv, int32_t d) {
    if (T < 0 || T >= (int64_t(1) << 31) - 256) return fail(PP_ERR_INVALID_ARG, "T=%lld out of range", (long long)T);
    if (hq <= 0 || hkv <= 0 || hq > 256 || hq % hkv != 0)
        return fail(PP_ERR_INVALID_ARG, "need 0 < hkv, hq %% hkv == 0, hq <= 256 (hq=%d hkv=%d)", hq, hkv);
    if (d != 64 && d != 128) return fail(PP_ERR_INVALID_ARG, "head dim %d not in {64, 128}", d);
    return PP_OK;
}

// A call's second kernel, launched as the first one's programmatic dependent: its blocks are made ready while the first
// ends, and griddepcontrol.wait, which it begins with, holds them until the first's writes are seen. In a row of
// pp_paged_decode calls 1.2 to 2.4 us less; in a graph no difference. (With the first kernel releasing its dependents at
// its start, not at its end, a graph was 0.2 to 1.1 us slower.)
template <typename... P, typename... A>
pp_status launch_second(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t s, const A &...args) {
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    PP_CUDA(cudaLaunchKernelEx(&cfg, kernel, P(args)...));
    return PP_OK;
}

// cudaFuncAttributeMaxDynamicSharedMemorySize of a kernel, raised once to the most that it is ever launched with; `done`
// holds a bit for each device. (The attribute calls take longer than a launch of a few microseconds' work.)
template <typename K> pp_status allow_smem(K kernel, int bytes, std::atomic<uint64_t> *done) {
    int dev = 0;
    PP_CUDA(cudaGetDevice(&dev));
    if (dev < 0 || dev >= kMaxDevices) return fail(PP_ERR_CUDA, "device index %d out of range", dev);
    if (!(done->load(std::memory_order_acquire) >> dev & 1)) {
        PP_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
        done->fetch_or(uint64_t(1) << dev, std::memory_order_release);
    }
    return PP_OK;
}

int grid_for(int sm_count, int per_sm, int64_t work) {
    int64_t g = int64_t(sm_count) * per_sm;
    if (work < g) g = work;
    return int(g < 1 ? 1 : g);
}

// Scratch of pp_attn_bwd_noalloc (see include/pp.h): compiled into the library so that callers who cannot
// allocate still get a backward. Host code must not use the symbol's host-side name as a device address; the
// device address is looked up once per device below.
static __device__ __align__(256) unsigned char g_noalloc_scratch[PP_NOALLOC_SCRATCH_BYTES];
void *g_noalloc_ptr[kMaxDevices] = {};

pp_status noalloc_scratch(void **out) {
    int dev = 0;
    PP_CUDA(cudaGetDevice(&dev));
    if (dev < 0 || dev >= kMaxDevices) return fail(PP_ERR_CUDA, "device index %d out of range", dev);
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g_noalloc_ptr[dev]) {
        void *p = nullptr;
        cudaError_t e = cudaGetSymbolAddress(&p, g_noalloc_scratch);   // with `dev` current
        if (e != cudaSuccess || !p)
            return fail(PP_ERR_CUDA, "cudaGetSymbolAddress(noalloc scratch): %s", cudaGetErrorString(e));
        g_noalloc_ptr[dev] = p;
    }
    *out = g_noalloc_ptr[dev];
    return PP_OK;
}

// ---- q/k norm with the rotation

bool bad_align(const void *p, int64_t a = 16) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

// Arrays of int32 or float.
template <typename... A> bool bad_words(const A *...p) { return (bad_align(p, 4) || ...); }

// theta^(-2m/d) / (2 pi) in fp64, computed once per (theta, d) and thread.
const pp::QknTurns &qkn_turns(float theta, int32_t d) {
    thread_local pp::QknTurns t;
    thread_local float have_theta = -1.f;
    thread_local int32_t have_d = 0;
    if (have_theta != theta || have_d != d) {
        for (int m = 0; m < d / 2; ++m)
            t.w[m] = std::pow(double(theta), -2.0 * m / d) / 6.283185307179586476925286766559;
        have_theta = theta;
        have_d = d;
    }
    return t;
}

struct QknSide {
    const void *x, *w, *g;
    void *y;
    int64_t xs, gs, ys;
    int32_t heads;
};

pp_status qkn_check(const QknSide &s, int32_t d, int64_t es, bool bwd, const char *what) {
    const int64_t dense = int64_t(s.heads) * d;
    if (!s.x) return PP_OK;
    if (!s.y || (bwd && !s.g)) return fail(PP_ERR_INVALID_ARG, "%s: NULL pointer argument", what);
    if (s.xs < dense || s.ys < dense || (bwd && s.gs < dense))
        return fail(PP_ERR_INVALID_ARG, "%s: token stride below heads * d", what);
    if (bad_align(s.x) || bad_align(s.y) || bad_align(s.w) || bad_align(s.g) || s.xs * es % 16 || s.ys * es % 16 ||
        (bwd && s.gs * es % 16))
        return fail(PP_ERR_INVALID_ARG, "%s: pointers and token strides must be multiples of 16 bytes", what);
    if ((s.y == s.x && s.ys != s.xs) || (bwd && s.y == s.g && s.ys != s.gs))
        return fail(PP_ERR_INVALID_ARG, "%s: an output over its input needs the same token stride", what);
    return PP_OK;
}

// Blocks and heads per warp of each side. A warp takes a token's heads together, so that its angles are formed once,
// unless that leaves the GPU without work (few tokens): then the heads are dealt out, one warp's row group at a time.
template <typename T, int D, bool BWD>
pp_status qkn_launch(const QknSide &q, const QknSide &k, const int32_t *pos, int64_t T_, float eps, float theta,
                     int sm_count, float *part, int32_t *nq, int32_t *nk, cudaStream_t s) {
    constexpr int R = pp::QknRow<D>::R;
    const int64_t warps = int64_t(sm_count) * (BWD ? pp::QKN_BLOCKS_BWD * 8 : 32);
    auto side = [&](const QknSide &x) {
        pp::QknPart<T> p{};
        p.x = static_cast<const T *>(x.x);
        p.w = static_cast<const T *>(x.w);
        p.g = static_cast<const T *>(x.g);
        p.y = static_cast<T *>(x.y);
        p.xs = x.xs;
        p.gs = x.gs;
        p.ys = x.ys;
        p.heads = x.heads;
        int64_t groups = (x.heads + R - 1) / R, per = groups;
        while (per > 1 && T_ * ((groups + per - 1) / per) < warps) per = (per + 1) / 2;
        p.per = int32_t(per * R);
        const int64_t units = T_ * ((x.heads + p.per - 1) / p.per);
        const int64_t blocks = (units + pp::QKN_WARPS - 1) / pp::QKN_WARPS;
        const int64_t most = BWD ? pp::QKN_MAX_BLOCKS / 2 : (int64_t(1) << 30);
        p.blocks = x.x ? int32_t(std::min(blocks, most)) : 0;
        return p;
    };
    pp::QknPart<T> pq = side(q), pk = side(k);
    if (BWD) {                       // persistent: three blocks to an SM, shared out by the sides' rows
        const int64_t room = int64_t(sm_count) * pp::QKN_BLOCKS_BWD;
        if (int64_t(pq.blocks) + pk.blocks > room) {
            const double share = q.x ? double(q.heads) / (q.heads + (k.x ? k.heads : 0)) : 0.0;
            const int32_t bq = int32_t(std::min<int64_t>(pq.blocks, std::max<int64_t>(q.x ? 1 : 0, int64_t(room * share))));
            const int32_t bk = int32_t(std::min<int64_t>(pk.blocks, std::max<int64_t>(k.x ? 1 : 0, room - bq)));
            pq.blocks = bq;
            pk.blocks = bk;
        }
    }
    *nq = pq.blocks;
    *nk = pk.blocks;
    if (pq.blocks + pk.blocks == 0) return PP_OK;
    pp::k_qk_norm_rope<T, D, BWD><<<pq.blocks + pk.blocks, pp::QKN_WARPS * 32, 0, s>>>(pq, pk, pos, T_, eps,
                                                                                     qkn_turns(theta, D), part);
    PP_CUDA(cudaGetLastError());
    return PP_OK;
}

template <bool BWD>
pp_status qkn_call(const QknSide &q, const QknSide &k, const int32_t *pos, int64_t T, int32_t d, float eps, float theta,
                   pp_dtype dt, float *part, int32_t *nq, int32_t *nk, cudaStream_t s) {
    DeviceInfo *di;
    pp_status st = device_info(&di);
    if (st != PP_OK) return st;
    const float th = theta == 0.f ? 10000.f : theta;
    if (dt == PP_BF16)
        return d == 128 ? qkn_launch<__nv_bfloat16, 128, BWD>(q, k, pos, T, eps, th, di->sm_count, part, nq, nk, s)
                        : qkn_launch<__nv_bfloat16, 64, BWD>(q, k, pos, T, eps, th, di->sm_count, part, nq, nk, s);
    return d == 128 ? qkn_launch<float, 128, BWD>(q, k, pos, T, eps, th, di->sm_count, part, nq, nk, s)
                    : qkn_launch<float, 64, BWD>(q, k, pos, T, eps, th, di->sm_count, part, nq, nk, s);
}

// dw partials: one row of d for each block. At most one block for 8 units, a unit at least one row.
int64_t qkn_part_bytes(int64_t T, int64_t heads, int32_t d) {
    const int64_t blocks = std::min<int64_t>(pp::QKN_MAX_BLOCKS, T * heads / pp::QKN_WARPS + 2);
    return (blocks * d * 4 + 255) / 256 * 256;
}

pp_status qkn_scalars(int64_t T, int32_t hq, int32_t hkv, int32_t d, float eps, float theta, pp_dtype dt) {
    pp_status st = check_heads(T, hq, hkv, d);
    if (st != PP_OK) return st;
    if (dt != PP_BF16 && dt != PP_FP32) return fail(PP_ERR_INVALID_ARG, "unknown dtype %d", int(dt));
    if (!(theta >= 0.f) || std::isinf(theta)) return fail(PP_ERR_INVALID_ARG, "theta must be finite and >= 0");
    if (!(eps >= 0.f) || std::isinf(eps)) return fail(PP_ERR_INVALID_ARG, "eps must be finite and >= 0");
    return PP_OK;
}

// ---- paged cache
int page_log2(int32_t page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : page == 128 ? 7 : -1; }

pp_status check_pool(int32_t num_pages, int32_t page_size) {
    if (page_log2(page_size) < 0) return fail(PP_ERR_INVALID_ARG, "page_size %d not in {16, 32, 64, 128}", page_size);
    if (num_pages < 1 || int64_t(num_pages) * page_size >= (int64_t(1) << 31))
        return fail(PP_ERR_INVALID_ARG, "need num_pages >= 1 and num_pages * page_size < 2^31 (%d, %d)", num_pages,
                    page_size);
    return PP_OK;
}

pp_status check_segments(int32_t G, int32_t nseg, int64_t max_pages, int32_t page_size) {
    if (G < 1 || nseg < G) return fail(PP_ERR_INVALID_ARG, "need num_groups >= 1 and num_segments >= num_groups");
    if (nseg > pp::PAGES_MAX_SEGS)
        return fail(PP_ERR_UNSUPPORTED, "at most %d segments (got %d)", pp::PAGES_MAX_SEGS, nseg);
    if (max_pages < 1 || max_pages > (int64_t(1) << 30) / page_size)
        return fail(PP_ERR_INVALID_ARG, "need max_pages >= 1 and max_pages * page_size <= 2^30");
    return PP_OK;
}

// 3-D map over a pool's (page, head) blocks of `rows` rows of `width` bytes: keys are rows of 128 bytes, values rows of a
// page's tokens. Box = 64 tokens of a block, or all it has, swizzled by the width of the box.
pp_status make_page_map(CUtensorMap *m, const void *base, int width, int rows, int64_t blocks, bool keys) {
    EncodeTiledFn enc;
    pp_status st = get_encoder(&enc);
    if (st != PP_OK) return st;
    const int bw = keys ? width : std::min(width, 64), br = keys ? std::min(rows, 64) : rows;
    cuuint64_t dims[3] = {cuuint64_t(width), cuuint64_t(rows), cuuint64_t(blocks)};
    cuuint64_t strides[2] = {cuuint64_t(width), cuuint64_t(width) * rows};
    cuuint32_t box[3] = {cuuint32_t(bw), cuuint32_t(br), 1};
    cuuint32_t estr[3] = {1, 1, 1};
    const CUtensorMapSwizzle sw = bw == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                                  : bw == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                  : bw == 32 ? CU_TENSOR_MAP_SWIZZLE_32B
                                             : CU_TENSOR_MAP_SWIZZLE_NONE;
    CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(PP_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", int(r));
    return PP_OK;
}

template <typename T>
pp_status store_rows(const void *k, const void *v, int64_t ks, int64_t vs, const int32_t *slots, int64_t n,
                            int32_t hkv, void *kp, void *vp, float *ksc, float *vsc, bool e4m3, int32_t num_pages,
                            int32_t page_size, int sm_count, cudaStream_t s) {
    pp::CacheStoreArgs<T> a{};
    a.rows[0] = static_cast<const T *>(k);
    a.rows[1] = static_cast<const T *>(v);
    a.stride[0] = ks;
    a.stride[1] = vs;
    a.pages[0] = static_cast<uint8_t *>(kp);
    a.pages[1] = static_cast<uint8_t *>(vp);
    a.scale[0] = ksc;
    a.scale[1] = vsc;
    a.slots = slots;
    a.n = n;
    a.hkv = hkv;
    a.num_pages = num_pages;
    a.page_log2 = page_log2(page_size);
    // few rows: windows of 8 and a head to a block, so that appended tokens (a warp each) spread over the SMs (128 rows of 8
    // heads 6.5 us, with windows of a page 28.9); many: a page's worth (88,685 rows 125 us, with windows of 8 456), and as
    // many heads as leave each SM a dozen blocks, so that a block's look at the slots serves them all (with a head to a
    // block 175 us). Skipped rows count as rows here: 128 of a buffer of 4096 take 32 us.
    a.window = (n + 7) / 8 * hkv * 2 <= int64_t(sm_count) * 16 ? 8 : page_size;
    const int64_t windows = (n + a.window - 1) / a.window;
    a.heads = 1;
    while (a.window > 8 && a.heads < hkv && windows * 2 * ((hkv + 2 * a.heads - 1) / (2 * a.heads)) >= int64_t(sm_count) * 12) a.heads *= 2;
    a.parts = 2 * ((hkv + a.heads - 1) / a.heads);
    const unsigned grid = static_cast<unsigned>(windows * a.parts);
    auto pick = [&](auto units) {
        constexpr int U = decltype(units)::value;
        if (e4m3) pp::k_cache_store<T, pp::CACHE_E4M3, U><<<grid, pp::CACHE_THREADS, 0, s>>>(a);
        else pp::k_cache_store<T, pp::CACHE_INT8, U><<<grid, pp::CACHE_THREADS, 0, s>>>(a);
    };
    const int units = page_size / 4 * (pp::CACHE_D * int(sizeof(T)) / 16);       // of four tokens and 16 bytes of d
    if (units <= pp::CACHE_THREADS) pick(std::integral_constant<int, 1>{});
    else if (units <= 2 * pp::CACHE_THREADS) pick(std::integral_constant<int, 2>{});
    else pick(std::integral_constant<int, 4>{});
    PP_CUDA(cudaGetLastError());
    return PP_OK;
}

}  // namespace

// =====================================================================================================================
extern "C" {

const char *pp_last_error(void) { return g_last_error.c_str(); }

const char *pp_version(void) { return "libpp 0.1 (sm_100a)"; }

pp_status pp_meta_bounds(int32_t num_groups, int32_t num_segments, int64_t total_tokens, int32_t num_heads_q,
                         int32_t num_heads_kv, int64_t *meta_bytes) {
    if (!meta_bytes) return fail(PP_ERR_INVALID_ARG, "meta_bytes is NULL");
    if (num_groups < 1) return fail(PP_ERR_INVALID_ARG, "num_groups must be >= 1");
    if (num_segments < num_groups) return fail(PP_ERR_INVALID_ARG, "num_segments < num_groups");
    pp_status st = check_heads(total_tokens, num_heads_q, num_heads_kv, 128);
    if (st != PP_OK) return st;
    *meta_bytes = pp::meta_layout(total_tokens, num_groups, num_segments, num_heads_q, num_heads_kv).total_bytes;
    return PP_OK;
}

pp_status pp_build_meta(const pp_group_desc *groups_d, int32_t num_groups, const int32_t *cu_seqlens_d,
                        int32_t num_segments, int64_t total_tokens, int32_t num_heads_q, int32_t num_heads_kv,
                        int32_t *pos_ids_d, void *meta_d, int64_t meta_bytes, void *stream) {
    int64_t need = 0;
    pp_status st = pp_meta_bounds(num_groups, num_segments, total_tokens, num_heads_q, num_heads_kv, &need);
    if (st != PP_OK) return st;
    if (!groups_d || !cu_seqlens_d || !meta_d || (total_tokens > 0 && !pos_ids_d))
        return fail(PP_ERR_INVALID_ARG, "NULL device pointer");
    if (reinterpret_cast<uintptr_t>(meta_d) % 256) return fail(PP_ERR_INVALID_ARG, "meta_d not 256-byte aligned");
    if (meta_bytes < need)
        return fail(PP_ERR_WORKSPACE, "meta buffer %lld bytes < %lld needed", (long long)meta_bytes, (long long)need);
    DeviceInfo *di;
    if ((st = device_info(&di)) != PP_OK) return st;
    cudaStream_t s = as_stream(stream);
    const pp::MetaHeader h = pp::meta_layout(total_tokens, num_groups, num_segments, num_heads_q, num_heads_kv);
    pp::k_meta_header<<<1, 1, 0, s>>>(meta_d, h);
    PP_CUDA(cudaGetLastError());
    char *base = reinterpret_cast<char *>(meta_d);
    int32_t *qoff = reinterpret_cast<int32_t *>(base + h.off_scratch);
    int32_t *koff = qoff + (num_groups + 1);
    int32_t *tmp = koff + (num_groups + 1);
    pp::BWork *bw_tmp = reinterpret_cast<pp::BWork *>(base + h.off_bw_tmp);
    pp::k_meta_groups<1024><<<1, 1024, 0, s>>>(groups_d, cu_seqlens_d, meta_d, qoff, koff);
    PP_CUDA(cudaGetLastError());
    if (total_tokens > 0) {
        pp::k_meta_tokens<<<grid_for(di->sm_count, 4, (total_tokens + 255) / 256), 256, 0, s>>>(cu_seqlens_d, meta_d,
                                                                                                  pos_ids_d);
        PP_CUDA(cudaGetLastError());
    }
    const int64_t ntiles = h.cap_qt > h.cap_kt ? h.cap_qt : h.cap_kt;
    pp::k_meta_tiles<<<grid_for(di->sm_count, 2, (ntiles + 127) / 128), 128, 0, s>>>(meta_d, qoff, koff);
    PP_CUDA(cudaGetLastError());
    pp::k_meta_sort<1024><<<1, 1024, 0, s>>>(meta_d, tmp, bw_tmp);
    PP_CUDA(cudaGetLastError());
    return PP_OK;
}

pp_status pp_meta_tiles(const void *meta_d, int32_t which, int32_t *tiles_d, int64_t capacity, int32_t *count_d,
                        void *stream) {
    if (!meta_d || !count_d || (capacity > 0 && !tiles_d)) return fail(PP_ERR_INVALID_ARG, "NULL pointer");
    if (which != PP_PASS_FWD && which != PP_PASS_BWD) return fail(PP_ERR_INVALID_ARG, "which must be fwd or bwd");
    DeviceInfo *di;
    pp_status st = device_info(&di);
    if (st != PP_OK) return st;
    cudaStream_t s = as_stream(stream);
    PP_CUDA(cudaMemsetAsync(count_d, 0, sizeof(int32_t), s));
    pp::k_meta_expand<<<di->sm_count, 128, 0, s>>>(meta_d, which, tiles_d, capacity, count_d);
    PP_CUDA(cudaGetLastError());
    return PP_OK;
}

pp_status pp_meta_schedule(const void *meta_d, int32_t which, int32_t *records_d, int64_t capacity, int32_t *count_d,
                           void *stream) {
    if (!meta_d || !count_d || (capacity > 0 && !records_d)) return fail(PP_ERR_INVALID_ARG, "NULL pointer");
    if (which != PP_PASS_FWD && which != PP_PASS_BWD) return fail(PP_ERR_INVALID_ARG, "which must be fwd or bwd");
    DeviceInfo *di;
    pp_status st = device_info(&di);
    if (st != PP_OK) return st;
    cudaStream_t s = as_stream(stream);
    PP_CUDA(cudaMemsetAsync(count_d, 0, sizeof(int32_t), s));
    pp::k_meta_schedule<<<di->sm_count, 128, 0, s>>>(meta_d, which, records_d, capacity, count_d);
    PP_CUDA(cudaGetLastError());
    return PP_OK;
}

pp_status pp_rope(void *q, void *k, const int32_t *pos_ids_d, int64_t T, int32_t hq, int32_t hkv, int32_t d,
                  float theta, pp_dtype dt, int32_t inverse, void *stream) {
    pp_status st = check_heads(T, hq, hkv, d);
    if (st != PP_OK) return st;
    if (dt != PP_BF16 && dt != PP_FP32) return fail(PP_ERR_INVALID_ARG, "unknown dtype %d", int(dt));
    if (!(theta >= 0.f) || std::isinf(theta)) return fail(PP_ERR_INVALID_ARG, "theta must be finite and >= 0");
    if (T == 0 || (!q && !k)) return PP_OK;
    if (!pos_ids_d) return fail(PP_ERR_INVALID_ARG, "pos_ids_d is NULL");
    if ((q && reinterpret_cast<uintptr_t>(q) % 16) || (k && reinterpret_cast<uintptr_t>(k) % 16))
        return fail(PP_ERR_INVALID_ARG, "q/k must be 16-byte aligned");
    DeviceInfo *di;
    if ((st = device_info(&di)) != PP_OK) return st;
    const double th = theta == 0.f ? 10000.0 : double(theta);
    const int grid = grid_for(di->sm_count, 8, (T + pp::ROPE_TOK - 1) / pp::ROPE_TOK);
    cudaStream_t s = as_stream(stream);
    if (dt == PP_BF16)
        pp::k_rope<__nv_bfloat16><<<grid, pp::ROPE_THREADS, 0, s>>>(
            static_cast<__nv_bfloat16 *>(q), static_cast<__nv_bfloat16 *>(k), pos_ids_d, T, hq, hkv, d, std::log2(th),
            inverse);
    else
        pp::k_rope<float><<<grid, pp::ROPE_THREADS, 0, s>>>(static_cast<float *>(q), static_cast<float *>(k),
                                                             pos_ids_d, T, hq, hkv, d, std::log2(th), inverse);
    PP_CUDA(cudaGetLastError());
    return PP_OK;
}

pp_status pp_workspace_bytes(int32_t which, int64_t T, int32_t hq, int32_t hkv, int32_t d, int64_t *bytes) {
    if (!bytes) return fail(PP_ERR_INVALID_ARG, "bytes is NULL");
    pp_status st = check_heads(T, hq, hkv, d);
    if (st != PP_OK) return st;
    if (which == PP_PASS_FWD) {
        *bytes = 256;
    } else if (which == PP_PASS_BWD) {
        *bytes = pp::bwd_workspace_layout(T, hq, hkv, d).total;
    } else {
        return fail(PP_ERR_INVALID_ARG, "which must be fwd or bwd");
    }
    return PP_OK;
}

pp_status pp_bwd_ds_bytes(const pp_group_desc *groups_host, int32_t G, const int32_t *cu_host, int32_t nseg,
                          int32_t hq, int32_t hkv, int64_t *bytes) {
    if (!groups_host || !cu_host || !bytes) return fail(PP_ERR_INVALID_ARG, "NULL pointer argument");
    if (G < 0 || nseg < 0 || hq <= 0 || hkv <= 0 || hq % hkv != 0)
        return fail(PP_ERR_INVALID_ARG, "need G, num_segments >= 0 and hq a multiple of hkv");
    const int64_t r = hq / hkv;
    // one step per (key tile, attending query tile, q head): key tile b of a group of length L, prefix P, covers
    // keys [128 b, 128 b + 128); its queries run from its own first row to e = L for a prefix tile, else to the end
    // of the segment of its last key (the same rule as the schedule builder's)
    int64_t steps = 0;
    int32_t s = 0;
    for (int32_t g = 0; g < G; ++g) {
        const int32_t P = groups_host[g].prefix_len, k = groups_host[g].num_suffixes;
        if (k < 0 || P < 0 || s + 1 + int64_t(k) > nseg) return fail(PP_ERR_INVALID_ARG, "descriptors exceed num_segments");
        for (int32_t j = s; j <= s + k; ++j)
            if (cu_host[j + 1] < cu_host[j]) return fail(PP_ERR_INVALID_ARG, "segment bounds must not decrease");
        const int32_t start = cu_host[s], end = cu_host[s + 1 + k];
        const int32_t L = end - start;
        if (cu_host[s + 1] - start != P) return fail(PP_ERR_INVALID_ARG, "prefix length disagrees with segments");
        int32_t seg = s + 1;                                        // segment of the current key (responses)
        for (int32_t y0 = 0; y0 < L; y0 += pp::BWD_BN) {
            const int32_t ylast = std::min(y0 + pp::BWD_BN, L) - 1;
            int32_t e = L;
            if (y0 >= P) {
                while (seg < s + 1 + k && cu_host[seg + 1] - start <= ylast) ++seg;
                e = cu_host[seg + 1] - start;
            }
            const int64_t qa = y0 / pp::BWD_BM, qb = (e + pp::BWD_BM - 1) / pp::BWD_BM;
            steps += (qb - qa) * r * hkv;                          // every q head of every kv head
        }
        s += 1 + k;
    }
    if (s != nseg) return fail(PP_ERR_INVALID_ARG, "num_segments must equal sum_g (1 + k_g)");
    *bytes = pp::BWD_DS_ALIGN + steps * pp::BWD_DS_TILE_BYTES;
    return PP_OK;
}

// Exact (chunk, query) pair count of the decode plan, from host copies of the descriptors and segment bounds.
static pp_status decode_pairs(const pp_group_desc *groups, int32_t G, const int32_t *cu, int32_t nseg, int64_t *pairs) {
    int64_t np = 0;
    int32_t s = 0;
    auto nch = [&](int32_t seg) -> int64_t {
        const int64_t len = int64_t(cu[seg + 1]) - cu[seg];
        return len > 0 ? (len + pp::DEC_CH - 1) / pp::DEC_CH : 0;
    };
    for (int32_t g = 0; g < G; ++g) {
        const int32_t k = groups[g].num_suffixes;
        if (k < 0 || s + 1 + int64_t(k) > nseg) return fail(PP_ERR_INVALID_ARG, "descriptors exceed num_segments");
        np += nch(s) * k;
        for (int32_t i = 0; i < k; ++i) np += nch(s + 1 + i);
        s += 1 + k;
    }
    if (s != nseg) return fail(PP_ERR_INVALID_ARG, "num_segments must equal sum_g (1 + k_g)");
    *pairs = np;
    return PP_OK;
}

pp_status pp_decode_workspace_bytes(const pp_group_desc *groups_host, int32_t G, const int32_t *cu_host, int32_t nseg,
                                    int32_t hq, int64_t *bytes) {
    if (!groups_host || !cu_host || !bytes) return fail(PP_ERR_INVALID_ARG, "NULL pointer argument");
    if (G < 1 || nseg < G || hq < 1) return fail(PP_ERR_INVALID_ARG, "need G >= 1, num_segments >= G, hq >= 1");
    int64_t np;
    pp_status st = decode_pairs(groups_host, G, cu_host, nseg, &np);
    if (st != PP_OK) return st;
    *bytes = pp::dec_plan_layout(cu_host[nseg], G, nseg, hq, np).total;
    return PP_OK;
}

pp_status pp_decode_attn(const void *q, const void *k_cache, const void *v_cache, const pp_group_desc *groups_d,
                         int32_t G, const int32_t *cu_d, int32_t nseg, int64_t T, int32_t hq, int32_t hkv, int32_t d,
                         float softmax_scale, void *o, float *lse, void *workspace, int64_t ws_bytes, void *stream) {
    pp_status st = check_heads(T, hq, hkv, d);
    if (st != PP_OK) return st;
    if (d != pp::DEC_D) return fail(PP_ERR_UNSUPPORTED, "decode supports head dim 128 only (got %d)", d);
    if (G < 1 || nseg < G) return fail(PP_ERR_INVALID_ARG, "need G >= 1 and num_segments >= G");
    const int32_t n_resp = nseg - G;
    if (n_resp == 0) return PP_OK;
    if (!q || !k_cache || !v_cache || !groups_d || !cu_d || !o || !lse || !workspace)
        return fail(PP_ERR_INVALID_ARG, "NULL pointer argument");
    const void *ptrs[4] = {q, k_cache, v_cache, o};
    for (const void *ptr : ptrs)
        if (reinterpret_cast<uintptr_t>(ptr) % 16) return fail(PP_ERR_INVALID_ARG, "q, k, v, o must be 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(workspace) % 256) return fail(PP_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    if (!(softmax_scale >= 0.f) || std::isinf(softmax_scale)) return fail(PP_ERR_INVALID_ARG, "bad softmax_scale");
    const int r = hq / hkv;
    if (r > 128) return fail(PP_ERR_UNSUPPORTED, "decode supports at most 128 q heads per kv head (got %d)", r);
    const int rb = 128 / r;                                  // responses per query block (r * rb <= 128 rows)
    const pp::DecPlan base = pp::dec_plan_layout(T, G, nseg, hq, 0);
    const int64_t rec = 4 * int64_t(hq) * pp::DEC_REC + 32;   // one record per q head, and one job entry
    if (ws_bytes < base.total + rec) return fail(PP_ERR_WORKSPACE, "workspace too small for the decode plan");
    int64_t mp = (ws_bytes - base.total) / rec;               // upper bound; trimmed for the sections' alignment
    while (mp > 0 && pp::dec_plan_layout(T, G, nseg, hq, mp).total > ws_bytes) --mp;
    const pp::DecPlan p = pp::dec_plan_layout(T, G, nseg, hq, mp);
    DeviceInfo *di;
    if ((st = device_info(&di)) != PP_OK) return st;
    CUtensorMap mq, mk, mv;
    if ((st = make_map_3d_box(&mq, q, n_resp, hq, d, r, rb)) != PP_OK) return st;
    if ((st = make_map_3d(&mk, k_cache, T, hkv, d, pp::DEC_CH)) != PP_OK) return st;
    if ((st = make_map_3d(&mv, v_cache, T, hkv, d, pp::DEC_CH)) != PP_OK) return st;
    const float scale = softmax_scale == 0.f ? 1.f / std::sqrt(float(d)) : softmax_scale;
    cudaStream_t s = as_stream(stream);
    const int32_t *gd = reinterpret_cast<const int32_t *>(groups_d);
    pp::k_dec_plan<<<1, 1024, 0, s>>>(gd, G, cu_d, nseg, T, rb, workspace, p);
    PP_CUDA(cudaGetLastError());
    const int smem = int(sizeof(pp::DecSmem)) + 1024;
    PP_CUDA(cudaFuncSetAttribute(pp::k_dec_chunk, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    pp::k_dec_chunk<<<di->sm_count, pp::DEC_THREADS, smem, s>>>(mq, mk, mv, hq, hkv, rb, n_resp,
                                                                  scale * 1.4426950408889634f, workspace, p);
    PP_CUDA(cudaGetLastError());
    pp::k_dec_combine<<<grid_for(di->sm_count, 3, (int64_t(n_resp) * hq + pp::DEC_COMB_WARPS - 1) / pp::DEC_COMB_WARPS),
                        pp::DEC_COMB_WARPS * 32, 0, s>>>(hq, n_resp, workspace, p, static_cast<__nv_bfloat16 *>(o), lse);
    PP_CUDA(cudaGetLastError());
    return PP_OK;
}

pp_status pp_pack_batch(const int32_t *prompts, const uint8_t *prompt_mask, int32_t Lp, const int32_t *responses,
                        const uint8_t *response_mask, int32_t Lr, const int64_t *uids, int32_t bs,
                        int32_t *packed_ids, int64_t capacity, pp_group_desc *groups, int32_t *cu_seqlens,
                        int32_t *sample_offsets, int32_t *counts, void *stream) {
    if (bs < 0 || bs > pp::PACK_MAX_BATCH)
        return fail(bs < 0 ? PP_ERR_INVALID_ARG : PP_ERR_UNSUPPORTED, "bs must be in [0, %d] (got %d)",
                    pp::PACK_MAX_BATCH, bs);
    if (Lp < 0 || Lr < 0) return fail(PP_ERR_INVALID_ARG, "negative row length");
    const int64_t worst = int64_t(bs) * (int64_t(Lp) + Lr);
    if (worst >= (int64_t(1) << 31)) return fail(PP_ERR_INVALID_ARG, "bs * (Lp + Lr) must fit int32");
    if (capacity < worst) return fail(PP_ERR_INVALID_ARG, "packed_ids capacity %lld < bs * (Lp + Lr) = %lld",
                                      (long long)capacity, (long long)worst);
    if (!cu_seqlens || !counts) return fail(PP_ERR_INVALID_ARG, "NULL pointer argument");
    cudaStream_t s = as_stream(stream);
    if (bs == 0) {
        PP_CUDA(cudaMemsetAsync(counts, 0, 3 * sizeof(int32_t), s));
        PP_CUDA(cudaMemsetAsync(cu_seqlens, 0, sizeof(int32_t), s));
        return PP_OK;
    }
    if (!uids || !groups || !sample_offsets || (worst > 0 && !packed_ids) || (Lp > 0 && (!prompts || !prompt_mask)) ||
        (Lr > 0 && (!responses || !response_mask)))
        return fail(PP_ERR_INVALID_ARG, "NULL pointer argument");
    DeviceInfo *di;
    pp_status st;
    if ((st = device_info(&di)) != PP_OK) return st;
    pp::k_pack_count<<<bs, pp::PACK_THREADS, 0, s>>>(prompt_mask, Lp, response_mask, Lr, sample_offsets);
    PP_CUDA(cudaGetLastError());
    const int smem = 4 * bs * int(sizeof(int32_t));
    PP_CUDA(cudaFuncSetAttribute(pp::k_pack_layout, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    pp::k_pack_layout<<<1, pp::PACK_LAYOUT_THREADS, smem, s>>>(uids, bs, sample_offsets,
                                                               reinterpret_cast<int32_t *>(groups), cu_seqlens,
                                                               counts);
    PP_CUDA(cudaGetLastError());
    pp::k_pack_gather<<<bs, pp::PACK_THREADS, 0, s>>>(prompts, prompt_mask, Lp, responses, response_mask, Lr,
                                                      sample_offsets, packed_ids);
    PP_CUDA(cudaGetLastError());
    return PP_OK;
}

pp_status pp_response_logprobs(const void *logits, pp_dtype dt, int64_t V, const int32_t *token_ids,
                               const void *meta_d, int64_t T, float temperature, float *out, void *stream) {
    if (T < 0 || T >= (int64_t(1) << 31)) return fail(PP_ERR_INVALID_ARG, "T out of range (%lld)", (long long)T);
    if (V < 1) return fail(PP_ERR_INVALID_ARG, "V must be >= 1 (got %lld)", (long long)V);
    if (dt != PP_BF16 && dt != PP_FP32) return fail(PP_ERR_INVALID_ARG, "unknown dtype %d", int(dt));
    if (!(temperature > 0.f) || std::isinf(temperature))
        return fail(PP_ERR_INVALID_ARG, "temperature must be finite and > 0");
    if (T == 0) return PP_OK;
    if (!logits || !token_ids || !meta_d || !out) return fail(PP_ERR_INVALID_ARG, "NULL pointer argument");
    if (reinterpret_cast<uintptr_t>(logits) % (dt == PP_BF16 ? 2 : 4))
        return fail(PP_ERR_INVALID_ARG, "logits must be aligned to their element size");
    DeviceInfo *di;
    pp_status st;
    if ((st = device_info(&di)) != PP_OK) return st;
    const int grid = grid_for(di->sm_count, 8, T);
    const float inv_temp = 1.f / temperature;
    const float c2 = float(1.4426950408889634 / double(temperature));
    cudaStream_t s = as_stream(stream);
    if (dt == PP_BF16)
        pp::k_response_logprobs<__nv_bfloat16><<<grid, pp::LP_THREADS, 0, s>>>(
            static_cast<const __nv_bfloat16 *>(logits), V, token_ids, meta_d, c2, inv_temp, out);
    else
        pp::k_response_logprobs<float><<<grid, pp::LP_THREADS, 0, s>>>(static_cast<const float *>(logits), V,
                                                                       token_ids, meta_d, c2, inv_temp, out);
    PP_CUDA(cudaGetLastError());
    return PP_OK;
}

pp_status pp_attn_fwd(const void *q, const void *k, const void *v, const void *meta_d, int64_t T, int32_t hq,
                      int32_t hkv, int32_t d, float softmax_scale, pp_dtype dt, void *o, float *lse,
                      void *workspace, int64_t ws_bytes, void *stream) {
    pp_status st = check_heads(T, hq, hkv, d);
    if (st != PP_OK) return st;
    if (T == 0) return PP_OK;
    if (!q || !k || !v || !meta_d || !o || !lse) return fail(PP_ERR_INVALID_ARG, "NULL pointer");
    if (dt != PP_BF16 && dt != PP_FP32) return fail(PP_ERR_INVALID_ARG, "unknown dtype %d", int(dt));
    int64_t need = 0;
    pp_workspace_bytes(PP_PASS_FWD, T, hq, hkv, d, &need);
    if (ws_bytes < need || !workspace) return fail(PP_ERR_WORKSPACE, "forward workspace too small");
    if (!(softmax_scale >= 0.f) || std::isinf(softmax_scale)) return fail(PP_ERR_INVALID_ARG, "bad softmax_scale");
    const float scale = softmax_scale == 0.f ? 1.f / std::sqrt(float(d)) : softmax_scale;
    DeviceInfo *di;
    if ((st = device_info(&di)) != PP_OK) return st;
    cudaStream_t s = as_stream(stream);
    if (dt == PP_FP32) {
        const size_t smem = size_t(2) * pp::FWD_BN * d * sizeof(float);
        const int64_t work = (T / pp::FWD_BM + 1024) * hq;
        if (d == 64) {
            PP_CUDA(cudaFuncSetAttribute(pp::k_attn_fwd_simt<float, 64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         int(smem)));
            pp::k_attn_fwd_simt<float, 64><<<grid_for(di->sm_count, 2, work), 128, smem, s>>>(
                static_cast<const float *>(q), static_cast<const float *>(k), static_cast<const float *>(v), meta_d,
                static_cast<float *>(o), lse, hq, hkv, scale);
        } else {
            PP_CUDA(cudaFuncSetAttribute(pp::k_attn_fwd_simt<float, 128>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)));
            pp::k_attn_fwd_simt<float, 128><<<grid_for(di->sm_count, 1, work), 128, smem, s>>>(
                static_cast<const float *>(q), static_cast<const float *>(k), static_cast<const float *>(v), meta_d,
                static_cast<float *>(o), lse, hq, hkv, scale);
        }
        PP_CUDA(cudaGetLastError());
        return PP_OK;
    }
    CUtensorMap mq, mk, mv;
    if ((st = make_map_3d(&mq, q, T, hq, d, pp::FWD_BM)) != PP_OK) return st;
    if ((st = make_map_3d(&mk, k, T, hkv, d, pp::FWD_BN)) != PP_OK) return st;
    if ((st = make_map_3d(&mv, v, T, hkv, d, pp::FWD_BN)) != PP_OK) return st;
    if (reinterpret_cast<uintptr_t>(o) % 16) return fail(PP_ERR_INVALID_ARG, "o must be 16-byte aligned");
    const float sl2 = scale * 1.4426950408889634f;
    const int grid = di->sm_count;
    if (d == 128) {
        const size_t smem = sizeof(pp::FwdSmem<128>) + 1024;
        PP_CUDA(cudaFuncSetAttribute(pp::k_attn_fwd_tc<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)));
        pp::k_attn_fwd_tc<128><<<grid, pp::FWD_THREADS, smem, s>>>(mq, mk, mv, meta_d,
                                                                     static_cast<__nv_bfloat16 *>(o), lse, hq, hkv, sl2);
    } else {
        const size_t smem = sizeof(pp::FwdSmem<64>) + 1024;
        PP_CUDA(cudaFuncSetAttribute(pp::k_attn_fwd_tc<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)));
        pp::k_attn_fwd_tc<64><<<grid, pp::FWD_THREADS, smem, s>>>(mq, mk, mv, meta_d,
                                                                   static_cast<__nv_bfloat16 *>(o), lse, hq, hkv, sl2);
    }
    PP_CUDA(cudaGetLastError());
    return PP_OK;
}

pp_status pp_attn_bwd(const void *q, const void *k, const void *v, const void *o, const float *lse,
                      const void *dout, const void *meta_d, int64_t T, int32_t hq, int32_t hkv, int32_t d,
                      float softmax_scale, void *dq, void *dk, void *dv, void *workspace, int64_t ws_bytes,
                      void *stream) {
    pp_status st = check_heads(T, hq, hkv, d);
    if (st != PP_OK) return st;
    if (T == 0) return PP_OK;
    if (!q || !k || !v || !o || !lse || !dout || !meta_d || !dq || !dk || !dv)
        return fail(PP_ERR_INVALID_ARG, "NULL pointer");
    int64_t need = 0;
    pp_workspace_bytes(PP_PASS_BWD, T, hq, hkv, d, &need);
    if (ws_bytes < need || !workspace) return fail(PP_ERR_WORKSPACE, "backward workspace %lld < %lld bytes",
                                                   (long long)ws_bytes, (long long)need);
    if (reinterpret_cast<uintptr_t>(workspace) % 256) return fail(PP_ERR_INVALID_ARG, "workspace not 256-aligned");
    if (!(softmax_scale >= 0.f) || std::isinf(softmax_scale)) return fail(PP_ERR_INVALID_ARG, "bad softmax_scale");
    const float scale = softmax_scale == 0.f ? 1.f / std::sqrt(float(d)) : softmax_scale;
    DeviceInfo *di;
    if ((st = device_info(&di)) != PP_OK) return st;
    return pp::launch_bwd(q, k, v, o, lse, dout, meta_d, T, hq, hkv, d, scale, dq, dk, dv, workspace, ws_bytes,
                          di->sm_count, as_stream(stream), make_map_3d, make_map_3d_box, fail);
}

pp_status pp_attn_bwd_noalloc(const void *q, const void *k, const void *v, const void *o, const float *lse,
                              const void *dout, const void *meta_d, int64_t T, int32_t hq, int32_t hkv, int32_t d,
                              float softmax_scale, void *dq, void *dk, void *dv, void *stream) {
    pp_status st = check_heads(T, hq, hkv, d);
    if (st != PP_OK) return st;
    int64_t need = 0;
    if ((st = pp_workspace_bytes(PP_PASS_BWD, T, hq, hkv, d, &need)) != PP_OK) return st;
    if (need > PP_NOALLOC_SCRATCH_BYTES)
        return fail(PP_ERR_WORKSPACE,
                    "pp_attn_bwd_noalloc: these sizes need %lld bytes of scratch but the built-in array holds %lld; "
                    "call pp_attn_bwd with a caller workspace instead",
                    (long long)need, (long long)PP_NOALLOC_SCRATCH_BYTES);
    if (T == 0) return PP_OK;
    void *scratch = nullptr;
    if ((st = noalloc_scratch(&scratch)) != PP_OK) return st;
    return pp_attn_bwd(q, k, v, o, lse, dout, meta_d, T, hq, hkv, d, softmax_scale, dq, dk, dv, scratch,
                       PP_NOALLOC_SCRATCH_BYTES, stream);
}

pp_status pp_qk_norm_rope(const void *q, const void *k, int64_t q_stride, int64_t k_stride, const void *wq,
                          const void *wk, const int32_t *pos_ids_d, int64_t T, int32_t hq, int32_t hkv, int32_t d,
                          float eps, float theta, pp_dtype dt, void *q_out, void *k_out, int64_t qo_stride,
                          int64_t ko_stride, void *stream) {
    pp_status st = qkn_scalars(T, hq, hkv, d, eps, theta, dt);
    if (st != PP_OK) return st;
    if (T == 0 || (!q && !k)) return PP_OK;
    if (!pos_ids_d) return fail(PP_ERR_INVALID_ARG, "pos_ids_d is NULL");
    if (bad_words(pos_ids_d)) return fail(PP_ERR_INVALID_ARG, "pos_ids_d must be 4-byte aligned");
    const int64_t es = dt == PP_BF16 ? 2 : 4;
    const QknSide sq{q, wq, nullptr, q_out, q_stride, 0, qo_stride, hq}, sk{k, wk, nullptr, k_out, k_stride, 0, ko_stride, hkv};
    if ((st = qkn_check(sq, d, es, false, "q")) != PP_OK || (st = qkn_check(sk, d, es, false, "k")) != PP_OK) return st;
    int32_t nq, nk;
    return qkn_call<false>(sq, sk, pos_ids_d, T, d, eps, theta, dt, nullptr, &nq, &nk, as_stream(stream));
}

pp_status pp_qk_norm_rope_bwd_bytes(int64_t T, int32_t hq, int32_t hkv, int32_t d, int64_t *bytes) {
    if (!bytes) return fail(PP_ERR_INVALID_ARG, "bytes is NULL");
    pp_status st = check_heads(T, hq, hkv, d);
    if (st != PP_OK) return st;
    *bytes = qkn_part_bytes(T, int64_t(hq) + hkv, d);
    return PP_OK;
}

pp_status pp_qk_norm_rope_bwd(const void *q, const void *k, int64_t q_stride, int64_t k_stride, const void *wq,
                              const void *wk, const int32_t *pos_ids_d, int64_t T, int32_t hq, int32_t hkv, int32_t d,
                              float eps, float theta, pp_dtype dt, const void *gq, const void *gk, int64_t gq_stride,
                              int64_t gk_stride, void *dq, void *dk, int64_t dq_stride, int64_t dk_stride, float *dwq,
                              float *dwk, void *workspace, int64_t ws_bytes, void *stream) {
    pp_status st = qkn_scalars(T, hq, hkv, d, eps, theta, dt);
    if (st != PP_OK) return st;
    cudaStream_t s = as_stream(stream);
    const int64_t es = dt == PP_BF16 ? 2 : 4;
    const QknSide sq{q, wq, gq, dq, q_stride, gq_stride, dq_stride, hq}, sk{k, wk, gk, dk, k_stride, gk_stride, dk_stride, hkv};
    if (T > 0) {
        if ((q || k) && !pos_ids_d) return fail(PP_ERR_INVALID_ARG, "pos_ids_d is NULL");
        if (bad_words(pos_ids_d)) return fail(PP_ERR_INVALID_ARG, "pos_ids_d must be 4-byte aligned");
        if ((st = qkn_check(sq, d, es, true, "q")) != PP_OK || (st = qkn_check(sk, d, es, true, "k")) != PP_OK) return st;
    }
    const int64_t need = qkn_part_bytes(T, int64_t(q ? hq : 0) + (k ? hkv : 0), d);
    if (!workspace || ws_bytes < need)
        return fail(PP_ERR_WORKSPACE, "workspace %lld < %lld bytes", (long long)ws_bytes, (long long)need);
    if (bad_align(workspace, 256)) return fail(PP_ERR_INVALID_ARG, "workspace not 256-byte aligned");
    if (bad_words(dwq, dwk)) return fail(PP_ERR_INVALID_ARG, "dwq and dwk must be 4-byte aligned");
    int32_t nq = 0, nk = 0;
    float *part = static_cast<float *>(workspace);
    if (T > 0 && (q || k) && (st = qkn_call<true>(sq, sk, pos_ids_d, T, d, eps, theta, dt, part, &nq, &nk, s)) != PP_OK)
        return st;
    if (dwq || dwk) {                // with no rows of a side its sum is 0
        const float *sums = part;
        if (nq + nk > 0) return launch_second(pp::k_qk_norm_dw, dim3(d / 32, 2), 1024, s, sums, int(d), int(nq), int(nk), dwq, dwk);
        pp::k_qk_norm_dw<<<dim3(d / 32, 2), 1024, 0, s>>>(sums, d, 0, 0, dwq, dwk);
        PP_CUDA(cudaGetLastError());
    }
    return PP_OK;
}

pp_status pp_pages_resize(const int32_t *group_start_d, int32_t G, const int32_t *seg_group_d, int32_t nseg,
                          const int32_t *old_lens_d, const int32_t *new_lens_d, int32_t page_size,
                          int32_t *page_table_d, int64_t max_pages, int32_t *free_pages_d, int32_t num_pages,
                          const int32_t *n_free_in, int32_t *n_free_out, int32_t *slots_d, int32_t *pos_ids_d,
                          int64_t capacity, int32_t *counts_d, void *stream) {
    pp_status st = check_pool(num_pages, page_size);
    if (st != PP_OK) return st;
    if ((st = check_segments(G, nseg, max_pages, page_size)) != PP_OK) return st;
    if (capacity < 0 || capacity >= (int64_t(1) << 31)) return fail(PP_ERR_INVALID_ARG, "capacity out of range");
    if (!group_start_d || !seg_group_d || !old_lens_d || !new_lens_d || !page_table_d || !free_pages_d || !n_free_in ||
        !n_free_out || !counts_d || (capacity > 0 && (!slots_d || !pos_ids_d)))
        return fail(PP_ERR_INVALID_ARG, "NULL pointer argument");
    if (bad_words(group_start_d, seg_group_d, old_lens_d, new_lens_d, page_table_d, free_pages_d, n_free_in, n_free_out, slots_d,
                  pos_ids_d, counts_d))
        return fail(PP_ERR_INVALID_ARG, "int32 arrays must be 4-byte aligned");
    DeviceInfo *di;
    if ((st = device_info(&di)) != PP_OK) return st;
    const pp::PagesArgs a{group_start_d, seg_group_d, old_lens_d, new_lens_d, page_table_d, free_pages_d, n_free_in,
                          n_free_out, slots_d, pos_ids_d, counts_d, max_pages, capacity, G, nseg, page_log2(page_size),
                          num_pages};
    const int smem = 3 * (nseg + 1) * int(sizeof(int32_t));
    static std::atomic<uint64_t> allowed{0};
    if ((st = allow_smem(pp::k_pages_resize, 3 * (pp::PAGES_MAX_SEGS + 1) * int(sizeof(int32_t)), &allowed)) != PP_OK) return st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 8;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(at[0].val.clusterDim.x);
    cfg.blockDim = dim3(pp::PAGES_THREADS);
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = as_stream(stream);
    cfg.attrs = at;
    cfg.numAttrs = 1;
    PP_CUDA(cudaLaunchKernelEx(&cfg, pp::k_pages_resize, a));
    return PP_OK;
}

pp_status pp_cache_store(const void *k, const void *v, int64_t k_stride, int64_t v_stride, pp_dtype dt,
                         const int32_t *slots_d, int64_t n, int32_t hkv, int32_t d, void *k_pages, void *v_pages,
                         float *k_scale, float *v_scale, pp_dtype codes, int32_t num_pages, int32_t page_size,
                         void *stream) {
    pp_status st = check_heads(n, hkv, hkv, d);
    if (st != PP_OK) return st;
    if (d != pp::CACHE_D) return fail(PP_ERR_UNSUPPORTED, "the paged cache supports head dim 128 only (got %d)", d);
    if (dt != PP_BF16 && dt != PP_FP32) return fail(PP_ERR_INVALID_ARG, "unknown dtype %d", int(dt));
    if (codes != PP_E4M3 && codes != PP_INT8) return fail(PP_ERR_INVALID_ARG, "codes must be PP_E4M3 or PP_INT8");
    if ((st = check_pool(num_pages, page_size)) != PP_OK) return st;
    if (n == 0) return PP_OK;
    if (!k || !v || !slots_d || !k_pages || !v_pages || !k_scale || !v_scale)
        return fail(PP_ERR_INVALID_ARG, "NULL pointer argument");
    const int64_t es = dt == PP_BF16 ? 2 : 4;
    if (k_stride < int64_t(hkv) * d || v_stride < int64_t(hkv) * d)
        return fail(PP_ERR_INVALID_ARG, "row stride below hkv * d");
    if (bad_align(k) || bad_align(v) || bad_align(k_pages) || bad_align(v_pages) || k_stride * es % 16 || v_stride * es % 16)
        return fail(PP_ERR_INVALID_ARG, "k, v, pages and row strides must be multiples of 16 bytes");
    if (bad_words(slots_d, k_scale, v_scale)) return fail(PP_ERR_INVALID_ARG, "slots_d and scales must be 4-byte aligned");
    DeviceInfo *di;
    if ((st = device_info(&di)) != PP_OK) return st;
    auto go = dt == PP_BF16 ? store_rows<__nv_bfloat16> : store_rows<float>;
    return go(k, v, k_stride, v_stride, slots_d, n, hkv, k_pages, v_pages, k_scale, v_scale, codes == PP_E4M3, num_pages,
              page_size, di->sm_count, as_stream(stream));
}

pp_status pp_paged_decode_bytes(int32_t n_resp, int32_t hq, int32_t hkv, int64_t *bytes) {
    if (!bytes) return fail(PP_ERR_INVALID_ARG, "bytes is NULL");
    pp_status st = check_heads(0, hq, hkv, 128);
    if (st != PP_OK) return st;
    if (n_resp < 0 || n_resp > pp::PAGES_MAX_SEGS) return fail(PP_ERR_INVALID_ARG, "n_resp out of range (%d)", n_resp);
    *bytes = pp::paged_workspace(n_resp, hq).total;
    return PP_OK;
}

pp_status pp_paged_decode(const void *q, const void *k_pages, const void *v_pages, const float *k_scale,
                          const float *v_scale, pp_dtype codes, int32_t num_pages, int32_t page_size,
                          const int32_t *group_start_d, int32_t G, const int32_t *seg_group_d, int32_t nseg,
                          const int32_t *lens_d, const int32_t *page_table_d, int64_t max_pages, int32_t hq,
                          int32_t hkv, int32_t d, float softmax_scale, void *o, float *lse, void *workspace,
                          int64_t ws_bytes, void *stream) {
    pp_status st = check_heads(0, hq, hkv, d);
    if (st != PP_OK) return st;
    if (d != pp::CACHE_D) return fail(PP_ERR_UNSUPPORTED, "the paged cache supports head dim 128 only (got %d)", d);
    if (codes != PP_E4M3 && codes != PP_INT8) return fail(PP_ERR_INVALID_ARG, "codes must be PP_E4M3 or PP_INT8");
    if ((st = check_pool(num_pages, page_size)) != PP_OK) return st;
    if (int64_t(num_pages) * hkv >= (int64_t(1) << 31))
        return fail(PP_ERR_UNSUPPORTED, "num_pages * hkv must be below 2^31");
    if ((st = check_segments(G, nseg, max_pages, page_size)) != PP_OK) return st;
    if (!(softmax_scale >= 0.f) || std::isinf(softmax_scale)) return fail(PP_ERR_INVALID_ARG, "bad softmax_scale");
    const int32_t n_resp = nseg - G;
    if (n_resp == 0) return PP_OK;
    if (!q || !k_pages || !v_pages || !k_scale || !v_scale || !group_start_d || !seg_group_d || !lens_d ||
        !page_table_d || !o || !lse)
        return fail(PP_ERR_INVALID_ARG, "NULL pointer argument");
    if (bad_align(q) || bad_align(k_pages) || bad_align(v_pages) || bad_align(o))
        return fail(PP_ERR_INVALID_ARG, "q, pages and o must be 16-byte aligned");
    if (bad_words(k_scale, v_scale, group_start_d, seg_group_d, lens_d, page_table_d, lse))
        return fail(PP_ERR_INVALID_ARG, "scales, descriptors, lens_d, page_table_d and lse must be 4-byte aligned");
    int64_t need = 0;
    if ((st = pp_paged_decode_bytes(n_resp, hq, hkv, &need)) != PP_OK) return st;
    if (!workspace || ws_bytes < need)
        return fail(PP_ERR_WORKSPACE, "workspace %lld < %lld bytes", (long long)ws_bytes, (long long)need);
    if (bad_align(workspace, 256)) return fail(PP_ERR_INVALID_ARG, "workspace not 256-byte aligned");
    DeviceInfo *di;
    if ((st = device_info(&di)) != PP_OK) return st;
    const float scale = softmax_scale == 0.f ? 1.f / std::sqrt(float(d)) : softmax_scale;
    const int32_t lg = page_log2(page_size);
    const pp::PagedWorkspace w = pp::paged_workspace(n_resp, hq);
    char *ws = static_cast<char *>(workspace);
    const pp::PagedArgs a{static_cast<const __nv_bfloat16 *>(q), static_cast<const uint8_t *>(k_pages),
                          static_cast<const uint8_t *>(v_pages), k_scale, v_scale, group_start_d, seg_group_d, lens_d,
                          page_table_d, static_cast<__nv_bfloat16 *>(o), lse, reinterpret_cast<pp::PagedSegRec *>(ws + w.off_seg),
                          reinterpret_cast<int4 *>(ws),
                          reinterpret_cast<float2 *>(ws + w.off_ml), reinterpret_cast<float *>(ws + w.off_part),
                          int32_t(max_pages), G, nseg, hq, hkv, hq / hkv, 65536 / (hq / hkv) + 1, num_pages, lg, scale * 1.4426950408889634f,
                          1.f / float(hq / hkv)};
    CUtensorMap mk, mv;
    if ((st = make_page_map(&mk, k_pages, 128, page_size, int64_t(num_pages) * hkv, true)) != PP_OK) return st;
    if ((st = make_page_map(&mv, v_pages, page_size, 128, int64_t(num_pages) * hkv, false)) != PP_OK) return st;
    cudaStream_t s = as_stream(stream);
    auto kernel = codes == PP_E4M3 ? pp::k_paged_decode<pp::CACHE_E4M3> : pp::k_paged_decode<pp::CACHE_INT8>;
    const int smem = int(sizeof(pp::PagedSmem)) + 1024, grid = std::min(di->sm_count, pp::PD_MAX_CTAS);
    static std::atomic<uint64_t> allowed[2] = {};
    if ((st = allow_smem(kernel, smem, &allowed[codes == PP_E4M3])) != PP_OK) return st;
    kernel<<<grid, pp::PD_THREADS, smem, s>>>(mk, mv, a);
    PP_CUDA(cudaGetLastError());
    const bool alone = int64_t(n_resp) * hq > pp::PD_COMB_ALONE;
    const dim3 rows(nseg, alone ? (hq + pp::PD_COMB_WARPS - 1) / pp::PD_COMB_WARPS : hq);
    return launch_second(alone ? pp::k_paged_combine<true> : pp::k_paged_combine<false>, rows, pp::PD_COMB_WARPS * 32, s, a);
}

pp_status pp_selftest_bounded_wait(int64_t limit_ns, unsigned long long *waited_ns_d, void *stream) {
    if (limit_ns < 1000 || limit_ns > 2000000000ll)
        return fail(PP_ERR_INVALID_ARG, "limit_ns must be in [1e3, 2e9] (got %lld)", (long long)limit_ns);
    if (!waited_ns_d) return fail(PP_ERR_INVALID_ARG, "waited_ns_d is NULL");
    DeviceInfo *di;
    pp_status st = device_info(&di);
    if (st != PP_OK) return st;
    pp::k_selftest_wait<<<1, 32, 0, as_stream(stream)>>>(uint64_t(limit_ns), waited_ns_d);
    PP_CUDA(cudaGetLastError());
    return PP_OK;
}

pp_status pp_get_status(void *stream) {
    cudaError_t e = cudaStreamSynchronize(as_stream(stream));
    if (e != cudaSuccess) return fail(PP_ERR_CUDA, "stream synchronize: %s", cudaGetErrorString(e));
    int32_t word = 0, zero = 0;
    e = cudaMemcpyFromSymbol(&word, pp::g_dev_err, sizeof(word));
    if (e != cudaSuccess) return fail(PP_ERR_CUDA, "reading the device error word: %s", cudaGetErrorString(e));
    if (word == 0) return PP_OK;
    e = cudaMemcpyToSymbol(pp::g_dev_err, &zero, sizeof(zero));
    if (e != cudaSuccess) return fail(PP_ERR_CUDA, "clearing the device error word: %s", cudaGetErrorString(e));
    if (word & pp::DEVERR_TIMEOUT) return fail(PP_ERR_DEVICE_TIMEOUT, "a kernel's bounded wait ran out (0x%x)", word);
    if (word == pp::DEVERR_NO_ROOM)
        return fail(PP_ERR_DEVICE_INPUT, "a resize of the paged cache needs more pages or slots than there are; it was not made (0x%x)", word);
    return fail(PP_ERR_DEVICE_INPUT, "inconsistent descriptors, segment boundaries, token ids or cache pages (0x%x)", word);
}

}  // extern "C"
