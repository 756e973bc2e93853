// pp_cache.cuh - the paged 8-bit cache: its codes, and the kernel that appends rows to it (pp.h, pp_cache_store).
//
// A page holds `page` tokens of every kv head. Keys lie as [page][head][token][d], values transposed as
// [page][head][d][token], so that both are read by the decode step in the order its products take them
// (pp_paged.cuh). A (page, head) block of keys, and one of values, has one scale 2^e: the smallest e in
// [CACHE_E_MIN, CACHE_E_MAX] with max |x| <= 448 * 2^e (e4m3) or 127 * 2^e (int8). A power of two makes the division
// exact, so an element is rounded once, to nearest even, and a page that is re-scaled is not rounded again but where
// its codes lose their last bits. Codes of e4m3 keep 4 significant bits whatever e is, so the power of two costs them
// nothing in range or precision; int8 gives up at most one of its 8 bits.
//
// The rows of one page that stand together in a call are one append, whatever the order and the gaps of their slots: one
// owner forms their one scale. Appending to a page that already holds tokens keeps the larger of its scale and the one that
// the new rows need; if it grows, the codes already there are re-rounded to it. Values that are not finite do not count for
// the scale.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>
#include "pp_build.cuh"   // set_dev_err
#include "pp_ptx.cuh"     // packed fp32 pairs
#include "pp_rope.cuh"    // RopeVec

namespace pp {

constexpr int CACHE_D = 128;
constexpr int CACHE_E_MIN = -40, CACHE_E_MAX = 56;   // every ratio of two scales stays far inside fp32's range
constexpr int CACHE_THREADS = 256;
// Rows of a run that one warp takes. Measured with 128 and 512 runs of 1, 2, 4 and 8 bf16 rows, 8 heads, pages of 64: up
// to 4 rows 7.0, 8.0, 12.0, 17.5 and 14.8, 20.1, 44.7, 57.5 us; up to 8 rows (longer code) 7.0, 8.3, 11.7, 18.8 and 15.6,
// 21.4, 46.0, 59.4; single rows only 6.6, 12.1, 13.6, 17.0 and 14.6, 36.0, 51.5, 55.8.
constexpr int CACHE_SHORT = 4;
constexpr int CACHE_APART = 256;      // rows of a page are one append if each is at most this many rows after the one before

enum CacheFmt : int { CACHE_E4M3 = 0, CACHE_INT8 = 1 };

template <int FMT> __device__ __forceinline__ float cache_scale(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int ex = int(b >> 23) - 127;               // amax = (1 + mantissa) 2^ex; below 2^-126 the clamp takes over
    const uint32_t man = b & 0x7fffffu;
    // 448 = 1.75 * 2^8, 127 = 1.984375 * 2^6
    int e = FMT == CACHE_E4M3 ? ex - 8 + (man > 0x600000u) : ex - 6 + (man > 0x7e0000u);
    e = max(CACHE_E_MIN, min(CACHE_E_MAX, e));
    return __uint_as_float(uint32_t(e + 127) << 23);
}
// Four values, in units of the scale, to four codes (byte i = value i). NaN becomes e4m3's NaN, or 0 in int8.
template <int FMT> __device__ __forceinline__ uint32_t cache_code4(float a, float b, float c, float d) {
    if (FMT == CACHE_E4M3) {
        uint16_t lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
        return uint32_t(lo) | uint32_t(hi) << 16;
    }
    auto one = [](float x) { return uint32_t(max(-127, min(127, __float2int_rn(x)))) & 0xffu; };
    return one(a) | one(b) << 8 | one(c) << 16 | one(d) << 24;
}
template <int FMT> __device__ __forceinline__ void cache_value4(uint32_t w, float (&x)[4]) {
    if (FMT == CACHE_E4M3) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t h;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(w >> (16 * i))));
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = float(int8_t(w >> (8 * i)));
    }
}
template <int FMT> __device__ __forceinline__ uint32_t cache_recode4(uint32_t w, float ratio) {
    float x[4];
    cache_value4<FMT>(w, x);
    return cache_code4<FMT>(x[0] * ratio, x[1] * ratio, x[2] * ratio, x[3] * ratio);
}
__device__ __forceinline__ float finite_abs(float x) {
    const float a = fabsf(x);
    return a < INFINITY ? a : 0.f;                    // NaN compares false
}

// The largest |x| of 16-byte vectors: a plain maximum over all (two bf16 to an instruction), which an infinity or NaN
// shows in; only then are the vectors looked through again for the largest finite one.
template <typename T> struct CacheMax;
template <> struct CacheMax<__nv_bfloat16> {
    __nv_bfloat162 m = __floats2bfloat162_rn(0.f, 0.f);
    __device__ __forceinline__ void add(const uint4 &v) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) m = __hmax2_nan(m, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i])));
    }
    __device__ __forceinline__ float get() const { return __bfloat162float(__hmax_nan(m.x, m.y)); }
};
template <> struct CacheMax<float> {
    float m = 0.f;
    __device__ __forceinline__ void add(const float4 &v) {
        const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(f[i])));
    }
    __device__ __forceinline__ float get() const { return m; }
};
__device__ __forceinline__ float max_nan(float a, float b) {
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(b));
    return a;
}
// Four values times inv, none beyond the largest code, to codes. For int8 adding 1.5 * 2^23 leaves the nearest integer
// (ties to even) in the low bits; with a power of two for inv the product is exact, so the fused form rounds the same.
template <int FMT> __device__ __forceinline__ uint32_t cache_code4_in(float2 a, float2 b, float2 inv) {
    if (FMT == CACHE_E4M3) {
        const float2 x = fmul2(a, inv), y = fmul2(b, inv);
        return cache_code4<FMT>(x.x, x.y, y.x, y.y);
    }
    const float2 big = make_float2(12582912.f, 12582912.f), x = ffma2(a, inv, big), y = ffma2(b, inv, big);
    return __byte_perm(__byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x0040),
                       __byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x0040), 0x5410);
}

template <typename T> struct CacheStoreArgs {
    const T *rows[2];                 // keys, values: [n, hkv, d]
    int64_t stride[2];                // elements between rows
    uint8_t *pages[2];
    float *scale[2];                  // [num_pages, hkv]
    const int32_t *slots;
    int64_t n;
    int32_t hkv, num_pages, page_log2;
    int32_t window, heads;            // rows and heads of a block
    uint32_t parts;                   // blocks of a window: keys and values, and their heads
};

// Re-round the codes of a block's first `o0` tokens after its scale grew by 1 / ratio; `who` of `many` threads.
template <int FMT>
__device__ __forceinline__ void cache_rescale(uint8_t *blk, bool val, int page, int o0, float ratio, int who, int many) {
    if (!val) {                                       // keys: o0 whole rows
        uint32_t *w = reinterpret_cast<uint32_t *>(blk);
        for (int i = who; i < o0 * (CACHE_D / 4); i += many) w[i] = cache_recode4<FMT>(w[i], ratio);
    } else {                                          // values: the first o0 bytes of every d's row
        const int nw = (o0 + 3) >> 2;
        for (int i = who; i < nw * CACHE_D; i += many) {
            const int d = i / nw, c = i - d * nw;
            uint32_t *w = reinterpret_cast<uint32_t *>(blk + d * page) + c;
            const uint32_t keep = 4 * c + 4 <= o0 ? 0u : 0xffffffffu << (8 * (o0 - 4 * c));
            const uint32_t old = *w;
            *w = (cache_recode4<FMT>(old, ratio) & ~keep) | (old & keep);
        }
    }
}

// 1 + the rows after i that go on with its run (at most a page).
__device__ __forceinline__ int cache_run_len(const uint32_t *cont, int i) {
    int j = i + 1;
    while (j < 256) {
        const uint32_t w = cont[j >> 5] >> (j & 31);
        const int ones = ~w ? __ffs(~w) - 1 : 32;
        const int room = 32 - (j & 31);
        j += min(ones, room);
        if (ones < room) break;
    }
    return j - i;
}

// The long look at the slots, for windows whose rows may stand apart: from row w0 - CACHE_THREADS on; bits of slots from there,
// and of the rows from w0 on that belong to the append of the last row with a slot before them.
constexpr int CACHE_LOOK = 2 * CACHE_THREADS;         // from w0 on: a window, a page's run after it and CACHE_APART more
static_assert(CACHE_LOOK >= 2 * 128 + CACHE_APART && CACHE_APART <= CACHE_THREADS, "rows looked at");
struct CacheLook {
    int32_t slot[CACHE_THREADS + CACHE_LOOK];         // -1: a row without one
    uint32_t valid[(CACHE_THREADS + CACHE_LOOK) / 32], join[CACHE_LOOK / 32];
};
// Sets `head` to the rows of the window that begin an append of one run, `apart` to those whose append has more rows. For the
// whole block.
static __device__ __noinline__ void cache_look_apart(const int32_t *slots, int64_t n, int64_t w0, int window, int lg, int64_t limit,
                                                     const uint32_t *cont, uint32_t *head, uint32_t *apart, CacheLook &k) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int W = CACHE_THREADS / 32;
    for (int z = 0; z < 3; ++z) {
        const int64_t i = w0 + tid + (z - 1) * CACHE_THREADS;
        int32_t slot = i >= 0 && i < n ? slots[i] : -1;
        if (slot >= limit) slot = -1;
        k.slot[z * CACHE_THREADS + tid] = slot;
        const uint32_t bv = __ballot_sync(0xffffffffu, slot >= 0);
        if (lane == 0) k.valid[z * W + warp] = bv;
    }
    __syncthreads();
    bool begins = false;
    for (int z = 0; z < 2; ++z) {
        const int r = (z + 1) * CACHE_THREADS + tid;  // in k.slot
        const int32_t slot = k.slot[r];
        bool join = false;
        if (slot >= 0) {
            int p = r - 1;                            // the last row with a slot, if it is near enough
            while (p >= r - CACHE_APART && k.slot[p] < 0) {
                const uint32_t w = k.valid[p >> 5] << (31 - (p & 31));
                p = w ? p - __clz(w) : (p & ~31) - 1;
            }
            join = p >= r - CACHE_APART && k.slot[p] >> lg == slot >> lg;
        }
        const uint32_t bj = __ballot_sync(0xffffffffu, join);
        if (lane == 0) k.join[z * W + warp] = bj;
        if (z == 0) begins = slot >= 0 && !join && tid < window;
    }
    __syncthreads();
    bool more = false;
    if (begins) {                                     // does the next row with a slot join its first run?
        const int from = tid + cache_run_len(cont, tid);
        for (int j = from, end = min(CACHE_LOOK, from + CACHE_APART); j < end; j = (j | 31) + 1) {
            const uint32_t w = k.valid[W + (j >> 5)] >> (j & 31);
            if (w) {
                const int next = j + __ffs(w) - 1;
                more = k.join[next >> 5] >> (next & 31) & 1;
                break;
            }
        }
    }
    const uint32_t bb = __ballot_sync(0xffffffffu, begins && !more), bm = __ballot_sync(0xffffffffu, more);
    if (lane == 0 && warp < 4) {
        head[warp] = bb;
        apart[warp] = bm;
    }
    __syncthreads();
}

// A page's rows that are not one run: from row i0 on, skipped rows and rows in any order among them, up to the last that
// follows the one before within CACHE_APART rows with no other page's row between. The whole block, a warp a row, each row
// read twice: ten times as slow as a run (a row left out of each of 1386 pages of 64, 8 heads: 1084 us, whole pages 103), but
// slots of pp_pages_resize are runs. s_row: 128 ints, s_red: 8 words, both free on entry.
template <typename T, int FMT>
static __device__ __noinline__ void cache_store_apart(const T *rows, int64_t stride, const int32_t *slots, int64_t n, int64_t i0, int lg,
                                                      int32_t num_pages, int hkv, bool val, int h0, int h1, uint8_t *pages,
                                                      float *scales, int32_t *s_row, uint32_t *s_red) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int page = 1 << lg;
    const int32_t pg = slots[i0] >> lg;
    const int64_t limit = int64_t(num_pages) << lg;
    auto slot_of = [&](int64_t i) {                       // of a row of any page, else -1
        const int32_t s = i < n ? slots[i] : -1;
        return s < limit ? s : -1;
    };
    int64_t last = i0;                                    // the same for all threads
    for (int64_t base = i0 + 1; base < n && base - last <= CACHE_APART; base += 32) {
        const int32_t s = slot_of(base + lane);           // every warp for itself: 32 rows at a time
        const uint32_t other = __ballot_sync(0xffffffffu, s >= 0 && s >> lg != pg);
        uint32_t same = __ballot_sync(0xffffffffu, s >= 0 && s >> lg == pg);
        if (other) same &= (other & (0u - other)) - 1;    // those before the first other
        bool end = other != 0;
        for (; same; same &= same - 1) {
            const int64_t i = base + __ffs(same) - 1;
            if (i - last > CACHE_APART) {
                end = true;
                break;
            }
            last = i;
        }
        if (end) break;
    }
    const int64_t len = last - i0 + 1;
    rows += i0 * stride;
    // the row of each place; of a slot that is named twice, the last
    __syncthreads();
    if (tid < page) s_row[tid] = -1;
    __syncthreads();
    for (int64_t t = tid; t < len; t += CACHE_THREADS) {
        const int32_t s = slot_of(i0 + t);
        if (s >= 0) atomicMax(&s_row[s & (page - 1)], int32_t(t));
    }
    __syncthreads();
    int o0 = 0;
    while (o0 < page - 1 && s_row[o0] < 0) ++o0;           // row i0 has one
    auto load = [&](int64_t t, int h, float (&x)[4]) {    // a lane four elements
        const T *row = rows + t * stride + h * CACHE_D + 4 * lane;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = static_cast<float>(row[e]);
    };
#pragma unroll 1
    for (int h = h0; h < h1; ++h) {
        const int64_t at = int64_t(pg) * hkv + h;
        uint8_t *blk = pages + (at << lg) * CACHE_D;
        const float old = o0 > 0 ? scales[at] : 0.f;
        float amax = 0.f;
#pragma unroll 1
        for (int64_t t = warp; t < len; t += CACHE_THREADS / 32)
            if (slot_of(i0 + t) >= 0) {
                float x[4];
                load(t, h, x);
                for (int e = 0; e < 4; ++e) amax = fmaxf(amax, finite_abs(x[e]));
            }
#pragma unroll
        for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (lane == 0) s_red[warp] = __float_as_uint(amax);
        __syncthreads();
        for (int k = 0; k < CACHE_THREADS / 32; ++k) amax = fmaxf(amax, __uint_as_float(s_red[k]));
        const float sc = fmaxf(old, cache_scale<FMT>(amax)), inv = 1.f / sc;
        if (o0 > 0 && sc > old) cache_rescale<FMT>(blk, val, page, o0, old * inv, tid, CACHE_THREADS);
        if (tid == 0) scales[at] = sc;
        __syncthreads();                                  // the re-rounded words are written before the new bytes
#pragma unroll 1
        for (int o = o0 + warp; o < page; o += CACHE_THREADS / 32) {
            const int32_t t = s_row[o];
            if (t < 0) continue;
            float x[4];
            load(t, h, x);
            const uint32_t w = cache_code4<FMT>(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
            if (!val) reinterpret_cast<uint32_t *>(blk + o * CACHE_D)[lane] = w;
            else
                for (int e = 0; e < 4; ++e) blk[(4 * lane + e) * page + o] = uint8_t(w >> (8 * e));
        }
    }
    __syncthreads();
}

// grid windows * parts, a window's blocks next to each other so that its rows' heads are read at about the same time: a
// block takes the appends that begin in its window of rows, for some heads' keys (even part) or values (odd). An append
// is all rows of one page that stand together, skipped rows among them: those of one (page, head) block, which one block
// or warp therefore owns. Nearly always it is a run, slots that ascend by one row by row; what is not goes to
// cache_store_apart. Runs of up to CACHE_SHORT rows (an appended token) go to a warp each; longer ones to the whole block,
// rows held in registers between the maximum and the codes, so that every row is read once, and the next head's rows
// asked for before this one's codes are written. A decode step (128 rows of 8 heads, 6.5 us) is bound by latency: slots,
// rows and scale, codes. A prefill (88,685 bf16 rows of 8 heads, 545 MB read and written in 125 us: 4.4 TB/s, 67 % of a
// plain copy's rate) by what stands between the loads: the block's maximum and its barriers, with 29 warps to an SM and
// two thirds of the issue slots taken. (The next head's rows asked for before the maximum, at 80 registers a thread and
// three blocks to an SM: 144 us.)
// UNITS: units of a thread, enough for a whole page.
template <typename T, int FMT, int UNITS>
__global__ void __launch_bounds__(CACHE_THREADS, UNITS == 1 ? 4 : UNITS == 2 ? 3 : 2) k_cache_store(const CacheStoreArgs<T> a) {
    using RV = RopeVec<T>;
    using V = typename RV::V;
    constexpr int N = RV::N, VR = CACHE_D / N;        // elements of a vector, vectors of a row
    constexpr int MAX_PAGE = 128;
    static_assert(sizeof(CacheLook) <= sizeof(uint32_t) * 2 * CACHE_D * (MAX_PAGE / 4 + 1), "a look fits s_v");
    __shared__ uint32_t s_cont[8], s_head[4], s_apart[4];
    __shared__ float s_max[2][CACHE_THREADS / 32], s_wild[CACHE_THREADS / 32];
    __shared__ uint32_t s_v[2][CACHE_D][MAX_PAGE / 4 + 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int lg = a.page_log2, page = 1 << lg;
    const uint32_t window = blockIdx.x / a.parts, part = blockIdx.x - window * a.parts;
    const bool val = part & 1;
    const int h0 = int(part >> 1) * a.heads, h1 = min(a.hkv, h0 + a.heads);
    const T *rows = val ? a.rows[1] : a.rows[0];
    const int64_t stride = val ? a.stride[1] : a.stride[0];
    uint8_t *pages = val ? a.pages[1] : a.pages[0];
    float *scales = val ? a.scale[1] : a.scale[0];
    const int64_t w0 = int64_t(window) * a.window;
    const int64_t limit = int64_t(a.num_pages) << lg;
    bool odd;                                         // rows of a page may stand apart
    {   // bit i of s_cont: row w0 + i goes on with the run of the row before it; of s_head: an append begins there
        const int64_t i = w0 + tid;
        const int32_t slot = i < a.n ? a.slots[i] : -1, before = i > 0 && i < a.n ? a.slots[i - 1] : -1;
        const bool valid = slot >= 0 && slot < limit, known = before >= 0 && before < limit;
        const bool same = valid && known && before >> lg == slot >> lg, cont = same && slot == before + 1;
        const uint32_t bc = __ballot_sync(0xffffffffu, cont);
        const uint32_t bh = __ballot_sync(0xffffffffu, valid && !cont && tid < a.window);
        if (lane == 0) {
            s_cont[warp] = bc;
            if (warp < 4) {
                s_head[warp] = bh;
                s_apart[warp] = 0;
            }
        }
        if (slot >= limit && tid < a.window && h0 == 0 && !val) set_dev_err(DEVERR_BAD_PAGES);
        // a row after a skipped one, or in its page but not the next; or skipped rows to the end of the look
        odd = valid ? i > 0 && (!known || (same && !cont)) : tid == CACHE_THREADS - 1 && i < a.n;
    }
    if (__syncthreads_or(odd))
        cache_look_apart(a.slots, a.n, w0, a.window, lg, limit, s_cont, s_head, s_apart, *reinterpret_cast<CacheLook *>(s_v));
    auto run_len = [&](int i) { return cache_run_len(s_cont, i); };
    // ---- short runs: one warp each, a lane four elements of every row
    int ord = 0;
    for (int wd = 0; wd < (a.window + 31) / 32; ++wd) {
        for (uint32_t b = s_head[wd]; b; b &= b - 1) {
            const int i = wd * 32 + __ffs(b) - 1, len = run_len(i);
            if (len > CACHE_SHORT || (ord++ & 7) != warp) continue;
            const int32_t slot = a.slots[w0 + i];
            const int o0 = slot & (page - 1);
#pragma unroll 1
            for (int h = h0; h < h1; ++h) {
                const int64_t at = int64_t(slot >> lg) * a.hkv + h;
                uint8_t *blk = pages + (at << lg) * CACHE_D;
                float x[CACHE_SHORT][4], amax = 0.f;
#pragma unroll
                for (int t = 0; t < CACHE_SHORT; ++t) {
                    if (t < len) {
                        const T *row = rows + (w0 + i + t) * stride + h * CACHE_D + 4 * lane;
                        if constexpr (N == 8) {
                            const uint2 u = *reinterpret_cast<const uint2 *>(row);
                            x[t][0] = __uint_as_float(u.x << 16);
                            x[t][1] = __uint_as_float(u.x & 0xffff0000u);
                            x[t][2] = __uint_as_float(u.y << 16);
                            x[t][3] = __uint_as_float(u.y & 0xffff0000u);
                        } else {
                            const float4 u = *reinterpret_cast<const float4 *>(row);
                            x[t][0] = u.x;
                            x[t][1] = u.y;
                            x[t][2] = u.z;
                            x[t][3] = u.w;
                        }
                    } else {
                        x[t][0] = x[t][1] = x[t][2] = x[t][3] = 0.f;
                    }
                }
                const float old = o0 > 0 ? scales[at] : 0.f;
#pragma unroll
                for (int t = 0; t < CACHE_SHORT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) amax = fmaxf(amax, finite_abs(x[t][e]));
#pragma unroll
                for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                const float sc = fmaxf(old, cache_scale<FMT>(amax)), inv = 1.f / sc;
                if (o0 > 0 && sc > old) {
                    cache_rescale<FMT>(blk, val, page, o0, old * inv, lane, 32);
                    __syncwarp();                     // its last word of values may hold the first new byte
                }
                if (lane == 0) scales[at] = sc;
#pragma unroll
                for (int t = 0; t < CACHE_SHORT; ++t) {
                    if (t >= len) break;
                    const uint32_t w = cache_code4<FMT>(x[t][0] * inv, x[t][1] * inv, x[t][2] * inv, x[t][3] * inv);
                    if (!val) {
                        reinterpret_cast<uint32_t *>(blk + (o0 + t) * CACHE_D)[lane] = w;
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) blk[(4 * lane + e) * page + o0 + t] = uint8_t(w >> (8 * e));
                    }
                }
            }
        }
    }
    // ---- long runs: the whole block; a unit is four tokens (at a multiple of four in the page) of one vector of d
    int par = 0;                                      // of the heads done: s_max and s_v alternate, one barrier apart
    for (int wd = 0; wd < (a.window + 31) / 32; ++wd) {
        for (uint32_t b = s_head[wd]; b; b &= b - 1) {
            const int i = wd * 32 + __ffs(b) - 1, len = run_len(i);
            if (len <= CACHE_SHORT) continue;
            const int32_t slot = a.slots[w0 + i];
            const int o0 = slot & (page - 1), o1 = o0 + len;
            const int q0 = o0 >> 2, units = (((o1 + 3) >> 2) - q0) * VR;
            const T *base = rows + (w0 + i - o0) * stride;             // row of the page's token 0
            V x[UNITS][4];
            auto load = [&](int h) {
#pragma unroll
                for (int k = 0; k < UNITS; ++k) {
                    const int u = tid + k * CACHE_THREADS, tok = 4 * (q0 + u / VR);
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        x[k][t] = V{};
                        if (u < units && tok + t >= o0 && tok + t < o1)
                            x[k][t] = reinterpret_cast<const V *>(base + int64_t(tok + t) * stride + h * CACHE_D)[u % VR];
                    }
                }
            };
            load(h0);
#pragma unroll 1
            for (int h = h0; h < h1; ++h, par ^= 1) {
                const int64_t at = int64_t(slot >> lg) * a.hkv + h;
                uint8_t *blk = pages + (at << lg) * CACHE_D;
                const float old = o0 > 0 ? scales[at] : 0.f;
                auto block_max = [&](float m, float *of) {  // over the block's threads; NaN if any is
#pragma unroll
                    for (int o = 16; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
                    if (lane == 0) of[warp] = m;
                    __syncthreads();
#pragma unroll
                    for (int k = 0; k < CACHE_THREADS / 32; ++k) m = max_nan(m, of[k]);
                    return m;
                };
                CacheMax<T> cm;
#pragma unroll
                for (int k = 0; k < UNITS; ++k)
#pragma unroll
                    for (int t = 0; t < 4; ++t) cm.add(x[k][t]);
                float amax = block_max(cm.get(), s_max[par]);
                bool wild = !(amax <= (FMT == CACHE_E4M3 ? 448.f : 127.f) * 0x1p56f);      // the same for all
                if (wild) {
                    amax = 0.f;
#pragma unroll
                    for (int k = 0; k < UNITS; ++k)
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            float f[N];
                            RV::unpack(x[k][t], f);
#pragma unroll
                            for (int e = 0; e < N; ++e) amax = fmaxf(amax, finite_abs(f[e]));
                        }
                    amax = block_max(amax, s_wild);
                    __syncthreads();                  // s_wild has no turn of its own
                }
                const float sc = fmaxf(old, cache_scale<FMT>(amax)), inv = 1.f / sc;
                if (o0 > 0 && sc > old) cache_rescale<FMT>(blk, val, page, o0, old * inv, tid, CACHE_THREADS);
                if (tid == 0) scales[at] = sc;
                uint32_t w[UNITS][4][N / 4];          // token t, codes of d = N * vector ...
                auto encode = [&](auto code4) {
#pragma unroll
                    for (int k = 0; k < UNITS; ++k)
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            float f[N];
                            RV::unpack(x[k][t], f);
#pragma unroll
                            for (int e = 0; e < N / 4; ++e)
                                w[k][t][e] = code4(make_float2(f[4 * e], f[4 * e + 1]), make_float2(f[4 * e + 2], f[4 * e + 3]));
                        }
                };
                if (FMT == CACHE_INT8 && wild)
                    encode([&](float2 p, float2 q) { return cache_code4<FMT>(p.x * inv, p.y * inv, q.x * inv, q.y * inv); });
                else
                    encode([&](float2 p, float2 q) { return cache_code4_in<FMT>(p, q, make_float2(inv, inv)); });
                if (h + 1 < h1) load(h + 1);
#pragma unroll
                for (int k = 0; k < UNITS; ++k) {
                    const int u = tid + k * CACHE_THREADS, qd = q0 + u / VR, dv = u % VR;
                    if (u >= units) break;
                    if (!val) {
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            const int tok = 4 * qd + t;
                            if (tok < o0 || tok >= o1) continue;
                            uint32_t *dst = reinterpret_cast<uint32_t *>(blk + tok * CACHE_D) + dv * (N / 4);
                            if constexpr (N == 8) *reinterpret_cast<uint2 *>(dst) = make_uint2(w[k][t][0], w[k][t][1]);
                            else *dst = w[k][t][0];
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < N / 4; ++e) {             // transpose the 4 tokens x 4 d of byte codes
                            const uint32_t w0 = w[k][0][e], w1 = w[k][1][e], w2 = w[k][2][e], w3 = w[k][3][e];
                            const uint32_t lo = __byte_perm(w0, w1, 0x5140), hi = __byte_perm(w2, w3, 0x5140);
                            const uint32_t lo2 = __byte_perm(w0, w1, 0x7362), hi2 = __byte_perm(w2, w3, 0x7362);
                            uint32_t *col = &s_v[par][N * dv + 4 * e][qd];
                            constexpr int S = MAX_PAGE / 4 + 1;
                            col[0] = __byte_perm(lo, hi, 0x5410);
                            col[S] = __byte_perm(lo, hi, 0x7632);
                            col[2 * S] = __byte_perm(lo2, hi2, 0x5410);
                            col[3 * S] = __byte_perm(lo2, hi2, 0x7632);
                        }
                    }
                }
                if (val) {                            // rows of d: 16 bytes at a time, single bytes at a ragged end
                    __syncthreads();
                    const int c0 = o0 >> 4, nc = ((o1 + 15) >> 4) - c0, lc = 32 - __clz(nc - 1);     // 2^lc >= nc
                    for (int u = tid; u < CACHE_D << lc; u += CACHE_THREADS) {
                        const int d = u >> lc, c = c0 + (u & ((1 << lc) - 1));
                        if (c >= c0 + nc) continue;
                        uint8_t *dst = blk + d * page + 16 * c;
                        const uint32_t *src = &s_v[par][d][4 * c];
                        if (16 * c >= o0 && 16 * c + 16 <= o1) {
                            *reinterpret_cast<uint4 *>(dst) = make_uint4(src[0], src[1], src[2], src[3]);
                        } else {
                            for (int j = max(o0 - 16 * c, 0); j < min(o1 - 16 * c, 16); ++j)
                                dst[j] = uint8_t(src[j >> 2] >> (8 * (j & 3)));
                        }
                    }
                }
            }
        }
    }
    if (s_apart[0] | s_apart[1] | s_apart[2] | s_apart[3]) {
        __syncthreads();                              // s_v is no longer read
        for (int wd = 0; wd < 4; ++wd)
            for (uint32_t b = s_apart[wd]; b; b &= b - 1)
                cache_store_apart<T, FMT>(rows, stride, a.slots, a.n, w0 + wd * 32 + __ffs(b) - 1, lg, a.num_pages, a.hkv, val, h0, h1,
                                          pages, scales, reinterpret_cast<int32_t *>(s_v[0][0]), reinterpret_cast<uint32_t *>(s_wild));
    }
}

}  // namespace pp
