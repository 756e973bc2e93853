// pp_paged.cuh - one decoding step over the paged 8-bit cache (pp.h, pp_paged_decode).
//
// Keys and values enter as codes: k_j = sk c_j, v_j = sv u_j with one sk and one sv for each (page, head) block. Every
// code, e4m3 or int8, is a number that f16 holds exactly, and so is a query row times its own power of two (2^-e with
// 2^e <= max |q| < 2^(e+1)), but for elements 2^-14 below the row's largest, which keep what is above 2^-24 of it. So
// the products run on the f16 tensor cores with no rounding of the keys and values, and the scales enter the softmax:
//   x_j = (c_j . q 2^-e) 2^e scale log2(e) sk_j + log2(sv_j)
//   p_j = 2^(x_j - m),  O = sum_j p_j u_j,  L = sum_j p_j / sv_j,  o = O / L,  LSE = ln 2 (m + log2 L).
// Taking log2(sv) into the exponent keeps p_j, which f16 has to hold, at most 2^15 whatever the blocks' scales are:
// m trails the true maximum by at most 8 and carries an offset of 7, so p reaches down to 2^-31 of its maximum before
// an f16 loses it (a spike over a long, flat context keeps its tail). L is summed in fp32 from the unrounded p.
// An f16 keeps 11 bits of p, 2^-12 of it at most off; o is off by some 2^-13 before its own rounding to bf16, which takes
// up to 2^-8: against 64 bits o is 1.670e-3 off (one response, root mean square, relative) where fp32 throughout gives
// 1.666e-3, and a few elements in 100 become the other neighbour. With p as two f16 and two products (22 bits) it was 1.666e-3
// too, at 62.7, 86.5 and 34.8 us where one product takes 58.5, 80.1 and 32.8 (the three large cases below, calls in a row):
// one is kept.
//
// Work: a job is 64 keys of one segment, one kv head and up to 16 query rows: (response, q head) pairs that see the
// segment, which for a prefix are those of all the group's responses. Jobs lie in the order (segment, head, rows,
// keys) and every warp takes an equal, contiguous share of them. Consecutive jobs of one (segment, head, rows), an
// item, accumulate in registers; an item cut between warps leaves one partial record for each. Row x of an item's
// records lies at (its place among all items' rows) + 16 * warp, both of which grow with the job order, so no two
// records meet and no count has to be scanned for it.
//
// A warp does all of a job: the pages come by bulk tensor copies into its stage (16 KB; the next job's are sent for into
// L2 meanwhile), and 16 keys at a time it forms S^T = K Q^T (m16n8k16, the keys as operand A), the softmax, and O^T += V^T
// P^T, with the codes converted in registers on their way from shared memory to operand A. Which keys and which d a
// lane's fragments stand for is free, as sums do not mind: they are chosen so that a lane reads 32 consecutive codes of
// a key and 4 consecutive keys of a d, for which the value pages are stored transposed, and so that 16 keys lie in one
// page: one sk and one sv.
//
// Measured (32 q and 8 kv heads, e4m3, pages of 64; both kernels): 16 groups of 8 responses, 88,685 tokens (184 MB), 56.2
// us, 3.3 TB/s or half the copy rate; 17 groups of 4, 147,786 tokens (304 MB), 77.3 us, 3.9 TB/s; 4 groups of 4 behind
// prefixes of 4096 to 8192 (31 MB, int8, 28 / 4 heads, pages of 128) 28.1 us; one response of 19 tokens 14.0 us. What
// bounds it: each warp waits for its pages and then for its own chains of products, 12 warps to an SM issue in 40 % of the
// cycles, some 15,000 of the 97,000 cycles pass before the first product (descriptors, page numbers, scales, queries, and
// code fetched for the first time), and the longest share ends as much after the mean.
// Tried and slower or no faster: two stages of 32 keys (70.6 and 97.8 us where one of 64 took 64.4 and 86.4), 32 keys at a
// time for up to 8 rows (no change), two warps that run through the loops' code while the others count (+2 us), fewer
// blocks for little work (no change).
// The warp-level MMA is a choice by measurement: with tcgen05 (keys and values as operand A of M = 128, queries as N;
// loaders, converters, softmax and issuers as roles of one CTA) a job passed through five hand-overs of 100 to 300 cycles
// each and these, not the tensor cores (2 % busy), bounded it: 103 and 110 us where this form began with 64 and 86.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include "pp_attn_fwd.cuh"  // bwait
#include "pp_cache.cuh"
#include "pp_paged_shares.cuh"
#include "pp_pages.cuh"     // PAGES_MAX_SEGS
#include "pp_ptx.cuh"

namespace pp {

constexpr int PD_BATCH = 16;          // jobs that a warp decodes at a time
constexpr int PD_THREADS = PD_WARPS * 32;
constexpr int PD_RUNS = 2048;         // runs of segments that a block keeps the sums before: of 1, 2 or 4 segments
static_assert(4 * PD_RUNS >= PAGES_MAX_SEGS, "runs");
constexpr float PD_OFF = 7.f;         // p = 2^(x - max + 7) at the maximum
constexpr float PD_LAZY = 8.f;        // the maximum may be exceeded by this before the sums are rescaled

struct alignas(16) PagedSegRec {
    int32_t off;                               // units before the segment
    int32_t item, last;                        // units of an item (0: no keys), and before its last job
    int32_t nblk;                              // blocks of query rows
    int32_t row, qrows, qbase;                 // first record row, query rows of a kv head, first response that sees it
    int32_t first;                             // the group's prefix segment, -1 for a prefix
};
struct PagedArgs {
    const __nv_bfloat16 *q;                    // [n_resp, hq, 128]
    const uint8_t *k_pages, *v_pages;
    const float *k_scale, *v_scale;            // [num_pages, hkv]
    const int32_t *group_start, *seg_group, *lens, *table;
    __nv_bfloat16 *o;
    float *lse;
    struct PagedSegRec *seg;                   // workspace: of each segment what the combine kernel needs
    int4 *total;                               // workspace: units in all, or -1 where the descriptors do not fit; their shares
    float2 *ml;                                // workspace: (max - 7, sum) of each record row
    float *part;                               // workspace: [rows][128] un-normalised outputs
    int32_t max_pages, G, nseg, hq, hkv, r, r_magic, num_pages, page_log2;   // r = hq / hkv, 65536 / r + 1
    float sl2, inv_r;                          // softmax scale * log2(e); 1 / r
};

struct PagedWorkspace {
    int64_t off_seg, off_ml, off_part, total;
};
__host__ inline PagedWorkspace paged_workspace(int32_t n_resp, int32_t hq) {
    const int64_t rows = paged_rows(n_resp, hq);
    auto up = [](int64_t x) { return (x + 255) & ~int64_t(255); };
    PagedWorkspace w{};
    w.off_seg = 256;
    w.off_ml = up(w.off_seg + 32 * PAGES_MAX_SEGS);
    w.off_part = up(w.off_ml + 8 * rows);
    w.total = up(w.off_part + 4 * CACHE_D * rows);
    return w;
}

// A segment as the work list sees it.
struct PagedSeg {
    int32_t len, nch;         // tokens, chunks
    int32_t r0, kg;           // first response ordinal and responses of its group
    int32_t qbase, qrows;     // first response that sees it; query rows of one kv head
    int32_t nblk;             // blocks of query rows
    int32_t place;            // in its group, 0 the prefix
    bool prefix, ok;
};
__device__ __forceinline__ PagedSeg paged_seg(const PagedArgs &a, int s) {
    PagedSeg d{};
    const int32_t len = a.lens[s], g = a.seg_group[s], gp = s > 0 ? a.seg_group[s - 1] : -1;
    d.ok = g >= 0 && g < a.G && len >= 0 && len <= a.max_pages << a.page_log2;      // at most 2^30
    if (!d.ok) return d;
    const int32_t b = a.group_start[g], e = a.group_start[g + 1];
    d.prefix = s == b;
    d.place = s - b;
    // groups follow one another without gaps, from segment 0 to the last
    d.ok = b >= 0 && b <= s && e > s && e <= a.nseg && (d.prefix ? g == gp + 1 : g == gp) &&
           (s != a.nseg - 1 || (g == a.G - 1 && e == a.nseg));
    if (!d.ok) return d;
    d.len = len;
    d.nch = (len + PD_CH - 1) / PD_CH;
    d.r0 = b - g;
    d.kg = e - b - 1;
    d.qbase = d.prefix ? d.r0 : s - g - 1;
    d.qrows = (d.prefix ? d.kg : 1) * a.r;
    d.nblk = (d.qrows + PD_RB - 1) / PD_RB;
    return d;
}
__device__ __forceinline__ int paged_run_log2(const PagedArgs &a) { return a.nseg <= PD_RUNS ? 0 : a.nseg <= 2 * PD_RUNS ? 1 : 2; }

// Four codes to two f16 pairs, exactly.
template <int FMT> __device__ __forceinline__ void codes_f16(uint32_t w, uint32_t &a, uint32_t &b) {
    if (FMT == CACHE_E4M3) {
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(a), "=r"(b) : "r"(w));
    } else {                                               // 1024 + (c + 128), then minus 1152
        const uint32_t x = w ^ 0x80808080u;
        const uint32_t u = __byte_perm(x, 0x64646464u, 0x4140), v = __byte_perm(x, 0x64646464u, 0x4342);
        const __half2 off = __half2half2(__ushort_as_half(0x6480));
        const __half2 ha = __hsub2(*reinterpret_cast<const __half2 *>(&u), off);
        const __half2 hb = __hsub2(*reinterpret_cast<const __half2 *>(&v), off);
        a = *reinterpret_cast<const uint32_t *>(&ha);
        b = *reinterpret_cast<const uint32_t *>(&hb);
    }
}

// The slow path of a wait, out of line.
static __device__ __noinline__ bool pwait_slow(uint64_t *bar, uint32_t parity, volatile int *abort_flag) {
    return bwait(bar, parity, abort_flag);
}
__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}
__device__ __forceinline__ float rcp_approx(float x) {     // within one step
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// D (16 x 8) += A (16 x 16) B (16 x 8), f16 in, fp32 out.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// An 8 x 8 matrix of f16, a lane two neighbours of row lane / 4, to its transpose.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <int N> struct PagedInt {
    static constexpr int value = N;
};

// A job, decoded: 16 of a warp's at a time, a lane one, so that the chain of loads behind it (segment, page table,
// scales) is waited for once in 16 jobs.
struct PagedJob {
    int32_t blk[4];           // of each 16 keys: (page, head) block
    float sk[4], lsv[4];      // key scale, log2 of the value scale
    int32_t seg;              // the segment
    int32_t key0, nk;         // first key, keys
    int32_t flags;            // 1: the warp's first job of its item, 2: its last
    int32_t nrows, head;      // query row i is q head head * r + (hh + i) % r of response resp + (hh + i) / r
    int32_t resp, hh;
    int32_t rec;              // record row of query row 0
};
// A warp's keys and values lie page by page (of 64 tokens at most) in the swizzle of their row's width: keys 128 bytes,
// values as many as a page's tokens.
struct PagedSmem {
    alignas(1024) uint8_t k[PD_WARPS][PD_CH * CACHE_D];
    alignas(1024) uint8_t v[PD_WARPS][PD_CH * CACHE_D];
    PagedJob job[PD_WARPS][PD_BATCH];
    int32_t run_off[PD_RUNS + 1], run_unit[PD_RUNS + 1];   // jobs, and units, before each run of segments
    uint64_t full[PD_WARPS];
    longlong2 sum[PD_WARPS];                               // of each warp's threads: jobs, units
    int abort_flag, bad;
};
static_assert(sizeof(PagedSmem) + 1024 <= 232448, "paged decode shared memory exceeds 227 KB");

// What a warp holds of an item of up to 8 NB query rows, in the layout of the MMA's fragments: lane (g, c) = (lane / 4,
// lane % 4) has, for each 8 rows, the f16 of row g (32 elements from 32 c on), and of rows 2 c and 2 c + 1 the factor of
// S, the maximum so far and its part of the sum, and O^T at d = 16 t + g and 8 further.
template <int NB> struct PagedItem {
    uint32_t q[NB][8][2];
    float o[NB][8][4];
    float cq[NB][2], m[NB][2], l[NB][2];
};

// Query row n of a job as f16, scaled to [1, 2) (the largest and smallest rows to [2^-6, 4)): a lane 32 elements from 32 (lane % 4) on; and the factor that takes its
// products back to exponents. Rows past the last are zeros.
struct PagedRow {
    uint32_t q[16];
    float f;
};
static __device__ __noinline__ PagedRow paged_row_f16(const PagedArgs &a, const PagedJob &e, int n, int c) {
    uint4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = make_uint4(0, 0, 0, 0);
    if (n < e.nrows) {
        const int hh = e.hh + n, more = (hh * a.r_magic) >> 16;        // hh / r, as hh < r + 16 and r <= 256
        const int64_t row = int64_t(e.resp + more) * a.hq + e.head * a.r + (hh - more * a.r);
        const uint4 *src = reinterpret_cast<const uint4 *>(a.q + row * CACHE_D + 32 * c);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = src[i];
    }
    const uint32_t x[16] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w,
                            w[2].x, w[2].y, w[2].z, w[2].w, w[3].x, w[3].y, w[3].z, w[3].w};
    float mx = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) mx = fmax3(mx, fabsf(bf16lo(x[i])), fabsf(bf16hi(x[i])));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    // e = 0 for a row of zeros or with an infinity or NaN, which f16 keeps; at most 126, so that 2^-e is a normal number
    int e2 = int(__float_as_uint(mx) >> 23) - 127;
    e2 = mx == 0.f || e2 == 128 ? 0 : min(max(e2, -120), 126);
    const float down = __uint_as_float(uint32_t(127 - e2) << 23);
    PagedRow out;
#pragma unroll
    for (int i = 0; i < 16; ++i) out.q[i] = pack_f16x2(bf16lo(x[i]) * down, bf16hi(x[i]) * down);
    out.f = a.sl2 * __uint_as_float(uint32_t(127 + e2) << 23);
    return out;
}

template <int NB>
__device__ __forceinline__ void paged_begin(PagedItem<NB> &it, const PagedArgs &a, const PagedJob &st, int lane) {
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int h = 0; h < NB; ++h) {
        const PagedRow row = paged_row_f16(a, st, g + 8 * h, c);
#pragma unroll
        for (int i = 0; i < 16; ++i) it.q[h][i >> 1][i & 1] = row.q[i];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            it.cq[h][e] = __shfl_sync(0xffffffffu, row.f, 4 * (2 * c + e));
            it.m[h][e] = -INFINITY;
            it.l[h][e] = 0.f;
        }
#pragma unroll
        for (int t = 0; t < 8; ++t) it.o[h][t][0] = it.o[h][t][1] = it.o[h][t][2] = it.o[h][t][3] = 0.f;
    }
}

// S^T = K Q^T of 16 keys: row g of the MMA's tile is key 4 (g / 2) + g % 2 and row g + 8 the key two further; step s holds
// d = 32 c + 4 s ..., so a lane reads 32 consecutive codes of a key (two 16-byte chunks, in the 128-byte swizzle).
template <int FMT, int NB>
__device__ __forceinline__ void paged_scores(const PagedItem<NB> &it, const uint8_t *k, int swz, int c, float (&x)[NB][4]) {
    uint4 w[2][2];
#pragma unroll
    for (int z = 0; z < 2; ++z)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[z][i] = *reinterpret_cast<const uint4 *>(k + 2 * z * CACHE_D + (((2 * c + i) ^ (swz + 2 * z)) << 4));
    float d[NB][2][4];                                     // two sums each, so that fewer products wait for one another
#pragma unroll
    for (int h = 0; h < NB; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i) d[h][i][0] = d[h][i][1] = d[h][i][2] = d[h][i][3] = 0.f;
#pragma unroll
    for (int s = 0; s < 8; ++s) {
        uint32_t f[4];
        auto word = [&](int z) { const uint4 v = w[z][s >> 2]; return (s & 3) == 0 ? v.x : (s & 3) == 1 ? v.y : (s & 3) == 2 ? v.z : v.w; };
        codes_f16<FMT>(word(0), f[0], f[2]);
        codes_f16<FMT>(word(1), f[1], f[3]);
#pragma unroll
        for (int h = 0; h < NB; ++h) mma_f16(d[h][s >> 2], f, it.q[h][s][0], it.q[h][s][1]);
    }
#pragma unroll
    for (int h = 0; h < NB; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[h][e] = d[h][0][e] + d[h][1][e];
}

// The softmax of 16 keys: p as the MMA's B operand. in0, in1: the lane's keys are inside the segment.
template <int NB>
__device__ __forceinline__ void paged_softmax(PagedItem<NB> &it, float (&x)[NB][4], float sk, float lsv, bool in0, bool in1,
                                              uint32_t (&pb)[NB][2]) {
    bool more = false;
#pragma unroll
    for (int h = 0; h < NB; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float f = it.cq[h][e] * sk;
            x[h][e] = in0 ? fmaf(x[h][e], f, lsv) : -INFINITY;         // past the end a page may hold anything
            x[h][2 + e] = in1 ? fmaf(x[h][2 + e], f, lsv) : -INFINITY;
            more |= fmaxf(x[h][e], x[h][2 + e]) > it.m[h][e] + (PD_OFF + PD_LAZY);
        }
    // a new maximum where the old one is exceeded by more than PD_LAZY, as it always is (from -inf) at first
    if (__any_sync(0xffffffffu, more)) {
#pragma unroll
        for (int h = 0; h < NB; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float w = fmaxf(x[h][e], x[h][2 + e]);
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, o));
                w = fmaxf(it.m[h][e], w - PD_OFF);
                const float fac = it.m[h][e] == w ? 1.f : ex2_approx(it.m[h][e] - w);
                it.m[h][e] = w;
                it.l[h][e] *= fac;
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    it.o[h][t][e] *= fac;
                    it.o[h][t][2 + e] *= fac;
                }
            }
    }
    const float isv = ex2_approx(-lsv);
#pragma unroll
    for (int h = 0; h < NB; ++h) {
        // where no key so far gives a number (NaN alone) m is -inf: any m will do
        const float m0 = it.m[h][0] == -INFINITY ? 0.f : it.m[h][0], m1 = it.m[h][1] == -INFINITY ? 0.f : it.m[h][1];
        const float p0 = ex2_approx(x[h][0] - m0), p1 = ex2_approx(x[h][1] - m1);
        const float p2 = ex2_approx(x[h][2] - m0), p3 = ex2_approx(x[h][3] - m1);
        it.l[h][0] = fmaf(p0 + p2, isv, it.l[h][0]);
        it.l[h][1] = fmaf(p1 + p3, isv, it.l[h][1]);
        pb[h][0] = transpose8(pack_f16x2(p0, p1));
        pb[h][1] = transpose8(pack_f16x2(p2, p3));
    }
}

// O^T += V^T P^T over 16 keys: tile t's rows are d = 16 t + row, and a lane reads keys 4 c ... 4 c + 3 of a d in one word.
// keep: the bytes of it that are inside the segment; the others count as 0, not as 0 * NaN.
template <int FMT, int NB>
__device__ __forceinline__ void paged_output(PagedItem<NB> &it, const uint8_t *v, int v_row, uint32_t keep,
                                             const uint32_t (&pb)[NB][2]) {
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        const uint32_t w0 = *reinterpret_cast<const uint32_t *>(v + 16 * t * v_row) & keep;
        const uint32_t w1 = *reinterpret_cast<const uint32_t *>(v + (16 * t + 8) * v_row) & keep;
        uint32_t f[4];
        codes_f16<FMT>(w0, f[0], f[2]);
        codes_f16<FMT>(w1, f[1], f[3]);
#pragma unroll
        for (int h = 0; h < NB; ++h) mma_f16(it.o[h][t], f, pb[h][0], pb[h][1]);
    }
}

template <int NB>
__device__ __forceinline__ void paged_record(PagedItem<NB> &it, const PagedArgs &a, int32_t rec, int nrows, int lane) {
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int h = 0; h < NB; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float l = it.l[h][e];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            const int n = 8 * h + 2 * c + e;
            if (n < nrows) {
                const int64_t row = int64_t(rec) + n;
                if (g == 0) a.ml[row] = make_float2(it.m[h][e], l);       // -inf: no key gave a number above it
                float *dst = a.part + row * CACHE_D + g;
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    dst[16 * t] = it.o[h][t][e];
                    dst[16 * t + 8] = it.o[h][t][2 + e];
                }
            }
        }
}

// The segment that job (BY units: unit) `at` lies in, with what it has to be known by; `before`: jobs before it, `within`:
// where in the segment. Out of line, as the other parts that are not a loop: an instruction that is run for the first
// time on an SM costs some 20 cycles to fetch, and two callers fetch this one once.
struct PagedPlace {
    int32_t s, len, r0, kg, before;
    uint32_t within, nch, nblk;
    bool prefix;
};
static __device__ __noinline__ PagedPlace paged_place(const PagedArgs &a, const int32_t *run_off, const int32_t *run_unit, int n_run,
                                                      int32_t at, bool units) {
    const int32_t *off = units ? run_unit : run_off;
    int lo = 0, hi = n_run;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= at) lo = mid; else hi = mid;
    }
    PagedPlace p;
    p.within = at - off[lo];
    p.before = run_off[lo];
#pragma unroll 1
    for (p.s = lo << paged_run_log2(a);; ++p.s) {          // paged_seg, that the scan has checked
        p.len = a.lens[p.s];
        const int32_t g = a.seg_group[p.s], b = a.group_start[g];
        p.kg = a.group_start[g + 1] - b - 1;
        p.r0 = b - g;
        p.prefix = p.s == b;
        const int32_t qrows = (p.prefix ? p.kg : 1) * a.r;
        p.nch = uint32_t(p.len + PD_CH - 1) / PD_CH;
        p.nblk = uint32_t(qrows + PD_RB - 1) / PD_RB;
        const uint32_t items = p.nblk * a.hkv, here = items * (units ? paged_item(p.nch, qrows) : p.nch);
        if (p.within < here) return p;
        p.within -= here;
        p.before += items * p.nch;
    }
}
// The first job that begins at unit u or after it.
__device__ __forceinline__ int32_t paged_job_at(const PagedArgs &a, const int32_t *run_off, const int32_t *run_unit, int n_run,
                                                int32_t u, int32_t n_units) {
    const PagedPlace p = paged_place(a, run_off, run_unit, n_run, min(u, n_units - 1), true);
    const int32_t qrows = (p.prefix ? p.kg : 1) * a.r, cost = paged_cost(qrows);
    const uint32_t item = paged_item(p.nch, qrows), i = p.within / item;
    const int32_t rest = p.within - i * item + (u >= n_units);           // past the last unit: after the last job
    return p.before + int32_t(i) * p.nch + paged_job_from(rest, cost);
}
// Jobs base ... base + PD_BATCH - 1 of a warp's: what they are (a lane a job), then their pages (a lane two of the 4 x 16
// sixteens of keys).
static __device__ __noinline__ void paged_decode_jobs(const PagedArgs &a, PagedJob *job, const int32_t *run_off, const int32_t *run_unit,
                                                      int n_run, int32_t j_begin, int32_t n_mine, int32_t who, int32_t base, int lane) {
    const int lg = a.page_log2;
    const int32_t j = base + lane;
    if (lane < PD_BATCH && j < n_mine) {
        const PagedPlace p = paged_place(a, run_off, run_unit, n_run, j_begin + j, false);
        const uint32_t idx = p.within / p.nch, chunk = p.within - idx * p.nch, head = idx / p.nblk, rb = idx - head * p.nblk;
        const int qrows = (p.prefix ? p.kg : 1) * a.r, rho = rb * PD_RB, qbase = p.prefix ? p.r0 : p.s - (a.seg_group[p.s]) - 1;
        PagedJob &e = job[lane];
        e.seg = p.s;
        e.key0 = chunk * PD_CH;
        e.nk = min(PD_CH, p.len - int(chunk) * PD_CH);
        e.flags = (chunk == 0 || j == 0 ? 1 : 0) | (chunk == p.nch - 1 || j + 1 == n_mine ? 2 : 0);
        e.nrows = min(PD_RB, qrows - rho);
        e.head = head;
        const uint32_t first = uint32_t(rho) / uint32_t(a.r);
        e.resp = qbase + first;
        e.hh = rho - first * a.r;
        e.rec = paged_row(p.prefix, p.r0, p.kg, qbase, a.hq) + head * qrows + rho + who * PD_RB;
    }
    __syncwarp();
    int32_t id[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int k = (lane >> 2) + 8 * i, at = 16 * (lane & 3);
        id[i] = base + k < n_mine && at < job[k].nk ? a.table[int64_t(job[k].seg) * a.max_pages + ((job[k].key0 + at) >> lg)] : 0;
    }
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int k = (lane >> 2) + 8 * i;
        const bool out = id[i] < 0 || id[i] >= a.num_pages;
        bad |= out;
        job[k].blk[lane & 3] = (out ? 0 : id[i]) * a.hkv + job[k].head;              // below 2^31: checked on the host
    }
    if (bad) set_dev_err(DEVERR_BAD_PAGES);
    __syncwarp();
}
// Their scales: apart, so that the first job's pages are asked for before they are waited for.
static __device__ __noinline__ void paged_decode_scales(const PagedArgs &a, PagedJob *job, int32_t n_mine, int32_t base, int lane) {
    float sk[2], sv[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int k = (lane >> 2) + 8 * i;
        const bool in = base + k < n_mine && 16 * (lane & 3) < job[k].nk;
        const int32_t blk = job[k].blk[lane & 3];
        sk[i] = in ? a.k_scale[blk] : 0.f;
        sv[i] = in ? a.v_scale[blk] : 1.f;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        job[(lane >> 2) + 8 * i].sk[lane & 3] = sk[i];
        job[(lane >> 2) + 8 * i].lsv[lane & 3] = __log2f(sv[i]);
    }
    __syncwarp();
}

// tmK, tmV: 3-D maps over the pools, (128, page, num_pages * hkv) and (page, 128, num_pages * hkv) bytes, boxes of one
// block or, for pages of 128 tokens, half of one.
template <int FMT>
__global__ void __launch_bounds__(PD_THREADS, 1)
k_paged_decode(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const PagedArgs a) {
    extern __shared__ uint8_t smem_raw[];
    PagedSmem &sm = *reinterpret_cast<PagedSmem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int lg = a.page_log2;
    volatile int *abort_flag = &sm.abort_flag;

    if (lane == 0) {
        mbar_init(&sm.full[warp], 1);
        fence_mbar_init();
    }
    if (threadIdx.x == 0) {
        sm.bad = 0;
        sm.abort_flag = 0;
    }
    __syncthreads();
    // the queries, which the items' first jobs will wait for
    for (int64_t i = (int64_t(blockIdx.x) * PD_THREADS + threadIdx.x) * 64, n = int64_t(a.nseg - a.G) * a.hq * CACHE_D; i < n;
         i += int64_t(gridDim.x) * PD_THREADS * 64)
        prefetch_l2(a.q + i);
    // ---- jobs and units before each run of segments: a thread sums the `each` runs from first on
    const int rl = paged_run_log2(a), n_run = (a.nseg + (1 << rl) - 1) >> rl;
    const bool lister = blockIdx.x == 0;                   // writes what the combine kernel needs of each segment
    const int each = (n_run + PD_THREADS - 1) / PD_THREADS, first = min(int(threadIdx.x) * each, n_run), last = min(first + each, n_run);
    int64_t jobs = 0, units = 0, all_units;
    bool bad = false;
#pragma unroll 1
    for (int s = first << rl; s < min(last << rl, a.nseg); ++s) {
        const PagedSeg d = paged_seg(a, s);
        bad |= !d.ok;
        // the page numbers will be read next: the first 128 of them (more are rarely one warp's)
        const int npg = (d.len + (1 << lg) - 1) >> lg;
#pragma unroll 1
        for (int i = 0; i < min(npg, 128); i += 32) prefetch_l2(a.table + int64_t(s) * a.max_pages + i);
        if ((s & ((1 << rl) - 1)) == 0) {                  // so far in the thread; garbage past 2^31, which the total catches
            sm.run_off[s >> rl] = int32_t(jobs);
            sm.run_unit[s >> rl] = int32_t(units);
        }
        const int32_t item = paged_item(d.nch, d.qrows);
        if (lister)
            a.seg[s] = PagedSegRec{int32_t(units), item, paged_start(d.nch - 1, d.qrows), d.nblk, paged_row(d.prefix, d.r0, d.kg, d.qbase, a.hq), d.qrows, d.qbase,
                                   d.ok && !d.prefix ? s - d.place : -1};
        const int32_t items = d.nblk * a.hkv;
        jobs += int64_t(d.nch) * items;
        units += int64_t(item) * items;
    }
    // what the threads before have: both counts saturate far past the limit of 2^31
    {
        int64_t ju = min(jobs, int64_t(1) << 31), uu = min(units, int64_t(1) << 31);
        const int64_t j_own = ju, u_own = uu;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, ju, o), y = __shfl_up_sync(0xffffffffu, uu, o);
            if (lane >= o) ju += x, uu += y;
        }
        if (lane == 31) sm.sum[warp] = make_longlong2(ju, uu);
        if (bad) sm.bad = 1;
        __syncthreads();
        int64_t j_all = 0, u_all = 0;
        jobs = ju - j_own;
        units = uu - u_own;
#pragma unroll 1
        for (int w = 0; w < PD_WARPS; ++w) {
            const longlong2 x = sm.sum[w];
            if (w < warp) jobs += x.x, units += x.y;
            j_all += x.x;
            u_all += x.y;
        }
        if (threadIdx.x == 0) sm.run_off[n_run] = int32_t(j_all), sm.run_unit[n_run] = int32_t(u_all);
        all_units = u_all;
    }
    const bool ok = !sm.bad && all_units < (int64_t(1) << 31);            // jobs are fewer than units
    const int32_t n_units = ok ? int32_t(all_units) : 0;
#pragma unroll 1
    for (int i = first; i < last; ++i) {
        sm.run_off[i] += int32_t(jobs);
        sm.run_unit[i] += int32_t(units);
    }
    if (lister) {
        if (ok)
#pragma unroll 1
            for (int s = first << rl; s < min(last << rl, a.nseg); ++s) a.seg[s].off += int32_t(units);
        if (threadIdx.x == 0 && !ok) set_dev_err(DEVERR_BAD_PAGES);
    }
    __syncthreads();
    // neighbouring shares go to different SMs: with few jobs every SM has some
    const int32_t who = warp * gridDim.x + blockIdx.x;
    const PagedShare share(n_units, gridDim.x * PD_WARPS);
    if (lister && threadIdx.x == 0) *a.total = make_int4(ok ? n_units : -1, share.many, share.per, share.more);
    if (n_units == 0 || who >= share.many) return;
    // lane 0 finds the share's first job, lane 1 the next share's
    const int32_t edge = paged_job_at(a, sm.run_off, sm.run_unit, n_run, share.begin(who + (lane & 1)), n_units);
    const int32_t j_begin = __shfl_sync(0xffffffffu, edge, 0), n_mine = __shfl_sync(0xffffffffu, edge, 1) - j_begin;

    uint64_t *full = &sm.full[warp];
    const uint32_t lead = elect_one();
    // the keys and values of job j, page by page
    const uint32_t lt = min(lg, 6), bytes = uint32_t(CACHE_D) << lt;
    auto fetch = [&](int32_t j) {
        const PagedJob &e = sm.job[warp][j & (PD_BATCH - 1)];
        const uint32_t np = uint32_t(e.nk + (1 << lt) - 1) >> lt;
        const int off = lg == 7 ? e.key0 & 64 : 0;         // half of a page of 128
        if (lead) {
            mbar_arrive_expect_tx(full, 2 * np * bytes);
#pragma unroll 1
            for (uint32_t i = 0; i < np; ++i) {
                const int32_t b = e.blk[i << (lt - 4)];
                tma_load_3d(sm.k[warp] + i * bytes, &tmK, 0, off, b, full);
                tma_load_3d(sm.v[warp] + i * bytes, &tmV, off, 0, b, full);
            }
        }
    };
    // the next job's pages into L2 while this one is worked on: there is no room for them in shared memory yet
    auto ahead = [&](int32_t j) {
        if (j < n_mine && (j & (PD_BATCH - 1)) != 0) {     // decoded
            const PagedJob &e = sm.job[warp][j & (PD_BATCH - 1)];
            const uint32_t np = uint32_t(e.nk + (1 << lt) - 1) >> lt;
            const int off = lg == 7 ? e.key0 & 64 : 0;
            if (lead)
#pragma unroll 1
                for (uint32_t i = 0; i < np; ++i) {
                    const int32_t b = e.blk[i << (lt - 4)];
                    tma_prefetch_3d(&tmK, 0, off, b);
                    tma_prefetch_3d(&tmV, off, 0, b);
                }
        }
    };
    auto arrived = [&](uint64_t *bar, int32_t j) -> bool {
        return __all_sync(0xffffffffu, mbar_try_wait(bar, j & 1) || pwait_slow(bar, j & 1, abort_flag));
    };

    const int g = lane >> 2, c = lane & 3;
    const int key = 4 * (g >> 1) + (g & 1);                // a lane's keys of 16 are key and key + 2
    // of 16 keys: the lane's row of codes, and its word of d = g (in the swizzle of v_row-byte rows)
    const int v_row = min(1 << lg, 64);
    const int v_swz = v_row == 64 ? (g >> 1) & 3 : v_row == 32 ? (g >> 2) & 1 : 0;
    int32_t j = 0;
    // the jobs of one item from j on, of up to 8 NB rows; false if a wait ran out
    auto item = [&](auto nb) -> bool {
        constexpr int NB = decltype(nb)::value;
        PagedItem<NB> it;
        paged_begin<NB>(it, a, sm.job[warp][j & (PD_BATCH - 1)], lane);
#pragma unroll 1
        for (;;) {
            const PagedJob &e = sm.job[warp][j & (PD_BATCH - 1)];
            const int flags = e.flags, nk = e.nk, rec = e.rec, nrows = e.nrows;
            ahead(j + 1);
            if (!arrived(full, j)) return false;
#pragma unroll 1
            for (int s = 0; 16 * s < nk; ++s) {
                const int left = nk - 16 * s;
                float x[NB][4];
                // the swizzle goes by the row: 16 s adds nothing to its low three bits
                paged_scores<FMT, NB>(it, sm.k[warp] + (16 * s + key) * CACHE_D, key & 7, c, x);
                uint32_t pb[NB][2];
                paged_softmax<NB>(it, x, e.sk[s], e.lsv[s], key < left, key + 2 < left, pb);
                const int cut = left - 4 * c, in_page = (16 * s) & (v_row - 1);
                const uint32_t keep = cut >= 4 ? 0xffffffffu : cut <= 0 ? 0u : 0xffffffffu >> (8 * (4 - cut));
                paged_output<FMT, NB>(it, sm.v[warp] + (16 * s - in_page) * CACHE_D + g * v_row + (((in_page >> 4) ^ v_swz) << 4) + 4 * c,
                                      v_row, keep, pb);
            }
            __syncwarp();                                  // the pages are read
            if (j + 1 < n_mine) {
                const bool batch = ((j + 1) & (PD_BATCH - 1)) == 0;
                if (batch) paged_decode_jobs(a, sm.job[warp], sm.run_off, sm.run_unit, n_run, j_begin, n_mine, who, j + 1, lane);
                fetch(j + 1);
                if (batch) paged_decode_scales(a, sm.job[warp], n_mine, j + 1, lane);
            }
            if (flags & 2) paged_record<NB>(it, a, rec, nrows, lane);
            ++j;
            if (flags & 2) return true;
        }
    };
    paged_decode_jobs(a, sm.job[warp], sm.run_off, sm.run_unit, n_run, j_begin, n_mine, who, 0, lane);
    fetch(0);
    paged_decode_scales(a, sm.job[warp], n_mine, 0, lane);
    while (j < n_mine)
        if (!(sm.job[warp][j & (PD_BATCH - 1)].nrows <= 8 ? item(PagedInt<1>{}) : item(PagedInt<2>{}))) break;
    if (j < n_mine) {                                      // after an abort: no copy may be in flight when the warp ends
        int never = 0;
        bwait(full, j & 1, &never);
    }
}

// The outputs of a response from the records of its prefix's items and of its own, one for each warp that had a share of
// an item. Eight warps to a block, a lane four of the 128 outputs. ALONE: a warp takes a q head; otherwise a block takes
// one and its warps deal the records out. A block a head shortens the chain of records where a head has many; a warp a head
// needs an eighth of the blocks. Which of the two it is goes by the heads in all, as the host does not know the lengths:
// with equal responses the warps cut an item into 16 * warps / heads + 2 records on average, 14 above PD_COMB_ALONE heads.
// Measured, both kernels, L2 flushed, a block a head and a warp a head (32 / 8 heads; groups of 8 responses of 600 tokens behind
// 500): 1024 heads 36.9 and 38.9 us, 2048 49.2 and 47.1, 2304 51.2 and 49.2, 2560 57.3 and 53.2, 4096 73.7 and 67.6; unlike lengths, to 16384
// (2176 heads, calls in a row) 80.3 and 87.8; 448 heads behind 6000 tokens 38.9 and 57.3; 8192 heads of 20 tokens 53.2 and 36.9. The rule
// does not see one long response among many short: behind 131,072 tokens beside 126 of 100 (4064 heads) its heads have some
// 180 records each, and a warp a head takes 139 us where a block takes 98; behind 32,768, 86 and 57. (Dealing such a head out
// to its block's warps, whose other heads are as long: 121 and 72, and 0.5 us more elsewhere.) Bound by latency: the shares, a
// record's two numbers, its outputs.
constexpr int PD_COMB_WARPS = 8, PD_COMB_ALONE = 2304;
template <bool ALONE>
__global__ void __launch_bounds__(PD_COMB_WARPS * 32) k_paged_combine(const PagedArgs a) {
    __shared__ float s_l[PD_COMB_WARPS];
    __shared__ float4 s_o[PD_COMB_WARPS][32];
    const int n_resp = a.nseg - a.G, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int h = ALONE ? blockIdx.y * PD_COMB_WARPS + warp : blockIdx.y;
    wait_first();
    const int4 all = *a.total;
    const int32_t n_units = all.x, first = a.seg[blockIdx.x].first;
    // an even lane has to do with the prefix, an odd one with the response
    const PagedSegRec d = a.seg[lane & 1 ? int(blockIdx.x) : n_units < 0 ? 0 : max(first, 0)];
    // with descriptors that do not fit any response may be this one: all of o and lse become NaN
    const int resp = n_units < 0 ? (int(blockIdx.x) < n_resp ? int(blockIdx.x) : -1)
                                 : first < 0 ? -1 : __shfl_sync(0xffffffffu, d.qbase, 1);
    if (resp < 0 || h >= a.hq) return;
    float M = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    int total = 0;
    if (n_units > 0) {
        // lanes 0 and 1: the first warp with a part of the item, lanes 2 and 3: the last
        const int kh = int((float(h) + 0.5f) * a.inv_r), rho = (resp - d.qbase) * a.r + (h - kh * a.r);
        const int32_t u = d.off + (kh * d.nblk + rho / PD_RB) * d.item + (lane & 2 ? d.last : 0);
        const int32_t who = d.item > 0 ? PagedShare(all.y, all.z, all.w).warp_of(u) + (lane & 2 ? 1 : 0) : 0;
        const int32_t at = d.row + kh * d.qrows + rho + who * PD_RB;   // record row of the first piece, which it is for lanes 0 and 1
        int64_t row[2];
        int n[2];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            row[z] = __shfl_sync(0xffffffffu, at, z);
            n[z] = __shfl_sync(0xffffffffu, who, z + 2) - __shfl_sync(0xffffffffu, who, z);
        }
        total = n[0] + n[1];
        auto rec = [&](int j) { return j < n[0] ? row[0] + int64_t(j) * PD_RB : row[1] + int64_t(j - n[0]) * PD_RB; };
        for (int j = lane; j < total; j += 32) M = fmaxf(M, a.ml[rec(j)].x);
#pragma unroll
        for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll 4
        for (int j = ALONE ? 0 : warp; j < total; j += ALONE ? 1 : PD_COMB_WARPS) {
            const int64_t x = rec(j);
            const float2 ml = a.ml[x];
            const float4 v = *reinterpret_cast<const float4 *>(a.part + x * CACHE_D + 4 * lane);
            const float g = ml.x == M ? 1.f : ex2_approx(ml.x - M);    // a NaN maximum stays one
            L = fmaf(ml.y, g, L);
            acc.x = fmaf(v.x, g, acc.x);
            acc.y = fmaf(v.y, g, acc.y);
            acc.z = fmaf(v.z, g, acc.z);
            acc.w = fmaf(v.w, g, acc.w);
        }
    }
    if (!ALONE) {
        s_o[warp][lane] = acc;
        if (lane == 0) s_l[warp] = L;
        __syncthreads();
        if (warp > 0) return;
        for (int k = 1; k < PD_COMB_WARPS; ++k) {
            const float4 v = s_o[k][lane];
            L += s_l[k];
            acc.x += v.x;
            acc.y += v.y;
            acc.z += v.z;
            acc.w += v.w;
        }
    }
    const float nan = __int_as_float(0x7fc00000), inv = n_units < 0 ? nan : total ? rcp_approx(L) : 0.f;
    __nv_bfloat162 *orow = reinterpret_cast<__nv_bfloat162 *>(a.o + (int64_t(resp) * a.hq + h) * CACHE_D + 4 * lane);
    orow[0] = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
    orow[1] = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
    if (lane == 0)
        a.lse[int64_t(h) * n_resp + resp] = n_units < 0 ? nan : total ? (M + __log2f(L)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace pp
