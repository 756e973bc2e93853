// pp_pages.cuh - block tables, slot maps and the free list of a paged cache, built on the device from the segments'
// lengths (pp.h, pp_pages_resize).
//
// Segment s holds old[s] tokens in ceil(old / page) pages and shall hold new[s]. Pages given back go onto the end of
// the free list in the order of (segment, place); pages needed are taken off its end, one after another, in the same
// order. With R pages given back and free[0 .. F) at the start, the i-th page needed is free[F + R - 1 - i]. The slot
// of a new token is table[s][place / page] * page + place % page, and its position id is its place in a prefix, or the
// prefix's new length plus its place in a response.
//
// One launch of one cluster of 8 CTAs, bound by latency: every CTA scans the segments for itself (three running
// counts in shared memory), so nothing is passed between CTAs but the free list, and the cluster barrier stands
// between pages given back and pages taken. A step of 144 segments takes 7.7 us (with one CTA 7.9), a prefill that maps
// 147,786 tokens 15.5 (with one CTA 64). A count that does not fit is seen by every CTA alike before any write, and so is a
// page id outside the pool among those given back, so the call changes everything or nothing.
#pragma once
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include "pp_build.cuh"   // block_exclusive_scan_multi, set_dev_err

namespace pp {

constexpr int PAGES_THREADS = 1024;
constexpr int PAGES_MAX_SEGS = 8192;      // three int32 counts of each segment in one CTA's shared memory

struct PagesArgs {
    const int32_t *group_start, *seg_group, *old_lens, *new_lens;
    int32_t *table, *free_pages;
    const int32_t *n_free_in;
    int32_t *n_free_out, *slots, *pos, *counts;
    int64_t max_pages, room;
    int32_t G, nseg, page_log2, num_pages;
};

// The segment that item i of a running count belongs to: off[s] <= i < off[s + 1].
__device__ __forceinline__ int seg_of(const int32_t *off, int nseg, int32_t i) {
    int lo = 0, hi = nseg;                               // off[lo] <= i < off[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= i) lo = mid; else hi = mid;
    }
    return lo;
}

// Whether one of the R pages given back that this thread of its CTA looks at is none of the pool's. Every CTA looks at all:
// handing the parts' answers round the cluster takes a second barrier, which few pages do not pay for (without a look, with
// this one, with the barrier: 144 pages given back 4.9, 5.6 and 6.9 us; 9,216 pages 5.9, 12.0 and 8.5) and which waits for
// CTAs that must have seen the same lengths.
static __device__ __noinline__ bool pages_out(const int32_t *back, int nseg, const int32_t *new_lens, int lg, const int32_t *table,
                                              int64_t max_pages, int32_t R, int32_t num_pages) {
    bool out = false;
#pragma unroll 4
    for (int32_t i = threadIdx.x; i < R; i += PAGES_THREADS) {
        const int s = seg_of(back, nseg, i);
        const int32_t n = new_lens[s];
        const int64_t at = int64_t(n >> lg) + ((n & ((1 << lg) - 1)) != 0) + (i - back[s]);
        const int32_t id = table[s * max_pages + at];
        out |= id < 0 || id >= num_pages;
    }
    return out;
}

__global__ void __launch_bounds__(PAGES_THREADS) k_pages_resize(const PagesArgs a) {
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    extern __shared__ int32_t sh[];
    int32_t *tok = sh, *need = sh + (a.nseg + 1), *back = sh + 2 * (a.nseg + 1);
    __shared__ int32_t s_tmp[3 * 32];
    __shared__ unsigned long long s_tok, s_need, s_back;
    __shared__ int s_bad;
    const int tid = threadIdx.x, lg = a.page_log2, page = 1 << lg;
    if (tid == 0) {
        s_tok = s_need = s_back = 0;
        s_bad = 0;
    }
    __syncthreads();
    const int32_t n_free = *a.n_free_in;
    unsigned long long t_tok = 0, t_need = 0, t_back = 0;
    bool bad = false;
    for (int s = tid; s < a.nseg; s += PAGES_THREADS) {
        const int32_t o = a.old_lens[s], n = a.new_lens[s], g = a.seg_group[s];
        const bool ok = o >= 0 && n >= 0 && o <= a.max_pages << lg && n <= a.max_pages << lg && g >= 0 && g < a.G &&
                        a.group_start[g] >= 0 && a.group_start[g] <= s && a.group_start[g + 1] > s;
        const int32_t po = ok ? (o >> lg) + ((o & (page - 1)) != 0) : 0, pn = ok ? (n >> lg) + ((n & (page - 1)) != 0) : 0;
        bad |= !ok;
        tok[s] = ok && n > o ? n - o : 0;
        need[s] = pn > po ? pn - po : 0;
        back[s] = po > pn ? po - pn : 0;
        t_tok += tok[s];
        t_need += need[s];
        t_back += back[s];
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        t_tok += __shfl_xor_sync(0xffffffffu, t_tok, o);
        t_need += __shfl_xor_sync(0xffffffffu, t_need, o);
        t_back += __shfl_xor_sync(0xffffffffu, t_back, o);
    }
    if ((tid & 31) == 0 && (t_tok | t_need | t_back)) {
        atomicAdd(&s_tok, t_tok);
        atomicAdd(&s_need, t_need);
        atomicAdd(&s_back, t_back);
    }
    if (bad) s_bad = 1;
    if (tid == 0) tok[a.nseg] = need[a.nseg] = back[a.nseg] = 0;
    __syncthreads();
    // 64-bit totals, so a sum past 2^31 is refused rather than wrapped
    const bool fits = !s_bad && n_free >= 0 && n_free <= a.num_pages && s_back <= (unsigned long long)(a.num_pages - n_free);
    bool ok = fits && s_tok <= (unsigned long long)a.room && s_need <= (unsigned long long)n_free + s_back;
    int32_t err = fits ? DEVERR_NO_ROOM : DEVERR_BAD_PAGES;              // where it is not ok
    const int64_t nthreads = int64_t(cluster.num_blocks()) * PAGES_THREADS;
    const int64_t me = int64_t(cluster.block_rank()) * PAGES_THREADS + tid;
    int32_t R = ok ? int32_t(s_back) : 0, K = ok ? int32_t(s_need) : 0, NT = ok ? int32_t(s_tok) : 0;
    if (ok) {
        int32_t *const arrs[3] = {tok, need, back};
        int32_t tots[3];
        block_exclusive_scan_multi<PAGES_THREADS, 3>(arrs, a.nseg + 1, s_tmp, tots);
        __syncthreads();
        if (R > 0 && __syncthreads_or(pages_out(back, a.nseg, a.new_lens, lg, a.table, a.max_pages, R, a.num_pages))) {
            ok = false;
            err = DEVERR_BAD_PAGES;
            R = K = NT = 0;
        }
        for (int64_t i = me; i < R; i += nthreads) {
            const int s = seg_of(back, a.nseg, int32_t(i));
            const int32_t n = a.new_lens[s];
            const int64_t at = int64_t(n >> lg) + ((n & (page - 1)) != 0) + (i - back[s]);
            a.free_pages[n_free + i] = a.table[s * a.max_pages + at];
        }
    }
    cluster.sync();                                      // n_free is read and the pages given back are listed
    if (me == 0) {
        *a.n_free_out = n_free + R - K;
        a.counts[0] = NT;
        a.counts[1] = K;
        a.counts[2] = R;
        a.counts[3] = ok ? 1 : 0;
        if (!ok) set_dev_err(err);
    }
    const int32_t top = n_free + R - 1;
    for (int64_t i = me; i < K; i += nthreads) {
        const int s = seg_of(need, a.nseg, int32_t(i));
        const int32_t o = a.old_lens[s];
        const int64_t at = int64_t(o >> lg) + ((o & (page - 1)) != 0) + (i - need[s]);
        a.table[s * a.max_pages + at] = a.free_pages[top - i];
    }
    // four tokens to a thread at a time: one search, and one look at the table for all that share a page
    const bool v4 = ((reinterpret_cast<uintptr_t>(a.slots) | reinterpret_cast<uintptr_t>(a.pos)) & 15) == 0;
    for (int64_t i0 = 4 * me; i0 < a.room; i0 += 4 * nthreads) {
        int32_t slot[4] = {-1, -1, -1, -1}, pos[4] = {0, 0, 0, 0};
        if (i0 < NT) {
            int s = seg_of(tok, a.nseg, int32_t(i0));
            int seg = -1, page_at = -1;
            int32_t o = 0, id = 0, before = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int32_t i = int32_t(i0) + e;
                if (i >= NT) break;
                while (i >= tok[s + 1]) ++s;
                if (s != seg) {
                    seg = s;
                    page_at = -1;
                    o = a.old_lens[s];
                    const int32_t first = a.group_start[a.seg_group[s]];
                    before = s == first ? 0 : a.new_lens[first];
                }
                const int32_t at = o + (i - tok[s]);
                if (at >> lg != page_at) {
                    page_at = at >> lg;
                    const int32_t held = (o >> lg) + ((o & (page - 1)) != 0);
                    // a page taken by this call is read off the free list: its table entry may be another CTA's write
                    id = page_at < held ? a.table[s * a.max_pages + page_at] : a.free_pages[top - (need[s] + page_at - held)];
                    if (id < 0 || id >= a.num_pages) {     // the table or the free list names a page outside the pool
                        set_dev_err(DEVERR_BAD_PAGES);
                        id = -1;
                    }
                }
                pos[e] = at + before;
                slot[e] = id < 0 ? -1 : (id << lg) + (at & (page - 1));
            }
        }
        if (v4 && i0 + 4 <= a.room) {
            *reinterpret_cast<int4 *>(a.slots + i0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
            *reinterpret_cast<int4 *>(a.pos + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        } else {
            for (int e = 0; e < 4 && i0 + e < a.room; ++e) {
                a.slots[i0 + e] = slot[e];
                a.pos[i0 + e] = pos[e];
            }
        }
    }
}

}  // namespace pp
