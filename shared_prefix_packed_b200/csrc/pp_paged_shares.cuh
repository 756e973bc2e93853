// pp_paged_shares.cuh - the arithmetic of pp_paged_decode's work list (pp_paged.cuh): what jobs cost, which warp has which,
// and where the records of its items lie. Plain integers, compiled for the host too.
#pragma once
#include <cstdint>

namespace pp {

constexpr int PD_CH = 64;             // keys of a job
constexpr int PD_RB = 16;             // query rows of a job, at most
constexpr int PD_WARPS = 12;
constexpr int PD_MAX_CTAS = 148;      // what a workspace is sized for

// What a job costs, in units that the warps' shares are equal in: one of up to 8 query rows, one of up to 16, and the
// first of an item more (its queries and its record). Measured on 16 groups of 8 responses (prefixes of 256 to 1024
// tokens, 64 to 2048 of their own) and 17 of 4 (to 16384 and 4096), 32 / 8 heads: with equal numbers of jobs 64.4 and 86.4
// us, with 2, 3 and 1 units 56.3 and 80.7, with 2, 3, 2 57.3 and 81.0, with 2, 3, 3 56.8 and 81.3, with 1, 2, 2 58.7 and 91.4.
constexpr int PD_COST8 = 2, PD_COST16 = 3, PD_COST_ITEM = 1;

__host__ __device__ __forceinline__ int32_t paged_cost(int32_t qrows) { return qrows <= 8 ? PD_COST8 : PD_COST16; }
// Units of an item of nch jobs, and before its job k.
__host__ __device__ __forceinline__ int32_t paged_item(int32_t nch, int32_t qrows) {
    return nch ? PD_COST_ITEM + nch * paged_cost(qrows) : 0;
}
__host__ __device__ __forceinline__ int32_t paged_start(int32_t k, int32_t qrows) {
    return k ? PD_COST_ITEM + k * paged_cost(qrows) : 0;
}
// The first job of an item that begins at its unit `at` or after it: job k > 0 begins at PD_COST_ITEM + k cost.
__host__ __device__ __forceinline__ int32_t paged_job_from(int32_t at, int32_t cost) {
    if (at == 0) return 0;
    const int32_t k = (at - PD_COST_ITEM + cost - 1) / cost;
    return k > 1 ? k : 1;
}
// First record row of a segment's items, without the warp's part: prefixes and responses in order, each hq rows for every
// response that sees it. r0: responses before the group, kg: those in it, qbase: the first that sees the segment.
__host__ __device__ __forceinline__ int32_t paged_row(bool prefix, int32_t r0, int32_t kg, int32_t qbase, int32_t hq) {
    return (prefix ? 2 * r0 : r0 + kg + qbase) * hq;
}
// Record rows of a call.
__host__ __device__ __forceinline__ int64_t paged_rows(int32_t n_resp, int32_t hq) {
    return 2 * int64_t(n_resp) * hq + int64_t(PD_MAX_CTAS) * PD_WARPS * PD_RB;
}

// The shares of n units among up to `warps` warps: a job is its warp's whose share holds its first unit. As many warps
// take part as leave each the units of the longest job, so every one of them has a job, and the warps that have a part
// of an item follow one another.
struct PagedShare {
    int32_t many, per, more;                               // warps, units of a warp, warps with one more
    __host__ __device__ PagedShare(int32_t n, int32_t warps) {
        const int32_t most = n / (PD_COST_ITEM + PD_COST16);
        many = most < 1 ? 1 : most < warps ? most : warps;
        per = n / many;
        more = n - per * many;
    }
    __host__ __device__ PagedShare(int32_t many_, int32_t per_, int32_t more_) : many(many_), per(per_), more(more_) {}
    __host__ __device__ int32_t begin(int32_t w) const { return w >= many ? per * many + more : per * w + (w < more ? w : more); }
    __host__ __device__ int32_t warp_of(int32_t u) const {
        const int32_t cut = more * (per + 1);
        const bool low = u < cut;
        return (low ? 0 : more) + int32_t(uint32_t(low ? u : u - cut) / uint32_t(low ? per + 1 : per));
    }
};

}  // namespace pp
