// gdr_paged.cuh -- the paged key/value cache as its kernels see it: which
// sequence owns a packed row, and where a token lies in the pages.
#pragma once

#include "gdr.h"
#include "gdr_common.cuh"

namespace gdr {
namespace paged {

constexpr int D = 256;
constexpr int kBadPage = GDR_ERR_INVALID_ARG;
constexpr int64_t kTooLong = 0x7fffff00;  // 2^31 - 256: no sequence has so many tokens
constexpr float kScaleMin = 9.094947017729282e-13f;  // 2^-40: a row of zeros keeps a usable scale

// The sequence that owns packed row t: the s with cu[s] <= t < cu[s + 1], or n_seq
// when no sequence owns it.  One whole warp calls it; every lane gets s.  cu
// never decreases, so s is the number of ends cu[1 ..] that are <= t: each round
// looks at 32 ends spread over what is left and keeps the stretch between two
// of them, log_32(n_seq) dependent loads in all.
__device__ __forceinline__ int find_sequence(const int32_t *cu, int n_seq, int t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = n_seq;  // the answer is in [lo, lo + n]
    while (n > 0) {
        const int step = (n + 31) >> 5;
        const int64_t i = lo + (int64_t)(lane + 1) * step;  // the end with this number, 1-based
        const bool past = i <= lo + n && __ldg(cu + i) <= t;
        const int k = __popc(__ballot_sync(kFullMask, past));
        const int left = n - k * step;
        lo += k * step;
        n = left < step - 1 ? left : step - 1;
    }
    return lo;
}

// Row of token t of sequence s of kv head g in the [n_pages, H_kv, page_size]
// rows of the cache, or -1 when the token has no valid page.
__device__ __forceinline__ int cache_row(const gdr_kv_pages &c, int shift, int s, int g, int64_t t) {
    const int64_t i = t >> shift;
    if (t < 0 || t + 1 >= kTooLong || i >= c.table_width) return -1;
    const int page = __ldg(c.page_table + s * c.table_stride + i);
    if (page < 0 || page >= c.n_pages) return -1;
    return (page * c.H_kv + g) * c.page_size + (int)(t & (c.page_size - 1));
}

inline int log2_of(int power) {
    int s = 0;
    while ((1 << s) < power) ++s;
    return s;
}

}  // namespace paged
}  // namespace gdr
