// vc_paged.cuh -- device-side view of a batch over the paged cache: which rows
// and positions a sequence has, and where a position lies.  Everything read
// from cu, kv_len and table is clamped or checked here, so that no value in
// them leads outside the caller's buffers.
#pragma once
#include <cstdint>

#include "vc_internal.h"

namespace vc {

struct SeqInfo {
    int q0, n;  // first row of the call and number of rows
    int L;      // tokens in the cache
};

__device__ __forceinline__ void flag_invalid(int32_t* dev_status) {
    if (dev_status) atomicMax(reinterpret_cast<int*>(dev_status), (int)VC_ERR_INVALID_ARG);
}

__device__ __forceinline__ SeqInfo seq_info(const CacheView& c, int b) {
    SeqInfo s;
    const int a = __ldg(c.cu + b), e = __ldg(c.cu + b + 1), len = __ldg(c.kv_len + b);
    s.q0 = min(max(a, 0), c.T);
    s.n = min(max(e, s.q0), c.T) - s.q0;
    s.L = min(max(len, 0), c.cols << c.page_log2);
    return s;
}

// Whether cu[b], cu[b+1] and kv_len[b] keep the batch's rules.
__device__ __forceinline__ bool seq_valid(const CacheView& c, int b) {
    const int a = __ldg(c.cu + b), e = __ldg(c.cu + b + 1), len = __ldg(c.kv_len + b);
    return a >= 0 && e >= a && e <= c.T && len >= 0 && len <= (c.cols << c.page_log2);
}

// Page of position p (0 <= p < cols * page_size), or -1 where it is not there.
__device__ __forceinline__ int page_of(const CacheView& c, int b, int p) {
    const int pg = __ldg(c.table + (int64_t)b * c.s_table + (p >> c.page_log2));
    return (pg >= 0 && pg < c.pages) ? pg : -1;
}

}  // namespace vc
