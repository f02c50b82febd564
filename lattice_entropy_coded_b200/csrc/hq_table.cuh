// hq_table.cuh -- searches in a KV cache's append table.
#pragma once

#include <stdint.h>

#include "hq_device.cuh"

namespace hq {

// The append table is searched through a sample of it in shared memory (all of it up to TOP appends):
// one load's latency for the sample instead of one for every step of a search, which on a short cache
// was most of a kernel's time.
struct TopRow {
    uint64_t first_chunk;
    int64_t token0;
};
template <int TOP>
struct Table {
    const hq_kv_append_row *rows;
    const TopRow *top;
    uint64_t n_appends, heads, stride, n;   // sample s is append s * stride
    __device__ __forceinline__ Table(const hq_kv_append_row *table, uint64_t appends, int h, const TopRow *t)
        : rows(table), top(t), n_appends(appends), heads((uint64_t)h) {
        stride = (n_appends + TOP - 1) / TOP;
        n = (n_appends + stride - 1) / stride;
    }
    // by the whole CTA; the caller synchronises
    __device__ __forceinline__ void load(TopRow *t) const {
        for (uint64_t i = threadIdx.x; i < n; i += blockDim.x)
            t[i] = *reinterpret_cast<const TopRow *>(&rows[i * stride]);
    }
    // the last append whose first chunk is at most x (CHUNK), or whose first token is; 0 if none
    template <bool CHUNK>
    __device__ __forceinline__ uint64_t find(int64_t x) const {
        uint64_t lo = 0, hi = n - 1;
        while (lo < hi) {
            const uint64_t mid = (lo + hi + 1) >> 1;
            if ((CHUNK ? (int64_t)top[mid].first_chunk : top[mid].token0) <= x) lo = mid; else hi = mid - 1;
        }
        if (stride == 1) return lo;
        lo *= stride;
        hi = min(lo + stride, n_appends) - 1;
        while (lo < hi) {
            const uint64_t mid = (lo + hi + 1) >> 1;
            if ((CHUNK ? (int64_t)rows[mid].first_chunk : rows[mid].token0) <= x) lo = mid; else hi = mid - 1;
        }
        return lo;
    }
    // the append of per-head chunk i (chunks of an append lie head-major: its first is heads times the
    // per-head chunks before it), and of token t
    __device__ __forceinline__ uint64_t append_of(uint64_t i) const { return find<true>((int64_t)(i * heads)); }
    __device__ __forceinline__ uint64_t append_of_token(int64_t t) const { return find<false>(t); }
};

}  // namespace hq
