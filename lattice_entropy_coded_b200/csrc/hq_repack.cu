// hq_repack.cu -- hq_kv_repack: ranges of a compressed KV cache's tokens copied into another
// cache, re-cut into full chunks.  The symbols of a token do not depend on where its chunk
// starts (its dither counter is its position), so nothing is decoded: a tile's bits are one
// run of each plane of its chunk, and a new chunk's planes are those runs joined.
//
// Two launches.  The first finds, one warp to a new chunk, each tile's chunk in the source
// and the run of its unary bits there (the 128-th terminators, by population counts), and
// writes 16 bytes per tile and the new chunk's words.  The second sums the words of the
// chunks before its own (contiguous) chunks, which costs each CTA a few bytes per chunk
// read from L2 and no third launch, and assembles the planes, a lane to a word: every word
// joins the bits of at most two tiles (a tile holds 128 unary bits or more, 16 coset bits,
// and at least 64 remainder bits where it has any).
// Bound: the stream's bytes, read twice (the second time from L2 up to its size) and
// written once.
#include <cuda_runtime.h>
#include <stdint.h>

#include "hq_device.cuh"

namespace hq {

namespace {

constexpr int kMaxRanges = 32;
constexpr int kRepackWarps = 8;

struct RepackRange {
    int64_t begin, end;
    uint64_t first_chunk;   // its first chunk in the new cache
};

struct RepackArgs {
    const uint32_t *src_words;
    uint64_t src_cap;
    const uint64_t *src_offsets;
    uint64_t src_chunks;
    const hq_kv_append_row *src_table;
    uint64_t src_appends;
    const hq_stats *src_stats;
    uint32_t *words;
    uint64_t cap;
    uint64_t *offsets;
    hq_kv_append_row *table;
    uint64_t *tail;
    hq_stats *stats;
    uint4 *tiles;          // per new tile: source chunk's first word | tile << 48 | its tiles << 56, unary start, length
    uint32_t *sizes;       // per new chunk: words
    uint64_t n_chunks;
    int heads, n_ranges, e8;
    uint32_t rem_bits;     // remainder bits of a tile
    RepackRange range[kMaxRanges];
};

// Append row of the last append that starts at or before token t (row 0 if none).
__device__ __forceinline__ uint64_t row_of_token(const hq_kv_append_row *table, uint64_t n, int64_t t) {
    uint64_t lo = 0, hi = n - 1;
    while (lo < hi) {
        const uint64_t mid = (lo + hi + 1) >> 1;
        if (table[mid].token0 <= t) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// 32 bits of the stream from absolute bit b on; `need` of them are used, and the second word is
// read only if they reach into it.
__device__ __forceinline__ uint32_t stream_bits(const uint32_t *w, uint64_t b, uint32_t need) {
    const uint32_t *p = w + (b >> 5);
    const uint32_t sh = (uint32_t)b & 31u;
    const uint32_t a0 = __ldg(p);
    const uint32_t a1 = sh + need > 32u ? __ldg(p + 1) : 0u;
    return __funnelshift_r(a0, a1, sh);
}

__device__ __forceinline__ uint32_t coset_words(const RepackArgs &a, uint32_t n) {
    return a.e8 ? (16u * n + 31u) >> 5 : 0u;
}
__device__ __forceinline__ uint32_t rem_words(const RepackArgs &a, uint32_t n) { return (n * a.rem_bits + 31u) >> 5; }

// Which range and which tokens new chunk c holds.
struct NewChunk {
    int r, h;
    int64_t t0;
    uint32_t n;
};
__device__ __forceinline__ NewChunk new_chunk(const RepackArgs &a, uint64_t c) {
    NewChunk g;
    g.r = 0;
    while (g.r + 1 < a.n_ranges && a.range[g.r + 1].first_chunk <= c) g.r++;
    const int64_t T = a.range[g.r].end - a.range[g.r].begin;
    unsigned long long h, j;
    divmod_u64(c - a.range[g.r].first_chunk, (unsigned long long)((T + 31) / 32), h, j);
    g.h = (int)h;
    g.t0 = a.range[g.r].begin + 32 * (int64_t)j;
    const int64_t left = a.range[g.r].end - g.t0;
    g.n = (uint32_t)(left < 32 ? left : 32);
    return g;
}

// First unary bit of every tile of a chunk of n tiles (start[0 .. n]) by the whole warp; false unless
// the plane of nu words holds exactly 128 n terminators.
__device__ __forceinline__ bool tile_starts(const uint32_t *un, uint32_t nu, uint32_t n, uint32_t *start, int lane) {
    uint32_t seen = 0;
    if (lane == 0) start[0] = 0;
    for (uint32_t i0 = 0; i0 < nu; i0 += 128) {
        uint32_t w[4];
#pragma unroll
        for (int u = 0; u < 4; u++) {
            const uint32_t i = i0 + 32u * u + lane;
            w[u] = i < nu ? __ldg(un + i) : 0u;
        }
#pragma unroll
        for (int u = 0; u < 4; u++) {
            const uint32_t p = __popc(w[u]);
            uint32_t incl = p;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            const uint32_t before = seen + incl - p;
            // the word holds terminators before .. before + p - 1; number 128 t - 1 ends tile t - 1
            const uint32_t t = (before + 128u) >> 7;
            if (128u * t - 1u < before + p && t <= n) {
                uint32_t x = w[u];
                for (uint32_t d = 128u * t - 1u - before; d; d--) x &= x - 1u;
                start[t] = (i0 + 32u * u + lane) * 32u + (uint32_t)__ffs((int)x);
            }
            seen += __shfl_sync(0xffffffffu, incl, 31);
        }
    }
    __syncwarp();
    return seen == 128u * n;
}

__global__ void __launch_bounds__(kRepackWarps * 32) repack_measure(const __grid_constant__ RepackArgs a) {
    __shared__ uint32_t starts[kRepackWarps][36];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x == 0) {
        if (threadIdx.x < (unsigned)a.n_ranges) {
            const RepackRange r = a.range[threadIdx.x];
            hq_kv_append_row row = a.src_table[row_of_token(a.src_table, a.src_appends, r.begin)];
            row.first_chunk = r.first_chunk;
            row.token0 = r.begin;
            row.tokens = (int32_t)(r.end - r.begin);
            a.table[threadIdx.x] = row;
        }
        if (threadIdx.x == 0) {
            hq_stats z = {};
            z.max_symbol = a.src_stats->max_symbol;
            z.max_abs_code = a.src_stats->max_abs_code;
            *a.stats = z;
        }
    }
    const uint64_t c = (uint64_t)blockIdx.x * kRepackWarps + warp;
    if (c >= a.n_chunks) return;
    const NewChunk g = new_chunk(a, c);
    // the lane's token in the source; its scale has to be that of the range's first token
    const int64_t t = g.t0 + ((uint32_t)lane < g.n ? lane : (int)g.n - 1);
    const hq_kv_append_row ref = a.src_table[row_of_token(a.src_table, a.src_appends, a.range[g.r].begin)];
    const hq_kv_append_row row = a.src_table[row_of_token(a.src_table, a.src_appends, t)];
    const int64_t in = t - row.token0;
    bool ok = in >= 0 && in < row.tokens && __float_as_uint(row.alpha) == __float_as_uint(ref.alpha) &&
              __float_as_uint(row.scale_inv) == __float_as_uint(ref.scale_inv);
    uint64_t chunk = 0, w0 = 0;
    uint32_t n = 0, nu = 0, head_words = 0;
    const uint32_t ti = (uint32_t)in & 31u;
    if (ok) {
        const int64_t left = (int64_t)row.tokens - (in & ~INT64_C(31));
        n = (uint32_t)(left < 32 ? left : 32);
        chunk = row.first_chunk + (uint64_t)g.h * (uint64_t)(((int64_t)row.tokens + 31) / 32) + (uint64_t)(in >> 5);
        ok = chunk < a.src_chunks;
    }
    if (ok) {
        w0 = a.src_offsets[chunk];
        const uint64_t w1 = a.src_offsets[chunk + 1];
        head_words = coset_words(a, n) + rem_words(a, n);
        ok = w0 <= w1 && w1 <= a.src_cap && w1 - w0 >= head_words && w1 - w0 - head_words < (kMaxUnaryBits / 32u);
        nu = ok ? (uint32_t)(w1 - w0) - head_words : 0u;
    }
    uint32_t ustart = 0, uend = 0;
    // short chunks of up to four tiles (one-token appends): the lane reads its chunk's plane by itself
    const bool alone = ok && n <= 4u && nu <= 256u;
    if (alone) {
        const uint32_t *un = a.src_words + w0 + head_words;
        uint32_t seen = 0;
        for (uint32_t i = 0; i < nu; i++) {
            const uint32_t w = __ldg(un + i), p = __popc(w);
            const uint32_t e0 = 128u * ti, e1 = e0 + 128u;   // terminators before the tile, and up to its last
            if (seen < e0 && seen + p >= e0) {
                uint32_t x = w;
                for (uint32_t d = e0 - 1u - seen; d; d--) x &= x - 1u;
                ustart = i * 32u + (uint32_t)__ffs((int)x);
            }
            if (seen < e1 && seen + p >= e1) {
                uint32_t x = w;
                for (uint32_t d = e1 - 1u - seen; d; d--) x &= x - 1u;
                uend = i * 32u + (uint32_t)__ffs((int)x);
            }
            seen += p;
        }
        ok = seen == 128u * n;
    }
    // larger ones: the warp reads each distinct chunk once
    unsigned todo = __ballot_sync(0xffffffffu, ok && !alone);
    while (todo) {
        const int lead = __ffs((int)todo) - 1;
        const uint64_t lc = __shfl_sync(0xffffffffu, (unsigned long long)chunk, lead);
        const uint64_t lw = __shfl_sync(0xffffffffu, (unsigned long long)(w0 + head_words), lead);
        const uint32_t ln = __shfl_sync(0xffffffffu, n, lead), lu = __shfl_sync(0xffffffffu, nu, lead);
        const bool good = tile_starts(a.src_words + lw, lu, ln, starts[warp], lane);
        const bool mine = ok && !alone && chunk == lc;
        if (mine) {
            if (good) {
                ustart = starts[warp][ti];
                uend = starts[warp][ti + 1];
            } else {
                ok = false;
            }
        }
        todo &= ~__ballot_sync(0xffffffffu, mine || (todo >> lane & 1u && chunk == lc));
        __syncwarp();
    }
    // a tile that is not there, or not sound, becomes one of zero symbols (128 terminators)
    uint32_t len = ok ? uend - ustart : 128u;
    unsigned long long bits = (uint32_t)lane < g.n ? len : 0u;
#pragma unroll
    for (int o = 16; o; o >>= 1) bits += __shfl_xor_sync(0xffffffffu, bits, o);
    if (bits >= kMaxUnaryBits) {   // tiles of enormous symbols that together exceed what a chunk may hold
        ok = false;
        len = 128u;
        bits = 128ull * g.n;
    }
    const uint64_t tag = ok ? w0 | (uint64_t)ti << 48 | (uint64_t)n << 56 : 0ull;
    if ((uint32_t)lane < g.n) a.tiles[c * 32 + lane] = make_uint4((uint32_t)tag, (uint32_t)(tag >> 32), ustart, len);
    if (lane == 0) a.sizes[c] = coset_words(a, g.n) + rem_words(a, g.n) + (uint32_t)((bits + 31) >> 5);
}

// Sum over the CTA of one value per thread; the same in all.
__device__ __forceinline__ unsigned long long cta_sum(unsigned long long v, unsigned long long *tmp) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int i = 0; i < kRepackWarps; i++) v += tmp[i];
    return v;
}

__global__ void __launch_bounds__(kRepackWarps * 32) repack_copy(const __grid_constant__ RepackArgs a) {
    __shared__ unsigned long long tmp[kRepackWarps];
    __shared__ unsigned long long src[kRepackWarps][32];   // first word of each tile's source chunk
    __shared__ uint32_t info[kRepackWarps][32];            // tile | its chunk's tiles << 8 (0: zero symbols)
    __shared__ uint32_t from[kRepackWarps][32];            // its first unary bit there
    __shared__ uint32_t at[kRepackWarps][33];              // and in the new plane
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint64_t per = (a.n_chunks + gridDim.x - 1) / gridDim.x;
    const uint64_t c0 = per * blockIdx.x, c1 = min(a.n_chunks, c0 + per);
    if (c0 >= c1) return;
    unsigned long long before = 0;
    for (uint64_t i = threadIdx.x; i < c0; i += blockDim.x) before += a.sizes[i];
    unsigned long long base = cta_sum(before, tmp);
    unsigned long long payload = 0;
    uint32_t status = 0;
    for (uint64_t cb = c0; cb < c1; cb += kRepackWarps) {
        const uint64_t c = cb + warp;
        const bool on = c < c1;
        const uint32_t size = on ? a.sizes[c] : 0u;
        __syncthreads();
        if (lane == 0) tmp[warp] = size;
        __syncthreads();
        unsigned long long w0 = base, all = 0;
#pragma unroll
        for (int i = 0; i < kRepackWarps; i++) {
            if (i < warp) w0 += tmp[i];
            all += tmp[i];
        }
        base += all;
        if (!on) continue;
        const NewChunk g = new_chunk(a, c);
        const bool mine = (uint32_t)lane < g.n;
        uint4 d = make_uint4(0u, 0u, 0u, 0u);
        if (mine) d = a.tiles[c * 32 + lane];
        uint32_t incl = mine ? d.w : 0u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        src[warp][lane] = ((unsigned long long)(d.y & 0xFFFFu) << 32) | d.x;
        info[warp][lane] = ((d.y >> 16) & 0xFFu) | ((d.y >> 24) << 8);
        from[warp][lane] = d.z;
        at[warp][lane + 1] = incl;
        if (lane == 0) at[warp][0] = 0;
        __syncwarp();
        if (mine && (d.y >> 24) == 0) status |= HQ_ST_CORRUPT;
        const uint32_t nbits = at[warp][32];
        if (lane == 0) payload += (unsigned long long)nbits + g.n * (a.rem_bits + (a.e8 ? 16u : 0u));
        const uint32_t nc = coset_words(a, g.n), nr = rem_words(a, g.n), nu = (nbits + 31u) >> 5;
        const uint32_t total = nc + nr + nu;
        if (lane == 0) a.offsets[c] = w0;
        for (uint32_t i = lane; i < total; i += 32) {
            uint32_t v = 0;
            if (i < nc) {
#pragma unroll
                for (int u = 0; u < 2; u++) {
                    const uint32_t t = 2u * i + u;
                    const uint32_t f = t < g.n ? info[warp][t] : 0u;
                    if (f) v |= (stream_bits(a.src_words, src[warp][t] * 32 + 16u * (f & 0xFFu), 16u) & 0xFFFFu)
                                << (16 * u);
                }
            } else if (i < nc + nr) {
                const uint32_t b = 32u * (i - nc), t = b / a.rem_bits, skip = b - t * a.rem_bits;
                const uint32_t have = min(32u, a.rem_bits - skip);
                uint32_t f = info[warp][t];
                if (f) {
                    const uint64_t s = (src[warp][t] + coset_words(a, f >> 8)) * 32 + (uint64_t)(f & 0xFFu) * a.rem_bits;
                    v = stream_bits(a.src_words, s + skip, have);
                    if (have < 32u) v &= (1u << have) - 1u;
                }
                if (have < 32u && t + 1 < g.n && (f = info[warp][t + 1])) {
                    const uint64_t s =
                        (src[warp][t + 1] + coset_words(a, f >> 8)) * 32 + (uint64_t)(f & 0xFFu) * a.rem_bits;
                    v |= stream_bits(a.src_words, s, 32u - have) << have;
                }
            } else {
                const uint32_t b = 32u * (i - nc - nr);
                uint32_t t = 0;
#pragma unroll
                for (int o = 16; o; o >>= 1)
                    if (t + o < g.n && at[warp][t + o] <= b) t += o;
                const uint32_t skip = b - at[warp][t];
                const uint32_t have = min(32u, at[warp][t + 1] - b);
                uint32_t f = info[warp][t];
                v = 0xFFFFFFFFu;
                if (f)
                    v = stream_bits(a.src_words,
                                    (src[warp][t] + coset_words(a, f >> 8) + rem_words(a, f >> 8)) * 32 +
                                        from[warp][t] + skip, have);
                if (have < 32u) {
                    v &= (1u << have) - 1u;
                    if (t + 1 < g.n) {
                        f = info[warp][t + 1];
                        uint32_t x = 0xFFFFFFFFu;
                        if (f)
                            x = stream_bits(a.src_words,
                                            (src[warp][t + 1] + coset_words(a, f >> 8) + rem_words(a, f >> 8)) * 32 +
                                                from[warp][t + 1], 32u - have);
                        v |= x << have;
                    }
                }
            }
            if (w0 + i < a.cap) a.words[w0 + i] = v;
        }
        if (w0 + total > a.cap) status |= HQ_ST_CAPACITY;
        if (c + 1 == a.n_chunks && lane == 0) {
            a.offsets[c + 1] = w0 + total;
            a.tail[0] = w0 + total;
            a.tail[1] = w0 + total;
            a.stats->stream_words = w0 + total;
        }
        __syncwarp();
    }
    payload = cta_sum(payload, tmp);
    if (threadIdx.x == 0) atomicAdd(reinterpret_cast<unsigned long long *>(&a.stats->payload_bits), payload);
    status = __reduce_or_sync(0xffffffffu, status);
    if (lane == 0 && status) atomicOr(&a.stats->status, status);
}

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

// The ranges' chunks (0 for none), or -1 if a range is empty, out of order or beyond `tokens`.
int64_t chunks_of_ranges(int32_t heads, const int64_t *ranges, int32_t n, int64_t tokens) {
    int64_t last = 0;
    uint64_t chunks = 0;
    for (int32_t i = 0; i < n; i++) {
        const int64_t b = ranges[2 * i], e = ranges[2 * i + 1];
        if (b < last || e <= b || e > tokens || e - b > INT64_C(0x7FFFFFFF)) return -1;
        chunks += (uint64_t)heads * (uint64_t)((e - b + 31) / 32);
        last = e;
    }
    return (int64_t)chunks;
}

// Whether two buffers share a byte.
bool overlap(const void *a, uint64_t na, const void *b, uint64_t nb) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return na && nb && x < y + nb && y < x + na;
}

}  // namespace

}  // namespace hq

using namespace hq;

extern "C" int hq_kv_repack_workspace_bytes(int32_t heads, const int64_t *h_ranges, int32_t n_ranges, size_t *bytes) {
    if (!bytes || heads <= 0 || n_ranges < 0 || (n_ranges && !h_ranges)) return HQ_EINVAL;
    if (n_ranges > kMaxRanges) return HQ_EUNSUPPORTED;
    const int64_t c = chunks_of_ranges(heads, h_ranges, n_ranges, INT64_MAX);
    if (c < 0) return HQ_EINVAL;
    if (c > (INT64_C(1) << 31)) return HQ_EUNSUPPORTED;
    *bytes = ((size_t)c * (32 * sizeof(uint4) + sizeof(uint32_t)) + 255) & ~(size_t)255;
    return HQ_OK;
}

extern "C" int hq_kv_repack(const hq_kv_cache *src, hq_kv_cache *dst, const int64_t *h_ranges, int32_t n_ranges,
                            void *workspace, size_t ws_bytes, void *cuda_stream) {
    if (!src || !dst || src == dst || !src->d_words || !dst->d_words || n_ranges < 0 || (n_ranges && !h_ranges))
        return HQ_EINVAL;
    if (n_ranges > kMaxRanges) return HQ_EUNSUPPORTED;
    const hq_params &p = src->params, &d = dst->params;
    if (src->heads <= 0 || dst->heads != src->heads || dst->head_dim != src->head_dim || d.lattice != p.lattice ||
        d.rice_k != p.rice_k || k_last_of(d) != k_last_of(p) || d.seed != p.seed || d.dither != p.dither ||
        d.rotation != p.rotation)
        return HQ_EINVAL;
    if (overlap(src->d_words, 4 * src->cap_words, dst->d_words, 4 * dst->cap_words) ||
        overlap(src->d_offsets, 8 * src->offsets_cap, dst->d_offsets, 8 * dst->offsets_cap) ||
        overlap(src->d_table, 32 * src->table_cap, dst->d_table, 32 * dst->table_cap) ||
        overlap(src->d_tail, 16, dst->d_tail, 16) || overlap(src->d_stats, sizeof(hq_stats), dst->d_stats, sizeof(hq_stats)))
        return HQ_EINVAL;
    const int64_t chunks = chunks_of_ranges(src->heads, h_ranges, n_ranges, src->tokens);
    if (chunks < 0) return HQ_EINVAL;
    if ((uint64_t)chunks + 1 > dst->offsets_cap || (uint64_t)n_ranges > dst->table_cap) return HQ_EINVAL;
    if (chunks > (INT64_C(1) << 31)) return HQ_EUNSUPPORTED;
    cudaStream_t s = (cudaStream_t)cuda_stream;
    if (chunks == 0) {
        if (cudaMemsetAsync(dst->d_tail, 0, 2 * sizeof(uint64_t), s) != cudaSuccess ||
            cudaMemsetAsync(dst->d_stats, 0, sizeof(hq_stats), s) != cudaSuccess ||
            cudaMemsetAsync(dst->d_offsets, 0, sizeof(uint64_t), s) != cudaSuccess)
            return HQ_ECUDA;
        dst->tokens = 0;
        dst->chunks = 0;
        dst->appends = 0;
        return HQ_OK;
    }
    size_t need = 0;
    int rc = hq_kv_repack_workspace_bytes(src->heads, h_ranges, n_ranges, &need);
    if (rc) return rc;
    if (!workspace || !aligned(workspace, 16) || ws_bytes < need) return HQ_EINVAL;
    RepackArgs a;
    a.src_words = src->d_words;
    a.src_cap = src->cap_words;
    a.src_offsets = src->d_offsets;
    a.src_chunks = src->chunks;
    a.src_table = src->d_table;
    a.src_appends = src->appends;
    a.src_stats = src->d_stats;
    a.words = dst->d_words;
    a.cap = dst->cap_words;
    a.offsets = dst->d_offsets;
    a.table = dst->d_table;
    a.tail = dst->d_tail;
    a.stats = dst->d_stats;
    a.tiles = (uint4 *)workspace;
    a.sizes = (uint32_t *)((char *)workspace + (size_t)chunks * 32 * sizeof(uint4));
    a.n_chunks = (uint64_t)chunks;
    a.heads = src->heads;
    a.n_ranges = n_ranges;
    a.e8 = p.lattice == HQ_E8;
    const int n = p.lattice == HQ_E8 ? 8 : p.lattice == HQ_D4 ? 4 : p.lattice == HQ_A2 ? 2 : 1;
    a.rem_bits = (uint32_t)(kTile / n) * (uint32_t)((n - 1) * p.rice_k + k_last_of(p));
    uint64_t first = 0;
    for (int32_t i = 0; i < n_ranges; i++) {
        a.range[i] = {h_ranges[2 * i], h_ranges[2 * i + 1], first};
        first += (uint64_t)src->heads * (uint64_t)((a.range[i].end - a.range[i].begin + 31) / 32);
    }
    const uint64_t ctas = (a.n_chunks + kRepackWarps - 1) / kRepackWarps;
    repack_measure<<<(unsigned)ctas, kRepackWarps * 32, 0, s>>>(a);
    if (cudaGetLastError() != cudaSuccess) return HQ_ECUDA;
    // all resident at once (8 CTAs of 256 threads per SM): each sums the sizes before its own chunks
    const uint64_t most = 148 * 8;
    repack_copy<<<(unsigned)(ctas < most ? ctas : most), kRepackWarps * 32, 0, s>>>(a);
    if (cudaGetLastError() != cudaSuccess) return HQ_ECUDA;
    dst->tokens = h_ranges[2 * n_ranges - 1];
    dst->chunks = (uint64_t)chunks;
    dst->appends = (uint64_t)n_ranges;
    return HQ_OK;
}
