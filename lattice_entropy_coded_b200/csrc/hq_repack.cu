// hq_repack.cu -- hq_kv_repack: ranges of a compressed KV cache's tokens copied into another
// cache, re-cut into full chunks.  The symbols of a token do not depend on where its chunk
// starts (its dither counter is its position), so nothing is decoded: a tile's bits are one
// run of each plane of its chunk, and a new chunk's planes are those runs joined.
//
// Two launches.  The first finds, one warp to a new chunk, each tile's chunk in the source and the
// run of its unary bits there, and writes 16 bytes per tile and the new chunk's words.  A new chunk
// that is a whole chunk of the source (a fork of full chunks) needs only its terminators counted;
// else the warp finds every 128th terminator of each chunk it touches, and tiles in chunks of their
// own (one-token appends) are counted by their lanes.  The second launch sums the words before its
// chunks and copies the planes run by run (tiles that follow one another in one source chunk), a lane
// to a word: a funnel shift of two source words, and a second pair where two runs meet in a word
// (never three: a tile has 128 unary bits or more, 16 coset bits, 64 remainder bits or none).
// Bound: the stream's bytes, read twice (the second time from L2 up to its size) and written once, of which a
// fork of 65535 tokens x 8 heads at 4 bits (33 MB) gets 1.5 TB/s (43 us; 10 us at the copy rate); short calls
// by their two launches and dependent loads (16 us).
#include <cuda_runtime.h>
#include <stdint.h>

#include "hq_decode.cuh"
#include "hq_table.cuh"

namespace hq {

namespace {

constexpr int kMaxRanges = 32;
constexpr int kRepackWarps = 4;
constexpr int kTop = 512;   // rows of the append table sampled into shared memory

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
    uint64_t *sums;        // per CTA of the first launch: words of its chunks
    uint64_t n_chunks;
    int heads, n_ranges, e8;
    uint32_t rem_bits;     // remainder bits of a tile
    RepackRange range[kMaxRanges];
};

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
// the plane of nu words holds exactly 128 n terminators.  128 words at a time, as the attention's scan:
// population counts, two sets of 32 scanned in one register (twice); a word that holds the last terminator of a
// tile (at most one) notes itself, and each lane then finds its tile's bit.
__device__ __forceinline__ bool tile_starts(const uint32_t *un, uint32_t nu, uint32_t n, uint32_t *start, int lane) {
    uint32_t seen = 0;
    __syncwarp();   // the last chunk's starts have been read
    for (uint32_t i0 = 0; i0 < nu; i0 += 128) {
        uint32_t p[4];
#pragma unroll
        for (int u = 0; u < 4; u++) {
            const uint32_t i = i0 + 32u * u + lane;
            p[u] = i < nu ? __popc(__ldg(un + i)) : 0u;
        }
#pragma unroll
        for (int h = 0; h < 2; h++) {
            uint32_t both = p[2 * h] | p[2 * h + 1] << 16;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, both, o);
                if (lane >= o) both += v;
            }
            const uint32_t all = __shfl_sync(0xffffffffu, both, 31);
            const uint32_t b0 = seen + (both & 0xFFFFu) - p[2 * h];
            const uint32_t b1 = seen + (all & 0xFFFFu) + (both >> 16) - p[2 * h + 1];
            const uint32_t i = i0 + 64u * h + lane;
            // word i holds terminators b .. b + p - 1; number 128 t - 1 ends tile t - 1
            if ((b0 >> 7) != ((b0 + p[2 * h]) >> 7) && b0 < 128u * n) start[(b0 >> 7) + 1u] = i * 32u + (127u - (b0 & 127u));
            if ((b1 >> 7) != ((b1 + p[2 * h + 1]) >> 7) && b1 < 128u * n)
                start[(b1 >> 7) + 1u] = (i + 32u) * 32u + (127u - (b1 & 127u));
            seen += (all & 0xFFFFu) + (all >> 16);
        }
    }
    __syncwarp();
    if (seen != 128u * n) return false;
    uint32_t v = 0;
    if ((uint32_t)lane < n) {
        v = start[lane + 1];
        v = (v & ~31u) + select_bit(__ldg(un + (v >> 5)), v & 31u) + 1u;
    }
    __syncwarp();
    if ((uint32_t)lane < n) start[lane + 1] = v;
    if (lane == 0) start[0] = 0;
    __syncwarp();
    return true;
}

__global__ void __launch_bounds__(kRepackWarps * 32, 12) repack_measure(const __grid_constant__ RepackArgs a) {
    __shared__ uint32_t starts[kRepackWarps][36];
    __shared__ TopRow top[kTop];
    __shared__ uint32_t size_of[kRepackWarps];
    cudaTriggerProgrammaticLaunchCompletion();   // the second launch may come up; it waits for this grid's end
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Table<kTop> tab(a.src_table, a.src_appends, a.heads, top);
    tab.load(top);
    __syncthreads();
    if (blockIdx.x == 0) {
        if (threadIdx.x < (unsigned)a.n_ranges) {
            const RepackRange r = a.range[threadIdx.x];
            hq_kv_append_row row = a.src_table[tab.append_of_token(r.begin)];
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
    uint32_t size = 0;
    if (c < a.n_chunks) {
        const NewChunk g = new_chunk(a, c);
        const bool mine = (uint32_t)lane < g.n;
        // the lane's token in the source; its scale has to be that of the range's first token
        const int64_t t = g.t0 + (mine ? lane : (int)g.n - 1);
        const uint64_t at = tab.append_of_token(t), at0 = tab.append_of_token(a.range[g.r].begin);
        const hq_kv_append_row row = a.src_table[at], ref = a.src_table[at0];
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
        uint32_t ustart = 0, len = 0;
        const uint32_t *un = a.src_words + w0 + head_words;
        // every tile of one source chunk: the new chunk is that chunk
        const uint64_t c0 = __shfl_sync(0xffffffffu, (unsigned long long)chunk, 0);
        bool whole = __all_sync(0xffffffffu, ok && chunk == c0 && n == g.n && (!mine || ti == (uint32_t)lane));
        if (whole) {
            uint32_t ones = 0;
            for (uint32_t i0 = 0; i0 < nu; i0 += 256) {
                uint32_t w[8];
#pragma unroll
                for (int u = 0; u < 8; u++) w[u] = i0 + 32u * u + lane < nu ? __ldg(un + i0 + 32u * u + lane) : 0u;
#pragma unroll
                for (int u = 0; u < 8; u++) ones += __popc(w[u]);
            }
            ones = __reduce_add_sync(0xffffffffu, ones);
            const uint32_t last = nu ? __ldg(un + nu - 1) : 0u;
            whole = ones == 128u * n && last != 0u;   // else found out tile by tile
            if (whole && lane == 0) len = nu * 32u - (uint32_t)__clz((int)last);   // lane 0's run is the chunk's
        }
        if (!whole) {
            // a tile in a chunk of its own
            const bool alone = ok && n == 1u && nu <= 256u;
            if (alone) {
                uint32_t ones = 0, last = 0;
                for (uint32_t i0 = 0; i0 < nu; i0 += 8) {
                    uint32_t w[8];
#pragma unroll
                    for (int u = 0; u < 8; u++) w[u] = i0 + u < nu ? __ldg(un + i0 + u) : 0u;
#pragma unroll
                    for (int u = 0; u < 8; u++) {
                        ones += __popc(w[u]);
                        if (w[u]) last = (i0 + u) * 32u + 32u - (uint32_t)__clz((int)w[u]);
                    }
                }
                ok = ones == 128u;
                len = last;
            }
            // larger ones: the warp reads each distinct chunk once
            unsigned todo = __ballot_sync(0xffffffffu, ok && !alone);
            while (todo) {
                const int lead = __ffs((int)todo) - 1;
                const uint64_t lc = __shfl_sync(0xffffffffu, (unsigned long long)chunk, lead);
                const uint64_t lw = __shfl_sync(0xffffffffu, (unsigned long long)(w0 + head_words), lead);
                const uint32_t ln = __shfl_sync(0xffffffffu, n, lead), lu = __shfl_sync(0xffffffffu, nu, lead);
                const bool good = tile_starts(a.src_words + lw, lu, ln, starts[warp], lane);
                const bool here = ok && !alone && chunk == lc;
                if (here) {
                    if (good) {
                        ustart = starts[warp][ti];
                        len = starts[warp][ti + 1] - ustart;
                    } else {
                        ok = false;
                    }
                }
                todo &= ~__ballot_sync(0xffffffffu, here);
            }
            // a tile that is not there, or not sound, becomes one of zero symbols (128 terminators)
            if (!ok) {
                ustart = 0;
                len = 128u;
            }
        }
        unsigned long long bits = mine ? len : 0u;
#pragma unroll
        for (int o = 16; o; o >>= 1) bits += __shfl_xor_sync(0xffffffffu, bits, o);
        if (bits >= kMaxUnaryBits) {   // tiles of enormous symbols that together exceed what a chunk may hold
            ok = false;
            ustart = 0;
            len = 128u;
            bits = 128ull * g.n;
        }
        const uint64_t tag = ok ? w0 | (uint64_t)ti << 48 | (uint64_t)n << 56 : 0ull;
        if (mine) a.tiles[c * 32 + lane] = make_uint4((uint32_t)tag, (uint32_t)(tag >> 32), ustart, len);
        size = coset_words(a, g.n) + rem_words(a, g.n) + (uint32_t)((bits + 31) >> 5);
        if (lane == 0) a.sizes[c] = size;
    }
    if (lane == 0) size_of[warp] = size;
    __syncthreads();
    if (threadIdx.x == 0) {
        uint64_t sum = 0;
        for (int i = 0; i < kRepackWarps; i++) sum += size_of[i];
        a.sums[blockIdx.x] = sum;
    }
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

// One plane of a new chunk: `words` words at dst (of which those below `room` exist), of runs whose first bits
// are at[r] (at[runs] the end) and come from absolute source bit from[r] on (kNoSource: `fill` instead).
constexpr unsigned long long kNoSource = ~0ull;
__device__ __forceinline__ uint32_t run_bits(const RepackArgs &a, unsigned long long from, uint32_t skip, uint32_t need,
                                             uint32_t fill) {
    return from == kNoSource ? fill : stream_bits(a.src_words, from + skip, need);
}
// Word i, from the run that holds its first bit and the one after it.
__device__ __forceinline__ uint32_t plane_word(const RepackArgs &a, uint32_t i, const unsigned long long *from,
                                               const uint32_t *at, int runs, uint32_t fill) {
    const uint32_t b = 32u * i;
    int r = 0;
    if (runs > 1) {
#pragma unroll
        for (int o = 16; o; o >>= 1)
            if (r + o < runs && at[r + o] <= b) r += o;
    }
    const uint32_t left = at[r + 1] - b, have = min(32u, left);
    uint32_t v = run_bits(a, from[r], b - at[r], have, fill);
    if (have < 32u) {
        v &= (1u << have) - 1u;
        if (r + 1 < runs) {
            // the next run's first bits (its end may lie in this word too: bits behind it are the plane's
            // padding, or of a third run, which no plane has)
            const uint32_t more = min(32u - have, at[r + 2] - at[r + 1]);
            uint32_t x = run_bits(a, from[r + 1], 0u, more, fill);
            if (more < 32u) x &= (1u << more) - 1u;
            v |= x << have;
        }
    }
    return v;
}
// Words [i0, i1) of a plane, 32 bits of the source from bit b on each: a word to a lane, eight in flight.
__device__ __forceinline__ void copy_run(const uint32_t *words, uint32_t *dst, uint32_t i0, uint32_t i1,
                                         unsigned long long b, int lane) {
    const uint32_t *p = words + (b >> 5);
    const uint32_t sh = (uint32_t)b & 31u, n = i1 - i0;
    dst += i0;
    for (uint32_t k0 = lane; k0 < n; k0 += 256) {
        uint32_t lo[8], hi[8];
#pragma unroll
        for (int u = 0; u < 8; u++) {
            const uint32_t k = k0 + 32u * u;
            lo[u] = k < n ? __ldg(p + k) : 0u;
            hi[u] = sh && k < n ? __ldg(p + k + 1) : 0u;
        }
#pragma unroll
        for (int u = 0; u < 8; u++)
            if (k0 + 32u * u < n) dst[k0 + 32u * u] = __funnelshift_r(lo[u], hi[u], sh);
    }
}
constexpr int kFewRuns = 8;   // up to which a plane's whole words are copied run by run
__device__ __forceinline__ void copy_plane(const RepackArgs &a, uint32_t *dst, uint64_t room, uint32_t words,
                                           const unsigned long long *from, const uint32_t *at, int runs, uint32_t fill,
                                           int lane) {
    if (words == 0) return;
    if (runs > kFewRuns || room < words) {
#pragma unroll 4
        for (uint32_t i = lane; i < words; i += 32) {
            const uint32_t v = plane_word(a, i, from, at, runs, fill);
            if (i < room) dst[i] = v;
        }
        return;
    }
    for (int r = 0; r < runs; r++) {
        const uint32_t i0 = (at[r] + 31u) >> 5, i1 = at[r + 1] >> 5;   // the words that lie in the run alone
        if (i0 >= i1) continue;
        if (from[r] == kNoSource) {
            for (uint32_t i = i0 + lane; i < i1; i += 32) dst[i] = fill;
        } else {
            copy_run(a.src_words, dst, i0, i1, from[r] + (32u * i0 - at[r]), lane);
        }
    }
    // the words that runs end in
    if (lane < runs && (at[lane + 1] & 31u)) {
        const uint32_t i = at[lane + 1] >> 5;
        dst[i] = plane_word(a, i, from, at, runs, fill);
    }
}

__global__ void __launch_bounds__(kRepackWarps * 32, 12) repack_copy(const __grid_constant__ RepackArgs a) {
    __shared__ unsigned long long tmp[kRepackWarps];
    __shared__ unsigned long long from[kRepackWarps][3][32];   // first source bit of each run, by plane
    __shared__ uint32_t at[kRepackWarps][3][34];               // and its first bit in the new plane
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // whole blocks of the first launch
    const uint64_t blocks = (a.n_chunks + kRepackWarps - 1) / kRepackWarps;
    const uint64_t b0 = blocks * blockIdx.x / gridDim.x, b1 = blocks * (blockIdx.x + 1) / gridDim.x;
    const uint64_t c0 = b0 * kRepackWarps, c1 = min(a.n_chunks, b1 * kRepackWarps);
    cudaGridDependencySynchronize();
    if (c0 >= c1) return;
    unsigned long long before = 0;
    for (uint64_t i = threadIdx.x; i < b0; i += blockDim.x) before += a.sums[i];
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
        uint32_t incl = d.w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        const uint32_t nbits = __shfl_sync(0xffffffffu, incl, 31);
        // runs: a tile that does not follow the one before it in one source chunk starts one
        const uint32_t px = __shfl_up_sync(0xffffffffu, d.x, 1), py = __shfl_up_sync(0xffffffffu, d.y, 1);
        const uint32_t n = d.y >> 24, ti = (d.y >> 16) & 0xFFu;
        const bool first = mine && (lane == 0 || n == 0u || px != d.x || d.y != py + 0x10000u);
        const unsigned heads = __ballot_sync(0xffffffffu, first);
        const int runs = __popc(heads);
        const uint32_t nc = coset_words(a, g.n), nr = rem_words(a, g.n), nu = (nbits + 31u) >> 5;
        if (first) {
            const int r = __popc(heads & ((1u << lane) - 1u));
            const unsigned long long src = (unsigned long long)(d.y & 0xFFFFu) << 32 | d.x;
            const uint32_t snc = coset_words(a, n), snr = rem_words(a, n);
            from[warp][0][r] = n ? src * 32 + 16u * ti : kNoSource;
            from[warp][1][r] = n ? (src + snc) * 32 + (unsigned long long)ti * a.rem_bits : kNoSource;
            from[warp][2][r] = n ? (src + snc + snr) * 32 + d.z : kNoSource;
            at[warp][0][r] = 16u * lane;
            at[warp][1][r] = a.rem_bits * lane;
            at[warp][2][r] = incl - d.w;
        }
        if (lane == 0) {
            at[warp][0][runs] = 16u * g.n;
            at[warp][1][runs] = a.rem_bits * g.n;
            at[warp][2][runs] = nbits;
            a.offsets[c] = w0;
            payload += (unsigned long long)nbits + g.n * (a.rem_bits + (a.e8 ? 16u : 0u));
        }
        __syncwarp();
        if (mine && n == 0u) status |= HQ_ST_CORRUPT;
        const uint32_t total = nc + nr + nu;
        // words of this chunk that the buffer has room for
        const uint64_t room = w0 < a.cap ? a.cap - w0 : 0ull;
        uint32_t *const dst = a.words + w0;
        // all tiles of a source chunk: its words as they are
        const bool whole = runs == 1 && __shfl_sync(0xffffffffu, n == g.n && ti == 0u, 0);
        if (whole && room >= total) {
            copy_run(a.src_words, dst, 0u, total, ((unsigned long long)(__shfl_sync(0xffffffffu, d.y, 0) & 0xFFFFu) << 32 |
                                                   __shfl_sync(0xffffffffu, d.x, 0)) * 32ull, lane);
        } else {
            copy_plane(a, dst, room, nc, from[warp][0], at[warp][0], runs, 0u, lane);
            copy_plane(a, dst + nc, room > nc ? room - nc : 0ull, nr, from[warp][1], at[warp][1], runs, 0u, lane);
            copy_plane(a, dst + nc + nr, room > nc + nr ? room - nc - nr : 0ull, nu, from[warp][2], at[warp][2], runs, ~0u,
                       lane);
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
    // tiles, sums by CTA, sizes
    *bytes = ((size_t)c * (32 * sizeof(uint4) + sizeof(uint32_t)) + ((size_t)c / kRepackWarps + 1) * sizeof(uint64_t) + 255) &
             ~(size_t)255;
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
    a.sums = (uint64_t *)((char *)workspace + (size_t)chunks * 32 * sizeof(uint4));
    a.sizes = (uint32_t *)(a.sums + chunks / kRepackWarps + 1);
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
    // all resident at once (12 CTAs per SM): each sums the sizes before its own chunks
    const uint64_t most = 148 * 12;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(ctas < most ? ctas : most));
    cfg.blockDim = dim3(kRepackWarps * 32);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, repack_copy, a) != cudaSuccess) return HQ_ECUDA;
    dst->tokens = h_ranges[2 * n_ranges - 1];
    dst->chunks = (uint64_t)chunks;
    dst->appends = (uint64_t)n_ranges;
    return HQ_OK;
}
