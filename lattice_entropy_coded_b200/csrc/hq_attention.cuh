// hq_attention.cuh -- attention of a few query tokens over compressed K and V caches
// (hq_kv_attention, hq_kv_tree_attention), without writing K or V to memory.
//
// Mathematics.  A cached vector is x = M z e with z = lattice point - dither, e the append's
// scale and M the inverse rotation (D H_128, or Q^T for a dense rotation), the same for every
// token.  So q . x = (M^T q) . z e, and sum_t p_t x_t = M (sum_t p_t e_t z_t): the queries are
// rotated once, the output once, and no token's tile is transformed.  The softmax runs over
// the tokens as they come, with the running maximum and sum of each row.
//
// Two launches: attention_kernel, a grid of (splits of the tokens) x (KV heads) x (blocks of
// query rows), leaves a partial (maximum, sum, 128 sums of values) per row and split, in the
// rotated domain; attention_combine joins the splits, turns the result back, adds the drafted
// tokens of a tree (whose K and V are plain bf16) and writes the output.
//
// The products run on the tensor cores in fp16 with fp32 sums (mma.sync m16n8k16):
//  * z / 64 in fp16: exact for codes up to 2048 without dither, else rounded by at most 2^-11
//    of its value, and finite over the codec's whole range (|z| < 2^21 + 2 < 64 * 65504);
//  * the rotated queries as the sum of two fp16 (scaled by a power of two per row): 2^-22;
//  * the weights p in [0, 1] in fp16: 2^-11 of their value (2^-25 below 2^-14).
// A lane of the Rice decoder holds 32 consecutive coordinates of one token; a step of 16
// contracted coordinates takes 4 from each of the 4 lanes of a token, and the queries are laid
// out in the same order, so K goes from the decoder's registers into the product as it is.
//
// Bound: the decoder's integer work (see hq_decode.cuh), not bytes nor products.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "hq_decode.cuh"

namespace hq {

constexpr int kAttnMaxQueries = 64;   // query tokens of a call (a draft's mask is one word)
constexpr int kAttnMaxGroup = 64;
constexpr int kAttnWarps = 8;
constexpr int kAttnTokens = 16 * kAttnWarps;   // tokens of one step of a CTA: two decoder rounds per warp
constexpr int kAttnStage = 704;                // staged words of a chunk (5.5 bits per scalar)
constexpr int kAttnCtas = 2 * 148;             // resident CTAs the splits aim at

struct AttnArgs {
    const uint32_t *words[2];       // K, V
    uint64_t cap[2];
    const uint64_t *offsets[2];
    const hq_kv_append_row *table[2];
    hq_stats *stats[2];
    uint64_t seed[2];
    const float *rot[2];
    int k[2], k_last[2];
    uint64_t n_chunks, n_appends;
    int64_t len, window, sinks;
    int heads, group, n_q, rows;    // rows = n_q * group query rows per KV head
    int splits, row_pad;            // row_pad: rows rounded up to whole blocks
    float scale_log2;               // scale * log2(e)
    const uint16_t *q;
    int64_t q_ld_tok, q_ld_head;
    const unsigned long long *mask; // tree: visible drafts of each query, or null
    const uint16_t *kd, *vd;
    int64_t d_ld_tok, d_ld_head;
    float *part;                    // [split][head][row_pad][128]
    float2 *ml;                     // [split][head][row_pad]: maximum (of log2 weights), sum
    void *out;
    int out_fp32;
    int64_t out_ld_tok, out_ld_head;
    float *lse;
    float scale;
};

cudaError_t launch_attention(int lattice, int dither, const AttnArgs &a, cudaStream_t s);
cudaError_t launch_attention_z(int dither, const AttnArgs &a, cudaStream_t s);
cudaError_t launch_attention_a2(int dither, const AttnArgs &a, cudaStream_t s);
cudaError_t launch_attention_d4(int dither, const AttnArgs &a, cudaStream_t s);
cudaError_t launch_attention_e8(int dither, const AttnArgs &a, cudaStream_t s);

// Query rows of one CTA for a call of `rows` rows: blocks of 16 up to 16 rows, of 32 beyond.
inline int attn_row_block(int rows) { return rows <= 16 ? 16 : 32; }
// Splits of the tokens: the CTAs of all heads and row blocks together fill the GPU once.
inline int attn_splits(int heads, int rows, uint64_t chunks_per_head) {
    const int rb = attn_row_block(rows);
    const int64_t base = (int64_t)heads * ((rows + rb - 1) / rb);
    int64_t s = kAttnCtas / base;
    const int64_t steps = (int64_t)((2 * chunks_per_head + kAttnWarps - 1) / kAttnWarps);
    if (s > steps) s = steps;
    return (int)(s < 1 ? 1 : s);
}

namespace {

constexpr float kNegInf = -INFINITY;

__device__ __forceinline__ uint32_t h2_pack(float a, float b) {
    __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&h);
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], const void *p) {
    const unsigned sa = (unsigned)__cvta_generic_to_shared(p);
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(sa) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], const void *p) {
    const unsigned sa = (unsigned)__cvta_generic_to_shared(p);
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(sa) : "memory");
}

// ------------------------------------------------------------------ where tokens are
// The append that holds per-head chunk i (chunks of an append lie head-major, so its first chunk is
// heads times the per-head chunks before it).
struct AttnRow {
    uint64_t append;
    hq_kv_append_row row;
    uint64_t base, count;   // per-head chunks before the append, and in it
};
__device__ __forceinline__ void load_row(const AttnArgs &a, uint64_t append, AttnRow &r) {
    r.append = append;
    r.row = a.table[0][append];
    unsigned long long rem, base;
    divmod_u64(r.row.first_chunk, (unsigned long long)a.heads, base, rem);
    r.base = base;
    r.count = (uint64_t)(((int64_t)r.row.tokens + 31) / 32);
}
__device__ __forceinline__ void find_row(const AttnArgs &a, uint64_t i, AttnRow &r) {
    if (i >= r.base && i < r.base + r.count) return;
    if (i >= r.base + r.count && r.append + 1 < a.n_appends) {
        load_row(a, r.append + 1, r);
        if (i >= r.base && i < r.base + r.count) return;
    }
    const uint64_t first = i * (uint64_t)a.heads;
    uint64_t lo = 0, hi = a.n_appends - 1;
    while (lo < hi) {
        const uint64_t mid = (lo + hi + 1) >> 1;
        if (a.table[0][mid].first_chunk <= first) lo = mid; else hi = mid - 1;
    }
    load_row(a, lo, r);
}
// Per-head chunks that lie wholly before token t (round_up: that hold any token before t).
__device__ __forceinline__ uint64_t chunks_before(const AttnArgs &a, int64_t t, bool round_up) {
    uint64_t lo = 0, hi = a.n_appends - 1;
    while (lo < hi) {
        const uint64_t mid = (lo + hi + 1) >> 1;
        if (a.table[0][mid].token0 <= t) lo = mid; else hi = mid - 1;
    }
    AttnRow r;
    load_row(a, lo, r);
    const int64_t in = t - r.row.token0;
    if (in <= 0) return r.base;
    const uint64_t n = (uint64_t)(round_up ? (in + 31) / 32 : in / 32);
    return r.base + (in >= r.row.tokens ? r.count : n < r.count ? n : r.count);
}

// One warp's part of a step: two decoder rounds (16 tokens) of one chunk.
struct Piece {
    bool on;              // there is one
    int r0;               // its first round
    int n;                // tokens of the chunk
    int64_t t0;           // position of the chunk's first token
    float e[2];           // K's and V's scale
    bool same;            // V's append is K's
    uint64_t chunk;       // chunk index (K's and V's)
};

// ------------------------------------------------------------------ E8 dither
// d = w - Q(w) of dither_block<HQ_E8>, bit for bit, for an eighth of its work.  With w uniform on
// [0, 4)^8, let c_i = (w_i mod 2) - 1 and b_i = |c_i|: c_i is w_i's residual to the nearest odd
// integer (candidate B), and c_i - sign(c_i), of size 1 - b_i, the one to the nearest even integer
// (candidate A).  The squared distances' difference is then linear in the b_i:
//   (|w - A|^2 - |w - B|^2) / 2 = 4 - sum b + 2 p_A min b - 2 p_B (1 - max b),
// the last terms being the parity fixes (the largest residual r becomes 2 - r), with the parities
// of the rounded halves from the two top bits of each w: p_B the XOR of the "w >= 2", p_A of the
// "1 <= w < 3".  So one pass over c serves both candidates.  Everything is exact in units of 2^-22
// but the sum (within 16 units).  The reading compares fp32 distances, which are off by less than
// 2^-16 here (the bound at Lattice<HQ_E8>): a difference within 2^-12, a coordinate on a rounding
// border (b = 0 or 1) or two equal largest residuals under a fix goes to the reading's own code
// instead, about one block in 4000.
constexpr float kDitherUnit = 4194304.0f;       // 2^22: d is returned in units of 2^-22
constexpr uint64_t kSplitGolden = 0x9E3779B97F4A7C15ull;

// Two hashes' worth of a pair: generator state z (s + (i + 1) golden) -> w of the even and the odd
// coordinate as 32-bit fixed point (bits 8..31 of each count).
__device__ __forceinline__ void dither_pair(uint64_t z, uint32_t &even, uint32_t &odd) {
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    // h = z ^ (z >> 31): bits 40..63 are z's own, bits 8..31 take z's bits 39..62
    even = (uint32_t)(z >> 32);
    odd = (uint32_t)z ^ (even << 1);
}

__device__ __noinline__ void e8_dither_reading(const uint32_t *x, float *d) {
    float w[8], p[8];
    int32_t q[8];
    for (int i = 0; i < 8; i++) w[i] = __fmul_rn((float)(x[i] >> 8), 0x1p-22f);
    Lattice<HQ_E8>::nearest(w, q);
    Lattice<HQ_E8>::point(q, p);
    for (int i = 0; i < 8; i++) d[i] = __fmul_rn(__fsub_rn(w[i], p[i]), kDitherUnit);
}

// The block whose first pair has generator state z0; d in units of 2^-22.
__device__ __forceinline__ void e8_dither(uint64_t z0, float (&d)[8]) {
    uint32_t x[8];
    float c[8];
#pragma unroll
    for (int i = 0; i < 4; i++) dither_pair(z0 + (uint64_t)i * kSplitGolden, x[2 * i], x[2 * i + 1]);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        // 2^23 + (w mod 2), less 2^23 + 1 (units of 2^-22): exact
        const float2 f = make_float2(__uint_as_float(((x[2 * i] >> 8) & 0x7FFFFFu) | 0x4B000000u),
                                     __uint_as_float(((x[2 * i + 1] >> 8) & 0x7FFFFFu) | 0x4B000000u));
        const float2 r = f2_sub(f, make_float2(8388608.0f + kDitherUnit, 8388608.0f + kDitherUnit));
        c[2 * i] = r.x;
        c[2 * i + 1] = r.y;
    }
    const uint32_t par = (x[0] ^ x[1] ^ x[2]) ^ (x[3] ^ x[4] ^ x[5]) ^ (x[6] ^ x[7]);
    const bool pb = (int32_t)par < 0, pa = (int32_t)(par ^ (par << 1)) < 0;
    float lo = fabsf(c[0]), hi = lo;
#pragma unroll
    for (int i = 1; i < 8; i++) {
        lo = fminf(lo, fabsf(c[i]));
        hi = fmaxf(hi, fabsf(c[i]));
    }
    const float s0 = __fadd_rn(__fadd_rn(fabsf(c[0]), fabsf(c[1])), __fadd_rn(fabsf(c[2]), fabsf(c[3])));
    const float s1 = __fadd_rn(__fadd_rn(fabsf(c[4]), fabsf(c[5])), __fadd_rn(fabsf(c[6]), fabsf(c[7])));
    const float half = __fsub_rn(__fsub_rn(4.0f * kDitherUnit, s0), s1);
    const float diff = __fadd_rn(half, __fsub_rn(pa ? __fadd_rn(lo, lo) : 0.0f,
                                                 pb ? __fmul_rn(2.0f, __fsub_rn(kDitherUnit, hi)) : 0.0f));
    const bool odd = diff > 0.0f, fix = odd ? pb : pa;
    // d = c - sign(c) m: m = 0 (B) or 1 (A), and for the coordinate of the fix 2 (B) or -1 (A)
    const float m0 = odd ? 0.0f : kDitherUnit, m1 = odd ? 2.0f * kDitherUnit : -kDitherUnit;
    const float at = fix ? (odd ? hi : lo) : -1.0f;
    float m[8];
    float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < 8; i++) m[i] = fabsf(c[i]) == at ? m1 : m0;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        sum = f2_add(sum, make_float2(m[2 * i], m[2 * i + 1]));
        const float2 r = f2_sub(make_float2(c[2 * i], c[2 * i + 1]),
                                make_float2(__uint_as_float(__float_as_uint(m[2 * i]) ^ (__float_as_uint(c[2 * i]) & 0x80000000u)),
                                            __uint_as_float(__float_as_uint(m[2 * i + 1]) ^
                                                            (__float_as_uint(c[2 * i + 1]) & 0x80000000u))));
        d[2 * i] = r.x;
        d[2 * i + 1] = r.y;
    }
    const float want = fix ? __fadd_rn(__fmul_rn(7.0f, m0), m1) : __fmul_rn(8.0f, m0);
    if (fabsf(diff) <= 1024.0f || lo == 0.0f || hi == kDitherUnit || __fadd_rn(sum.x, sum.y) != want) {
        float t[8];
        e8_dither_reading(x, t);
#pragma unroll
        for (int i = 0; i < 8; i++) d[i] = t[i];
    }
}

// ------------------------------------------------------------------ decode
// Forms of the Rice code: no remainders at all (k = 0: the 2-bit caches), remainders read four
// windows at a time (k <= 4, one parameter), or bit by bit.
enum AttnForm { kFormUnary = 0, kFormWindows = 1, kFormGeneral = 2 };

// Unary pairs of E8 at k = 0: the next 10 stream bits -> both codewords.  Bits 0..4 their length,
// byte 1 and byte 2 the two codes 2 m + 128 (2 m the zigzag inverse doubled), bit 24 the parity of
// m of both, bit 25 of the first, bit 31 set if both codewords end inside the 10 bits (one pair in
// 2000 does not at 2 bits per scalar).
constexpr int kPairBits = 10;
__device__ __forceinline__ uint32_t pair_entry(uint32_t w) {
    const uint32_t t0 = (uint32_t)__ffs((int)(w | 0x80000000u)) - 1u;
    const uint32_t t1 = t0 < 31u ? (uint32_t)__ffs((int)((w >> (t0 + 1u)) | 0x80000000u)) - 1u : 31u;
    if (t0 + t1 + 2u > (uint32_t)kPairBits) return 0u;
    const uint32_t a = t0 ^ (0u - (t0 & 1u)), b = t1 ^ (0u - (t1 & 1u));   // 2 m
    return 0x80000000u | (t0 + t1 + 2u) | ((a + 128u) & 0xFFu) << 8 | ((b + 128u) & 0xFFu) << 16 |
           (((a ^ b) >> 1) & 1u) << 24 | ((a >> 1) & 1u) << 25;
}

// The 32 codes (minus dither) of a lane's quarter of a tile, times `scale`, as 16 fp16 pairs.
template <int LAT, bool DITHER, int FORM, bool STAGED>
__device__ __forceinline__ bool decode_quarter(const uint32_t *src, uint32_t nc, uint32_t nr, uint32_t nu, int k, int kl,
                                               uint32_t bp, uint32_t segi, int q, unsigned long long e0, uint64_t seed,
                                               float scale, const uint32_t *pairs, uint32_t (&w)[16]) {
    using L = Lattice<LAT>;
    constexpr int N = L::N;
    const uint32_t *un = src + nc + nr;
    const uint32_t pk = 1u << k, pkl = 1u << kl;
    const uint32_t gbits = group_rem_bits<N>(k, kl), lane_bits = 4u * gbits;
    bool ok = true;
    uint32_t rx[4] = {0u, 0u, 0u, 0u};
    if (FORM == kFormWindows && k > 0) rem_windows(src + nc + segi * (uint32_t)k, k, rx);
    const uint32_t cw = (LAT == HQ_E8) ? src[segi >> 3] : 0u;
    const uint32_t coset = (cw >> (4 * (segi & 7u))) & 0xFu;
    const float2 s2 = make_float2(scale, scale);
    // E8 with dither: d comes in units of 2^-22
    const float2 sd2 = make_float2(__fmul_rn(scale, -0x1p-22f), __fmul_rn(scale, -0x1p-22f));
    const uint64_t z0 = (seed ^ kDitherSalt) + ((e0 >> 1) + (uint64_t)(16 * q) + 1ull) * kSplitGolden;
#pragma unroll
    for (int g = 0; g < 4; g++) {
        float u[8];
        if constexpr (LAT == HQ_E8 && FORM == kFormUnary && STAGED) {
            // The plane's terminators were counted, so a lane's 32 codewords end inside it (or in the pad
            // behind its last word, which the second word of a window may reach).
            const uint32_t c = (coset >> g) & 1u;
            uint32_t e[4], used = 0;
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const uint32_t *p = un + ((bp + used) >> 5);
                uint32_t x = __funnelshift_r(p[0], p[1], bp + used);
                e[2 * h] = pairs[x & ((1u << kPairBits) - 1u)];
                x = __funnelshift_r(x, 0u, e[2 * h]);
                e[2 * h + 1] = pairs[x & ((1u << kPairBits) - 1u)];
                used += (e[2 * h] + e[2 * h + 1]) & 0x1Fu;
            }
            if ((int32_t)(e[0] & e[1] & e[2] & e[3]) < 0) {
                bp += used;
                // the stripped parity of m_7: that of m_0 .. m_6
                const uint32_t p7 = ((e[0] ^ e[1] ^ e[2]) >> 24 ^ e[3] >> 25) & 1u;
                const float off = __fsub_rn((float)(int)c, 8388608.0f + 128.0f);
                const float2 o2 = make_float2(off, off);
#pragma unroll
                for (int h = 0; h < 4; h++) {
                    const float2 f = make_float2(__uint_as_float(__byte_perm(e[h], 0x4B000000u, 0x7441)),
                                                 __uint_as_float(__byte_perm(e[h], 0x4B000000u, 0x7442)));
                    const float2 r = f2_add(f, o2);
                    u[2 * h] = r.x;
                    u[2 * h + 1] = r.y;
                }
                // 2 (2 m_7 + p) + c from 2 m_7 + c
                u[7] = __fadd_rn(__fadd_rn(u[7], u[7]), (float)((int)(2u * p7) - (int)c));
            } else {
                uint32_t zq[8];
                unary4<STAGED>(un, nu, bp, ok, zq);
                unary4<STAGED>(un, nu, bp, ok, zq + 4);
                int32_t qq[8];
                e8_codes_from_symbols(zq, c, qq);
                decoded_point<HQ_E8>(qq, u);
            }
        } else {
            uint32_t qv[8], rv[8];
            unary4<STAGED>(un, nu, bp, ok, qv);
            unary4<STAGED>(un, nu, bp, ok, qv + 4);
            if (FORM == kFormGeneral) {
                rem_group_mixed<N, STAGED>(src + nc, nr, segi * lane_bits, g, k, kl, gbits, rv);
            } else if (FORM == kFormWindows) {
                const uint32_t mask = (1u << k) - 1u;
                uint32_t xw = rx[g];
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    rv[i] = xw & mask;
                    xw >>= k;
                }
            }
#pragma unroll
            for (int bb = 0; bb < 8 / N; bb++) {
                int32_t qq[N];
                float p[N];
                uint32_t zb[N];
#pragma unroll
                for (int i = 0; i < N; i++)
                    zb[i] = FORM == kFormUnary ? qv[bb * N + i]
                                               : imad(qv[bb * N + i], (N > 1 && i == N - 1) ? pkl : pk, rv[bb * N + i]);
                if constexpr (LAT == HQ_E8) {
                    e8_codes_from_symbols(zb, (coset >> g) & 1u, qq);
                } else {
                    int32_t m[N];
#pragma unroll
                    for (int i = 0; i < N; i++) m[i] = unzigzag(zb[i]);
                    L::reinsert(m, 0u, qq);
                }
                decoded_point<LAT>(qq, p);
                if (DITHER && LAT != HQ_E8) {
                    float d[N];
                    dither_block<LAT>(seed, e0 + (unsigned long long)(32 * q + 8 * g + bb * N), d);
#pragma unroll
                    for (int i = 0; i < N; i++) p[i] = __fsub_rn(p[i], d[i]);
                }
#pragma unroll
                for (int i = 0; i < N; i++) u[bb * N + i] = p[i];
            }
        }
        if constexpr (DITHER && LAT == HQ_E8) {
            float d[8];
            e8_dither(z0 + (uint64_t)(4 * g) * kSplitGolden, d);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const float2 x = f2_fma(make_float2(d[2 * j], d[2 * j + 1]), sd2, f2_mul(make_float2(u[2 * j], u[2 * j + 1]), s2));
                w[4 * g + j] = h2_pack(x.x, x.y);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const float2 x = f2_mul(make_float2(u[2 * j], u[2 * j + 1]), s2);
                w[4 * g + j] = h2_pack(x.x, x.y);
            }
        }
    }
    return ok && bp <= nu * 32u;
}

// ------------------------------------------------------------------ shared memory
template <int MB>
struct AttnSmem {
    static constexpr int R = 16 * MB;
    uint4 qh[MB * 8 * 32], ql[MB * 8 * 32];     // query fragments (two fp16 parts)
    uint32_t v[kAttnTokens * 64];               // V: [token][128] fp16, 16-byte pieces swizzled by the token
    uint32_t p[R * (kAttnTokens / 2)];          // weights: [row][token] fp16, swizzled by the row
    uint32_t stage[kAttnWarps][2][kAttnStage + kStagePad];
    uint32_t start[kAttnWarps][128];
    uint32_t sign[4];
    uint32_t pairs[1 << kPairBits];             // E8 at k = 0 (pair_entry)
    float wmax[2][kAttnWarps][R];               // row maxima of each warp's tokens, by parity of the step
    float rescale[R];                           // of the sums, this step
    float qscale[R];                            // undoes a row's power-of-two scale, with the softmax scale
    int64_t qpos[R];
    float lsum[kAttnWarps][R];
    float xs[kAttnWarps][128];
    uint64_t range[3];
    float eref[kAttnWarps];
};

// Unnormalised H_128 of a row held 4 coordinates to a lane (4 lane ..), the whole warp.
__device__ __forceinline__ void fwht_row(float (&u)[4], int lane) {
    const float t0 = __fadd_rn(u[0], u[1]), t1 = __fsub_rn(u[0], u[1]), t2 = __fadd_rn(u[2], u[3]),
                t3 = __fsub_rn(u[2], u[3]);
    u[0] = __fadd_rn(t0, t2);
    u[1] = __fadd_rn(t1, t3);
    u[2] = __fsub_rn(t0, t2);
    u[3] = __fsub_rn(t1, t3);
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const float sg = (lane & m) ? -1.0f : 1.0f;
#pragma unroll
        for (int i = 0; i < 4; i++) u[i] = __fmaf_rn(sg, u[i], __shfl_xor_sync(0xffffffffu, u[i], m));
    }
}

// Rotated query row (u = M^T q, 4 values per lane: coordinates 4 lane ..), unnormalised for H_128.
__device__ __forceinline__ void rotate_query(const AttnArgs &a, float (&u)[4], const uint32_t *sign, float *xs, int lane) {
    if (a.rot[0]) {
        reinterpret_cast<float4 *>(xs)[lane] = make_float4(u[0], u[1], u[2], u[3]);
        __syncwarp();
        const float *Q = a.rot[0] + 4 * lane * 128;
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int j = 0; j < 32; j++) {
            const float4 x = reinterpret_cast<const float4 *>(xs)[j];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float4 m = __ldg(reinterpret_cast<const float4 *>(Q + i * 128) + j);
                acc[i] = __fmaf_rn(m.w, x.w, __fmaf_rn(m.z, x.z, __fmaf_rn(m.y, x.y, __fmaf_rn(m.x, x.x, acc[i]))));
            }
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; i++) u[i] = acc[i];
        return;
    }
    // signs: column c = 4 lane + i; word c / 32 holds even columns in bits 0.., odd in bits 16..
    const uint32_t e = sign[lane >> 3];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int c = (4 * lane + i) & 31;
        if ((e >> ((c >> 1) + 16 * (c & 1))) & 1u) u[i] = -u[i];
    }
    fwht_row(u, lane);
}

template <int LAT, bool DITHER, int FORM, int MB>
__global__ void __launch_bounds__(kAttnWarps * 32, 2) attention_kernel(const __grid_constant__ AttnArgs a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    AttnSmem<MB> &sm = *reinterpret_cast<AttnSmem<MB> *>(smem_raw);
    constexpr int R = 16 * MB;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g8 = lane >> 2, t4 = lane & 3;
    const int split = blockIdx.x, head = blockIdx.y, row0 = blockIdx.z * R;

    // ---- which chunks the queries can see, the queries themselves
    if (threadIdx.x == 0) {
        const int64_t pmin = a.mask ? a.len - 1 : a.len - a.n_q;   // of any query: a bound is enough here
        const uint64_t all = chunks_before(a, a.len, true);
        uint64_t ia = all, ib = all;
        if (a.window > 0) {
            ia = a.sinks > 0 ? chunks_before(a, a.sinks < a.len ? a.sinks : a.len, true) : 0;
            const int64_t lo = pmin - a.window + 1;
            ib = lo > 0 ? chunks_before(a, lo, false) : 0;
            if (ib < ia) ib = ia;
        }
        sm.range[0] = ia;
        sm.range[1] = ib;
        sm.range[2] = all;
    }
    build_sign_table(sm.sign, 1, a.seed[0]);
    if (LAT == HQ_E8 && FORM == kFormUnary)
        for (int i = threadIdx.x; i < (1 << kPairBits); i += blockDim.x) sm.pairs[i] = pair_entry((uint32_t)i);
    for (int r = threadIdx.x; r < R; r += blockDim.x) {
        int64_t pos = INT64_MIN / 2;      // a row past the last sees nothing
        if (row0 + r < a.rows) {
            const int i = (row0 + r) / a.group;
            pos = a.len - a.n_q + i;
            if (a.mask) {
                const unsigned long long all = a.n_q < 64 ? (1ull << a.n_q) - 1ull : ~0ull;
                pos = a.len - 1 + __popcll(a.mask[i] & all);
            }
        }
        sm.qpos[r] = pos;
    }
    __syncthreads();
    for (int r = warp; r < R; r += kAttnWarps) {
        float u[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (row0 + r < a.rows) {
            const int i = (row0 + r) / a.group, qh = head * a.group + (row0 + r) - i * a.group;
            const uint2 x = *reinterpret_cast<const uint2 *>(a.q + i * a.q_ld_tok + qh * a.q_ld_head + 4 * lane);
            u[0] = __uint_as_float(x.x << 16);
            u[1] = __uint_as_float(x.x & 0xFFFF0000u);
            u[2] = __uint_as_float(x.y << 16);
            u[3] = __uint_as_float(x.y & 0xFFFF0000u);
        }
        rotate_query(a, u, sm.sign, sm.xs[warp], lane);
        float top = fmaxf(fmaxf(fabsf(u[0]), fabsf(u[1])), fmaxf(fabsf(u[2]), fabsf(u[3])));
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
        // power of two that brings the row's largest value into [1, 2) (rows of zeros, infinities: 1)
        const int ex = (int)(__float_as_uint(top) >> 23) - 127;
        const float down = (ex >= -126 && ex <= 126) ? __uint_as_float((uint32_t)(127 - ex) << 23) : 1.0f;
        const float up = (ex >= -126 && ex <= 126) ? __uint_as_float((uint32_t)(127 + ex) << 23) : 1.0f;
        // fragment of coordinate c for row r: step s = (c mod 32) / 4 of lane quarter c / 32
#pragma unroll
        for (int pr = 0; pr < 2; pr++) {
            const float x0 = __fmul_rn(u[2 * pr], down), x1 = __fmul_rn(u[2 * pr + 1], down);
            const uint32_t hi = h2_pack(x0, x1);
            const __half2 hh = *reinterpret_cast<const __half2 *>(&hi);
            const uint32_t lo = h2_pack(__fsub_rn(x0, __low2float(hh)), __fsub_rn(x1, __high2float(hh)));
            // coordinates 4 lane + 2 pr: quarter lane / 8, step lane % 8, register pair pr
            const int slot = ((r >> 4) * 8 + (lane & 7)) * 32 + (r & 7) * 4 + (lane >> 3);
            const int reg = ((r >> 3) & 1) + 2 * pr;
            reinterpret_cast<uint32_t *>(sm.qh)[slot * 4 + reg] = hi;
            reinterpret_cast<uint32_t *>(sm.ql)[slot * 4 + reg] = lo;
        }
        if (lane == 0) sm.qscale[r] = __fmul_rn(up, a.scale_log2);
    }
    const uint64_t ia = sm.range[0], ib = sm.range[1], ie = sm.range[2];
    const uint64_t nvis = ia + (ie - ib);
    const uint64_t steps = (2 * nvis + kAttnWarps - 1) / kAttnWarps;
    // this CTA's steps: an even share
    const uint64_t st0 = steps * (uint64_t)split / (uint64_t)a.splits;
    const uint64_t st1 = steps * (uint64_t)(split + 1) / (uint64_t)a.splits;

    // ---- V is summed in units of the largest scale among this CTA's appends
    float eref = 0.0f;
    if (st0 < st1) {
        const uint64_t v0 = st0 * kAttnWarps / 2, v1 = min(nvis, (st1 * kAttnWarps + 1) / 2);
        AttnRow lo, hi;
        load_row(a, 0, lo);
        hi = lo;
        find_row(a, v0 < ia ? v0 : v0 - ia + ib, lo);
        find_row(a, v1 - 1 < ia ? v1 - 1 : v1 - 1 - ia + ib, hi);
        for (uint64_t i = lo.append + threadIdx.x; i <= hi.append; i += blockDim.x)
            eref = fmaxf(eref, a.table[1][i].scale_inv);
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) eref = fmaxf(eref, __shfl_xor_sync(0xffffffffu, eref, m));
    }
    if (lane == 0) sm.eref[warp] = eref;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kAttnWarps; i++) eref = fmaxf(eref, sm.eref[i]);

    float m_run[MB][2], l_run[MB][2], acc[2 * MB][4];
#pragma unroll
    for (int mb = 0; mb < MB; mb++) {
        m_run[mb][0] = m_run[mb][1] = kNegInf;
        l_run[mb][0] = l_run[mb][1] = 0.0f;
    }
#pragma unroll
    for (int n = 0; n < 2 * MB; n++) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;

    AttnRow row;
    load_row(a, 0, row);
    auto piece_of = [&](uint64_t step) {
        Piece p;
        const uint64_t pi = step * kAttnWarps + warp, v = pi >> 1;
        p.on = step < st1 && v < nvis;
        p.r0 = (int)(pi & 1) * 2;
        p.n = 0;
        p.same = true;
        if (p.on) {
            const uint64_t i = v < ia ? v : v - ia + ib;
            find_row(a, i, row);
            const uint64_t j = i - row.base;
            p.t0 = row.row.token0 + 32 * (int64_t)j;
            const int64_t left = (int64_t)row.row.tokens - 32 * (int64_t)j;
            p.n = (int)(left < 32 ? left : 32);
            p.on = p.n > 8 * p.r0;
            p.chunk = row.row.first_chunk + (uint64_t)head * row.count + j;
            const hq_kv_append_row vr = a.table[1][row.append];
            p.same = vr.first_chunk == row.row.first_chunk && vr.token0 == row.row.token0 && vr.tokens == row.row.tokens;
            p.e[0] = row.row.scale_inv;
            p.e[1] = vr.scale_inv;
        }
        return p;
    };
    // valid words of a piece's chunk in cache `which`, staged
    auto words_of = [&](const Piece &p, int which) {
        ChunkWords cw = {0, 0, false, nullptr, 0, 0};
        if (p.on && p.chunk < a.n_chunks) {
            cw.w0 = a.offsets[which][p.chunk];
            const uint64_t w1 = a.offsets[which][p.chunk + 1];
            cw.ok = cw.w0 <= w1 && w1 <= a.cap[which] && (which == 0 || p.same);
            cw.nw = cw.ok ? w1 - cw.w0 : 0ull;
            cw.src = a.words[which] + cw.w0;
        }
        return cw;
    };
    auto stage = [&](const ChunkWords &cw, int which) {
        uint32_t *st = sm.stage[warp][which];
        if (cw.nw <= (unsigned long long)kAttnStage) {
            const uint32_t n = (uint32_t)cw.nw;
            for (uint32_t i = lane; i < n; i += 32) {
                const unsigned sa = (unsigned)__cvta_generic_to_shared(st + i);
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(sa), "l"(cw.src + i) : "memory");
            }
            if (lane < kStagePad) st[n + lane] = 0u;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    uint32_t status[2] = {0u, 0u};
    Piece cur = piece_of(st0);
    ChunkWords cw[2] = {words_of(cur, 0), words_of(cur, 1)};
    stage(cw[0], 0);
    stage(cw[1], 1);
    for (uint64_t step = st0; step < st1; step++) {
        const Piece next = piece_of(step + 1);
        float s[MB][2][4];
#pragma unroll
        for (int mb = 0; mb < MB; mb++)
#pragma unroll
            for (int rr = 0; rr < 2; rr++) s[mb][rr][0] = s[mb][rr][1] = s[mb][rr][2] = s[mb][rr][3] = 0.0f;
#pragma unroll 1
        for (int which = 0; which < 2; which++) {
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncwarp();
            const ChunkWords c = which ? cw[1] : cw[0];
            const int k = which ? a.k[1] : a.k[0], kl = which ? a.k_last[1] : a.k_last[0];
            const uint64_t seed = which ? a.seed[1] : a.seed[0];
            const uint32_t nt = (uint32_t)cur.n, nsym = nt * kTile, nseg = 4u * nt;
            const uint32_t nc = (LAT == HQ_E8) ? (16u * nt + 31u) / 32u : 0u;
            const uint32_t nr = (nt * tile_rem_bits<Lattice<LAT>::N>(k, kl) + 31u) >> 5;
            bool ok = cur.on && c.ok && c.nw >= (unsigned long long)(nc + nr) &&
                      (c.nw - nc - nr) < (unsigned long long)(kMaxUnaryBits / 32u);
            const uint32_t nu = ok ? (uint32_t)(c.nw - nc - nr) : 0u;
            const bool staged = c.nw <= (unsigned long long)kAttnStage;
            uint32_t *startbit = sm.start[warp];
            if (which == 1) __syncthreads();   // V's and the weights' buffers are free (the last step's sums are done)
            if (staged)
                ok = find_segment_starts(sm.stage[warp][which] + nc + nr, nu, nsym, nseg, ok, startbit, lane);
            else
                ok = find_segment_starts(c.src + nc + nr, nu, nsym, nseg, ok, startbit, lane);
            // V in units of eref; both in units of 64
            const float zs = which && cur.on ? __fmul_rn(__fdiv_rn(cur.e[1], eref), 0.015625f) : 0.015625f;
            bool bad = cur.on && !ok;
#pragma unroll 1
            for (int rr = 0; rr < 2; rr++) {
                const int ti = 8 * (cur.r0 + rr) + g8;
                const bool valid = cur.on && ti < cur.n;
                uint32_t w[16];
                bool lane_ok = ok;
                if (ok && valid) {
                    const uint32_t segi = 32u * (uint32_t)(cur.r0 + rr) + lane;
                    const unsigned long long e0 = (unsigned long long)(((cur.t0 + ti) * a.heads + head) * kTile);
                    if (staged)
                        lane_ok = decode_quarter<LAT, DITHER, FORM, true>(sm.stage[warp][which], nc, nr, nu, k, kl,
                                                                             startbit[segi], segi, t4, e0, seed, zs, sm.pairs, w);
                    else
                        lane_ok = decode_quarter<LAT, DITHER, FORM, false>(c.src, nc, nr, nu, k, kl, startbit[segi],
                                                                              segi, t4, e0, seed, zs, sm.pairs, w);
                }
                const unsigned bad_lanes = __ballot_sync(0xffffffffu, valid && !lane_ok);
                // a tile that did not decode counts as zeros, as a read stores it
                const bool zero = !valid || ((bad_lanes >> (lane & ~3)) & 0xFu);
                bad |= bad_lanes != 0u;
                if (zero) {
#pragma unroll
                    for (int j = 0; j < 16; j++) w[j] = 0u;
                }
                if (which == 0) {
#pragma unroll
                    for (int st = 0; st < 8; st++) {
#pragma unroll
                        for (int mb = 0; mb < MB; mb++) {
                            const uint4 fh = sm.qh[(mb * 8 + st) * 32 + lane], fl = sm.ql[(mb * 8 + st) * 32 + lane];
                            const uint32_t ah[4] = {fh.x, fh.y, fh.z, fh.w}, al[4] = {fl.x, fl.y, fl.z, fl.w};
                            if (rr == 0) {
                                mma16816(s[mb][0], ah, w[2 * st], w[2 * st + 1]);
                                mma16816(s[mb][0], al, w[2 * st], w[2 * st + 1]);
                            } else {
                                mma16816(s[mb][1], ah, w[2 * st], w[2 * st + 1]);
                                mma16816(s[mb][1], al, w[2 * st], w[2 * st + 1]);
                            }
                        }
                    }
                } else {
                    const int tok = 16 * warp + 8 * rr + g8;
                    uint4 *dst = reinterpret_cast<uint4 *>(sm.v + tok * 64);
#pragma unroll
                    for (int c4 = 0; c4 < 4; c4++)
                        dst[(4 * t4 + c4) ^ (tok & 7)] = make_uint4(w[4 * c4], w[4 * c4 + 1], w[4 * c4 + 2], w[4 * c4 + 3]);
                }
            }
            if (bad) status[which] |= HQ_ST_CORRUPT;
            __syncwarp();
            // the next piece's words, behind the other cache's decode
            cw[which] = words_of(next, which);
            stage(cw[which], which);
            if (which == 0) {
                // scores, masks, and the maximum of each row over this warp's tokens
                const float ek = cur.on ? __fmul_rn(cur.e[0], 64.0f) : 0.0f;
#pragma unroll
                for (int mb = 0; mb < MB; mb++) {
#pragma unroll
                    for (int hf = 0; hf < 2; hf++) {
                        const int r = 16 * mb + 8 * hf + g8;
                        const float qs = __fmul_rn(sm.qscale[r], ek);
                        const int64_t pos = sm.qpos[r];
                        float top = kNegInf;
#pragma unroll
                        for (int rr = 0; rr < 2; rr++) {
#pragma unroll
                            for (int cc = 0; cc < 2; cc++) {
                                const int ti = 8 * (cur.r0 + rr) + 2 * t4 + cc;
                                const int64_t t = cur.t0 + ti;
                                const bool see = cur.on && ti < cur.n && t < a.len && t <= pos &&
                                                 (a.window <= 0 || t > pos - a.window || t < a.sinks);
                                float &x = s[mb][rr][2 * hf + cc];
                                x = see ? __fmul_rn(x, qs) : kNegInf;
                                top = fmaxf(top, x);
                            }
                        }
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                        if (t4 == 0) sm.wmax[step & 1][warp][r] = top;
                    }
                }
            }
        }
        __syncthreads();   // the row maxima and V are there
#pragma unroll
        for (int mb = 0; mb < MB; mb++) {
#pragma unroll
            for (int hf = 0; hf < 2; hf++) {
                const int r = 16 * mb + 8 * hf + g8;
                float m = m_run[mb][hf];
#pragma unroll
                for (int i = 0; i < kAttnWarps; i++) m = fmaxf(m, sm.wmax[step & 1][i][r]);
                const float base = m == kNegInf ? 0.0f : m;   // a row that has seen nothing yet: weights exp2(-inf) = 0
                const float f = ex2(__fsub_rn(m_run[mb][hf], base));
                m_run[mb][hf] = m;
                if (warp == 0 && t4 == 0) sm.rescale[r] = f;
                float sum = 0.0f;
#pragma unroll
                for (int rr = 0; rr < 2; rr++) {
                    const float p0 = ex2(__fsub_rn(s[mb][rr][2 * hf], base)), p1 = ex2(__fsub_rn(s[mb][rr][2 * hf + 1], base));
                    sum = __fadd_rn(sum, __fadd_rn(p0, p1));
                    sm.p[r * (kAttnTokens / 2) + 4 * ((2 * warp + rr) ^ (r & 7)) + t4] = h2_pack(p0, p1);
                }
                l_run[mb][hf] = __fmaf_rn(l_run[mb][hf], f, sum);
            }
        }
        __syncthreads();   // the weights are there
        {
            // sums of this warp's 16 coordinates over the step's tokens: V^T (16 x 16) times P^T (16 x 8 rows)
#pragma unroll
            for (int n = 0; n < 2 * MB; n++) {
                const float f0 = sm.rescale[8 * n + 2 * t4], f1 = sm.rescale[8 * n + 2 * t4 + 1];
                acc[n][0] = __fmul_rn(acc[n][0], f0);
                acc[n][1] = __fmul_rn(acc[n][1], f1);
                acc[n][2] = __fmul_rn(acc[n][2], f0);
                acc[n][3] = __fmul_rn(acc[n][3], f1);
            }
#pragma unroll
            for (int ks = 0; ks < kAttnTokens / 16; ks++) {
                uint32_t av[4];
                const int tok = 16 * ks + 8 * (lane >> 4) + (lane & 7);
                ldsm4t(av, sm.v + tok * 64 + 4 * ((2 * warp + ((lane >> 3) & 1)) ^ (tok & 7)));
#pragma unroll
                for (int n2 = 0; n2 < MB; n2++) {
                    uint32_t bp[4];
                    const int r = 16 * n2 + 8 * (lane >> 4) + (lane & 7);
                    ldsm4(bp, sm.p + r * (kAttnTokens / 2) + 4 * ((2 * ks + ((lane >> 3) & 1)) ^ (r & 7)));
                    mma16816(acc[2 * n2], av, bp[0], bp[1]);
                    mma16816(acc[2 * n2 + 1], av, bp[2], bp[3]);
                }
            }
        }
        cur = next;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");

    // ---- the split's partial results
    const int64_t pbase = ((int64_t)split * a.heads + head) * a.row_pad + row0;
    const float eo = __fmul_rn(eref, 64.0f);
#pragma unroll
    for (int n = 0; n < 2 * MB; n++) {
        float *o = a.part + (pbase + 8 * n + 2 * t4) * kTile + 16 * warp + g8;
        o[0] = __fmul_rn(acc[n][0], eo);
        o[kTile] = __fmul_rn(acc[n][1], eo);
        o[8] = __fmul_rn(acc[n][2], eo);
        o[kTile + 8] = __fmul_rn(acc[n][3], eo);
    }
#pragma unroll
    for (int mb = 0; mb < MB; mb++) {
#pragma unroll
        for (int hf = 0; hf < 2; hf++) {
            float l = l_run[mb][hf];
            l = __fadd_rn(l, __shfl_xor_sync(0xffffffffu, l, 1));
            l = __fadd_rn(l, __shfl_xor_sync(0xffffffffu, l, 2));
            if (t4 == 0) sm.lsum[warp][16 * mb + 8 * hf + g8] = l;
        }
    }
    __syncthreads();
    if (warp == 0 && t4 == 0) {
#pragma unroll
        for (int mb = 0; mb < MB; mb++) {
#pragma unroll
            for (int hf = 0; hf < 2; hf++) {
                const int r = 16 * mb + 8 * hf + g8;
                float l = 0.0f;
                for (int i = 0; i < kAttnWarps; i++) l = __fadd_rn(l, sm.lsum[i][r]);
                a.ml[pbase + r] = make_float2(m_run[mb][hf], l);
            }
        }
    }
#pragma unroll
    for (int which = 0; which < 2; which++) {
        const uint32_t st = __reduce_or_sync(0xffffffffu, status[which]);
        if (lane == 0 && st) atomicOr(&a.stats[which]->status, st);
    }
}

template <int LAT, bool DITHER, int FORM, int MB>
cudaError_t launch_mb(const AttnArgs &a, cudaStream_t s) {
    auto kern = attention_kernel<LAT, DITHER, FORM, MB>;
    static LaunchPlan plan;
    const size_t smem = sizeof(AttnSmem<MB>);
    unsigned grid = 0;
    cudaError_t e = plan.grid(kern, kAttnWarps * 32, smem, 1, grid);
    if (e != cudaSuccess) return e;
    const dim3 g((unsigned)a.splits, (unsigned)a.heads, (unsigned)(a.row_pad / (16 * MB)));
    kern<<<g, kAttnWarps * 32, smem, s>>>(a);
    return cudaGetLastError();
}

template <int LAT, bool DITHER>
cudaError_t launch_lat(const AttnArgs &a, cudaStream_t s) {
    const bool unary = a.k[0] == 0 && a.k[1] == 0 && a.k_last[0] == 0 && a.k_last[1] == 0;
    const bool general = a.k[0] > 4 || a.k[1] > 4 || a.k_last[0] != a.k[0] || a.k_last[1] != a.k[1];
    const bool small = attn_row_block(a.rows) == 16;
    if (unary) return small ? launch_mb<LAT, DITHER, kFormUnary, 1>(a, s) : launch_mb<LAT, DITHER, kFormUnary, 2>(a, s);
    if (general)
        return small ? launch_mb<LAT, DITHER, kFormGeneral, 1>(a, s) : launch_mb<LAT, DITHER, kFormGeneral, 2>(a, s);
    return small ? launch_mb<LAT, DITHER, kFormWindows, 1>(a, s) : launch_mb<LAT, DITHER, kFormWindows, 2>(a, s);
}

}  // namespace

}  // namespace hq
