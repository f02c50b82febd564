// hq_attention.cuh -- attention of a few query tokens over compressed K and V caches
// (hq_kv_attention, hq_kv_tree_attention), without writing K or V to memory.
//
// Mathematics.  A cached vector is x = M z e with z = lattice point - dither, e the append's
// scale and M the inverse rotation (D H_128, or Q^T for a dense rotation), the same for every
// token.  So q . x = (M^T q) . z e, and sum_t p_t x_t = M (sum_t p_t e_t z_t): the queries are
// rotated once, the output once, and no token's tile is transformed.  The softmax runs over
// the tokens as they come, with the running maximum and sum of each row.
//
// Two launches: attention_kernel (up to 16 query rows of a KV head) or attention_wide (up to 256), a grid
// of (splits of the tokens) x (KV heads) x (blocks of rows), leaves a partial (maximum, sum, 128 sums of
// values) per row and split, in the rotated domain; attention_combine joins the splits, turns the result
// back, adds the drafted tokens of a tree (whose K and V are plain bf16) and writes the output.
//
// The products run on the tensor cores in fp16 with fp32 sums:
//  * z / 256 in fp16: exact for codes up to 2048 without dither, else rounded by at most 2^-11 of its value (or
//    2^-17), and finite over the codec's whole range (symbols below 2^22, so |z| < 2^23 + 4 < 256 * 65504: E8's last
//    code of a block is 4 m + 2 p + c, with |m| up to 2^21);
//  * the rotated queries as the sum of two fp16 (scaled by a power of two per row): 2^-22;
//  * the weights w = p e in fp16, e V's scale: it goes into the weights' exponent (log2 p + log2 e), so the
//    row's running maximum is that of p e, and tokens whose scales lie far apart keep their bits whichever of
//    them a row sees.  Held as up to 2^15 times the row's largest: 2^-11 of their value, or 2^-36 of the
//    largest where they are below 2^-25 of it (a long cache's many small weights beside one large, as of a
//    sink).  The softmax's sum adds w / e in fp32.
// In attention_kernel a lane of the Rice decoder holds 32 consecutive coordinates of one token; a step of
// 16 contracted coordinates (mma.sync m16n8k16) takes 4 from each of the 4 lanes of a token, and the queries
// are laid out in the same order, so K goes from the decoder's registers into the product as it is.
//
// Bound: the decoder's integer work, not bytes nor products: 38 lane-instructions a code with dither (E8, 2
// bits), at 3.4 of 4 issued a cycle. One query over 8 x 32768 tokens at 2 bits: 174 us (104 of them the
// decode's at that rate); 64 drafts: 297 us.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "hq_decode.cuh"
#include "hq_table.cuh"

namespace hq {

constexpr int kAttnMaxQueries = 64;   // query tokens of a call (a draft's mask is one word)
constexpr int kAttnMaxGroup = 64;
constexpr int kAttnWarps = 8;
constexpr int kAttnStage = 704;                // staged words of a chunk (5.5 bits per scalar)
constexpr int kAttnCtas = 2 * 148;             // resident CTAs the splits aim at
constexpr uint32_t kAttnWaitPolls = 1u << 20;  // polls of 1 us for the tensor cores before giving up

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
    int splits, row_pad;            // row_pad: rows of a head in `part`
    int short_steps;                // a step is one chunk (RW = 1), not four
    uint32_t wait_limit;            // kAttnWaitPolls, or what a test lowered it to
    float scale_log2;               // scale * log2(e)
    const uint16_t *q;
    int64_t q_ld_tok, q_ld_head;
    const unsigned long long *mask; // tree: visible drafts of each query, or null
    const uint16_t *kd, *vd;
    int64_t d_ld_tok, d_ld_head;
    float *part;                    // [split][head][row_pad][128]
    float2 *ml;                     // [split][head][row_pad]: log2 of the unit of both sums, the softmax's sum
    void *out;
    int out_fp32;
    int64_t out_ld_tok, out_ld_head;
    float *lse;
};

cudaError_t launch_attention(int lattice, int dither, const AttnArgs &a, cudaStream_t s);
cudaError_t launch_attention_z(int dither, const AttnArgs &a, cudaStream_t s);
cudaError_t launch_attention_a2(int dither, const AttnArgs &a, cudaStream_t s);
cudaError_t launch_attention_d4(int dither, const AttnArgs &a, cudaStream_t s);
cudaError_t launch_attention_e8(int dither, const AttnArgs &a, cudaStream_t s);

// Query rows of one CTA: one block of 16 (attention_kernel), or up to 256 in blocks of 128 (attention_wide).
// Over 8 heads, E8 at 2 bits: 16 rows of 32768 tokens take 170 us by the first, about 224 by the second; 20 rows
// 354 (two blocks, so every token twice) and 224; of 4099 tokens 35 and 43, 58 and 43.
constexpr int kNarrowRows = 16;
inline int attn_row_pad(int rows) { return rows <= kNarrowRows ? 16 : (rows + 127) / 128 * 128; }
// Whether steps are of one chunk, whose rounds four warps share, instead of a chunk to a warp: while
// that leaves at most two such steps to a CTA (short caches, where the time is that of one step: 300 tokens
// of 8 heads 27 us so and 31 with a chunk to a warp, ncu; 4100 tokens, at 3.5 steps to a CTA, 43 and 33).
inline bool attn_short(int heads, int rows, uint64_t chunks_per_head) {
    return rows <= kNarrowRows && (uint64_t)heads * chunks_per_head <= 2 * (uint64_t)kAttnCtas;
}
// Splits of the tokens: the CTAs of all heads and row blocks together fill the GPU once.
inline int attn_splits(int heads, int rows, uint64_t chunks_per_head, bool short_steps) {
    const int64_t base = rows <= kNarrowRows ? heads : (int64_t)heads * ((rows + 255) / 256);
    int64_t s = (rows <= kNarrowRows ? kAttnCtas : kAttnCtas / 2) / base;
    const int64_t steps = (int64_t)(short_steps ? chunks_per_head : (chunks_per_head + 3) / 4);
    if (s > steps) s = steps;
    return (int)(s < 1 ? 1 : s);
}

namespace {

constexpr int kTop = 128;   // rows of the append table sampled into shared memory
constexpr float kNegInf = -INFINITY;
constexpr float kCodeUnit = 256.0f;  // of the codes in fp16
constexpr float kTopBits = 15.0f;   // the largest weight in fp16 (up to 65504): 2^15

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
__device__ __forceinline__ void find_row(const AttnArgs &a, const Table<kTop> &t, uint64_t i, AttnRow &r) {
    if (i >= r.base && i < r.base + r.count) return;
    load_row(a, t.append_of(i), r);
}
// Per-head chunks that lie wholly before token t (round_up: that hold any token before t).
__device__ __forceinline__ uint64_t chunks_before(const AttnArgs &a, const Table<kTop> &tab, int64_t t, bool round_up) {
    AttnRow r;
    load_row(a, tab.append_of_token(t), r);
    const int64_t in = t - r.row.token0;
    if (in <= 0) return r.base;
    const uint64_t n = (uint64_t)(round_up ? (in + 31) / 32 : in / 32);
    return r.base + (in >= r.row.tokens ? r.count : n < r.count ? n : r.count);
}

// One warp's part of a step: a chunk of K or V.
struct Piece {
    bool on, ok;          // there is one; the tables agree on it
    int n;                // its tokens
    int64_t t0;           // position of the first
    float e;              // the append's scale
    uint64_t w0, w1;      // its words, as the offsets have them
};

// ------------------------------------------------------------------ E8 dither
// d = w - Q(w) of dither_block<HQ_E8>, bit for bit, in one pass over both candidates.  With w uniform
// on [0, 4)^8, let c_i be w_i's residual to the nearest odd integer (candidate B) and b_i = |c_i|; the
// one to the nearest even integer (candidate A) is c_i - sign(c_i), of size 1 - b_i.  The squared
// distances' difference is then linear in the b_i:
//   D = (|w - A|^2 - |w - B|^2) / 2 = 4 - sum b + 2 p_A min b - 2 p_B (1 - max b),
// the last terms being the parity fixes (the largest residual r becomes 2 - r), with the parities of
// the rounded halves from the two top bits of each w: p_B the XOR of the "w >= 2", p_A of the
// "1 <= w < 3".  Everything is exact in units of 2^-22 but the sum (within 16 units).  The reading
// compares fp32 distances, which are off by less than 2^-16 here (the bound at Lattice<HQ_E8>): a
// difference within 2^-12, a coordinate on a rounding border (b = 0 or 1) or two equal largest
// residuals under a fix goes to the reading's own code instead, about one block in 4000.
//
// Bound by the ALU pipe (half the FMA pipe's rate), so what can be is put on the FMA pipe: w mod 2 by
// one mad.hi that also sets the exponent, and the search for the largest residual by
// saturate(size + 1 - largest), 1 at the largest and 0 elsewhere as sizes are whole units.  24.8
// lane-instructions per element, 11.3 of them the hash, 59.5 us for 67 million elements alone
// (dither_block: about 34).
constexpr float kDitherUnit = 4194304.0f;       // 2^22: d is returned in units of 2^-22
constexpr uint64_t kSplitGolden = 0x9E3779B97F4A7C15ull;

// A pair's hash from its generator state z (s + (i + 1) golden): w of the even and the odd coordinate
// as 32-bit fixed point (bits 8..31 of each count).
__device__ __forceinline__ void dither_pair(uint64_t z, uint32_t &even, uint32_t &odd) {
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    // h = z ^ (z >> 31): bits 40..63 are z's own, bits 8..31 take z's bits 39..62
    even = (uint32_t)(z >> 32);
    odd = (uint32_t)z ^ (even << 1);
}

__device__ __noinline__ void e8_dither_reading(uint64_t z0, float *d) {
    float w[8], p[8];
    int32_t q[8];
    for (int i = 0; i < 4; i++) {
        uint32_t x, y;
        dither_pair(z0 + (uint64_t)i * kSplitGolden, x, y);
        w[2 * i] = __fmul_rn((float)(x >> 8), 0x1p-22f);
        w[2 * i + 1] = __fmul_rn((float)(y >> 8), 0x1p-22f);
    }
    Lattice<HQ_E8>::nearest(w, q);
    Lattice<HQ_E8>::point(q, p);
    for (int i = 0; i < 8; i++) d[i] = __fmul_rn(__fsub_rn(w[i], p[i]), kDitherUnit);
}

__device__ __forceinline__ float add_sat(float a, float b) {
    float r;
    asm("add.rn.sat.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// bits 8..30 of x (w mod 2 in units of 2^-22) plus 2^23, as a float
__device__ __forceinline__ float frac2(uint32_t x) {
    uint32_t r;
    asm("mad.hi.u32 %0, %1, %2, %3;" : "=r"(r) : "r"(x * 2u), "r"(1u << 23), "r"(0x4B000000u));
    return __uint_as_float(r);
}

// The block whose first pair has generator state z0; d in units of 2^-22.
__device__ __forceinline__ void e8_dither(uint64_t z0, float (&d)[8]) {
    constexpr float U = kDitherUnit;
    float c[8];
    uint32_t xe = 0, xo = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        uint32_t x, y;
        dither_pair(z0 + (uint64_t)i * kSplitGolden, x, y);
        xe ^= x;
        xo ^= y;
        const float2 r = f2_sub(make_float2(frac2(x), frac2(y)), make_float2(8388608.0f + U, 8388608.0f + U));
        c[2 * i] = r.x;
        c[2 * i + 1] = r.y;
    }
    const uint32_t par = xe ^ xo;
    const bool pb = (int32_t)par < 0, pa = (int32_t)(par ^ (par << 1)) < 0;
    float lo = fabsf(c[0]), hi = lo;
#pragma unroll
    for (int i = 1; i < 8; i++) {
        lo = fminf(lo, fabsf(c[i]));
        hi = fmaxf(hi, fabsf(c[i]));
    }
    const float s0 = __fadd_rn(__fadd_rn(fabsf(c[0]), fabsf(c[1])), __fadd_rn(fabsf(c[2]), fabsf(c[3])));
    const float s1 = __fadd_rn(__fadd_rn(fabsf(c[4]), fabsf(c[5])), __fadd_rn(fabsf(c[6]), fabsf(c[7])));
    const float diff = __fadd_rn(__fsub_rn(__fsub_rn(4.0f * U, s0), s1),
                                 __fsub_rn(pa ? __fadd_rn(lo, lo) : 0.0f, pb ? __fmaf_rn(-2.0f, hi, 2.0f * U) : 0.0f));
    const bool odd = diff > 0.0f, fix = odd ? pb : pa;
    // signed sizes |c| - m (A's turned); the fix takes the largest by 2 the other way
    const float m = odd ? 0.0f : -U, turn = odd ? -2.0f * U : 2.0f * U, top = odd ? hi : __fsub_rn(U, lo);
    const float shift = fix ? __fsub_rn(1.0f, top) : -INFINITY;
    float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float t0 = __fadd_rn(fabsf(c[2 * i]), m), t1 = __fadd_rn(fabsf(c[2 * i + 1]), m);
        const float2 e = make_float2(add_sat(fabsf(t0), shift), add_sat(fabsf(t1), shift));
        sum = f2_add(sum, e);
        const float2 r = f2_fma(e, make_float2(turn, turn), make_float2(t0, t1));
        d[2 * i] = __uint_as_float(__float_as_uint(r.x) ^ (__float_as_uint(c[2 * i]) & 0x80000000u));
        d[2 * i + 1] = __uint_as_float(__float_as_uint(r.y) ^ (__float_as_uint(c[2 * i + 1]) & 0x80000000u));
    }
    if (fabsf(diff) <= 1024.0f || lo == 0.0f || hi == U || __fadd_rn(sum.x, sum.y) != (fix ? 1.0f : 0.0f)) {
        float r[8];
        e8_dither_reading(z0, r);
#pragma unroll
        for (int i = 0; i < 8; i++) d[i] = r[i];
    }
}

// ------------------------------------------------------------------ decode
// Forms of the Rice code: no remainders at all (k = 0: the 2-bit caches), or any parameters.
enum AttnForm { kFormUnary = 0, kFormGeneral = 1 };

// Codewords two at a time: the next 10 unary bits -> both quotients.  Bits 0..4 their length, byte 1 and
// byte 2 the quotients, bit 31 set if both end inside the 10 bits (at 2 bits per scalar one pair in 2000
// does not).  CODES (E8 without remainders): bytes 1 and 2 are the codes 2 m + 128 instead (2 m the zigzag
// inverse doubled), bit 24 the parity of m of both, bit 25 of the first.
constexpr int kPairBits = 10;
template <bool CODES>
__device__ __forceinline__ uint32_t pair_entry(uint32_t w) {
    const uint32_t t0 = (uint32_t)__ffs((int)(w | 0x80000000u)) - 1u;
    const uint32_t t1 = t0 < 31u ? (uint32_t)__ffs((int)((w >> (t0 + 1u)) | 0x80000000u)) - 1u : 31u;
    if (t0 + t1 + 2u > (uint32_t)kPairBits) return 0u;
    if (!CODES) return 0x80000000u | (t0 + t1 + 2u) | t0 << 8 | t1 << 16;
    const uint32_t a = t0 ^ (0u - (t0 & 1u)), b = t1 ^ (0u - (t1 & 1u));   // 2 m
    return 0x80000000u | (t0 + t1 + 2u) | ((a + 128u) & 0xFFu) << 8 | ((b + 128u) & 0xFFu) << 16 |
           (((a ^ b) >> 1) & 1u) << 24 | ((a >> 1) & 1u) << 25;
}
// Four pairs from unary bit bp on; whether all of them ended in time, and their length.  The plane's
// terminators were counted, so a lane's codewords end inside it (or in the pad behind its last word,
// which the second word of a window may reach).
__device__ __forceinline__ bool read_pairs(const uint32_t *un, uint32_t bp, const uint32_t *pairs, uint32_t (&e)[4],
                                           uint32_t &used) {
    used = 0;
#pragma unroll
    for (int h = 0; h < 2; h++) {
        const uint32_t *p = un + ((bp + used) >> 5);
        uint32_t x = __funnelshift_r(p[0], p[1], bp + used);
        e[2 * h] = pairs[x & ((1u << kPairBits) - 1u)];
        x = __funnelshift_r(x, 0u, e[2 * h]);
        e[2 * h + 1] = pairs[x & ((1u << kPairBits) - 1u)];
        used += (e[2 * h] + e[2 * h + 1]) & 0x1Fu;
    }
    return (int32_t)(e[0] & e[1] & e[2] & e[3]) < 0;
}

// What a lane decodes in a round: its quarter of a tile, 32 codes in four blocks of 8.
struct Quarter {
    const uint32_t *un, *rem;       // unary and remainder planes
    uint32_t nu, nr;                // their words
    uint32_t bp;                    // next unary bit
    uint32_t rb;                    // next remainder bit
    uint32_t coset;                 // E8: coset bits of the blocks left
    unsigned long long e0;          // dither counter of the next element (E8: the pair's generator state)
    bool ok;
};
template <int LAT, int FORM>
__device__ __forceinline__ void open_quarter(Quarter &t, const uint32_t *src, uint32_t nc, uint32_t nr, uint32_t nu, int k,
                                             int kl, uint64_t seed, uint32_t start, uint32_t segi,
                                             unsigned long long e0) {
    t.rem = src + nc;
    t.un = src + nc + nr;
    t.nu = nu;
    t.nr = nr;
    t.bp = start;
    t.rb = FORM == kFormUnary ? 0u : segi * 4u * group_rem_bits<Lattice<LAT>::N>(k, kl);
    t.coset = LAT == HQ_E8 ? src[segi >> 3] >> (4 * (segi & 7u)) : 0u;
    t.e0 = e0 + 32ull * (segi & 3u);
    if (LAT == HQ_E8) t.e0 = (seed ^ kDitherSalt) + ((t.e0 >> 1) + 1ull) * kSplitGolden;
    t.ok = true;
}

// The next 8 codes (minus dither) times `scale`, as 4 fp16 pairs.
template <int LAT, bool DITHER, int FORM, bool STAGED>
__device__ __forceinline__ void decode_block(Quarter &t, int k, int kl, uint64_t seed, float scale, const uint32_t *pairs,
                                             uint32_t (&w)[4]) {
    using L = Lattice<LAT>;
    constexpr int N = L::N;
    float u[8];
    const uint32_t c = t.coset & 1u;
    t.coset >>= 1;
    if constexpr (LAT == HQ_E8 && FORM == kFormUnary && STAGED) {
        uint32_t e[4], used;
        if (read_pairs(t.un, t.bp, pairs, e, used)) {
            t.bp += used;
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
            unary4<STAGED>(t.un, t.nu, t.bp, t.ok, zq);
            unary4<STAGED>(t.un, t.nu, t.bp, t.ok, zq + 4);
            int32_t qq[8];
            e8_codes_from_symbols(zq, c, qq);
            decoded_point<HQ_E8>(qq, u);
        }
    } else {
        uint32_t qv[8], rv[8];
        uint32_t e[4], used;
        if (STAGED && read_pairs(t.un, t.bp, pairs, e, used)) {
            t.bp += used;
#pragma unroll
            for (int h = 0; h < 4; h++) {
                qv[2 * h] = __byte_perm(e[h], 0u, 0x4441);
                qv[2 * h + 1] = __byte_perm(e[h], 0u, 0x4442);
            }
        } else {
            unary4<STAGED>(t.un, t.nu, t.bp, t.ok, qv);
            unary4<STAGED>(t.un, t.nu, t.bp, t.ok, qv + 4);
        }
        if (FORM == kFormGeneral) {
            const uint32_t gbits = group_rem_bits<N>(k, kl);
            rem_group_mixed<N, STAGED>(t.rem, t.nr, t.rb, 0, k, kl, gbits, rv);
            t.rb += gbits;
        }
        const uint32_t pk = 1u << k, pkl = 1u << kl;
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
                e8_codes_from_symbols(zb, c, qq);
            } else {
                int32_t m[N];
#pragma unroll
                for (int i = 0; i < N; i++) m[i] = unzigzag(zb[i]);
                L::reinsert(m, 0u, qq);
            }
            decoded_point<LAT>(qq, p);
            if (DITHER && LAT != HQ_E8) {
                float d[N];
                dither_block<LAT>(seed, t.e0 + (unsigned long long)(bb * N), d);
#pragma unroll
                for (int i = 0; i < N; i++) p[i] = __fsub_rn(p[i], d[i]);
            }
#pragma unroll
            for (int i = 0; i < N; i++) u[bb * N + i] = p[i];
        }
    }
    const float2 s2 = make_float2(scale, scale);
    if constexpr (DITHER && LAT == HQ_E8) {
        float d[8];   // in units of 2^-22
        e8_dither(t.e0, d);
        const float sd = __fmul_rn(scale, -0x1p-22f);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const float2 x = f2_fma(make_float2(d[2 * j], d[2 * j + 1]), make_float2(sd, sd),
                                    f2_mul(make_float2(u[2 * j], u[2 * j + 1]), s2));
            w[j] = h2_pack(x.x, x.y);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const float2 x = f2_mul(make_float2(u[2 * j], u[2 * j + 1]), s2);
            w[j] = h2_pack(x.x, x.y);
        }
    }
    t.e0 += LAT == HQ_E8 ? 4ull * kSplitGolden : 8ull;
}
__device__ __forceinline__ bool close_quarter(const Quarter &t) { return t.ok && t.bp <= t.nu * 32u; }

// ------------------------------------------------------------------ segment starts
// Where the 32-symbol segments [s0, s1) of a chunk start (s1 - s0 = 32 rounds' worth of what the warp
// decodes): seg[s] = 32 i + n says that terminator 32 s - 1 is the n-th (0-based) set bit of unary word i.
// 128 words at a time, a lane to four words: population counts, a scan of two packed in one register, and
// every word that holds a boundary (at most one) notes it; each lane finds the bit itself for the segments
// it decodes (segment_start).  Words wholly before or behind the wanted segments are only counted.  False
// unless the plane holds exactly nsym terminators.
__device__ __forceinline__ bool scan_segments(const uint32_t *un, uint32_t nu, uint32_t nsym, uint32_t s0, uint32_t s1,
                                              uint32_t *seg, int lane) {
    uint32_t seen = 0;
    const uint32_t want0 = 32u * s0, want1 = 32u * s1;   // terminators want0 - 1 .. want1 - 33 are looked for
    for (uint32_t i0 = 0; i0 < nu; i0 += 128) {
        uint32_t p[4];
#pragma unroll
        for (int u = 0; u < 4; u++) p[u] = i0 + 32u * u + lane < nu ? __popc(un[i0 + 32u * u + lane]) : 0u;
        const uint32_t total = __reduce_add_sync(0xffffffffu, (p[0] + p[1]) + (p[2] + p[3]));
        if (seen + total >= want0 && seen < want1) {
            uint32_t both[2] = {p[0] | p[1] << 16, p[2] | p[3] << 16};
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const uint32_t v = __shfl_up_sync(0xffffffffu, both[h], o);
                    if (lane >= o) both[h] += v;
                }
            }
            uint32_t before = seen;
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const uint32_t all = __shfl_sync(0xffffffffu, both[h], 31), i = i0 + 64u * h + lane;
                const uint32_t b0 = before + (both[h] & 0xFFFFu) - p[2 * h];
                const uint32_t b1 = before + (all & 0xFFFFu) + (both[h] >> 16) - p[2 * h + 1];
                // a boundary past the last segment means a corrupt plane: not noted, and found by the count
                if ((b0 >> 5) != ((b0 + p[2 * h]) >> 5) && b0 < nsym) seg[(b0 >> 5) + 1u] = i * 32u + (31u - (b0 & 31u));
                if ((b1 >> 5) != ((b1 + p[2 * h + 1]) >> 5) && b1 < nsym)
                    seg[(b1 >> 5) + 1u] = (i + 32u) * 32u + (31u - (b1 & 31u));
                before += (all & 0xFFFFu) + (all >> 16);
            }
        }
        seen += total;
    }
    __syncwarp();
    return seen == nsym;
}
__device__ __forceinline__ uint32_t segment_start(const uint32_t *un, const uint32_t *seg, uint32_t s) {
    if (s == 0u) return 0u;
    const uint32_t v = seg[s];
    return (v & ~31u) + select_bit(un[v >> 5], v & 31u) + 1u;
}

// ------------------------------------------------------------------ shared memory
// RW: decoder rounds (8 tokens) of a warp in a step of 32 RW tokens.  Half of the CTA's warps decode K,
// half V: a chunk each (RW = 4), or a round of one chunk (RW = 1).
template <int RW>
struct AttnSmem {
    static constexpr int R = 16, NT = 32 * RW, SP = NT + 8;
    uint4 qh[8 * 32], ql[8 * 32];               // query fragments (two fp16 parts)
    uint32_t v[NT * 64];                        // V: [token][128] fp16, 16-byte pieces swizzled by the token
    uint32_t p[R * (NT / 2)];                   // weights: [row][token] fp16, pieces swizzled by the row
    float sc[R * SP];                           // scores (log2)
    uint32_t stage[kAttnWarps][2][kAttnStage + kStagePad];
    uint32_t seg[kAttnWarps][129];
    uint32_t sign[4];
    uint32_t pairs[1 << kPairBits];             // pair_entry
    float rescale[R];                           // of the sums, this step
    float qscale[R];                            // undoes a row's power-of-two scale, with the softmax scale
    int64_t qpos[R];
    float xs[kAttnWarps][128];
    uint64_t range[3];
    int64_t span[2];                            // first and last position of the CTA's queries
    float2 ev[4];                               // V's scales of the step's chunks: vscale
    TopRow top[kTop];
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

// ------------------------------------------------------------------ what both kernels share
// Chunks of a head that some query may see: [0, range[0]) and [range[1], range[2]), one bound each by the
// first threads of warps 5 to 7 (range[0] and range[1] still to be put in order: see_bounds).
__device__ __forceinline__ void visible_range(const AttnArgs &a, const Table<kTop> &tab, uint64_t *range) {
    if (threadIdx.x == 160) range[2] = chunks_before(a, tab, a.len, true);
    if (threadIdx.x == 192 && a.window > 0)
        range[0] = a.sinks > 0 ? chunks_before(a, tab, a.sinks < a.len ? a.sinks : a.len, true) : 0;
    if (threadIdx.x == 224 && a.window > 0) {
        const int64_t lo = (a.mask ? a.len - 1 : a.len - a.n_q) - a.window + 1;   // of any query: a bound is enough
        range[1] = lo > 0 ? chunks_before(a, tab, lo, false) : 0;
    }
}
__device__ __forceinline__ void see_bounds(const AttnArgs &a, const uint64_t *range, uint64_t &ia, uint64_t &ib, uint64_t &ie) {
    ie = range[2];
    ia = a.window > 0 ? range[0] : ie;
    ib = a.window > 0 ? range[1] : ie;
    if (ib < ia) ib = ia;
}
// Bounds of the positions of query rows [row0, row0 + n): in order without a tree, at most their count
// apart with one.
__device__ __forceinline__ void query_span(const AttnArgs &a, int row0, int n, int64_t *span) {
    const int i0 = row0 / a.group, i1 = min(a.rows - 1, row0 + n - 1) / a.group;
    span[0] = a.mask ? a.len - 1 : a.len - a.n_q + i0;
    span[1] = a.mask ? a.len - 1 + a.n_q : a.len - a.n_q + i1;
}
// Position of a query row; one past the last sees nothing.
__device__ __forceinline__ int64_t query_position(const AttnArgs &a, int row) {
    if (row >= a.rows) return INT64_MIN / 2;
    const int i = row / a.group;
    if (!a.mask) return a.len - a.n_q + i;
    const unsigned long long all = a.n_q < 64 ? (1ull << a.n_q) - 1ull : ~0ull;
    return a.len - 1 + __popcll(a.mask[i] & all);
}
// A query row, rotated, times the power of two that brings its largest value into [1, 2) (rows of zeros,
// infinities: 1), 4 coordinates to a lane; up: the power's inverse.  Whole warp.
__device__ __forceinline__ void load_query(const AttnArgs &a, int head, int row, const uint32_t *sign, float *xs, int lane,
                                           float (&u)[4], float &up) {
    u[0] = u[1] = u[2] = u[3] = 0.0f;
    if (row < a.rows) {
        const int i = row / a.group, qh = head * a.group + row - i * a.group;
        const uint2 x = *reinterpret_cast<const uint2 *>(a.q + i * a.q_ld_tok + qh * a.q_ld_head + 4 * lane);
        u[0] = __uint_as_float(x.x << 16);
        u[1] = __uint_as_float(x.x & 0xFFFF0000u);
        u[2] = __uint_as_float(x.y << 16);
        u[3] = __uint_as_float(x.y & 0xFFFF0000u);
    }
    rotate_query(a, u, sign, xs, lane);
    float top = fmaxf(fmaxf(fabsf(u[0]), fabsf(u[1])), fmaxf(fabsf(u[2]), fabsf(u[3])));
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
    const int ex = (int)(__float_as_uint(top) >> 23) - 127;
    const bool in = ex >= -126 && ex <= 126;
    const float down = in ? __uint_as_float((uint32_t)(127 - ex) << 23) : 1.0f;
    up = in ? __uint_as_float((uint32_t)(127 + ex) << 23) : 1.0f;
#pragma unroll
    for (int j = 0; j < 4; j++) u[j] = __fmul_rn(u[j], down);
}
// What V's scale e of a chunk's append does to its weights: (log2 of 256 e, 1 / (256 e)), codes being in units of
// 256.  The first is added to the scores, the second takes it out of the softmax's sum again.
__device__ __forceinline__ float2 vscale(float e) {
    const float x = __fmul_rn(e, kCodeUnit);
    return make_float2(log2f(x), __fdiv_rn(1.0f, x));
}

// The cache that a warp decodes: K (0) or V (1).
struct Source {
    const uint32_t *words;
    const uint64_t *offsets;
    uint64_t cap, seed;
    int which, k, kl;
    AttnRow row;
    bool same;    // V: its append covers the same tokens as K's
    float e;      // the append's scale in this cache
    __device__ __forceinline__ void init(const AttnArgs &a, int w) {
        which = w;
        words = a.words[w];
        offsets = a.offsets[w];
        cap = a.cap[w];
        seed = a.seed[w];
        k = a.k[w];
        kl = a.k_last[w];
        row.base = row.count = 0;   // none yet
    }
    // visible chunk v
    __device__ __forceinline__ Piece piece(const AttnArgs &a, const Table<kTop> &tab, int head, uint64_t v, bool on, uint64_t nvis, uint64_t ia,
                                           uint64_t ib) {
        Piece p;
        p.on = on && v < nvis;
        p.ok = false;
        p.n = 0;
        p.t0 = 0;
        p.e = 0.0f;
        p.w0 = p.w1 = 0;
        if (p.on) {
            const uint64_t i = v < ia ? v : v - ia + ib;
            if (!(i >= row.base && i < row.base + row.count)) {
                find_row(a, tab, i, row);
                same = true;
                e = row.row.scale_inv;
                if (which) {
                    const hq_kv_append_row vr = a.table[1][row.append];
                    same = vr.first_chunk == row.row.first_chunk && vr.token0 == row.row.token0 &&
                           vr.tokens == row.row.tokens;
                    e = vr.scale_inv;
                }
            }
            const uint64_t j = i - row.base;
            p.t0 = row.row.token0 + 32 * (int64_t)j;
            const int64_t left = (int64_t)row.row.tokens - 32 * (int64_t)j;
            p.n = (int)(left < 32 ? left : 32);
            const uint64_t chunk = row.row.first_chunk + (uint64_t)head * row.count + j;
            p.e = e;
            p.ok = same && chunk < a.n_chunks;
            if (p.ok) {
                p.w0 = offsets[chunk];
                p.w1 = offsets[chunk + 1];
            }
        }
        return p;
    }
    // its words into a stage, by `of` threads (nothing for a chunk that is not sound or does not fit)
    __device__ __forceinline__ void stage(const Piece &p, uint32_t *st, int me, int of) const {
        if (p.on && p.ok && p.w0 <= p.w1 && p.w1 <= cap && p.w1 - p.w0 <= (unsigned long long)kAttnStage) {
            const uint32_t n = (uint32_t)(p.w1 - p.w0);
            const uint32_t *src = words + p.w0;
            for (uint32_t i = me; i < n; i += of) {
                const unsigned sa = (unsigned)__cvta_generic_to_shared(st + i);
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(sa), "l"(src + i) : "memory");
            }
            if (me < kStagePad) st[n + me] = 0u;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
};
// A piece's planes, in words.
struct Planes {
    uint32_t nc, nr, nu, nsym;
    bool ok, staged;
};
template <int LAT, int FORM>
__device__ __forceinline__ Planes planes_of(const Source &s, const Piece &p) {
    Planes r;
    const uint32_t nt = (uint32_t)p.n;
    r.nsym = nt * kTile;
    r.nc = (LAT == HQ_E8) ? (16u * nt + 31u) / 32u : 0u;
    r.nr = FORM == kFormUnary ? 0u : (nt * tile_rem_bits<Lattice<LAT>::N>(s.k, s.kl) + 31u) >> 5;
    r.ok = p.on && p.ok && p.w0 <= p.w1 && p.w1 <= s.cap;
    const unsigned long long nw = r.ok ? p.w1 - p.w0 : 0ull;
    r.ok = r.ok && nw >= (unsigned long long)(r.nc + r.nr) && (nw - r.nc - r.nr) < (unsigned long long)(kMaxUnaryBits / 32u);
    r.nu = r.ok ? (uint32_t)(nw - r.nc - r.nr) : 0u;
    r.staged = nw <= (unsigned long long)kAttnStage;
    return r;
}
// Whether every query sees every token of a whole chunk.
__device__ __forceinline__ bool all_see(const AttnArgs &a, const Piece &p, const int64_t *span) {
    const int64_t tl = p.t0 + 31;
    return p.on && p.n == 32 && tl < a.len && tl <= span[0] &&
           (a.window <= 0 || p.t0 > span[1] - a.window || tl < a.sinks);
}
// One round of a sound chunk: each lane decodes its quarter of a tile and hands every block (8 codes as 4
// words) to `use`.  A lane whose tile is not there decodes the chunk's first segment and scales it to zero,
// so the warp runs one path.  Returns the lanes whose tile did not decode.
template <int LAT, bool DITHER, int FORM, bool STAGED, typename F>
__device__ __forceinline__ unsigned decode_round(const uint32_t *p, const Planes &pl, const Source &src, const uint32_t *seg,
                                                 uint32_t segi, bool valid, unsigned long long e0, float scale,
                                                 const uint32_t *pairs, F &&use) {
    if (!valid) {
        segi = 0u;   // its start needs no note
        scale = 0.0f;
    }
    Quarter t;
    open_quarter<LAT, FORM>(t, p, pl.nc, pl.nr, pl.nu, src.k, src.kl, src.seed,
                           segment_start(p + pl.nc + pl.nr, seg, segi), segi, e0);
#pragma unroll
    for (int g = 0; g < 4; g++) {
        uint32_t w[4];
        decode_block<LAT, DITHER, FORM, STAGED>(t, src.k, src.kl, src.seed, scale, pairs, w);
        use(g, w);
    }
    return __ballot_sync(0xffffffffu, valid && !close_quarter(t));
}
template <int LAT, bool DITHER, int FORM, typename F>
__device__ __forceinline__ unsigned decode_round(bool ok, bool staged, const uint32_t *st, const uint32_t *gsrc,
                                                 const Planes &pl, const Source &src, const uint32_t *seg, uint32_t segi,
                                                 bool valid, unsigned long long e0, float scale, const uint32_t *pairs,
                                                 F &&use) {
    if (ok && staged) return decode_round<LAT, DITHER, FORM, true>(st, pl, src, seg, segi, valid, e0, scale, pairs, use);
    if (ok) return decode_round<LAT, DITHER, FORM, false>(gsrc, pl, src, seg, segi, valid, e0, scale, pairs, use);
#pragma unroll
    for (int g = 0; g < 4; g++) {
        const uint32_t w[4] = {0u, 0u, 0u, 0u};
        use(g, w);
    }
    return 0u;
}

template <int LAT, bool DITHER, int FORM, int RW>
__global__ void __launch_bounds__(kAttnWarps * 32, 2) attention_kernel(const __grid_constant__ AttnArgs a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    using Smem = AttnSmem<RW>;
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
    constexpr int R = Smem::R, NT = Smem::NT, SP = Smem::SP, KW = kAttnWarps / 2;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g8 = lane >> 2, t4 = lane & 3;
    const int split = blockIdx.x, head = blockIdx.y, row0 = blockIdx.z * R;

    cudaTriggerProgrammaticLaunchCompletion();   // the combine may come up; it waits for this grid's end
    // ---- which chunks the queries can see, the queries themselves
    const Table<kTop> tab(a.table[0], a.n_appends, a.heads, sm.top);
    tab.load(sm.top);
    if (threadIdx.x == 128) query_span(a, row0, R, sm.span);
    build_sign_table(sm.sign, 1, a.seed[0]);
    for (int i = threadIdx.x; i < (1 << kPairBits); i += blockDim.x)
        sm.pairs[i] = pair_entry<LAT == HQ_E8 && FORM == kFormUnary>((uint32_t)i);
    for (int r = threadIdx.x; r < R; r += blockDim.x) sm.qpos[r] = query_position(a, row0 + r);
    __syncthreads();
    visible_range(a, tab, sm.range);
    __syncwarp();
    for (int r = warp; r < R; r += kAttnWarps) {
        float u[4] = {}, up = 1.0f;
        if (row0 + r < a.rows) load_query(a, head, row0 + r, sm.sign, sm.xs[warp], lane, u, up);
        // fragment of coordinate c for row r: step s = (c mod 32) / 4 of lane quarter c / 32
#pragma unroll
        for (int pr = 0; pr < 2; pr++) {
            const float x0 = u[2 * pr], x1 = u[2 * pr + 1];
            const uint32_t hi = h2_pack(x0, x1);
            const __half2 hh = *reinterpret_cast<const __half2 *>(&hi);
            const uint32_t lo = h2_pack(__fsub_rn(x0, __low2float(hh)), __fsub_rn(x1, __high2float(hh)));
            // coordinates 4 lane + 2 pr: quarter lane / 8, step lane % 8, register pair pr
            const int slot = (lane & 7) * 32 + (r & 7) * 4 + (lane >> 3);
            const int reg = ((r >> 3) & 1) + 2 * pr;
            reinterpret_cast<uint32_t *>(sm.qh)[slot * 4 + reg] = hi;
            reinterpret_cast<uint32_t *>(sm.ql)[slot * 4 + reg] = lo;
        }
        if (lane == 0) sm.qscale[r] = __fmul_rn(up, a.scale_log2);
    }
    __syncthreads();
    uint64_t ia, ib, ie;
    see_bounds(a, sm.range, ia, ib, ie);
    const uint64_t nvis = ia + (ie - ib);
    const uint64_t steps = (nvis + RW - 1) / RW;
    // this CTA's steps: an even share
    const uint64_t st0 = steps * (uint64_t)split / (uint64_t)a.splits;
    const uint64_t st1 = steps * (uint64_t)(split + 1) / (uint64_t)a.splits;

    // softmax state of row tid / 16, the same in its 16 threads but for the sums
    float m_run = kNegInf, l_run = 0.0f, acc[2][4] = {};

    // ---- this warp's part of a step: a chunk (RW = 4) or a round of one (RW = 1), of K or of V
    const int which = warp / KW, wi = warp % KW, ci = RW == 4 ? wi : 0;
    Source src;
    src.init(a, which);
    uint32_t status = 0u;
    int buf = 0;
    Piece cur = src.piece(a, tab, head, st0 * RW + ci, st0 < st1, nvis, ia, ib);
    src.stage(cur, sm.stage[warp][0], lane, 32);
    Piece next = src.piece(a, tab, head, (st0 + 1) * RW + ci, st0 + 1 < st1, nvis, ia, ib);
    for (uint64_t step = st0; step < st1; step++, buf ^= 1) {
        // the next chunk's words behind this one's decode, and the offsets of the one after it
        src.stage(next, sm.stage[warp][buf ^ 1], lane, 32);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncwarp();
        const Planes pl = planes_of<LAT, FORM>(src, cur);
        const bool staged = pl.staged;
        const uint32_t *const st = sm.stage[warp][buf], *const gsrc = src.words + cur.w0;
        uint32_t *const seg = sm.seg[warp];
        bool ok = pl.ok;
        const uint32_t seg0 = RW == 4 ? 0u : 32u * wi, seg1 = RW == 4 ? 128u : seg0 + 32u;
        if (staged)
            ok = scan_segments(st + pl.nc + pl.nr, pl.nu, pl.nsym, seg0, seg1, seg, lane) && ok;
        else
            ok = scan_segments(gsrc + pl.nc + pl.nr, pl.nu, pl.nsym, seg0, seg1, seg, lane) && ok;
        const int r0 = RW == 4 ? 0 : wi;
        // codes in units of 256; K's scales go into the scores, V's into the weights
        const float ek = cur.on ? __fmul_rn(cur.e, kCodeUnit) : 0.0f;
        if (which && r0 == 0 && lane == 0) sm.ev[ci] = cur.on ? vscale(cur.e) : make_float2(0.0f, 1.0f);
        const bool open = all_see(a, cur, sm.span);
        bool bad = cur.on && !ok;
#pragma unroll 1
        for (int rr = 0; rr < RW; rr++) {
            const int ti = 8 * (r0 + rr) + g8;
            const bool valid = cur.on && ti < cur.n;
            const int tok = (RW == 4 ? 32 * wi + 8 * rr : 8 * wi);   // the round's first token in the step
            uint32_t w[16];
            const unsigned long long e0 = (unsigned long long)(((cur.t0 + ti) * a.heads + head) * kTile);
            // a tile that did not decode counts as zeros, as a read stores it
            const unsigned lost = decode_round<LAT, DITHER, FORM>(
                ok, staged, st, gsrc, pl, src, seg, 32u * (uint32_t)(r0 + rr) + lane, valid, e0, 1.0f / kCodeUnit, sm.pairs,
                [&](int g, const uint32_t (&x)[4]) {
#pragma unroll
                    for (int i = 0; i < 4; i++) w[4 * g + i] = x[i];
                });
            float s[2][4] = {};
            uint4 *const dst = reinterpret_cast<uint4 *>(sm.v + (tok + g8) * 64);
            if (which == 0) {
#pragma unroll
                for (int h = 0; h < 8; h++) {
                    const uint4 fh = sm.qh[h * 32 + lane], fl = sm.ql[h * 32 + lane];
                    const uint32_t ah[4] = {fh.x, fh.y, fh.z, fh.w}, al[4] = {fl.x, fl.y, fl.z, fl.w};
                    mma16816(s[0], ah, w[2 * h], w[2 * h + 1]);
                    mma16816(s[1], al, w[2 * h], w[2 * h + 1]);
                }
            } else {
#pragma unroll
                for (int g = 0; g < 4; g++)
                    dst[(4 * t4 + g) ^ g8] = make_uint4(w[4 * g], w[4 * g + 1], w[4 * g + 2], w[4 * g + 3]);
            }
            bad |= lost != 0u;
            if (which == 0) {
#pragma unroll
                for (int hf = 0; hf < 2; hf++) {
                    const int r = 8 * hf + g8;
                    const float qs = __fmul_rn(sm.qscale[r], ek);
                    float x[2];
#pragma unroll
                    for (int cc = 0; cc < 2; cc++) {
                        x[cc] = __fmul_rn(__fadd_rn(s[0][2 * hf + cc], s[1][2 * hf + cc]), qs);
                        if (lost && ((lost >> (4 * (2 * t4 + cc))) & 0xFu)) x[cc] = 0.0f;
                        if (!open) {
                            const int tc = 8 * (r0 + rr) + 2 * t4 + cc;
                            const int64_t tt = cur.t0 + tc, pos = sm.qpos[r];
                            const bool see = cur.on && tc < cur.n && tt < a.len && tt <= pos &&
                                             (a.window <= 0 || tt > pos - a.window || tt < a.sinks);
                            if (!see) x[cc] = kNegInf;
                        }
                    }
                    *reinterpret_cast<float2 *>(sm.sc + r * SP + tok + 2 * t4) = make_float2(x[0], x[1]);
                }
            } else if ((lost >> (lane & ~3)) & 0xFu) {
#pragma unroll
                for (int g = 0; g < 4; g++) dst[(4 * t4 + g) ^ g8] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
        if (bad) status |= HQ_ST_CORRUPT;
        const Piece after = src.piece(a, tab, head, (step + 2) * RW + ci, step + 2 < st1, nvis, ia, ib);
        __syncthreads();   // scores and V are there
        {
            // softmax: 16 threads to a row, NT / 16 tokens each
            constexpr int PT = NT / 16;
            const int r = threadIdx.x >> 4, j = threadIdx.x & 15;
            float x[PT];
            const float *sc = sm.sc + r * SP + PT * j;
            if constexpr (PT == 8) {
                const float4 y0 = reinterpret_cast<const float4 *>(sc)[0], y1 = reinterpret_cast<const float4 *>(sc)[1];
                x[0] = y0.x; x[1] = y0.y; x[2] = y0.z; x[3] = y0.w;
                x[4] = y1.x; x[5] = y1.y; x[6] = y1.z; x[7] = y1.w;
            } else {
                const float2 y = *reinterpret_cast<const float2 *>(sc);
                x[0] = y.x; x[1] = y.y;
            }
            const float2 e = sm.ev[PT * j / 32];   // a thread's tokens are of one chunk
            float m = m_run;
#pragma unroll
            for (int i = 0; i < PT; i++) {
                x[i] = __fadd_rn(x[i], e.x);
                m = fmaxf(m, x[i]);
            }
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float top = m == kNegInf ? 0.0f : m;   // a row that has seen nothing yet: weights exp2(-inf) = 0
            const float f = ex2(__fsub_rn(m_run, top)), base = __fsub_rn(top, kTopBits);
            m_run = m;
            if (j == 0) sm.rescale[r] = f;
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < PT; i++) {
                x[i] = ex2(__fsub_rn(x[i], base));
                sum = __fadd_rn(sum, x[i]);
            }
            l_run = __fmaf_rn(l_run, f, __fmul_rn(sum, e.y));
            if constexpr (PT == 8)
                *reinterpret_cast<uint4 *>(sm.p + r * (NT / 2) + 4 * (j ^ (r & 7))) =
                    make_uint4(h2_pack(x[0], x[1]), h2_pack(x[2], x[3]), h2_pack(x[4], x[5]), h2_pack(x[6], x[7]));
            else   // four pieces to a row of 32 tokens
                sm.p[r * (NT / 2) + 4 * ((j >> 2) ^ ((r >> 1) & 3)) + (j & 3)] = h2_pack(x[0], x[1]);
        }
        __syncthreads();   // the weights are there
        {
            // sums of this warp's 16 coordinates over the step's tokens: V^T (16 x 16) times P^T (16 x 8 rows)
            float o[2][4] = {};
#pragma unroll
            for (int ks = 0; ks < NT / 16; ks++) {
                uint32_t av[4];
                const int tok = 16 * ks + 8 * (lane >> 4) + (lane & 7);
                ldsm4t(av, sm.v + tok * 64 + 4 * ((2 * warp + ((lane >> 3) & 1)) ^ (tok & 7)));
                uint32_t bp[4];
                const int r = 8 * (lane >> 4) + (lane & 7), piece = 2 * ks + ((lane >> 3) & 1);
                ldsm4(bp, sm.p + r * (NT / 2) + 4 * (RW == 4 ? piece ^ (r & 7) : piece ^ ((r >> 1) & 3)));
                mma16816(o[0], av, bp[0], bp[1]);
                mma16816(o[1], av, bp[2], bp[3]);
            }
#pragma unroll
            for (int n = 0; n < 2; n++) {
                const float f0 = sm.rescale[8 * n + 2 * t4], f1 = sm.rescale[8 * n + 2 * t4 + 1];
                acc[n][0] = __fmaf_rn(acc[n][0], f0, o[n][0]);
                acc[n][1] = __fmaf_rn(acc[n][1], f1, o[n][1]);
                acc[n][2] = __fmaf_rn(acc[n][2], f0, o[n][2]);
                acc[n][3] = __fmaf_rn(acc[n][3], f1, o[n][3]);
            }
        }
        __syncthreads();   // V, the scores and the weights may be written again
        cur = next;
        next = after;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");

    // ---- the split's partial results
    const int64_t pbase = ((int64_t)split * a.heads + head) * a.row_pad + row0;
#pragma unroll
    for (int n = 0; n < 2; n++) {
        float *o = a.part + (pbase + 8 * n + 2 * t4) * kTile + 16 * warp + g8;
        o[0] = acc[n][0];
        o[kTile] = acc[n][1];
        o[8] = acc[n][2];
        o[kTile + 8] = acc[n][3];
    }
    {
        float l = l_run;
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) l = __fadd_rn(l, __shfl_xor_sync(0xffffffffu, l, o));
        if ((threadIdx.x & 15) == 0) a.ml[pbase + (threadIdx.x >> 4)] = make_float2(__fsub_rn(m_run, kTopBits), l);
    }
    status = __reduce_or_sync(0xffffffffu, status);
    if (lane == 0 && status) atomicOr(&a.stats[which]->status, status);
}

// ------------------------------------------------------------------ many rows
// attention_wide: up to 256 query rows of a KV head in one CTA (draft trees), so that a token is decoded
// once for all of them.  16 warps, one CTA per SM; a step is four chunks (128 tokens), decoded by 8 warps
// for K and 8 for V (two to a chunk, two rounds each) into two shared-memory tiles, [token][128] fp16 in
// panels of 64 coordinates with the 128-byte swizzle.  The products run on tcgen05 with their sums in
// TMEM, a block of 128 rows at a time:
//   S (128 rows x 128 tokens) = Q K^T, Q as two fp16: the upper part from shared memory, the lower
//     part from TMEM, K with the contracted coordinate contiguous;
//   O (128 rows x 128 coordinates) += P V, P in fp16 from TMEM over S's columns, V as it lies (the
//     contracted token in steps of 128 bytes).
// TMEM: O of both blocks (256 columns), S / P (128), Q's lower part (2 x 64): all 512.
// Softmax: a thread holds 32 tokens (one chunk) of one row; four threads share a row and exchange their
// maxima through shared memory.  A row's maximum is moved only when a new one is 2^4 larger, so O is
// hardly ever rescaled; weights stand at 2^11 of the row's largest and reach 2^15 before that.
constexpr int kWideThreads = 512;
constexpr int kWideRows = 256;
constexpr float kLazyMax = 4.0f;

struct WideInfo {
    int64_t t0;
    float ek;
    int n, open;
};
struct WideSmem {
    uint4 qh[2][2048];                          // upper part of Q: [block][panel][row][8 pieces], swizzled
    uint4 k[2048], v[2048];                     // [panel][token][8 pieces], swizzled
    uint32_t stage[kAttnWarps][2][kAttnStage + kStagePad];   // per chunk of a step (4 of K, 4 of V)
    uint32_t seg[16][132];
    uint32_t pairs[1 << kPairBits];
    float qscale[kWideRows];
    int64_t qpos[kWideRows];
    float mx[4][128];
    WideInfo info[4];
    float2 ev[4];                               // vscale of the step's chunks
    uint64_t bar[3];                            // S is there; O is there; all that was issued is done
    uint64_t range[3];
    int64_t span[2];
    uint32_t sign[4];
    uint32_t tmem;
    TopRow top[kTop];
};

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
// The first poll does not wait, each other up to 1 us.
__device__ __forceinline__ bool bar_wait(uint64_t *bar, uint32_t parity, uint32_t polls) {
    const uint32_t a = smem_u32(bar);
    uint32_t done;
    asm volatile("{\n.reg .pred p;\nmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
                 : "=r"(done) : "r"(a), "r"(parity) : "memory");
    if (done) return true;
    for (uint32_t i = 1; i < polls; i++) {
        asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\nselp.u32 %0, 1, 0, p;\n}"
                     : "=r"(done) : "r"(a), "r"(parity), "r"(1000u) : "memory");
        if (done) return true;
    }
    return false;
}
// Shared-memory operand descriptor, 128-byte swizzle: strides in bytes.
__device__ __forceinline__ uint64_t smem_desc(const void *p, uint32_t lead, uint32_t stride) {
    return (uint64_t)((smem_u32(p) & 0x3FFFFu) >> 4) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(stride >> 4) << 32 |
           1ull << 46 | 2ull << 61;
}
// fp16 x fp16 -> fp32, M = N = 128; the second operand with the contracted index contiguous or not.
constexpr uint32_t kIdescK = 1u << 4 | (128u >> 3) << 17 | (128u >> 4) << 24;
constexpr uint32_t kIdescMN = kIdescK | 1u << 16;
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add) : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
                 ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add) : "memory");
}
__device__ __forceinline__ void umma_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t (&r)[32], uint32_t at) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,"
                 "%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                   "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                   "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(at) : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t at, const uint32_t (&r)[32]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
                 "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,"
                 "%29,%30,%31,%32};"
                 ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
                   "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
                   "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
                   "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]) : "memory");
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
                 ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
                   "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]) : "memory");
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

template <int LAT, bool DITHER, int FORM>
__global__ void __launch_bounds__(kWideThreads, 1) attention_wide(const __grid_constant__ AttnArgs a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    // the swizzle counts from 1024-byte lines
    WideSmem &sm = *reinterpret_cast<WideSmem *>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g8 = lane >> 2, t4 = lane & 3;
    const int split = blockIdx.x, head = blockIdx.y, row0 = blockIdx.z * kWideRows;
    const int rows = min(a.rows - row0, kWideRows), nb = rows > 128 ? 2 : 1;
    cudaTriggerProgrammaticLaunchCompletion();   // the combine may come up; it waits for this grid's end

    if (threadIdx.x == 0) {
        query_span(a, row0, rows, sm.span);
        for (int i = 0; i < 3; i++)
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_u32(&sm.bar[i])) : "memory");
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sm.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    const Table<kTop> tab(a.table[0], a.n_appends, a.heads, sm.top);
    tab.load(sm.top);
    build_sign_table(sm.sign, 1, a.seed[0]);
    for (int i = threadIdx.x; i < (1 << kPairBits); i += blockDim.x)
        sm.pairs[i] = pair_entry<LAT == HQ_E8 && FORM == kFormUnary>((uint32_t)i);
    for (int r = threadIdx.x; r < kWideRows; r += blockDim.x) sm.qpos[r] = query_position(a, row0 + r);
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tm = sm.tmem, tmS = tm + 256u, tmQ = tm + 384u;
    const uint32_t lane_base = (uint32_t)(warp & 3) << 21;   // this warp's 32 TMEM lanes (lane in bits 16..)
    visible_range(a, tab, sm.range);
    __syncwarp();

    // ---- queries: upper parts to their tiles, lower parts through the K and V tiles to TMEM
#pragma unroll 4
    for (int r = warp; r < 128 * nb; r += 16) {
        float u[4] = {}, up = 1.0f;
        if (r < rows) load_query(a, head, row0 + r, sm.sign, reinterpret_cast<float *>(sm.seg[warp]), lane, u, up);
        const uint32_t h0 = h2_pack(u[0], u[1]), h1 = h2_pack(u[2], u[3]);
        const __half2 a0 = *reinterpret_cast<const __half2 *>(&h0), a1 = *reinterpret_cast<const __half2 *>(&h1);
        const uint32_t l0 = h2_pack(__fsub_rn(u[0], __low2float(a0)), __fsub_rn(u[1], __high2float(a0)));
        const uint32_t l1 = h2_pack(__fsub_rn(u[2], __low2float(a1)), __fsub_rn(u[3], __high2float(a1)));
        // coordinates 4 lane ..: panel lane / 16, piece (lane mod 16) / 2 of 8 coordinates, half lane & 1
        const int b = r >> 7, rr = r & 127;
        uint2 *qh = reinterpret_cast<uint2 *>(&sm.qh[b][(lane >> 4) * 1024 + rr * 8 + (((lane & 15) >> 1) ^ (rr & 7))]);
        qh[lane & 1] = make_uint2(h0, h1);
        uint2 *ql = reinterpret_cast<uint2 *>(&(b ? sm.v : sm.k)[rr * 16 + ((lane >> 1) ^ (rr & 15))]);
        ql[lane & 1] = make_uint2(l0, l1);
        if (lane == 0) sm.qscale[r] = __fmul_rn(up, a.scale_log2);
    }
    __syncthreads();
    const int row = (warp & 3) * 32 + lane, grp = warp >> 2;   // this thread's row of a block, and its quarter of the tokens
    for (int b = 0; b < nb; b++) {
        uint32_t r[16];
#pragma unroll
        for (int c = 0; c < 4; c++) {
            const uint4 x = (b ? sm.v : sm.k)[row * 16 + ((4 * grp + c) ^ (row & 15))];
            r[4 * c] = x.x; r[4 * c + 1] = x.y; r[4 * c + 2] = x.z; r[4 * c + 3] = x.w;
        }
        tmem_st16(tmQ + 64u * b + 16u * grp + lane_base, r);
    }
    uint64_t ia, ib, ie;
    see_bounds(a, sm.range, ia, ib, ie);
    const uint64_t nvis = ia + (ie - ib), steps = (nvis + 3) / 4;
    const uint64_t st0 = steps * (uint64_t)split / (uint64_t)a.splits;
    const uint64_t st1 = steps * (uint64_t)(split + 1) / (uint64_t)a.splits;
    __syncthreads();   // the lower parts have been read: K and V may be written

    const int which = warp >> 3, ci = (warp & 7) >> 1, r0 = 2 * (warp & 1), chunk_slot = 4 * which + ci;
    Source src;
    src.init(a, which);
    float m_run[2] = {kNegInf, kNegInf}, l_run[2] = {0.0f, 0.0f};
    uint32_t status = 0u;
    bool dead = false;
    int buf = 0;
    uint32_t s_count = 0;   // commits of S so far
    Piece cur = src.piece(a, tab, head, st0 * 4 + ci, st0 < st1, nvis, ia, ib);
    src.stage(cur, sm.stage[chunk_slot][0], threadIdx.x & 63, 64);
    Piece next = src.piece(a, tab, head, (st0 + 1) * 4 + ci, st0 + 1 < st1, nvis, ia, ib);
    for (uint64_t step = st0; step < st1; step++, buf ^= 1) {
        src.stage(next, sm.stage[chunk_slot][buf ^ 1], threadIdx.x & 63, 64);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        // the chunk's words come from both of its warps
        asm volatile("bar.sync %0, 64;" ::"r"(1 + chunk_slot) : "memory");
        const Planes pl = planes_of<LAT, FORM>(src, cur);
        const bool staged = pl.staged;
        const uint32_t *const st = sm.stage[chunk_slot][buf], *const gsrc = src.words + cur.w0;
        uint32_t *const seg = sm.seg[warp];
        bool ok = pl.ok;
        const uint32_t seg0 = 32u * r0, seg1 = seg0 + 64u;
        if (staged)
            ok = scan_segments(st + pl.nc + pl.nr, pl.nu, pl.nsym, seg0, seg1, seg, lane) && ok;
        else
            ok = scan_segments(gsrc + pl.nc + pl.nr, pl.nu, pl.nsym, seg0, seg1, seg, lane) && ok;
        if (which == 0 && r0 == 0 && lane == 0) {
            WideInfo &w = sm.info[ci];
            w.t0 = cur.t0;
            w.n = cur.on ? cur.n : 0;
            w.ek = cur.on ? __fmul_rn(cur.e, kCodeUnit) : 0.0f;
            w.open = all_see(a, cur, sm.span);
        }
        if (which == 1 && r0 == 0 && lane == 0) sm.ev[ci] = cur.on ? vscale(cur.e) : make_float2(0.0f, 1.0f);
        // V's tile is free when the last step's sums are done
        if (which == 1 && step > st0) dead |= !bar_wait(&sm.bar[1], (uint32_t)(step - st0 - 1) & 1u, a.wait_limit);
        uint4 *const tile = which ? sm.v : sm.k;
        bool bad = cur.on && !ok;
#pragma unroll 1
        for (int rr = 0; rr < 2; rr++) {
            const int ti = 8 * (r0 + rr) + g8;
            const bool valid = cur.on && ti < cur.n;
            // token 32 ci + ti: panel t4 / 2, pieces 4 (t4 & 1) ..
            const int tok = 32 * ci + ti;
            uint4 *const dst = tile + (t4 >> 1) * 1024 + tok * 8;
            const unsigned long long e0 = (unsigned long long)(((cur.t0 + ti) * a.heads + head) * kTile);
            // a tile that did not decode counts as zeros, as a read stores it
            const unsigned lost = decode_round<LAT, DITHER, FORM>(
                ok, staged, st, gsrc, pl, src, seg, 32u * (uint32_t)(r0 + rr) + lane, valid, e0, 1.0f / kCodeUnit, sm.pairs,
                [&](int g, const uint32_t (&w)[4]) {
                    dst[(4 * (t4 & 1) + g) ^ (tok & 7)] = make_uint4(w[0], w[1], w[2], w[3]);
                });
            bad |= lost != 0u;
            if ((lost >> (lane & ~3)) & 0xFu) {
#pragma unroll
                for (int g = 0; g < 4; g++) dst[(4 * (t4 & 1) + g) ^ (tok & 7)] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
        if (bad) status |= HQ_ST_CORRUPT;
        // (found here, not before the decode: it would take registers from it)
        const Piece after = src.piece(a, tab, head, (step + 2) * 4 + ci, step + 2 < st1, nvis, ia, ib);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        dead = __syncthreads_or(dead);   // K, V and the chunks' records are there
        if (dead) break;
        auto issue_s = [&](int b) {
#pragma unroll
            for (int ks = 0; ks < 8; ks++) {
                const int at = (ks >> 2) * 1024 + (ks & 3) * 2;
                umma_ss(tmS, smem_desc(&sm.qh[b][at], 16, 1024), smem_desc(&sm.k[at], 16, 1024), kIdescK, ks > 0);
            }
#pragma unroll
            for (int ks = 0; ks < 8; ks++)
                umma_ts(tmS, tmQ + 64u * b + 8u * ks, smem_desc(&sm.k[(ks >> 2) * 1024 + (ks & 3) * 2], 16, 1024), kIdescK, true);
            umma_commit(&sm.bar[0]);
        };
        if (threadIdx.x == 0) {
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            issue_s(0);
        }
        const WideInfo info = sm.info[grp];
        const float2 ev = sm.ev[grp];
        for (int b = 0; b < nb; b++) {
            dead |= !bar_wait(&sm.bar[0], s_count & 1u, a.wait_limit);
            s_count++;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const bool live = 128 * b + (warp & 3) * 32 < rows;   // rows past the last are left out
            const int r = 128 * b + row;
            float x[32], top = kNegInf;
            if (live) {
                uint32_t raw[32];
                tmem_ld32(raw, tmS + 32u * grp + lane_base);
                const float qs = __fmul_rn(sm.qscale[r], info.ek);
#pragma unroll
                for (int i = 0; i < 32; i++) x[i] = __fmaf_rn(__uint_as_float(raw[i]), qs, ev.x);
                if (!info.open) {
                    const int64_t pos = sm.qpos[r];
#pragma unroll
                    for (int i = 0; i < 32; i++) {
                        const int64_t t = info.t0 + i;
                        const bool see = i < info.n && t < a.len && t <= pos &&
                                         (a.window <= 0 || t > pos - a.window || t < a.sinks);
                        if (!see) x[i] = kNegInf;
                    }
                }
#pragma unroll
                for (int i = 0; i < 32; i++) top = fmaxf(top, x[i]);
                sm.mx[grp][row] = top;
            }
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            dead = __syncthreads_or(dead);
            if (dead) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            if (live) {
#pragma unroll
                for (int i = 0; i < 4; i++) top = fmaxf(top, sm.mx[i][row]);
                float m = b ? m_run[1] : m_run[0], l = b ? l_run[1] : l_run[0], f = 1.0f;
                if (top > __fadd_rn(m, kLazyMax) || (m == kNegInf && top != kNegInf)) {
                    f = m == kNegInf ? 0.0f : ex2(__fsub_rn(m, top));
                    m = top;
                }
                if (__any_sync(0xffffffffu, f != 1.0f) && step > st0) {
                    // the sums of the last step are there: its barrier has been passed or is passed here
                    dead |= !bar_wait(&sm.bar[1], (uint32_t)(step - st0 - 1) & 1u, a.wait_limit);
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    uint32_t o[32];
                    tmem_ld32(o, tm + 128u * b + 32u * grp + lane_base);
#pragma unroll
                    for (int i = 0; i < 32; i++) o[i] = __float_as_uint(__fmul_rn(__uint_as_float(o[i]), f));
                    tmem_st32(tm + 128u * b + 32u * grp + lane_base, o);
                }
                const float base = m == kNegInf ? 0.0f : __fsub_rn(m, kTopBits - kLazyMax);
                uint32_t pw[16];
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; i++) {
                    const float p0 = ex2(__fsub_rn(x[2 * i], base)), p1 = ex2(__fsub_rn(x[2 * i + 1], base));
                    sum = __fadd_rn(sum, __fadd_rn(p0, p1));
                    pw[i] = h2_pack(p0, p1);
                }
                l = __fmaf_rn(l, f, __fmul_rn(sum, ev.y));
                m_run[b ? 1 : 0] = m;
                l_run[b ? 1 : 0] = l;
                tmem_st16(tmS + 16u * grp + lane_base, pw);
            }
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            dead = __syncthreads_or(dead);
            if (dead) break;
            if (threadIdx.x == 0) {
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
                for (int ks = 0; ks < 8; ks++)
                    umma_ts(tm + 128u * b, tmS + 8u * ks, smem_desc(&sm.v[ks * 128], 16384, 1024), kIdescMN,
                            step > st0 || ks > 0);
                if (b + 1 < nb)
                    issue_s(b + 1);   // after the product above has read the weights in its place
                else
                    umma_commit(&sm.bar[1]);
            }
        }
        if (dead) break;   // the same in all threads: the barriers above
        cur = next;
        next = after;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (st0 < st1 && !dead) dead = !bar_wait(&sm.bar[1], (uint32_t)(st1 - st0 - 1) & 1u, a.wait_limit);
    dead = __syncthreads_or(dead);
    if (dead) {
        // given up: products that are still in flight read this CTA's shared memory and write its TMEM (the wait
        // for them is never the lowered one)
        if (threadIdx.x == 0) {
            umma_commit(&sm.bar[2]);
            bar_wait(&sm.bar[2], 0u, kAttnWaitPolls);
        }
        __syncthreads();
    }
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");

    // ---- the split's partial results
    for (int b = 0; b < nb; b++) {
        const bool live = 128 * b + (warp & 3) * 32 < rows;
        const int64_t at = ((int64_t)split * a.heads + head) * a.row_pad + row0 + 128 * b + row;
        if (live) {
            uint32_t o[32] = {};
            if (st0 < st1 && !dead) tmem_ld32(o, tm + 128u * b + 32u * grp + lane_base);
            float4 *dst = reinterpret_cast<float4 *>(a.part + at * kTile + 32 * grp);
#pragma unroll
            for (int i = 0; i < 8; i++)
                dst[i] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]), __uint_as_float(o[4 * i + 2]),
                                     __uint_as_float(o[4 * i + 3]));
            sm.mx[grp][row] = b ? l_run[1] : l_run[0];
        }
        __syncthreads();
        if (live && grp == 0)
            a.ml[at] = make_float2(__fsub_rn(b ? m_run[1] : m_run[0], kTopBits - kLazyMax),
                                   __fadd_rn(__fadd_rn(sm.mx[0][row], sm.mx[1][row]), __fadd_rn(sm.mx[2][row], sm.mx[3][row])));
        __syncthreads();
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (warp == 0) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tm) : "memory");
    }
    if (dead) status |= HQ_ST_TIMEOUT;
    status = __reduce_or_sync(0xffffffffu, status);
    if (lane == 0 && status) atomicOr(&a.stats[which]->status, status);
}

template <int LAT, bool DITHER, int FORM, int RW>
cudaError_t launch_rw(const AttnArgs &a, cudaStream_t s) {
    auto kern = attention_kernel<LAT, DITHER, FORM, RW>;
    static LaunchPlan plan;
    const size_t smem = sizeof(AttnSmem<RW>);
    unsigned grid = 0;
    cudaError_t e = plan.grid(kern, kAttnWarps * 32, smem, 1, grid);
    if (e != cudaSuccess) return e;
    const dim3 g((unsigned)a.splits, (unsigned)a.heads, (unsigned)(a.row_pad / 16));
    kern<<<g, kAttnWarps * 32, smem, s>>>(a);
    return cudaGetLastError();
}

template <int LAT, bool DITHER, int FORM>
cudaError_t launch_wide(const AttnArgs &a, cudaStream_t s) {
    auto kern = attention_wide<LAT, DITHER, FORM>;
    static LaunchPlan plan;
    const size_t smem = sizeof(WideSmem) + 1024;   // room to align
    unsigned grid = 0;
    cudaError_t e = plan.grid(kern, kWideThreads, smem, 1, grid);
    if (e != cudaSuccess) return e;
    const dim3 g((unsigned)a.splits, (unsigned)a.heads, (unsigned)((a.rows + kWideRows - 1) / kWideRows));
    kern<<<g, kWideThreads, smem, s>>>(a);
    return cudaGetLastError();
}

template <int LAT, bool DITHER, int FORM>
cudaError_t launch_form(const AttnArgs &a, cudaStream_t s) {
    if (a.rows > kNarrowRows) return launch_wide<LAT, DITHER, FORM>(a, s);
    return a.short_steps ? launch_rw<LAT, DITHER, FORM, 1>(a, s) : launch_rw<LAT, DITHER, FORM, 4>(a, s);
}

template <int LAT, bool DITHER>
cudaError_t launch_lat(const AttnArgs &a, cudaStream_t s) {
    if (a.k[0] == 0 && a.k[1] == 0 && a.k_last[0] == 0 && a.k_last[1] == 0) return launch_form<LAT, DITHER, kFormUnary>(a, s);
    return launch_form<LAT, DITHER, kFormGeneral>(a, s);
}

}  // namespace

}  // namespace hq
