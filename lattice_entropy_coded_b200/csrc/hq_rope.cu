// hq_rope.cu -- hq_qk_norm_rope: the RMS norm of every query and key head vector and
// its position rotation in one pass, from a projection's output to the layouts that
// hq_kv_append (keys) and hq_kv_attention (queries) take.
//
// One head vector x of 128 (bf16): y = x / sqrt(mean x^2 + eps) * w, then pairs (a, b) of
// the first rot_dim coordinates turn by pos * inv_freq[i]: (a cos - b sin, b cos + a sin).
// All in fp32, rounded to bf16 once.  The angle is reduced to a fraction of a turn in
// double (pos * inv_freq reaches 10^6 radians, where fp32 holds 2^-4 of a radian), so that
// far positions turn as exactly as near ones.
//
// The pass is bound by its bytes (2 read, 2 written per element, 6 operations): half a
// warp holds a head vector, 8 elements to a lane in two 8-byte pieces that are both ends of
// 4 pairs, so the rotation needs no exchange and the norm four shuffles.  A half-warp keeps
// its token's 4 angles and the side's 8 weights and walks over heads, so the sines cost one
// evaluation per token and lane; short calls spread a token's heads over more half-warps instead.
// 8191 tokens of 32 + 8 heads: 35 us, 4.8 TB/s (74 % of a copy).  Four CTAs to an SM at 64 registers (by events on
// a cold L2: three 51 us, four 47, five 62); 8 pairs to a lane instead of 4 60 us, the next heads' loads ahead of
// this one's arithmetic 47 to 68 us, the fast sines no difference.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "hq_device.cuh"

namespace hq {

namespace {

struct RopeSide {
    const uint16_t *x;
    uint16_t *y;
    const uint16_t *w;
    int64_t ld_tok, ld_head, out_tok, out_head;
    int heads;
};

struct RopeArgs {
    RopeSide side[2];
    const double *inv_freq;
    const int64_t *pos;
    int64_t pos0, tokens;
    int rot, interleaved, norm, splits, per_split;
    float eps;
};

constexpr int kRopeThreads = 256;
constexpr int kRopeUnroll = 4;   // head vectors whose loads are in flight at once

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t bf_pack(float a, float b) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&h);
}

// The lane's 8 elements are 4 pairs (a, b).  kHalves, kPairs (rot_dim % 8 == 0): the a's and the b's
// are each an aligned run of four, or the pairs one run of eight; the pairs that do not turn are such
// runs too.  kSingles: any other rot_dim, element by element.
enum RopeForm { kHalves = 0, kPairs = 1, kSingles = 2 };

template <int FORM>
__device__ __forceinline__ int pair_of(int j, int u) { return FORM == kSingles ? j + 16 * u : 4 * j + u; }

struct Lane8 {
    float2 a[2], b[2];   // pairs 0..3: (a0, a1), (a2, a3) and the b's
};
template <int FORM>
struct LaneMap {
    int oa, ob;       // first coordinates of the two runs of four
    int ca[4], cb[4]; // kSingles: the coordinates
    __device__ __forceinline__ void init(const RopeArgs &a, int j) {
        const int half = a.rot >> 1;
        if (FORM == kPairs) {
            oa = 8 * j;
            ob = 8 * j + 4;
        } else if (4 * j < half) {
            oa = 4 * j;
            ob = half + 4 * j;
        } else {
            oa = a.rot + 8 * (j - half / 4);
            ob = oa + 4;
        }
        if (FORM == kSingles) {
#pragma unroll
            for (int u = 0; u < 4; u++) {
                const int p = pair_of<FORM>(j, u);
                const bool halves = !a.interleaved && p < half;
                ca[u] = halves ? p : 2 * p;
                cb[u] = halves ? p + half : 2 * p + 1;
            }
        }
    }
    __device__ __forceinline__ Lane8 load(const uint16_t *x) const {
        Lane8 r;
        if (FORM == kSingles) {
            float f[8];
#pragma unroll
            for (int u = 0; u < 4; u++) {
                f[u] = __uint_as_float((uint32_t)x[ca[u]] << 16);
                f[4 + u] = __uint_as_float((uint32_t)x[cb[u]] << 16);
            }
            r.a[0] = make_float2(f[0], f[1]);
            r.a[1] = make_float2(f[2], f[3]);
            r.b[0] = make_float2(f[4], f[5]);
            r.b[1] = make_float2(f[6], f[7]);
            return r;
        }
        const uint2 p = *reinterpret_cast<const uint2 *>(x + oa), q = *reinterpret_cast<const uint2 *>(x + ob);
        if (FORM == kPairs) {
            r.a[0] = make_float2(bf_lo(p.x), bf_lo(p.y));
            r.b[0] = make_float2(bf_hi(p.x), bf_hi(p.y));
            r.a[1] = make_float2(bf_lo(q.x), bf_lo(q.y));
            r.b[1] = make_float2(bf_hi(q.x), bf_hi(q.y));
        } else {
            r.a[0] = make_float2(bf_lo(p.x), bf_hi(p.x));
            r.a[1] = make_float2(bf_lo(p.y), bf_hi(p.y));
            r.b[0] = make_float2(bf_lo(q.x), bf_hi(q.x));
            r.b[1] = make_float2(bf_lo(q.y), bf_hi(q.y));
        }
        return r;
    }
    __device__ __forceinline__ void store(uint16_t *y, const Lane8 &r) const {
        if (FORM == kSingles) {
            const float f[8] = {r.a[0].x, r.a[0].y, r.a[1].x, r.a[1].y, r.b[0].x, r.b[0].y, r.b[1].x, r.b[1].y};
#pragma unroll
            for (int u = 0; u < 4; u++) {
                y[ca[u]] = (uint16_t)bf_pack(f[u], 0.0f);
                y[cb[u]] = (uint16_t)bf_pack(f[4 + u], 0.0f);
            }
        } else if (FORM == kPairs) {
            *reinterpret_cast<uint2 *>(y + oa) = make_uint2(bf_pack(r.a[0].x, r.b[0].x), bf_pack(r.a[0].y, r.b[0].y));
            *reinterpret_cast<uint2 *>(y + ob) = make_uint2(bf_pack(r.a[1].x, r.b[1].x), bf_pack(r.a[1].y, r.b[1].y));
        } else {
            *reinterpret_cast<uint2 *>(y + oa) = make_uint2(bf_pack(r.a[0].x, r.a[0].y), bf_pack(r.a[1].x, r.a[1].y));
            *reinterpret_cast<uint2 *>(y + ob) = make_uint2(bf_pack(r.b[0].x, r.b[0].y), bf_pack(r.b[1].x, r.b[1].y));
        }
    }
};

// Pairs turned in place.  A pair that does not turn is to pass as it is, but a 1 - b 0 is NaN beside an infinity:
// without PLAIN it is left out (bit u of `still`: pair u of the lane).  (8191 tokens with the norm: 33.0 us if
// nothing is left out, 33.5 with the two forms and a branch, 34.2 to 34.9 with a choice for every pair.)
template <int FORM, bool PLAIN>
__device__ __forceinline__ void turn(Lane8 (&v)[kRopeUnroll], const float2 (&c)[2], const float2 (&s)[2], uint32_t still) {
#pragma unroll
    for (int n = 0; n < kRopeUnroll; n++)
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const float2 a = v[n].a[i], b = v[n].b[i], bs = f2_mul(b, s[i]), as = f2_mul(a, s[i]);
            v[n].a[i] = f2_fma(a, c[i], make_float2(-bs.x, -bs.y));
            v[n].b[i] = f2_fma(b, c[i], as);
            if (!PLAIN) {
                if (still >> (2 * i) & 1u) v[n].a[i].x = a.x, v[n].b[i].x = b.x;
                if (still >> (2 * i + 1) & 1u) v[n].a[i].y = a.y, v[n].b[i].y = b.y;
            }
        }
}

template <int FORM>
__global__ void __launch_bounds__(kRopeThreads, FORM == kSingles ? 2 : 4) norm_rope_kernel(const __grid_constant__ RopeArgs a) {
    const int j = threadIdx.x & 15;
    const unsigned mine = 0xFFFFu << (threadIdx.x & 16);   // the half-warp: its two may walk different heads
    const int64_t unit = ((int64_t)blockIdx.x * kRopeThreads + threadIdx.x) >> 4;
    const int64_t tok = a.splits == 1 ? unit : unit / a.splits;
    const int part = a.splits == 1 ? 0 : (int)(unit - tok * a.splits);
    if (tok >= a.tokens) return;
    LaneMap<FORM> map;
    map.init(a, j);
    float2 c[2], s[2];
    uint32_t still = 0;   // the lane's pairs that do not turn
    {
        const double pos = (double)(a.pos ? a.pos[tok] : a.pos0 + tok);
        float cc[4], ss[4];
#pragma unroll
        for (int u = 0; u < 4; u++) {
            const int p = pair_of<FORM>(j, u);
            cc[u] = 1.0f;
            ss[u] = 0.0f;
            if (2 * p >= a.rot) still |= 1u << u;
            if (2 * p < a.rot) {
                const double t = pos * a.inv_freq[p] * 0.15915494309189533577;   // of a turn: 1 / (2 pi)
                sincospif((float)(2.0 * (t - rint(t))), &ss[u], &cc[u]);
            }
        }
        c[0] = make_float2(cc[0], cc[1]);
        c[1] = make_float2(cc[2], cc[3]);
        s[0] = make_float2(ss[0], ss[1]);
        s[1] = make_float2(ss[2], ss[3]);
    }
    const int all = a.side[0].heads + a.side[1].heads;
    const int h0 = part * a.per_split, h1 = min(all, h0 + a.per_split);
#pragma unroll 1
    for (int which = 0; which < 2; which++) {
        const RopeSide &sd = a.side[which];
        const int first = which ? a.side[0].heads : 0;
        const int lo = max(h0 - first, 0), hi = min(h1 - first, sd.heads);
        if (lo >= hi) continue;
        const uint16_t *x = sd.x + tok * sd.ld_tok;
        uint16_t *y = sd.y + tok * sd.out_tok;
        Lane8 w;
        const float2 one = make_float2(1.0f, 1.0f);
        w.a[0] = w.a[1] = w.b[0] = w.b[1] = one;
        if (a.norm && sd.w) w = map.load(sd.w);
        for (int h = lo; h < hi; h += kRopeUnroll) {
            Lane8 v[kRopeUnroll];
#pragma unroll
            for (int n = 0; n < kRopeUnroll; n++)   // past the last: the last again, not stored
                v[n] = map.load(x + (int64_t)min(h + n, hi - 1) * sd.ld_head);
            bool plain = false;   // nothing but finite numbers, as the sums of squares tell (weights are finite)
            if (a.norm) {
                float ss[kRopeUnroll];
#pragma unroll
                for (int n = 0; n < kRopeUnroll; n++) {
                    float2 q = f2_mul(v[n].a[0], v[n].a[0]);
                    q = f2_fma(v[n].a[1], v[n].a[1], q);
                    q = f2_fma(v[n].b[0], v[n].b[0], q);
                    q = f2_fma(v[n].b[1], v[n].b[1], q);
                    ss[n] = __fadd_rn(q.x, q.y);
                }
#pragma unroll
                for (int m = 1; m <= 8; m <<= 1)
#pragma unroll
                    for (int n = 0; n < kRopeUnroll; n++) ss[n] = __fadd_rn(ss[n], __shfl_xor_sync(mine, ss[n], m));
                plain = __fadd_rn(__fadd_rn(ss[0], ss[1]), __fadd_rn(ss[2], ss[3])) <= 3.4028235e38f;
#pragma unroll
                for (int n = 0; n < kRopeUnroll; n++) {
                    const float r = rsqrtf(__fmaf_rn(ss[n], 1.0f / 128.0f, a.eps));
                    const float2 r2 = make_float2(r, r);
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        v[n].a[i] = f2_mul(f2_mul(v[n].a[i], r2), w.a[i]);
                        v[n].b[i] = f2_mul(f2_mul(v[n].b[i], r2), w.b[i]);
                    }
                }
            }
            if (plain)
                turn<FORM, true>(v, c, s, still);
            else
                turn<FORM, false>(v, c, s, still);
#pragma unroll
            for (int n = 0; n < kRopeUnroll; n++)
                if (h + n < hi) map.store(y + (int64_t)(h + n) * sd.out_head, v[n]);
        }
    }
}

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

// One side's pointers and strides: HQ_OK, or HQ_EINVAL.
int check_side(const void *x, int64_t ld_tok, int64_t ld_head, const void *w, void *y, int64_t out_tok,
               int64_t out_head, int heads, int64_t tokens) {
    if (heads == 0) return HQ_OK;
    if (!x || !y || !aligned(x, 16) || !aligned(y, 16) || !aligned(w, 16)) return HQ_EINVAL;
    if (ld_tok < 0 || ld_tok % 8 || ld_head < 0 || ld_head % 8) return HQ_EINVAL;
    if (out_tok < 0 || out_tok % 8 || out_head < 0 || out_head % 8) return HQ_EINVAL;
    if (!vectors_apart(tokens, out_tok, heads, out_head)) return HQ_EINVAL;
    // in place only vector by vector: under other strides one half-warp would write what another has yet to read
    if (x == y && ((tokens > 1 && ld_tok != out_tok) || (heads > 1 && ld_head != out_head))) return HQ_EINVAL;
    return HQ_OK;
}

}  // namespace

}  // namespace hq

extern "C" int hq_qk_norm_rope(const void *q, int64_t q_ld_token, int64_t q_ld_head, int32_t heads_q, const void *k,
                               int64_t k_ld_token, int64_t k_ld_head, int32_t heads_k, int64_t tokens,
                               const hq_rope_spec *spec, const void *d_wq, const void *d_wk,
                               const double *d_inv_freq, const int64_t *d_pos, int64_t pos0, void *q_out,
                               int64_t qo_ld_token, int64_t qo_ld_head, void *k_out, int64_t ko_ld_token,
                               int64_t ko_ld_head, void *cuda_stream) {
    using namespace hq;
    if (!spec || tokens < 0 || heads_q < 0 || heads_k < 0) return HQ_EINVAL;
    if (spec->rot_dim < 0 || spec->rot_dim > kTile || spec->rot_dim % 2) return HQ_EINVAL;
    if (spec->interleaved != 0 && spec->interleaved != 1) return HQ_EINVAL;
    if (spec->norm != 0 && spec->norm != 1) return HQ_EINVAL;
    if (!(spec->eps >= 0.0f) || !isfinite(spec->eps)) return HQ_EINVAL;
    if (heads_q > 65536 || heads_k > 65536 || tokens > (INT64_C(1) << 31)) return HQ_EUNSUPPORTED;
    if (tokens == 0 || heads_q + heads_k == 0) return HQ_OK;
    int rc = check_side(q, q_ld_token, q_ld_head, d_wq, q_out, qo_ld_token, qo_ld_head, heads_q, tokens);
    if (rc) return rc;
    if ((rc = check_side(k, k_ld_token, k_ld_head, d_wk, k_out, ko_ld_token, ko_ld_head, heads_k, tokens)))
        return rc;
    if (spec->rot_dim && (!d_inv_freq || !aligned(d_inv_freq, 8))) return HQ_EINVAL;
    if (d_pos && !aligned(d_pos, 8)) return HQ_EINVAL;
    RopeArgs a;
    a.side[0] = {(const uint16_t *)q, (uint16_t *)q_out, (const uint16_t *)d_wq, q_ld_token, q_ld_head, qo_ld_token,
                 qo_ld_head, heads_q};
    a.side[1] = {(const uint16_t *)k, (uint16_t *)k_out, (const uint16_t *)d_wk, k_ld_token, k_ld_head, ko_ld_token,
                 ko_ld_head, heads_k};
    a.inv_freq = d_inv_freq;
    a.pos = d_pos;
    a.pos0 = pos0;
    a.tokens = tokens;
    a.rot = spec->rot_dim;
    a.interleaved = spec->interleaved;
    a.norm = spec->norm;
    a.eps = spec->eps;
    // a token's heads over as many half-warps as the GPU holds (148 SMs x 4 CTAs x 256 threads), one head each
    // at the least: every half-warp starts with its token's position and sines, so no more (8191 tokens, cold
    // L2: 47 us with twice as many, 39 so)
    const int heads = heads_q + heads_k;
    const int64_t want = (INT64_C(148) * 64) / tokens;
    int64_t splits = want < 1 ? 1 : want;
    if (splits > heads) splits = heads;
    a.per_split = (int)((heads + splits - 1) / splits);
    a.splits = (heads + a.per_split - 1) / a.per_split;
    const int64_t units = tokens * a.splits, per_cta = kRopeThreads / 16;
    const int64_t grid = (units + per_cta - 1) / per_cta;
    cudaStream_t s = (cudaStream_t)cuda_stream;
    if (a.rot % 8 != 0)
        norm_rope_kernel<kSingles><<<(unsigned)grid, kRopeThreads, 0, s>>>(a);
    else if (a.interleaved)
        norm_rope_kernel<kPairs><<<(unsigned)grid, kRopeThreads, 0, s>>>(a);
    else
        norm_rope_kernel<kHalves><<<(unsigned)grid, kRopeThreads, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? HQ_OK : HQ_ECUDA;
}
