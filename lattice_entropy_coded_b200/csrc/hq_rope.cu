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
// its token's 4 angles and walks over heads, so the sines cost one evaluation per token and
// lane; short calls spread a token's heads over more half-warps instead.
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

// The lane's 8 elements: 4 pairs (a, b), pair u at coordinates pa(u), pb(u), and the index of its
// angle (pairs past rot_dim / 2 do not turn).  VEC: the a's and the b's are each one aligned run of
// four, or (interleaved) the pairs one run of eight; otherwise (rot_dim % 8 != 0) single elements.
template <bool VEC>
struct PairMap {
    int oa, ob;   // VEC: first coordinates of the two runs of four
    int pair0;    // VEC: index of the lane's first pair
    __device__ __forceinline__ void init(const RopeArgs &a, int j) {
        const int half = a.rot >> 1;
        pair0 = 4 * j;
        if (a.interleaved) {
            oa = 8 * j;
            ob = 8 * j + 4;
        } else if (4 * j < half) {
            oa = 4 * j;
            ob = half + 4 * j;
        } else {
            oa = a.rot + 8 * (j - half / 4);
            ob = oa + 4;
        }
    }
    __device__ __forceinline__ static int pair(int j, int u) { return VEC ? 4 * j + u : j + 16 * u; }
    __device__ __forceinline__ static int pa(const RopeArgs &a, int p) {
        const int half = a.rot >> 1;
        return a.interleaved ? 2 * p : p < half ? p : 2 * p;
    }
    __device__ __forceinline__ static int pb(const RopeArgs &a, int p) {
        const int half = a.rot >> 1;
        return a.interleaved ? 2 * p + 1 : p < half ? p + half : 2 * p + 1;
    }
};

template <bool VEC>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_kernel(const __grid_constant__ RopeArgs a) {
    const int j = threadIdx.x & 15;
    const int64_t unit = ((int64_t)blockIdx.x * kRopeThreads + threadIdx.x) >> 4;
    int64_t tok;
    int part;
    if (a.splits == 1) {
        tok = unit;
        part = 0;
    } else {
        tok = unit / a.splits;
        part = (int)(unit - tok * a.splits);
    }
    // both half-warps of a warp take part in the shuffles; one past the end does nothing else
    const bool live = tok < a.tokens;
    PairMap<VEC> map;
    map.init(a, j);
    float c[4], s[4];
    const double pos = live ? (double)(a.pos ? a.pos[tok] : a.pos0 + tok) : 0.0;
#pragma unroll
    for (int u = 0; u < 4; u++) {
        const int p = PairMap<VEC>::pair(j, u);
        c[u] = 1.0f;
        s[u] = 0.0f;
        if (2 * p < a.rot) {
            const double turns = pos * a.inv_freq[p] * 0.15915494309189533577;   // 1 / (2 pi)
            sincospif((float)(2.0 * (turns - rint(turns))), &s[u], &c[u]);
        }
    }
    const int hall = a.side[0].heads + a.side[1].heads;
    const int h0 = part * a.per_split, h1 = min(hall, h0 + a.per_split);
    for (int h = h0; h < h0 + a.per_split; h += kRopeUnroll) {
        float va[kRopeUnroll][4], vb[kRopeUnroll][4];
#pragma unroll
        for (int n = 0; n < kRopeUnroll; n++) {
            const bool on = live && h + n < h1;
            const int which = h + n < a.side[0].heads ? 0 : 1;
            const RopeSide &sd = a.side[which];
            const int hh = h + n - (which ? a.side[0].heads : 0);
            const uint16_t *x = sd.x + tok * sd.ld_tok + (int64_t)hh * sd.ld_head;
            if (VEC) {
                uint2 ra = make_uint2(0u, 0u), rb = ra;
                if (on) {
                    ra = *reinterpret_cast<const uint2 *>(x + map.oa);
                    rb = *reinterpret_cast<const uint2 *>(x + map.ob);
                }
                const float f[8] = {bf_lo(ra.x), bf_hi(ra.x), bf_lo(ra.y), bf_hi(ra.y),
                                    bf_lo(rb.x), bf_hi(rb.x), bf_lo(rb.y), bf_hi(rb.y)};
#pragma unroll
                for (int u = 0; u < 4; u++) {
                    va[n][u] = a.interleaved ? f[2 * u] : f[u];
                    vb[n][u] = a.interleaved ? f[2 * u + 1] : f[4 + u];
                }
            } else {
#pragma unroll
                for (int u = 0; u < 4; u++) {
                    const int p = PairMap<VEC>::pair(j, u);
                    va[n][u] = on ? __uint_as_float((uint32_t)x[PairMap<VEC>::pa(a, p)] << 16) : 0.0f;
                    vb[n][u] = on ? __uint_as_float((uint32_t)x[PairMap<VEC>::pb(a, p)] << 16) : 0.0f;
                }
            }
        }
        if (a.norm) {
            float ss[kRopeUnroll];
#pragma unroll
            for (int n = 0; n < kRopeUnroll; n++) {
                ss[n] = 0.0f;
#pragma unroll
                for (int u = 0; u < 4; u++) ss[n] = __fmaf_rn(vb[n][u], vb[n][u], __fmaf_rn(va[n][u], va[n][u], ss[n]));
            }
#pragma unroll
            for (int m = 1; m <= 8; m <<= 1)
#pragma unroll
                for (int n = 0; n < kRopeUnroll; n++)
                    ss[n] = __fadd_rn(ss[n], __shfl_xor_sync(0xffffffffu, ss[n], m));
#pragma unroll
            for (int n = 0; n < kRopeUnroll; n++) {
                const float r = rsqrtf(__fmaf_rn(ss[n], 1.0f / 128.0f, a.eps));
                const uint16_t *w = a.side[h + n < a.side[0].heads ? 0 : 1].w;
#pragma unroll
                for (int u = 0; u < 4; u++) {
                    const int p = PairMap<VEC>::pair(j, u);
                    const int ia = VEC ? (a.interleaved ? map.oa + 2 * u : map.oa + u) : PairMap<VEC>::pa(a, p);
                    const int ib = VEC ? (a.interleaved ? map.oa + 2 * u + 1 : map.ob + u) : PairMap<VEC>::pb(a, p);
                    va[n][u] = __fmul_rn(va[n][u], r);
                    vb[n][u] = __fmul_rn(vb[n][u], r);
                    if (w) {
                        va[n][u] = __fmul_rn(va[n][u], __uint_as_float((uint32_t)__ldg(w + ia) << 16));
                        vb[n][u] = __fmul_rn(vb[n][u], __uint_as_float((uint32_t)__ldg(w + ib) << 16));
                    }
                }
            }
        }
#pragma unroll
        for (int n = 0; n < kRopeUnroll; n++) {
            if (!(live && h + n < h1)) continue;
            const int which = h + n < a.side[0].heads ? 0 : 1;
            const RopeSide &sd = a.side[which];
            const int hh = h + n - (which ? a.side[0].heads : 0);
            uint16_t *y = sd.y + tok * sd.out_tok + (int64_t)hh * sd.out_head;
            float ya[4], yb[4];
#pragma unroll
            for (int u = 0; u < 4; u++) {
                ya[u] = __fmaf_rn(va[n][u], c[u], -__fmul_rn(vb[n][u], s[u]));
                yb[u] = __fmaf_rn(vb[n][u], c[u], __fmul_rn(va[n][u], s[u]));
            }
            if (VEC) {
                uint2 ra, rb;
                if (a.interleaved) {
                    ra = make_uint2(bf_pack(ya[0], yb[0]), bf_pack(ya[1], yb[1]));
                    rb = make_uint2(bf_pack(ya[2], yb[2]), bf_pack(ya[3], yb[3]));
                } else {
                    ra = make_uint2(bf_pack(ya[0], ya[1]), bf_pack(ya[2], ya[3]));
                    rb = make_uint2(bf_pack(yb[0], yb[1]), bf_pack(yb[2], yb[3]));
                }
                *reinterpret_cast<uint2 *>(y + map.oa) = ra;
                *reinterpret_cast<uint2 *>(y + map.ob) = rb;
            } else {
#pragma unroll
                for (int u = 0; u < 4; u++) {
                    const int p = PairMap<VEC>::pair(j, u);
                    y[PairMap<VEC>::pa(a, p)] = (uint16_t)bf_pack(ya[u], 0.0f);
                    y[PairMap<VEC>::pb(a, p)] = (uint16_t)bf_pack(yb[u], 0.0f);
                }
            }
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
    // two vectors never share their output
    if ((tokens > 1 && out_tok < kTile) || (heads > 1 && out_head < kTile)) return HQ_EINVAL;
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
    // a token's heads over as many half-warps as keep the GPU's (148 SMs x 2048 threads) busy, one to
    // kRopeUnroll heads each at the least
    const int heads = heads_q + heads_k;
    const int64_t want = (INT64_C(148) * 128) / tokens;
    int64_t splits = want < 1 ? 1 : want;
    if (splits > heads) splits = heads;
    a.per_split = (int)((heads + splits - 1) / splits);
    a.splits = (heads + a.per_split - 1) / a.per_split;
    const int64_t units = tokens * a.splits, per_cta = kRopeThreads / 16;
    const int64_t grid = (units + per_cta - 1) / per_cta;
    cudaStream_t s = (cudaStream_t)cuda_stream;
    if (a.rot % 8 == 0)
        norm_rope_kernel<true><<<(unsigned)grid, kRopeThreads, 0, s>>>(a);
    else
        norm_rope_kernel<false><<<(unsigned)grid, kRopeThreads, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? HQ_OK : HQ_ECUDA;
}
