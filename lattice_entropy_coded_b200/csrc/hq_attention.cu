// hq_attention.cu -- the entry points of attention over compressed KV caches, their argument
// checks, and the kernel that joins the splits' partial results (hq_attention.cuh).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "hq_attention.cuh"

namespace hq {

namespace {

constexpr int kCombineWarps = 8;
// Rows of all heads up to which a CTA's warps share one row (32 rows: 16 us with a warp each, 6 so; 2048 rows, a
// whole call: 325 and 339 us).
constexpr int kCombineSpread = 512;

// A query row: the splits' sums rescaled to a common maximum and added, turned back (D H_128, or Q^T),
// the visible drafts added, divided by the sum of all weights.  Bound by the latency of its loads (a few
// MB from L2): every warp asks for eight splits at a time, and with few rows (W = 8) the eight warps of
// a CTA share one row, else (W = 1) each has its own.
template <int W>
__global__ void __launch_bounds__(kCombineWarps * 32) attention_combine(const __grid_constant__ AttnArgs a) {
    constexpr int RPC = kCombineWarps / W;   // rows of a CTA
    __shared__ uint32_t sign[4];
    __shared__ float4 xs[kCombineWarps][32];
    __shared__ float ls[kCombineWarps];
    __shared__ float ps[RPC][kAttnMaxQueries];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % W;
    build_sign_table(sign, 1, a.seed[1]);
    const int row = blockIdx.x * RPC + warp / W, head = blockIdx.y;
    const bool on = row < a.rows;
    const int qi = on ? row / a.group : 0, qh = head * a.group + row - qi * a.group;
    const int64_t d_head = head * a.d_ld_head + 4 * lane;

    // drafts that the row sees (one later than the query, or outside its window, is not visible whatever
    // the mask says), and their log2 weights
    unsigned long long mine = 0;
    if (a.mask && on) {
        const unsigned long long all = a.n_q < 64 ? (1ull << a.n_q) - 1ull : ~0ull, given = a.mask[qi] & all;
        const int64_t pos = a.len - 1 + __popcll(given);
        unsigned half[2];
#pragma unroll
        for (int u = 0; u < 2; u++) {
            const int j = lane + 32 * u;
            bool see = ((given >> j) & 1ull) != 0ull;
            if (see) {
                const int64_t t = a.len - 1 + __popcll(a.mask[j] & all);
                see = t <= pos && (a.window <= 0 || t > pos - a.window || t < a.sinks);
            }
            half[u] = __ballot_sync(0xffffffffu, see);
        }
        mine = (unsigned long long)half[1] << 32 | half[0];
        const uint2 qr = *reinterpret_cast<const uint2 *>(a.q + qi * a.q_ld_tok + qh * a.q_ld_head + 4 * lane);
        const float q[4] = {__uint_as_float(qr.x << 16), __uint_as_float(qr.x & 0xFFFF0000u),
                            __uint_as_float(qr.y << 16), __uint_as_float(qr.y & 0xFFFF0000u)};
        // four at a time; the warps of a row take turns
        int turn = 0;
        for (unsigned long long left = mine; left; turn++) {
            int j[4];
            uint2 kr[4];
            float s[4];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                j[i] = left ? __ffsll((long long)left) - 1 : -1;
                left &= left - 1;
            }
            if (turn % W != part) continue;
#pragma unroll
            for (int i = 0; i < 4; i++)
                kr[i] = j[i] >= 0 ? *reinterpret_cast<const uint2 *>(a.kd + j[i] * a.d_ld_tok + d_head) : make_uint2(0u, 0u);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                s[i] = __fmul_rn(q[0], __uint_as_float(kr[i].x << 16));
                s[i] = __fmaf_rn(q[1], __uint_as_float(kr[i].x & 0xFFFF0000u), s[i]);
                s[i] = __fmaf_rn(q[2], __uint_as_float(kr[i].y << 16), s[i]);
                s[i] = __fmaf_rn(q[3], __uint_as_float(kr[i].y & 0xFFFF0000u), s[i]);
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1)
#pragma unroll
                for (int i = 0; i < 4; i++) s[i] = __fadd_rn(s[i], __shfl_xor_sync(0xffffffffu, s[i], o));
#pragma unroll
            for (int i = 0; i < 4; i++)
                if (lane == 0 && j[i] >= 0) ps[warp / W][j[i]] = __fmul_rn(s[i], a.scale_log2);
        }
    }
    // what the splits left
    cudaGridDependencySynchronize();
    const int64_t step = (int64_t)a.heads * a.row_pad, at = (int64_t)head * a.row_pad + row;
    float m = kNegInf;
    if (on)
        for (int sp = lane; sp < a.splits; sp += 32) m = fmaxf(m, a.ml[sp * step + at].x);
    __syncthreads();   // the drafts' weights and the signs are there
    if (mine)
        for (int j = lane; j < a.n_q; j += 32)
            if ((mine >> j) & 1ull) m = fmaxf(m, ps[warp / W][j]);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float base = m == kNegInf ? 0.0f : m;
    float l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (on) {
        // this warp's splits part, part + W, ...: weights by lane, then their sums
        for (int s0 = 0; s0 < a.splits; s0 += 32 * W) {
            const int sp = s0 + lane * W + part;
            float f = 0.0f;
            if (sp < a.splits) {
                const float2 ml = a.ml[sp * step + at];
                f = ml.y == 0.0f ? 0.0f : ex2(__fsub_rn(ml.x, base));   // 0: the split saw nothing of this row
                l = __fmaf_rn(ml.y, f, l);
            }
            const int n = min(32, (a.splits - s0 - part + W - 1) / W);
            for (int i0 = 0; i0 < n; i0 += 8) {
                float4 x[8];
#pragma unroll
                for (int i = 0; i < 8; i++)
                    x[i] = i0 + i < n ? *reinterpret_cast<const float4 *>(
                                            a.part + ((s0 + (i0 + i) * W + part) * step + at) * kTile + 4 * lane)
                                      : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const float fi = __shfl_sync(0xffffffffu, f, (i0 + i) & 31);
                    o.x = __fmaf_rn(x[i].x, fi, o.x);
                    o.y = __fmaf_rn(x[i].y, fi, o.y);
                    o.z = __fmaf_rn(x[i].z, fi, o.z);
                    o.w = __fmaf_rn(x[i].w, fi, o.w);
                }
            }
        }
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) l = __fadd_rn(l, __shfl_xor_sync(0xffffffffu, l, s));
    }
    if (W > 1) {
        xs[warp][lane] = o;
        if (lane == 0) ls[warp] = l;
        __syncthreads();
        if (part) return;
#pragma unroll
        for (int i = 1; i < W; i++) {
            const float4 x = xs[warp + i][lane];
            o.x = __fadd_rn(o.x, x.x);
            o.y = __fadd_rn(o.y, x.y);
            o.z = __fadd_rn(o.z, x.z);
            o.w = __fadd_rn(o.w, x.w);
            l = __fadd_rn(l, ls[warp + i]);
        }
    }
    if (!on) return;
    // back from the rotated domain
    float o4[4] = {o.x, o.y, o.z, o.w};
    if (a.rot[1]) {
        xs[warp][lane] = o;
        __syncwarp();
        o4[0] = o4[1] = o4[2] = o4[3] = 0.0f;
#pragma unroll 8
        for (int i = 0; i < 128; i++) {
            const float z = reinterpret_cast<const float *>(xs[warp])[i];
            const float4 q = __ldg(reinterpret_cast<const float4 *>(a.rot[1] + i * 128) + lane);
            o4[0] = __fmaf_rn(q.x, z, o4[0]);
            o4[1] = __fmaf_rn(q.y, z, o4[1]);
            o4[2] = __fmaf_rn(q.z, z, o4[2]);
            o4[3] = __fmaf_rn(q.w, z, o4[3]);
        }
    } else {
        fwht_row(o4, lane);
        const uint32_t e = sign[lane >> 3];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int c = (4 * lane + i) & 31;
            if ((e >> ((c >> 1) + 16 * (c & 1))) & 1u) o4[i] = -o4[i];
        }
    }
    // what an invisible draft holds does not matter: only those of `mine` are read
    for (unsigned long long left = mine; left;) {
        int j[4];
        uint2 vr[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            j[i] = left ? __ffsll((long long)left) - 1 : -1;
            left &= left - 1;
        }
#pragma unroll
        for (int i = 0; i < 4; i++)
            vr[i] = j[i] >= 0 ? *reinterpret_cast<const uint2 *>(a.vd + j[i] * a.d_ld_tok + d_head) : make_uint2(0u, 0u);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float p = j[i] >= 0 ? ex2(__fsub_rn(ps[warp / W][j[i] < 0 ? 0 : j[i]], base)) : 0.0f;
            l = __fadd_rn(l, p);
            o4[0] = __fmaf_rn(p, __uint_as_float(vr[i].x << 16), o4[0]);
            o4[1] = __fmaf_rn(p, __uint_as_float(vr[i].x & 0xFFFF0000u), o4[1]);
            o4[2] = __fmaf_rn(p, __uint_as_float(vr[i].y << 16), o4[2]);
            o4[3] = __fmaf_rn(p, __uint_as_float(vr[i].y & 0xFFFF0000u), o4[3]);
        }
    }
    const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);   // a row that sees nothing: zeros
#pragma unroll
    for (int i = 0; i < 4; i++) o4[i] = __fmul_rn(o4[i], inv);
    const int64_t off = qi * a.out_ld_tok + qh * a.out_ld_head + 4 * lane;
    if (a.out_fp32) {
        *reinterpret_cast<float4 *>((float *)a.out + off) = make_float4(o4[0], o4[1], o4[2], o4[3]);
    } else {
        __nv_bfloat162 b0 = __floats2bfloat162_rn(o4[0], o4[1]), b1 = __floats2bfloat162_rn(o4[2], o4[3]);
        *reinterpret_cast<uint2 *>((uint16_t *)a.out + off) =
            make_uint2(*reinterpret_cast<uint32_t *>(&b0), *reinterpret_cast<uint32_t *>(&b1));
    }
    if (a.lse && lane == 0)
        a.lse[(int64_t)qi * a.heads * a.group + qh] =
            l == 0.0f ? kNegInf : __fmul_rn(__fadd_rn(m, log2f(l)), 0.69314718055994530942f);
}

// The combine may start while the splits run: its own inputs come first, and it waits for theirs.
template <int W>
cudaError_t launch_combine(const AttnArgs &a, cudaStream_t s) {
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((unsigned)((a.rows + kCombineWarps / W - 1) / (kCombineWarps / W)), (unsigned)a.heads);
    c.blockDim = dim3(kCombineWarps * 32);
    c.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = at;
    c.numAttrs = a.splits ? 1 : 0;
    return cudaLaunchKernelEx(&c, attention_combine<W>, a);
}

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

int check_spec(const hq_attn_spec *sp) {
    if (!sp || sp->len < 0 || sp->window < 0 || sp->sinks < 0 || !isfinite(sp->scale)) return HQ_EINVAL;
    if (sp->n_q < 0 || sp->group < 1) return HQ_EINVAL;
    if (sp->n_q > kAttnMaxQueries || sp->group > kAttnMaxGroup || sp->len > (INT64_C(1) << 40)) return HQ_EUNSUPPORTED;
    return HQ_OK;
}

int attend(const hq_kv_cache *k, const hq_kv_cache *v, const hq_attn_spec *sp, const void *d_q, int64_t q_ld_token,
           int64_t q_ld_head, bool tree, const void *d_kd, const void *d_vd, int64_t d_ld_token, int64_t d_ld_head,
           const uint64_t *d_mask, void *out, int out_dtype, int64_t out_ld_token, int64_t out_ld_head, float *d_lse,
           void *workspace, size_t ws_bytes, void *cuda_stream) {
    int rc = check_spec(sp);
    if (rc) return rc;
    if (!k || !v || k == v || !k->d_words || !v->d_words || k->heads <= 0 || k->heads != v->heads) return HQ_EINVAL;
    if (k->head_dim != kTile || v->head_dim != kTile) return HQ_EUNSUPPORTED;
    if (out_dtype != 0 && out_dtype != 1) return HQ_EINVAL;
    // the two caches' appends have to cover the same tokens (the device tables are compared too)
    if (sp->len > k->tokens || sp->len > v->tokens || k->chunks != v->chunks || k->appends != v->appends) return HQ_EINVAL;
    if (k->params.lattice != v->params.lattice || k->params.dither != v->params.dither) return HQ_EUNSUPPORTED;
    if (!tree && sp->n_q > sp->len) return HQ_EINVAL;   // the queries are the last cached tokens
    if (k->heads > 65535) return HQ_EUNSUPPORTED;       // a grid dimension
    if (sp->n_q == 0) return HQ_OK;
    const int m = out_dtype ? 4 : 8, n_heads = k->heads * sp->group;
    if (!d_q || !aligned(d_q, 16) || q_ld_token < 0 || q_ld_token % 8 || q_ld_head < 0 || q_ld_head % 8) return HQ_EINVAL;
    if (!out || !aligned(out, 16) || out_ld_token < 0 || out_ld_token % m || out_ld_head < 0 || out_ld_head % m)
        return HQ_EINVAL;
    if (!vectors_apart(sp->n_q, out_ld_token, n_heads, out_ld_head)) return HQ_EINVAL;
    if (d_lse && !aligned(d_lse, 4)) return HQ_EINVAL;
    if (tree && (!d_kd || !aligned(d_kd, 16) || !d_vd || !aligned(d_vd, 16) || d_ld_token < 0 || d_ld_token % 8 ||
                 d_ld_head < 0 || d_ld_head % 8 || !d_mask || !aligned(d_mask, 8)))
        return HQ_EINVAL;
    size_t need = 0;
    if ((rc = hq_kv_attention_workspace_bytes(k->heads, sp, &need))) return rc;
    if (!workspace || !aligned(workspace, 16) || ws_bytes < need) return HQ_EINVAL;
    AttnArgs a;
    memset(&a, 0, sizeof(a));
    const hq_kv_cache *c[2] = {k, v};
    for (int i = 0; i < 2; i++) {
        a.words[i] = c[i]->d_words;
        a.cap[i] = c[i]->cap_words;
        a.offsets[i] = c[i]->d_offsets;
        a.table[i] = c[i]->d_table;
        a.stats[i] = c[i]->d_stats;
        a.seed[i] = c[i]->params.seed;
        a.rot[i] = c[i]->params.rotation;
        a.k[i] = c[i]->params.rice_k;
        a.k_last[i] = k_last_of(c[i]->params);
    }
    a.n_chunks = k->chunks;
    a.n_appends = k->appends;
    a.len = sp->len;
    a.window = sp->window > sp->len + kAttnMaxQueries ? 0 : sp->window;   // sees everything
    a.sinks = sp->sinks > sp->len + kAttnMaxQueries ? sp->len + kAttnMaxQueries : sp->sinks;
    a.heads = k->heads;
    a.group = sp->group;
    a.n_q = sp->n_q;
    a.rows = sp->n_q * sp->group;
    a.row_pad = attn_row_pad(a.rows);
    a.scale_log2 = (float)((double)sp->scale * 1.4426950408889634074);
    a.q = (const uint16_t *)d_q;
    a.q_ld_tok = q_ld_token;
    a.q_ld_head = q_ld_head;
    if (tree) {
        a.mask = (const unsigned long long *)d_mask;
        a.kd = (const uint16_t *)d_kd;
        a.vd = (const uint16_t *)d_vd;
        a.d_ld_tok = d_ld_token;
        a.d_ld_head = d_ld_head;
    }
    a.wait_limit = spin_limit() < kAttnWaitPolls ? spin_limit() : kAttnWaitPolls;
    a.out = out;
    a.out_fp32 = out_dtype;
    a.out_ld_tok = out_ld_token;
    a.out_ld_head = out_ld_head;
    a.lse = d_lse;
    cudaStream_t s = (cudaStream_t)cuda_stream;
    const bool cached = sp->len > 0 && k->chunks > 0;
    if (cached) {
        const ChunkCount see = visible_chunks(*k, a.window, a.window + sp->n_q + a.sinks);
        a.short_steps = attn_short(a.heads, a.rows, see.likely);
        a.splits = attn_splits(a.heads, a.rows, see.most, a.short_steps);
        a.part = (float *)workspace;
        a.ml = (float2 *)(a.part + (size_t)a.splits * a.heads * a.row_pad * kTile);
        if (launch_attention(k->params.lattice, k->params.dither, a, s) != cudaSuccess) return HQ_ECUDA;
    }
    const bool spread = (int64_t)a.rows * a.heads <= kCombineSpread;
    return (spread ? launch_combine<kCombineWarps>(a, s) : launch_combine<1>(a, s)) == cudaSuccess ? HQ_OK : HQ_ECUDA;
}

}  // namespace

cudaError_t launch_attention(int lattice, int dither, const AttnArgs &a, cudaStream_t s) {
    switch (lattice) {
    case HQ_Z: return launch_attention_z(dither, a, s);
    case HQ_A2: return launch_attention_a2(dither, a, s);
    case HQ_D4: return launch_attention_d4(dither, a, s);
    case HQ_E8: return launch_attention_e8(dither, a, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace hq

using namespace hq;

extern "C" {

int hq_kv_attention_workspace_bytes(int32_t heads, const hq_attn_spec *spec, size_t *bytes) {
    const int rc = check_spec(spec);
    if (rc) return rc;
    if (!bytes || heads <= 0) return HQ_EINVAL;
    const int rows = spec->n_q * spec->group;
    // as many splits as any cache of this many heads may take
    const size_t splits = (size_t)attn_splits(heads, rows, UINT64_C(1) << 40, false);
    *bytes = (splits * (size_t)heads * (size_t)attn_row_pad(rows) * (kTile * sizeof(float) + sizeof(float2)) + 255) &
             ~(size_t)255;
    return HQ_OK;
}

int hq_kv_attention(const hq_kv_cache *k, const hq_kv_cache *v, const hq_attn_spec *spec, const void *d_q,
                    int64_t q_ld_token, int64_t q_ld_head, void *out, int out_dtype, int64_t out_ld_token,
                    int64_t out_ld_head, float *d_lse, void *workspace, size_t ws_bytes, void *cuda_stream) {
    return attend(k, v, spec, d_q, q_ld_token, q_ld_head, false, nullptr, nullptr, 0, 0, nullptr, out, out_dtype,
                  out_ld_token, out_ld_head, d_lse, workspace, ws_bytes, cuda_stream);
}

int hq_kv_tree_attention(const hq_kv_cache *k, const hq_kv_cache *v, const hq_attn_spec *spec, const void *d_q,
                         int64_t q_ld_token, int64_t q_ld_head, const void *d_kd, const void *d_vd, int64_t d_ld_token,
                         int64_t d_ld_head, const uint64_t *d_mask, void *out, int out_dtype, int64_t out_ld_token,
                         int64_t out_ld_head, float *d_lse, void *workspace, size_t ws_bytes, void *cuda_stream) {
    return attend(k, v, spec, d_q, q_ld_token, q_ld_head, true, d_kd, d_vd, d_ld_token, d_ld_head, d_mask, out,
                  out_dtype, out_ld_token, out_ld_head, d_lse, workspace, ws_bytes, cuda_stream);
}

}  // extern "C"
