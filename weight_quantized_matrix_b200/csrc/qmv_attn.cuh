// qmv_attn.cuh -- device pieces of the paged attention kernels.
#pragma once

#include "qmv_attn_mma.cuh"
#include "qmv_paged.cuh"

namespace qmv {

__device__ __forceinline__ float ld_elem(const float* p) { return __ldg(p); }
__device__ __forceinline__ float ld_elem(const __half* p) { return __half2float(*p); }
__device__ __forceinline__ float ld_elem(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st_elem(float* p, float v) { *p = v; }
__device__ __forceinline__ void st_elem(__half* p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void st_elem(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Element offset of key / value row j of sequence b, kv head hk; -1 when the
// page table has no page of the cache there.
__device__ __forceinline__ long long key_place(const AttnParams& p, int b, int hk, int j) {
    const int e = j / p.page;
    if (e >= p.max_pages) return -1;
    const int pg = __ldg(p.table + (long long)b * p.max_pages + e);
    if ((unsigned)pg >= (unsigned)p.n_pages) return -1;
    return (long long)pg * p.page_s + (long long)(j - e * p.page) * p.tok_s + (long long)hk * p.head_s;
}

// Dot product -> score in units of log2: scale, then the cap c tanh(s / c), then
// the distance bias.  EXACT (fp32 elements) takes tanhf.  For 16-bit elements
// (the hardware's tanh approximation has an error of 2^-11, which the cap would
// multiply into the score): up to |t| = |s / c| = 0.7 tanh's odd polynomial, fitted
// to 2^-25 of t, so that a score far below its cap keeps its own precision
// whatever the cap is; beyond, 1 - 2 / (2^(2t log2 e) + 1), whose absolute error of
// 2^-21 is 2^-20 of the result there, with exact limits at both ends.
template <bool EXACT> struct ScoreMod {
    static constexpr float kBend = 0.7f;
    float pre, post;            // scale / c and c log2 e; without a cap scale log2 e
    bool cap;
    __device__ explicit ScoreMod(const AttnParams& p) {
        cap = p.softcap > 0.0f;
        pre = cap ? p.scale / p.softcap : p.scale * kLog2e;
        post = p.softcap * kLog2e;
    }
    // (tanh(t) - t) / t^3 as a polynomial in u = t^2, pairwise
    __device__ static __forceinline__ float2 bend(float2 u) {
        float2 r = fma2(make_float2(-0.00515510421f, -0.00515510421f), u, make_float2(0.0201116465f, 0.0201116465f));
        r = fma2(r, u, make_float2(-0.0535669848f, -0.0535669848f));
        r = fma2(r, u, make_float2(0.133292437f, 0.133292437f));
        return fma2(r, u, make_float2(-0.333331972f, -0.333331972f));
    }
    // c tanh(t) of two scores, each by the form for its size
    __device__ __forceinline__ float2 capped(float2 t) const {
        const float2 w = mul2(t, make_float2(post, post)), u = mul2(t, t);
        float2 v = fma2(mul2(w, u), bend(u), w);
        const float2 x = mul2(t, make_float2(2.0f * kLog2e, 2.0f * kLog2e));
        if (!(fabsf(t.x) <= kBend)) v.x = fmaf(-post, __fdividef(2.0f, ex2(x.x) + 1.0f), post);
        if (!(fabsf(t.y) <= kBend)) v.y = fmaf(-post, __fdividef(2.0f, ex2(x.y) + 1.0f), post);
        return v;
    }
    __device__ __forceinline__ float apply(float dot, float slope_log2, int away) const {
        float s = dot * pre;
        if (cap) {
            if constexpr (EXACT) s = post * tanhf(s);
            else s = capped(make_float2(s, s)).x;
        }
        return fmaf(slope_log2, (float)away, s);
    }
    // Scale and cap of N scores.  Where every |s / c| of the warp is at most 0.7
    // (scores seldom come near their cap) the polynomial alone: no exponential and
    // no division, which are the scarce units in a softmax.
    template <int N> __device__ __forceinline__ void scaled(float (&x)[N]) const {
        const float2 pre2 = make_float2(pre, pre);
        if (cap) {
            float big = 0.0f;
#pragma unroll
            for (int c = 0; c < N; c += 2) big = max3(fabsf(x[c]), fabsf(x[c + 1]), big);
            if (__all_sync(0xFFFFFFFFu, big * pre <= kBend)) {
                const float2 post2 = make_float2(post, post);
#pragma unroll
                for (int c = 0; c < N; c += 2) {
                    const float2 t = mul2(make_float2(x[c], x[c + 1]), pre2), u = mul2(t, t);
                    const float2 w = mul2(t, post2), v = fma2(mul2(w, u), bend(u), w);
                    x[c] = v.x;
                    x[c + 1] = v.y;
                }
            } else {
#pragma unroll
                for (int c = 0; c < N; c += 2) {
                    const float2 v = capped(mul2(make_float2(x[c], x[c + 1]), pre2));
                    x[c] = v.x;
                    x[c + 1] = v.y;
                }
            }
        } else {
#pragma unroll
            for (int c = 0; c < N; c += 2) {
                const float2 v = mul2(make_float2(x[c], x[c + 1]), pre2);
                x[c] = v.x;
                x[c + 1] = v.y;
            }
        }
    }
    // N scores of consecutive keys, the first `away` from the row's position.
    template <int N> __device__ __forceinline__ void apply_all(float (&x)[N], float slope_log2, int away) const {
        scaled(x);
        if (slope_log2 != 0.0f) {
            const float a0 = (float)away;
            const float2 a2 = make_float2(a0, a0), s2 = make_float2(slope_log2, slope_log2);
#pragma unroll
            for (int c = 0; c < N; c += 2) {
                const float2 v = fma2(s2, add2(a2, make_float2((float)c, (float)(c + 1))), make_float2(x[c], x[c + 1]));
                x[c] = v.x;
                x[c + 1] = v.y;
            }
        }
    }
};

}  // namespace qmv
