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

// Dot product -> score in units of log2: scale, then the cap c tanh(s / c),
// then the distance bias.  EXACT (fp32 elements) takes tanhf.  For 16-bit
// elements tanh(x) = 1 - 2 / (2^(2x log2 e) + 1), with exact limits at both ends and
// an absolute error below 2^-20 (the hardware's tanh approximation has 2^-11,
// which the cap would multiply into the score).
template <bool EXACT> struct ScoreMod {
    float pre, post;
    bool cap;
    __device__ explicit ScoreMod(const AttnParams& p) {
        cap = p.softcap > 0.0f;
        pre = !cap ? p.scale * kLog2e : EXACT ? p.scale / p.softcap : p.scale / p.softcap * (2.0f * kLog2e);
        post = p.softcap * kLog2e;
    }
    __device__ __forceinline__ float apply(float dot, float slope_log2, int away) const {
        float s = dot * pre;
        if (cap) {
            if constexpr (EXACT) {
                s = post * tanhf(s);
            } else {
                float e;
                asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(s));
                s = fmaf(-post, __fdividef(2.0f, e + 1.0f), post);
            }
        }
        return fmaf(slope_log2, (float)away, s);
    }
    // N scores of consecutive keys, the first `away` from the row's position.
    // Where every |s / c| of the warp is at most 0.7 (scores seldom come near their
    // cap) tanh is its odd polynomial, fitted to 2^-26 there: no exponential and
    // no division, which are the scarce units in a softmax.
    template <int N> __device__ __forceinline__ void apply_all(float (&x)[N], float slope_log2, int away) const {
        const float2 pre2 = make_float2(pre, pre);
        if (cap) {
            float big = 0.0f;
#pragma unroll
            for (int c = 0; c < N; c += 2) big = max3(fabsf(x[c]), fabsf(x[c + 1]), big);
            const float half = pre * (0.5f * kLn2);             // pre holds 2 log2 e / c
            if (__all_sync(0xFFFFFFFFu, big * half <= 0.7f)) {
                const float2 h2 = make_float2(half, half), post2 = make_float2(post, post);
#pragma unroll
                for (int c = 0; c < N; c += 2) {
                    const float2 t = mul2(make_float2(x[c], x[c + 1]), h2), u = mul2(t, t);
                    float2 r = fma2(make_float2(-0.00515510421f, -0.00515510421f), u, make_float2(0.0201116465f, 0.0201116465f));
                    r = fma2(r, u, make_float2(-0.0535669848f, -0.0535669848f));
                    r = fma2(r, u, make_float2(0.133292437f, 0.133292437f));
                    r = fma2(r, u, make_float2(-0.333331972f, -0.333331972f));
                    const float2 w = mul2(t, post2), v = fma2(mul2(w, u), r, w);
                    x[c] = v.x;
                    x[c + 1] = v.y;
                }
            } else {
#pragma unroll
                for (int c = 0; c < N; ++c) x[c] = apply(x[c], 0.0f, 0);
            }
        } else {
#pragma unroll
            for (int c = 0; c < N; c += 2) {
                const float2 v = mul2(make_float2(x[c], x[c + 1]), pre2);
                x[c] = v.x;
                x[c + 1] = v.y;
            }
        }
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
