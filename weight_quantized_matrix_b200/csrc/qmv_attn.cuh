// qmv_attn.cuh -- device pieces of the paged attention kernels.
#pragma once

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
};

}  // namespace qmv
