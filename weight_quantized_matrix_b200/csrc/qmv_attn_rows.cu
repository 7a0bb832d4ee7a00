// qmv_attn_rows.cu -- attention over a paged cache, one warp per query row: the
// path for every head size, stride and alignment.
//
// Mathematics: one pass over the row's visible keys with the running maximum
// m and sum l of the softmax (scores times log2 e, so that exp is exp2):
//     m' = max(m, s);  l = l 2^(m - m') + 2^(s - m');  o = o 2^(m - m') + 2^(s - m') v
// and at the end o / l, lse = ln 2 (m + log2 l).  All of it fp32; the output is
// rounded once.  Lane l holds dims l, l + 32, ...; a score is a butterfly sum.
// Keys go four at a time so that their loads overlap.  Keys the row does not
// see are never read.
#include "qmv_attn.cuh"

namespace qmv {

namespace {

constexpr int kRowWarps = 4;
constexpr int kRowDims = 8;             // 32 * 8 = 256 dims at most

template <class T>
__global__ void __launch_bounds__(kRowWarps * 32) attn_rows_kernel(const __grid_constant__ AttnParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long rows = (long long)p.T * p.Hq;
    const ScoreMod<true> mod(p);
    for (long long r = (long long)blockIdx.x * kRowWarps + (threadIdx.x >> 5); r < rows;
         r += (long long)gridDim.x * kRowWarps) {
        const int t = (int)(r / p.Hq), h = (int)(r - (long long)t * p.Hq);
        const int b = seq_of_row(p.q_starts, p.n_seqs, t);
        if (b < 0) continue;
        const int len = max(0, __ldg(p.kv_lens + b));
        const int pos = len - __ldg(p.q_starts + b + 1) + t;
        int lo, hi;
        visible_keys(p, pos, len, lo, hi);
        const float slope = p.slopes ? __ldg(p.slopes + h) * kLog2e : 0.0f;
        float q[kRowDims], o[kRowDims];
#pragma unroll
        for (int i = 0; i < kRowDims; ++i) {
            const int d = lane + 32 * i;
            q[i] = d < p.D ? ld_elem(static_cast<const T*>(p.q) + t * p.q_ts + h * p.q_hs + d) : 0.0f;
            o[i] = 0.0f;
        }
        float m = -INFINITY, l = 0.0f;
        for (unsigned j0 = lo; j0 < (unsigned)hi; j0 += 4) {          // (hi may be the last int)
            long long at[4];
            float s[4];
            bool bad[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int j = (int)min(j0 + u, (unsigned)hi - 1);
                at[u] = key_place(p, b, h / p.G, j);
                bad[u] = at[u] < 0;
                if (bad[u]) at[u] = 0;
                s[u] = 0.0f;
#pragma unroll
                for (int i = 0; i < kRowDims; ++i) {
                    const int d = lane + 32 * i;
                    if (d < p.D && !bad[u]) s[u] = fmaf(q[i], ld_elem(static_cast<const T*>(p.k) + at[u] + d), s[u]);
                }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
#pragma unroll
                for (int w = 16; w > 0; w >>= 1) s[u] += __shfl_xor_sync(0xFFFFFFFFu, s[u], w);
                s[u] = mod.apply(s[u], slope, (int)(j0 + u - (unsigned)pos));
                if (bad[u]) s[u] = NAN;
                if (j0 + u >= (unsigned)hi) s[u] = -INFINITY;
            }
            float mn = m;
#pragma unroll
            for (int u = 0; u < 4; ++u) mn = fmaxf(mn, s[u]);
            const float base = mn == -INFINITY ? 0.0f : mn;      // every score -inf so far: weights 0
            const float f = exp2f(m - base);
            l *= f;
#pragma unroll
            for (int i = 0; i < kRowDims; ++i) o[i] *= f;
            m = mn;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (j0 + u >= (unsigned)hi) break;
                const float w = exp2f(s[u] - base);
                l += w;
#pragma unroll
                for (int i = 0; i < kRowDims; ++i) {
                    const int d = lane + 32 * i;
                    if (d < p.D && !bad[u]) o[i] = fmaf(w, ld_elem(static_cast<const T*>(p.v) + at[u] + d), o[i]);
                    if (bad[u]) o[i] = NAN;
                }
            }
        }
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
        for (int i = 0; i < kRowDims; ++i) {
            const int d = lane + 32 * i;
            if (d < p.D)
                st_elem(static_cast<T*>(p.out) + t * p.o_ts + h * p.o_hs + d, l == 0.0f ? 0.0f : o[i] * inv);
        }
        if (p.lse && lane == 0) p.lse[(long long)t * p.Hq + h] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
    }
}

}  // namespace

cudaError_t launch_attn_rows(int dtype, const AttnParams& p, cudaStream_t st) {
    const long long rows = (long long)p.T * p.Hq;
    long long grid = (rows + kRowWarps - 1) / kRowWarps;
    if (grid > (1 << 20)) grid = 1 << 20;
    const dim3 g((unsigned)grid), blk(kRowWarps * 32);
    switch (dtype) {
        case 0: return launch_dependent(attn_rows_kernel<float>, g, blk, 0, st, p);
        case 1: return launch_dependent(attn_rows_kernel<__half>, g, blk, 0, st, p);
        case 2: return launch_dependent(attn_rows_kernel<__nv_bfloat16>, g, blk, 0, st, p);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace qmv
