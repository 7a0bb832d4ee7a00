// qmv_attn_f32.cu -- attention over a paged cache for fp32 elements.
//
// The products are fp32 FMAs (the tensor cores have no fp32 form; splitting the
// operands would lose to the copies at the few rows this type is decoded with).
// One-token and drafted decode is bound by the keys and values, which a unit's 16
// packed rows share; long chunks are bound by the FMAs and the shared-memory
// reads that feed them.
//  * As in qmv_attn_few.cu every warp streams its own 16 keys of a tile through its
//    own ring (cp.async, 16-byte chunks, XOR-swizzled).
//  * Scores: a lane makes 4 keys of up to 4 rows from half of the dims, so that
//    shared memory feeds the FMAs.  Units of up to 4, 8 or 16 rows run code of
//    that size.
//  * Weights go through shared memory; for the second product a lane owns D / 32
//    dims of every row, V is read once for all rows.
//  * DP = 64, 128 or 256 dims, padded with zeros in shared memory only.
// Measured: 12 sequences of 2-5 new tokens over 100-2100 keys, 16 heads of 64: 43 us =
// 2.8 TB/s; one token of 8 sequences over 4000 keys, 8 kv heads of 128, 74 us = 3.5 TB/s:
// bound by the latency of a step's instructions, at one or two warps a scheduler.
// 1000 tokens over 2000 keys, 32 heads of 128: 1140 us = 22 TFLOP/s, so bound, too
// (issue slots 32 % busy); 1290 with a lane a key and all rows.  At 256 dims the
// kernel spills 326 bytes a thread.
#include <algorithm>

#include "qmv_attn_mma.cuh"
#include "qmv_attn_sched.cuh"

namespace qmv {

namespace {

constexpr int kRows = 16;

template <int DP> struct F32Geom {
    static constexpr int WARPS = DP == 64 ? 4 : 2;
    static constexpr int TILE = 16 * WARPS;
    static constexpr int STAGES = 3;
    static constexpr int PER_SM = DP == 256 ? 1 : 2;
    static constexpr int ROWB = DP * 4;
    static constexpr int STEP = 2 * 16 * ROWB;
    static constexpr int RING = WARPS * STAGES * STEP;
    static constexpr int QH = DP / 2 + 4;                    // floats of half a query row; the halves fall on other banks
    static constexpr int SMEM = RING + kRows * 2 * QH * 4;
};
static_assert(kJoinBytes <= F32Geom<64>::RING, "joined in the ring");

// A unit's rows as the steps need them.
struct Rows {
    int lo[kRows], hi[kRows], pos[kRows];       // keys the row sees, its position
    float slope[kRows];
};

// The weights of the first 4 rows: lane = (key, half of the dims) makes its key's
// scores of all rows (few rows want the reads in flight, not their reuse: one
// token of 32 heads on 8 over 8 x 4000 keys takes 75 us this way and 82 the other).
// m and l are all rows', l of the lane's key.
template <int DP, bool MOD>
__device__ __forceinline__ void f32_weights4(const unsigned char* kb, const float* s_q, float (&s_p)[16][kRows], const Rows& rows,
                                             const ScoreMod<true>& mod, int j0, bool full, float2 (&o)[kRows / 2][DP / 32],
                                             float (&m)[kRows / 4], float (&l)[kRows / 4]) {
    using Gm = F32Geom<DP>;
    constexpr int R = 4, ROWB = Gm::ROWB, CPR = DP / 4, VEC = DP / 32;
    const int lane = threadIdx.x & 31, key = lane & 15, hf = lane >> 4, j = j0 + key;
    float x[R], mx[R];
#pragma unroll
    for (int r = 0; r < R; ++r) x[r] = 0.0f;
#pragma unroll 4
    for (int c = 0; c < CPR / 2; ++c) {
        const float4 kv = *reinterpret_cast<const float4*>(kb + key * ROWB + (((hf * (CPR / 2) + c) ^ (key & 7)) << 4));
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float4 qv = *reinterpret_cast<const float4*>(s_q + (r * 2 + hf) * Gm::QH + c * 4);
            x[r] = fmaf(qv.x, kv.x, x[r]);
            x[r] = fmaf(qv.y, kv.y, x[r]);
            x[r] = fmaf(qv.z, kv.z, x[r]);
            x[r] = fmaf(qv.w, kv.w, x[r]);
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) x[r] += __shfl_xor_sync(0xFFFFFFFFu, x[r], 16);
    if constexpr (MOD) {                        // each half of the warp takes half of the rows
#pragma unroll
        for (int r = 0; r < R / 2; ++r) {
            const int mr = hf ? r + R / 2 : r;
            const float y = mod.apply(hf ? x[r + R / 2] : x[r], rows.slope[mr], j - rows.pos[mr]);
            const float z = __shfl_xor_sync(0xFFFFFFFFu, y, 16);
            x[r] = hf ? z : y;
            x[r + R / 2] = hf ? y : z;
        }
    } else {
#pragma unroll
        for (int r = 0; r < R; ++r) x[r] = __fmul_rn(x[r], mod.pre);     // rounded alike for the maximum and the weight
    }
    if (!full) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (j < rows.lo[r] || j >= rows.hi[r]) x[r] = -INFINITY;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) mx[r] = x[r];
#pragma unroll
    for (int w = 8; w > 0; w >>= 1)
#pragma unroll
        for (int r = 0; r < R; ++r) mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xFFFFFFFFu, mx[r], w));
    bool raise = false;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        mx[r] = fmaxf(mx[r], m[r]);
        raise |= mx[r] > m[r];
    }
    if (raise) {                                // the same for every lane
        float f[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            f[r] = mx[r] > m[r] ? ex2(m[r] - mx[r]) : 1.0f;
            l[r] *= f[r];
            m[r] = mx[r];
        }
#pragma unroll
        for (int u = 0; u < VEC; ++u) {
            o[0][u] = mul2(o[0][u], make_float2(f[0], f[1]));
            o[1][u] = mul2(o[1][u], make_float2(f[2], f[3]));
        }
    }
    __syncwarp();
#pragma unroll
    for (int r = 0; r < R; ++r) {
        x[r] = ex2(x[r] - (mx[r] == -INFINITY ? 0.0f : mx[r]));
        l[r] += x[r];                           // summed over the 16 lanes of a half at the end
    }
    if (hf == 0) *reinterpret_cast<float4*>(&s_p[4 * (key & 3) + (key >> 2)][0]) = make_float4(x[0], x[1], x[2], x[3]);
    __syncwarp();
}

// The weights of a step of 16 keys (j0 on) against the first R = 8 or 16 rows: lane = (kl, rg,
// hf) makes keys kl + 4 i, i < 4, of rows rg + 4 r from half hf of the dims: 8
// 16-byte reads without conflicts feed 64 products (R = 16; with a lane a key and
// all rows it is 17).  The halves then swap sums, and each goes on with two of the
// keys; m and l are the lane's rows'.  Weights go through s_p, key kl + 4 i at
// 4 kl + i, row rg + 4 r at rg RL + r.
template <int DP, bool MOD, int R>
__device__ __forceinline__ void f32_weights(const unsigned char* kb, const float* s_q, float (&s_p)[16][kRows],
                                         float (&s_f)[kRows], const Rows& rows, const ScoreMod<true>& mod, int j0, bool full,
                                         float2 (&o)[kRows / 2][DP / 32], float (&m)[kRows / 4], float (&l)[kRows / 4]) {
    using Gm = F32Geom<DP>;
    constexpr int ROWB = Gm::ROWB, CPR = DP / 4, VEC = DP / 32, RL = R / 4;
    const int lane = threadIdx.x & 31, kl = lane & 3, rg = (lane >> 2) & 3, hf = lane >> 4;
    float2 s[4][RL];            // even and odd dims
    float x[2][RL], mx[RL];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < RL; ++r) s[i][r] = make_float2(0.0f, 0.0f);
#pragma unroll 2
    for (int c = 0; c < CPR / 2; ++c) {
        const int cc = hf * (CPR / 2) + (c ^ (hf << 2));        // the halves read other banks
        float4 kv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int key = kl + 4 * i;
            kv[i] = *reinterpret_cast<const float4*>(kb + key * ROWB + ((cc ^ (key & 7)) << 4));
        }
#pragma unroll
        for (int r = 0; r < RL; ++r) {
            const float4 qv = *reinterpret_cast<const float4*>(s_q + ((rg + 4 * r) * 2 + hf) * Gm::QH + (c ^ (hf << 2)) * 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[i][r] = fma2(make_float2(qv.x, qv.y), make_float2(kv[i].x, kv[i].y), s[i][r]);
                s[i][r] = fma2(make_float2(qv.z, qv.w), make_float2(kv[i].z, kv[i].w), s[i][r]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < RL; ++r)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const float a = s[u][r].x + s[u][r].y, b = s[2 + u][r].x + s[2 + u][r].y;
            x[u][r] = (hf ? b : a) + __shfl_xor_sync(0xFFFFFFFFu, hf ? a : b, 16);
        }
    const int j = j0 + kl + 8 * hf;                             // the lane's keys: j and j + 4
#pragma unroll
    for (int r = 0; r < RL; ++r)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if constexpr (MOD) x[u][r] = mod.apply(x[u][r], rows.slope[rg + 4 * r], j + 4 * u - rows.pos[rg + 4 * r]);
            else x[u][r] = __fmul_rn(x[u][r], mod.pre);
        }
    if (!full) {
#pragma unroll
        for (int r = 0; r < RL; ++r) {
            const int lo = rows.lo[rg + 4 * r], hi = rows.hi[rg + 4 * r];
#pragma unroll
            for (int u = 0; u < 2; ++u)
                if (j + 4 * u < lo || j + 4 * u >= hi) x[u][r] = -INFINITY;
        }
    }
    // all rows' maxima side by side: a butterfly's latency is paid once
    bool raise = false;
#pragma unroll
    for (int r = 0; r < RL; ++r) mx[r] = fmaxf(x[0][r], x[1][r]);
#pragma unroll
    for (int w = 1; w <= 16; w = w == 2 ? 16 : w * 2)
#pragma unroll
        for (int r = 0; r < RL; ++r) mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xFFFFFFFFu, mx[r], w));
#pragma unroll
    for (int r = 0; r < RL; ++r) {
        mx[r] = fmaxf(mx[r], m[r]);
        raise |= mx[r] > m[r];
    }
    raise = __any_sync(0xFFFFFFFFu, raise);
    __syncwarp();                               // every lane is done with s_p and s_f
    if (raise) {
#pragma unroll
        for (int r = 0; r < RL; ++r) {
            const float f = mx[r] > m[r] ? ex2(m[r] - mx[r]) : 1.0f;
            l[r] *= f;
            m[r] = mx[r];
            if (kl == 0 && hf == 0) s_f[rg * RL + r] = f;
        }
    }
    __syncwarp();
#pragma unroll
    for (int r = 0; r < RL; ++r) {
        const float ref = mx[r] == -INFINITY ? 0.0f : mx[r];
        const float e0 = ex2(x[0][r] - ref), e1 = ex2(x[1][r] - ref);
        l[r] += e0 + e1;                        // summed over the row's 8 lanes at the end
        x[0][r] = e0;
        x[1][r] = e1;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        float* to = &s_p[4 * kl + 2 * hf + u][rg * RL];
        if constexpr (RL == 4) *reinterpret_cast<float4*>(to) = make_float4(x[u][0], x[u][1], x[u][2], x[u][3]);
        else *reinterpret_cast<float2*>(to) = make_float2(x[u][0], x[u][1]);
    }
    __syncwarp();
    if (raise) {
#pragma unroll
        for (int r = 0; r < R / 2; ++r) {
            const float2 f = *reinterpret_cast<const float2*>(&s_f[2 * r]);
#pragma unroll
            for (int u = 0; u < VEC; ++u) o[r][u] = mul2(o[r][u], f);
        }
    }
}

// One step: weights, then the second product with lane = dims, two rows to an FMA.
template <int DP, bool MOD, int R>
__device__ __forceinline__ void f32_step(const unsigned char* kb, const unsigned char* vb, const float* s_q, float (&s_p)[16][kRows],
                                         float (&s_f)[kRows], const Rows& rows, const ScoreMod<true>& mod, int j0, bool full,
                                         float2 (&o)[kRows / 2][DP / 32], float (&m)[kRows / 4], float (&l)[kRows / 4]) {
    constexpr int ROWB = F32Geom<DP>::ROWB, VEC = DP / 32, RL = R / 4;
    const int lane = threadIdx.x & 31;
    if constexpr (R == 4) f32_weights4<DP, MOD>(kb, s_q, s_p, rows, mod, j0, full, o, m, l);
    else f32_weights<DP, MOD, R>(kb, s_q, s_p, s_f, rows, mod, j0, full, o, m, l);
#pragma unroll 2
    for (int k4 = 0; k4 < 16; k4 += 4) {
        float v[4][VEC];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int key = k4 / 4 + 4 * k;
            const unsigned char* row = vb + key * ROWB;
            if constexpr (VEC == 2) {
                const float2 f = *reinterpret_cast<const float2*>(row + (((lane >> 1) ^ (key & 7)) << 4) + (lane & 1) * 8);
                v[k][0] = f.x; v[k][1] = f.y;
            } else {
#pragma unroll
                for (int u = 0; u < VEC; u += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(row + (((lane + u * 8) ^ (key & 7)) << 4));
                    v[k][u] = f.x; v[k][u + 1] = f.y; v[k][u + 2] = f.z; v[k][u + 3] = f.w;
                }
            }
        }
        // Unseen keys weigh exactly 0, which finite values leave 0.
        bool plain = full;
        if (!full) {
            float z = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int u = 0; u < VEC; ++u) z = fmaf(v[k][u], 0.0f, z);
            plain = __all_sync(0xFFFFFFFFu, z == 0.0f);
        }
        if (plain) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float2 vv[VEC];
#pragma unroll
                for (int u = 0; u < VEC; ++u) vv[u] = make_float2(v[k][u], v[k][u]);
#pragma unroll
                for (int r = 0; r < R; r += 4) {
                    const float4 w = *reinterpret_cast<const float4*>(&s_p[k4 + k][r]);
#pragma unroll
                    for (int u = 0; u < VEC; ++u) {
                        o[r / 2][u] = fma2(make_float2(w.x, w.y), vv[u], o[r / 2][u]);
                        o[r / 2 + 1][u] = fma2(make_float2(w.z, w.w), vv[u], o[r / 2 + 1][u]);
                    }
                }
            }
        } else {
            // a key the row does not see takes no part, whatever its value holds
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int lo = rows.lo[r / RL + 4 * (r % RL)], hi = rows.hi[r / RL + 4 * (r % RL)];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int jk = j0 + k4 / 4 + 4 * k;
                    if (jk < lo || jk >= hi) continue;
                    const float w = s_p[k4 + k][r];
#pragma unroll
                    for (int u = 0; u < VEC; ++u) {
                        float& d = r % 2 ? o[r / 2][u].y : o[r / 2][u].x;
                        d = fmaf(w, v[k][u], d);
                    }
                }
            }
        }
    }
}

template <int DP, bool MOD>
__global__ void __launch_bounds__(F32Geom<DP>::WARPS * 32, F32Geom<DP>::PER_SM)
attn_f32_kernel(const __grid_constant__ AttnParams p, int page_shift) {
    using Gm = F32Geom<DP>;
    constexpr int WARPS = Gm::WARPS, NTH = WARPS * 32, STAGES = Gm::STAGES, ROWB = Gm::ROWB, CPR = DP / 4, VEC = DP / 32;           // a lane owns VEC dims
    extern __shared__ __align__(1024) unsigned char ring[];
    float* s_q = reinterpret_cast<float*>(ring + Gm::RING);
    __shared__ SchedSmem sm;
    __shared__ __align__(16) float s_p[WARPS][16][kRows];
    __shared__ __align__(16) float s_f[WARPS][kRows];
    __shared__ float s_m[WARPS][kRows], s_l[WARPS][kRows];
    __shared__ Rows rows;
    __shared__ int s_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned char* mine = ring + warp * STAGES * Gm::STEP;
    const uint32_t mine_a = s_addr(mine);
    const int chunks = p.D / 4;
    grid_dependency_wait();
    grid_launch_dependents();

    Sched<kRows, Gm::TILE> sc;
    sc.template init<NTH>(p, sm, 12);
    const ScoreMod<true> mod(p);
    const int page16 = (int)(p.page_s / 4), tok16 = (int)(p.tok_s / 4);

    while (sc.live) {
        int k0, k1;
        sc.piece(k0, k1);
        const SeqInfo s = sc.s;
        const int rbase = sc.i * kRows, nrows = min(kRows, s.n * p.G - rbase);
        int ulo, uhi;
        rows_keys(p, s, rbase, rbase + nrows - 1, ulo, uhi);
        const char* kh = static_cast<const char*>(p.k) + (long long)sc.h * p.head_s * 4;
        const char* vh = static_cast<const char*>(p.v) + (long long)sc.h * p.head_s * 4;
        const int* trow = p.table + (long long)sc.b * p.max_pages;
        auto place = [&](int t) -> int {
            const int j = (int)((unsigned)t * Gm::TILE + warp * 16 + (lane & 15));
            if (t >= k1 || j < ulo || j >= uhi) return -1;
            const int e = page_shift >= 0 ? j >> page_shift : j / p.page;
            if (e >= p.max_pages) return -2;
            const int pg = __ldg(trow + e);
            if ((unsigned)pg >= (unsigned)p.n_pages) return -2;
            return pg * page16 + (j - e * p.page) * tok16;
        };
        auto issue = [&](int t, int slot, int at) {
            if (t < k1) {
                const uint32_t base = mine_a + slot * Gm::STEP;
                if (chunks == CPR && __all_sync(0xFFFFFFFFu, at >= 0)) {
#pragma unroll 8
                    for (int u = 0; u < 16 * CPR / 32; ++u) {
                        const int id = u * 32 + lane, r = id / CPR, c = id % CPR;
                        const long long off = (long long)__shfl_sync(0xFFFFFFFFu, at, r) * 16 + c * 16;
                        const uint32_t d = base + r * ROWB + ((c ^ (r & 7)) << 4);
                        cp16(d, kh + off);
                        cp16(d + 16 * ROWB, vh + off);
                    }
                    cp_commit();
                    return;
                }
#pragma unroll 8
                for (int u = 0; u < 16 * CPR / 32; ++u) {
                    const int id = u * 32 + lane, r = id / CPR, c = id % CPR;
                    const int a = __shfl_sync(0xFFFFFFFFu, at, r);
                    const uint32_t d = base + r * ROWB + ((c ^ (r & 7)) << 4);
                    const bool rd = a >= 0 && c < chunks;
                    const long long off = rd ? (long long)a * 16 + c * 16 : 0;
                    cp16_or_zero(d, kh + off, rd);
                    cp16_or_zero(d + 16 * ROWB, vh + off, rd);
                }
                if (__any_sync(0xFFFFFFFFu, at == -2)) {            // keys of NaN, once the copies have landed
                    cp_commit();
                    cp_wait<0>();
                    __syncwarp();
                    if (lane < 16 && at == -2)
                        *reinterpret_cast<uint4*>(mine + slot * Gm::STEP + lane * ROWB + ((lane & 7) << 4)) =
                            make_uint4(~0u, ~0u, ~0u, ~0u);
                    return;
                }
            }
            cp_commit();
        };
        constexpr int AHEAD = 4;
        int at[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) at[u] = place(k0 + u);
        auto issue_next = [&](int t, int slot) {
            const int now = at[0];
#pragma unroll
            for (int u = 0; u + 1 < AHEAD; ++u) at[u] = at[u + 1];
            at[AHEAD - 1] = place(t + AHEAD);
            issue(t, slot, now);
        };

        // ---- queries and the rows' keys --------------------------------------
        for (int x = threadIdx.x; x < kRows * CPR; x += NTH) {
            const int r = x / CPR, c = x % CPR, pr = rbase + min(r, nrows - 1), ti = token_of(p, pr);
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (r < nrows && c < chunks)
                v = *reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + (long long)(s.t0 + ti) * p.q_ts +
                                                     (long long)(sc.h * p.G + pr - ti * p.G) * p.q_hs + c * 4);
            *reinterpret_cast<float4*>(s_q + (r * 2 + c / (CPR / 2)) * Gm::QH + c % (CPR / 2) * 4) = v;
        }
        if (threadIdx.x < kRows) {
            const int r = threadIdx.x, pr = rbase + min(r, nrows - 1), ti = token_of(p, pr), h = sc.h * p.G + pr - ti * p.G;
            int lo, hi;
            rows.pos[r] = s.len - s.n + ti;
            visible_keys(p, rows.pos[r], s.len, lo, hi);
            rows.lo[r] = r < nrows ? lo : 0;
            rows.hi[r] = r < nrows ? hi : 0;
            rows.slope[r] = p.slopes ? __ldg(p.slopes + h) * kLog2e : 0.0f;
        }
        __syncthreads();
        // keys that every row sees (bounds ascend with the row)
        const int alo = rows.lo[nrows - 1], ahi = rows.hi[0];

        float2 o[kRows / 2][VEC];
        float m[kRows / 4], l[kRows / 4];        // of rows r (4 rows), (lane / 4) % 4 + 4 r (more)
#pragma unroll
        for (int r = 0; r < kRows / 4; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.0f;
        }
#pragma unroll
        for (int r = 0; r < kRows / 2; ++r) {
#pragma unroll
            for (int u = 0; u < VEC; ++u) o[r][u] = make_float2(0.0f, 0.0f);
        }
        // the first STAGES - 1 rounds only fill the ring
        int slot = 0, fill = 0;
#pragma unroll 1
        for (int t = k0 - (STAGES - 1); t < k1; ++t) {
            if (t >= k0) {
                cp_wait<STAGES - 2>();
                __syncwarp();
            }
            issue_next(t + STAGES - 1, fill);                   // the stage read last time
            fill = fill + 1 == STAGES ? 0 : fill + 1;
            if (t < k0) continue;
            const unsigned char* kb = mine + slot * Gm::STEP;
            const unsigned char* vb = kb + 16 * ROWB;
            slot = slot + 1 == STAGES ? 0 : slot + 1;
            const int j0 = t * Gm::TILE + warp * 16;
            if (j0 >= uhi || j0 <= ulo - 16) continue;
            const bool full = j0 >= alo && j0 <= ahi - 16;

            // as many rows as the unit has, in fours
            if (nrows <= 4) f32_step<DP, MOD, 4>(kb, vb, s_q, s_p[warp], s_f[warp], rows, mod, j0, full, o, m, l);
            else if (nrows <= 8) f32_step<DP, MOD, 8>(kb, vb, s_q, s_p[warp], s_f[warp], rows, mod, j0, full, o, m, l);
            else f32_step<DP, MOD, 16>(kb, vb, s_q, s_p[warp], s_f[warp], rows, mod, j0, full, o, m, l);
        }
        cp_wait<0>();
        __syncthreads();

        // ---- the warps' results meet in the ring ------------------------------
        float* red = reinterpret_cast<float*>(ring);            // [warp][row][DP]
        const int lg_rl = nrows <= 4 ? 0 : nrows <= 8 ? 1 : 2;
#pragma unroll
        for (int r = 0; r < kRows / 4; ++r) {
            l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 1);
            l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 2);
            if (nrows <= 4) {
                l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 4);
                l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 8);
                if (lane == 0) { s_m[warp][r] = m[r]; s_l[warp][r] = l[r]; }
            } else {
                l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 16);
                const int at_row = (lane >> 2 & 3) + 4 * r;
                if ((lane & 0x13) == 0) { s_m[warp][at_row] = m[r]; s_l[warp][at_row] = l[r]; }
            }
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (r >= 4 << lg_rl) break;         // places no step filled
            float* d = red + (warp * kRows + (r >> lg_rl) + 4 * (r & ((1 << lg_rl) - 1))) * DP;
            float e[VEC];
#pragma unroll
            for (int u = 0; u < VEC; ++u) e[u] = r % 2 ? o[r / 2][u].y : o[r / 2][u].x;
            if constexpr (VEC == 2) {
                *reinterpret_cast<float2*>(d + lane * 2) = make_float2(e[0], e[1]);
            } else {
#pragma unroll
                for (int u = 0; u < VEC; u += 4)
                    *reinterpret_cast<float4*>(d + (lane + u * 8) * 4) = make_float4(e[u], e[u + 1], e[u + 2], e[u + 3]);
            }
        }
        __syncthreads();
        const bool part = sc.shared();
        float* slot_o = part ? attn_slot(p, blockIdx.x, sc.w0 >= sc.us ? 0 : 1, kRows) : nullptr;
        auto store = [&](int r, int d, float4 v, float mm, float ll) {
            const int pr = rbase + r, ti = token_of(p, pr), h = sc.h * p.G + pr - ti * p.G;
            const long long row = s.t0 + ti;
            if (ll == 0.0f) v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
            float* to = static_cast<float*>(p.out) + row * p.o_ts + (long long)h * p.o_hs + d;
            to[0] = v.x * inv; to[1] = v.y * inv; to[2] = v.z * inv; to[3] = v.w * inv;
            if (d == 0 && p.lse) p.lse[row * p.Hq + h] = ll == 0.0f ? -INFINITY : (mm + log2f(ll)) * kLn2;
        };
#pragma unroll 1
        for (int x = threadIdx.x; x < nrows * (DP / 4); x += NTH) {
            const int r = x / (DP / 4), d = (x % (DP / 4)) * 4;
            if (d >= p.D) continue;
            float mm = s_m[0][r];
#pragma unroll
            for (int w = 1; w < WARPS; ++w) mm = fmaxf(mm, s_m[w][r]);
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            float ll = 0.0f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                const float f = part_weight(s_m[w][r], s_l[w][r], mm);
                const float4 u = *reinterpret_cast<const float4*>(red + (w * kRows + r) * DP + d);
                v.x = fmaf(u.x, f, v.x); v.y = fmaf(u.y, f, v.y); v.z = fmaf(u.z, f, v.z); v.w = fmaf(u.w, f, v.w);
                ll = fmaf(s_l[w][r], f, ll);
            }
            if (part) {
                __stcg(reinterpret_cast<float4*>(slot_o + r * p.D + d), v);
                if (d == 0) { __stcg(slot_o + kRows * p.D + r, mm); __stcg(slot_o + kRows * p.D + kRows + r, ll); }
            } else {
                store(r, d, v, mm, ll);
            }
        }
        if (part && attn_arrive(p, sc, &s_flag)) attn_join<NTH>(p, sc, nrows, ring, store);
        __syncthreads();
        sc.next(p);
    }
}

template <int DP, bool MOD> cudaError_t launch_dm(const AttnParams& p, cudaStream_t st) {
    using Gm = F32Geom<DP>;
    static std::atomic<unsigned> configured{0};
    auto kern = attn_f32_kernel<DP, MOD>;
    const cudaError_t e = allow_smem(kern, configured, Gm::SMEM);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, dim3((unsigned)(std::min(api_sms(), 148) * Gm::PER_SM)), dim3(Gm::WARPS * 32), Gm::SMEM, st, p,
                            page_shift_of(p.page));
}

template <int DP> cudaError_t launch_d(const AttnParams& p, cudaStream_t st) {
    return p.softcap > 0.0f || p.slopes ? launch_dm<DP, true>(p, st) : launch_dm<DP, false>(p, st);
}

}  // namespace

cudaError_t launch_attn_f32(const AttnParams& p, cudaStream_t st) {
    return p.D <= 64 ? launch_d<64>(p, st) : p.D <= 128 ? launch_d<128>(p, st) : launch_d<256>(p, st);
}

}  // namespace qmv
