// qmv_attn_few.cu -- attention over a paged cache for few query rows a kv head
// (one-token decode, drafted tokens): 16-bit types.
//
// Bound by the keys and values, which are read once per kv head: a unit's 16 packed
// rows (the G query heads of 16 / G tokens) share them.
//  * Each of the 4 warps streams its own 16 of a tile's 64 keys through its own
//    ring in shared memory (cp.async, 16-byte chunks, XOR-swizzled so that
//    ldmatrix is free of conflicts); a warp waits only for its own copies, and
//    no block-wide barrier lies inside the key loop.  2 blocks an SM keep about
//    190 KB in flight (D = 128), four times what the latency needs.
//  * S = Q K^T and O += P V run on mma.sync m16n8k16 (fp32 accumulators in
//    registers): 16 rows is the whole problem, so the 128-row tcgen05 tiles would be
//    7/8 empty, and at 16 rows the products take a fifth of the copy's time.
//  * The running maximum, the weights' sum and the output are per warp, and meet
//    once per unit in shared memory.  The output is rescaled only when a maximum
//    grows.  The weights are rounded to the element type for the second
//    product (their sum is not): the error is that of rounding the output.  For
//    f16 they are taken times 2^15, so that the row's largest is 2^15 and those down
//    to 2^-29 of it keep all their bits (as they are, 2^-14 would be the end, and a
//    long tail below 2^-25 of a large weight would be lost from the output but not
//    from the sum).
//  * The heads' dims are padded to DP = 64, 128 or 256 with zeros in shared
//    memory only.
// Measured (bf16, 32 query and 8 kv heads of 128): one token over 131001 keys 93 us =
// 5.8 TB/s, 90 % of a copy's rate; 64 tokens over 300-8000 keys each 185 us, 90 %;
// one token over 517 keys 12.6 us, all latency.  64 tokens of 16 heads on 4 of 256:
// 220 us = 4.9 TB/s (one block an SM; that form spills 34 bytes a thread, 70 with cap
// or bias).
#include <limits.h>

#include <algorithm>

#include "qmv_attn_mma.cuh"
#include "qmv_attn_sched.cuh"

namespace qmv {

namespace {

constexpr int kRows = 16;

// WARPS 4: two blocks an SM (one at DP = 256); 8: one, for batches of fewer units
// than SMs, whose blocks then take 128 keys a step.
template <int DP, int WARPS> struct FewGeom {
    static constexpr int TILE = 16 * WARPS;                // keys of a tile, 16 a warp
    static constexpr int STAGES = DP == 64 ? 6 : 3;
    static constexpr int PER_SM = DP == 256 || WARPS == 8 ? 1 : 2;
    static constexpr int ROWB = DP * 2;                    // bytes of a key in shared memory
    static constexpr int STEP = 2 * 16 * ROWB;             // a warp's K and V of one tile
    static constexpr int RING = WARPS * STAGES * STEP;
};
static_assert(4 * kRows * 256 * 4 <= FewGeom<256, 4>::RING && 4 * kRows * 64 * 4 <= FewGeom<64, 4>::RING, "joined in the ring");
static_assert(kJoinBytes <= FewGeom<64, 4>::RING, "joined in the ring");

template <class T, int DP, int WARPS, bool MOD>
__global__ void __launch_bounds__(WARPS * 32, FewGeom<DP, WARPS>::PER_SM) attn_few_kernel(const __grid_constant__ AttnParams p,
                                                                                       int page_shift) {
    using Gm = FewGeom<DP, WARPS>;
    constexpr int STAGES = Gm::STAGES, ROWB = Gm::ROWB, KS = DP / 16, NT = DP / 8, CPR = DP / 8;
    extern __shared__ __align__(1024) unsigned char ring[];
    __shared__ SchedSmem sm;
    __shared__ float s_m[WARPS][kRows], s_l[WARPS][kRows];
    __shared__ int s_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gid = lane >> 2, tig = lane & 3;
    unsigned char* mine = ring + warp * STAGES * Gm::STEP;
    const uint32_t mine_a = s_addr(mine);
    const int chunks = p.D / 8;                     // 16-byte chunks of a head
    grid_dependency_wait();
    grid_launch_dependents();

    Sched<kRows, Gm::TILE> sc;
    sc.template init<WARPS * 32>(p, sm, 768 / Gm::TILE);
    const ScoreMod<false> mod(p);
    const float scale2 = p.scale * kLog2e;
    constexpr float kUp = __is_same(T, __half) ? 15.0f : 0.0f;      // log2 of what weights are taken times
    const int page16 = (int)(p.page_s / 8), tok16 = (int)(p.tok_s / 8);

    while (sc.live) {
        int k0, k1;
        sc.piece(k0, k1);
        const SeqInfo s = sc.s;
        const int rbase = sc.i * kRows, nrows = min(kRows, s.n * p.G - rbase);
        int ulo, uhi;                               // keys that any row of the unit sees
        rows_keys(p, s, rbase, rbase + nrows - 1, ulo, uhi);
        // this lane's chunk of the head's rows
        const char* kl = static_cast<const char*>(p.k) + (long long)sc.h * p.head_s * 2 + lane % CPR * 16;
        const char* vl = static_cast<const char*>(p.v) + (long long)sc.h * p.head_s * 2 + lane % CPR * 16;
        const int* trow = p.table + (long long)sc.b * p.max_pages;

        // lanes r and r + 16: place of key r of this warp's step t, in units of 16
        // bytes; -1 outside the unit's keys, -2 on a bad page
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
#pragma unroll
                    for (int u = 0; u < 16 * CPR / 32; ++u) {
                        const int id = u * 32 + lane, r = id / CPR, c = id % CPR;
                        const long long off = (long long)__shfl_sync(0xFFFFFFFFu, at, r) * 16;
                        const uint32_t d = base + r * ROWB + ((c ^ (r & 7)) << 4);
                        cp16(d, kl + off);
                        cp16(d + 16 * ROWB, vl + off);
                    }
                } else {
#pragma unroll 2
                    for (int u = 0; u < 16 * CPR / 32; ++u) {
                        const int id = u * 32 + lane, r = id / CPR, c = id % CPR;
                        const int a = __shfl_sync(0xFFFFFFFFu, at, r);
                        const uint32_t d = base + r * ROWB + ((c ^ (r & 7)) << 4);
                        const bool rd = a >= 0 && c < chunks;
                        const long long off = rd ? (long long)a * 16 : -16 * c;
                        cp16_or_zero(d, kl + off, rd);
                        cp16_or_zero(d + 16 * ROWB, vl + off, rd);
                    }
                    if (__any_sync(0xFFFFFFFFu, at == -2)) {        // keys of NaN, once the copies have landed
                        cp_commit();
                        cp_wait<0>();
                        __syncwarp();
                        if (lane < 16 && at == -2)
                            *reinterpret_cast<uint4*>(mine + slot * Gm::STEP + lane * ROWB + ((lane & 7) << 4)) =
                                make_uint4(~0u, ~0u, ~0u, ~0u);
                        return;
                    }
                }
            }
            cp_commit();
        };

        // ---- queries: A fragments, rows gid and gid + 8 ---------------------
        uint32_t qf[KS][4];
        int lo[2], hi[2], pos[2];
        float slope[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = gid + 8 * e;
            const bool in = r < nrows;
            const int pr = rbase + (in ? r : 0), ti = token_of(p, pr), h = sc.h * p.G + pr - ti * p.G;
            pos[e] = s.len - s.n + ti;
            visible_keys(p, pos[e], s.len, lo[e], hi[e]);
            if (!in) lo[e] = hi[e] = 0;
            slope[e] = MOD && p.slopes ? __ldg(p.slopes + h) * kLog2e : 0.0f;
            const T* qr = static_cast<const T*>(p.q) + (long long)(s.t0 + ti) * p.q_ts + (long long)h * p.q_hs;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int d = k * 16 + u * 8 + tig * 2;
                    qf[k][e + 2 * u] = in && d < p.D ? *reinterpret_cast<const uint32_t*>(qr + d) : 0u;
                }
            }
        }
        // keys that every row sees: no masks there
        int alo = max(lo[0], nrows > gid + 8 ? lo[1] : 0), ahi = min(gid < nrows ? hi[0] : INT_MAX, gid + 8 < nrows ? hi[1] : INT_MAX);
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) {
            alo = max(alo, __shfl_xor_sync(0xFFFFFFFFu, alo, w));
            ahi = min(ahi, __shfl_xor_sync(0xFFFFFFFFu, ahi, w));
        }
        float o[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

        // places of the next AHEAD steps to issue: the table's latency is behind
        // as many steps
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
        // The first STAGES - 1 rounds only fill the ring.  (One copy of the code for
        // them too: unrolled fills made the kernel 160 KB, and a short call waited
        // for its instructions.)
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
            const uint32_t kb = mine_a + slot * Gm::STEP, vb = kb + 16 * ROWB;
            slot = slot + 1 == STAGES ? 0 : slot + 1;
            const int j0 = t * Gm::TILE + warp * 16;
            if (j0 >= uhi || j0 <= ulo - 16) continue;

            // ---- S = Q K^T: 16 rows x 16 keys ---------------------------------
            float sa[2][4] = {}, sb[2][4] = {};     // two chains of half the dims
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint32_t f[4];                      // keys 0-7 / 8-15 x dims 0-7 / 8-15
                const int r = (lane & 7) + ((lane >> 4) << 3), c = 2 * k + ((lane >> 3) & 1);
                ldsm4(kb + r * ROWB + ((c ^ (r & 7)) << 4), f);
                if (k & 1) {
                    mma<T>(sb[0], qf[k], f[0], f[1]);
                    mma<T>(sb[1], qf[k], f[2], f[3]);
                } else {
                    mma<T>(sa[0], qf[k], f[0], f[1]);
                    mma<T>(sa[1], qf[k], f[2], f[3]);
                }
            }
            // element (n, 2e + u): row gid + 8 e, key j0 + 8 n + 2 tig + u
            const bool full = j0 >= alo && j0 <= ahi - 16;
            float mx[2] = {m[0], m[1]};
            float sc8[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) sc8[x] = sa[x / 4][x % 4] + sb[x / 4][x % 4];
            if constexpr (MOD) mod.scaled(sc8);
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int e = x >> 1, j = j0 + 8 * n + 2 * tig + (x & 1);
                    if constexpr (MOD) sa[n][x] = fmaf(slope[e], (float)(j - pos[e]), sc8[4 * n + x]);
                    else sa[n][x] = __fmul_rn(sc8[4 * n + x], scale2);     // rounded alike for the maximum and the weight
                }
            if (!full) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int e = x >> 1, j = j0 + 8 * n + 2 * tig + (x & 1);
                        if (j < lo[e] || j >= hi[e]) sa[n][x] = -INFINITY;
                    }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e)
                mx[e] = fmaxf(fmaxf(fmaxf(sa[0][2 * e], sa[0][2 * e + 1]), fmaxf(sa[1][2 * e], sa[1][2 * e + 1])), mx[e]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xFFFFFFFFu, mx[e], 1));
                mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xFFFFFFFFu, mx[e], 2));
            }
            if (__any_sync(0xFFFFFFFFu, mx[0] > m[0] || mx[1] > m[1])) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float f = m[e] == -INFINITY ? 0.0f : ex2(m[e] - mx[e]);
                    l[e] *= f;
#pragma unroll
                    for (int n = 0; n < NT; ++n) { o[n][2 * e] *= f; o[n][2 * e + 1] *= f; }
                    m[e] = mx[e];
                }
            }
            const float base[2] = {m[0] == -INFINITY ? 0.0f : m[0], m[1] == -INFINITY ? 0.0f : m[1]};
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    // (m + 15 is not the same: scores of 2^24 and more would round it)
                    sa[n][x] = ex2((sa[n][x] - base[x >> 1]) + kUp);
                    l[x >> 1] += sa[n][x];
                }
            // ---- O += P V -----------------------------------------------------
            // Where some rows see a key and others do not, an infinite or NaN
            // value must not reach the others through 0 * v: such a step (no
            // finite model makes one) adds key by key.
            bool odd = false;
            if (!full) {
#pragma unroll 1
                for (int u = 0; u < 16 * CPR / 32; ++u) {
                    const uint4 w = *reinterpret_cast<const uint4*>(mine + (vb - mine_a) + (u * 32 + lane) * 16);
                    odd |= odd_word<T>(w.x) || odd_word<T>(w.y) || odd_word<T>(w.z) || odd_word<T>(w.w);
                }
                odd = __any_sync(0xFFFFFFFFu, odd);
            }
            if (!odd) {
                uint32_t pf[4] = {pack2<T>(sa[0][0], sa[0][1]), pack2<T>(sa[0][2], sa[0][3]),
                                  pack2<T>(sa[1][0], sa[1][1]), pack2<T>(sa[1][2], sa[1][3])};
#pragma unroll
                for (int n = 0; n < NT; n += 2) {
                    uint32_t f[4];                  // keys 0-7 / 8-15 of dims 8n.., then of the next 8
                    const int r = lane & 15, c = n + (lane >> 4);
                    ldsm4t(vb + r * ROWB + ((c ^ (r & 7)) << 4), f);
                    mma<T>(o[n], pf, f[0], f[1]);
                    mma<T>(o[n + 1], pf, f[2], f[3]);
                }
            } else {
#pragma unroll 1
                for (int k = 0; k < 16; ++k) {
                    const int j = j0 + k, src = (lane & ~3) | ((k & 7) >> 1);
                    const float c0 = k & 8 ? (k & 1 ? sa[1][1] : sa[1][0]) : (k & 1 ? sa[0][1] : sa[0][0]);
                    const float c1 = k & 8 ? (k & 1 ? sa[1][3] : sa[1][2]) : (k & 1 ? sa[0][3] : sa[0][2]);
                    const float p0 = __shfl_sync(0xFFFFFFFFu, c0, src), p1 = __shfl_sync(0xFFFFFFFFu, c1, src);
                    const bool v0 = j >= lo[0] && j < hi[0], v1 = j >= lo[1] && j < hi[1];
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float2 w = unpack2<T>(*reinterpret_cast<const uint32_t*>(
                            mine + (vb - mine_a) + k * ROWB + ((n ^ (k & 7)) << 4) + tig * 4));
                        if (v0) { o[n][0] = fmaf(p0, w.x, o[n][0]); o[n][1] = fmaf(p0, w.y, o[n][1]); }
                        if (v1) { o[n][2] = fmaf(p1, w.x, o[n][2]); o[n][3] = fmaf(p1, w.y, o[n][3]); }
                    }
                }
            }
        }
        cp_wait<0>();
        __syncthreads();

        // ---- the warps' results meet in the ring ------------------------------
        float* red = reinterpret_cast<float*>(ring);            // [warp][row][DP]
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], 1);
            l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], 2);
            // what the weights are relative to, from here on
            if (tig == 0) { s_m[warp][gid + 8 * e] = m[e] - kUp; s_l[warp][gid + 8 * e] = l[e]; }
#pragma unroll
            for (int n = 0; n < NT; ++n)
                *reinterpret_cast<float2*>(red + (warp * kRows + gid + 8 * e) * DP + n * 8 + tig * 2) =
                    make_float2(o[n][2 * e], o[n][2 * e + 1]);
        }
        __syncthreads();
        const bool part = sc.shared();
        float* slot_o = part ? attn_slot(p, blockIdx.x, sc.w0 >= sc.us ? 0 : 1, kRows) : nullptr;
        auto store = [&](int r, int d, float4 v, float mm, float ll) {
            const int pr = rbase + r, ti = token_of(p, pr), h = sc.h * p.G + pr - ti * p.G;
            const long long row = s.t0 + ti;
            const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;    // no key: 0 even where a sum is not a number
            if (ll == 0.0f) v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            T* to = static_cast<T*>(p.out) + row * p.o_ts + (long long)h * p.o_hs + d;
            st_elem(to, v.x * inv); st_elem(to + 1, v.y * inv); st_elem(to + 2, v.z * inv); st_elem(to + 3, v.w * inv);
            if (d == 0 && p.lse) p.lse[row * p.Hq + h] = ll == 0.0f ? -INFINITY : (mm + log2f(ll)) * kLn2;
        };
#pragma unroll 1
        for (int x = threadIdx.x; x < nrows * (DP / 4); x += WARPS * 32) {
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
        if (part && attn_arrive(p, sc, &s_flag)) attn_join<WARPS * 32>(p, sc, nrows, ring, store);
        __syncthreads();
        sc.next(p);
    }
}

template <class T, int DP, int WARPS, bool MOD> cudaError_t launch_tdm(const AttnParams& p, cudaStream_t st) {
    using Gm = FewGeom<DP, WARPS>;
    static std::atomic<unsigned> configured{0};
    auto kern = attn_few_kernel<T, DP, WARPS, MOD>;
    const cudaError_t e = allow_smem(kern, configured, Gm::RING);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, dim3((unsigned)(std::min(api_sms(), 148) * Gm::PER_SM)), dim3(WARPS * 32), Gm::RING, st, p,
                            page_shift_of(p.page));
}

template <class T, int DP, int WARPS> cudaError_t launch_tdw(const AttnParams& p, cudaStream_t st) {
    return p.softcap > 0.0f || p.slopes ? launch_tdm<T, DP, WARPS, true>(p, st) : launch_tdm<T, DP, WARPS, false>(p, st);
}

template <class T, int DP> cudaError_t launch_td(const AttnParams& p, long long units, cudaStream_t st) {
    if constexpr (DP < 256) {
        // Fewer units than SMs: a short call's time is its steps' latency, and 8
        // warps halve the steps (517 keys: 12.4 us, 15.5 with 4); a long one has fewer
        // parts to join.  More units: two blocks an SM fill each other's gaps.
        if (units <= api_sms()) return launch_tdw<T, DP, 8>(p, st);
    }
    return launch_tdw<T, DP, 4>(p, st);
}

template <class T> cudaError_t launch_t(const AttnParams& p, long long units, cudaStream_t st) {
    return p.D <= 64 ? launch_td<T, 64>(p, units, st) : p.D <= 128 ? launch_td<T, 128>(p, units, st) : launch_td<T, 256>(p, units, st);
}

}  // namespace

cudaError_t launch_attn_few(int dtype, const AttnParams& p, int max_q_len, cudaStream_t st) {
    const long long units = (long long)p.n_seqs * p.Hkv * (((long long)max_q_len * p.G + kRows - 1) / kRows);
    return dtype == 1 ? launch_t<__half>(p, units, st) : launch_t<__nv_bfloat16>(p, units, st);
}

}  // namespace qmv
