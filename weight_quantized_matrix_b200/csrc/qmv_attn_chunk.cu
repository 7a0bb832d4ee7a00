// qmv_attn_chunk.cu -- attention over a paged cache for many query rows a kv
// head (chunks of new tokens): 16-bit types, heads of up to 128 dims, on the
// 5th-generation tensor cores.
//
// Bound by the products (4 D flops a pair of row and key) and, at the same size, by
// the exponentials (one a pair: 16 a clock and SM, so a 128 x 128 tile takes
// 1024 clocks, as its two products do at D = 128; at D = 64 twice as long).
//
// One block an SM, 384 threads; a unit is 256 packed rows in two halves of 128:
//   warps 0-3, 4-7  softmax of half 0 / 1: thread = row.  S is read from tensor
//              memory (tcgen05.ld), the weights are written back over it in the
//              element type as the second product's A operand.
//   warp 8     lane 0 issues tcgen05.mma: S_h = Q_h K^T (A, B shared, 128-byte
//              swizzle), O_h += P_h V (A tensor memory, B shared, V as it
//              lies: dims contiguous, the MN-major form).  While one half's
//              softmax runs, the tensor cores do the other half's products.
//   warps 9-11 copy K and V: tiles all of whose keys are seen by some row go by
//              tensor copies, one a page (or 128 rows) and 64 dims, where pages are
//              powers of two from 8 up; other pages, and the tiles at the ends,
//              go by cp.async, 16 bytes at a time, with zeros for keys no row
//              sees.  Q goes by cp.async.
// Tensor memory: S_0 S_1 (128 columns each, P_h in the lower half of S_h), O_0 O_1.
// K and V tiles of 128 keys alternate in a ring of 5 slots.
//
// The running maximum is only raised when a row's new maximum exceeds it by 2^8:
// softmax is invariant to the reference that is subtracted, and with a slack of
// 8 in log2 neither the weights (<= 256) nor their fp32 sums can overflow; the
// output is rescaled in tensor memory, rarely, by the softmax warps themselves.
// The weights are rounded to the element type for the second product, their
// sum is not: an error of the size of the output's own rounding.
//
// Every wait is bounded (about one second); one that runs out ORs a code into
// the fault word (1: softmax, 2: copies, 8: products), raises a flag that ends
// every other wait, and the block frees its tensor memory and ends.
#include <limits.h>

#include <algorithm>

#include "qmv_attn_mma.cuh"
#include "qmv_attn_sched.cuh"

namespace qmv {

namespace {

constexpr int kThreads = 384;
constexpr int kRows = 256, kHalf = 128;
constexpr int kTile = 128;
constexpr int kLoaders = 3;                  // warps
constexpr int kSoftRegs = 216, kOtherRegs = 72;      // 256 x 216 + 128 x 72 = 384 x 168
constexpr float kSlack = 8.0f;               // log2

template <int DP> struct ChunkGeom {
    static constexpr int SLOT = kTile * DP * 2;                 // bytes of a K or V tile
    static constexpr int SLOTS = DP == 64 ? 8 : 5;
    static constexpr int QB = kHalf * DP * 2;                   // bytes of half a unit's queries
    static constexpr int RING = 2 * QB;                         // ring's place
    static constexpr int SMEM = RING + SLOTS * SLOT + 1024;     // slack to round the base up to 1024
};

struct Bars {
    uint64_t kv_full[8], kv_empty[8], q_full, q_empty, s_full[2], p_full[2], pv_done[2], drain;
    uint32_t tmem;
    volatile int abort;
    int skip[2];             // this step's second product was done by the softmax warps
    int flag[2];
};

struct ChunkArgs {
    CUtensorMap kmap, vmap;  // the cache as boxes of 64 dims x box_rows rows of a page
    int box_rows;            // 0: no boxes (pages that are no power of two, or below 8 rows)
    int page_shift;          // log2 of the page, -1 if it is no power of two
    int out_vec;             // 16-byte stores
};

// The wait of every role: false once the block has given up.
struct Waiter {
    Bars* b;
    unsigned* fault;
    unsigned code;
    bool ok;
    __device__ __forceinline__ bool operator()(const uint64_t& bar, uint32_t parity) {
        if (!ok) return false;
        const uint32_t a = s_addr(&bar);
        if (mbar_try_sleep(a, parity)) return true;
        const uint64_t t0 = now_ns();
        for (;;) {
            if (mbar_try_sleep(a, parity)) return true;
            if (b->abort || now_ns() - t0 > kWaitNs) {
                if (!b->abort && fault) atomicOr(fault, code);
                b->abort = 1;
                return ok = false;
            }
        }
    }
};

// The same for a whole warp, with one answer.
__device__ __forceinline__ bool warp_wait(Waiter& w, const uint64_t& bar, uint32_t parity) {
    const bool r = w(bar, parity);
    return w.ok = __all_sync(0xFFFFFFFFu, r);
}

// Key tiles of half h inside the unit's piece [k0, k1).
__device__ __forceinline__ void half_tiles(const AttnParams& p, const SeqInfo& s, int rbase, int h, int k0, int k1, int& a,
                                           int& b) {
    const int r0 = rbase + h * kHalf, r1 = min(r0 + kHalf, s.n * p.G) - 1;
    a = b = k0;
    if (r0 > r1) return;
    int lo, hi;
    rows_keys(p, s, r0, r1, lo, hi);
    a = max(k0, lo / kTile);
    b = min(k1, (hi + kTile - 1) / kTile);
    if (a >= b) a = b = k0;
}

template <class T, int DP, bool MOD>
__global__ void __launch_bounds__(kThreads, 1) attn_chunk_kernel(const __grid_constant__ AttnParams p,
                                                                 const __grid_constant__ ChunkArgs g) {
    using Gm = ChunkGeom<DP>;
    constexpr int CPR = DP / 8, SLOTS = Gm::SLOTS;
    extern __shared__ unsigned char raw[];
    unsigned char* smem = raw + ((1024u - (s_addr(raw) & 1023u)) & 1023u);
    __shared__ Bars bars;
    __shared__ SchedSmem sm;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t q_a = s_addr(smem), ring_a = q_a + Gm::RING;

    if (threadIdx.x == 0) {
        for (int i = 0; i < SLOTS; ++i) { mbar_init1(&bars.kv_full[i], kLoaders); mbar_init1(&bars.kv_empty[i], 1); }
        mbar_init1(&bars.q_full, kLoaders);
        mbar_init1(&bars.q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init1(&bars.s_full[i], 1);
            mbar_init1(&bars.p_full[i], 4);
            mbar_init1(&bars.pv_done[i], 1);
            bars.skip[i] = 0;
        }
        mbar_init1(&bars.drain, 1);
        bars.abort = 0;
        fence_mbar_init();
    }
    if (warp == 8) tm_alloc(s_addr(&bars.tmem), 512);
    grid_dependency_wait();
    grid_launch_dependents();
    tc_before();
    __syncthreads();
    tc_after();
    constexpr uint32_t tm = 0;                   // all 512 columns: tensor memory's start

    Sched<kRows, kTile> sc;
    sc.init<kThreads, 32>(p, sm, 4);

    if (warp >= 8) {
        reg_dec<kOtherRegs>();
        if (warp == 8) {
            // ------------------------------------------------ the products ----
            // The whole warp walks through this with the same values, so that
            // descriptors live in uniform registers; one lane issues.  (With one
            // lane in the loop alone the issue took 150 clocks a product.)
            Waiter wait{&bars, p.fault, 8u, true};
            constexpr uint32_t FMT = __is_same(T, __half) ? 0u : 1u;
            constexpr uint32_t ID_S = (1u << 4) | (FMT << 7) | (FMT << 10) | ((kTile / 8u) << 17) | (8u << 24);
            constexpr uint32_t ID_O = (1u << 4) | (FMT << 7) | (FMT << 10) | (1u << 16) | ((DP / 8u) << 17) | (8u << 24);
            const uint32_t q_d = desc_lo(q_a, 16), ring_k = desc_lo(ring_a, 16), ring_v = desc_lo(ring_a, 128 * 128);
            constexpr uint32_t HI = desc_hi(1024);
            const bool one = elect_one();
            int n = 0;                              // tiles of K and V taken from the ring so far
            int npiece = 0;
            int pv[2] = {0, 0}, pf[2] = {0, 0};      // products O and weights P so far
            auto full = [&](int x) { return warp_wait(wait, bars.kv_full[x % SLOTS], (uint32_t)(x / SLOTS) & 1u); };
            auto release = [&](int x) { if (one) commit(&bars.kv_empty[x % SLOTS]); };
            auto qk = [&](int h, int x) {
                // S_h is free once the product that read its weights is done
                if (pv[h] > 0 && !warp_wait(wait, bars.pv_done[h], (uint32_t)(pv[h] - 1) & 1u)) return;
                tc_after();
                const uint32_t a = q_d + h * (Gm::QB / 16), b = ring_k + x % SLOTS * (Gm::SLOT / 16);
                if (one) {
#pragma unroll
                    for (int k = 0; k < DP / 16; ++k) {
                        const uint32_t o = ((k / 4) * (128 * 128) + (k % 4) * 32) / 16;
                        mma_ss(h * 128, a + o, b + o, HI, ID_S, k > 0);
                    }
                    commit(&bars.s_full[h]);
                }
            };
            while (sc.live && wait.ok) {
                int k0, k1, a[2], b[2];
                sc.piece(k0, k1);
                for (int h = 0; h < 2; ++h) half_tiles(p, sc.s, sc.i * kRows, h, k0, k1, a[h], b[h]);
                if (k0 < k1) {
                    if (!warp_wait(wait, bars.q_full, (uint32_t)npiece & 1u)) break;
                    if (!full(2 * n)) break;
                    tc_after();
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (a[h] <= k0 && k0 < b[h]) qk(h, 2 * n);
                    release(2 * n);
                    if (k1 - k0 == 1 && one) commit(&bars.q_empty);
                    for (int j = k0; j < k1; ++j, ++n) {
                        const bool more = j + 1 < k1;
                        if (!full(2 * n + 1)) break;
                        if (more && !full(2 * n + 2)) break;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (a[h] <= j && j < b[h]) {
                                if (!warp_wait(wait, bars.p_full[h], (uint32_t)pf[h]++ & 1u)) break;
                                tc_after();
                                const bool skip = *(volatile int*)&bars.skip[h] != 0;
                                const uint32_t v = ring_v + (2 * n + 1) % SLOTS * (Gm::SLOT / 16);
                                if (one) {
                                    if (!skip) {
                                        const bool acc = j > a[h];
#pragma unroll
                                        for (int k = 0; k < kTile / 16; ++k)
                                            mma_ts(256 + h * DP, h * 128 + k * 8, v + k * (16 * 128 / 16), HI, ID_O, acc || k > 0);
                                    }
                                    commit(&bars.pv_done[h]);
                                }
                                ++pv[h];
                            }
                            if (more && a[h] <= j + 1 && j + 1 < b[h]) qk(h, 2 * n + 2);
                        }
                        if (!wait.ok) break;
                        release(2 * n + 1);
                        if (more) release(2 * n + 2);
                        if (j + 2 == k1 && one) commit(&bars.q_empty);
                    }
                    ++npiece;
                }
                if (wait.ok) sc.next(p);
            }
            // nothing of this block's is in flight when it ends
            if (one) commit(&bars.drain);
            const uint64_t t0 = now_ns();
            while (!mbar_try_sleep(s_addr(&bars.drain), 0u) && now_ns() - t0 < kWaitNs) {}
            __syncwarp();
        } else {
            // -------------------------------------------------- the copies ----
            Waiter wait{&bars, p.fault, 2u, true};
            const int w = warp - 9;
            const int chunks = p.D / 8;
            const int page16 = (int)(p.page_s / 8), tok16 = (int)(p.tok_s / 8);
            constexpr int PER = 8 * CPR / 32;            // copies a lane makes of 8 rows
            constexpr int LAG = 2;                       // slots in flight behind the one being issued
            int filled = 0, told = 0;                    // slots filled, slots reported full
            auto tell = [&]() {
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive1(&bars.kv_full[told % SLOTS]);
                ++told;
            };
            // boxes: pieces of box_rows rows x 64 dims, shared out over warps and lanes
            const bool boxes = g.box_rows > 0;
            const int pieces = boxes ? kTile / g.box_rows : 0, items = pieces * (DP / 64), item = lane * kLoaders + w;
            const uint32_t my_bytes = (uint32_t)((items - w + kLoaders - 1) / kLoaders) * g.box_rows * 128u;
            auto tell_all = [&]() {
                cp_wait<0>();
                while (told < filled) tell();
            };
            int npiece = 0;
            while (sc.live && wait.ok) {
                int k0, k1;
                sc.piece(k0, k1);
                if (k0 < k1) {
                    const SeqInfo s = sc.s;
                    const int rbase = sc.i * kRows, nrows = min(kRows, s.n * p.G - rbase);
                    int ulo, uhi;
                    rows_keys(p, s, rbase, rbase + nrows - 1, ulo, uhi);
                    const char* kl = static_cast<const char*>(p.k) + (long long)sc.h * p.head_s * 2 + lane % CPR * 16;
                    const char* vl = static_cast<const char*>(p.v) + (long long)sc.h * p.head_s * 2 + lane % CPR * 16;
                    const int* trow = p.table + (long long)sc.b * p.max_pages;
                    // this warp's rows of a tile: the 8-row groups w, w + 3, ..
                    auto place = [&](int j0, int u) -> int {
                        const int lr = u * 32 + lane, row = (w + kLoaders * (lr >> 3)) * 8 + (lr & 7), j = j0 + row;
                        if (row >= kTile || j < ulo || j >= uhi) return -1;
                        const int e = g.page_shift >= 0 ? j >> g.page_shift : j / p.page;
                        if (e >= p.max_pages) return -2;
                        const int pg = __ldg(trow + e);
                        if ((unsigned)pg >= (unsigned)p.n_pages) return -2;
                        return pg * page16 + (j - e * p.page) * tok16;
                    };
                    // page of this lane's piece of a tile, -1 where it must go row by row
                    auto page_of = [&](int j0) -> int {
                        const int x = j0 + lane * g.box_rows;
                        if (lane >= pieces) return 0;
                        const int e = x >> g.page_shift;
                        if (j0 < ulo || j0 + kTile > uhi || e >= p.max_pages) return -1;
                        const int pg = __ldg(trow + e);
                        return (unsigned)pg < (unsigned)p.n_pages ? pg : -1;
                    };
                    int at0 = place(k0 * kTile, 0), at1 = place(k0 * kTile, 1);
                    int pg = boxes ? page_of(k0 * kTile) : -1;
                    // ---- queries, once the first products of the unit before are done ----
                    tell_all();
                    if (npiece > 0 && !warp_wait(wait, bars.q_empty, (uint32_t)(npiece - 1) & 1u)) break;
                    for (int gr = w; gr < kRows / 8; gr += kLoaders) {
                        const int r = gr * 8 + (lane & 7), pr = rbase + min(r, nrows - 1), ti = pr / p.G;
                        const long long off = ((long long)(s.t0 + ti) * p.q_ts + (long long)(sc.h * p.G + pr - ti * p.G) * p.q_hs) * 2;
#pragma unroll
                        for (int u = 0; u < PER; ++u) {
                            const int id = u * 32 + lane, rr = id / CPR, c = id % CPR, row = gr * 8 + rr;
                            const long long o = __shfl_sync(0xFFFFFFFFu, off, rr);
                            const bool rd = row < nrows && c < chunks;
                            const uint32_t d = q_a + (row / kHalf) * Gm::QB + (c / 8) * (128 * 128) + (row % kHalf) * 128 +
                                               (((c & 7) ^ (row & 7)) << 4);
                            cp16_or_zero(d, static_cast<const char*>(p.q) + (rd ? o + c * 16 : 0), rd);
                        }
                    }
                    cp_commit();
                    cp_wait<0>();
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive1(&bars.q_full);
                    ++npiece;
                    // ---- keys and values ------------------------------------------
                    for (int j = k0; j < k1 && wait.ok; ++j) {
                        const bool by_box = boxes && __all_sync(0xFFFFFFFFu, pg >= 0);
                        const int npg = boxes ? page_of((j + 1) * kTile) : -1;
                        int n0 = 0, n1 = 0;
                        if (!boxes || !__all_sync(0xFFFFFFFFu, npg >= 0)) {
                            n0 = place((j + 1) * kTile, 0);
                            n1 = place((j + 1) * kTile, 1);
                        }
                        const int my_pg = __shfl_sync(0xFFFFFFFFu, pg, item / (DP / 64) & 31);
                        for (int kv = 0; kv < 2; ++kv) {
                            const int slot = filled % SLOTS;
                            if (filled >= SLOTS) {
                                const uint32_t ph = (uint32_t)(filled / SLOTS - 1) & 1u;
                                // about to wait: what is on its way is reported first
                                if (!__all_sync(0xFFFFFFFFu, mbar_test(s_addr(&bars.kv_empty[slot]), ph))) tell_all();
                                if (!warp_wait(wait, bars.kv_empty[slot], ph)) break;
                            }
                            if (by_box) {
                                tell_all();
                                if (lane == 0) mbar_expect(&bars.kv_full[slot], my_bytes);
                                __syncwarp();
                                if (item < items) {
                                    const int piece = item / (DP / 64), blk = item % (DP / 64);
                                    box_copy(ring_a + slot * Gm::SLOT + blk * (128 * 128) + piece * g.box_rows * 128,
                                             kv ? &g.vmap : &g.kmap, blk * 64, (j * kTile + piece * g.box_rows) & (p.page - 1),
                                             sc.h, my_pg, &bars.kv_full[slot]);
                                }
                                ++filled;
                                ++told;
                                continue;
                            }
                            const uint32_t base = ring_a + slot * Gm::SLOT;
                            const char* src = kv ? vl : kl;
#pragma unroll
                            for (int gi = 0; gi < (16 + kLoaders - 1) / kLoaders; ++gi) {
                                const int gr = w + kLoaders * gi;
                                if (gr >= 16) break;
#pragma unroll
                                for (int u = 0; u < PER; ++u) {
                                    const int id = u * 32 + lane, rr = id / CPR, c = id % CPR, row = gr * 8 + rr;
                                    const int at = __shfl_sync(0xFFFFFFFFu, gi < 4 ? at0 : at1, (gi & 3) * 8 + rr);
                                    const uint32_t d = base + (c / 8) * (128 * 128) + row * 128 + (((c & 7) ^ rr) << 4);
                                    if (at == -2 && kv == 0) {
                                        st_shared16(d, ~0u);                 // a key of NaN
                                    } else {
                                        const bool rd = at >= 0 && c < chunks;
                                        cp16_or_zero(d, src + (rd ? (long long)at * 16 : -16 * c), rd);
                                    }
                                }
                            }
                            cp_commit();
                            ++filled;
                            if (filled - told > LAG) { cp_wait<LAG>(); tell(); }
                        }
                        at0 = n0;
                        at1 = n1;
                        pg = npg;
                    }
                }
                sc.next(p);
            }
            tell_all();
        }
    } else {
        // ---------------------------------------------------- the softmax ----
        reg_inc<kSoftRegs>();
        const int h = warp >> 2;                         // half
        const int r = threadIdx.x & 127;                 // row of the half = lane of tensor memory
        const uint32_t lane_base = (uint32_t)(warp & 3) << 21;      // 32 lanes a warp, lane in bits 16..
        const uint32_t ts = tm + h * 128 + lane_base, to = tm + 256 + h * DP + lane_base;
        const ScoreMod<false> mod(p);
        const float scale2 = p.scale * kLog2e;
        Waiter wait{&bars, p.fault, 1u, true};
        int ns = 0;                                      // steps of this half so far
        int n0 = 0;                                      // tiles of all pieces before this one
        // A wait that gave up does not end these warps: they go through their
        // steps (without waiting), so that the barriers among them stay paired.
        while (sc.live) {
            int k0, k1, a, b;
            sc.piece(k0, k1);
            const SeqInfo s = sc.s;
            const int rbase = sc.i * kRows + h * kHalf, nrows = min(kHalf, s.n * p.G - rbase);
            half_tiles(p, s, sc.i * kRows, h, k0, k1, a, b);
            int lo = 0, hi = 0, pos = 0, ti = 0, head = 0;
            float slope = 0.0f;
            if (r < nrows) {
                const int pr = rbase + r;
                ti = pr / p.G;
                head = sc.h * p.G + pr - ti * p.G;
                pos = s.len - s.n + ti;
                visible_keys(p, pos, s.len, lo, hi);
                if (MOD && p.slopes) slope = __ldg(p.slopes + head) * kLog2e;
            }
            int part_lo = 0, part_hi = 0;                // keys that every row of the half sees
            if (nrows > 0) {
                int x;
                visible_keys(p, s.len - s.n + rbase / p.G, s.len, x, part_hi);
                visible_keys(p, s.len - s.n + (rbase + nrows - 1) / p.G, s.len, part_lo, x);
            }
            float m = -INFINITY, l = 0.0f;
            for (int j = a; j < b; ++j, ++ns) {
                warp_wait(wait, bars.s_full[h], (uint32_t)ns & 1u);
                tc_after();
                float x[128];
#pragma unroll
                for (int c = 0; c < 128; c += 32) tm_ld32(ts + c, x + c);
                tm_wait_ld();
                const int j0 = j * kTile;
                if constexpr (MOD) {
#pragma unroll
                    for (int c = 0; c < 128; ++c) x[c] = mod.apply(x[c], slope, j0 + c - pos);
                }
                // rows past the unit have queries of zero and need no mask
                const bool full = __all_sync(0xFFFFFFFFu, r >= nrows || (lo <= j0 && j0 + kTile <= hi));
                if (!full) {
#pragma unroll
                    for (int c = 0; c < 128; ++c)
                        if (j0 + c < lo || j0 + c >= hi) x[c] = -INFINITY;
                }
                float mx = -INFINITY;
                {
                    float mm[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                    for (int c = 4; c < 128; c += 4)
#pragma unroll
                        for (int u = 0; u < 4; ++u) mm[u] = fmaxf(mm[u], x[c + u]);
                    mx = fmaxf(fmaxf(mm[0], mm[1]), fmaxf(mm[2], mm[3]));
                }
                if constexpr (!MOD) mx *= scale2;
                if (mx == -INFINITY || mx != mx) mx = m;
                // raise the reference when it is left behind by more than the slack
                const bool raise = mx > m + kSlack || (m == -INFINITY && mx > m);
                if (__any_sync(0xFFFFFFFFu, raise)) {
                    const float f = raise ? (m == -INFINITY ? 0.0f : ex2(m - mx)) : 1.0f;
                    if (raise) { m = mx; l *= f; }
                    if (j > a) {
                        warp_wait(wait, bars.pv_done[h], (uint32_t)(ns - 1) & 1u);
                        tc_after();
#pragma unroll
                        for (int c = 0; c < DP; c += 16) {
                            float o[16];
                            tm_ld16(to + c, o);
                            tm_wait_ld();
#pragma unroll
                            for (int u = 0; u < 16; ++u) o[u] *= f;
                            tm_st16(to + c, reinterpret_cast<uint32_t*>(o));
                        }
                        tm_wait_st();
                    }
                }
                const float base = m == -INFINITY ? 0.0f : m;
                float ls[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int c = 0; c < 128; c += 32) {
                    uint32_t pk[16];
#pragma unroll
                    for (int u = 0; u < 32; u += 2) {
                        float e0, e1;
                        if constexpr (MOD) { e0 = ex2(x[c + u] - base); e1 = ex2(x[c + u + 1] - base); }
                        else { e0 = ex2(fmaf(x[c + u], scale2, -base)); e1 = ex2(fmaf(x[c + u + 1], scale2, -base)); }
                        ls[(u / 2) & 1] += e0;
                        ls[2 + ((u / 2) & 1)] += e1;
                        pk[u / 2] = pack2<T>(e0, e1);
                    }
                    tm_st16(ts + c / 2, pk);
                }
                l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
                tm_wait_st();
                // Where some rows see a key and others do not, an infinite or
                // NaN value must not reach the others through 0 * v: these
                // warps then add such a tile (no finite model makes one)
                // themselves, key by key.
                bool by_hand = false;
                if (j0 < part_lo || j0 + kTile > part_hi) {
                    {
                        const int x2 = 2 * (n0 + j - k0) + 1;
                        warp_wait(wait, bars.kv_full[x2 % SLOTS], (uint32_t)(x2 / SLOTS) & 1u);
                        const unsigned char* v = smem + Gm::RING + (x2 % SLOTS) * Gm::SLOT;
                        bool odd = false;
                        for (int u = r; u < Gm::SLOT / 16; u += kHalf) {
                            const uint4 q4 = reinterpret_cast<const uint4*>(v)[u];
                            odd |= odd_word<T>(q4.x) || odd_word<T>(q4.y) || odd_word<T>(q4.z) || odd_word<T>(q4.w);
                        }
                        by_hand = bar_or(1 + h, odd);
                        if (by_hand) {
                            if (j > a) warp_wait(wait, bars.pv_done[h], (uint32_t)(ns - 1) & 1u);
                            tc_after();
                            for (int c = 0; c < DP; c += 16) {
                                float o[16];
                                if (j > a) { tm_ld16(to + c, o); tm_wait_ld(); }
                                else {
#pragma unroll
                                    for (int u = 0; u < 16; ++u) o[u] = 0.0f;
                                }
                                for (int k = 0; k < kTile; k += 2) {
                                    uint32_t w2;
                                    tm_ld1(ts + k / 2, w2);
                                    tm_wait_ld();
                                    const float2 pw = unpack2<T>(w2);
#pragma unroll
                                    for (int e = 0; e < 2; ++e) {
                                        const int jk = j0 + k + e;
                                        if (jk < lo || jk >= hi) continue;
                                        const float pe = e ? pw.y : pw.x;
#pragma unroll
                                        for (int u = 0; u < 16; u += 8) {
                                            const int ch = (c + u) / 8;
                                            const uint4 vv = *reinterpret_cast<const uint4*>(
                                                v + (ch / 8) * (128 * 128) + (k + e) * 128 + (((ch & 7) ^ ((k + e) & 7)) << 4));
                                            const uint32_t vw[4] = {vv.x, vv.y, vv.z, vv.w};
#pragma unroll
                                            for (int t = 0; t < 4; ++t) {
                                                const float2 f2 = unpack2<T>(vw[t]);
                                                o[u + 2 * t] = fmaf(pe, f2.x, o[u + 2 * t]);
                                                o[u + 2 * t + 1] = fmaf(pe, f2.y, o[u + 2 * t + 1]);
                                            }
                                        }
                                    }
                                    __syncwarp();
                                }
                                tm_st16(to + c, reinterpret_cast<uint32_t*>(o));
                                tm_wait_st();
                            }
                        }
                    }
                }
                if (r == 0) bars.skip[h] = by_hand;
                tc_before();
                __syncwarp();
                if (lane == 0) mbar_arrive1(&bars.p_full[h]);
            }
            // ---- the half's result ---------------------------------------------
            const bool any = b > a;
            if (any) warp_wait(wait, bars.pv_done[h], (uint32_t)(ns - 1) & 1u);
            tc_after();
            const bool part = sc.shared();
            if (nrows > 0) {
                const bool empty = l == 0.0f;
                const float inv = empty ? 0.0f : 1.0f / l;
                float* so = attn_slot(p, blockIdx.x, sc.w0 >= sc.us ? 0 : 1, kRows);
                const long long row = s.t0 + ti;
                T* out = static_cast<T*>(p.out) + row * p.o_ts + (long long)head * p.o_hs;
#pragma unroll
                for (int c = 0; c < DP; c += 16) {
                    float o[16];
                    if (any) { tm_ld16(to + c, o); tm_wait_ld(); }
                    if (r < nrows && c < p.D) {
                        if (empty) {
#pragma unroll
                            for (int u = 0; u < 16; ++u) o[u] = 0.0f;
                        }
                        if (part) {
                            float* d = so + (size_t)(h * kHalf + r) * p.D + c;
#pragma unroll
                            for (int u = 0; u < 16; u += 4)
                                if (c + u < p.D) __stcg(reinterpret_cast<float4*>(d + u), make_float4(o[u], o[u + 1], o[u + 2], o[u + 3]));
                        } else {
                            put16<T>(out + c, o, inv, p.D - c, g.out_vec);
                        }
                    }
                }
                if (r < nrows) {
                    if (part) {
                        __stcg(so + (size_t)kRows * p.D + h * kHalf + r, m);
                        __stcg(so + (size_t)kRows * p.D + kRows + h * kHalf + r, l);
                    } else if (p.lse) {
                        p.lse[row * p.Hq + head] = empty ? -INFINITY : (m + log2f(l)) * kLn2;
                    }
                }
                if (part) {
                    const int c0 = sc.owner(sc.us), c1 = sc.owner(sc.us + sc.c - 1);
                    __threadfence();
                    bar_sync(1 + h, kHalf);
                    if (r == 0) {
                        const bool last = atomicAdd(p.counters + 2 * c0 + h, 1u) == (unsigned)(c1 - c0);
                        if (last) p.counters[2 * c0 + h] = 0u;
                        bars.flag[h] = last;
                    }
                    bar_sync(1 + h, kHalf);
                    if (bars.flag[h]) {
                        __threadfence();
                        if (r < nrows) {
                            const size_t ss = (size_t)kRows * (p.D + 2);
                            const float* st = p.partials + (size_t)kRows * p.D + h * kHalf + r;
                            auto slot = [&](int c) { return (size_t)(2 * c + (sc.part(c) >= sc.us ? 0 : 1)) * ss; };
                            float M = -INFINITY, L = 0.0f;
                            for (int c = c0; c <= c1; ++c) M = fmaxf(M, __ldcg(st + slot(c)));
                            for (int c = c0; c <= c1; ++c) {
                                const float pl = __ldcg(st + slot(c) + kRows);
                                L = fmaf(pl, part_weight(__ldcg(st + slot(c)), pl, M), L);
                            }
                            for (int d = 0; d < p.D; d += 16) {
                                float o[16];
#pragma unroll
                                for (int u = 0; u < 16; ++u) o[u] = 0.0f;
                                for (int c = c0; c <= c1; ++c) {
                                    const float* sp = p.partials + slot(c) + (size_t)(h * kHalf + r) * p.D + d;
                                    const float pl = __ldcg(st + slot(c) + kRows);
                                    const float f = part_weight(__ldcg(st + slot(c)), pl, M);
#pragma unroll
                                    for (int u = 0; u < 16; u += 4)
                                        if (d + u < p.D) {
                                            const float4 v4 = __ldcg(reinterpret_cast<const float4*>(sp + u));
                                            o[u] = fmaf(v4.x, f, o[u]); o[u + 1] = fmaf(v4.y, f, o[u + 1]);
                                            o[u + 2] = fmaf(v4.z, f, o[u + 2]); o[u + 3] = fmaf(v4.w, f, o[u + 3]);
                                        }
                                }
                                if (L == 0.0f) {
#pragma unroll
                                    for (int u = 0; u < 16; ++u) o[u] = 0.0f;
                                }
                                put16<T>(out + d, o, L == 0.0f ? 0.0f : 1.0f / L, p.D - d, g.out_vec);
                            }
                            if (p.lse) p.lse[row * p.Hq + head] = L == 0.0f ? -INFINITY : (M + log2f(L)) * kLn2;
                        }
                        bar_sync(1 + h, kHalf);
                    }
                }
            }
            tc_before();
            n0 += k1 - k0;
            sc.next(p);
        }
    }
    // ---- every role has ended: tensor memory goes back ------------------------
    tc_before();
    __syncthreads();
    tc_after();
    if (warp == 8) {
        tm_relinquish();
        tm_dealloc(tm, 512);
    }
}

template <class T, int DP, bool MOD> cudaError_t launch_tdm(const AttnParams& p, cudaStream_t st) {
    using Gm = ChunkGeom<DP>;
    static std::atomic<unsigned> configured{0};
    auto kern = attn_chunk_kernel<T, DP, MOD>;
    ChunkArgs g = {};
    g.page_shift = -1;
    if ((p.page & (p.page - 1)) == 0)
        for (g.page_shift = 0; (1 << g.page_shift) < p.page; ++g.page_shift) {}
    g.out_vec = ((reinterpret_cast<uintptr_t>(p.out) | (uintptr_t)(p.o_ts * 2) | (uintptr_t)(p.o_hs * 2)) & 15) == 0;
    // pages of 8 rows or more, a power of two: whole pieces by tensor copies
    if (g.page_shift >= 3) {
        const bool f16 = __is_same(T, __half);
        const int rows = std::min(p.page, kTile);
        if (api_encode_pages(&g.kmap, p.k, f16, p.D, p.page, p.Hkv, p.n_pages, p.tok_s, p.head_s, p.page_s, rows) &&
            api_encode_pages(&g.vmap, p.v, f16, p.D, p.page, p.Hkv, p.n_pages, p.tok_s, p.head_s, p.page_s, rows))
            g.box_rows = rows;
    }
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned bit = 1u << (dev & 31);
    if (!(configured.load(std::memory_order_acquire) & bit)) {
        // the warpgroups' shares are drawn from the launch's registers
        cudaFuncAttributes at;
        e = cudaFuncGetAttributes(&at, kern);
        if (e == cudaSuccess && at.numRegs * kThreads < 256 * kSoftRegs + 128 * kOtherRegs) e = cudaErrorInvalidConfiguration;
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Gm::SMEM);
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit, std::memory_order_acq_rel);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::min(api_sms(), 148));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Gm::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p, g);
}

template <class T, int DP> cudaError_t launch_td(const AttnParams& p, cudaStream_t st) {
    return p.softcap > 0.0f || p.slopes ? launch_tdm<T, DP, true>(p, st) : launch_tdm<T, DP, false>(p, st);
}

template <class T> cudaError_t launch_t(const AttnParams& p, cudaStream_t st) {
    return p.D <= 64 ? launch_td<T, 64>(p, st) : launch_td<T, 128>(p, st);
}

}  // namespace

cudaError_t launch_attn_chunk(int dtype, const AttnParams& p, cudaStream_t st) {
    return dtype == 1 ? launch_t<__half>(p, st) : launch_t<__nv_bfloat16>(p, st);
}

}  // namespace qmv
