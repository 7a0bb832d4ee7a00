// qmv_attn_chunk.cu -- attention over a paged cache for many query rows a kv
// head (chunks of new tokens): 16-bit types, heads of up to 128 dims, on the
// 5th-generation tensor cores.
//
// Bound by the products (4 D flops a pair of row and key) and, at nearly the same
// size, by the exponentials (one a pair, 16 a clock and SM: a 128 x 64 tile
// takes 512 clocks, as its two products do at D = 128; at D = 64 they take half).
//
// One block an SM, 512 threads; a unit is 256 packed rows in two halves of 128:
//   warps 0-3, 4-7  softmax of half 0 / 1: thread = row.  S is read from tensor
//              memory (tcgen05.ld) and given back at once; the weights go to
//              tensor memory in the element type as the second product's A.
//   warps 8, 9 one lane each issues the half's tcgen05.mma: S = Q K^T (A, B
//              shared, 128-byte swizzle), O += P V (A tensor memory, B shared, V as
//              it lies: dims contiguous, the MN-major form).  The next step's S
//              is made while this step's exponentials run.
//   warps 12-15 copy K and V: tiles all of whose keys are seen by some row go by
//              tensor copies, one a page (or 64 rows) and 64 dims, where pages are
//              powers of two from 8 up; other pages, and the tiles at the ends,
//              go by cp.async, 16 bytes at a time, with zeros for keys no row
//              sees.  Q goes by cp.async.
//   warp 10    hands the block's units out, one after the other.
// Tensor memory: S_0, S_1 (64 columns each), 2 x P_0, 2 x P_1 (32 each), O_0, O_1.
// K and V tiles of 64 keys alternate in a ring.
//
// The running maximum is only raised when a row's new maximum exceeds it by 2^8:
// softmax is invariant to the reference that is subtracted, and with a slack of
// 8 in log2 neither the weights (<= 256) nor their fp32 sums can overflow; the
// output is rescaled in tensor memory, rarely, by the softmax warps themselves.
// The weights are rounded to the element type for the second product, their
// sum is not: an error of the size of the output's own rounding (the largest
// weight among them, since the reference may lie below it).  For f16 they
// are taken times 2^7 (2^15 at most, with the slack): those down to 2^-21 of the
// reference keep all their bits, the rest are off by up to 2^-32 of it.
//
// Every wait is bounded (about one second, not counting rows summed again); one
// that runs out ORs a code into the fault word (1: softmax, 2: copies, 8:
// products, 16: scheduling), raises a flag that ends every other wait, and the
// block frees its tensor memory and ends.
//
// Measured (bf16, 32 query and 8 kv heads of 128): 4096 tokens over 16384 keys,
// causal, 1000 us = 960 TFLOP/s, 58 % of the GEMM burst rate (69 % of the
// sustained one), tensor pipe and exponential unit each 52 % busy: softmax and
// products wait for each other.  Forms of the same call on the way: one warp that issues both halves'
// products 1330 us; tiles of 128 keys 1160; a single S beside P 1190; four warps that
// copy, one a ring slot, 1136; the scheduling warp 1125; turns at the
// exponentials 1022; one issuing lane 1005.  A quarter of the exponentials as
// polynomials: 1087 where 1042 was without.
#include <algorithm>

#include "qmv_attn_mma.cuh"
#include "qmv_attn_sched.cuh"

namespace qmv {

namespace {

constexpr int kThreads = 512;
constexpr int kRows = 256, kHalf = 128;
constexpr int kTile = 64;
constexpr int kLoaders = 4;                  // warps
constexpr int kSoftRegs = 176, kOtherRegs = 80;      // 256 x 176 + 256 x 80 = 512 x 128
constexpr float kSlack = 8.0f;               // log2
constexpr float kLarge = 65536.0f;           // references (log2) beyond which rows are summed again
template <class T> constexpr float kUp = __is_same(T, __half) ? 7.0f : 0.0f;     // log2 of what weights are taken times

template <int DP> struct ChunkGeom {
    static constexpr int SLOT = kTile * DP * 2;                 // bytes of a K or V tile
    static constexpr int SLOTS = DP == 64 ? 16 : 10;
    static constexpr int QB = kHalf * DP * 2;                   // bytes of half a unit's queries
    static constexpr int RING = 2 * QB;                         // ring's place
    static constexpr int SMEM = RING + SLOTS * SLOT + 1024;     // slack to round the base up to 1024
};

// One unit, or this block's part of it, as the scheduling warp hands it out.
struct Piece {
    int live;                // 0: no more
    int t0, n, len;          // the sequence: first row, new tokens, keys
    int b, h, rbase;         // sequence, kv head, first packed row
    int k0, k1;              // key tiles
    int ulo, uhi;            // keys that any row sees
    int a[2], e[2];          // key tiles of each half
    int shared;              // other blocks have parts of the unit
    int slot;                // this block's partial result
    int c0, c1, slot0;       // first and last block of the unit; the first one's partial result
};
constexpr int kPieces = 4;
constexpr int kReaders = 2 + kLoaders + 8;   // warps that read a piece

struct Bars {
    uint64_t kv_full[16], kv_empty[16], q_full, q_empty, s_full[2], s_empty[2], p_full[2][2], pv_done[2][2], drain[2];
    uint64_t pc_full[kPieces], pc_empty[kPieces];
    uint32_t tmem;
    volatile int abort;
    int busy;                // warps that sum rows again: nobody gives up meanwhile
    int turn[4];             // taken while a warp of the scheduler's pair has its exponentials
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
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) {
        if (mbar_try_sleep(bar, parity)) return true;
        uint64_t t0 = now_ns();
        while (ok) {
            if (mbar_try_sleep(bar, parity)) return true;
            if (*(volatile int*)&b->busy) t0 = now_ns();
            if (b->abort || now_ns() - t0 > kWaitNs) {
                if (!b->abort && fault) atomicOr(fault, code);
                b->abort = 1;
                ok = false;
            }
        }
        return false;
    }
};

// The same for a whole warp, with one answer.  The warp is converged after it, as
// the .aligned tcgen05 instructions that follow need it to be: lanes leave the
// polling loop one by one, and neither a vote nor a shuffle brings them back
// into step.
__device__ __forceinline__ bool warp_wait_all(Waiter& w, uint32_t bar, uint32_t parity) {
    const bool r = w(bar, parity);
    w.ok = __all_sync(0xFFFFFFFFu, r && w.ok);      // one lane of a warp may have given up alone
    __syncwarp();
    return w.ok;
}

// The two softmax warps of a scheduler (one of each half) take turns at their
// exponentials.  At once they take twice as long each, fall into step and leave
// the exponentials' unit idle for the rest of the step; in turns one warp's
// exponentials run beside the other's loads, maxima and waits.  Only the speed
// depends on it: after a while a warp goes on without its turn.
__device__ __forceinline__ void take_turn(int* turn) {
    if ((threadIdx.x & 31) == 0) {
        for (int i = 0; i < 200 && atomicExch(turn, 1) != 0; ++i) {}
    }
    __syncwarp();
}
__device__ __forceinline__ void give_turn(int* turn) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) *(volatile int*)turn = 0;
}

// One row over keys [k0, k1) of its sequence, by a warp (lane = dims lane, lane +
// 32, ..), reading only the keys the row sees: for rows whose sums came out
// infinite or NaN (there, and only there, a value that some rows see and others
// do not may have reached the others through 0 * v), and for rows of huge scores.
template <class T, int DP, bool MOD>
__device__ __forceinline__ void exact_row(const AttnParams& p, const ScoreMod<false>& mod, int b, int hk, const T* q, int pos,
                                          int k0, int k1, float slope, float (&o)[DP / 32], float& m, float& l) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < DP / 32; ++i) o[i] = 0.0f;
    m = -INFINITY;
    l = 0.0f;
#pragma unroll 1
    for (unsigned j0 = k0; j0 < (unsigned)k1; j0 += 32) {           // (k1 may be the last int)
        // 32 scores, a key a lane
        const bool in = j0 + lane < (unsigned)k1;
        const long long at = in ? key_place(p, b, hk, (int)(j0 + lane)) : -1;
        float s = 0.0f;
#pragma unroll 2
        for (int c = 0; c < p.D && at >= 0; c += 8) {
            const uint4 kq = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p.k) + at + c));
            const uint4 qq = __ldg(reinterpret_cast<const uint4*>(q + c));
            const uint32_t kw[4] = {kq.x, kq.y, kq.z, kq.w}, qw[4] = {qq.x, qq.y, qq.z, qq.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 a = unpack2<T>(kw[e]), x = unpack2<T>(qw[e]);
                s = fmaf(a.x, x.x, s);
                s = fmaf(a.y, x.y, s);
            }
        }
        s = MOD ? mod.apply(s, slope, (int)(j0 + lane - (unsigned)pos)) : __fmul_rn(s, p.scale * kLog2e);
        s = !in ? -INFINITY : at < 0 ? NAN : s;
        float mn = s;
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, w));
        mn = fmaxf(m, mn);
        const float base = mn == -INFINITY ? 0.0f : mn, f = ex2(m - base), w = in ? ex2(s - base) : 0.0f;
        m = mn;
        float sum = w;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, x);
        l = fmaf(l, f, sum);
#pragma unroll
        for (int i = 0; i < DP / 32; ++i) o[i] *= f;
#pragma unroll 4
        for (int x = 0; x < 32; ++x) {
            const float wx = __shfl_sync(0xFFFFFFFFu, w, x);
            const long long ax = __shfl_sync(0xFFFFFFFFu, at, x);
            if (j0 + x >= (unsigned)k1) continue;
#pragma unroll
            for (int i = 0; i < DP / 32; ++i) {
                const int d = lane + 32 * i;
                if (ax < 0) o[i] = NAN;
                else if (d < p.D) o[i] = fmaf(wx, ld_elem(static_cast<const T*>(p.v) + ax + d), o[i]);
            }
        }
    }
}

template <class T, int DP, bool MOD>
__global__ void __launch_bounds__(kThreads, 1) attn_chunk_kernel(const __grid_constant__ AttnParams p,
                                                                 const __grid_constant__ ChunkArgs g) {
    using Gm = ChunkGeom<DP>;
    constexpr int CPR = DP / 8, SLOTS = Gm::SLOTS;
    extern __shared__ unsigned char raw[];
    unsigned char* smem = raw + ((1024u - (s_addr(raw) & 1023u)) & 1023u);
    __shared__ Bars bars;
    __shared__ Piece pieces_s[kPieces];
    __shared__ SchedSmem sm;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t q_a = s_addr(smem), ring_a = q_a + Gm::RING;

    if (threadIdx.x == 0) {
        for (int i = 0; i < SLOTS; ++i) { mbar_init1(&bars.kv_full[i], 1); mbar_init1(&bars.kv_empty[i], 2); }
        mbar_init1(&bars.q_full, kLoaders);
        mbar_init1(&bars.q_empty, 2);
        for (int i = 0; i < 2; ++i) {
            mbar_init1(&bars.s_full[i], 1);
            mbar_init1(&bars.s_empty[i], 4);
            for (int u = 0; u < 2; ++u) {
                mbar_init1(&bars.p_full[i][u], 4);
                mbar_init1(&bars.pv_done[i][u], 1);
            }
            mbar_init1(&bars.drain[i], 1);
        }
        for (int i = 0; i < kPieces; ++i) { mbar_init1(&bars.pc_full[i], 1); mbar_init1(&bars.pc_empty[i], kReaders); }
        for (int i = 0; i < 4; ++i) bars.turn[i] = 0;
        bars.abort = 0;
        bars.busy = 0;
        fence_mbar_init();
    }
    __syncwarp();
    if (warp == 8) tm_alloc(s_addr(&bars.tmem), 512);
    grid_dependency_wait();
    grid_launch_dependents();
    tc_before();
    __syncthreads();
    tc_after();
    constexpr uint32_t tm = 0;                   // all 512 columns: tensor memory's start

    Sched<kRows, kTile> sc;
    sc.template init<kThreads>(p, sm, 8);

    // Pieces are read in order by every role but the scheduling warp: take()
    // waits for the next one, done() gives it back.
    int np = 0;
    auto take = [&](Waiter& w) -> const Piece* {
        if (!warp_wait_all(w, s_addr(&bars.pc_full[np % kPieces]), (uint32_t)(np / kPieces) & 1u)) return nullptr;
        const Piece* pc = &pieces_s[np % kPieces];
        return pc->live ? pc : nullptr;
    };
    auto done = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive1(&bars.pc_empty[np % kPieces]);
        ++np;
    };

    __syncwarp();
    if (warp >= 8) {
        reg_dec<kOtherRegs>();
        if (warp == 10) {
            // ---------------------------------------------- the scheduling ----
            Waiter wait{&bars, p.fault, 16u, true};
#pragma unroll 1
            for (;; ++np) {
                if (np >= kPieces &&
                    !warp_wait_all(wait, s_addr(&bars.pc_empty[np % kPieces]), (uint32_t)(np / kPieces - 1) & 1u))
                    break;
                if (lane == 0) {
                    Piece& pc = pieces_s[np % kPieces];
                    pc.live = sc.live;
                    if (sc.live) {
                        const int rbase = sc.i * kRows, rows = sc.s.n * p.G;
                        int k0, k1;
                        sc.piece(k0, k1);
                        pc.t0 = sc.s.t0; pc.n = sc.s.n; pc.len = sc.s.len;
                        pc.b = sc.b; pc.h = sc.h; pc.rbase = rbase;
                        pc.k0 = k0; pc.k1 = k1;
                        rows_keys(p, sc.s, rbase, min(rbase + kRows, rows) - 1, pc.ulo, pc.uhi);
#pragma unroll 1
                        for (int h = 0; h < 2; ++h) {
                            const int r0 = rbase + h * kHalf, r1 = min(r0 + kHalf, rows) - 1;
                            int a = k0, e = k0;
                            if (r0 <= r1) {
                                int lo, hi;
                                rows_keys(p, sc.s, r0, r1, lo, hi);
                                if (lo < hi) {
                                    a = max(k0, lo / kTile);
                                    e = min(k1, (hi - 1) / kTile + 1);
                                    if (a >= e) a = e = k0;
                                }
                            }
                            pc.a[h] = a; pc.e[h] = e;
                        }
                        pc.shared = sc.shared();
                        pc.slot = 2 * blockIdx.x + (sc.w0 >= sc.us ? 0 : 1);
                        pc.c0 = sc.owner(sc.us);
                        pc.c1 = sc.owner(sc.us + sc.c - 1);
                        pc.slot0 = 2 * pc.c0 + (sc.part(pc.c0) >= sc.us ? 0 : 1);
                    }
                    mbar_arrive1(&bars.pc_full[np % kPieces]);
                }
                __syncwarp();
                if (!sc.live) break;
                sc.next(p);
            }
        } else if (warp < 10) {
            // ------------------------------------------------ the products ----
            // One warp a half, of which one lane walks the steps.  These warps share their schedulers with
            // the softmax and wait for every instruction of their own: slots,
            // phases and descriptors are counted up, not computed.
            const int h = warp - 8;
            Waiter wait{&bars, p.fault, 8u, true};
            constexpr uint32_t FMT = __is_same(T, __half) ? 0u : 1u;
            constexpr uint32_t ID_S = (1u << 4) | (FMT << 7) | (FMT << 10) | ((kTile / 8u) << 17) | (8u << 24);
            constexpr uint32_t ID_O = (1u << 4) | (FMT << 7) | (FMT << 10) | (1u << 16) | ((DP / 8u) << 17) | (8u << 24);
            constexpr uint32_t HI = desc_hi(1024);
            constexpr uint32_t LBO_K = 1u << 16, LBO_V = (kTile * 128u / 16) << 16;
            const uint32_t q_d = desc_lo(q_a + h * Gm::QB, 16), ring_d = ring_a >> 4;
            const uint32_t ts = tm + h * 64, tp = tm + 128 + h * 64, to = tm + 256 + h * DP;
            const uint32_t full_a = s_addr(bars.kv_full), empty_a = s_addr(bars.kv_empty), sf_a = s_addr(&bars.s_full[h]),
                           se_a = s_addr(&bars.s_empty[h]), pf_a = s_addr(&bars.p_full[h]), pv_a = s_addr(&bars.pv_done[h]),
                           qe_a = s_addr(&bars.q_empty);
            const bool one = elect_one();
            // K and V of a step are slots 2 n and 2 n + 1 of the ring, which has an
            // even number: K tiles live in even slots.
            int ks = 0, vs = 1;                     // next slots
            uint32_t kph = 0, vph = 0, qph = 0;     // phases of the slots, of Q
            int sn = 0, pn = 0;                     // first and second products of this half so far
            auto qk = [&](bool mine) {              // takes a K tile; S = Q K^T
                wait(full_a + ks * 8, kph);
                if (mine) {
                    // the softmax holds the S before in registers
                    if (sn > 0) wait(se_a, (uint32_t)(sn - 1) & 1u);
                    tc_after();
                    if (wait.ok) {
                        const uint32_t b = (ring_d + ks * (Gm::SLOT / 16)) | LBO_K;
#pragma unroll
                        for (int k = 0; k < DP / 16; ++k) {
                            const uint32_t o = (k % 4) * (32 / 16);
                            mma_ss(ts, q_d + (k / 4) * (kHalf * 128 / 16) + o, b + (k / 4) * (kTile * 128 / 16) + o, HI, ID_S, k > 0);
                        }
                        commit(sf_a);
                    }
                    ++sn;
                }
                if (wait.ok) commit(empty_a + ks * 8);
                ks += 2;
                if (ks == SLOTS) { ks = 0; kph ^= 1u; }
            };
#pragma unroll 1
            while (const Piece* pc = take(wait)) {
                const int k0 = pc->k0, k1 = pc->k1, a = pc->a[h], e = pc->e[h];
                if (one && k0 < k1) {
                    wait(s_addr(&bars.q_full), qph);
                    qph ^= 1u;
                    // first products k0 .. k1 - 1, each one step ahead of its second
#pragma unroll 1
                    for (int j = k0 - 1; j < k1 && wait.ok; ++j) {
                        if (j + 1 < k1) {
                            qk(a <= j + 1 && j + 1 < e);
                            if (j + 2 == k1) commit(qe_a);
                        }
                        if (j < k0) continue;
                        wait(full_a + vs * 8, vph);
                        if (a <= j && j < e) {
                            const int u = pn & 1;
                            wait(pf_a + u * 8, (uint32_t)(pn >> 1) & 1u);
                            tc_after();
                            if (wait.ok) {
                                const uint32_t v = (ring_d + vs * (Gm::SLOT / 16)) | LBO_V, w = tp + u * 32;
                                mma_ts(to, w, v, HI, ID_O, j > a);
#pragma unroll
                                for (int k = 1; k < kTile / 16; ++k)
                                    mma_ts(to, w + k * 8, v + k * (16 * 128 / 16), HI, ID_O, true);
                                commit(pv_a + u * 8);
                            }
                            ++pn;
                        }
                        if (wait.ok) commit(empty_a + vs * 8);
                        vs += 2;
                        if (vs > SLOTS) { vs = 1; vph ^= 1u; }
                    }
                }
                done();
            }
            // nothing of this block's is in flight when it ends
            const uint32_t dr_a = s_addr(&bars.drain[h]);
            if (one) commit(dr_a);
            const uint64_t t0 = now_ns();
            while (!mbar_try_sleep(dr_a, 0u) && now_ns() - t0 < kWaitNs) {}
            __syncwarp();
        } else if (warp >= kThreads / 32 - kLoaders) {
            // -------------------------------------------------- the copies ----
            // Item x in the order of the ring (K and V of a tile in turn) is filled by
            // warp x % 4 alone: a warp's K or V, every second tile.  (All four warps on
            // each tile took 1000 clocks a slot, the time of one warp's instructions,
            // and bound the kernel.)
            Waiter wait{&bars, p.fault, 2u, true};
            const int w = warp - (kThreads / 32 - kLoaders), kv = w & 1;
            const int chunks = p.D / 8;
            const int page16 = (int)(p.page_s / 8), tok16 = (int)(p.tok_s / 8);
            constexpr int PER = 8 * CPR / 32;            // copies a lane makes of 8 rows
            const uint32_t full_a = s_addr(bars.kv_full), empty_a = s_addr(bars.kv_empty);
            const int pieces = g.box_rows > 0 ? kTile / g.box_rows : 0, items = pieces * (DP / 64);
            const CUtensorMap* map = kv ? &g.vmap : &g.kmap;
            int slot = w, fills = 0;
            uint32_t sph = 1;                            // a fresh barrier's phase of parity 1 is over
            int pend = -1;                               // slot whose cp.async copies are not reported yet
            auto tell = [&]() {
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive1(&bars.kv_full[pend]);
                pend = -1;
            };
            auto flush = [&]() {
                if (pend >= 0) { cp_wait<0>(); tell(); }
            };
            int npiece = 0, n0 = 0;                      // pieces and tiles before this one
#pragma unroll 1
            while (const Piece* pc = take(wait)) {
                const int k0 = pc->k0, k1 = pc->k1;
                if (k0 < k1) {
                    const int rbase = pc->rbase, nrows = min(kRows, pc->n * p.G - rbase), ulo = pc->ulo, uhi = pc->uhi, hk = pc->h;
                    const char* src = static_cast<const char*>(kv ? p.v : p.k) + (long long)hk * p.head_s * 2 + lane % CPR * 16;
                    const int* trow = p.table + (long long)pc->b * p.max_pages;
                    // place of key j, in units of 16 bytes; -1 where no row sees it, -2 on a bad page
                    auto place = [&](int j) -> int {
                        if (j < ulo || j >= uhi) return -1;
                        const int e = g.page_shift >= 0 ? j >> g.page_shift : j / p.page;
                        if (e >= p.max_pages) return -2;
                        const int pg = __ldg(trow + e);
                        if ((unsigned)pg >= (unsigned)p.n_pages) return -2;
                        return pg * page16 + (j - e * p.page) * tok16;
                    };
                    // page of this lane's box of a tile, -1 where the tile must go row by row
                    auto page_of = [&](int tile) -> int {
                        const int j0 = (int)((unsigned)tile * kTile);      // past the last int: negative, no tile
                        if (lane >= items) return 0;
                        const int e = (j0 + lane / (DP / 64) * g.box_rows) >> g.page_shift;
                        if (j0 < ulo || j0 > uhi - kTile || e >= p.max_pages) return -1;
                        const int pg = __ldg(trow + e);
                        return (unsigned)pg < (unsigned)p.n_pages ? pg : -1;
                    };
                    int j = k0 + (((n0 ^ (w >> 1)) & 1));         // this warp's first tile
                    int pg = items > 0 ? page_of(j) : -1;
                    // ---- queries, once the first products of the unit before are done ----
                    flush();
                    if (npiece > 0 && !warp_wait_all(wait, s_addr(&bars.q_empty), (uint32_t)(npiece - 1) & 1u)) break;
#pragma unroll 1
                    for (int gr = w; gr < kRows / 8; gr += kLoaders) {
                        const int r = gr * 8 + (lane & 7), pr = rbase + min(r, nrows - 1), ti = token_of(p, pr);
                        const long long off = ((long long)(pc->t0 + ti) * p.q_ts + (long long)(hk * p.G + pr - ti * p.G) * p.q_hs) * 2;
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
                    // ---- keys or values ---------------------------------------------
#pragma unroll 1
                    for (; j < k1; j += 2) {
                        const uint32_t base = ring_a + slot * Gm::SLOT;
                        // test hook (qmv_test_skip_last_copy): block 0's first K tile never comes
                        if (p.test_skip && blockIdx.x == 0 && w == 0 && fills == 0) {
                            pg = -1;
                        } else if (__all_sync(0xFFFFFFFFu, pg >= 0)) {
                            const int npg = page_of(j + 2);
                            flush();
                            if (!warp_wait_all(wait, empty_a + slot * 8, sph)) break;
                            if (lane == 0) mbar_expect(&bars.kv_full[slot], (uint32_t)Gm::SLOT);
                            __syncwarp();
                            if (lane < items) {
                                const int piece = lane / (DP / 64), blk = lane % (DP / 64);
                                box_copy(base + blk * (kTile * 128) + piece * g.box_rows * 128, map, blk * 64,
                                         (j * kTile + piece * g.box_rows) & (p.page - 1), hk, pg, &bars.kv_full[slot]);
                            }
                            pg = npg;
                        } else {
                            const int at[2] = {place(j * kTile + lane), place(j * kTile + 32 + lane)};
                            if (items > 0) pg = page_of(j + 2);
                            // about to wait: what is on its way is reported first
                            if (pend >= 0 && !__all_sync(0xFFFFFFFFu, mbar_test(empty_a + slot * 8, sph))) flush();
                            if (!warp_wait_all(wait, empty_a + slot * 8, sph)) break;
#pragma unroll 1
                            for (int gr = 0; gr < kTile / 8; ++gr) {
#pragma unroll
                                for (int u = 0; u < PER; ++u) {
                                    const int id = u * 32 + lane, rr = id / CPR, c = id % CPR;
                                    const int ra = __shfl_sync(0xFFFFFFFFu, gr < 4 ? at[0] : at[1], (gr & 3) * 8 + rr);
                                    const uint32_t d = base + (c / 8) * (kTile * 128) + (gr * 8 + rr) * 128 + (((c & 7) ^ rr) << 4);
                                    if (ra == -2 && kv == 0) {
                                        st_shared16(d, ~0u);                 // a key of NaN
                                    } else {
                                        const bool rd = ra >= 0 && c < chunks;
                                        cp16_or_zero(d, src + (rd ? (long long)ra * 16 : -16 * c), rd);
                                    }
                                }
                            }
                            cp_commit();
                            if (pend >= 0) { cp_wait<1>(); tell(); }
                            pend = slot;
                        }
                        ++fills;
                        slot += 4;
                        if (slot >= SLOTS) { slot -= SLOTS; sph ^= 1u; }
                    }
                    n0 += k1 - k0;
                }
                done();
            }
            cp_wait<0>();
            if (pend >= 0) tell();
            if (!wait.ok) {
                // given up: this warp's tensor copies land before the block ends
                const uint64_t t0 = now_ns();
                for (int f = max(0, fills - (SLOTS + 3) / 4); f < fills; ++f) {
                    const int x = w + 4 * f;
                    while (!mbar_test(full_a + x % SLOTS * 8, (uint32_t)(x / SLOTS) & 1u) && now_ns() - t0 < kWaitNs) {}
                }
                __syncwarp();
            }
        }
    } else {
        // ---------------------------------------------------- the softmax ----
        // Nothing here waits for another warp but on the bounded barriers: a warp
        // that gives up leaves the others free to do so.
        reg_inc<kSoftRegs>();
        const int h = warp >> 2;                         // half
        const int r = threadIdx.x & 127;                 // row of the half = lane of tensor memory
        const uint32_t lane_base = (uint32_t)(warp & 3) << 21;      // 32 lanes a warp, lane in bits 16..
        const uint32_t ts = tm + h * 64 + lane_base, tp0 = tm + 128 + h * 64 + lane_base, to = tm + 256 + h * DP + lane_base;
        const ScoreMod<false> mod(p);
        const float scale2 = p.scale * kLog2e;
        Waiter wait{&bars, p.fault, 1u, true};
        int ns = 0;                                      // steps of this half so far
#pragma unroll 1
        while (const Piece* pc = take(wait)) {
            const int a = pc->a[h], e = pc->e[h];
            const int rbase = pc->rbase + h * kHalf, nrows = min(kHalf, pc->n * p.G - rbase);
            int lo = 0, hi = 0, pos = 0, ti = 0, head = 0;
            float slope = 0.0f;
            if (r < nrows) {
                const int pr = rbase + r;
                ti = token_of(p, pr);
                head = pc->h * p.G + pr - ti * p.G;
                pos = pc->len - pc->n + ti;
                visible_keys(p, pos, pc->len, lo, hi);
                if (MOD && p.slopes) slope = __ldg(p.slopes + head) * kLog2e;
            }
            float m = -INFINITY, l = 0.0f;
#pragma unroll 1
            for (int j = a; j < e && wait.ok; ++j, ++ns) {
                const int u2 = ns & 1;                   // which P of the half
                const uint32_t tp = tp0 + u2 * 32;
                if (!warp_wait_all(wait, s_addr(&bars.s_full[h]), (uint32_t)ns & 1u)) break;
                tc_after();
                float x[kTile];
                tm_ld32(ts, x);
                tm_ld32(ts + 32, x + 32);
                const int j0 = j * kTile;
                // rows past the unit have queries of zero and need no mask
                const bool full = __all_sync(0xFFFFFFFFu, r >= nrows || (lo <= j0 && j0 <= hi - kTile));
                tm_wait_ld();
                tc_before();
                __syncwarp();
                if (lane == 0) mbar_arrive1(&bars.s_empty[h]);      // the next S may be written
                if constexpr (MOD) mod.template apply_all<kTile>(x, slope, j0 - pos);
                if (!full) {
#pragma unroll
                    for (int c = 0; c < kTile; ++c)
                        if (j0 + c < lo || j0 + c >= hi) x[c] = -INFINITY;
                }
                float mx;
                {
                    float mm[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                    for (int c = 4; c + 8 <= kTile; c += 8)
#pragma unroll
                        for (int u = 0; u < 4; ++u) mm[u] = max3(mm[u], x[c + u], x[c + 4 + u]);
#pragma unroll
                    for (int u = 0; u < 4; ++u) mm[u] = fmaxf(mm[u], x[kTile - 4 + u]);
                    mx = fmaxf(fmaxf(mm[0], mm[1]), fmaxf(mm[2], mm[3]));
                }
                if constexpr (!MOD) mx = __fmul_rn(mx, scale2);
                if (mx == -INFINITY || mx != mx) mx = m;
                // raise the reference when it is left behind by more than the slack
                const bool raise = mx - m > kSlack;
                if (__any_sync(0xFFFFFFFFu, raise)) {
                    const float f = raise ? (m == -INFINITY ? 0.0f : ex2(m - mx)) : 1.0f;
                    if (raise) { m = mx; l *= f; }
                    if (j > a) {
                        if (!warp_wait_all(wait, s_addr(&bars.pv_done[h][u2 ^ 1]), (uint32_t)((ns - 1) >> 1) & 1u)) break;
                        tc_after();
#pragma unroll 1
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
                // this P was last read by the second product two steps ago
                if (ns >= 2 && !warp_wait_all(wait, s_addr(&bars.pv_done[h][u2]), (uint32_t)((ns >> 1) - 1) & 1u)) break;
                take_turn(&bars.turn[warp & 3]);
                tc_after();
                const float away = m == -INFINITY ? 0.0f : kUp<T> - m;
                const float2 nb = make_float2(away, away), sc2 = make_float2(MOD ? 1.0f : scale2, MOD ? 1.0f : scale2);
                float2 ls[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
                for (int c = 0; c < kTile; c += 32) {
                    uint32_t pk[16];
#pragma unroll
                    for (int u = 0; u < 32; u += 2) {
                        float2 w = fma2(make_float2(x[c + u], x[c + u + 1]), sc2, nb);
                        w.x = ex2(w.x);
                        w.y = ex2(w.y);
                        ls[(u / 2) & 1] = add2(ls[(u / 2) & 1], w);
                        pk[u / 2] = pack2<T>(w.x, w.y);
                    }
                    tm_st16(tp + c / 2, pk);
                }
                give_turn(&bars.turn[warp & 3]);
                l += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
                tm_wait_st();
                tc_before();
                __syncwarp();
                if (lane == 0) mbar_arrive1(&bars.p_full[h][u2]);
            }
            if (!wait.ok) break;
            m -= kUp<T>;                                 // what the weights are relative to, from here on
            // ---- the rows' result ----------------------------------------------
            const bool any = e > a;
            if (any && !warp_wait_all(wait, s_addr(&bars.pv_done[h][(ns - 1) & 1]), (uint32_t)((ns - 1) >> 1) & 1u)) break;
            tc_after();
            const bool mine = r < nrows, empty = l == 0.0f, part = pc->shared;
            const float inv = empty ? 0.0f : 1.0f / l;
            const long long row = pc->t0 + ti;
            T* out = static_cast<T*>(p.out) + row * p.o_ts + (long long)head * p.o_hs;
            // a partial result holds 4 dims of all rows side by side: lanes are rows
            const size_t ss = (size_t)kRows * (p.D + 2);
            const int at = h * kHalf + r;                // row of the unit
            float* so = p.partials + pc->slot * ss;
            bool odd = false;                            // a sum that is not finite
#pragma unroll 1
            for (int c = 0; c < p.D; c += 16) {
                float o[16];
                __syncwarp();
                if (any) { tm_ld16(to + c, o); tm_wait_ld(); }
#pragma unroll
                for (int u = 0; u < 16; ++u) odd |= !(fabsf(o[u]) < INFINITY);
                if (empty) {
#pragma unroll
                    for (int u = 0; u < 16; ++u) o[u] = 0.0f;
                }
                if (mine && part) {
#pragma unroll
                    for (int u = 0; u < 16; u += 4)
                        if (c + u < p.D)
                            __stcg(reinterpret_cast<float4*>(so) + (size_t)((c + u) / 4) * kRows + at, make_float4(o[u], o[u + 1], o[u + 2], o[u + 3]));
                } else if (mine) {
                    put16<T>(out + c, o, inv, p.D - c, g.out_vec);
                }
            }
            tc_before();
            if (mine && part) {
                __stcg(so + (size_t)kRows * p.D + at, m);
                __stcg(so + (size_t)kRows * p.D + kRows + at, l);
            } else if (mine && p.lse) {
                p.lse[row * p.Hq + head] = empty ? -INFINITY : (m + log2f(l)) * kLn2;
            }
            // An FMA does not round its product, as the maximum's was: with references
            // this large the weights are off by 2^(up to 2^-24 m), all of a row alike,
            // down to none and up to infinity.  (Rounding the products in the loop
            // where a warp has such rows cost 1.4 % of every call.)
            const bool large = !MOD && m != -INFINITY && fabsf(m) > kLarge;
            unsigned again = __ballot_sync(0xFFFFFFFFu, mine && any && (large || (odd && !empty)));
            if (again && lane == 0) atomicAdd(&bars.busy, 1);      // may take long; it waits for nothing
            const bool busy = again != 0;
#pragma unroll 1
            while (again) {
                const int src = __ffs(again) - 1;
                again &= again - 1;
                __syncwarp();
                auto of = [&](int v) { return __shfl_sync(0xFFFFFFFFu, v, src); };
                const int sti = of(ti), shead = of(head), spos = of(pos), slo = max(of(lo), a * kTile), shi = (int)min((unsigned)of(hi), (unsigned)e * kTile);
                const float sslope = __shfl_sync(0xFFFFFFFFu, slope, src);
                float o[DP / 32], sm2, sl;
                exact_row<T, DP, MOD>(p, mod, pc->b, pc->h, static_cast<const T*>(p.q) + (long long)(pc->t0 + sti) * p.q_ts + (long long)shead * p.q_hs,
                                      spos, slo, shi, sslope, o, sm2, sl);
                const int sat = h * kHalf + (r & ~31) + src;
                const long long srow = pc->t0 + sti;
#pragma unroll
                for (int i = 0; i < DP / 32; ++i) {
                    const int d = lane + 32 * i;
                    if (d >= p.D) continue;
                    if (part) __stcg(so + ((size_t)(d / 4) * kRows + sat) * 4 + d % 4, sl == 0.0f ? 0.0f : o[i]);
                    else st_elem(static_cast<T*>(p.out) + srow * p.o_ts + (long long)shead * p.o_hs + d, sl == 0.0f ? 0.0f : o[i] / sl);
                }
                if (lane == 0 && part) {
                    __stcg(so + (size_t)kRows * p.D + sat, sm2);
                    __stcg(so + (size_t)kRows * p.D + kRows + sat, sl);
                } else if (lane == 0 && p.lse) {
                    p.lse[srow * p.Hq + shead] = sl == 0.0f ? -INFINITY : (sm2 + log2f(sl)) * kLn2;
                }
            }
            if (busy && lane == 0) atomicAdd(&bars.busy, -1);
            if (part && nrows > (r & ~31)) {             // this warp has rows
                // A warp joins its own rows: the last of the unit's blocks to
                // have written them does.
                const int c0 = pc->c0, c1 = pc->c1;
                __threadfence();
                __syncwarp();
                int last = 0;
                if (lane == 0) {
                    unsigned* cnt = p.counters + 8 * c0 + warp;
                    last = atomicAdd(cnt, 1u) == (unsigned)(c1 - c0);
                    if (last) *cnt = 0u;
                }
                last = __shfl_sync(0xFFFFFFFFu, last, 0);
                if (last) {
                    __threadfence();
                    if (mine) {
                        const float* st = p.partials + (size_t)kRows * p.D + at;
                        auto slot = [&](int c) { return (size_t)(c == c0 ? pc->slot0 : 2 * c) * ss; };
                        float M = -INFINITY, L = 0.0f;
#pragma unroll 1
                        for (int c = c0; c <= c1; ++c) M = fmaxf(M, __ldcg(st + slot(c)));
#pragma unroll 1
                        for (int c = c0; c <= c1; ++c) {
                            const float pl = __ldcg(st + slot(c) + kRows);
                            L = fmaf(pl, part_weight(__ldcg(st + slot(c)), pl, M), L);
                        }
                        const float iL = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll 1
                        for (int d = 0; d < p.D; d += 16) {
                            float o[16];
#pragma unroll
                            for (int u = 0; u < 16; ++u) o[u] = 0.0f;
#pragma unroll 2
                            for (int c = c0; c <= c1; ++c) {
                                const float4* sp = reinterpret_cast<const float4*>(p.partials + slot(c)) + (size_t)(d / 4) * kRows + at;
                                const float pl = __ldcg(st + slot(c) + kRows);
                                const float f = part_weight(__ldcg(st + slot(c)), pl, M);
#pragma unroll
                                for (int u = 0; u < 16; u += 4)
                                    if (d + u < p.D) {
                                        const float4 v4 = __ldcg(sp + (size_t)(u / 4) * kRows);
                                        o[u] = fmaf(v4.x, f, o[u]); o[u + 1] = fmaf(v4.y, f, o[u + 1]);
                                        o[u + 2] = fmaf(v4.z, f, o[u + 2]); o[u + 3] = fmaf(v4.w, f, o[u + 3]);
                                    }
                            }
                            if (L == 0.0f) {
#pragma unroll
                                for (int u = 0; u < 16; ++u) o[u] = 0.0f;
                            }
                            put16<T>(out + d, o, iL, p.D - d, g.out_vec);
                        }
                        if (p.lse) p.lse[row * p.Hq + head] = L == 0.0f ? -INFINITY : (M + log2f(L)) * kLn2;
                    }
                }
            }
            done();
        }
    }
    // ---- every role has ended: tensor memory goes back ------------------------
    tc_before();
    __syncthreads();
    tc_after();
    __syncwarp();
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
    g.page_shift = page_shift_of(p.page);
    g.out_vec = ((reinterpret_cast<uintptr_t>(p.out) | (uintptr_t)(p.o_ts * 2) | (uintptr_t)(p.o_hs * 2)) & 15) == 0;
    // pages of 8 rows or more, a power of two: whole pieces by tensor copies
    if (g.page_shift >= 3) {
        const bool f16 = __is_same(T, __half);
        const int rows = std::min(p.page, kTile);
        if (api_encode_pages(&g.kmap, p.k, f16, p.D, p.page, p.Hkv, p.n_pages, p.tok_s, p.head_s, p.page_s, rows) &&
            api_encode_pages(&g.vmap, p.v, f16, p.D, p.page, p.Hkv, p.n_pages, p.tok_s, p.head_s, p.page_s, rows))
            g.box_rows = rows;
    }
    // the warpgroups' shares are drawn from the launch's registers
    cudaFuncAttributes at;
    cudaError_t e = cudaFuncGetAttributes(&at, kern);
    if (e == cudaSuccess && at.numRegs * kThreads < 256 * (kSoftRegs + kOtherRegs)) e = cudaErrorInvalidConfiguration;
    if (e == cudaSuccess) e = allow_smem(kern, configured, Gm::SMEM);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, dim3((unsigned)std::min(api_sms(), 148)), dim3(kThreads), Gm::SMEM, st, p, g);
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
