// qmv_attn_sched.cuh -- how the attention kernels share out their work.
//
// A unit is (sequence b, kv head h, row tile i): ROWS consecutive packed rows of
// a sequence (packed row r is query head h G + r % G of new token r / G, so the
// G query heads that share a kv head share its keys), over the keys that any of
// them sees, in key tiles of TK.  All units' key tiles, laid end to end in the
// order (b, h, i), are cut into equal parts, one a block: every block streams
// the same number of key tiles whatever the lengths are, and nothing but the
// device's length lists decides the cut (a captured call can be replayed with
// other lengths).  Each block finds its own part: it sums the units' tile
// counts over the sequences with a block-wide scan.
//
// A block that ends one unit and begins another pays two joins, of about ten
// tiles' time each.  Few tiles a block are therefore cut at the units' own ends
// (every unit into parts of Q tiles, the last one shorter), if that gives no more
// parts than blocks at the even share or 5/4 of it; failing that, in eighths of
// the even share (at least 4 tiles), so that short units stay whole.  (12 fp32
// sequences of 100-2100 keys: 46 us, and 54 with whole parts of up to twice the share
// and quarters.)
//
// A block whose part ends or begins inside a unit leaves that unit's partial
// result (unnormalised sums, maxima, weights) in the workspace and counts
// itself in on the unit's counter; the last block to arrive joins the parts in
// block order, writes the unit's output and sets the counter back to zero.  No
// block waits for another, and the order of every sum depends on the arguments
// alone.  Without a workspace a unit belongs whole to the block in whose part it
// begins.
#pragma once

#include "qmv_attn.cuh"

namespace qmv {

constexpr int kAttnCounters = 4096;                     // unsigned words at the workspace's start
constexpr size_t kAttnPartialsAt = kAttnCounters * 4;   // byte offset of the partial results

struct SeqInfo {
    int t0, n, len;         // first row, new tokens, keys
};

__device__ __forceinline__ SeqInfo seq_info(const AttnParams& p, int b) {
    SeqInfo s;
    s.t0 = row_start(p.q_starts, b, p.T);
    s.n = max(0, row_start(p.q_starts, b + 1, p.T) - s.t0);
    s.len = max(0, __ldg(p.kv_lens + b));
    return s;
}

// Keys [lo, hi) that any of the packed rows r0..r1 of a sequence sees (0, 0: none).
__device__ __forceinline__ void rows_keys(const AttnParams& p, const SeqInfo& s, int r0, int r1, int& lo, int& hi) {
    int x;
    visible_keys(p, s.len - s.n + token_of(p, r0), s.len, lo, x);
    visible_keys(p, s.len - s.n + token_of(p, r1), s.len, x, hi);
    if (lo >= hi) lo = hi = 0;
}

// Row tile i of a sequence: its first key tile and the number of key tiles (0:
// the unit sees no key; it still counts as one tile of work).
template <int ROWS, int TK>
__device__ __forceinline__ int unit_tiles(const AttnParams& p, const SeqInfo& s, int i, int& first) {
    int lo, hi;
    rows_keys(p, s, i * ROWS, min((i + 1) * ROWS, s.n * p.G) - 1, lo, hi);
    first = lo / TK;
    return hi > lo ? (hi - 1) / TK + 1 - first : 0;
}

constexpr int kAlignTiles = 64;         // parts up to this many tiles end with their units
constexpr long long kMostTiles = 1LL << 26;     // of a unit: 2^31 keys in tiles of 32

struct SchedSmem {
    long long warp_sum[32];
    long long seq_at;       // chunks before the sequence in which the block's part begins
    int seq;                // that sequence
    int per_head;           // its chunks per kv head
};

// One block's walk over its part.  Work is counted in chunks of Q key tiles of a
// unit (its last chunk may be shorter): Q = 1 unless parts are to end with their
// units, or there are 2^30 tiles or more.  (Tiles are counted in 64 bits, chunks
// fit an int.)
template <int ROWS, int TK> struct Sched {
    int W, w0, w1;          // all chunks, this block's part
    int q, rem;             // W = nblk q + rem: the first rem blocks take q + 1 chunks
    int us;                 // first chunk of the current unit
    int nblk, b, h, i, c;   // blocks with a part; current unit and its chunks
    int first, nt;          // its first key tile and number of key tiles
    int Q;
    SeqInfo s;
    bool split, live;

    __device__ __forceinline__ int chunks(int tiles) const {
        return tiles <= Q ? 1 : Q == 1 ? tiles : (tiles - 1) / Q + 1;
    }
    __device__ __forceinline__ int part(int blk) const { return blk * q + min(blk, rem); }
    __device__ __forceinline__ int owner(int w) const {
        const int big = rem * (q + 1);
        return w < big ? w / (q + 1) : rem + (w - big) / q;
    }
    __device__ __forceinline__ void load_unit(const AttnParams& p) {
        nt = unit_tiles<ROWS, TK>(p, s, i, first);
        c = chunks(nt);
    }
    __device__ __forceinline__ void next(const AttnParams& p) {
        us += c;
        if (us >= w1) { live = false; return; }
        if (++i * ROWS >= s.n * p.G) {
            i = 0;
            if (++h == p.Hkv) {
                h = 0;
#pragma unroll 1
                do {
                    if (++b >= p.n_seqs) { live = false; return; }
                    s = seq_info(p, b);
                } while (s.n == 0);
            }
        }
        load_unit(p);
    }
    // Every thread of the block calls this (NT threads).  A sequence's units are
    // counted by 1 to 32 lanes, as many as leave every sequence a place in one
    // round (one lane for all 60 units of 120 tokens x 8 heads: the call takes 44 us,
    // so 24).
    template <int NT> __device__ __forceinline__ void init(const AttnParams& p, SchedSmem& sm, int min_tiles) {
        const int tid = threadIdx.x, lane = tid & 31;
        int lg = 5;
        while (lg > 0 && (long long)p.n_seqs << lg > NT) --lg;
        const int lps = 1 << lg, sub = tid & (lps - 1), seqs = NT >> lg;
        const int rounds = (p.n_seqs + seqs - 1) >> (__ffs(seqs) - 1);
        int kept = -2;          // tiles of the lane's only unit, -1 for none, in the one round; -2: not known
        auto cost = [&](int bb) {
            long long v = 0;
            if (kept >= -1) {
                if (kept >= 0) v = chunks(kept);
            } else if (bb < p.n_seqs) {
                const SeqInfo si = seq_info(p, bb);
                const int nq = (si.n * p.G + ROWS - 1) / ROWS;
                if (nq <= lps && rounds == 1) kept = -1;
                int f;
#pragma unroll 1
                for (int k = sub; k < nq; k += lps) {
                    const int tiles = unit_tiles<ROWS, TK>(p, si, k, f);
                    if (kept == -1) kept = tiles;
                    v += chunks(tiles);
                }
            }
            // one unit a sequence: its first lane, which alone is read, holds the sum
            if (__any_sync(0xFFFFFFFFu, sub != 0 && v != 0)) {
#pragma unroll 1
                for (int w = lps >> 1; w > 0; w >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, w);
            }
            return v;
        };
        // inclusive scan over the block (the value counts once a sequence)
        auto scan = [&](long long c1, long long& total) {
            long long v = sub == 0 ? c1 * p.Hkv : 0;
#pragma unroll
            for (int w = 1; w < 32; w <<= 1) {
                const long long u = __shfl_up_sync(0xFFFFFFFFu, v, w);
                if (lane >= w) v += u;
            }
            __syncthreads();
            if (lane == 31) sm.warp_sum[tid >> 5] = v;
            __syncthreads();
            long long before = 0;
            total = 0;
#pragma unroll
            for (int w = 0; w < NT / 32; ++w) {
                const long long u = sm.warp_sum[w];
                if (w < (tid >> 5)) before += u;
                total += u;
            }
            return v + before;
        };
        split = p.partials != nullptr;
        live = false;
        Q = 1;
        long long v = 0;
        int pass = 0;           // 0: count tiles, 1, 2: parts of each, 5/4 each tiles end with their units, 3: they do not
        int each = 0;           // tiles a block
        long long incl = 0, all;
#pragma unroll 1
        for (;;) {
            all = 0;
#pragma unroll 1
            for (int r = 0; r < rounds; ++r) {
                v = cost(r * seqs + (tid >> lg));
                long long total;
                incl = scan(v, total);
                all += total;
            }
            if (pass == 0) {
                if (all <= 0) return;
                if (all >> 30) {
                    Q = (int)min(all >> 29, kMostTiles) + 1;
                    pass = 3;
                    continue;
                }
                each = (int)(((unsigned)all + gridDim.x - 1) / gridDim.x);
                if (split && each <= kAlignTiles) {
                    Q = max(each, min_tiles);
                    pass = 1;
                    continue;
                }
            } else if (pass < 3 && all > (long long)gridDim.x) {
                ++pass;
                Q = pass == 3 ? max(4, each / 8) : max(min_tiles, each * 5 / 4);
                continue;
            } else if (all >> 31) {
                // many units of one chunk: an int holds those of all rows there can
                // be; more are lists that do not ascend, which nothing is run for
                if (Q > kMostTiles) return;
                Q = (int)min(Q * 8LL, kMostTiles + 1);
                continue;
            }
            break;
        }
        W = (int)all;
        nblk = pass == 1 || pass == 2 ? W : min((int)gridDim.x, W);
        if ((int)blockIdx.x >= nblk) return;
        q = W / nblk;
        rem = W - q * nblk;
        w0 = part(blockIdx.x);
        w1 = part(blockIdx.x + 1);
        long long base = 0;
#pragma unroll 1
        for (int r = 0; r < rounds; ++r) {
            long long total = all;
            if (rounds > 1) {
                v = cost(r * seqs + (tid >> lg));
                incl = scan(v, total);
            }
            const long long end = base + incl, beg = end - v * p.Hkv;
            if (sub == 0 && beg <= w0 && w0 < end) {
                sm.seq = r * seqs + (tid >> lg);
                sm.seq_at = beg;
                sm.per_head = (int)v;
            }
            base += total;
            if (base > w0) break;       // the same for every thread
        }
        __syncthreads();
        b = sm.seq;
        s = seq_info(p, b);
        int off = w0 - (int)sm.seq_at;
        h = off / sm.per_head;
        off -= h * sm.per_head;
        i = 0;
        if (s.n * p.G > ROWS) {             // 32 units at a time
#pragma unroll 1
            for (;; i += 32) {
                int f, cc = 0;
                if ((i + lane) * ROWS < s.n * p.G) cc = chunks(unit_tiles<ROWS, TK>(p, s, i + lane, f));
                int upto = cc;
#pragma unroll
                for (int w = 1; w < 32; w <<= 1) {
                    const int u = __shfl_up_sync(0xFFFFFFFFu, upto, w);
                    if (lane >= w) upto += u;
                }
                const unsigned here = __ballot_sync(0xFFFFFFFFu, off < upto);
                const int at = here ? __ffs(here) - 1 : 31;
                off -= __shfl_sync(0xFFFFFFFFu, here ? upto - cc : upto, at);
                if (here || (i + 32) * ROWS >= s.n * p.G) {     // (the bound: lists that change meanwhile end, too)
                    i += at;
                    break;
                }
            }
        }
        load_unit(p);
        us = w0 - off;
        live = true;
        if (!split && off > 0) next(p);     // the unit belongs to the block before
    }
    // Key tiles [k0, k1) of the current unit that are this block's.
    __device__ __forceinline__ void piece(int& k0, int& k1) const {
        if (split) {
            k0 = first + (max(w0, us) - us) * Q;
            k1 = first + min((min(w1, us + c) - us) * Q, nt);
        } else {
            k0 = first;
            k1 = first + nt;
        }
    }
    // Whether other blocks hold parts of the current unit.
    __device__ __forceinline__ bool shared() const { return split && (us < w0 || us + c > w1); }
};

// Partial result of a block: slot 0 for the unit its part begins in, 1 for the
// one it ends in.  Per slot ROWS x D sums, then ROWS maxima (log2) and sums of
// weights.
__device__ __forceinline__ float* attn_slot(const AttnParams& p, int blk, int which, int rows) {
    return p.partials + ((size_t)blk * 2 + which) * ((size_t)rows * (p.D + 2));
}

// Counts this block in on the current unit; true in the last one to arrive.
// Every thread of the block has written its share before.
template <int ROWS, int TK>
__device__ __forceinline__ bool attn_arrive(const AttnParams& p, const Sched<ROWS, TK>& sc, int* s_flag) {
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        const int c0 = sc.owner(sc.us), c1 = sc.owner(sc.us + sc.c - 1);
        const bool last = atomicAdd(p.counters + c0, 1u) == (unsigned)(c1 - c0);
        if (last) p.counters[c0] = 0u;
        *s_flag = last;
    }
    __syncthreads();
    const bool last = *s_flag != 0;
    if (last) __threadfence();
    return last;
}

// Weight of a partial result whose maximum (log2) is m among ones of maximum M:
// 0 for one without keys.
__device__ __forceinline__ float part_weight(float m, float l, float M) {
    return l == 0.0f ? 0.0f : exp2f(m == -INFINITY && M == -INFINITY ? 0.0f : m - M);
}

// The last block joins the parts of the current unit (whole block; NT threads;
// at most kJoinParts parts and kJoinRows rows).  store(row, dim, 4 sums, m, l)
// gets every 4 dims of every row.
constexpr int kJoinParts = 296, kJoinRows = 16;
constexpr int kJoinBytes = kJoinParts * 4 + 2 * kJoinRows * kJoinParts * 4 + 2 * kJoinRows * 4;
template <int NT, int ROWS, int TK, class Store>
__device__ __forceinline__ void attn_join(const AttnParams& p, const Sched<ROWS, TK>& sc, int nrows, void* buf, Store store) {
    static_assert(ROWS <= kJoinRows, "join buffer");
    const int c0 = sc.owner(sc.us), np = sc.owner(sc.us + sc.c - 1) - c0 + 1;
    float* s_f = static_cast<float*>(buf);              // [row][np]: maximum, then weight
    float* s_l = s_f + ROWS * np;
    float* s_M = s_l + ROWS * np;
    float* s_L = s_M + ROWS;
    int* s_slot = reinterpret_cast<int*>(s_L + ROWS);
    const int tid = threadIdx.x, lane = tid & 31;
    for (int i = tid; i < np; i += NT) s_slot[i] = (c0 + i) * 2 + (sc.part(c0 + i) >= sc.us ? 0 : 1);
    __syncthreads();
    const size_t ss = (size_t)ROWS * (p.D + 2);
#pragma unroll 1
    for (int x = tid; x < nrows * np; x += NT) {
        const int r = x / np, i = x - r * np;
        const float* so = p.partials + s_slot[i] * ss + ROWS * p.D;
        s_f[x] = __ldcg(so + r);
        s_l[x] = __ldcg(so + ROWS + r);
    }
    __syncthreads();
    for (int r = tid >> 5; r < nrows; r += NT / 32) {
        float M = -INFINITY, L = 0.0f;
        for (int i = lane; i < np; i += 32) M = fmaxf(M, s_f[r * np + i]);
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, w));
        for (int i = lane; i < np; i += 32) {
            const float l = s_l[r * np + i], f = part_weight(s_f[r * np + i], l, M);
            s_f[r * np + i] = f;
            L = fmaf(l, f, L);
        }
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) L += __shfl_xor_sync(0xFFFFFFFFu, L, w);
        if (lane == 0) { s_M[r] = M; s_L[r] = L; }
    }
    __syncthreads();
    const int vecs = p.D / 4;
#pragma unroll 1
    for (int x = tid; x < nrows * vecs; x += NT) {
        const int r = x / vecs, d = (x - r * vecs) * 4;
        const float* so = p.partials + r * p.D + d;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
        for (int i = 0; i < np; ++i) {
            const float4 u = __ldcg(reinterpret_cast<const float4*>(so + s_slot[i] * ss));
            const float f = s_f[r * np + i];
            v.x = fmaf(u.x, f, v.x); v.y = fmaf(u.y, f, v.y); v.z = fmaf(u.z, f, v.z); v.w = fmaf(u.w, f, v.w);
        }
        store(r, d, v, s_M[r], s_L[r]);
    }
}

}  // namespace qmv
