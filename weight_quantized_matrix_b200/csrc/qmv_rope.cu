// qmv_rope.cu -- the rotary rotation of query / key heads, and the append of
// rotated keys and of values to a paged cache (one kernel for both).
//
// Mathematics.  Pair i of a head of a token at position p turns by the angle
// a = p * inv_freq[i]:  (x, y) -> m (x cos a - y sin a), m (x sin a + y cos a).
// p has up to 31 bits and inv_freq 24, so an fp32 product loses the angle of a
// far position; the product and its reduction to a fraction of one turn are
// done in fp64 and only that fraction, in [-1/2, 1/2], is rounded to fp32 for
// sincospif (angle error below 2^-24 turns up to angles of 2^29, 2^-23 at the last
// int; that is fp64's own rounding).  The rotation itself is fp32, rounded
// once to the element type.
//
// Memory-bound: every element is read once and written once.  A block takes
// `tpb` tokens (as many as give its 256 threads up to three items each); its threads
// first load their vectors, then look the tokens up and share out their cosines
// and sines through shared memory (one evaluation per token and pair, for all
// heads), then rotate and store.  A work item is the pair of vectors a rotation mixes:
// dims (i, i + rot/2) of the half layout, or 2 consecutive vectors of the
// interleaved one and of the parts that are copied (dims >= rot, V).
#include "qmv_paged.cuh"

namespace qmv {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 32;      // tokens of a block
constexpr int kItems = 2;           // items a thread holds at once

template <int BYTES> struct VecOf;
template <> struct VecOf<16> { using type = uint4; };
template <> struct VecOf<8> { using type = uint2; };
template <> struct VecOf<4> { using type = uint32_t; };
template <> struct VecOf<2> { using type = uint16_t; };

template <class T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <class T, int E> union Vec {
    typename VecOf<(int)sizeof(T) * E>::type raw;
    T e[E];
    __device__ Vec() {}
};

// n / d for n < 2^31: by the reciprocal where that is exact (n d < 2^32), else plainly.
struct Div {
    unsigned d, mul;                // mul 0: plain
    __device__ __forceinline__ int operator()(int n) const {
        return mul ? (int)__umulhi((unsigned)n, mul) : n / (int)d;
    }
};
Div make_div(long long d, long long max_n) {
    Div v{(unsigned)d, 0u};
    if (d > 1 && max_n * d < (1LL << 32)) v.mul = (unsigned)((1ULL << 32) / d + 1);
    return v;
}

struct RopeShape {
    int tpb, heads, ipr_rot, ipr_copy, per_tok;     // heads that turn; items of a turning and of a copied head, of a token
    Div by_tok, by_rot, by_copy;
};

struct Smem {
    int seq_page[kMaxTokens];       // page id of the token, -1: not stored
    int row[kMaxTokens];            // row inside the page
    int pos[kMaxTokens];            // position that turns the heads
    int live[kMaxTokens];           // 0: row outside every sequence
};

// One work item: two vectors of a head, at dims a and b.
struct Item {
    int lt, h, a, b;                // token of the block, head
    int cs;                         // index of the first cos / sin of a token, -1: copied
    int n;                          // vectors (a head's last pair may hold one)
    int n_turn;                     // interleaved: how many of them turn
};

template <int E> __device__ __forceinline__ Item item_of(const RopeParams& p, const RopeShape& g, int i) {
    Item it;
    it.lt = g.by_tok(i);
    int r = i - it.lt * g.per_tok, j;
    const bool turns = r < g.heads * g.ipr_rot;
    if (turns) {                    // the leading p.skip heads are left alone
        it.h = g.by_rot(r);
        j = r - it.h * g.ipr_rot;
        it.h += p.skip;
    } else {
        r -= g.heads * g.ipr_rot;
        it.h = g.by_copy(r);
        j = r - it.h * g.ipr_copy;
        it.h += p.H - p.n_kv;
    }
    it.cs = -1;
    it.n = it.n_turn = 2;
    const int rot = p.inv_freq ? p.rot : 0;
    if (turns && !p.interleaved && j * E < rot / 2) {
        it.a = j * E;
        it.b = it.a + rot / 2;
        it.cs = it.a;
    } else {
        // two consecutive vectors
        it.a = turns && !p.interleaved ? rot + (j - rot / 2 / E) * 2 * E : j * 2 * E;
        it.b = it.a + E;
        if (turns && p.interleaved && it.a < rot) it.cs = it.a / 2;
        if (it.b >= rot) it.n_turn = 1;
        if (it.b >= p.D) { it.n = 1; it.b = it.a; }
    }
    return it;
}

template <class T, int E>
__device__ __forceinline__ void turn(const RopeParams& p, const float2* cs, const Item& it, Vec<T, E>& a, Vec<T, E>& b) {
    if (!p.interleaved || E == 1) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float2 c = cs[e];
            const float x = to_f(a.e[e]), y = to_f(b.e[e]);
            a.e[e] = from_f<T>(fmaf(x, c.x, -(y * c.y)));
            b.e[e] = from_f<T>(fmaf(x, c.y, y * c.x));
        }
    } else {
        // pair k of a vector: elements 2k, 2k + 1
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            Vec<T, E>& w = v ? b : a;
            if (v >= it.n_turn) break;
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float2 c = cs[v * (E / 2) + e / 2];
                const float x = to_f(w.e[e]), y = to_f(w.e[e + 1]);
                w.e[e] = from_f<T>(fmaf(x, c.x, -(y * c.y)));
                w.e[e + 1] = from_f<T>(fmaf(x, c.y, y * c.x));
            }
        }
    }
}

template <class T, int E>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p,
                                                        const __grid_constant__ RopeShape g) {
    using V = typename VecOf<(int)sizeof(T) * E>::type;
    extern __shared__ __align__(16) float2 cs[];        // [tpb][rot / 2]
    __shared__ Smem s;
    const long long t0 = (long long)blockIdx.x * g.tpb;
    const int ntok = (int)min((long long)g.tpb, p.T - t0), items = ntok * g.per_tok;
    grid_dependency_wait();
    grid_launch_dependents();
    // this thread's first items are on their way before anything else is known
    Item it[kItems];
    Vec<T, E> a[kItems], b[kItems];
    auto load = [&](int i0) {
#pragma unroll
        for (int u = 0; u < kItems; ++u) {
            const int i = i0 + u * kThreads;
            if (i < items) {
                it[u] = item_of<E>(p, g, i);
                const T* x = static_cast<const T*>(p.src) + (t0 + it[u].lt) * p.src_ts + it[u].h * p.src_hs;
                a[u].raw = *reinterpret_cast<const V*>(x + it[u].a);
                b[u].raw = *reinterpret_cast<const V*>(x + it[u].b);
            }
        }
    };
    load(threadIdx.x);
    if ((int)threadIdx.x < ntok) {
        const int i = threadIdx.x, t = (int)t0 + i;
        int live = 1, pos = 0, page = -1, row = 0;
        if (p.n_kv > 0) {
            const int q = seq_of_row(p.q_starts, p.n_seqs, t);
            live = q >= 0;
            if (live) {
                const int place = __ldg(p.kv_lens + q) - __ldg(p.q_starts + q + 1) + t;
                pos = place;
                if (place >= 0 && place / p.page < p.max_pages) {
                    page = __ldg(p.table + (long long)q * p.max_pages + place / p.page);
                    row = place % p.page;
                    if (page >= p.n_pages) page = -1;
                }
            }
        }
        if (p.positions) pos = __ldg(p.positions + t);
        s.live[i] = live; s.pos[i] = pos; s.seq_page[i] = page; s.row[i] = row;
    }
    __syncthreads();
    const int half = p.inv_freq ? p.rot / 2 : 0;
    for (int k = threadIdx.x; k < ntok * half; k += kThreads) {
        const int lt = k / half;
        const double turns = (double)s.pos[lt] * (double)__ldg(p.inv_freq + (k - lt * half)) * 0.15915494309189535;
        float sn, c;
        sincospif(2.0f * (float)(turns - rint(turns)), &sn, &c);
        cs[k] = make_float2(c * p.magnitude, sn * p.magnitude);
    }
    __syncthreads();
    for (int i0 = threadIdx.x; i0 < items; i0 += kItems * kThreads) {
        if (i0 != (int)threadIdx.x) load(i0);
#pragma unroll
        for (int u = 0; u < kItems; ++u) {
            if (i0 + u * kThreads >= items || !s.live[it[u].lt]) continue;
            const int lt = it[u].lt, h = it[u].h;
            T* d;
            if (h < p.n_dst) {
                d = static_cast<T*>(p.dst) + (t0 + lt) * p.dst_ts + h * p.dst_hs;
            } else {
                const int pg = s.seq_page[lt];
                if (pg < 0) continue;
                const bool isv = h >= p.n_dst + p.n_kv;
                d = static_cast<T*>(isv ? p.v : p.k) + (long long)pg * p.page_s + (long long)s.row[lt] * p.tok_s +
                    (long long)(h - p.n_dst - (isv ? p.n_kv : 0)) * p.head_s;
            }
            const bool rot = it[u].cs >= 0;
            if (rot) turn<T, E>(p, cs + lt * half + it[u].cs, it[u], a[u], b[u]);
            if (rot || p.copy_tail) {
                *reinterpret_cast<V*>(d + it[u].a) = a[u].raw;
                if (it[u].n == 2) *reinterpret_cast<V*>(d + it[u].b) = b[u].raw;
            }
        }
    }
}

template <class T, int E> cudaError_t launch_te(const RopeParams& p, cudaStream_t st) {
    const int rot = p.inv_freq ? p.rot : 0;
    // items per head: pairs of the half layout plus pairs of copied vectors
    const int ipr_rot = p.interleaved ? (p.D + 2 * E - 1) / (2 * E) : rot / 2 / E + (p.D - rot + 2 * E - 1) / (2 * E);
    const int ipr_copy = (p.D + 2 * E - 1) / (2 * E);
    const long long per_tok = (long long)(p.H - p.n_kv - p.skip) * ipr_rot + (long long)p.n_kv * ipr_copy;
    if (per_tok == 0) return cudaSuccess;
    if (per_tok > 0x3FFFFFF) return cudaErrorInvalidValue;
    // tokens of a block: up to 3 items a thread; fewer when that would leave
    // multiprocessors idle.  (One token a warp without block barriers, or
    // blocks that walk over tokens with the next one's loads ahead, measured no
    // faster: 8192 x 32 x 128 f16 rows 29-42 and 25-35 us.)
    long long tpb = 3 * kThreads / per_tok;
    tpb = tpb < 1 ? 1 : tpb > kMaxTokens ? kMaxTokens : tpb;
    const long long fill = ((long long)p.T + api_sms() - 1) / api_sms();
    if (tpb > fill) tpb = fill;
    const long long grid = (p.T + tpb - 1) / tpb;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    const size_t smem = (size_t)tpb * (rot / 2) * sizeof(float2);
    RopeShape g = {};
    g.tpb = (int)tpb;
    g.heads = p.H - p.n_kv - p.skip;
    g.ipr_rot = ipr_rot;
    g.ipr_copy = ipr_copy;
    g.per_tok = (int)per_tok;
    g.by_tok = make_div(per_tok, tpb * per_tok);
    g.by_rot = make_div(ipr_rot, per_tok);
    g.by_copy = make_div(ipr_copy, per_tok);
    // smem: at most 32 tokens x 128 pairs x 8 bytes = 32 KB
    return launch_dependent(rope_kernel<T, E>, dim3((unsigned)grid), dim3(kThreads), smem, st, p, g);
}

template <class T> cudaError_t launch_t(const RopeParams& p, int vec_bytes, cudaStream_t st) {
    constexpr int ES = (int)sizeof(T);
    if (vec_bytes >= 16) return launch_te<T, 16 / ES>(p, st);
    if (vec_bytes == 8) return launch_te<T, 8 / ES>(p, st);
    if constexpr (ES == 2) {
        if (vec_bytes == 4) return launch_te<T, 2>(p, st);
    }
    return launch_te<T, 1>(p, st);
}

}  // namespace

cudaError_t launch_rope(int dtype, const RopeParams& p, int vec_bytes, cudaStream_t st) {
    switch (dtype) {
        case 0: return launch_t<float>(p, vec_bytes, st);
        case 1: return launch_t<__half>(p, vec_bytes, st);
        case 2: return launch_t<__nv_bfloat16>(p, vec_bytes, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace qmv
