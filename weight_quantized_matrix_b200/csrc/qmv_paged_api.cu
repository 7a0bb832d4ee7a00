// qmv_paged_api.cu -- C entries of the rotary rotation, the append to a paged
// cache and the attention over it: argument checks and the choice of kernel.
#include <float.h>
#include <math.h>

#include <initializer_list>

#include "qmv.h"
#include "qmv_attn_sched.cuh"

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int elem_bytes(int dtype) { return dtype == QMV_F32 ? 4 : 2; }

bool known_dtype(int dtype) { return dtype == QMV_F32 || dtype == QMV_F16 || dtype == QMV_BF16; }

// Largest of 16, 8, 4, 2 that divides every given byte count.
int common_vec(std::initializer_list<long long> bytes) {
    long long all = 16;
    for (long long b : bytes) all |= b < 0 ? -b : b;
    return (int)(all & -all);
}

// Whether rows of `D` elements at a * sa + b * sb (+ c * sc) can share an
// element: strides taken from the smallest, each must clear what lies inside.
bool disjoint(int D, int n, const long long* size, const long long* stride) {
    long long s[3], c[3];
    int m = 0;
    for (int i = 0; i < n; ++i)
        if (size[i] > 1) { s[m] = stride[i]; c[m] = size[i]; ++m; }
    for (int i = 0; i < m; ++i)
        for (int j = i + 1; j < m; ++j)
            if (s[j] < s[i]) { long long t = s[i]; s[i] = s[j]; s[j] = t; t = c[i]; c[i] = c[j]; c[j] = t; }
    long long span = D;
    for (int i = 0; i < m; ++i) {
        if (s[i] < span) return false;
        span = s[i] * (c[i] - 1) + span;
    }
    return true;
}

int check_rotation(int D, int rot_dim, int layout) {
    if (layout != QMV_ROPE_HALF && layout != QMV_ROPE_INTERLEAVED) return QMV_EUNSUPPORTED;
    if (rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > D) return QMV_EINVAL;
    return QMV_OK;
}

int check_cache(const qmv_paged_kv* kv) {
    if (!kv) return QMV_EINVAL;
    if (!known_dtype(kv->dtype)) return QMV_EUNSUPPORTED;
    if (kv->n_pages < 1 || kv->page_size < 1 || kv->n_kv_heads < 1 || kv->head_dim < 1 || kv->n_seqs < 0 ||
        kv->max_pages < 1)
        return QMV_EINVAL;
    if (kv->head_dim > QMV_MAX_HEAD_DIM || kv->n_seqs > (1 << 30)) return QMV_EUNSUPPORTED;
    const long long size[3] = {kv->n_pages, kv->page_size, kv->n_kv_heads};
    const long long stride[3] = {kv->page_stride, kv->token_stride, kv->head_stride};
    if (!disjoint(kv->head_dim, 3, size, stride)) return QMV_EINVAL;
    return QMV_OK;
}

// Which kernel of the 16-bit types: 16 rows a kv head and unit, keys streamed by
// warp, or 256 rows on the tensor cores.  Measured, heads of 128, 4 query heads
// a kv head (us, few / many): 32 sequences of 4000 keys, 16 rows 90 / 137, 24
// rows 175 / 138; one of 100000, 32 rows 141 / 164, 48 rows 200 / 167; one of 2000,
// 96 rows 23 / 32; 80 tokens alone 18 / 12, after 600 keys 31 / 21; 12 x 20 tokens
// 30 / 18, 12 x 160 178 / 27; 12 x 20 of 8 heads on one after 600 keys 15 / 30.
// So: up to 16 rows the first; up to 32 while its units leave SMs free (it reads
// keys twice, from the second-level cache); and more while its units all find an
// SM and its tiles, by the longest sequence the table can hold, are so few that
// a call's latency decides.  Many heads of few rows leave the second one's units
// as many and nearly empty (12 x 40 tokens, 16 heads of 64: 13 / 19), so up to 48
// rows then too.
bool many_rows(const qmv::AttnParams& p, int max_q_len) {
    const double rows = (double)max_q_len * p.G, sms = qmv::api_sms(), heads = (double)p.n_seqs * p.Hkv;
    const double units = heads * ceil(rows / 16), tiles = (double)p.max_pages * p.page / 64;
    if (rows <= 16 || (rows <= 32 && units <= 2 * sms)) return false;
    if (units > sms && (rows > 48 || heads <= sms)) return true;
    return units * tiles > 24 * sms;
}

int check_cache_pointers(const qmv_paged_kv* kv) {
    if (!kv->k || !kv->v || !kv->page_table || !kv->q_starts || !kv->kv_lens) return QMV_EINVAL;
    const size_t eb = (size_t)elem_bytes(kv->dtype);
    if (!aligned(kv->k, eb) || !aligned(kv->v, eb) || !aligned(kv->page_table, 4) || !aligned(kv->q_starts, 4) ||
        !aligned(kv->kv_lens, 4))
        return QMV_EALIGN;
    return QMV_OK;
}

}  // namespace

extern "C" {

int qmv_rope_frequencies(float* inv_freq, float* magnitude, int rot_dim, double base, int scaling, double factor,
                         int original_length, double turns_fast, double turns_slow) {
    if (scaling < QMV_ROPE_PLAIN || scaling > QMV_ROPE_BANDED) return QMV_EUNSUPPORTED;
    if (!inv_freq || !magnitude || rot_dim < 2 || rot_dim % 2 != 0) return QMV_EINVAL;
    if (!(base > 1.0) || !(base < 1e300)) return QMV_EINVAL;
    if (scaling != QMV_ROPE_PLAIN && (!(factor >= 1.0) || !(factor < 1e9))) return QMV_EINVAL;
    if (scaling == QMV_ROPE_BASE && rot_dim <= 2 && factor > 1.0) return QMV_EINVAL;
    if (scaling == QMV_ROPE_BANDED && (original_length < 1 || !(turns_slow > 0.0) || !(turns_fast > turns_slow)))
        return QMV_EINVAL;
    const double kTwoPi = 6.283185307179586;
    if (scaling == QMV_ROPE_BASE) base *= pow(factor, (double)rot_dim / (rot_dim - 2));
    double first = 0.0, last = 0.0;
    if (scaling == QMV_ROPE_BANDED) {
        // index of the pair that makes the given number of turns over the trained length
        const double per = (double)rot_dim / (2.0 * log(base));
        first = floor(per * log(original_length / (turns_fast * kTwoPi)));
        last = ceil(per * log(original_length / (turns_slow * kTwoPi)));
        if (first < 0.0) first = 0.0;
        if (last > rot_dim - 1) last = rot_dim - 1;
        if (last <= first) last = first + 0.001;
    }
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = pow(base, -2.0 * i / rot_dim);
        if (scaling == QMV_ROPE_LINEAR) f /= factor;
        if (scaling == QMV_ROPE_BANDED) {
            double w = (i - first) / (last - first);        // 0: kept, 1: stretched
            w = w < 0.0 ? 0.0 : w > 1.0 ? 1.0 : w;
            f = f * (1.0 - w) + f / factor * w;
        }
        inv_freq[i] = (float)f;
    }
    *magnitude = scaling == QMV_ROPE_BANDED ? (float)(0.1 * log(factor) + 1.0) : 1.0f;
    return QMV_OK;
}

int qmv_rope(const void* x, void* y, const int* positions, const float* inv_freq, int T, int H, int D, int rot_dim,
             int layout, float magnitude, long long x_token_stride, long long x_head_stride, long long y_token_stride,
             long long y_head_stride, int dtype, void* stream) {
    if (!known_dtype(dtype)) return QMV_EUNSUPPORTED;
    if (T < 0 || H < 0 || D < 1) return QMV_EINVAL;
    if (D > QMV_MAX_HEAD_DIM) return QMV_EUNSUPPORTED;
    int st = check_rotation(D, rot_dim, layout);
    if (st != QMV_OK) return st;
    if (T == 0 || H == 0) return QMV_OK;
    const long long size[2] = {T, H}, ys[2] = {y_token_stride, y_head_stride};
    if (x_token_stride < 0 || x_head_stride < 0 || !disjoint(D, 2, size, ys)) return QMV_EINVAL;
    if (!x || !y || !positions || !inv_freq) return QMV_EINVAL;
    const long long es = elem_bytes(dtype);
    if (!aligned(x, es) || !aligned(y, es) || !aligned(positions, 4) || !aligned(inv_freq, 4)) return QMV_EALIGN;
    const bool in_place = x == y && x_token_stride == y_token_stride && x_head_stride == y_head_stride;
    if (!in_place) {
        const char* x0 = static_cast<const char*>(x);
        const char* y0 = static_cast<const char*>(y);
        const char* x1 = x0 + ((T - 1LL) * x_token_stride + (H - 1LL) * x_head_stride + D) * es;
        const char* y1 = y0 + ((T - 1LL) * y_token_stride + (H - 1LL) * y_head_stride + D) * es;
        if (x0 < y1 && y0 < x1) return QMV_EINVAL;
    }
    qmv::RopeParams p = {};
    p.src = x; p.src_ts = x_token_stride; p.src_hs = x_head_stride;
    p.dst = y; p.dst_ts = y_token_stride; p.dst_hs = y_head_stride;
    p.n_dst = p.H = H;
    p.T = T; p.D = D; p.rot = rot_dim; p.interleaved = layout == QMV_ROPE_INTERLEAVED;
    p.positions = positions; p.inv_freq = inv_freq; p.magnitude = magnitude;
    p.copy_tail = !in_place;
    const int vec = common_vec({(long long)reinterpret_cast<uintptr_t>(x), (long long)reinterpret_cast<uintptr_t>(y),
                                x_token_stride * es, x_head_stride * es, y_token_stride * es, y_head_stride * es,
                                D * es, (p.interleaved ? rot_dim : rot_dim / 2) * es});
    return qmv::api_finish(qmv::launch_rope(dtype, p, vec, static_cast<cudaStream_t>(stream)));
}

int qmv_kv_append(const void* qkv, long long qkv_stride, const qmv_paged_kv* kv, const int* positions,
                  const float* inv_freq, void* q_out, long long q_out_stride, int T, int n_q_heads, int rot_dim,
                  int layout, float magnitude, void* stream) {
    int st = check_cache(kv);
    if (st != QMV_OK) return st;
    if (T < 0 || n_q_heads < 0) return QMV_EINVAL;
    const int D = kv->head_dim;
    if (inv_freq) {
        st = check_rotation(D, rot_dim, layout);
        if (st != QMV_OK) return st;
    }
    const long long wide = ((long long)n_q_heads + 2LL * kv->n_kv_heads) * D;
    if (qkv_stride < wide) return QMV_EINVAL;
    if (q_out && (n_q_heads < 1 || q_out_stride < (long long)n_q_heads * D)) return QMV_EINVAL;
    if (T == 0 || kv->n_seqs == 0) return QMV_OK;
    if (!qkv) return QMV_EINVAL;
    st = check_cache_pointers(kv);
    if (st != QMV_OK) return st;
    const long long es = elem_bytes(kv->dtype);
    if (!aligned(qkv, es) || (q_out && !aligned(q_out, es)) || (inv_freq && !aligned(inv_freq, 4)) ||
        (positions && !aligned(positions, 4)))
        return QMV_EALIGN;
    if (q_out && (q_out != qkv || q_out_stride != qkv_stride)) {
        // only the very same place may be shared with the rows that are read
        const char* a0 = static_cast<const char*>(qkv);
        const char* b0 = static_cast<const char*>(q_out);
        const char* a1 = a0 + ((T - 1LL) * qkv_stride + wide) * es;
        const char* b1 = b0 + ((T - 1LL) * q_out_stride + (long long)n_q_heads * D) * es;
        if (a0 < b1 && b0 < a1) return QMV_EINVAL;
    }
    qmv::RopeParams p = {};
    p.src = qkv; p.src_ts = qkv_stride; p.src_hs = D;
    p.dst = q_out; p.dst_ts = q_out_stride; p.dst_hs = D;
    p.skip = q_out ? 0 : n_q_heads;
    p.n_dst = n_q_heads; p.n_kv = kv->n_kv_heads; p.H = n_q_heads + 2 * kv->n_kv_heads;
    p.T = T; p.D = D; p.rot = inv_freq ? rot_dim : 0; p.interleaved = layout == QMV_ROPE_INTERLEAVED;
    p.positions = positions; p.inv_freq = inv_freq; p.magnitude = magnitude;
    p.copy_tail = 1;
    p.k = kv->k; p.v = kv->v;
    p.page_s = kv->page_stride; p.tok_s = kv->token_stride; p.head_s = kv->head_stride;
    p.table = kv->page_table; p.q_starts = kv->q_starts; p.kv_lens = kv->kv_lens;
    p.n_seqs = kv->n_seqs; p.n_pages = kv->n_pages; p.page = kv->page_size; p.max_pages = kv->max_pages;
    const int vec = common_vec(
        {(long long)reinterpret_cast<uintptr_t>(qkv), (long long)reinterpret_cast<uintptr_t>(q_out), qkv_stride * es,
         q_out ? q_out_stride * es : 0, (long long)reinterpret_cast<uintptr_t>(kv->k),
         (long long)reinterpret_cast<uintptr_t>(kv->v), kv->page_stride * es, kv->token_stride * es,
         kv->head_stride * es, D * es, inv_freq ? (p.interleaved ? rot_dim : rot_dim / 2) * es : 0});
    return qmv::api_finish(qmv::launch_rope(kv->dtype, p, vec, static_cast<cudaStream_t>(stream)));
}

int qmv_paged_attention(const void* q, const qmv_paged_kv* kv, void* out, float* lse, int T, int n_q_heads,
                        float scale, int causal, int window, float softcap, const float* slopes,
                        long long q_token_stride, long long q_head_stride, long long out_token_stride,
                        long long out_head_stride, int max_q_len, void* workspace, void* stream) {
    int st = check_cache(kv);
    if (st != QMV_OK) return st;
    if (T < 0 || n_q_heads < 1 || n_q_heads % kv->n_kv_heads != 0 || max_q_len < 0) return QMV_EINVAL;
    // row counts are rounded up to a step of 32 tiles of 256 rows in an int
    if ((long long)T * n_q_heads > 0x7FFFFFFF - 33 * 256) return QMV_EUNSUPPORTED;
    if (causal != 0 && causal != 1) return QMV_EINVAL;
    if (window < 0 || !(softcap >= 0.0f) || isinf(softcap * qmv::kLog2e) || !(scale > 0.0f) || isinf(scale * qmv::kLog2e)) return QMV_EINVAL;
    // a subnormal quotient has too few bits for the scores it is multiplied into
    if (softcap > 0.0f && (isinf(scale / softcap * (2.0f * qmv::kLog2e)) || scale / softcap < FLT_MIN)) return QMV_EINVAL;
    const int D = kv->head_dim;
    const long long size[2] = {T, n_q_heads}, os[2] = {out_token_stride, out_head_stride};
    if (q_token_stride < 0 || q_head_stride < 0 || !disjoint(D, 2, size, os)) return QMV_EINVAL;
    if (T == 0 || kv->n_seqs == 0) return QMV_OK;
    if (!q || !out) return QMV_EINVAL;
    st = check_cache_pointers(kv);
    if (st != QMV_OK) return st;
    const size_t eb = (size_t)elem_bytes(kv->dtype);
    if (!aligned(q, eb) || !aligned(out, eb) || (lse && !aligned(lse, 4)) || (slopes && !aligned(slopes, 4)) ||
        (workspace && !aligned(workspace, 16)))
        return QMV_EALIGN;
    qmv::AttnParams p = {};
    p.q = q; p.k = kv->k; p.v = kv->v; p.out = out; p.lse = lse;
    p.table = kv->page_table; p.q_starts = kv->q_starts; p.kv_lens = kv->kv_lens; p.slopes = slopes;
    p.q_ts = q_token_stride; p.q_hs = q_head_stride; p.o_ts = out_token_stride; p.o_hs = out_head_stride;
    p.page_s = kv->page_stride; p.tok_s = kv->token_stride; p.head_s = kv->head_stride;
    p.T = T; p.Hq = n_q_heads; p.Hkv = kv->n_kv_heads; p.G = n_q_heads / kv->n_kv_heads; p.D = D;
    p.n_seqs = kv->n_seqs; p.n_pages = kv->n_pages; p.page = kv->page_size; p.max_pages = kv->max_pages;
    // exact for r G < 2^32 (G > 1; r < T G)
    if (p.G > 1 && (long long)T * p.G * p.G < (1LL << 32)) p.g_mul = (unsigned)((1ULL << 32) / p.G + 1);
    p.causal = causal;
    p.window = window;
    p.scale = scale; p.softcap = softcap;
    if (workspace) {
        p.counters = static_cast<unsigned*>(workspace);
        p.partials = reinterpret_cast<float*>(static_cast<char*>(workspace) + qmv::kAttnPartialsAt);
    }
    auto s = static_cast<cudaStream_t>(stream);
    // 16-byte copies of whole heads: the kernels that stream keys and values
    const int vec = common_vec({(long long)reinterpret_cast<uintptr_t>(q), (long long)reinterpret_cast<uintptr_t>(kv->k),
                                (long long)reinterpret_cast<uintptr_t>(kv->v), q_token_stride * (long long)eb,
                                q_head_stride * (long long)eb, kv->page_stride * (long long)eb,
                                kv->token_stride * (long long)eb, kv->head_stride * (long long)eb, D * (long long)eb});
    // whose places (in 16 bytes) fit an int: caches of up to 32 GiB a tensor
    const long long per16 = 16 / (long long)eb;
    const bool near = (kv->n_pages - 1LL) * kv->page_stride + (kv->page_size - 1LL) * kv->token_stride <= (per16 << 31) - per16;
    if (vec == 16 && near && kv->dtype == QMV_F32) return qmv::api_finish(qmv::launch_attn_f32(p, s));
    if (vec == 16 && near) {
        p.fault = qmv::api_fault_word();
        if (!p.fault) return QMV_ECUDA;
        p.test_skip = qmv::api_test_skip();
        const int most = max_q_len > 0 && max_q_len < T ? max_q_len : T;
        if (D <= 128 && many_rows(p, most)) return qmv::api_finish(qmv::launch_attn_chunk(kv->dtype, p, s));
        return qmv::api_finish(qmv::launch_attn_few(kv->dtype, p, most, s));
    }
    return qmv::api_finish(qmv::launch_attn_rows(kv->dtype, p, s));
}

}  // extern "C"
