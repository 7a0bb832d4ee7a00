// qmv_paged.cuh -- what the paged-cache entry points share: the launch
// parameters, the batch description read on the device (sequence of a token,
// visible keys of a row, page of a position) and the host-side launch helpers.
#pragma once

#include <atomic>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace qmv {

// Implemented in qmv_api.cu for the C entries that live in other files.
int api_finish(cudaError_t e);      // QMV_OK, or QMV_ECUDA (recorded for qmv_last_cuda_error)
int api_sms();                      // multiprocessors of the current device
unsigned* api_fault_word();         // fault word of the current device, null if unknown
bool api_pdl();                     // programmatic dependent launch (off with QMV_PDL=0)
int api_test_skip();                // whether qmv_test_skip_last_copy is on
bool api_encode_pages(CUtensorMap* m, const void* base, bool f16, int D, int page, int heads, int pages, long long tok_s,
                      long long head_s, long long page_s, int rows);

// Rotation and append: rows of heads, `n_rot` rotated ones first.
struct RopeParams {
    const void* src;                // row t, head h at src + t * src_ts + h * src_hs
    long long src_ts, src_hs;
    void* dst;                      // heads [0, n_dst) go to dst + t * dst_ts + h * dst_hs
    long long dst_ts, dst_hs;
    int skip;                       // append: leading heads that are left alone (no q_out)
    int n_dst;                      // heads written to dst (q); the next n_kv are K, then n_kv V
    int n_kv;
    int H;                          // heads of a row: n_dst + 2 n_kv
    int T, D, rot, interleaved;
    const int* positions;           // [T], or null: the token's place in its sequence
    const float* inv_freq;          // [rot / 2], or null: no rotation
    float magnitude;
    int copy_tail;                  // 1: write dims >= rot of dst too (0: in place, they are there)
    // paged cache (append)
    void* k;
    void* v;
    long long page_s, tok_s, head_s;
    const int* table;
    const int* q_starts;
    const int* kv_lens;
    int n_seqs, n_pages, page, max_pages;
};

struct AttnParams {
    const void* q;
    const void* k;
    const void* v;
    void* out;
    float* lse;                     // [T, Hq] or null
    const int* table;               // [n_seqs, max_pages]
    const int* q_starts;            // [n_seqs + 1]
    const int* kv_lens;             // [n_seqs]
    const float* slopes;            // [Hq] or null
    long long q_ts, q_hs, o_ts, o_hs;
    long long page_s, tok_s, head_s;
    int T, Hq, Hkv, G, D;
    unsigned g_mul;                 // ceil(2^32 / G) where rows / G is exact by it, else 0
    int n_seqs, n_pages, page, max_pages;
    int causal, window;             // window 0: none
    float scale, softcap;           // softcap 0: none
    unsigned* counters;             // workspace, null: no split over the keys
    float* partials;
    unsigned* fault;
    int test_skip;                  // tests only (qmv_test_skip_last_copy)
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ------------------------------------------------------------ device side --
// q_starts[b], kept inside the T rows that exist whatever the table holds.
__device__ __forceinline__ int row_start(const int* q_starts, int b, int T) {
    return min(max(__ldg(q_starts + b), 0), T);
}

// Sequence that holds row t (the last b with q_starts[b] <= t), or -1 when t
// lies before the first or behind the last sequence.
__device__ __forceinline__ int seq_of_row(const int* q_starts, int n_seqs, int t) {
    if (t < __ldg(q_starts) || t >= __ldg(q_starts + n_seqs)) return -1;
    int lo = 0, hi = n_seqs;        // q_starts[lo] <= t < q_starts[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(q_starts + mid) <= t) lo = mid; else hi = mid;
    }
    return lo;
}

// Keys [lo, hi) that the token at position pos of a sequence of len keys sees.
__device__ __forceinline__ void visible_keys(const AttnParams& p, int pos, int len, int& lo, int& hi) {
    hi = p.causal ? min(len, pos + 1) : len;
    lo = p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0;
    if (hi < 0) hi = 0;
}

// Packed row r (new token r / G, head r % G of its kv head) -> token.
__device__ __forceinline__ int token_of(const AttnParams& p, int r) {
    return p.g_mul ? (int)__umulhi((unsigned)r, p.g_mul) : p.G == 1 ? r : r / p.G;
}

__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// -------------------------------------------------------------- host side --
// Lets a kernel use `smem` bytes of dynamic shared memory, once per device.
template <class Kern>
inline cudaError_t allow_smem(Kern kern, std::atomic<unsigned>& configured, int smem) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned bit = 1u << (dev & 31);
    if (configured.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) configured.fetch_or(bit, std::memory_order_acq_rel);
    return e;
}

// Launch with programmatic dependent launch: the kernel may begin while the
// kernel before it drains, and waits for it before it touches memory.  Without it
// (api_pdl) the kernel's wait returns at once.
template <class Kern, class... Args>
inline cudaError_t launch_dependent(Kern kern, dim3 grid, dim3 block, size_t smem, cudaStream_t st, const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = api_pdl() ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// log2 of the page size, -1 if it is no power of two.
inline int page_shift_of(int page) {
    if (page & (page - 1)) return -1;
    int s = 0;
    while ((1 << s) < page) ++s;
    return s;
}

cudaError_t launch_rope(int dtype, const RopeParams& p, int vec_bytes, cudaStream_t st);
cudaError_t launch_attn_few(int dtype, const AttnParams& p, int max_q_len, cudaStream_t st);
cudaError_t launch_attn_chunk(int dtype, const AttnParams& p, cudaStream_t st);
cudaError_t launch_attn_f32(const AttnParams& p, cudaStream_t st);
cudaError_t launch_attn_rows(int dtype, const AttnParams& p, cudaStream_t st);

}  // namespace qmv
