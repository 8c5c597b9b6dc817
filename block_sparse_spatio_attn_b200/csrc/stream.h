// stream.h -- what the streaming attention calls share: the window mask's arithmetic and the
// parameters their kernels take.
#pragma once
#include <cstddef>
#include <cstdint>

#include "svga_internal.h"

namespace svga {

constexpr int kMaxMask = 1 << 24;  // largest window, sinks, block and token count

// ------------------------------------------------------------------------- the mask
// The keys query position p keeps are [lo, hi) and [0, sk); all three never decrease
// with p, so a run of queries keeps nothing outside [lo(first), hi(last)) and
// [0, sk(last)), and everything inside [lo(last), hi(first)) and [0, sk(first)).
struct MaskRange {
    int lo, hi, sk;
};

struct Mask {
    int causal, window, sinks, block;
};

__host__ __device__ __forceinline__ int floor_div(int a, int b)
{
    const int q = a / b;
    return (a % b != 0 && a < 0) ? q - 1 : q;
}

__host__ __device__ __forceinline__ int clamp_tokens(long long x, int n)
{
    return x < 0 ? 0 : (x > n ? n : (int)x);
}

__host__ __device__ __forceinline__ MaskRange mask_range(const Mask &m, int p, int nk)
{
    // block indices times block pass 32 bits: window and block are up to 2^24 each
    const long long b = m.block == 1 ? p : floor_div(p, m.block);
    const int own_end = clamp_tokens((b + 1) * m.block, nk);  // end of the query's own block
    MaskRange r;
    if (m.window < 0) {
        r.hi = m.causal ? own_end : nk;
        r.lo = 0;
        r.sk = 0;
        return r;
    }
    r.hi = m.causal ? own_end : clamp_tokens((b + m.window + 1) * m.block, nk);
    const int lo = clamp_tokens((b - m.window) * m.block, nk);
    r.lo = lo < r.hi ? lo : r.hi;
    const int sk = m.causal ? own_end : nk;
    r.sk = m.sinks < sk ? m.sinks : sk;
    return r;
}

// The queries that keep key j (0 <= j < nk) are the rows [first, end) of 0 .. nq - 1, with
// off = nk - nq: the inverse of mask_range, contiguous for every mask.
__host__ __device__ __forceinline__ void mask_rows(const Mask &m, int j, int nq, int off,
                                                   int &first, int &end)
{
    const long long b = m.block == 1 ? j : j / m.block;
    const bool sink = m.window >= 0 && j < m.sinks;
    long long a = 0, e = (long long)nq + off;  // positions
    bool all_before = false;
    if (m.causal)
        a = b * m.block;
    else if (m.window >= 0 && !sink)
        a = (b - m.window) * m.block;
    else
        all_before = true;
    if (m.window >= 0 && !sink) e = (b + m.window + 1) * m.block;
    first = all_before ? 0 : clamp_tokens(a - off, nq);
    end = clamp_tokens(e - off, nq);
    if (end < first) end = first;
}

// The 128-key chunks one run of query positions [p0, p1] visits: [0, a) for the sinks and
// [w0, w1) for the window (overlapping chunks count once), and the ones every query of
// the run keeps whole.
struct ChunkList {
    int a, w0, w1;   // visited
    int fa, f0, f1;  // full: c < fa, or f0 <= c < f1
    __host__ __device__ __forceinline__ bool visits(int c) const
    {
        return c < a || (c >= w0 && c < w1);
    }
    __host__ __device__ __forceinline__ bool full(int c) const
    {
        return c < fa || (c >= f0 && c < f1);
    }
};

// From the ranges of the run's first and last query.
template <int KN>
__host__ __device__ __forceinline__ ChunkList chunk_list(const MaskRange &r0, const MaskRange &r1)
{
    ChunkList c;
    c.a = (r1.sk + KN - 1) / KN;
    c.w0 = r0.lo / KN;
    c.w1 = r1.hi > r0.lo ? (r1.hi + KN - 1) / KN : c.w0;
    c.fa = r0.sk / KN;
    c.f0 = r1.lo <= r0.sk ? 0 : (r1.lo + KN - 1) / KN;  // sinks that reach the window join it
    c.f1 = r0.hi / KN;
    return c;
}

template <int KN>
__host__ __device__ __forceinline__ ChunkList chunk_list(const Mask &m, int p0, int p1, int nk)
{
    return chunk_list<KN>(mask_range(m, p0, nk), mask_range(m, p1, nk));
}

// The merged chunk list of two consecutive runs of queries.  The windows of consecutive
// positions touch or overlap, so every chunk of the list is visited by one of the runs.
__host__ __device__ __forceinline__ void merge_lists(const ChunkList &l0, const ChunkList &l1,
                                                     bool valid1, int &a, int &skip, int &end)
{
    a = l0.a;
    int w0 = l0.w0, w1 = l0.w1;
    if (valid1) {
        a = l1.a > a ? l1.a : a;
        if (l1.w1 > l1.w0) {
            if (w1 <= w0 || l1.w0 < w0) w0 = l1.w0;
            if (l1.w1 > w1) w1 = l1.w1;
        }
    }
    skip = w0 > a ? w0 : a;
    end = w1 > skip ? w1 : skip;
}

// The queries that keep any of the keys [k0, k1), in [first, end), and the ones that keep all of
// them, [all_first, all_end), from the queries of three keys: the first (a sink, if one is
// among them), the last, and the first that is no sink.  Each key's queries are contiguous, a
// sink's run to the end, and first rows and (sinks aside) ends never decrease with the key.
struct BlockRows {
    int first, end, all_first, all_end;
};

__host__ __device__ __forceinline__ int block_key(const Mask &m, int k0, int k1, int e)
{
    if (e == 0) return k0;
    if (e == 1) return k1 - 1;
    const int key = m.sinks < k1 - 1 ? m.sinks : k1 - 1;
    return key > k0 ? key : k0;
}

__host__ __device__ __forceinline__ BlockRows block_rows(const Mask &m, int k1, int nq, int first0,
                                                         int end0, int first1, int end1, int end2)
{
    BlockRows r;
    r.first = first0;
    r.end = end0 > end1 ? end0 : end1;
    r.all_first = first0 > first1 ? first0 : first1;
    r.all_end = m.window < 0 ? end0 : (m.sinks < k1 ? end2 : nq);
    return r;
}

#ifdef __CUDACC__
__device__ __forceinline__ MaskRange range_of_lane(const MaskRange &r, int lane)
{
    return {__shfl_sync(0xffffffffu, r.lo, lane), __shfl_sync(0xffffffffu, r.hi, lane),
            __shfl_sync(0xffffffffu, r.sk, lane)};
}
#endif

// --------------------------------------------------------------------------- splitting
// Division by a number the host knows: n / d = n ceil(2^shift / d) >> shift for 0 <= n < 2^31,
// with shift = 31 + ceil(log2 d) (the error n (2^shift mod d) / (d 2^shift) stays below 1 / d).
// A CTA's place among the items takes five divisions in a row before its first load, a hundred
// cycles or two each when the hardware's reciprocal has to do them.
struct FastDiv {
    uint32_t mul;
    int shift;
    __host__ __device__ __forceinline__ int of(int n) const
    {
        return (int)(((unsigned long long)(uint32_t)n * mul) >> shift);
    }
};

inline FastDiv fast_div(int d)
{
    int s = 0;
    while ((1ll << s) < d) ++s;
    return {(uint32_t)(((1ull << (31 + s)) + d - 1) / d), 31 + s};
}

// Work items in launch order, the first n1 of them split k1 ways and the others k2 ways over
// as many CTAs.  Parts of a split item leave partial sums in the workspace, in slots
// numbered over the split items' parts in launch order.
struct Split {
    int items, n1, k1, k2;
    __host__ __device__ __forceinline__ int k(int item) const { return item < n1 ? k1 : k2; }
    __host__ __device__ __forceinline__ long long ctas() const
    {
        return (long long)n1 * k1 + (long long)(items - n1) * k2;
    }
    // (by1, by2: division by k1 and k2)
    __device__ __forceinline__ void of_block(int blk, const FastDiv &by1, const FastDiv &by2,
                                             int &item, int &part) const
    {
        const bool head = blk < n1 * k1;
        const int r = head ? blk : blk - n1 * k1, q = head ? by1.of(r) : by2.of(r);
        item = head ? q : n1 + q;
        part = r - q * (head ? k1 : k2);
    }
    __host__ __device__ __forceinline__ long long slot(int item, int part) const
    {
        if (item < n1) return (long long)item * k1 + part;
        return (k1 > 1 ? (long long)n1 * k1 : 0) + (long long)(item - n1) * k2 + part;
    }
    __host__ __device__ __forceinline__ long long slots() const
    {
        return (k1 > 1 ? (long long)n1 * k1 : 0) + (k2 > 1 ? (long long)(items - n1) * k2 : 0);
    }
    // the items a join kernel has to visit: [from, to)
    __host__ __device__ __forceinline__ int split_from() const { return k1 > 1 ? 0 : n1; }
    __host__ __device__ __forceinline__ int split_to() const { return k2 > 1 ? items : n1; }
};

// ------------------------------------------------------------------- kernel parameters
// A strided tensor in kernel parameters (strides in elements).
struct View {
    char *p;
    long long sb, sh, st;
};

struct WindowShape {
    int batch, hq, hk, group, tq, tk;
    Mask mask;
    const int32_t *q_lens, *k_lens;
    int32_t *status;
};

// tensor_map.cu: map (64 columns, token, d / 64, head, batch) of a strided view of 16-bit
// elements, 128-byte swizzle: one copy brings box_rows tokens whole, their first 64 columns
// together and then their second.  A broadcast (stride 0) or one-entry
// dimension is mapped with extent 1: coordinates in it are multiplied by *mul_h / *mul_b
// (0 or 1).  False: the driver refused it.
bool make_view_map(void *map, const svga_view &v, int batch, int heads, int tokens, int d,
                   svga_dtype dt, int box_rows, int *mul_h, int *mul_b);
// Map of contiguous rows of 16-bit elements as (64 columns, rows, d / 64): one copy of a box
// brings box_rows whole rows, each 64 columns of them together.
bool make_rows_map(void *map, const void *base, long long rows, int d, svga_dtype dt,
                   int box_rows);
void *encode_tiled_entry();  // cuTensorMapEncodeTiled, or NULL

// rotary.cu
svga_status launch_rotary_table(const svga_rotary_spec *spec, double theta, float *table,
                                void *stream);
svga_status launch_rotary(const svga_view &src, const svga_view &dst, int batch, int heads,
                          int tokens, int d, svga_dtype dt, const svga_rotary_spec *spec,
                          const float *table, const int32_t *positions, long long first_token,
                          int inverse, int32_t *status, void *stream);
svga_status launch_append(const svga_view &k, const svga_view &v, int tokens,
                          const int32_t *new_lens, const svga_paged_cache *cache,
                          const svga_rotary_spec *spec, const float *table, void *stream);

// decode.cu
svga_status launch_decode(const svga_view &q, const svga_view &o, float *lse, int q_heads,
                          const svga_paged_cache *cache, const svga_window_mask *mask,
                          float scale, void *stream);

// window_fwd.cu, window_bwd.cu
size_t window_fwd_workspace(const svga_window_problem *p);
size_t window_bwd_workspace(const svga_window_problem *p);
svga_status launch_window_fwd(const svga_view &q, const svga_view &k, const svga_view &v,
                              const svga_view &o, float *lse, const svga_window_problem *p,
                              float scale, void *ws, void *stream);
svga_status launch_window_bwd(const svga_view &d_o, const svga_view &q, const svga_view &k,
                              const svga_view &v, const svga_view &o, const float *lse,
                              const svga_view &dq, const svga_view &dk, const svga_view &dv,
                              const svga_window_problem *p, float scale, void *ws, void *stream);

svga_status check_launch_of(const char *what);  // cudaGetLastError as a status

#ifdef __CUDACC__
// Launch of a kernel that begins while the one before it in the stream is still running and
// waits for it itself (pdl_wait, in every CTA, before it touches what that one writes).
template <typename... Params, typename... Args>
svga_status launch_after(void (*kernel)(Params...), dim3 grid, unsigned threads, size_t smem,
                         cudaStream_t st, const char *what, const Args &...args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) return check_launch_of(what);
    return SVGA_OK;
}
#endif

inline Mask to_mask(const svga_window_mask &m)
{
    return {m.causal, m.window, m.sinks, m.block};
}

inline WindowShape to_shape(const svga_window_problem *p)
{
    return {p->batch,  p->q_heads,  p->kv_heads,      p->q_heads / p->kv_heads,
            p->q_tokens, p->k_tokens, to_mask(p->mask), p->q_lens,
            p->k_lens, p->status};
}

}  // namespace svga
