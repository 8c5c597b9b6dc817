// decode.cu -- attention of one new token per sequence over a paged key-value cache.
//
//   o = sum_j exp(x_j - m) v_j / sum_j exp(x_j - m),  x_j = scale q . k_j, over the kept keys.
//
// Bound by HBM: every kept key and value row is read once, 4 d bytes a key and key head (by groups
// above 16 query heads once for every 16 of them).
//   * The query heads that share a key head are the 16 rows of one mma.sync tile (padded;
//     a group above 16 takes several tiles), so a key row is read once for 16 of them and
//     the FP32 pipe does not limit shared heads.  tcgen05 has nothing to add here: its
//     smallest tile has 64 query rows and the operand bytes, not the products, set the time.
//   * A cluster of CTAs splits the keys of one (sequence, key head): CTA r takes the r-th
//     run of 64-key chunks of the mask's chunk list (sinks, then window; chunks in between
//     are never read).  The CTAs join over distributed shared memory, so the call is one
//     launch with no workspace, and two calls can never share scratch.
//   * Warp 4 looks up pages and streams K and V with TMA through kStages stages of 64 keys: a
//     copy each of K and V per box of 16, 32 or 64 rows, as many as lie whole in a page, with
//     all their columns (64 at a time, 128-byte swizzle).  What it does per chunk bounds a CTA
//     alone: eight times 2 KB a tensor with a page look-up each chunk took 1.34 us, one copy
//     a tensor and look-ups a batch ahead 0.82 us (39 GB/s of K and V a CTA).
//   * Warps 0-3 take 16 keys of a chunk each, with a softmax state of their own: no warp waits
//     for another before the end.  Q sits in shared memory, read again for every chunk, to
//     leave registers.
//   * 96 KB of stages a CTA, two CTAs an SM.  One CTA an SM with eight warps and six stages
//     streams 59 GB/s, but what 160 or 256 CTAs gain by it they lose in their second round
//     (34 against 23 us, 80 against 70 us); chunks of 32 keys change nothing.
// Measured: 8 sequences of 16,384 to 32,768 keys, 32 heads on 4, 385 MB: 70 us, 5.5 TB/s (84 %
// of the measured copy); 16 sequences, 10 heads, 1,040 keys kept of up to 8,191, 85 MB: 23.5 us
// (160 CTAs, one a pair of sequence and head; its 17 or 18 chunks, one after the other, take 14.5
// us at the rate of a CTA alone).
// The running maximum moves only when a tile raises it (a warp vote), so O is rarely rescaled.
// P is rounded to the cache's type for its product with V (operands of one type; half a step
// relative, the weight of one rounding of O).  In fp16 it is held times 2^15 of the running
// maximum, the most its largest value allows: of smaller ones none is off by more than 2^-40 of
// the row's largest, so that a long tail of keys does not vanish (2^24 keys: 2^-16 of O).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "stream.h"
#include "svga_device.cuh"

namespace svga {
namespace {

constexpr int kWarps = 4;                     // consumer warps, 16 keys of a chunk each
constexpr int kThreads = 32 * (kWarps + 1);   // + the producer
constexpr int kChunk = 16 * kWarps;           // keys per stage
constexpr int kRows = 16;                     // query rows of a tile
constexpr int kStages = 3;
constexpr float kLog2e = 1.4426950408889634f;

struct DecodeParams {
    const char *q;
    char *o;
    float *lse;
    long long q_sb, q_sh, o_sb, o_sh;
    int hq, hk, group, tiles;  // tiles of 16 query heads per key head
    int pages, page_size, max_pages;
    int box;  // rows of a TMA box: 16, 32 or 64, whole inside a page
    const int32_t *page_table, *lens;
    Mask mask;
    float scale_log2;
    int32_t *status;
};

template <int D>
struct DecodeSmem {
    static constexpr int kTile = kChunk * D * 2;        // K or V of a chunk
    static constexpr int kStage = 2 * kTile;
    static constexpr int kData = kStages * kStage;
    static constexpr int kQ = kRows * D * 2;
    // the warps' partial results and the CTA's
    static constexpr int kJoin = (kWarps + 1) * kRows * (D + 2) * 4;
    static_assert(kJoin <= kData, "the join reuses the stages");
    static constexpr int kAlloc = kData + kQ + 256 + 1024;
};

struct DecodeBars {
    uint64_t full[kStages], empty[kStages];
    uint32_t boxes[kStages];  // which of the stage's boxes were loaded
    int abort;
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// c += a b for one 16 x 8 x 16 tile
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1)
{
    if constexpr (F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
    return r;
}

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 2) decode_kernel(const __grid_constant__ CUtensorMap tmK,
                                                          const __grid_constant__ CUtensorMap tmV,
                                                          const DecodeParams p)
{
    using S = DecodeSmem<D>;
    constexpr float kBelow = F16 ? 15.f : 0.f;  // log2: the reference lies below the maximum
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~uintptr_t(1023));
    const uint32_t sQ = smem_u32(smem + S::kData);
    DecodeBars *bar = reinterpret_cast<DecodeBars *>(smem + S::kData + S::kQ);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank(), ranks = (int)cluster_size();
    const int kvh = blockIdx.y / p.tiles, tile = blockIdx.y - kvh * p.tiles, b = blockIdx.z;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&bar->full[s]), 1);
            mbar_init(smem_u32(&bar->empty[s]), kWarps);
        }
        bar->abort = 0;
        fence_barrier_init();
    }
    pdl_wait();  // before anything in memory is looked at
    pdl_start();
    // the sequence, its kept keys and this CTA's share of their chunks
    int len = p.lens[b];
    if (len < 0 || len > p.max_pages * p.page_size) {
        if (threadIdx.x == 0 && rank == 0) report(p.status, SVGA_ERR_INVALID_ARG);
        len = 0;
    }
    const MaskRange mr = mask_range(p.mask, len - 1, len);
    const ChunkList cl = chunk_list<kChunk>(p.mask, len - 1, len - 1, len);
    const int skip = max(cl.a, cl.w0);  // first chunk behind the sinks
    const int all = len > 0 ? cl.a + max(cl.w1 - skip, 0) : 0;
    const int e0 = (int)((long long)rank * all / ranks);
    const int e1 = (int)((long long)(rank + 1) * all / ranks);
    auto chunk_of = [&](int e) { return e < cl.a ? e : skip + e - cl.a; };
    auto kept = [&](int j) { return j < mr.hi && (j >= mr.lo || j < mr.sk); };
    // the tile's query rows, 16-byte units permuted within a row so that ldmatrix meets no bank
    // twice; rows past the group are 0
    const int head0 = kvh * p.group + tile * kRows;
    const int rows = min(kRows, p.group - tile * kRows);
    for (int i = threadIdx.x; i < kRows * (D / 8); i += kThreads) {
        const int r = i / (D / 8), u = i - r * (D / 8);
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (r < rows)
            x = reinterpret_cast<const uint4 *>(p.q + 2 * (b * p.q_sb + (head0 + r) * p.q_sh))[u];
        st_shared_v4(sQ + r * (D * 2) + ((u ^ (r & 7)) << 4), x.x, x.y, x.z, x.w);
    }
    __syncthreads();

    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] = 0.f;

    if (warp == kWarps) {
        // ------------------------------------------------------------------ producer
        int issued = 0;
        // A chunk comes in `per` boxes of p.box rows, a copy each of K and V.  One pass of this
        // loop is what bounds a CTA alone, so it does little: the rows of the next 32 / per
        // chunks' boxes are looked up together, one lane a box, a batch ahead of their use.
        const int per = kChunk / p.box, batch = 32 / per, g = lane & (per - 1);
        auto row_at = [&](int e) {  // row of this lane's box in the batch from entry e on
            e += lane / per;
            if (e >= e1) return -1;
            const int j = chunk_of(e) * kChunk + g * p.box, slot = j / p.page_size;
            // any kept key: in [lo, hi), or below the end of the sinks
            if (j >= mr.hi || !(j + p.box > mr.lo || j < mr.sk)) return -1;
            const int page = p.page_table[(long long)b * p.max_pages + slot];
            if (page < 0 || page >= p.pages) {
                report(p.status, SVGA_ERR_INVALID_ARG);
                return -1;
            }
            return (page * p.hk + kvh) * p.page_size + j - slot * p.page_size;
        };
        int rows_now = row_at(e0), rows_next = row_at(e0 + batch);
        const int count = e1 - e0;
        for (int i = 0, s = 0, round = 0, at = 0; i < count; ++i) {
            if (at == batch) {
                at = 0;
                rows_now = rows_next;
                rows_next = row_at(e0 + i + batch);
            }
            const int row = __shfl_sync(0xffffffffu, rows_now, at * per + g);
            ++at;
            bool ok = true;
            if (round > 0)
                ok = mbar_wait(smem_u32(&bar->empty[s]), (round - 1) & 1, &bar->abort);
            if (!__all_sync(0xffffffffu, ok)) break;
            const bool load = lane < per && row >= 0;
            const uint32_t boxes = __ballot_sync(0xffffffffu, load);
            const uint32_t fb = smem_u32(&bar->full[s]);
            if (lane == 0) {
                bar->boxes[s] = boxes;
                mbar_arrive_expect_tx(fb, __popc(boxes) * p.box * D * 2 * 2);
            }
            __syncwarp();
            if (load) {
                const uint32_t dst = smem_u32(smem + s * S::kStage) + g * p.box * (D * 2);
                tma_load_3d(dst, &tmK, fb, 0, row, 0);
                tma_load_3d(dst + S::kTile, &tmV, fb, 0, row, 0);
            }
            issued = i + 1;
            if (++s == kStages) {
                s = 0;
                ++round;
            }
        }
        // every copy lands before the CTA can exit, whoever gave up waiting
        if (lane == 0)
            for (int i = max(0, issued - kStages); i < issued; ++i)
                mbar_wait_bounded(smem_u32(&bar->full[i % kStages]), (i / kStages) & 1);
    } else {
        // ----------------------------------------------------------------- consumers
        const int c0 = (lane & 3) * 2;
        const int mat = lane >> 3, mrow = lane & 7;
        // A box lies in a tile as its rows' first 64 columns, then their second: this warp's 16
        // rows, and the step from one half of the columns to the other
        const int box_at = warp * 16 / p.box;
        const uint32_t row_at = box_at * p.box * (D * 2) + (warp * 16 - box_at * p.box) * 128;
        const uint32_t half_step = p.box * 128;
        for (int i = 0; i < e1 - e0; ++i) {
            const int s = i % kStages;
            const bool ok = mbar_wait(smem_u32(&bar->full[s]), (i / kStages) & 1, &bar->abort);
            if (!__all_sync(0xffffffffu, ok)) break;
            const int j0 = chunk_of(e0 + i) * kChunk + warp * 16;  // this warp's 16 keys
            if ((bar->boxes[s] >> box_at) & 1u) {
                const uint32_t kb = smem_u32(smem + s * S::kStage) + row_at;
                float sc[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int x = 0; x < 4; ++x) sc[n][x] = 0.f;
                {
                    const int key = (mat >> 1) * 8 + mrow;
                    const uint32_t qrow = (mat & 1) * 8 + mrow;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const int col = kk * 16 + (mat & 1) * 8;
                        uint32_t kf[4], qf[4];
                        ldsm4(sQ + qrow * (D * 2) + (((2 * kk + (mat >> 1)) ^ mrow) << 4), qf);
                        ldsm4(kb + (col >> 6) * half_step + key * 128 +
                                  ((((col & 63) >> 3) ^ mrow) << 4),
                              kf);
                        mma16816<F16>(sc[0], qf, kf[0], kf[1]);
                        mma16816<F16>(sc[1], qf, kf[2], kf[3]);
                    }
                }
                // masked keys: score -inf, and their value rows read as 0 (a probability of 0
                // times an infinity or NaN left there would not be 0)
                const bool whole = (j0 >= mr.lo || j0 + 16 <= mr.sk) && j0 + 16 <= mr.hi;
                uint32_t vm0 = 0xffffffffu, vm1 = 0xffffffffu;
                if (!whole) {
                    vm0 = (kept(j0 + c0) ? 0xffffu : 0u) | (kept(j0 + c0 + 1) ? 0xffff0000u : 0u);
                    vm1 = (kept(j0 + c0 + 8) ? 0xffffu : 0u) |
                          (kept(j0 + c0 + 9) ? 0xffff0000u : 0u);
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint32_t bit = (x & 1) ? 0xffff0000u : 0xffffu;
                        if (!(vm0 & bit)) sc[0][x] = -INFINITY;
                        if (!(vm1 & bit)) sc[1][x] = -INFINITY;
                    }
                }
                uint32_t pa[4];
#pragma unroll
                for (int r = 0; r < 2; ++r) {  // rows r0, r0 + 8
                    float mx = fmaxf(fmaxf(sc[0][2 * r], sc[0][2 * r + 1]),
                                     fmaxf(sc[1][2 * r], sc[1][2 * r + 1]));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * p.scale_log2;
                    if (__any_sync(0xffffffffu, mx > m[r])) {
                        const float mn = fmaxf(m[r], mx);
                        const float f = m[r] == -INFINITY ? 0.f : exp2f(m[r] - mn);
                        m[r] = mn;
                        l[r] *= f;
#pragma unroll
                        for (int n = 0; n < D / 8; ++n) {
                            o[n][2 * r] *= f;
                            o[n][2 * r + 1] *= f;
                        }
                    }
                    const float ref = m[r] == -INFINITY ? 0.f : m[r] - kBelow;
                    float e[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        e[x] = fast_exp2(sc[x >> 1][2 * r + (x & 1)] * p.scale_log2 - ref);
                    l[r] += (e[0] + e[1]) + (e[2] + e[3]);
                    pa[r] = pack_16x2<F16>(e[0], e[1]);
                    pa[2 + r] = pack_16x2<F16>(e[2], e[3]);
                }
                const uint32_t vb = kb + S::kTile;
                const int key = (mat & 1) * 8 + mrow;
#pragma unroll
                for (int n = 0; n < D / 16; ++n) {
                    const int col = n * 16 + (mat >> 1) * 8;
                    uint32_t vf[4];
                    ldsm4_t(vb + (col >> 6) * half_step + key * 128 +
                                ((((col & 63) >> 3) ^ mrow) << 4),
                            vf);
                    mma16816<F16>(o[2 * n], pa, vf[0] & vm0, vf[1] & vm1);
                    mma16816<F16>(o[2 * n + 1], pa, vf[2] & vm0, vf[3] & vm1);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bar->empty[s]));
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {  // the quad's lanes hold parts of one row's sum
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        }
    }

    // ------------------------------------------------------------------------- join
    __syncthreads();  // every copy has landed and been read: the stages are free
    float *part = reinterpret_cast<float *>(smem);  // [warp][row][D]
    float *ml = part + kWarps * kRows * D;          // [warp][row] (m, l)
    if (warp < kWarps) {
        const int r0 = lane >> 2, c0 = (lane & 3) * 2;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = r0 + 8 * r;
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
                *reinterpret_cast<float2 *>(part + (warp * kRows + row) * D + n * 8 + c0) =
                    make_float2(o[n][2 * r], o[n][2 * r + 1]);
            if ((lane & 3) == 0)
                *reinterpret_cast<float2 *>(ml + 2 * (warp * kRows + row)) =
                    make_float2(m[r] - kBelow, l[r]);  // (sums are relative to the reference)
        }
    }
    __syncthreads();
    // First the warps of this CTA, into comb / cml, in warp order.
    float *comb = ml + 2 * kWarps * kRows;  // [row][D]
    float *cml = comb + kRows * D;          // [row] (m, l)
    for (int i = threadIdx.x; i < rows * (D / 2); i += kThreads) {
        const int row = i / (D / 2), c = 2 * (i - row * (D / 2));
        float2 s[kWarps];
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            s[w] = *reinterpret_cast<const float2 *>(ml + 2 * (w * kRows + row));
            mx = fmaxf(mx, s[w].x);
        }
        const float ref = mx == -INFINITY ? 0.f : mx;
        float sum = 0.f;
        float2 x = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float wgt = exp2f(s[w].x - ref);
            const float2 y = *reinterpret_cast<const float2 *>(part + (w * kRows + row) * D + c);
            sum += wgt * s[w].y;
            x.x += wgt * y.x;
            x.y += wgt * y.y;
        }
        *reinterpret_cast<float2 *>(comb + row * D + c) = x;
        if (c == 0) *reinterpret_cast<float2 *>(cml + 2 * row) = make_float2(mx, sum);
    }
    if (ranks > 1)
        cluster_sync_all();
    else
        __syncthreads();
    // Then the CTAs of the cluster, each joining its share of the values, in rank order.
    const bool failed = bar->abort != 0;
    for (int i = rank * kThreads + threadIdx.x; i < rows * (D / 2); i += ranks * kThreads) {
        const int row = i / (D / 2), c = 2 * (i - row * (D / 2));
        float mx = -INFINITY;
#pragma unroll 4
        for (int k = 0; k < ranks; ++k)
            mx = fmaxf(mx, *reinterpret_cast<const float *>(
                               __cluster_map_shared_rank(cml + 2 * row, k)));
        const float ref = mx == -INFINITY ? 0.f : mx;
        float sum = 0.f;
        float2 x = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int k = 0; k < ranks; ++k) {
            const float2 s =
                *reinterpret_cast<const float2 *>(__cluster_map_shared_rank(cml + 2 * row, k));
            const float2 y = *reinterpret_cast<const float2 *>(
                __cluster_map_shared_rank(comb + row * D + c, k));
            const float wgt = exp2f(s.x - ref);
            sum += wgt * s.y;
            x.x += wgt * y.x;
            x.y += wgt * y.y;
        }
        if (failed) continue;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        *reinterpret_cast<uint32_t *>(p.o + 2 * (b * p.o_sb + (head0 + row) * p.o_sh + c)) =
            pack_16x2<F16>(x.x * inv, x.y * inv);
        if (c == 0 && p.lse)
            p.lse[(long long)b * p.hq + head0 + row] =
                sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
    }
    if (ranks > 1) cluster_sync_all();  // no CTA leaves while another reads its shared memory
    if (threadIdx.x == 0 && failed) report(p.status, SVGA_ERR_TIMEOUT);
}

template <int D, bool F16>
svga_status launch(const svga_paged_cache *c, const DecodeParams &p, int ranks, cudaStream_t st)
{
    using S = DecodeSmem<D>;
    auto kfn = decode_kernel<D, F16>;
    alignas(64) CUtensorMap tk, tv;
    const long long rows = std::max(1ll, (long long)c->pages * c->kv_heads * c->page_size);
    // with no pages nothing is loaded; the maps then only have to be valid
    const void *kb = c->pages > 0 ? c->k_pages : p.q, *vb = c->pages > 0 ? c->v_pages : p.q;
    if (!make_rows_map(&tk, kb, rows, D, c->dtype, p.box) ||
        !make_rows_map(&tv, vb, rows, D, c->dtype, p.box)) {
        set_error("cuTensorMapEncodeTiled failed (driver entry point or arguments)");
        return SVGA_ERR_CUDA;
    }
    if (cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kAlloc) !=
            cudaSuccess ||
        cudaFuncSetAttribute(kfn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
            cudaSuccess) {
        set_error("cudaFuncSetAttribute failed: %s", cudaGetErrorString(cudaGetLastError()));
        return SVGA_ERR_CUDA;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ranks, c->kv_heads * p.tiles, c->batch);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::kAlloc;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ranks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kfn, tk, tv, p);
    if (e != cudaSuccess) {
        cudaGetLastError();
        set_error("decode launch failed: %s", cudaGetErrorString(e));
        return SVGA_ERR_CUDA;
    }
    return SVGA_OK;
}

// CTAs per (sequence, key head): doubled while the launch still fits the GPU's two slots an SM
// and every CTA keeps at least 128 keys of the longest sequence the page table could hold.  From
// 149 pairs of sequence and head on that is one each, whatever the lengths: a sequence much longer
// than the others is then one CTA's alone.
int choose_ranks(const svga_paged_cache *c, const Mask &m, int tiles)
{
    const int cap = c->max_pages * c->page_size;
    const ChunkList cl = chunk_list<kChunk>(m, cap - 1, cap - 1, cap);
    const int chunks = cap > 0 ? cl.a + std::max(cl.w1 - std::max(cl.a, cl.w0), 0) : 1;
    const long long clusters = (long long)c->batch * c->kv_heads * tiles;
    int ranks = 1;
    while (ranks < 16 && clusters * ranks * 2 <= 2 * 148 && chunks * kChunk >= 256 * ranks) ranks *= 2;
    return ranks;
}

}  // namespace

svga_status launch_decode(const svga_view &q, const svga_view &o, float *lse, int q_heads,
                          const svga_paged_cache *c, const svga_window_mask *mask, float scale,
                          void *stream)
{
    DecodeParams p{};
    p.q = static_cast<const char *>(q.data);
    p.o = static_cast<char *>(o.data);
    p.lse = lse;
    p.q_sb = q.stride_batch;
    p.q_sh = q.stride_head;
    p.o_sb = o.stride_batch;
    p.o_sh = o.stride_head;
    p.hq = q_heads;
    p.hk = c->kv_heads;
    p.group = q_heads / c->kv_heads;
    p.tiles = (p.group + kRows - 1) / kRows;
    p.pages = c->pages;
    p.page_size = c->page_size;
    p.max_pages = c->max_pages;
    p.box = 16;
    while (p.box < kChunk && c->page_size % (2 * p.box) == 0) p.box *= 2;
    p.page_table = c->page_table;
    p.lens = c->lens;
    p.mask = to_mask(*mask);
    p.scale_log2 = scale * kLog2e;
    p.status = c->status;
    const int ranks = choose_ranks(c, p.mask, p.tiles);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (c->head_dim == 128)
        return c->dtype == SVGA_F16 ? launch<128, true>(c, p, ranks, st)
                                    : launch<128, false>(c, p, ranks, st);
    return c->dtype == SVGA_F16 ? launch<64, true>(c, p, ranks, st)
                                : launch<64, false>(c, p, ranks, st);
}

}  // namespace svga
