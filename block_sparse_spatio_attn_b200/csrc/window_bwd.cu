// window_bwd.cu -- attention under a causal window with sinks, backward (sm_100a).
//
// With P = exp(scale Q K^T - lse) on the kept pairs and D = rowsum(dO o O):
//   dV = P^T dO,   dS = P o (dO V^T - D),   dQ = scale dS K,   dK = scale dS^T Q.
//
// Three launches, each begun while the one before it ends (programmatic dependent launch): the
// rows, one of dkdv's and dq's CTAs together, and a join where some of dkdv's items were split.
//   rows    D and lse of every query row in the exp2 domain, negated, 1 KB per 128 rows (fp16:
//           and the norms of dO and V);
//   dkdv    one CTA per 128 keys of a key head; walks the query blocks that keep any of
//           them, over all query heads of the group, with dK and dV in TMEM throughout, so
//           shared heads are summed without atomics and the order is fixed.  Sinks, which
//           every later query keeps, and launches of few key blocks are split over CTAs
//           that leave fp32 sums in the workspace, added in order by a join kernel;
//   dq      one CTA per 128 queries; walks their key chunks with dQ in TMEM.
// S and dO V^T are computed in both: 7 products instead of the 5 a single pass needs.  The
// single pass would add each dQ tile into memory from every CTA: 64 KB of fp32 atomics a
// tile pair, more than L2 takes at this rate, in an order that changes the bits.
//
// dkdv works on transposed tiles, S^T = K Q^T and dP^T = V dO^T (TMEM lane = key), so that P^T
// and dS^T are in place as the A operands of dV += P^T dO and dK += dS^T Q: nothing is
// transposed through shared memory.  TMEM: S^T | dP^T | dV | dK, 128 columns each; P^T and
// dS^T are written over the first half of what each softmax group read of S^T and dP^T.
//
// Warps 4-7 (group A) hold a lane's columns 0-63, warps 8-11 (B) columns 64-127, P staying in
// registers in fp32 between the two steps of a tile.
//
// P and dS are rounded to the tensors' type for their products (operands of one type): half a step
// relative.  fp16 has few exponents: dS is about |dO| |V| over the number of keys, which falls
// below its smallest step (2^-24) for small output gradients, and passes its largest value
// (65504) for large ones; and P is small where there are many keys.  So in fp16 both are held
// times powers of two that the sums are divided by at the end:
//   * P <= 1 times 2^14, by an addition to the exponent;
//   * |dS_ij| = P_ij |dO_i V_j - D_i| <= |dO_i| max_j |V_j| + |D_i|, a bound that is brought to
//     2^13 .. 2^14: in dq a query's own, in dkdv one for all the queries that a CTA visits.  The rows
//     kernel finds the norms (of V too), which every CTA takes the largest of before its loop.
// What falls below the normal range then is 2^-28 of the bound.  Rows that are not finite are left
// out of the norms, so that they do not reach other tiles than those that visit them.
//
// What bounds them.  A product of 128 x 128 tiles with both operands in shared memory reads
// 128 bytes a cycle there, all it has, so that barrier operations and loads of the other
// threads take some 200 cycles beside it; an issuing thread that waits before every product
// leaves the tensor pipe idle between them (one issuer: 2,870 cycles a step of dq, 967 of
// them in waits).  So
//   * two threads issue in dkdv (dV and S^T; dK and dP^T) and three in dq (S; dQ; dP), each the
//     products of its own accumulators and tiles, and each waits for its loads before it waits
//     for the softmax threads;
//   * dkdv: a step's S^T cannot be computed before the last P^T is used up, and no TMEM is
//     left for a second tile.  The groups are therefore two chains of their own (barriers, an
//     S^T product of 64 columns each, dV and dK products of 64 terms each): while one waits,
//     the other has the exponential unit and the tensor pipe.  dP^T, which the groups need later,
//     is one product of 128 columns: two of 64 take half as long again (2,048 causal tokens of
//     4 heads: 32.2 us against 33.2; S^T in one as well: 36);
//   * dq gives dS columns of its own (S | dP | dQ | dS | Q, the last two
//     64 columns of packed pairs each): S and dP are computed again as soon as they were
//     read, so the softmax threads wait for no product (with dS over dP the chain dS -> dQ ->
//     dP -> dS alone took 2,440 cycles a step).  Q as an operand in TMEM spares a quarter of
//     the shared memory's reads;
//   * shared memory holds, beside the resident tiles, three stages of the operand that is
//     needed longest (dkdv: Q, dq: K) and two of the other.
// Measured: 12,480 tokens, 4 heads of 128, frames of 960, window 2 and a sink frame: 295 us, 735
// TFLOP/s of the five products of kept pairs (in a loop; one launch alone 265); 75,600 tokens, 10
// heads, frames of 3,600, window 3 and a sink frame: 19.0 ms, 832 TFLOP/s; 2 x 2,001 tokens, 8 heads
// on 2, window of 512, fp16: 50 us (47.5 without the norms and powers of two).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "stream.h"
#include "svga_device.cuh"
#include "tile_out.cuh"

namespace svga {
namespace {

constexpr int kThreads = 384;
constexpr int kT = 128;  // rows and keys of a tile
constexpr int kSms = 148;
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kNegInfBits = 0xff800000u;
constexpr int kRegsLaunch = 168, kRegsLow = 96, kRegsHigh = 200;
static_assert(128 * kRegsLow + 256 * kRegsHigh <= kThreads * kRegsLaunch, "register split");

struct BwdParams {
    WindowShape s;
    View d_o, o, v, dq, dk, dv;
    const float *lse;
    float *stats;  // [batch * hq][query block][kStatRows][128]: -lse log2(e), -D and |dO|
    // fp16: the largest |dO| and |D| of parts of the query blocks, |V| of the key blocks
    float2 *most_q;  // [batch * hq][query block][kParts]
    float *most_v;   // [batch * hk][key block][kParts]
    float scale, scale_log2;
    int n_qblk, n_kblk;
    int n_dkdv;    // CTAs of dkdv
    Split split;   // over dkdv's items, key blocks ascending
    // the split's parts, (sequence, key head) and (sequence, query head) pairs, heads, the group
    FastDiv by_k1, by_k2, by_bk, by_hk, by_bq, by_hq, by_group;
    float *parts;  // [slot][dV, dK][128][d]
    int q_mb, q_mh, o_mb, o_mh, k_mb, k_mh, v_mb, v_mh;  // coordinate multipliers (o: dO)
};

template <int D>
struct Cfg {
    static constexpr int kTile = kT * D * 2;   // a 128-row tile of Q, K, V or dO
    static constexpr int kChunk = kT * 128;    // 64 columns of it
    static constexpr int kStats = 2 * kT * 4;  // a query block's statistics for dkdv
    static constexpr int kParts = kT * (D / 8) / 256;  // CTAs of the rows kernel to a block
    // dkdv: K, V, three stages of Q, two of dO with the block's statistics
    static constexpr int kQStages = 3, kOStages = 2;
    static constexpr int kKvData = (2 + kQStages + kOStages) * kTile + kOStages * kStats;
    // dq: Q (on its way to TMEM), dO, three stages of K, two of V
    static constexpr int kKStages = 3, kVStages = 2;
    static constexpr int kDqData = (2 + kKStages + kVStages) * kTile;
    static constexpr int kBars = 512;
    // one CTA per SM (each takes the whole TMEM): never less than half the shared memory.
    // No room is left to align the base by hand: the kernels check it.
    static constexpr int alloc(int data)
    {
        return data + kBars < 120 * 1024 ? 120 * 1024 : data + kBars;
    }
    static constexpr int kKvAlloc = alloc(kKvData), kDqAlloc = alloc(kDqData);
    static_assert(kKvAlloc <= 227 * 1024 && kDqAlloc <= 227 * 1024, "shared memory budget");
};

// fp16 holds P times 2^kPBits and dS times the power of two that brings its bound below 2^14.
constexpr int kPBits = 14;
template <bool F16>
constexpr int kStatRows = F16 ? 3 : 2;

// k with bound * 2^k in [2^13, 2^14) (a bound of 0, whose dS are 0, takes any)
__device__ __forceinline__ int bits_to_2_14(float bound)
{
    const int e = (__float_as_int(bound) >> 23) - 127;  // 2^e <= bound < 2^(e + 1)
    return min(max(13 - e, -64), 64);                   // (finite ones lie in -27 .. 61)
}

__device__ __forceinline__ float pow2(int k) { return __int_as_float((k + 127) << 23); }

__device__ __forceinline__ float warp_max(float x)
{
#pragma unroll
    for (int k = 16; k > 0; k /= 2) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, k));
    return x;
}

__device__ __forceinline__ int clamped_len(const int32_t *lens, int b, int most)
{
    return lens ? min(max(lens[b], 0), most) : most;
}

__device__ __forceinline__ uint32_t bits_below(int n)
{
    return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u);
}

template <bool F16>
__device__ __forceinline__ float2 unpack_16x2(uint32_t x)
{
    if constexpr (F16) {
        const __half2 h = *reinterpret_cast<const __half2 *>(&x);
        return __half22float2(h);
    } else {
        return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
    }
}

// 64 columns of a TMEM tile into registers
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&r)[64])
{
    tmem_ld32(taddr, *reinterpret_cast<uint32_t(*)[32]>(&r[0]));
    tmem_ld32(taddr + 32, *reinterpret_cast<uint32_t(*)[32]>(&r[32]));
}

// ----------------------------------------------------------------------------- rows
// D / 8 threads a row, kParts CTAs a block of 128.  Bound by HBM: dO and O are read once (fp16: and
// V, whose CTAs come last).  Rows past the sequence's end get -inf and 0: their P and dS are 0.
template <int D, bool F16>
__global__ void __launch_bounds__(256) bwd_rows_kernel(const BwdParams p)
{
    pdl_wait();
    pdl_start();
    constexpr int kPer = D / 8, kParts = Cfg<D>::kParts;
    const int q_ctas = p.s.batch * p.s.hq * p.n_qblk * kParts;
    const bool values = F16 && (int)blockIdx.x >= q_ctas;
    const int cta = blockIdx.x - (values ? q_ctas : 0), n_blk = values ? p.n_kblk : p.n_qblk;
    const int heads = values ? p.s.hk : p.s.hq;
    const long long row = (cta * 256ll + threadIdx.x) / kPer, bh = row / (n_blk * kT);
    const int b = (int)(bh / heads), h = (int)(bh - (long long)b * heads);
    const int t = (int)(row - bh * n_blk * kT), c = 8 * (int)(threadIdx.x % kPer);
    const bool there = t < (values ? clamped_len(p.s.k_lens, b, p.s.tk)
                                   : clamped_len(p.s.q_lens, b, p.s.tq));
    float sum = 0.f, square = 0.f;
    if (there) {
        const View &xv = values ? p.v : p.d_o;
        const uint4 x = *reinterpret_cast<const uint4 *>(
            xv.p + 2 * (b * xv.sb + h * xv.sh + t * xv.st + c));
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
        if (!values) {
            const uint4 y = *reinterpret_cast<const uint4 *>(
                p.o.p + 2 * (b * p.o.sb + h * p.o.sh + t * p.o.st + c));
            const uint32_t ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 u = unpack_16x2<F16>(xs[k]), v = unpack_16x2<F16>(ys[k]);
                sum += u.x * v.x + u.y * v.y;
            }
        }
        if constexpr (F16) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 u = unpack_16x2<F16>(xs[k]);
                square += u.x * u.x + u.y * u.y;
            }
        }
    }
#pragma unroll
    for (int k = kPer / 2; k > 0; k /= 2) {
        sum += __shfl_xor_sync(0xffffffffu, sum, k);
        if constexpr (F16) square += __shfl_xor_sync(0xffffffffu, square, k);
    }
    const float norm = sqrtf(square);
    if (c == 0 && !values) {
        const float lse = there ? p.lse[bh * p.s.tq + t] : -INFINITY;
        float *out =
            p.stats + (bh * p.n_qblk + t / kT) * kStatRows<F16> * kT + t % kT;
        // (an empty row keeps nothing)
        out[0] = lse == -INFINITY ? -INFINITY : -lse * kLog2e + (F16 ? (float)kPBits : 0.f);
        out[kT] = -sum;
        if constexpr (F16) out[2 * kT] = norm;
    }
    if constexpr (F16) {  // the CTA's largest norms
        __shared__ float2 most[8];
        const bool finite = norm < INFINITY && fabsf(sum) < INFINITY;
        const float2 m = {warp_max(finite ? norm : 0.f), warp_max(finite ? fabsf(sum) : 0.f)};
        if (threadIdx.x % 32 == 0) most[threadIdx.x / 32] = m;
        __syncthreads();
        if (threadIdx.x == 0) {
            float2 x = most[0];
            for (int w = 1; w < 8; ++w) x = {fmaxf(x.x, most[w].x), fmaxf(x.y, most[w].y)};
            if (values)
                p.most_v[cta] = x.x;
            else
                p.most_q[cta] = x;
        }
    }
}

// Rows [first, 128) of a swizzled 128-row tile read as 0 (whole rows: the swizzle permutes
// inside a row's 128 bytes).
template <int D>
__device__ __forceinline__ void zero_rows(uint32_t tile, int first, int lane)
{
    for (int u = first * 8 + lane; u < kT * 8; u += 32)
        for (int c = 0; c < D / 64; ++c)
            st_shared_v4(tile + c * Cfg<D>::kChunk + u * 16, 0u, 0u, 0u, 0u);
}

// Columns 64 g .. 64 g + 63 of a 128 x 128 product over D terms, both operands in shared
// memory: b's rows 64 g and up.
template <int D>
__device__ __forceinline__ void product_ss(uint32_t d, uint64_t a, uint64_t b, int g, uint32_t id)
{
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t at = ((kk >> 2) * Cfg<D>::kChunk + (kk & 3) * 32) >> 4;
        mma_ss(d + 64 * g, a + at, b + at + g * (64 * 128 >> 4), id, kk > 0 ? 1u : 0u);
    }
}

// A 128 x D product over terms 64 g .. 64 g + 63: a holds them as packed 16-bit pairs in
// columns 64 g .. 64 g + 31, b's rows are the terms.
__device__ __forceinline__ void product_ts(uint32_t d, uint32_t a, uint64_t b, int g, uint32_t id,
                                           bool accumulate)
{
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
        mma_ts(d, a + 64 * g + 8 * kk, b + (uint32_t)((4 * g + kk) * (2048 >> 4)), id,
               (accumulate || kk > 0) ? 1u : 0u);
}

// A 128 x 128 product over D terms, both operands in shared memory.
template <int D>
__device__ __forceinline__ void product_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id)
{
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t at = ((kk >> 2) * Cfg<D>::kChunk + (kk & 3) * 32) >> 4;
        mma_ss(d, a + at, b + at, id, kk > 0 ? 1u : 0u);
    }
}

// A 128 x D product over 128 terms: a holds them as packed pairs in 64 columns.
__device__ __forceinline__ void product_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id,
                                           bool accumulate)
{
#pragma unroll
    for (int kk = 0; kk < kT / 16; ++kk)
        mma_ts(d, a + 8 * kk, b + (uint32_t)(kk * (2048 >> 4)), id,
               (accumulate || kk > 0) ? 1u : 0u);
}

// A 128 x 128 product over D terms, a in TMEM as packed pairs, b's rows (K-major) the columns.
template <int D>
__device__ __forceinline__ void product_tk(uint32_t d, uint32_t a, uint64_t b, uint32_t id)
{
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
        mma_ts(d, a + 8 * kk, b + (uint32_t)(((kk >> 2) * Cfg<D>::kChunk + (kk & 3) * 32) >> 4), id,
               kk > 0 ? 1u : 0u);
}

// The base of the dynamic shared memory, on the 1024-byte boundary the swizzle needs.  The
// runtime places it there; should it ever not, the kernel reports instead of computing.
__device__ __forceinline__ bool smem_misplaced(const void *base, int32_t *status)
{
    if ((smem_u32(base) & 1023u) == 0) return false;
    pdl_wait();  // before anything in memory is touched
    if (threadIdx.x == 0) report(status, SVGA_ERR_ALIGNMENT);
    return true;
}

// ----------------------------------------------------------------------------- dkdv
// One CTA's work, worked out by warp 0, its lanes together, for all.
struct KvItem {
    int b, hk, nq, nk, off;
    int k0, k1;                // keys
    int qb0, n_blk;            // query blocks that keep any of them
    int all_first, all_end;    // the queries that keep all of them
    int steps, g0, blk0;       // this CTA's part of the group's blocks: how many, the first
    int ragged;                // block whose last rows lie past the sequence's end but inside
                               // the tensor, or -1
    int ksplit;
    long long slot;
};

__device__ __forceinline__ bool make_item(const BwdParams &p, int block, KvItem &it)
{
    int item, part;
    p.split.of_block(block, p.by_k1, p.by_k2, item, part);
    it.ksplit = p.split.k(item);
    it.slot = it.ksplit > 1 ? p.split.slot(item, part) : 0;
    const int bh = p.s.batch * p.s.hk;
    const int kblk = p.by_bk.of(item), r = item - kblk * bh;
    it.b = p.by_hk.of(r);
    it.hk = r - it.b * p.s.hk;
    it.nq = clamped_len(p.s.q_lens, it.b, p.s.tq);
    it.nk = clamped_len(p.s.k_lens, it.b, p.s.tk);
    const int nq = it.nq, off = it.off = it.nk - nq;
    const int k0 = it.k0 = kblk * kT, k1 = it.k1 = min(k0 + kT, it.nk);
    if (k0 >= it.nk) return false;
    int first, end;  // of three keys, a lane each
    mask_rows(p.s.mask, block_key(p.s.mask, k0, k1, threadIdx.x & 3), nq, off, first, end);
    const int first0 = __shfl_sync(0xffffffffu, first, 0), end0 = __shfl_sync(0xffffffffu, end, 0);
    const int first1 = __shfl_sync(0xffffffffu, first, 1), end1 = __shfl_sync(0xffffffffu, end, 1);
    const int end2 = __shfl_sync(0xffffffffu, end, 2);
    const BlockRows rows = block_rows(p.s.mask, k1, nq, first0, end0, first1, end1, end2);
    it.all_first = rows.all_first;
    it.all_end = rows.all_end;
    first = rows.first;
    end = rows.end;
    it.qb0 = first / kT;
    it.n_blk = end > first ? (end + kT - 1) / kT - it.qb0 : 0;
    const long long all = (long long)it.n_blk * p.s.group;
    int first_step = 0;
    it.steps = (int)all;
    it.g0 = 0;
    if (it.ksplit > 1) {
        first_step = (int)(part * all / it.ksplit);
        it.steps = (int)((part + 1) * all / it.ksplit) - first_step;
        it.g0 = it.n_blk > 0 ? first_step / it.n_blk : 0;
    }
    it.blk0 = first_step - it.g0 * it.n_blk;
    it.ragged =
        (p.s.q_lens && nq < p.s.tq && nq % kT && nq / kT == it.qb0 + it.n_blk - 1) ? it.n_blk - 1
                                                                                    : -1;
    return true;
}

struct KvBars {
    uint64_t kv_full;
    uint64_t q_full[3], q_empty[3];      // stages of Q
    uint64_t o_full[2], o_empty[2];      // stages of dO
    uint64_t st_full[2], st_empty[2];    // of the statistics (needed longer than dO)
    uint64_t s_full[2], dp_full;         // [group]: its columns of S^T are in TMEM; dP^T is
    uint64_t p_ready[2], ds_ready[2];    // [group]: its P^T / dS^T is (4 warps)
    uint64_t acc_done;                   // every product is done (both issuers)
    uint64_t drain[2];
    uint64_t zero_req[2], zero_done[2];  // Q, dO
    uint32_t tmem_base;
    int abort, some;
    KvItem item;
};
static_assert(sizeof(KvBars) <= 512, "barrier space");

template <int D, bool F16>
__device__ __forceinline__ void dkdv_cta(const CUtensorMap &tmQ, const CUtensorMap &tmO,
                                         const CUtensorMap &tmK, const CUtensorMap &tmV,
                                         const BwdParams &p, uint8_t *smem, int block)
{
    using C = Cfg<D>;
    constexpr uint32_t kS = 0, kDP = 128, kDV = 256, kDK = 384;
    uint8_t *sK = smem, *sV = smem + C::kTile;
    uint8_t *sQ = smem + 2 * C::kTile;              // [stage]
    uint8_t *sO = sQ + C::kQStages * C::kTile;      // [stage]
    uint8_t *sStats = sO + C::kOStages * C::kTile;  // [stage]
    KvBars *bar = reinterpret_cast<KvBars *>(smem + C::kKvData);
    volatile int *abort_flag = &bar->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmO);
        mbar_init(smem_u32(&bar->kv_full), 1);
        for (int i = 0; i < C::kQStages; ++i) {
            mbar_init(smem_u32(&bar->q_full[i]), 1);
            mbar_init(smem_u32(&bar->q_empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&bar->o_full[i]), 1);
            mbar_init(smem_u32(&bar->o_empty[i]), 2);  // dV and dP of the step are done
            mbar_init(smem_u32(&bar->st_full[i]), 1);
            mbar_init(smem_u32(&bar->st_empty[i]), 1);
            mbar_init(smem_u32(&bar->s_full[i]), 1);
            mbar_init(smem_u32(&bar->p_ready[i]), 4);
            mbar_init(smem_u32(&bar->ds_ready[i]), 4);
            mbar_init(smem_u32(&bar->zero_req[i]), 1);
            mbar_init(smem_u32(&bar->zero_done[i]), 1);
            mbar_init(smem_u32(&bar->drain[i]), 1);
        }
        mbar_init(smem_u32(&bar->dp_full), 1);
        mbar_init(smem_u32(&bar->acc_done), 2);
        bar->abort = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&bar->tmem_base), 512);
        tmem_relinquish();
    }
    // Q or dO of step i (query head h, block blk) into its stage
    auto fetch = [&](int i, bool o, int row, int h, int b) {
        const int st = i % (o ? C::kOStages : C::kQStages);
        const uint32_t fb = smem_u32(o ? &bar->o_full[st] : &bar->q_full[st]);
        mbar_arrive_expect_tx(fb, C::kTile);
        tma_load_5d(smem_u32((o ? sO : sQ) + st * C::kTile), o ? &tmO : &tmQ, fb, 0, row, 0,
                    h * (o ? p.o_mh : p.q_mh), b * (o ? p.o_mb : p.q_mb));
    };
    if (warp == 1) pdl_start();  // the next kernel, once this one has its TMEM
    // Before anything in memory is looked at: the lengths, where sequences have their own, then
    // the tensors.  (The rows kernel has waited for all that came before it when this one starts,
    // but only its end, which is waited for here, promises that their writes can be read.)
    if (p.s.q_lens || p.s.k_lens) pdl_wait();
    if (warp == 0) {
        __syncwarp();  // (or the item is worked out for lane 0 and for the others, one after the other)
        KvItem mine;
        const bool some = make_item(p, block, mine);  // false: past the sequence's keys
        pdl_wait();
        if (threadIdx.x == 0) {
            bar->item = mine;
            bar->some = some;
            if (some && mine.steps > 0) {  // on their way before the CTA meets
                const uint32_t kvf = smem_u32(&bar->kv_full);
                mbar_arrive_expect_tx(kvf, 2 * C::kTile);
                tma_load_5d(smem_u32(sK), &tmK, kvf, 0, mine.k0, 0, mine.hk * p.k_mh, mine.b * p.k_mb);
                tma_load_5d(smem_u32(sV), &tmV, kvf, 0, mine.k0, 0, mine.hk * p.v_mh, mine.b * p.v_mb);
                for (int o = 0; o < 2; ++o)
                    fetch(0, o, (mine.qb0 + mine.blk0) * kT, mine.hk * p.s.group + mine.g0, mine.b);
            }
        }
    }
    pdl_wait();  // (every thread: the rows' statistics)
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar->tmem_base;
    if (!bar->some) {
        if (warp == 1) tmem_dealloc(tmem, 512);
        return;
    }
    const KvItem &it = bar->item;
    const int b = it.b, hk = it.hk, nq = it.nq, nk = it.nk, off = it.off, k0 = it.k0;
    const int qb0 = it.qb0, n_blk = it.n_blk, steps = it.steps, ragged = it.ragged;

    if (warp < 4) {
        setmaxnreg_dec<kRegsLow>();
        if (threadIdx.x == 0 && steps > 0) {
            // -------------------------------------------------------- TMA producer
            int q_issued = 0, o_issued = 0, st_issued = 0, g = it.g0, blk = it.blk0;
            for (int i = 0; i < steps; ++i) {
                const int h = hk * p.s.group + g, row = (qb0 + blk) * kT;
                const int qs = i % C::kQStages, os = i % C::kOStages;
                const int qr = i / C::kQStages, orr = i / C::kOStages;
                if (qr > 0 && !mbar_wait(smem_u32(&bar->q_empty[qs]), (qr - 1) & 1, abort_flag))
                    break;
                if (i > 0) fetch(i, false, row, h, b);  // (the first are on their way)
                q_issued = i + 1;
                if (orr > 0 && !mbar_wait(smem_u32(&bar->o_empty[os]), (orr - 1) & 1, abort_flag))
                    break;
                if (i > 0) fetch(i, true, row, h, b);
                o_issued = i + 1;
                if (orr > 0 && !mbar_wait(smem_u32(&bar->st_empty[os]), (orr - 1) & 1, abort_flag))
                    break;
                const uint32_t fb = smem_u32(&bar->st_full[os]);
                mbar_arrive_expect_tx(fb, C::kStats);
                bulk_load(smem_u32(sStats + os * C::kStats),
                          p.stats + (((long long)b * p.s.hq + h) * p.n_qblk + qb0 + blk) *
                                        kStatRows<F16> * kT,
                          C::kStats, fb);
                st_issued = i + 1;
                if (++blk == n_blk) {
                    blk = 0;
                    ++g;
                }
            }
            // every copy lands before the CTA can exit, whichever role aborts
            mbar_wait_bounded(smem_u32(&bar->kv_full), 0);
            for (int i = max(q_issued - C::kQStages, 0); i < q_issued; ++i)
                mbar_wait_bounded(smem_u32(&bar->q_full[i % C::kQStages]), (i / C::kQStages) & 1);
            for (int i = max(o_issued - C::kOStages, 0); i < o_issued; ++i)
                mbar_wait_bounded(smem_u32(&bar->o_full[i % C::kOStages]), (i / C::kOStages) & 1);
            for (int i = max(st_issued - C::kOStages, 0); i < st_issued; ++i)
                mbar_wait_bounded(smem_u32(&bar->st_full[i % C::kOStages]), (i / C::kOStages) & 1);
        } else if ((warp == 1 || warp == 3) && steps > 0 && elect_one()) {
            // --------------------------------------------------------- MMA issuers
            // warp 1: S^T and dV, warp 3: dP^T and dK.  Each accumulator and tile belongs to
            // one of them, so its products stay in order.
            const int role = warp == 3;
            constexpr uint32_t idS = idesc_16_f32(F16, kT, 64, 0, 0);
            constexpr uint32_t idDP = idesc_16_f32(F16, kT, kT, 0, 0);
            constexpr uint32_t idA = idesc_16_f32(F16, kT, D, 0, 1);
            const uint64_t kmaj = smem_desc_sw128(0, 16, 1024);         // rows of terms
            const uint64_t nmaj = smem_desc_sw128(0, C::kChunk, 1024);  // terms down the rows
            const uint32_t aQ = smem_u32(sQ) >> 4, aO = smem_u32(sO) >> 4;
            // the stage of step i has landed (w: 0 Q, 1 dO)
            auto landed = [&](int i, int w) {
                return w ? mbar_wait(smem_u32(&bar->o_full[i % C::kOStages]),
                                     (i / C::kOStages) & 1, abort_flag)
                         : mbar_wait(smem_u32(&bar->q_full[i % C::kQStages]),
                                     (i / C::kQStages) & 1, abort_flag);
            };
            int blk[2] = {it.blk0, it.blk0}, cleaned[2] = {0, 0};  // walks of Q's and dO's steps
            // landed, and its rows past the sequence's end are 0 (asked of warp 2 once, by the
            // issuer whose first product on the stage it is)
            auto take = [&](int i, int w, bool ask) {
                if (!landed(i, w)) return false;
                const bool dirty = blk[w] == ragged;
                if (++blk[w] == n_blk) blk[w] = 0;
                if (!dirty) return true;
                if (ask) mbar_arrive(smem_u32(&bar->zero_req[w]));
                return mbar_wait(smem_u32(&bar->zero_done[w]), cleaned[w]++ & 1, abort_flag);
            };
            auto q_at = [&](int i) { return aQ + (i % C::kQStages) * (C::kTile >> 4); };
            auto o_at = [&](int i) { return aO + (i % C::kOStages) * (C::kTile >> 4); };
            bool ok = mbar_wait(smem_u32(&bar->kv_full), 0, abort_flag) && take(0, role, true);
            if (role == 0) {
                const uint64_t a = kmaj + (smem_u32(sK) >> 4);
                auto issue = [&](int i, int g) {
                    product_ss<D>(tmem + kS, a, kmaj + q_at(i), g, idS);
                    mma_commit(smem_u32(&bar->s_full[g]));
                };
                if (ok) {
                    issue(0, 0);
                    issue(0, 1);
                }
                for (int i = 0; ok && i < steps; ++i) {
                    const bool next = i + 1 < steps;
                    ok = take(i, 1, false) && (!next || take(i + 1, 0, true));
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        if (!ok || !(ok = mbar_wait(smem_u32(&bar->p_ready[g]), i & 1, abort_flag)))
                            break;
                        tc_fence_after();
                        product_ts(tmem + kDV, tmem + kS, nmaj + o_at(i), g, idA, i > 0 || g > 0);
                        if (g == 1) mma_commit(smem_u32(&bar->o_empty[i % C::kOStages]));
                        if (next) issue(i + 1, g);
                    }
                }
            } else {
                const uint64_t a = kmaj + (smem_u32(sV) >> 4);
                auto issue = [&](int i) {
                    product_ss<D>(tmem + kDP, a, kmaj + o_at(i), idDP);
                    mma_commit(smem_u32(&bar->dp_full));
                    mma_commit(smem_u32(&bar->o_empty[i % C::kOStages]));
                };
                if (ok) issue(0);
                for (int i = 0; ok && i < steps; ++i) {
                    const bool next = i + 1 < steps;
                    ok = landed(i, 0) && (!next || take(i + 1, 1, true));
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        if (!ok ||
                            !(ok = mbar_wait(smem_u32(&bar->ds_ready[g]), i & 1, abort_flag)))
                            break;
                        tc_fence_after();
                        product_ts(tmem + kDK, tmem + kDP, nmaj + q_at(i), g, idA, i > 0 || g > 0);
                        if (g == 1) {  // the last to use the step's Q; the statistics were read
                            mma_commit(smem_u32(&bar->q_empty[i % C::kQStages]));
                            mma_commit(smem_u32(&bar->st_empty[i % C::kOStages]));
                            if (next) issue(i + 1);
                        }
                    }
                }
            }
            if (ok) {
                mma_commit(smem_u32(&bar->acc_done));
            } else {
                mma_commit(smem_u32(&bar->drain[role]));
                mbar_wait_bounded(smem_u32(&bar->drain[role]), 0);
            }
        } else if (warp == 2 && ragged >= 0) {
            // ------------------------ rows of Q and dO past the sequence's end read as 0
            int time = 0;
            for (int i = ragged - it.blk0 + (ragged < it.blk0 ? n_blk : 0); i < steps;
                 i += n_blk, ++time) {
                bool ok = true;
                for (int w = 0; w < 2 && ok; ++w) {
                    ok = __all_sync(0xffffffffu, mbar_wait_long(smem_u32(&bar->zero_req[w]),
                                                                time & 1, abort_flag));
                    if (!ok) break;
                    zero_rows<D>(smem_u32(w ? sO + (i % C::kOStages) * C::kTile
                                            : sQ + (i % C::kQStages) * C::kTile),
                                 nq % kT, lane);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&bar->zero_done[w]));
                }
                if (!ok) break;
            }
        }
    } else {
        // ------------------------------------------------------ softmax warpgroups
        setmaxnreg_inc<kRegsHigh>();
        const int wg = (warp - 4) >> 2, quad = warp & 3, row = quad * 32 + lane;
        const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
        const uint32_t tS = tmem + lane_base + kS + 64 * wg;
        const uint32_t tDP = tmem + lane_base + kDP + 64 * wg;
        const int key = k0 + row;
        int ra = 0, re = 0;  // the queries that keep this lane's key
        if (key < nk) mask_rows(p.s.mask, key, nq, off, ra, re);
        const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
        bool ok = true;
        const int all_first = it.all_first, all_end = it.all_end;
        int blk = it.blk0;
        int s_bits = 0;  // fp16: dS is held times 2^s_bits
        if constexpr (F16) {
            if (steps > 0) {
                float most_o = 0.f, most_d = 0.f, most_v = 0.f;
                for (int i = lane; i < steps; i += 32) {
                    const int at = it.blk0 + i, g = at / n_blk;
                    const float4 *m = reinterpret_cast<const float4 *>(
                        p.most_q + (((long long)b * p.s.hq + hk * p.s.group + it.g0 + g) * p.n_qblk +
                                    qb0 + at - g * n_blk) *
                                       C::kParts);
#pragma unroll
                    for (int j = 0; j < C::kParts / 2; ++j) {
                        const float4 y = m[j];
                        most_o = fmaxf(most_o, fmaxf(y.x, y.z));
                        most_d = fmaxf(most_d, fmaxf(y.y, y.w));
                    }
                }
                if (lane < C::kParts)
                    most_v = p.most_v[(((long long)b * p.s.hk + hk) * p.n_kblk + k0 / kT) * C::kParts +
                                      lane];
                s_bits = bits_to_2_14(warp_max(most_o) * warp_max(most_v) + warp_max(most_d));
            }
        }
        // dS from P 2^kPBits, and back from either sum
        const float2 to_s = make_float2(pow2(s_bits - kPBits), pow2(s_bits - kPBits));
        const float back = F16 ? pow2(wg ? -s_bits : -kPBits) : 1.f;
        for (int i = 0; i < steps; ++i) {
            const int r0 = (qb0 + blk) * kT;
            if (++blk == n_blk) blk = 0;
            const bool full = r0 >= all_first && min(r0 + kT, nq) <= all_end;
            uint32_t keep[2] = {0u, 0u};
            if (!full) {  // kept columns of this thread's half: [c0, c1)
                const int c0 = ra - r0 - 64 * wg, c1 = re - r0 - 64 * wg;
                keep[0] = bits_below(c1) & ~bits_below(c0);
                keep[1] = bits_below(c1 - 32) & ~bits_below(c0 - 32);
            }
            const float4 *nl = reinterpret_cast<const float4 *>(
                                   sStats + (i % C::kOStages) * C::kStats) +
                               16 * wg;
            uint32_t x[64];
            float pr[64];
            ok = __all_sync(0xffffffffu,
                            mbar_wait(smem_u32(&bar->s_full[wg]), i & 1, abort_flag) &&
                                mbar_wait(smem_u32(&bar->st_full[i % C::kOStages]),
                                          (i / C::kOStages) & 1, abort_flag));
            tc_fence_after();
            if (!ok) break;
            tmem_ld64(tS, x);
            tmem_wait_ld();
            if (!full) {
#pragma unroll
                for (int c = 0; c < 64; ++c)
                    if (!((keep[c >> 5] >> (c & 31)) & 1u)) x[c] = kNegInfBits;
            }
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
                const float4 n = nl[c >> 2];
                const float2 u = ffma2(make_float2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])),
                                       sc2, make_float2(n.x, n.y));
                const float2 v =
                    ffma2(make_float2(__uint_as_float(x[c + 2]), __uint_as_float(x[c + 3])), sc2,
                          make_float2(n.z, n.w));
                pr[c] = fast_exp2(u.x);
                pr[c + 1] = fast_exp2(u.y);
                pr[c + 2] = fast_exp2(v.x);
                pr[c + 3] = fast_exp2(v.y);
            }
            {
                uint32_t pk[32];
#pragma unroll
                for (int c = 0; c < 32; ++c) pk[c] = pack_16x2<F16>(pr[2 * c], pr[2 * c + 1]);
                tmem_st32(tS, pk);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bar->p_ready[wg]));

            ok = __all_sync(0xffffffffu,
                            mbar_wait(smem_u32(&bar->dp_full), i & 1, abort_flag));
            tc_fence_after();
            if (!ok) break;
            tmem_ld64(tDP, x);
            tmem_wait_ld();
            {
                const float4 *nd = nl + kT / 4;
                uint32_t pk[32];
#pragma unroll
                for (int c = 0; c < 64; c += 4) {
                    const float4 n = nd[c >> 2];
                    float2 u = fadd2(make_float2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])),
                                     make_float2(n.x, n.y));
                    float2 v = fadd2(
                        make_float2(__uint_as_float(x[c + 2]), __uint_as_float(x[c + 3])),
                        make_float2(n.z, n.w));
                    u = ffma2(u, make_float2(pr[c], pr[c + 1]), make_float2(0.f, 0.f));
                    v = ffma2(v, make_float2(pr[c + 2], pr[c + 3]), make_float2(0.f, 0.f));
                    if constexpr (F16) {
                        u = ffma2(u, to_s, make_float2(0.f, 0.f));
                        v = ffma2(v, to_s, make_float2(0.f, 0.f));
                    }
                    pk[c / 2] = pack_16x2<F16>(u.x, u.y);
                    pk[c / 2 + 1] = pack_16x2<F16>(v.x, v.y);
                }
                if (!full) {  // 0 also where a dropped pair's product is not finite
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const uint32_t k2 = keep[c >> 4] >> (2 * (c & 15));
                        pk[c] &= ((k2 & 1u) ? 0xffffu : 0u) | ((k2 & 2u) ? 0xffff0000u : 0u);
                    }
                }
                tmem_st32(tDP, pk);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bar->ds_ready[wg]));
        }
        // ------------------------------- epilogue: group 0 stores dV, group 1 dK
        if (ok && steps > 0) {
            ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar->acc_done), 0, abort_flag));
            tc_fence_after();
        }
        if (ok) {  // through K's and V's tiles, whose products are done
            const uint32_t acc = tmem + lane_base + (wg ? kDK : kDV);
            const uint32_t tile = smem_u32(wg ? sK : sV);
            const int valid = nk - (key - lane);  // of the warp's rows
            if (it.ksplit > 1) {  // (a tile holds half of a row of fp32)
                char *dst = reinterpret_cast<char *>(
                    p.parts + ((it.slot * 2 + wg) * kT + row - lane) * D);
#pragma unroll 1
                for (int j = 0; j < 2; ++j) {
                    put_row_32<D / 2>(acc + j * (D / 2), tile, C::kChunk, row, back, steps > 0);
                    copy_rows_out<D / 8>(tile, C::kChunk, row - lane, 0, dst + 2 * D * j, 4 * D,
                                         valid, lane);
                }
            } else {
                const View &w = wg ? p.dk : p.dv;
                put_row_16<D, F16>(acc, tile, C::kChunk, row, 0, wg ? p.scale * back : back,
                                   steps > 0);
                copy_rows_out<D / 8>(tile, C::kChunk, row - lane, 0,
                                     w.p + 2 * (b * w.sb + hk * w.sh + (key - lane) * w.st),
                                     2 * w.st, valid, lane);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0 && bar->abort) report(p.s.status, SVGA_ERR_TIMEOUT);
}

// Adds the parts of dkdv's split items in part order: one thread per 8 values of a row.
template <int D, bool F16>
__global__ void __launch_bounds__(256) bwd_join_kernel(const BwdParams p)
{
    pdl_wait();  // the parts
    pdl_start();
    constexpr int kPer = D / 8;
    const long long i = blockIdx.x * 256ll + threadIdx.x;
    const int c = 8 * (int)(i % kPer);
    const long long row_all = i / kPer;
    const int row = (int)(row_all % kT), w = (int)(row_all / kT % 2);
    const long long it = p.split.split_from() + row_all / (2 * kT);
    if (it >= p.split.split_to()) return;
    const int item = (int)it, k = p.split.k(item);
    const int bh = p.s.batch * p.s.hk;
    const int kblk = p.by_bk.of(item), r = item - kblk * bh;
    const int b = p.by_hk.of(r), hk = r - b * p.s.hk, key = kblk * kT + row;
    if (key >= clamped_len(p.s.k_lens, b, p.s.tk)) return;
    const float *src = p.parts + ((p.split.slot(item, 0) * 2 + w) * kT + row) * D + c;
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int j = 0; j < k; ++j) {
        const float4 *at = reinterpret_cast<const float4 *>(src + (long long)j * 2 * kT * D);
        const float4 u = at[0], v = at[1];
        x[0] += u.x;
        x[1] += u.y;
        x[2] += u.z;
        x[3] += u.w;
        x[4] += v.x;
        x[5] += v.y;
        x[6] += v.z;
        x[7] += v.w;
    }
    const float f = w ? p.scale : 1.f;
    uint32_t y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = pack_16x2<F16>(x[2 * j] * f, x[2 * j + 1] * f);
    const View &to = w ? p.dk : p.dv;
    *reinterpret_cast<uint4 *>(to.p + 2 * (b * to.sb + hk * to.sh + key * to.st + c)) =
        make_uint4(y[0], y[1], y[2], y[3]);
}

// ------------------------------------------------------------------------------- dq
struct DqItem {
    int b, h, hk, blk, nq, nk;
    ChunkList list;
    int skip, E;  // the chunks: 0 .. list.a - 1, then skip, skip + 1, ...; how many
};

__device__ __forceinline__ bool make_item(const BwdParams &p, int block, DqItem &it)
{
    // last blocks first: the longest under a causal mask
    const int bh = p.s.batch * p.s.hq;
    const int slot = p.by_bq.of(block), r = block - slot * bh;
    it.b = p.by_hq.of(r);
    it.h = r - it.b * p.s.hq;
    it.hk = p.by_group.of(it.h);
    it.blk = p.n_qblk - 1 - slot;
    it.nq = clamped_len(p.s.q_lens, it.b, p.s.tq);
    it.nk = clamped_len(p.s.k_lens, it.b, p.s.tk);
    const int off = it.nk - it.nq, r0 = it.blk * kT;
    if (r0 >= it.nq) return false;
    // first and last query, a lane each
    const MaskRange mr = mask_range(
        p.s.mask, (threadIdx.x & 1 ? min(r0 + kT, it.nq) - 1 : r0) + off, it.nk);
    it.list = chunk_list<kT>(range_of_lane(mr, 0), range_of_lane(mr, 1));
    it.skip = max(it.list.a, it.list.w0);
    it.E = it.list.a + max(it.list.w1 - it.skip, 0);
    return true;
}

struct DqBars {
    uint64_t q_full;           // Q and dO are in shared memory
    uint64_t a_ready;          // Q is in TMEM (8 warps)
    uint64_t k_full[3], k_empty[3], v_full[2], v_empty[2];
    uint64_t s_full, s_free;   // S of a step is in TMEM, was read into registers (8 warps)
    uint64_t dp_full, dp_free; // the same of dP
    uint64_t ds_ready;         // dS is in its columns (8 warps)
    uint64_t dq_done;          // the dQ product that reads them is done
    uint64_t drain[3];
    uint64_t zero_done;
    uint32_t tmem_base;
    int abort, some;
    DqItem item;
};
static_assert(sizeof(DqBars) <= 512, "barrier space");

template <int D, bool F16>
__device__ __forceinline__ void dq_cta(const CUtensorMap &tmQ, const CUtensorMap &tmO,
                                       const CUtensorMap &tmK, const CUtensorMap &tmV,
                                       const BwdParams &p, uint8_t *smem, int block)
{
    using C = Cfg<D>;
    constexpr uint32_t kS = 0, kDP = 128, kDQ = 256, kDS = 384, kQ = 448;
    uint8_t *sQ = smem, *sO = smem + C::kTile;
    uint8_t *sK = smem + 2 * C::kTile;          // [stage]
    uint8_t *sV = sK + C::kKStages * C::kTile;  // [stage]
    DqBars *bar = reinterpret_cast<DqBars *>(smem + C::kDqData);
    volatile int *abort_flag = &bar->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmO);
        prefetch_tmap(&tmV);
        mbar_init(smem_u32(&bar->q_full), 1);
        mbar_init(smem_u32(&bar->a_ready), 8);
        for (int i = 0; i < C::kKStages; ++i) {
            mbar_init(smem_u32(&bar->k_full[i]), 1);
            mbar_init(smem_u32(&bar->k_empty[i]), 1);
            mbar_init(smem_u32(&bar->drain[i]), 1);
        }
        for (int i = 0; i < C::kVStages; ++i) {
            mbar_init(smem_u32(&bar->v_full[i]), 1);
            mbar_init(smem_u32(&bar->v_empty[i]), 1);
        }
        mbar_init(smem_u32(&bar->s_full), 1);
        mbar_init(smem_u32(&bar->s_free), 8);
        mbar_init(smem_u32(&bar->dp_full), 1);
        mbar_init(smem_u32(&bar->dp_free), 8);
        mbar_init(smem_u32(&bar->ds_ready), 8);
        mbar_init(smem_u32(&bar->dq_done), 1);
        mbar_init(smem_u32(&bar->zero_done), 1);
        bar->abort = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&bar->tmem_base), 512);
        tmem_relinquish();
    }
    // K or V of step i (chunk c of key head hk) into its stage
    auto fetch = [&](int i, bool v, int c, int hk, int b) {
        const int st = i % (v ? C::kVStages : C::kKStages);
        const uint32_t fb = smem_u32(v ? &bar->v_full[st] : &bar->k_full[st]);
        mbar_arrive_expect_tx(fb, C::kTile);
        tma_load_5d(smem_u32((v ? sV : sK) + st * C::kTile), v ? &tmV : &tmK, fb, 0, c * kT, 0,
                    hk * (v ? p.v_mh : p.k_mh), b * (v ? p.v_mb : p.k_mb));
    };
    if (warp == 1) pdl_start();  // the next kernel, once this one has its TMEM
    if (p.s.q_lens || p.s.k_lens) pdl_wait();  // as in dkdv_cta
    if (warp == 0) {
        __syncwarp();
        DqItem mine;
        const bool some = make_item(p, block, mine);  // false: past the sequence's queries
        pdl_wait();
        if (threadIdx.x == 0) {
            bar->item = mine;
            bar->some = some;
            if (some && mine.E > 0) {  // on their way before the CTA meets
                const uint32_t qf = smem_u32(&bar->q_full);
                mbar_arrive_expect_tx(qf, 2 * C::kTile);
                tma_load_5d(smem_u32(sQ), &tmQ, qf, 0, mine.blk * kT, 0, mine.h * p.q_mh, mine.b * p.q_mb);
                tma_load_5d(smem_u32(sO), &tmO, qf, 0, mine.blk * kT, 0, mine.h * p.o_mh, mine.b * p.o_mb);
                for (int v = 0; v < 2; ++v)
                    fetch(0, v, mine.list.a > 0 ? 0 : mine.skip, mine.hk, mine.b);
            }
        }
    }
    pdl_wait();  // (every thread: the rows' statistics)
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar->tmem_base;
    if (!bar->some) {
        if (warp == 1) tmem_dealloc(tmem, 512);
        return;
    }
    const DqItem &it = bar->item;
    const int b = it.b, h = it.h, hk = it.hk, blk = it.blk, nq = it.nq, nk = it.nk, E = it.E;
    const int off = nk - nq, r0 = blk * kT, sinks = it.list.a, skip = it.skip;
    auto chunk_of = [&](int e) { return e < sinks ? e : skip + e - sinks; };
    const int ragged = (p.s.k_lens && nk < p.s.tk && nk % kT) ? nk / kT : -1;

    if (warp < 4) {
        setmaxnreg_dec<kRegsLow>();
        // the ragged chunk, a sequence's last, is the last of the list where it is in it
        const bool clean = E > 0 && chunk_of(E - 1) == ragged;
        if (warp == 0 && E > 0) {
            // -------------------------------------------------------- TMA producer
            int k_issued = 0, v_issued = 0;
            if (threadIdx.x == 0) {
                for (int i = 0; i < E; ++i) {
                    const int c = chunk_of(i), ks = i % C::kKStages, vs = i % C::kVStages;
                    const int kr = i / C::kKStages, vr = i / C::kVStages;
                    if (kr > 0 && !mbar_wait(smem_u32(&bar->k_empty[ks]), (kr - 1) & 1, abort_flag))
                        break;
                    if (i > 0) fetch(i, false, c, hk, b);  // (the first are on their way)
                    k_issued = i + 1;
                    if (vr > 0 && !mbar_wait(smem_u32(&bar->v_empty[vs]), (vr - 1) & 1, abort_flag))
                        break;
                    if (i > 0) fetch(i, true, c, hk, b);
                    v_issued = i + 1;
                }
            }
            __syncwarp();
            if (clean && __shfl_sync(0xffffffffu, k_issued, 0) == E) {
                // keys past the sequence's end read as 0 (this warp filled the stage, so the
                // phase its parity names is the stage's current one)
                const int ks = (E - 1) % C::kKStages;
                const bool ok =
                    mbar_wait(smem_u32(&bar->k_full[ks]), ((E - 1) / C::kKStages) & 1, abort_flag);
                if (__all_sync(0xffffffffu, ok)) {
                    zero_rows<D>(smem_u32(sK + ks * C::kTile), nk % kT, lane);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&bar->zero_done));
                }
            }
            if (lane == 0) {  // every copy lands before the CTA can exit, whichever role aborts
                mbar_wait_bounded(smem_u32(&bar->q_full), 0);
                for (int i = max(k_issued - C::kKStages, 0); i < k_issued; ++i)
                    mbar_wait_bounded(smem_u32(&bar->k_full[i % C::kKStages]),
                                      (i / C::kKStages) & 1);
                for (int i = max(v_issued - C::kVStages, 0); i < v_issued; ++i)
                    mbar_wait_bounded(smem_u32(&bar->v_full[i % C::kVStages]),
                                      (i / C::kVStages) & 1);
            }
        } else if (warp >= 1 && E > 0 && elect_one()) {
            // --------------------------------------------------------- MMA issuers
            // warp 1: S, warp 2: dQ, warp 3: dP
            constexpr uint32_t idS = idesc_16_f32(F16, kT, kT, 0, 0);
            constexpr uint32_t idA = idesc_16_f32(F16, kT, D, 0, 1);
            const uint64_t kmaj = smem_desc_sw128(0, 16, 1024);
            const uint64_t nmaj = smem_desc_sw128(0, C::kChunk, 1024);
            const uint32_t aK = smem_u32(sK) >> 4, aV = smem_u32(sV) >> 4;
            auto k_landed = [&](int i) {
                return mbar_wait(smem_u32(&bar->k_full[i % C::kKStages]), (i / C::kKStages) & 1,
                                 abort_flag);
            };
            auto k_at = [&](int i) { return aK + (i % C::kKStages) * (C::kTile >> 4); };
            bool ok = true;
            if (warp == 1) {
                ok = mbar_wait(smem_u32(&bar->a_ready), 0, abort_flag);
                tc_fence_after();
                for (int i = 0; ok && i < E; ++i) {
                    ok = k_landed(i) &&
                         (!(clean && i == E - 1) ||
                          mbar_wait(smem_u32(&bar->zero_done), 0, abort_flag)) &&
                         (i == 0 || mbar_wait(smem_u32(&bar->s_free), (i - 1) & 1, abort_flag));
                    tc_fence_after();
                    if (!ok) break;
                    product_tk<D>(tmem + kS, tmem + kQ, kmaj + k_at(i), idS);
                    mma_commit(smem_u32(&bar->s_full));
                }
            } else if (warp == 2) {
                for (int i = 0; ok && i < E; ++i) {
                    ok = k_landed(i) && mbar_wait(smem_u32(&bar->ds_ready), i & 1, abort_flag);
                    tc_fence_after();
                    if (!ok) break;
                    product_ts(tmem + kDQ, tmem + kDS, nmaj + k_at(i), idA, i > 0);
                    mma_commit(smem_u32(&bar->dq_done));
                    mma_commit(smem_u32(&bar->k_empty[i % C::kKStages]));
                }
            } else {
                const uint64_t a = kmaj + (smem_u32(sO) >> 4);
                ok = mbar_wait(smem_u32(&bar->q_full), 0, abort_flag);
                for (int i = 0; ok && i < E; ++i) {
                    const int vs = i % C::kVStages;
                    ok = mbar_wait(smem_u32(&bar->v_full[vs]), (i / C::kVStages) & 1, abort_flag) &&
                         (i == 0 || mbar_wait(smem_u32(&bar->dp_free), (i - 1) & 1, abort_flag));
                    tc_fence_after();
                    if (!ok) break;
                    product_ss<D>(tmem + kDP, a, kmaj + aV + vs * (C::kTile >> 4), idS);
                    mma_commit(smem_u32(&bar->dp_full));
                    mma_commit(smem_u32(&bar->v_empty[vs]));
                }
            }
            if (!ok) {
                mma_commit(smem_u32(&bar->drain[warp - 1]));
                mbar_wait_bounded(smem_u32(&bar->drain[warp - 1]), 0);
            }
        }
    } else {
        // ------------------------------------------------------ softmax warpgroups
        setmaxnreg_inc<kRegsHigh>();
        const int wg = (warp - 4) >> 2, quad = warp & 3, row = quad * 32 + lane;
        const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
        const uint32_t tS = tmem + lane_base + kS + 64 * wg;
        const uint32_t tDP = tmem + lane_base + kDP + 64 * wg;
        const uint32_t tDS = tmem + lane_base + kDS + 32 * wg;
        const int qrow = r0 + row;
        MaskRange mr = {0, 0, 0};
        if (qrow < nq) mr = mask_range(p.s.mask, qrow + off, nk);
        const float *st =
            p.stats + (((long long)b * p.s.hq + h) * p.n_qblk + blk) * kStatRows<F16> * kT + row;
        float nl = st[0];
        const float nd = st[kT];
        float back = 1.f;
        bool ok = true;
        if (E > 0) {  // this lane's row of Q to TMEM as packed pairs, each group half of it
            ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar->q_full), 0, abort_flag));
            constexpr int kHalf = D / 4;  // 32-bit columns
            const uint32_t src = smem_u32(sQ) + row * 128;
#pragma unroll
            for (int j = 0; j < kHalf / 16; ++j) {
                uint32_t w[16];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    // 16-byte unit of the row: its 64-column chunk and place in the swizzle
                    const int unit = wg * (kHalf / 4) + 4 * j + u;
                    ld_shared_v4(src + (unit >> 3) * C::kChunk + (((unit & 7) ^ (row & 7)) << 4),
                                 w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
                }
                tmem_st16(tmem + lane_base + kQ + wg * kHalf + 16 * j, w);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(smem_u32(&bar->a_ready));
        }
        // fp16: this query's dS is held times 2^k, by way of P's exponent (after Q is on its way: S
        // is computed meanwhile)
        if constexpr (F16) {
            float most_v = 0.f;
            for (int i = lane; i < E; i += 32) {
                const float4 *m = reinterpret_cast<const float4 *>(
                    p.most_v + (((long long)b * p.s.hk + hk) * p.n_kblk + chunk_of(i)) * C::kParts);
#pragma unroll
                for (int j = 0; j < C::kParts / 4; ++j) {
                    const float4 y = m[j];
                    most_v = fmaxf(most_v, fmaxf(fmaxf(y.x, y.y), fmaxf(y.z, y.w)));
                }
            }
            const int k = bits_to_2_14(st[2 * kT] * warp_max(most_v) + fabsf(nd));
            nl += (float)(k - kPBits);
            back = pow2(-k);
        }
        const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), nl2 = make_float2(nl, nl),
                     nd2 = make_float2(nd, nd);
        const ChunkList list = it.list;
        for (int i = 0; ok && i < E; ++i) {
            const int c = chunk_of(i), base = c * kT + 64 * wg;
            const bool full = list.full(c);
            uint32_t keep[2] = {0u, 0u};
            if (!full) {
#pragma unroll
                for (int w = 0; w < 2; ++w)
                    keep[w] =
                        (bits_below(mr.hi - base - 32 * w) & ~bits_below(mr.lo - base - 32 * w)) |
                        bits_below(mr.sk - base - 32 * w);
            }
            uint32_t x[64];
            float pr[64];
            ok = __all_sync(0xffffffffu,
                            mbar_wait(smem_u32(&bar->s_full), i & 1, abort_flag));
            tc_fence_after();
            if (!ok) break;
            tmem_ld64(tS, x);
            tmem_wait_ld();
            tc_fence_before();  // S is in registers: its columns may take the next step's
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bar->s_free));
            if (!full) {
#pragma unroll
                for (int j = 0; j < 64; ++j)
                    if (!((keep[j >> 5] >> (j & 31)) & 1u)) x[j] = kNegInfBits;
            }
#pragma unroll
            for (int j = 0; j < 64; j += 2) {
                const float2 u = ffma2(make_float2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])),
                                       sc2, nl2);
                pr[j] = fast_exp2(u.x);
                pr[j + 1] = fast_exp2(u.y);
            }
            ok = __all_sync(0xffffffffu,
                            mbar_wait(smem_u32(&bar->dp_full), i & 1, abort_flag));
            tc_fence_after();
            if (!ok) break;
            tmem_ld64(tDP, x);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bar->dp_free));
            {
                uint32_t pk[32];
#pragma unroll
                for (int j = 0; j < 64; j += 2) {
                    float2 u = fadd2(make_float2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])),
                                     nd2);
                    u = ffma2(u, make_float2(pr[j], pr[j + 1]), make_float2(0.f, 0.f));
                    pk[j / 2] = pack_16x2<F16>(u.x, u.y);
                }
                if (!full) {  // 0 also where a dropped pair's product is not finite
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const uint32_t k2 = keep[j >> 4] >> (2 * (j & 15));
                        pk[j] &= ((k2 & 1u) ? 0xffffu : 0u) | ((k2 & 2u) ? 0xffff0000u : 0u);
                    }
                }
                if (i > 0) {  // the last step's dQ product reads the columns
                    ok = __all_sync(0xffffffffu,
                                    mbar_wait(smem_u32(&bar->dq_done), (i - 1) & 1, abort_flag));
                    tc_fence_after();
                    if (!ok) break;
                }
                tmem_st32(tDS, pk);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bar->ds_ready));
        }
        // ------------------------------------ epilogue: each group half the columns
        if (ok && E > 0) {
            ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar->dq_done), (E - 1) & 1, abort_flag));
            tc_fence_after();
        }
        if (ok) {  // through Q's tile, which went to TMEM before the first step
            put_row_16<D / 2, F16>(tmem + lane_base + kDQ + wg * (D / 2), smem_u32(sQ), C::kChunk,
                                   row, wg * (D / 16), p.scale * back, E > 0);
            copy_rows_out<D / 16>(smem_u32(sQ), C::kChunk, row - lane, wg * (D / 16),
                                  p.dq.p + 2 * (b * p.dq.sb + h * p.dq.sh + (qrow - lane) * p.dq.st +
                                                wg * (D / 2)),
                                  2 * p.dq.st, nq - (qrow - lane), lane);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0 && bar->abort) report(p.s.status, SVGA_ERR_TIMEOUT);
}

// dkdv's CTAs, the longer ones, then dq's: the two need nothing of each other, and in one launch
// dq's fill the SMs that dkdv's last round leaves idle.
template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 1)
    bwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmO,
               const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
               const __grid_constant__ BwdParams p)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_misplaced(smem, p.s.status)) return;
    if ((int)blockIdx.x < p.n_dkdv)
        dkdv_cta<D, F16>(tmQ, tmO, tmK, tmV, p, smem, blockIdx.x);
    else
        dq_cta<D, F16>(tmQ, tmO, tmK, tmV, p, smem, blockIdx.x - p.n_dkdv);
}

template <typename K>
svga_status prepare(K kfn, int smem, const char *what)
{
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, kfn) != cudaSuccess) {
        set_error("cudaFuncGetAttributes failed: %s", cudaGetErrorString(cudaGetLastError()));
        return SVGA_ERR_CUDA;
    }
    if (fa.numRegs < kRegsLaunch) {
        // the setmaxnreg split draws on the registers the CTA is launched with
        set_error("%s kernel built with %d registers/thread, the register split needs %d", what,
                  fa.numRegs, kRegsLaunch);
        return SVGA_ERR_UNSUPPORTED;
    }
    if (cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
        cudaSuccess) {
        set_error("cudaFuncSetAttribute(max dynamic shared memory) failed");
        return SVGA_ERR_CUDA;
    }
    return SVGA_OK;
}

template <int D, bool F16>
svga_status launch(const svga_view &d_o, const svga_view &q, const svga_view &k,
                   const svga_view &v, BwdParams &kp, const svga_window_problem *p,
                   cudaStream_t st)
{
    using C = Cfg<D>;
    svga_status rc;
    constexpr int kAlloc = C::kKvAlloc > C::kDqAlloc ? C::kKvAlloc : C::kDqAlloc;
    if ((rc = prepare(bwd_kernel<D, F16>, kAlloc, "window backward")) != SVGA_OK) return rc;
    alignas(64) CUtensorMap tq, to, tk, tv;
    // an empty side is never loaded: its maps only have to be valid
    const bool hq = p->q_tokens > 0, hk = p->k_tokens > 0;
    const svga_view &qs = hq ? q : k, &os = hq ? d_o : k, &ks = hk ? k : q, &vs = hk ? v : q;
    const int qb = hq ? p->batch : 1, qh = hq ? p->q_heads : 1, qt = std::max(p->q_tokens, 1);
    const int kb = hk ? p->batch : 1, kh = hk ? p->kv_heads : 1, kt = std::max(p->k_tokens, 1);
    if (!make_view_map(&tq, qs, qb, qh, qt, D, p->dtype, kT, &kp.q_mh, &kp.q_mb) ||
        !make_view_map(&to, os, qb, qh, qt, D, p->dtype, kT, &kp.o_mh, &kp.o_mb) ||
        !make_view_map(&tk, ks, kb, kh, kt, D, p->dtype, kT, &kp.k_mh, &kp.k_mb) ||
        !make_view_map(&tv, vs, kb, kh, kt, D, p->dtype, kT, &kp.v_mh, &kp.v_mb)) {
        set_error("cuTensorMapEncodeTiled failed (driver entry point or arguments)");
        return SVGA_ERR_CUDA;
    }
    if (hq) {
        const long long n = (long long)p->batch * p->q_heads * kp.n_qblk +
                            (F16 ? (long long)p->batch * p->kv_heads * kp.n_kblk : 0);
        rc = launch_after(bwd_rows_kernel<D, F16>, (unsigned)(n * C::kParts), 256, 0, st,
                          "window backward rows", kp);
        if (rc != SVGA_OK) return rc;
    }
    kp.n_dkdv = hk ? (int)kp.split.ctas() : 0;
    const long long n_dq = hq ? (long long)p->batch * p->q_heads * kp.n_qblk : 0;
    const unsigned grid = (unsigned)(kp.n_dkdv + n_dq);
    rc = launch_after(bwd_kernel<D, F16>, grid, kThreads, kAlloc, st, "window backward", tq, to, tk,
                      tv, kp);
    if (rc != SVGA_OK) return rc;
    if (hk && kp.split.slots() > 0) {
        const long long n =
            (long long)(kp.split.split_to() - kp.split.split_from()) * 2 * kT * (D / 8);
        rc = launch_after(bwd_join_kernel<D, F16>, (unsigned)((n + 255) / 256), 256, 0, st,
                          "window backward join", kp);
    }
    return rc;
}

View to_view(const svga_view &v)
{
    return {static_cast<char *>(v.data), v.stride_batch, v.stride_head, v.stride_token};
}

}  // namespace

// Floats of the workspace before the parts: the rows' statistics and, in fp16, the largest norms.
struct RowFloats {
    size_t stats, most_q, most_v;
    size_t all() const { return stats + most_q + most_v; }
};

static RowFloats row_floats(const svga_window_problem *p)
{
    const size_t q = (size_t)p->batch * p->q_heads * ((p->q_tokens + kT - 1) / kT);
    const size_t k = (size_t)p->batch * p->kv_heads * ((p->k_tokens + kT - 1) / kT);
    if (p->dtype != SVGA_F16) return {q * kStatRows<false> * kT, 0, 0};
    const int parts = p->head_dim == 128 ? Cfg<128>::kParts : Cfg<64>::kParts;
    return {q * kStatRows<true> * kT, q * parts * 2, k * parts};
}

// How dkdv's items are split.  Items are key blocks; the ones that hold sinks, first in launch
// order, are kept by every later query of a causal mask, the others by a window of them.
// `per_sm` is the launch's work divided by the SMs, in steps of dkdv (dq has as many steps,
// at about three quarters of the time): a longer item holds up the whole launch, while parts
// cost their sums in memory and a join.  Sinks are split above per_sm, others, which overlap
// less, above 1.25 of it, and nothing into parts of fewer than 8 steps, unless the whole launch
// is less than one round of CTAs: then as finely as still fits in one, where that is not much
// coarser (3 x 1,176 tokens, 3 heads of 64 on 1, 30 items of 30 steps: in three 40 us, whole 52).  Measured (backward in
// all, us): 8,192 tokens causal, 8 heads on 2, per_sm 200: in two 367, unsplit 450; 13 frames of
// 960 tokens, per_sm 129, sinks of 98 steps: unsplit 252, sinks in two 260, in four 265; 2,048
// tokens causal, 4 heads, per_sm 6: unsplit 34, in two 37; 2 x 2,001 tokens in a window, per_sm
// 15, sinks of 64 steps: sinks in five and the others in two 48, unsplit 121; 1,000 tokens, 8
// heads of 64 on 2, a window of 300, one round: in five 21, in two 26, unsplit 36.
static Split choose_bwd_split(const svga_window_problem *p)
{
    const long long heads = (long long)p->batch * p->kv_heads;
    const int blocks = (p->k_tokens + kT - 1) / kT, group = p->q_heads / p->kv_heads;
    const long long n = heads * blocks;
    Split s = {(int)n, 0, 1, 1};
    if (n == 0 || p->q_tokens == 0) return s;
    const Mask m = to_mask(p->mask);
    const int sinks = m.window >= 0 ? std::min((std::min(m.sinks, p->k_tokens) + kT - 1) / kT, blocks) : 0;
    const int off = p->k_tokens - p->q_tokens;
    auto steps_of = [&](int kb) {
        const int k0 = kb * kT, k1 = std::min(k0 + kT, p->k_tokens);
        int first, end, x, end1;
        mask_rows(m, k0, p->q_tokens, off, first, end);
        mask_rows(m, k1 - 1, p->q_tokens, off, x, end1);
        end = std::max(end, end1);
        return end > first ? (long long)group * ((end + kT - 1) / kT - first / kT) : 0ll;
    };
    // the longest and the mean of either kind, over at most 64 blocks of each
    long long top[2] = {0, 0};
    double mean[2] = {0, 0};
    for (int w = 0; w < 2; ++w) {
        const int from = w ? sinks : 0, to = w ? blocks : sinks, stride = (to - from) / 64 + 1;
        int count = 0;
        for (int kb = from; kb < to; kb += stride, ++count) {
            const long long x = steps_of(kb);
            top[w] = std::max(top[w], x);
            mean[w] += x;
        }
        mean[w] /= std::max(count, 1);
    }
    const double per_sm = 1.75 * heads * (sinks * mean[0] + (blocks - sinks) * mean[1]) / kSms;
    auto parts = [](long long x, double most) {
        return (int)std::max(1ll, std::min(64ll, (long long)std::ceil(x / most)));
    };
    s.n1 = (int)(heads * sinks);
    s.k1 = parts(top[0], std::max(per_sm, 8.0));
    s.k2 = parts(top[1], std::max(1.25 * per_sm, 8.0));
    const long long free = kSms - (long long)p->batch * p->q_heads * ((p->q_tokens + kT - 1) / kT);
    Split one = s;
    for (double most = 2.0; n <= free; most *= 1.25) {  // one round in all: fill it
        one.k1 = parts(top[0], most);
        one.k2 = parts(top[1], most);
        if (one.ctas() <= free) {
            // (unless that leaves parts of more than twice the length)
            if (s.k1 <= 2 * one.k1 && s.k2 <= 2 * one.k2) s = one;
            break;
        }
    }
    return s;
}

size_t window_bwd_workspace(const svga_window_problem *p)
{
    return (row_floats(p).all() + (size_t)choose_bwd_split(p).slots() * 2 * kT * p->head_dim) *
           sizeof(float);
}

svga_status launch_window_bwd(const svga_view &d_o, const svga_view &q, const svga_view &k,
                              const svga_view &v, const svga_view &o, const float *lse,
                              const svga_view &dq, const svga_view &dk, const svga_view &dv,
                              const svga_window_problem *p, float scale, void *ws, void *stream)
{
    BwdParams kp{};
    kp.s = to_shape(p);
    kp.d_o = to_view(d_o);
    kp.o = to_view(o);
    kp.v = to_view(v);
    kp.dq = to_view(dq);
    kp.dk = to_view(dk);
    kp.dv = to_view(dv);
    kp.lse = lse;
    kp.stats = static_cast<float *>(ws);
    kp.scale = scale;
    kp.scale_log2 = scale * kLog2e;
    kp.n_qblk = (p->q_tokens + kT - 1) / kT;
    kp.n_kblk = (p->k_tokens + kT - 1) / kT;
    kp.split = choose_bwd_split(p);
    kp.by_k1 = fast_div(kp.split.k1);
    kp.by_k2 = fast_div(kp.split.k2);
    kp.by_bk = fast_div(p->batch * p->kv_heads);
    kp.by_hk = fast_div(p->kv_heads);
    kp.by_bq = fast_div(p->batch * p->q_heads);
    kp.by_hq = fast_div(p->q_heads);
    kp.by_group = fast_div(p->q_heads / p->kv_heads);
    const RowFloats n = row_floats(p);
    kp.most_q = reinterpret_cast<float2 *>(kp.stats + n.stats);
    kp.most_v = kp.stats + n.stats + n.most_q;
    kp.parts = kp.stats + n.all();
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (p->head_dim == 128)
        return p->dtype == SVGA_F16 ? launch<128, true>(d_o, q, k, v, kp, p, st)
                                    : launch<128, false>(d_o, q, k, v, kp, p, st);
    return p->dtype == SVGA_F16 ? launch<64, true>(d_o, q, k, v, kp, p, st)
                                : launch<64, false>(d_o, q, k, v, kp, p, st);
}

}  // namespace svga
