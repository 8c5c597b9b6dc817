// window_fwd.cu -- attention under a causal window with sinks, forward (sm_100a).
//
//   O_i = sum_j P_ij V_j / sum_j P_ij,  P_ij = exp(scale q_i . k_j - m_i),  j kept by the mask,
//   lse_i = m_i + ln sum_j P_ij.
//
// The design is the block-sparse kernel's (attention.cu: two 128-row query blocks a CTA,
// TMA ring, two tcgen05.mma issuers, S | P0 | P1 | O0 | O1 in TMEM, one row per softmax
// thread, the reference maximum of the first tile kept until a tile's sum would pass a
// limit).  The one S tile the two groups share keeps them half a visit apart, so that one has
// the exponential unit while the other waits; with a tile each (head_dim 64 has the room, and
// P over S would make it) they drift into step and both wait together: 115 us against 106 for
// 148 items of 64 chunks at head_dim 64, 173 against 140 at 128.  What differs:
//   * the visited key chunks need no map: the keys a run of queries keeps are [0, sk) and
//     [lo, hi), all monotone in the position (stream.h), so every role computes its list;
//   * rows are masked by those two intervals, two shifts a 32-key word;
//   * tensors are strided and batched (5-D tensor maps, one copy a tile), query heads share key
//     heads, every sequence may have its own lengths; rows of V past a sequence's end are set
//     to 0 in shared memory before they meet P (0 times a NaN left there is not 0);
//   * bf16 or fp16.  P is rounded to the tensors' type for its product with V, as the tensor
//     cores take operands of one type: half a step relative, the weight of one rounding of O.  It
//     reaches at most the tile-sum limit: 2^16 in bf16, 65504, the largest value, in fp16.  fp16
//     has few exponents below 1 (steps of 2^-24), and a long tail of keys that all round to 0
//     would be missing from O while it stays in the sum; there the reference lies 2^6 below the
//     first tile's maximum, so that a P is off by at most 2^-31 of the row's largest: n keys by
//     n 2^-31 together, half a step of O at 2^20 keys.  (2^8 would still fit a tile of equal
//     scores, but hardly any later rise: 2 x 4,000 tokens, 16 heads of 64 on 4, four sinks first: 84
//     us against 72.)  A maximum of few keys is soon passed by that of 128, so it is 2^5 below that
//     of two or three and 2^3 below a single key's (a P off by 2^-28; the same with one sink
//     first: 85 us with 2^6, 79 with 2^5, 72.8 so and with none);
//   * with few items for the GPU's SMs some or all key lists are split over CTAs that leave
//     fp32 partial rows in the workspace, joined in a fixed order by a second kernel, whose
//     launch overlaps the first (programmatic dependent launch);
//   * one query block's worth of rows (up to 128) and an even number of query heads to a key
//     head: the two blocks of a CTA are two heads over one stream of keys.
// Bound by the softmax threads: a chunk of both blocks takes 2,700 cycles, 2,048 of them the
// exponential unit's (16 a cycle and SM), 2,060 (head_dim 64: 1,260) the tensor pipe's; a warp
// alone keeps the exponential unit 72 % busy, and loads, barriers and the row's state take a
// visit 700 cycles beside it.  Four softmax warps a sub-partition with half a row each (2,740
// cycles), barriers tested ahead of need and a quarter of the exponentials as polynomials
// (3,300) did not help.  A CTA's start and end take 8,000 cycles (2,700 until its loads are
// out, 2,000 to the first S, 1,000 for the last P V, 2,000 for the rows).
// Measured: 12,480 tokens, 4 heads of 128, frames of 960, window 2 and a sink frame: 97 us, 900
// TFLOP/s of kept pairs (in a loop, where the power limit holds the clock near 1.3 GHz; one launch
// alone 90); 75,600 tokens, 10 heads of 128, frames of 3,600, window 3 and a sink frame: 4.94
// ms, 1,276 TFLOP/s; 2 x 4,000 tokens, 16 heads of 64 on 4, window of 1,024 tokens: 73 us.
// Query blocks are launched last first: under a causal mask those are the longest, and the
// hardware hands CTAs out in index order.  Neighbouring CTAs are heads of one group, so
// the K and V chunks they share meet in L2.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "stream.h"
#include "svga_device.cuh"
#include "tile_out.cuh"

namespace svga {
namespace {

constexpr int kThreads = 384;
constexpr int kKN = 128;  // keys per chunk
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kNegInfBits = 0xff800000u;
// registers: the producer / MMA warpgroup drops to kRegsLow, the softmax warpgroups rise to
// kRegsHigh (checked against the launch's on the host)
constexpr int kRegsLaunch = 168, kRegsLow = 120, kRegsHigh = 192;
static_assert(128 * kRegsLow + 256 * kRegsHigh <= kThreads * kRegsLaunch, "register split");
// TMEM columns: S of whichever group's turn it is, then a P tile (packed pairs) and an O a group
constexpr uint32_t kTmS = 0, kTmP = 128, kTmO = 256;
constexpr int kMinChunksPerSplit = 4;
constexpr int kSms = 148;

struct FwdParams {
    WindowShape s;
    View o;
    float *lse;
    float scale_log2;
    int n_pairs;    // items per (sequence, head or pair of heads)
    int by_heads;   // 1: an item's two blocks are block 0 of two heads
    Split split;    // over items, last query blocks first
    FastDiv by_k1, by_k2, by_bh, by_h;  // the split's parts, (sequence, head) pairs, heads
    int q_mb, q_mh, k_mb, k_mh, v_mb, v_mh;  // coordinate multipliers (0: broadcast)
    float *part_o;    // [slot][256][d], unnormalised
    float2 *part_ml;  // [slot][256] (reference maximum, sum)
};

template <int D>
struct Cfg {
    static constexpr int kQBytes = kBlockM * D * 2;
    static constexpr int kQChunk = kBlockM * 128;  // 64 columns x 128 rows
    static constexpr int kKVBytes = kKN * D * 2;
    static constexpr int kKVChunk = kKN * 128;
    static constexpr int kStages = D == 128 ? 5 : 8;
    static constexpr int kSmemData = 2 * kQBytes + kStages * kKVBytes;
    static constexpr int kSmemAlloc = kSmemData + 1024 + 1024;  // barriers, alignment slack
    // one CTA per SM: the TMEM of a CTA is the whole SM's
    static constexpr int kSmemLaunch = kSmemAlloc < 120 * 1024 ? 120 * 1024 : kSmemAlloc;
    static_assert(kSmemAlloc <= 227 * 1024, "shared memory budget");
};

constexpr uint32_t kV0 = 1, kF0 = 2, kV1 = 4, kF1 = 8;

// One CTA's work: two query blocks of one head and its share of their merged chunk list.
struct Item {
    int b, h, b0, nq, nk;
    bool valid1;
    int ksplit;
    long long slot;
    ChunkList l0, l1;
    int a, skip;  // merged list: chunks 0 .. a - 1, then skip, skip + 1, ...
    int e0, E;    // this CTA's entries
    __device__ __forceinline__ int chunk(int n) const
    {
        const int e = e0 + n;
        return e < a ? e : skip + e - a;
    }
    __device__ __forceinline__ uint32_t flags(int c) const
    {
        uint32_t f = l0.visits(c) ? kV0 | (l0.full(c) ? kF0 : 0u) : 0u;
        if (valid1 && l1.visits(c)) f |= kV1 | (l1.full(c) ? kF1 : 0u);
        return f;
    }
};

struct Barriers {
    uint64_t q_full;
    uint64_t kv_full[8], kv_empty[8];
    uint64_t s_full[2];    // [group]: that group's S is in the S columns
    uint64_t s_free;       // the S columns were read into registers (4 warps)
    uint64_t p_full[2];    // [group]: P of the group's tile is in its P columns (4 warps)
    uint64_t o_done[2];    // [group]: the group's last P V product is done
    uint64_t drain[2];     // abort: [issuer]: the MMAs that issuer started are done
    uint64_t zero_req, zero_done;  // the ragged V chunk landed / its rows past the end are 0
    uint32_t tmem_base;
    int abort;
    int some;   // the item has queries
    Item item;  // worked out by warp 3 for all: by every warp it took 2,000 cycles more
};

__device__ __forceinline__ int clamped_len(const int32_t *lens, int b, int most)
{
    return lens ? min(max(lens[b], 0), most) : most;
}

// Item `i` in launch order: its sequence, first head and first 128-row block.
__device__ __forceinline__ void place_item(const FwdParams &p, int i, int &b, int &h, int &b0)
{
    const int heads = p.by_heads ? p.s.hq / 2 : p.s.hq, bh = p.s.batch * heads;
    const int pair = p.by_bh.of(i), r = i - pair * bh;
    b = p.by_h.of(r);
    h = (r - b * heads) << p.by_heads;
    b0 = 2 * (p.n_pairs - 1 - pair);
}

// In two steps, by a whole warp: where the item's queries are (false: past the sequence's end),
// which is all their load needs, and which keys they visit.
__device__ __forceinline__ bool make_item(const FwdParams &p, Item &it, int &part)
{
    int item;
    p.split.of_block(blockIdx.x, p.by_k1, p.by_k2, item, part);
    place_item(p, item, it.b, it.h, it.b0);
    it.ksplit = p.split.k(item);
    it.slot = it.ksplit > 1 ? p.split.slot(item, part) : 0;
    it.nq = clamped_len(p.s.q_lens, it.b, p.s.tq);
    it.nk = clamped_len(p.s.k_lens, it.b, p.s.tk);
    const int r0 = it.b0 * kBlockM;
    it.valid1 = p.by_heads || r0 + kBlockM < it.nq;
    return r0 < it.nq;
}

__device__ __forceinline__ void make_lists(const FwdParams &p, Item &it, int part)
{
    const int off = it.nk - it.nq, r0 = it.b0 * kBlockM;
    // first and last query of the two blocks, a lane each
    const int lane = threadIdx.x & 31, e = lane & 3;
    const int row = e == 0 ? r0 : min(r0 + (e == 1 ? kBlockM : e == 2 ? kBlockM + 1 : 2 * kBlockM),
                                      it.nq) - 1;
    const MaskRange mr = mask_range(p.s.mask, row + off, it.nk);
    it.l0 = it.l1 = chunk_list<kKN>(range_of_lane(mr, 0), range_of_lane(mr, 1));
    const ChunkList l1 = chunk_list<kKN>(range_of_lane(mr, 2), range_of_lane(mr, 3));
    if (!p.by_heads && it.valid1) it.l1 = l1;
    int end;
    merge_lists(it.l0, it.l1, it.valid1, it.a, it.skip, end);
    const int all = it.a + end - it.skip;  // below 2^18; times a part's number below 2^31
    it.e0 = 0;
    it.E = all;
    if (it.ksplit > 1) {
        it.e0 = part * all / it.ksplit;
        it.E = (part + 1) * all / it.ksplit - it.e0;
    }
}

// bits [0, n) of a 32-bit word
__device__ __forceinline__ uint32_t bits_below(int n)
{
    return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u);
}

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 1)
    window_fwd_kernel(const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const FwdParams p)
{
    using C = Cfg<D>;
    constexpr float kSumLimit = F16 ? 65504.f : 65536.f;
    // log2: the reference lies this far below a maximum of `keys` scores
    auto below = [](int keys) {
        return !F16 ? 0.f : (keys >= 4 ? 6.f : (keys >= 2 ? 5.f : 3.f));
    };
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~uintptr_t(1023));
    uint8_t *sQ = smem;
    uint8_t *sKV = smem + 2 * C::kQBytes;
    Barriers *bar = reinterpret_cast<Barriers *>(smem + C::kSmemData);
    volatile int *abort_flag = &bar->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // warps 0 and 3 set up what the first loads need and start them, warp 2 the rest
    if (threadIdx.x == 64) {
        for (int s = 0; s < C::kStages; ++s) mbar_init(smem_u32(&bar->kv_empty[s]), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&bar->s_full[i]), 1);
            mbar_init(smem_u32(&bar->p_full[i]), 4);
            mbar_init(smem_u32(&bar->o_done[i]), 1);
            mbar_init(smem_u32(&bar->drain[i]), 1);
        }
        mbar_init(smem_u32(&bar->s_free), 4);
        mbar_init(smem_u32(&bar->zero_req), 1);
        mbar_init(smem_u32(&bar->zero_done), 1);
        bar->abort = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&bar->tmem_base), 512);
        tmem_relinquish();
    }
    // Before anything in memory is looked at: the lengths, where sequences have their own, then
    // the tensors.
    if (p.s.q_lens || p.s.k_lens) pdl_wait();
    Item it;
    // K (idx even) or V of entry idx / 2 into its stage
    auto fetch = [&](int idx) {
        const int s = idx % C::kStages, t = idx & 1, row = it.chunk(idx >> 1) * kKN;
        const int hk = it.h / p.s.group;
        const uint32_t fb = smem_u32(&bar->kv_full[s]);
        mbar_arrive_expect_tx(fb, C::kKVBytes);
        tma_load_5d(smem_u32(sKV + s * C::kKVBytes), t ? &tmV : &tmK, fb, 0, row, 0,
                    hk * (t ? p.v_mh : p.k_mh), it.b * (t ? p.v_mb : p.k_mb));
    };
    // Q and the first K and V are on their way before the CTA meets: warp 0 loads Q, which needs
    // only the item's place, while warp 3 works out the list of keys (one warp for both takes 500
    // cycles more).
    if (warp == 0) {
        const uint32_t qf = smem_u32(&bar->q_full);
        if (threadIdx.x == 0) {
            prefetch_tmap(&tmQ);
            mbar_init(qf, 1);
            fence_barrier_init();
        }
        __syncwarp();  // (or what follows is run for one lane and for the others one after the other)
        int part;
        const bool some = make_item(p, it, part);
        pdl_wait();
        if (some && threadIdx.x == 0) {
            const int nq_tiles = it.valid1 ? 2 : 1;
            mbar_arrive_expect_tx(qf, nq_tiles * C::kQBytes);
            for (int i = 0; i < nq_tiles; ++i)
                tma_load_5d(smem_u32(sQ + i * C::kQBytes), &tmQ, qf, 0,
                            (it.b0 + (p.by_heads ? 0 : i)) * kBlockM, 0,
                            (it.h + (p.by_heads ? i : 0)) * p.q_mh, it.b * p.q_mb);
        }
    } else if (warp == 3) {
        if (elect_one()) {
            prefetch_tmap(&tmK);
            prefetch_tmap(&tmV);
            for (int s = 0; s < C::kStages; ++s) mbar_init(smem_u32(&bar->kv_full[s]), 1);
            fence_barrier_init();
        }
        __syncwarp();
        int part;
        const bool some = make_item(p, it, part);
        if (some) make_lists(p, it, part);
        pdl_wait();
        if (elect_one()) {
            if (some && it.E > 0) {
                fetch(0);
                fetch(1);
            }
            bar->item = it;
            bar->some = some;
        }
    }
    pdl_wait();
    if (warp == 1) pdl_start();  // (the next kernel's CTAs find no TMEM left to wait for)
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar->tmem_base;
    if (!bar->some) {
        if (warp == 1) tmem_dealloc(tmem, 512);
        return;
    }

    if (warp < 4) {
        setmaxnreg_dec<kRegsLow>();
        it = bar->item;
        // the chunk whose last rows lie past the sequence's end but inside the tensor
        const int ragged = (p.s.k_lens && it.nk < p.s.tk && it.nk % kKN) ? it.nk / kKN : -1;
        // Two threads issue the products: warp 1's S = Q K^T, warp 3's O += P V.  Each waits on its
        // own barriers only, its loads before the softmax threads; the hazards between them go
        // through the softmax groups' barriers.  Both walk the visits: (entry n, group g), entries
        // ascending, group 0 before group 1.
        auto landed = [&](int idx) {
            return mbar_wait(smem_u32(&bar->kv_full[idx % C::kStages]), (idx / C::kStages) & 1,
                             abort_flag);
        };
        auto release = [&](int idx) {
            if (idx + C::kStages < 2 * it.E) mma_commit(smem_u32(&bar->kv_empty[idx % C::kStages]));
        };
        auto stage_at = [&](int idx) {
            return (smem_u32(sKV) >> 4) + (idx % C::kStages) * (C::kKVBytes >> 4);
        };
        auto give_up = [&](int i) {  // every MMA the thread issued ends before TMEM is freed
            mma_commit(smem_u32(&bar->drain[i]));
            mbar_wait_bounded(smem_u32(&bar->drain[i]), 0);
        };
        auto issue_s = [&]() {
            constexpr uint32_t id = idesc_16_f32(F16, kBlockM, kKN, 0, 0);
            const uint64_t desc = smem_desc_sw128(0, 16, 1024);
            bool ok = it.E == 0 || mbar_wait(smem_u32(&bar->q_full), 0, abort_flag);
            int k = 0;  // visits done
            for (int n = 0; ok && n < it.E; ++n) {
                const uint32_t f = it.flags(it.chunk(n));
                ok = landed(2 * n);
#pragma unroll 1
                for (int g = (f & kV0) ? 0 : 1; ok && g < 2; ++g) {
                    if (g == 1 && !(f & kV1)) break;
                    // once the owner of the previous visit has read its S
                    if (k > 0 && !(ok = mbar_wait(smem_u32(&bar->s_free), (k - 1) & 1, abort_flag)))
                        break;
                    tc_fence_after();
                    const uint64_t a0 = desc + ((smem_u32(sQ) + g * C::kQBytes) >> 4);
                    const uint64_t b0 = desc + stage_at(2 * n);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        mma_ss(tmem + kTmS,
                               a0 + (uint32_t)(((kk >> 2) * C::kQChunk + (kk & 3) * 32) >> 4),
                               b0 + (uint32_t)(((kk >> 2) * C::kKVChunk + (kk & 3) * 32) >> 4), id,
                               kk > 0 ? 1u : 0u);
                    mma_commit(smem_u32(&bar->s_full[g]));
                    if (g == 1 || !(f & kV1)) release(2 * n);
                    ++k;
                }
            }
            if (!ok) give_up(0);
        };
        auto issue_pv = [&]() {
            constexpr uint32_t id = idesc_16_f32(F16, kBlockM, D, 0, 1);
            const uint64_t desc = smem_desc_sw128(0, C::kKVChunk, 1024);
            bool ok = true;
            int done[2] = {0, 0};
            for (int n = 0; ok && n < it.E; ++n) {
                const int chunk = it.chunk(n);
                const uint32_t f = it.flags(chunk);
                ok = landed(2 * n + 1);
                if (ok && chunk == ragged) {  // warp 2 clears the rows past the end
                    mbar_arrive(smem_u32(&bar->zero_req));
                    ok = mbar_wait(smem_u32(&bar->zero_done), 0, abort_flag);
                }
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    if (!ok || !(f & (g ? kV1 : kV0))) continue;
                    ok = mbar_wait(smem_u32(&bar->p_full[g]), done[g] & 1, abort_flag);
                    tc_fence_after();
                    if (!ok) break;
                    const uint64_t b0 = desc + stage_at(2 * n + 1);
#pragma unroll
                    for (int kk = 0; kk < kKN / 16; ++kk)
                        mma_ts(tmem + kTmO + g * 128, tmem + kTmP + g * 64 + kk * 8,
                               b0 + (uint32_t)(kk * (2048 >> 4)), id,
                               (done[g] != 0 || kk > 0) ? 1u : 0u);
                    mma_commit(smem_u32(&bar->o_done[g]));
                    if (g == 1 || !(f & kV1)) release(2 * n + 1);
                    ++done[g];
                }
            }
            if (!ok) give_up(1);
        };
        if (threadIdx.x == 0) {
            // -------------------------------------------------------- TMA producer
            const uint32_t qf = smem_u32(&bar->q_full);
            int issued = min(2, 2 * it.E);  // the first K and V are on their way
            for (; issued < 2 * it.E; ++issued) {
                const int s = issued % C::kStages, round = issued / C::kStages;
                if (round > 0 && !mbar_wait(smem_u32(&bar->kv_empty[s]), (round - 1) & 1, abort_flag)) break;
                fetch(issued);
            }
            // every copy lands before the CTA can exit, whichever role aborts
            mbar_wait_bounded(qf, 0);
            for (int idx = max(issued - C::kStages, 0); idx < issued; ++idx)
                mbar_wait_bounded(smem_u32(&bar->kv_full[idx % C::kStages]),
                                  (idx / C::kStages) & 1);
        } else if (warp == 1) {
            if (elect_one()) issue_s();
        } else if (warp == 3) {
            if (elect_one()) issue_pv();
        } else if (warp == 2 && ragged >= 0) {
            // --------------------------------- rows of V past the sequence's end read as 0
            int n = it.E - 1;  // the ragged chunk is a sequence's last: its entry, if any
            while (n >= 0 && it.chunk(n) > ragged) --n;
            if (n >= 0 && it.chunk(n) == ragged) {
                const bool ok = mbar_wait_long(smem_u32(&bar->zero_req), 0, abort_flag);
                if (__all_sync(0xffffffffu, ok)) {
                    const uint32_t base =
                        smem_u32(sKV + ((2 * n + 1) % C::kStages) * C::kKVBytes);
                    for (int u = (it.nk % kKN) * 8 + lane; u < kKN * 8; u += 32)
                        for (int c = 0; c < D / 64; ++c)
                            st_shared_v4(base + c * C::kKVChunk + u * 16, 0u, 0u, 0u, 0u);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&bar->zero_done));
                }
            }
        }
    } else {
        // ------------------------------------------------------ softmax warpgroups
        setmaxnreg_inc<kRegsHigh>();
        const int wg = (warp - 4) >> 2, quad = warp & 3, row = quad * 32 + lane;
        const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
        const uint32_t tS = tmem + lane_base + kTmS;
        const uint32_t tP = tmem + lane_base + kTmP + wg * 64;
        const uint32_t tO = tmem + lane_base + kTmO + wg * 128;
        // what the loop needs of the item stays in registers, the rest in shared memory
        const Item &item = bar->item;
        const ChunkList list = wg ? item.l1 : item.l0;
        const bool mine = wg == 0 || item.valid1;
        const int first = item.e0, end = mine ? first + item.E : first;
        const int sinks = item.a, skip = item.skip;
        const int qrow = (item.b0 + (p.by_heads ? 0 : wg)) * kBlockM + row;
        const bool row_valid = qrow < item.nq;
        MaskRange mr = {0, 0, 0};
        if (row_valid) mr = mask_range(p.s.mask, qrow + item.nk - item.nq, item.nk);
        const float sl2 = p.scale_log2;
        float m_used = -INFINITY, l = 0.f;
        int visit = 0;
        bool ok = true;
        for (int e = first; e < end; ++e) {
            const int chunk = e < sinks ? e : skip + e - sinks;
            if (!list.visits(chunk)) continue;
            ok = __all_sync(0xffffffffu,
                            mbar_wait(smem_u32(&bar->s_full[wg]), visit & 1, abort_flag));
            tc_fence_after();
            if (!ok) break;
            uint32_t r[kKN];
#pragma unroll
            for (int j = 0; j < kKN / 32; ++j)
                tmem_ld32(tS + j * 32, *reinterpret_cast<uint32_t(*)[32]>(&r[j * 32]));
            tmem_wait_ld();
            tc_fence_before();  // S is in registers: its columns may take another visit's
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bar->s_free));
            int keys = kKN;  // the row keeps, of the chunk
            if (!list.full(chunk)) {
                const int k0 = chunk * kKN;
                keys = 0;
#pragma unroll
                for (int w = 0; w < kKN / 32; ++w) {
                    const int x = k0 + 32 * w;
                    const uint32_t keep = (bits_below(mr.hi - x) & ~bits_below(mr.lo - x)) |
                                          bits_below(mr.sk - x);
                    if (F16) keys += __popc(keep);
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (!((keep >> c) & 1u)) r[32 * w + c] = kNegInfBits;
                }
            }
            auto tile_max = [&]() {
                float a0 = -INFINITY, a1 = -INFINITY, a2 = -INFINITY, a3 = -INFINITY;
#pragma unroll
                for (int c = 0; c < kKN; c += 8) {
                    a0 = fmax3(a0, __uint_as_float(r[c]), __uint_as_float(r[c + 1]));
                    a1 = fmax3(a1, __uint_as_float(r[c + 2]), __uint_as_float(r[c + 3]));
                    a2 = fmax3(a2, __uint_as_float(r[c + 4]), __uint_as_float(r[c + 5]));
                    a3 = fmax3(a3, __uint_as_float(r[c + 6]), __uint_as_float(r[c + 7]));
                }
                return fmaxf(fmaxf(a0, a1), fmaxf(a2, a3)) * sl2;
            };
            if (m_used == -INFINITY) m_used = tile_max() - below(keys);
            if (visit > 0) {  // the previous P V reads the P columns this tile writes
                ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar->o_done[wg]),
                                                       (visit - 1) & 1, abort_flag));
                tc_fence_after();
                if (!ok) break;
            }
            float lt;
#pragma unroll 1
            for (int attempt = 0;; ++attempt) {
                const float ms = (m_used == -INFINITY) ? 0.f : m_used;
                const float2 sc2 = make_float2(sl2, sl2), nm2 = make_float2(-ms, -ms);
                float2 s0 = make_float2(0.f, 0.f), s1 = make_float2(0.f, 0.f);
#pragma unroll
                for (int j = 0; j < kKN / 32; ++j) {
                    uint32_t pk[16];
#pragma unroll
                    for (int c2 = 0; c2 < 16; ++c2) {
                        const int c = j * 32 + 2 * c2;
                        const float2 x = ffma2(
                            make_float2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), sc2, nm2);
                        const float2 ev = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                        if (c2 & 1)
                            s1 = fadd2(s1, ev);
                        else
                            s0 = fadd2(s0, ev);
                        pk[c2] = pack_16x2<F16>(ev.x, ev.y);
                    }
                    tmem_st16(tP + j * 16, pk);
                }
                lt = (s0.x + s0.y) + (s1.x + s1.y);
                const bool need = !(lt <= kSumLimit);
                if (attempt > 0 || !__any_sync(0xffffffffu, need)) break;
                // rare: O is rescaled to the tile's exact maximum and the tile is done again (of 128
                // terms whose sum passes the limit one is above 2^8: the reference rises)
                const float m_new = need ? fmaxf(m_used, tile_max() - below(kKN)) : m_used;
                const float fac = need ? fast_exp2(m_used - m_new) : 1.f;
                l *= fac;
                m_used = m_new;
                if (visit > 0) {
#pragma unroll 1
                    for (int j = 0; j < D / 32; ++j) {
                        uint32_t o[32];
                        tmem_ld32(tO + j * 32, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            o[c] = __float_as_uint(__uint_as_float(o[c]) * fac);
                        tmem_st32(tO + j * 32, o);
                    }
                    tmem_wait_st();
                }
            }
            l += lt;
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bar->p_full[wg]));
            ++visit;
        }
        // ----------------------------------------------------------------- epilogue
        if (ok && visit > 0) {
            ok = __all_sync(0xffffffffu,
                            mbar_wait(smem_u32(&bar->o_done[wg]), (visit - 1) & 1, abort_flag));
            tc_fence_after();
        }
        // a group without a visit waited for nothing yet: its Q tile, which the rows go out
        // through, may still be on its way
        if (ok && mine && visit == 0)
            ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar->q_full), 0, abort_flag));
        const Item &it = item;
        const bool split = it.ksplit > 1;
        if (ok && (wg == 0 || it.valid1)) {
            const float inv = split ? 1.f : (l == 0.f ? 0.f : 1.f / l);
            const int h = it.h + (p.by_heads ? wg : 0);
            const long long flat = ((long long)it.b * p.s.hq + h) * p.s.tq + qrow;
            const long long part = it.slot * 2 * kBlockM + wg * kBlockM + row;
            // through this group's Q tile, whose last product is done
            const uint32_t tile = smem_u32(sQ + wg * C::kQBytes);
            const int valid = it.nq - (qrow - lane);  // of the warp's rows
            if (!split) {
                put_row_16<D, F16>(tO, tile, C::kQChunk, row, 0, inv, visit > 0);
                copy_rows_out<D / 8>(tile, C::kQChunk, row - lane, 0,
                                     p.o.p + 2 * (it.b * p.o.sb + h * p.o.sh +
                                                  (qrow - lane) * p.o.st),
                                     2 * p.o.st, valid, lane);
            } else {  // the tile holds half of a row of fp32
#pragma unroll 1
                for (int j = 0; j < 2; ++j) {
                    put_row_32<D / 2>(tO + j * (D / 2), tile, C::kQChunk, row, 1.f, visit > 0);
                    copy_rows_out<D / 8>(tile, C::kQChunk, row - lane, 0,
                                         reinterpret_cast<char *>(p.part_o + (part - lane) * D +
                                                                  j * (D / 2)),
                                         4 * D, valid, lane);
                }
            }
            if (row_valid && split)
                p.part_ml[part] = make_float2(m_used, l);
            else if (row_valid && p.lse)
                p.lse[flat] = l == 0.f ? -INFINITY : (m_used + log2f(l)) * 0.6931471805599453f;
        }
    }

    // ---------------------------------------------------------------- teardown
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0 && bar->abort) report(p.s.status, SVGA_ERR_TIMEOUT);
}

// Join of the split items: one thread per 8 values of a row; the parts' maxima give the
// common scale, sums run in part order.  A part that saw no key of the row has l = 0.
template <bool F16>
__global__ void __launch_bounds__(256) join_kernel(const FwdParams p, int d)
{
    pdl_wait();  // the parts
    pdl_start();
    const int per = d / 8;
    const long long i = blockIdx.x * 256ll + threadIdx.x;
    const long long all = i / per;
    const int c = 8 * (int)(i - all * per), row = (int)(all % (2 * kBlockM));
    const long long it = p.split.split_from() + all / (2 * kBlockM);
    if (it >= p.split.split_to()) return;
    const int item = (int)it, k = p.split.k(item);
    int b, h, b0;
    place_item(p, item, b, h, b0);
    const int g = row / kBlockM;
    h += p.by_heads ? g : 0;
    const int t = (b0 + (p.by_heads ? 0 : g)) * kBlockM + row % kBlockM;
    if (t >= clamped_len(p.s.q_lens, b, p.s.tq)) return;
    const long long at = p.split.slot(item, 0) * 2 * kBlockM + row;
    constexpr int kStep = 2 * kBlockM;  // rows from one part's slot to the next
    float m = -INFINITY;
#pragma unroll 4
    for (int r = 0; r < k; ++r) m = fmaxf(m, p.part_ml[at + r * kStep].x);
    const float ref = m == -INFINITY ? 0.f : m;
    float l = 0.f, x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int r = 0; r < k; ++r) {
        const float2 ml = p.part_ml[at + r * kStep];
        const float4 *src =
            reinterpret_cast<const float4 *>(p.part_o + (at + r * kStep) * d + c);
        const float4 u = src[0], v = src[1];
        const float w = exp2f(ml.x - ref);
        l += w * ml.y;
        x[0] += w * u.x;
        x[1] += w * u.y;
        x[2] += w * u.z;
        x[3] += w * u.w;
        x[4] += w * v.x;
        x[5] += w * v.y;
        x[6] += w * v.z;
        x[7] += w * v.w;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint32_t y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = pack_16x2<F16>(x[2 * j] * inv, x[2 * j + 1] * inv);
    *reinterpret_cast<uint4 *>(p.o.p + 2 * (b * p.o.sb + h * p.o.sh + t * p.o.st + c)) =
        make_uint4(y[0], y[1], y[2], y[3]);
    if (c == 0 && p.lse)
        p.lse[((long long)b * p.s.hq + h) * p.s.tq + t] =
            l == 0.f ? -INFINITY : (ref + log2f(l)) * 0.6931471805599453f;
}

// Two heads a CTA: one query block of rows would leave the second group idle (and its S
// product's latency uncovered).
bool pair_heads(const svga_window_problem *p)
{
    return p->q_tokens <= kBlockM && (p->q_heads / p->kv_heads) % 2 == 0;
}

// Which items are split, from the shapes alone.  An item's list is as long as the shapes allow;
// the GPU runs kSms items at a time.
//   * less than one round of items: all split into as many parts as split_cost finds best.
//     Measured against none, the best of all and what fits one round (us): causal, 4 heads of
//     4,000 tokens, 64 items of 2 to 32 chunks: 33 (3 parts), 56, 33, 39; 8 heads, 128 items: 49
//     (2), 58, 49, 58; 1,000 tokens, 4 heads: 18 (4), 23, 18; one token over 2,000 keys, 8 heads
//     on 1: 14 (8), 31, 14;
//   * more, of lists of about one length (mean at least 0.65 of the longest): those behind the
//     last whole round are split to fill one more, where that shortens it by at least 8 chunks
//     (12,480 tokens of 4 heads, 196 items of 28 chunks: 88 us against 109 unsplit, all split in
//     two 111, the partial sums cost more; 512 items of 9 chunks: 80 against 76, so not there);
//   * nothing from eight rounds on, nor where a causal list without a window makes lengths run
//     from 1 to the longest: those are launched longest first and pack by themselves.
// A part of the second kind keeps at least kMinChunksPerSplit chunks.

// The time of n < kSms items split into k parts each, in chunks: a CTA's start and end cost 3, the
// join 3 and a quarter a part; past one round of CTAs the SMs share the sum, and the last
// CTAs leave half a part's time unused.
double split_cost(long long n, int k, double longest, double mean)
{
    constexpr double kCta = 3, kJoin = 3, kPart = 0.25;
    double t = longest / k + kCta;
    if (n * k > kSms)
        t = std::max(t, n * (mean + k * kCta) / kSms + 0.5 * (mean / k + kCta));
    return k > 1 ? t + kJoin + kPart * k : t;
}

Split choose_split(const svga_window_problem *p)
{
    const long long pairs = (p->q_tokens + 2 * kBlockM - 1) / (2 * kBlockM);
    const long long n = (long long)p->batch * (pair_heads(p) ? p->q_heads / 2 : p->q_heads) * pairs;
    Split s = {(int)n, (int)n, 1, 1};
    if (n == 0 || n >= 8 * kSms || n % kSms == 0 || p->k_tokens == 0) return s;
    const Mask m = to_mask(p->mask);
    const int off = p->k_tokens - p->q_tokens;
    long long longest = 0, sum = 0;
    for (int i = 0; i < pairs; ++i) {
        const int r0 = i * 2 * kBlockM, r1 = std::min(r0 + 2 * kBlockM, p->q_tokens) - 1;
        const ChunkList c = chunk_list<kKN>(m, r0 + off, r1 + off, p->k_tokens);
        const int len = c.a + std::max(c.w1 - std::max(c.a, c.w0), 0);
        longest = std::max<long long>(longest, len);
        sum += len;
    }
    if (n < kSms) {
        const double mean = (double)sum / pairs;
        double best = split_cost(n, 1, longest, mean);
        for (int k = 2; k <= std::min(longest, 64ll); ++k) {
            const double t = split_cost(n, k, longest, mean);
            if (t < best) {
                best = t;
                s.k1 = k;
            } else if (t > best + 2) {  // past the minimum: the parts' own cost grows from here
                break;
            }
        }
    } else if (20 * sum >= 13 * longest * pairs) {
        const int tail = (int)(n % kSms);
        const int k = (int)std::min<long long>(kSms / tail,
                                               std::max(1ll, longest / kMinChunksPerSplit));
        if (longest - longest / k >= 8) {
            s.n1 = (int)n - tail;
            s.k2 = k;
        }
    }
    return s;
}

template <int D, bool F16>
svga_status launch(const svga_view &q, const svga_view &k, const svga_view &v, FwdParams &kp,
                   const svga_window_problem *p, cudaStream_t st)
{
    using C = Cfg<D>;
    auto kfn = window_fwd_kernel<D, F16>;
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, kfn) != cudaSuccess) {
        set_error("cudaFuncGetAttributes failed: %s", cudaGetErrorString(cudaGetLastError()));
        return SVGA_ERR_CUDA;
    }
    if (fa.numRegs < kRegsLaunch) {
        // the setmaxnreg split draws on the registers the CTA is launched with
        set_error("window kernel built with %d registers/thread, the register split needs %d",
                  fa.numRegs, kRegsLaunch);
        return SVGA_ERR_UNSUPPORTED;
    }
    alignas(64) CUtensorMap tq, tk, tv;
    // without keys nothing is loaded: the maps of K and V then only have to be valid
    const svga_view &ks = p->k_tokens ? k : q, &vs = p->k_tokens ? v : q;
    const int kt = std::max(p->k_tokens, 1), kh = p->k_tokens ? p->kv_heads : 1;
    const int kb = p->k_tokens ? p->batch : 1;
    if (!make_view_map(&tq, q, p->batch, p->q_heads, p->q_tokens, D, p->dtype, kBlockM, &kp.q_mh,
                       &kp.q_mb) ||
        !make_view_map(&tk, ks, kb, kh, kt, D, p->dtype, kKN, &kp.k_mh, &kp.k_mb) ||
        !make_view_map(&tv, vs, kb, kh, kt, D, p->dtype, kKN, &kp.v_mh, &kp.v_mb)) {
        set_error("cuTensorMapEncodeTiled failed (driver entry point or arguments)");
        return SVGA_ERR_CUDA;
    }
    if (cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemLaunch) !=
        cudaSuccess) {
        set_error("cudaFuncSetAttribute(max dynamic shared memory) failed");
        return SVGA_ERR_CUDA;
    }
    svga_status rc = launch_after(kfn, (unsigned)kp.split.ctas(), kThreads, C::kSmemLaunch, st,
                                  "window attention", tq, tk, tv, kp);
    if (rc != SVGA_OK || kp.split.slots() == 0) return rc;
    const long long n = (long long)(kp.split.split_to() - kp.split.split_from()) * 2 * kBlockM *
                        (D / 8);
    return launch_after(join_kernel<F16>, (unsigned)((n + 255) / 256), 256, 0, st,
                        "window attention join", kp, D);
}

}  // namespace

size_t window_fwd_workspace(const svga_window_problem *p)
{
    return (size_t)choose_split(p).slots() * 2 * kBlockM * (p->head_dim * 4 + 8);
}

svga_status launch_window_fwd(const svga_view &q, const svga_view &k, const svga_view &v,
                              const svga_view &o, float *lse, const svga_window_problem *p,
                              float scale, void *ws, void *stream)
{
    FwdParams kp{};
    kp.s = to_shape(p);
    kp.o = {static_cast<char *>(o.data), o.stride_batch, o.stride_head, o.stride_token};
    kp.lse = lse;
    kp.scale_log2 = scale * kLog2e;
    kp.n_pairs = (p->q_tokens + 2 * kBlockM - 1) / (2 * kBlockM);
    kp.by_heads = pair_heads(p);
    kp.split = choose_split(p);
    const int heads = kp.by_heads ? p->q_heads / 2 : p->q_heads;
    kp.by_k1 = fast_div(kp.split.k1);
    kp.by_k2 = fast_div(kp.split.k2);
    kp.by_bh = fast_div(p->batch * heads);
    kp.by_h = fast_div(heads);
    kp.part_o = static_cast<float *>(ws);
    kp.part_ml = reinterpret_cast<float2 *>(kp.part_o + (size_t)kp.split.slots() * 2 * kBlockM *
                                                            p->head_dim);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (p->head_dim == 128)
        return p->dtype == SVGA_F16 ? launch<128, true>(q, k, v, kp, p, st)
                                    : launch<128, false>(q, k, v, kp, p, st);
    return p->dtype == SVGA_F16 ? launch<64, true>(q, k, v, kp, p, st)
                                : launch<64, false>(q, k, v, kp, p, st);
}

}  // namespace svga
