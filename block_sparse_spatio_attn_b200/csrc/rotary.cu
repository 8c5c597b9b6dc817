// rotary.cu -- rotary positions on the three axes of a video grid, and the append of rotated
// keys (and values) to a paged cache.
//
// A pair (x0, x1) of a head's values turns by its axis's angle a = x_axis * theta^(-j / n):
//   y0 = x0 cos a - x1 sin a,   y1 = x1 cos a + x0 sin a   (fp32, rounded once),
// the inverse (and so the backward pass) with -sin a.  cos and sin come from a table built
// in 64 bits, one row per position of each axis: 146 rows for 21 x 45 x 80 tokens, resident
// in L1.  Pure data movement otherwise: each value is read once and written once.
//
// One thread owns one 16-byte piece of a token's row (with halves layout the piece and its
// partner P values further) and walks the heads with it: the token's place and the
// piece's cos / sin are found once for all heads, and the coming heads' pieces are in flight
// in shared memory meanwhile (loads held in registers left 20 KB in flight an SM: 121 us for
// 75,600 tokens of 10 heads).
// Consecutive threads hold consecutive pieces, so rows move whole.  When there are few
// tokens (a decoding step) the heads are dealt over blocks instead, so that the launch
// still covers the GPU.
//
// Bound by HBM.  Measured: 75,600 tokens of 10 heads of 128 (bf16) into each head's order, 387 MB:
// 65 us in a loop, 6.0 TB/s (91 % of the measured copy); append of 2 x 12,480 tokens of 10 heads,
// 256 MB: 43 us, 6.0 TB/s; 64 single tokens of 16 heads: 3.6 us, the time of a launch.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "stream.h"
#include "svga_device.cuh"

namespace svga {
namespace {

constexpr int kThreads = 256;
constexpr int kSlots = 8;  // 16-byte vectors a thread has in flight

struct Orders {
    uint8_t order[kMaxHeads];
};
struct NoOrders {
    uint8_t unused;
};

enum { DST_PLAIN = 0, DST_ORDERED = 1, DST_PAGED = 2 };
enum { LAY_INTERLEAVED = 0, LAY_HALVES = 1, LAY_HALVES_ODD = 2 };

struct RotParams {
    View src, dst;
    View src2;  // paged: the values (copied, not turned)
    int batch, heads, tokens, d, units;
    int heads_per_thread;
    int F, gh, gw, S;
    int pf, ph, P;  // pairs of axis 0, of axis 1, of all
    const float2 *table;
    const int32_t *positions;
    long long first;
    int inverse, turn;
    int32_t *status;
    // paged
    char *k_pages, *v_pages;
    int pages, page_size, max_pages;
    const int32_t *page_table, *lens, *new_lens;
};

template <typename T>
struct Vec {
    static constexpr int N = 16 / sizeof(T);
    T x[N];
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float &y, float x) { y = x; }
__device__ __forceinline__ void from_f(__half &y, float x) { y = __float2half_rn(x); }
__device__ __forceinline__ void from_f(__nv_bfloat16 &y, float x) { y = __float2bfloat16_rn(x); }

// cos and sin of pair i at place (f, r, c)
__device__ __forceinline__ float2 pair_cs(const RotParams &p, int i, int f, int r, int c)
{
    const int pw = p.P - p.pf - p.ph;
    int at;
    if (i < p.pf)
        at = f * p.pf + i;
    else if (i < p.pf + p.ph)
        at = p.F * p.pf + r * p.ph + (i - p.pf);
    else
        at = p.F * p.pf + p.gh * p.ph + c * pw + (i - p.pf - p.ph);
    return p.table[at];
}

// The two values of a packed pair, and back.
__device__ __forceinline__ float2 pair_of(const __nv_bfloat16 *x)
{
    const uint32_t w = *reinterpret_cast<const uint32_t *>(x);
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 pair_of(const __half *x)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(x));
}
__device__ __forceinline__ float2 pair_of(const float *x)
{
    return *reinterpret_cast<const float2 *>(x);
}
__device__ __forceinline__ void set_pair(__nv_bfloat16 *x, float a, float b)
{
    *reinterpret_cast<uint32_t *>(x) = pack_bf16x2(a, b);
}
__device__ __forceinline__ void set_pair(__half *x, float a, float b)
{
    *reinterpret_cast<uint32_t *>(x) = pack_f16x2(a, b);
}
__device__ __forceinline__ void set_pair(float *x, float a, float b)
{
    *reinterpret_cast<float2 *>(x) = make_float2(a, b);
}

// The lanes of one row's pieces: `units` of them from lane `first` on.
__device__ __forceinline__ uint32_t row_lanes(int units, int first)
{
    return units >= 32 ? 0xffffffffu : ((1u << units) - 1u) << first;
}

// Turns the first np of the piece's NP pairs: within a (interleaved), or between a and c.
template <typename T, int LAY, int V, int NP>
__device__ __forceinline__ void turn_piece(T (&a)[V], T (&c)[V], const float (&cs)[NP],
                                           const float (&sn)[NP], int np)
{
    if constexpr (LAY == LAY_INTERLEAVED) {
#pragma unroll
        for (int j = 0; j < NP; ++j)
            if (j < np) {
                const float2 x = pair_of(a + 2 * j);
                set_pair(a + 2 * j, x.x * cs[j] - x.y * sn[j], x.y * cs[j] + x.x * sn[j]);
            }
    } else {  // whole vectors only: the halves layout has no partial piece
#pragma unroll
        for (int j = 0; j < NP; j += 2) {
            const float2 x = pair_of(a + j), y = pair_of(c + j);
            set_pair(a + j, x.x * cs[j] - y.x * sn[j], x.y * cs[j + 1] - y.y * sn[j + 1]);
            set_pair(c + j, y.x * cs[j] + x.x * sn[j], y.y * cs[j + 1] + x.y * sn[j + 1]);
        }
    }
}

template <typename T, int LAY, int DST, typename Ord>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotParams p,
                                                          const __grid_constant__ Ord ord)
{
    constexpr int V = Vec<T>::N;  // values of a piece
    // before anything in memory is looked at: tokens' places, where they are there, else the rows
    // (in between only threads without a token leave)
    const bool placed = DST == DST_PAGED || p.positions;
    if (placed) pdl_wait();
    const long long idx = blockIdx.x * (long long)kThreads + threadIdx.x;
    // 32-bit divisions where the piece index fits (64-bit ones cost a tenth of the kernel)
    const bool small = (long long)p.batch * p.tokens * p.units <= 0x7fffffffll;
    const long long tok_all = small ? (int)idx / p.units : idx / p.units;
    if (tok_all >= (long long)p.batch * p.tokens) return;
    const int unit = (int)(idx - tok_all * p.units);
    const int b = small ? (int)tok_all / p.tokens : (int)(tok_all / p.tokens);
    const int t = (int)(tok_all - (long long)b * p.tokens);
    const bool values = DST == DST_PAGED && blockIdx.z == 1;
    const bool turn = p.turn && !values;

    // the token's place in the grid
    long long pos;
    if (DST == DST_PAGED) {
        const int n = p.new_lens ? p.new_lens[b] : p.tokens;
        const int len = p.lens[b];
        if (n < 0 || n > p.tokens || len < 0) {
            if (unit == 0) report(p.status, SVGA_ERR_INVALID_ARG);
            return;
        }
        if (t >= n) return;
        pos = (long long)len - n + t;
    } else {
        pos = p.positions ? (long long)p.positions[tok_all] : p.first + t;
    }
    int f = 0, s = 0, row = 0, col = 0;
    if (p.turn || DST == DST_ORDERED) {  // (a value goes where its key does, or neither)
        if (pos < 0 || pos >= (long long)p.F * p.S) {
            if (!placed) pdl_wait();  // (the host refuses such a first token: a CTA waits all the same)
            if (unit == 0) report(p.status, SVGA_ERR_INVALID_ARG);
            return;
        }
        f = (int)(pos / p.S);
        s = (int)(pos - (long long)f * p.S);
        row = s / p.gw;
        col = s - row * p.gw;
    }
    long long paged_row = 0;  // row of head 0 in the page array
    if (DST == DST_PAGED) {
        const long long slot = pos < 0 ? -1 : pos / p.page_size;
        const int page = slot >= 0 && slot < p.max_pages
                             ? p.page_table[(long long)b * p.max_pages + slot]
                             : -1;
        if (page < 0 || page >= p.pages) {
            if (unit == 0) report(p.status, SVGA_ERR_INVALID_ARG);
            return;
        }
        paged_row = (long long)page * p.heads * p.page_size + (pos - slot * p.page_size);
    }

    // the piece: values lo .. lo + V - 1 and, with halves, hi .. hi + V - 1
    int lo, hi = -1, pair0 = -1;  // pair0 < 0: copied unchanged
    if (LAY != LAY_HALVES) {
        lo = unit * V;
        if (turn && lo < 2 * p.P) pair0 = LAY == LAY_INTERLEAVED ? lo / 2 : lo;
    } else {
        const int n = p.P / V;  // pieces of the turned half
        if (unit < n) {
            lo = unit * V;
            hi = lo + p.P;
            if (turn) pair0 = lo;
        } else {
            lo = 2 * p.P + (unit - n) * V;
        }
    }

    // rows of the ordered side: one offset per token order
    const View &sv = values ? p.src2 : p.src;
    const T *src = reinterpret_cast<const T *>(sv.p) + b * sv.sb;
    T *dst;
    long long src_at[3], dst_at[3], dst_sh;
    if constexpr (DST == DST_PAGED) {
        dst = reinterpret_cast<T *>(values ? p.v_pages : p.k_pages) + paged_row * p.d;
        dst_sh = (long long)p.page_size * p.d;
    } else {
        dst = reinterpret_cast<T *>(p.dst.p) + b * p.dst.sb;
        dst_sh = p.dst.sh;
    }
#pragma unroll
    for (int k = 0; k < (DST == DST_ORDERED ? 3 : 1); ++k) {
        const int at = DST == DST_ORDERED ? coord_to_pos(k, f, s, p.F, p.S) : t;
        src_at[k] = (p.inverse ? at : t) * sv.st;
        dst_at[k] = DST == DST_PAGED ? 0 : (p.inverse ? t : at) * p.dst.st;
    }

    struct alignas(V * sizeof(T)) Piece {
        T x[V];
    };
    // Heads go by one at a time, kDepth of them in flight: each thread copies its own pieces
    // of the coming heads into its own slots of shared memory (cp.async) and waits for
    // nothing but its own copies.
    constexpr int kVecs = LAY == LAY_HALVES ? 2 : 1;
    constexpr int kDepth = kSlots / kVecs;
    __shared__ uint4 slots[kSlots][kThreads];
    const int h0 = blockIdx.y * p.heads_per_thread;
    const int h1 = min(h0 + p.heads_per_thread, p.heads);
    auto pick = [&](const long long (&at)[3], int h) {
        if constexpr (DST == DST_ORDERED) {
            const int k = ord.order[h];
            return k == 0 ? at[0] : (k == 1 ? at[1] : at[2]);
        } else {
            return at[0];
        }
    };
    auto fetch = [&](int h) {
        if (h < h1) {
            const T *from = src + h * sv.sh + pick(src_at, h);
            const int at = (h - h0) % kDepth * kVecs;
            cp_async_16(smem_u32(&slots[at][threadIdx.x]), from + lo, 16);
            if (kVecs == 2 && hi >= 0)
                cp_async_16(smem_u32(&slots[at + 1][threadIdx.x]), from + hi, 16);
        }
        cp_async_commit();  // (an empty group where no head is left keeps the count)
    };
    if (!placed) pdl_wait();
    pdl_start();
    for (int u = 0; u < kDepth; ++u) fetch(h0 + u);

    // np of the piece's NP angles turn something; with odd halves one angle a value, and the
    // value it goes with (its sine taken negative in the first half) is another piece's
    constexpr int NP = LAY == LAY_INTERLEAVED ? V / 2 : V;
    const int last = LAY == LAY_HALVES_ODD ? 2 * p.P : p.P;
    const int np = pair0 < 0 ? 0 : min(NP, last - pair0);
    float cs[NP], sn[NP];
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        float2 a = make_float2(1.f, 0.f);
        if (j < np) {
            const int i = pair0 + j;
            const bool second = LAY == LAY_HALVES_ODD && i >= p.P;
            a = pair_cs(p, second ? i - p.P : i, f, row, col);
            if (LAY == LAY_HALVES_ODD && !second) a.y = -a.y;
        }
        cs[j] = a.x;
        sn[j] = p.inverse ? -a.y : a.y;
    }
    // the lanes that hold the row's other pieces (all of one row take the same branches)
    const uint32_t mine = row_lanes(p.units, (threadIdx.x & 31) - unit);
    for (int h = h0; h < h1; ++h) {
        Piece a, c;
        cp_async_wait<kDepth - 1>();
        const int at = (h - h0) % kDepth * kVecs;
        a = *reinterpret_cast<const Piece *>(&slots[at][threadIdx.x]);
        if constexpr (kVecs == 2) c = *reinterpret_cast<const Piece *>(&slots[at + 1][threadIdx.x]);
        if constexpr (LAY == LAY_HALVES_ODD) {
            __syncwarp(mine);  // the others' copies have landed too
            const T *whole = reinterpret_cast<const T *>(&slots[at][threadIdx.x - unit]);
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j < np) {
                    const int i = lo + j, other = i < p.P ? i + p.P : i - p.P;
                    from_f(a.x[j], to_f(a.x[j]) * cs[j] + to_f(whole[other]) * sn[j]);
                }
            __syncwarp(mine);  // and were read: the slot takes a later head
        } else if (np == NP) {
            turn_piece<T, LAY, V, NP>(a.x, c.x, cs, sn, NP);
        } else if (np > 0) {  // the piece the turned values end in: the rest stays as it is
            turn_piece<T, LAY, V, NP>(a.x, c.x, cs, sn, np);
        }
        fetch(h + kDepth);
        T *to = dst + h * dst_sh + pick(dst_at, h);
        *reinterpret_cast<Piece *>(to + lo) = a;
        if (kVecs == 2 && hi >= 0) *reinterpret_cast<Piece *>(to + hi) = c;
    }
}

// Table entry (position x, pair j of an axis with n pairs): the angle x * theta^(-j / n) in
// 64 bits.  One thread per entry; built once per grid.
__global__ void __launch_bounds__(kThreads) rotary_table_kernel(int F, int gh, int gw, int pf,
                                                                int ph, int pw, double theta,
                                                                float2 *table)
{
    const int i = blockIdx.x * kThreads + threadIdx.x;
    const int nf = F * pf, nh = gh * ph, nw = gw * pw;
    if (i >= nf + nh + nw) return;
    int k = i, n = pf;
    if (i >= nf + nh) {
        k = i - nf - nh;
        n = pw;
    } else if (i >= nf) {
        k = i - nf;
        n = ph;
    }
    const int x = k / n, j = k - x * n;
    double sn, cs;
    sincos((double)x * pow(theta, -(double)j / n), &sn, &cs);
    table[i] = make_float2((float)cs, (float)sn);
}

View to_view(const svga_view &v)
{
    return {static_cast<char *>(v.data), v.stride_batch, v.stride_head, v.stride_token};
}

// Grid of a launch: pieces over x, heads over y where the tokens alone give too few
// blocks.  Measured on 64 sequences of one token with 16 heads of 64: 16 heads a thread
// leave 2 blocks, one head a thread gives 32; at 75,600 tokens the table look-ups are
// shared by all heads of a thread.
template <typename T, int LAY, int DST, typename Ord>
svga_status launch(RotParams &p, const Ord &ord, cudaStream_t st)
{
    constexpr int V = Vec<T>::N;
    p.units = LAY == LAY_HALVES ? p.P / V + (p.d - 2 * p.P) / V : p.d / V;
    const long long pieces = (long long)p.batch * p.tokens * p.units;
    const long long blocks = (pieces + kThreads - 1) / kThreads;
    if (blocks == 0 || p.heads == 0) return SVGA_OK;
    if (blocks > 0x7fffffffll) {
        set_error("rotary: %lld blocks do not fit one launch", blocks);
        return SVGA_ERR_SHAPE;
    }
    int hpt = p.heads;
    while (hpt > 1 && blocks * ((p.heads + hpt - 1) / hpt) < 2 * 148) hpt = (hpt + 1) / 2;
    p.heads_per_thread = hpt;
    const dim3 grid((unsigned)blocks, (unsigned)((p.heads + hpt - 1) / hpt),
                    DST == DST_PAGED ? 2 : 1);
    return launch_after(rotary_kernel<T, LAY, DST, Ord>, grid, kThreads, 0, st, "rotary", p, ord);
}

template <typename T, int DST, typename Ord>
svga_status launch_layout(RotParams &p, bool interleaved, const Ord &ord, cudaStream_t st)
{
    if (interleaved) return launch<T, LAY_INTERLEAVED, DST>(p, ord, st);
    // halves: with P no multiple of a piece the two values of a pair sit at different places of
    // theirs, and pieces are turned through shared memory
    if (p.P % Vec<T>::N == 0) return launch<T, LAY_HALVES, DST>(p, ord, st);
    return launch<T, LAY_HALVES_ODD, DST>(p, ord, st);
}

template <int DST, typename Ord>
svga_status launch_type(RotParams &p, svga_dtype dt, bool interleaved, const Ord &ord,
                        cudaStream_t st)
{
    if (dt == SVGA_BF16) return launch_layout<__nv_bfloat16, DST>(p, interleaved, ord, st);
    if (dt == SVGA_F16) return launch_layout<__half, DST>(p, interleaved, ord, st);
    if constexpr (DST == DST_PAGED) {
        set_error("a paged cache holds bf16 or fp16");
        return SVGA_ERR_UNSUPPORTED;
    } else {
        return launch_layout<float, DST>(p, interleaved, ord, st);
    }
}

void set_spec(RotParams &p, const svga_rotary_spec *spec, const float *table)
{
    p.F = p.gh = p.gw = p.S = 1;
    if (!spec) return;
    p.F = spec->num_frames;
    p.gh = spec->grid_h;
    p.gw = spec->grid_w;
    p.S = p.gh * p.gw;
    p.pf = spec->pairs[0];
    p.ph = spec->pairs[1];
    p.P = p.pf + p.ph + spec->pairs[2];
    p.table = reinterpret_cast<const float2 *>(table);
    p.turn = 1;
}

}  // namespace

svga_status launch_rotary_table(const svga_rotary_spec *s, double theta, float *table,
                                void *stream)
{
    const int n = s->num_frames * s->pairs[0] + s->grid_h * s->pairs[1] + s->grid_w * s->pairs[2];
    if (n == 0) return SVGA_OK;
    rotary_table_kernel<<<(n + kThreads - 1) / kThreads, kThreads, 0,
                          static_cast<cudaStream_t>(stream)>>>(
        s->num_frames, s->grid_h, s->grid_w, s->pairs[0], s->pairs[1], s->pairs[2], theta,
        reinterpret_cast<float2 *>(table));
    return check_launch_of("rotary table");
}

svga_status launch_rotary(const svga_view &src, const svga_view &dst, int batch, int heads,
                          int tokens, int d, svga_dtype dt, const svga_rotary_spec *spec,
                          const float *table, const int32_t *positions, long long first_token,
                          int inverse, int32_t *status, void *stream)
{
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    RotParams p{};
    p.src = to_view(src);
    p.dst = to_view(dst);
    p.batch = batch;
    p.heads = heads;
    p.tokens = tokens;
    p.d = d;
    set_spec(p, spec, table);
    p.positions = positions;
    p.first = first_token;
    p.inverse = inverse;
    p.status = status;
    if (spec->order) {
        Orders o;
        for (int h = 0; h < heads; ++h) o.order[h] = (uint8_t)spec->order[h];
        return launch_type<DST_ORDERED>(p, dt, spec->interleaved != 0, o, st);
    }
    return launch_type<DST_PLAIN>(p, dt, spec->interleaved != 0, NoOrders{0}, st);
}

svga_status launch_append(const svga_view &k, const svga_view &v, int tokens,
                          const int32_t *new_lens, const svga_paged_cache *c,
                          const svga_rotary_spec *spec, const float *table, void *stream)
{
    RotParams p{};
    p.src = to_view(k);
    p.src2 = to_view(v);
    p.batch = c->batch;
    p.heads = c->kv_heads;
    p.tokens = tokens;
    p.d = c->head_dim;
    set_spec(p, spec, table);
    p.status = c->status;
    p.k_pages = static_cast<char *>(c->k_pages);
    p.v_pages = static_cast<char *>(c->v_pages);
    p.pages = c->pages;
    p.page_size = c->page_size;
    p.max_pages = c->max_pages;
    p.page_table = c->page_table;
    p.lens = c->lens;
    p.new_lens = new_lens;
    return launch_type<DST_PAGED>(p, c->dtype, !spec || spec->interleaved != 0, NoOrders{0},
                                  static_cast<cudaStream_t>(stream));
}

}  // namespace svga
