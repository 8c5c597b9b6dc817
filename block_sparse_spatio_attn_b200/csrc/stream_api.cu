// stream_api.cu -- the C entry points of the streaming attention calls: checks and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>

#include "stream.h"

namespace svga {

svga_status check_launch_of(const char *what)
{
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
        set_error("%s launch failed: %s", what, cudaGetErrorString(e));
        return SVGA_ERR_CUDA;
    }
    return SVGA_OK;
}

namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

svga_status bad(svga_status rc, const char *fmt, const char *name = "", long long x = 0,
                long long y = 0)
{
    set_error(fmt, name, x, y);
    return rc;
}

int elem_bytes(svga_dtype dt) { return dt == SVGA_F32 ? 4 : 2; }

svga_status check_dtype(svga_dtype dt, bool f32_too)
{
    if (dt == SVGA_BF16 || dt == SVGA_F16 || (f32_too && dt == SVGA_F32)) return SVGA_OK;
    set_error("dtype %d unsupported here (bf16 or fp16%s)", (int)dt, f32_too ? " or fp32" : "");
    return SVGA_ERR_UNSUPPORTED;
}

svga_status check_head_dim(int d)
{
    if (d == 64 || d == 128) return SVGA_OK;
    set_error("head_dim %d unsupported (64 or 128)", d);
    return SVGA_ERR_UNSUPPORTED;
}

svga_status check_word(const int32_t *p, const char *name)
{
    if (p && !aligned(p, 4)) return bad(SVGA_ERR_ALIGNMENT, "%s is not 4-byte aligned", name);
    return SVGA_OK;
}

// A view of batch x heads x tokens rows of d values.  `write`: rows must not overlap, so a
// stride must reach over everything the smaller strides span.  An empty view is not looked
// at beyond its pointer's presence.
svga_status check_view(const svga_view *v, const char *name, int batch, int heads, int tokens,
                       int d, svga_dtype dt, bool write)
{
    if (!v) return bad(SVGA_ERR_INVALID_ARG, "%s is NULL", name);
    if (batch == 0 || heads == 0 || tokens == 0) return SVGA_OK;
    if (!v->data) return bad(SVGA_ERR_INVALID_ARG, "%s has no data", name);
    const int e = elem_bytes(dt);
    if (!aligned(v->data, 16)) return bad(SVGA_ERR_ALIGNMENT, "%s is not 16-byte aligned", name);
    struct Dim {
        long long stride, n;
    } dims[3] = {{v->stride_token, tokens}, {v->stride_head, heads}, {v->stride_batch, batch}};
    for (const Dim &x : dims) {
        if (x.n == 1) continue;
        if (x.stride < 0 || x.stride > (1ll << 38))
            return bad(SVGA_ERR_SHAPE, "%s: stride %lld outside 0 .. 2^38", name, x.stride);
        if (x.stride * e % 16 != 0)
            return bad(SVGA_ERR_ALIGNMENT, "%s: stride of %lld elements is no multiple of 16 bytes",
                       name, x.stride);
    }
    if (tokens > 1 && v->stride_token < d)
        return bad(SVGA_ERR_SHAPE, "%s: token stride %lld below the %lld values of a row", name,
                   v->stride_token, d);
    if (write) {
        std::sort(dims, dims + 3, [](const Dim &a, const Dim &b) { return a.stride < b.stride; });
        long long span = d;
        for (const Dim &x : dims) {
            if (x.n == 1) continue;
            if (x.stride < span)
                return bad(SVGA_ERR_INVALID_ARG,
                           "%s is written, but a stride of %lld makes its rows overlap", name,
                           x.stride);
            span = x.stride * (x.n - 1) + span;
        }
    }
    return SVGA_OK;
}

// [first byte, last byte) a view touches
void extent(const svga_view *v, int batch, int heads, int tokens, int d, int e, const char **lo,
            const char **hi)
{
    const long long n = (batch > 1 ? (batch - 1) * v->stride_batch : 0) +
                        (heads > 1 ? (heads - 1) * v->stride_head : 0) +
                        (tokens > 1 ? (tokens - 1) * v->stride_token : 0) + d;
    *lo = static_cast<const char *>(v->data);
    *hi = *lo + n * e;
}

svga_status check_scale(float scale)
{
    if (!(scale > 0.f) || !(scale < 1e30f))
        return bad(SVGA_ERR_INVALID_ARG, "%sscale must be a positive finite number");
    return SVGA_OK;
}

svga_status check_mask(const svga_window_mask *m)
{
    if (!m) return bad(SVGA_ERR_INVALID_ARG, "%smask is NULL");
    if (m->causal != 0 && m->causal != 1)
        return bad(SVGA_ERR_INVALID_ARG, "%scausal must be 0 or 1");
    if (m->window < -1 || m->window > kMaxMask || m->sinks < 0 || m->sinks > kMaxMask ||
        m->block < 1 || m->block > kMaxMask) {
        set_error("mask outside its range: window %d (-1 .. 2^24), sinks %d (0 .. 2^24), block %d "
                  "(1 .. 2^24)",
                  m->window, m->sinks, m->block);
        return SVGA_ERR_INVALID_ARG;
    }
    return SVGA_OK;
}

svga_status check_window(const svga_window_problem *p)
{
    if (!p) return bad(SVGA_ERR_INVALID_ARG, "%sproblem is NULL");
    svga_status rc;
    if (p->batch < 0 || p->batch > 65535 || p->q_heads < 1 || p->kv_heads < 1 ||
        p->q_heads > kMaxHeads || p->q_heads % p->kv_heads != 0) {
        set_error("batch %d (0 .. 65535), q_heads %d (1 .. %d) or kv_heads %d (a divisor of q_heads) "
                  "out of range",
                  p->batch, p->q_heads, kMaxHeads, p->kv_heads);
        return SVGA_ERR_SHAPE;
    }
    if (p->q_tokens < 0 || p->k_tokens < 0 || p->q_tokens > kMaxTokens ||
        p->k_tokens > kMaxTokens) {
        set_error("q_tokens %d or k_tokens %d outside 0 .. %d", p->q_tokens, p->k_tokens,
                  kMaxTokens);
        return SVGA_ERR_SHAPE;
    }
    if ((rc = check_head_dim(p->head_dim)) != SVGA_OK ||
        (rc = check_dtype(p->dtype, false)) != SVGA_OK || (rc = check_mask(&p->mask)) != SVGA_OK ||
        (rc = check_word(p->q_lens, "q_lens")) != SVGA_OK ||
        (rc = check_word(p->k_lens, "k_lens")) != SVGA_OK ||
        (rc = check_word(p->status, "status")) != SVGA_OK)
        return rc;
    const long long blocks = (long long)p->batch * p->q_heads *
                             ((std::max(p->q_tokens, p->k_tokens) + 127) / 128);
    if (blocks > 0x7fffffffll / 64) {
        set_error("%lld 128-row blocks (batch x heads x tokens) do not fit one launch", blocks);
        return SVGA_ERR_SHAPE;
    }
    return SVGA_OK;
}

svga_status check_workspace(const void *ws, size_t have, size_t need)
{
    if (need == 0) return SVGA_OK;
    if (!ws || !aligned(ws, 256) || have < need) {
        set_error("workspace missing, not 256-byte aligned or smaller than the %zu bytes "
                  "svga_window_attention_size says",
                  need);
        return SVGA_ERR_WORKSPACE;
    }
    return SVGA_OK;
}

svga_status check_spec(const svga_rotary_spec *s, int head_dim)
{
    if (!s) return bad(SVGA_ERR_INVALID_ARG, "%sspec is NULL");
    if (s->num_frames < 1 || s->grid_h < 1 || s->grid_w < 1 ||
        (long long)s->grid_h * s->grid_w > kMaxTokens ||
        (long long)s->grid_h * s->grid_w * s->num_frames > 0x7fffffffll) {
        set_error("grid of %d frames x %d x %d must be positive, below 2^24 tokens a frame and 2^31 "
                  "in all",
                  s->num_frames, s->grid_h, s->grid_w);
        return SVGA_ERR_SHAPE;
    }
    int sum = 0;
    for (int a = 0; a < 3; ++a) {
        if (s->pairs[a] < 0 || s->pairs[a] > 64) {
            set_error("pairs[%d] = %d outside 0 .. 64", a, s->pairs[a]);
            return SVGA_ERR_SHAPE;
        }
        sum += s->pairs[a];
    }
    if (head_dim && sum > head_dim / 2) {
        set_error("%d pairs do not fit a head of %d values", sum, head_dim);
        return SVGA_ERR_SHAPE;
    }
    const long long entries = (long long)s->num_frames * s->pairs[0] +
                              (long long)s->grid_h * s->pairs[1] +
                              (long long)s->grid_w * s->pairs[2];
    if (entries > 0x3fffffffll) {
        set_error("a table of %lld entries is too large (below 2^30)", entries);
        return SVGA_ERR_SHAPE;
    }
    if (s->interleaved != 0 && s->interleaved != 1)
        return bad(SVGA_ERR_INVALID_ARG, "%sinterleaved must be 0 or 1");
    return SVGA_OK;
}

svga_status check_table(const svga_rotary_spec *s, const float *table)
{
    if (s->pairs[0] + s->pairs[1] + s->pairs[2] == 0) return SVGA_OK;
    if (!table) return bad(SVGA_ERR_INVALID_ARG, "%stable is NULL");
    if (!aligned(table, 16)) return bad(SVGA_ERR_ALIGNMENT, "%stable is not 16-byte aligned");
    return SVGA_OK;
}

svga_status check_cache(const svga_paged_cache *c)
{
    if (!c) return bad(SVGA_ERR_INVALID_ARG, "%scache is NULL");
    svga_status rc;
    if ((rc = check_head_dim(c->head_dim)) != SVGA_OK ||
        (rc = check_dtype(c->dtype, false)) != SVGA_OK)
        return rc;
    if (c->page_size < 16 || c->page_size > 1024 || c->page_size % 16 != 0) {
        set_error("page_size %d must be a multiple of 16 in 16 .. 1024", c->page_size);
        return SVGA_ERR_UNSUPPORTED;
    }
    if (c->pages < 0 || c->kv_heads < 1 || c->kv_heads > kMaxHeads || c->batch < 0 ||
        c->batch > 65535 || c->max_pages < 0 ||
        (long long)c->max_pages * c->page_size > kMaxTokens ||
        (long long)c->pages * c->kv_heads * c->page_size > 0x7fffffffll) {
        set_error("cache of %d pages x %d heads x %d rows (below 2^31 rows), batch %d (0 .. 65535) x "
                  "%d pages (at most 2^24 tokens) out of range",
                  c->pages, c->kv_heads, c->page_size, c->batch, c->max_pages);
        return SVGA_ERR_SHAPE;
    }
    if (c->batch == 0) return SVGA_OK;
    if ((c->pages > 0 && (!c->k_pages || !c->v_pages)) || !c->lens ||
        (c->max_pages > 0 && !c->page_table))
        return bad(SVGA_ERR_INVALID_ARG, "%sk_pages, v_pages, page_table and lens must be given");
    if (!aligned(c->k_pages, 16) || !aligned(c->v_pages, 16))
        return bad(SVGA_ERR_ALIGNMENT, "%sk_pages and v_pages must be 16-byte aligned");
    if ((rc = check_word(c->page_table, "page_table")) != SVGA_OK ||
        (rc = check_word(c->lens, "lens")) != SVGA_OK ||
        (rc = check_word(c->status, "status")) != SVGA_OK)
        return rc;
    return SVGA_OK;
}

}  // namespace
}  // namespace svga

using namespace svga;

extern "C" {

svga_status svga_rotary_table_size(const svga_rotary_spec *spec, size_t *bytes)
{
    const svga_status rc = check_spec(spec, 0);
    if (rc != SVGA_OK) return rc;
    if (bytes)
        *bytes = 8 * ((size_t)spec->num_frames * spec->pairs[0] +
                      (size_t)spec->grid_h * spec->pairs[1] + (size_t)spec->grid_w * spec->pairs[2]);
    return SVGA_OK;
}

svga_status svga_rotary_table(const svga_rotary_spec *spec, double theta, float *table,
                              svga_stream_t stream)
{
    svga_status rc = check_spec(spec, 0);
    if (rc != SVGA_OK || (rc = check_table(spec, table)) != SVGA_OK) return rc;
    if (!(theta > 1.0) || !(theta < 1e18))
        return bad(SVGA_ERR_INVALID_ARG, "%stheta must lie in (1, 1e18)");
    return launch_rotary_table(spec, theta, table, stream);
}

svga_status svga_rotary(const svga_view *src, const svga_view *dst, int batch, int heads,
                        int tokens, int head_dim, svga_dtype dtype, const svga_rotary_spec *spec,
                        const float *table, const int32_t *positions, int64_t first_token,
                        int inverse, int32_t *status, svga_stream_t stream)
{
    svga_status rc;
    if ((rc = check_dtype(dtype, true)) != SVGA_OK || (rc = check_head_dim(head_dim)) != SVGA_OK ||
        (rc = check_spec(spec, head_dim)) != SVGA_OK || (rc = check_table(spec, table)) != SVGA_OK)
        return rc;
    if (batch < 0 || heads < 1 || heads > kMaxHeads || tokens < 0 || tokens > kMaxTokens) {
        set_error("batch %d, heads %d (1 .. %d) or tokens %d (0 .. %d) out of range", batch, heads,
                  kMaxHeads, tokens, kMaxTokens);
        return SVGA_ERR_SHAPE;
    }
    if ((rc = check_view(src, "src", batch, heads, tokens, head_dim, dtype, false)) != SVGA_OK ||
        (rc = check_view(dst, "dst", batch, heads, tokens, head_dim, dtype, true)) != SVGA_OK ||
        (rc = check_word(positions, "positions")) != SVGA_OK ||
        (rc = check_word(status, "status")) != SVGA_OK)
        return rc;
    if (inverse != 0 && inverse != 1)
        return bad(SVGA_ERR_INVALID_ARG, "%sinverse must be 0 or 1");
    const long long grid = (long long)spec->num_frames * spec->grid_h * spec->grid_w;
    if (!positions && (first_token < 0 || first_token > grid - tokens))  // (a sum could wrap)
        return bad(SVGA_ERR_SHAPE, "%stokens from first_token %lld on pass the grid's %lld", "",
                   first_token, grid);
    if (spec->order) {
        if (positions || first_token != 0 || tokens != grid)
            return bad(SVGA_ERR_INVALID_ARG,
                       "%san order needs every token of the grid (%lld), no positions and "
                       "first_token 0",
                       "", grid);
        for (int h = 0; h < heads; ++h)
            if (spec->order[h] < SVGA_ORDER_FRAME_MAJOR ||
                spec->order[h] > SVGA_ORDER_TEMPORAL_MAJOR_STRICT) {
                set_error("head %d: order %d invalid", h, spec->order[h]);
                return SVGA_ERR_INVALID_ARG;
            }
    }
    if (batch == 0 || tokens == 0) return SVGA_OK;
    const char *s0, *s1, *d0, *d1;
    extent(src, batch, heads, tokens, head_dim, elem_bytes(dtype), &s0, &s1);
    extent(dst, batch, heads, tokens, head_dim, elem_bytes(dtype), &d0, &d1);
    if (s0 < d1 && d0 < s1) {
        const bool same = s0 == d0 && (batch == 1 || src->stride_batch == dst->stride_batch) &&
                          (heads == 1 || src->stride_head == dst->stride_head) &&
                          (tokens == 1 || src->stride_token == dst->stride_token);
        if (!same || spec->order)
            return bad(SVGA_ERR_INVALID_ARG,
                       "%ssrc and dst overlap (only the same view, without an order, is turned in "
                       "place)");
    }
    return launch_rotary(*src, *dst, batch, heads, tokens, head_dim, dtype, spec, table, positions,
                         first_token, inverse, status, stream);
}

svga_status svga_window_attention_size(const svga_window_problem *problem, size_t *fwd_bytes,
                                       size_t *bwd_bytes)
{
    const svga_status rc = check_window(problem);
    if (rc != SVGA_OK) return rc;
    if (fwd_bytes) *fwd_bytes = window_fwd_workspace(problem);
    if (bwd_bytes) *bwd_bytes = window_bwd_workspace(problem);
    return SVGA_OK;
}

svga_status svga_window_attention_fwd(const svga_view *q, const svga_view *k, const svga_view *v,
                                      const svga_view *o, float *lse,
                                      const svga_window_problem *p, float scale, void *workspace,
                                      size_t workspace_bytes, svga_stream_t stream)
{
    svga_status rc;
    if ((rc = check_window(p)) != SVGA_OK || (rc = check_scale(scale)) != SVGA_OK) return rc;
    const int B = p->batch, H = p->q_heads, G = p->kv_heads, d = p->head_dim;
    if ((rc = check_view(q, "q", B, H, p->q_tokens, d, p->dtype, false)) != SVGA_OK ||
        (rc = check_view(k, "k", B, G, p->k_tokens, d, p->dtype, false)) != SVGA_OK ||
        (rc = check_view(v, "v", B, G, p->k_tokens, d, p->dtype, false)) != SVGA_OK ||
        (rc = check_view(o, "o", B, H, p->q_tokens, d, p->dtype, true)) != SVGA_OK)
        return rc;
    if (lse && !aligned(lse, 4)) return bad(SVGA_ERR_ALIGNMENT, "%slse is not 4-byte aligned");
    if ((rc = check_workspace(workspace, workspace_bytes, window_fwd_workspace(p))) != SVGA_OK)
        return rc;
    if (B == 0 || p->q_tokens == 0) return SVGA_OK;
    if (o->data == q->data || o->data == k->data || o->data == v->data)
        return bad(SVGA_ERR_INVALID_ARG, "%so starts where q, k or v does: it is written while they "
                                         "are read");
    return launch_window_fwd(*q, *k, *v, *o, lse, p, scale, workspace, stream);
}

svga_status svga_window_attention_bwd(const svga_view *d_o, const svga_view *q, const svga_view *k,
                                      const svga_view *v, const svga_view *o, const float *lse,
                                      const svga_view *dq, const svga_view *dk,
                                      const svga_view *dv, const svga_window_problem *p,
                                      float scale, void *workspace, size_t workspace_bytes,
                                      svga_stream_t stream)
{
    svga_status rc;
    if ((rc = check_window(p)) != SVGA_OK || (rc = check_scale(scale)) != SVGA_OK) return rc;
    const int B = p->batch, H = p->q_heads, G = p->kv_heads, d = p->head_dim;
    const struct {
        const svga_view *v;
        const char *name;
        int heads, tokens;
        bool write;
    } views[] = {{d_o, "d_o", H, p->q_tokens, false}, {q, "q", H, p->q_tokens, false},
                 {k, "k", G, p->k_tokens, false},     {v, "v", G, p->k_tokens, false},
                 {o, "o", H, p->q_tokens, false},     {dq, "dq", H, p->q_tokens, true},
                 {dk, "dk", G, p->k_tokens, true},    {dv, "dv", G, p->k_tokens, true}};
    for (const auto &x : views)
        if ((rc = check_view(x.v, x.name, B, x.heads, x.tokens, d, p->dtype, x.write)) != SVGA_OK)
            return rc;
    if (B > 0 && p->q_tokens > 0 && !lse) return bad(SVGA_ERR_INVALID_ARG, "%slse is NULL");
    if (!aligned(lse, 4)) return bad(SVGA_ERR_ALIGNMENT, "%slse is not 4-byte aligned");
    if ((rc = check_workspace(workspace, workspace_bytes, window_bwd_workspace(p))) != SVGA_OK)
        return rc;
    if (B == 0 || (p->q_tokens == 0 && p->k_tokens == 0)) return SVGA_OK;
    for (const auto &x : views)
        for (const auto &y : views)
            if (&x != &y && x.write && x.tokens > 0 && y.tokens > 0 && x.v->data == y.v->data) {
                set_error("%s starts where %s does: it is written while that is read or written",
                          x.name, y.name);
                return SVGA_ERR_INVALID_ARG;
            }
    return launch_window_bwd(*d_o, *q, *k, *v, *o, lse, *dq, *dk, *dv, p, scale, workspace, stream);
}

svga_status svga_cache_append(const svga_view *k, const svga_view *v, int tokens,
                              const int32_t *new_lens, const svga_paged_cache *c,
                              const svga_rotary_spec *spec, const float *table,
                              svga_stream_t stream)
{
    svga_status rc;
    if ((rc = check_cache(c)) != SVGA_OK) return rc;
    if (tokens < 0 || tokens > kMaxTokens) {
        set_error("tokens %d outside 0 .. %d", tokens, kMaxTokens);
        return SVGA_ERR_SHAPE;
    }
    if ((rc = check_view(k, "k", c->batch, c->kv_heads, tokens, c->head_dim, c->dtype, false)) !=
            SVGA_OK ||
        (rc = check_view(v, "v", c->batch, c->kv_heads, tokens, c->head_dim, c->dtype, false)) !=
            SVGA_OK ||
        (rc = check_word(new_lens, "new_lens")) != SVGA_OK)
        return rc;
    if (spec) {
        if ((rc = check_spec(spec, c->head_dim)) != SVGA_OK ||
            (rc = check_table(spec, table)) != SVGA_OK)
            return rc;
        if (spec->order)
            return bad(SVGA_ERR_INVALID_ARG, "%sa cache holds positions in order: spec->order must "
                                             "be NULL");
    } else if (table) {
        return bad(SVGA_ERR_INVALID_ARG, "%sa table without a spec");
    }
    if (c->batch == 0 || tokens == 0) return SVGA_OK;
    if (c->k_pages == c->v_pages)
        return bad(SVGA_ERR_INVALID_ARG, "%sk_pages and v_pages start together: both are written");
    return launch_append(*k, *v, tokens, new_lens, c, spec, table, stream);
}

svga_status svga_cache_decode(const svga_view *q, const svga_view *o, float *lse, int q_heads,
                              const svga_paged_cache *c, const svga_window_mask *mask, float scale,
                              svga_stream_t stream)
{
    svga_status rc;
    if ((rc = check_cache(c)) != SVGA_OK || (rc = check_mask(mask)) != SVGA_OK ||
        (rc = check_scale(scale)) != SVGA_OK)
        return rc;
    if (q_heads < 1 || q_heads > kMaxHeads || q_heads % c->kv_heads != 0) {
        set_error("q_heads %d must be a multiple of kv_heads %d up to %d", q_heads, c->kv_heads,
                  kMaxHeads);
        return SVGA_ERR_SHAPE;
    }
    if ((rc = check_view(q, "q", c->batch, q_heads, 1, c->head_dim, c->dtype, false)) != SVGA_OK ||
        (rc = check_view(o, "o", c->batch, q_heads, 1, c->head_dim, c->dtype, true)) != SVGA_OK)
        return rc;
    if (lse && !aligned(lse, 4)) return bad(SVGA_ERR_ALIGNMENT, "%slse is not 4-byte aligned");
    if (c->batch == 0) return SVGA_OK;
    if (o->data == q->data || (c->pages > 0 && (o->data == c->k_pages || o->data == c->v_pages)))
        return bad(SVGA_ERR_INVALID_ARG, "%so starts where q or the cache does: it is written while "
                                         "they are read");
    return launch_decode(*q, *o, lse, q_heads, c, mask, scale, stream);
}

}  // extern "C"
