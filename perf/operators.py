"""What the operators of streaming video attention cost: rotary positions on three axes, causal
window attention with sinks (forward and backward), the append to a paged key-value cache and the
attention of one new token over it.

`own` chooses between the plain form (elementary torch operations in 32 bits) and the library's
calls; `perf/operators.py` is imported by a measuring program and is not part of the package.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
DEV = "cuda"

# The mask: query i sits at position p = i + (keys - queries) and sees key j when
#   (not causal or block(j) <= block(p)) and (window < 0 or |block(p) - block(j)| <= window or j < sinks)
# with block(x) = floor(x / block).


def _rotary(**kw):
    c = dict(op="rotary", batch=1, heads=1, frames=1, grid_h=1, grid_w=1, tokens=0, dim=128, pf=22, ph=21,
             pw=21, dtype="bf16", interleaved=True, inverse=False, ordered=False, token_major=False)
    c.update(kw)
    return c


def _attn(**kw):
    c = dict(op="fwd", batch=1, q_heads=1, kv_heads=1, q_tokens=1, k_tokens=1, dim=128, dtype="bf16",
             causal=True, window=-1, sinks=0, block=1, ragged=False, token_major=False)
    c.update(kw)
    return c


def _append(**kw):
    c = dict(op="append", batch=1, kv_heads=1, new=1, length=1, page=64, dim=128, dtype="bf16", rotate=True,
             frames=32, grid_h=32, grid_w=64, pf=22, ph=21, pw=21, interleaved=True)
    c.update(kw)
    return c


def _decode(**kw):
    c = dict(op="decode", batch=1, q_heads=1, kv_heads=1, length=1, page=64, dim=128, dtype="bf16", window=-1,
             sinks=0, block=1, ragged=True)
    c.update(kw)
    return c


def listed():
    return [
        # Q of the 75,600-token video layer straight from the projection ([tokens, heads, d]) into each head's
        # token order: what a denoising step does before its sparse attention
        _rotary(name="rotary_video_order", heads=10, frames=21, grid_h=45, grid_w=80, ordered=True, token_major=True),
        # the gradient of the rotated keys back to the projection's layout, in 32 bits, at the 12,480-token size
        _rotary(name="rotary_backward_f32", batch=2, heads=4, frames=13, grid_h=24, grid_w=40, dtype="f32", pf=16,
                ph=24, pw=24, interleaved=False, inverse=True, ordered=True),
        # the queries of one decoding step: one token of each of 64 sequences, each at a place of its own
        _rotary(name="rotary_step", batch=64, heads=16, frames=32, grid_h=32, grid_w=64, tokens=1, dim=64, pf=8,
                ph=12, pw=12, dtype="f16"),
        # frame-causal attention of a 13-frame clip: two frames back, the first frame stays visible
        _attn(name="window_frames", q_heads=4, kv_heads=4, q_tokens=12480, k_tokens=12480, block=960, window=2,
              sinks=960),
        # token-causal window over a discrete token stream, heads shared by four, from the projection's layout
        _attn(name="window_tokens_shared", batch=2, q_heads=16, kv_heads=4, q_tokens=4000, k_tokens=4000, dim=64,
              dtype="f16", window=1023, sinks=4, token_major=True),
        # a chunk of new tokens against a long cache, sequences of unequal length
        _attn(name="window_extend", batch=3, q_heads=8, kv_heads=2, q_tokens=100, k_tokens=16001, ragged=True),
        # training: gradients of the frame-causal clip
        _attn(name="backward_frames", op="bwd", q_heads=4, kv_heads=4, q_tokens=12480, k_tokens=12480, block=960,
              window=2, sinks=960),
        # training: token-causal window, shared heads, an odd length, a padded batch
        _attn(name="backward_tokens_shared", op="bwd", batch=2, q_heads=8, kv_heads=2, q_tokens=2001, k_tokens=2001,
              dtype="f16", window=511, sinks=4, ragged=True),
        # one decoding step's keys and values of 64 sequences, rotated on the way into their pages
        _append(name="append_step", batch=64, kv_heads=8, length=2048, page=16),
        # a whole 12,480-token clip into its pages
        _append(name="append_clip", batch=2, kv_heads=10, new=12480, length=12480, page=64, frames=13, grid_h=24,
                grid_w=40),
        # one token over long caches, eight query heads to a key head
        _decode(name="decode_long", batch=8, q_heads=32, kv_heads=4, length=32768, page=64),
        # one token of many sequences with a window and sinks over small pages, a head to each key head
        _decode(name="decode_window", batch=16, q_heads=10, kv_heads=10, length=8191, page=16, window=1023, sinks=16,
                dtype="f16"),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm where the range is wide."""
    if hi <= lo:
        return lo
    if hi <= 10 * max(1, lo):
        return rng.randint(lo, hi)
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(max(1, lo)), math.log(hi))))))


def _draw_pairs(rng, dim):
    total = dim // 2 if rng.random() < 0.7 else rng.randint(3, dim // 2)
    pf = rng.randint(1, total - 2)
    ph = rng.randint(1, total - pf - 1)
    return dict(pf=pf, ph=ph, pw=total - pf - ph)


def draw(rng):
    kind = rng.choice(["rotary", "fwd", "fwd", "bwd", "append", "decode", "decode"])
    dim = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "f16"])
    if kind == "rotary":
        dtype = rng.choice(["bf16", "f16", "f32"])
        if rng.random() < 0.3:  # single tokens of many sequences
            return _rotary(batch=_spread(rng, 1, 256), heads=rng.randint(1, 32), frames=32, grid_h=32, grid_w=64,
                           tokens=rng.randint(1, 9), dim=dim, dtype=dtype, interleaved=rng.random() < 0.5,
                           inverse=rng.random() < 0.3, token_major=rng.random() < 0.5, **_draw_pairs(rng, dim))
        frames, gh, gw = rng.randint(1, 21), _spread(rng, 1, 48), _spread(rng, 2, 80)
        room = max(1, 96_000_000 // (frames * gh * gw * dim))
        batch = rng.randint(1, min(3, room))
        return _rotary(batch=batch, heads=rng.randint(1, max(1, min(12, room // batch))), frames=frames, grid_h=gh,
                       grid_w=gw, dim=dim, dtype=dtype, interleaved=rng.random() < 0.5, inverse=rng.random() < 0.5,
                       ordered=rng.random() < 0.6, token_major=rng.random() < 0.5, **_draw_pairs(rng, dim))
    if kind in ("fwd", "bwd"):
        kv_heads, share = rng.randint(1, 4), rng.choice([1, 1, 2, 3, 4, 8])
        batch = rng.randint(1, 3)
        room = 600_000_000 // (batch * kv_heads * share)
        # a row that sees one key has a gradient of zero, which rounding alone then fills: training lengths are longer
        k_tokens = _spread(rng, 1 if kind == "fwd" else 64, min(16001, room))
        q_tokens = k_tokens if rng.random() < 0.6 else _spread(rng, 1, min(16001, room // k_tokens))
        q_tokens = min(q_tokens, max(1, room // k_tokens), 16001 if kind == "fwd" else k_tokens)
        block = 1 if rng.random() < 0.6 else _spread(rng, 2, 1000)
        blocks = k_tokens // block + 1
        return _attn(op=kind, batch=batch, q_heads=kv_heads * share, kv_heads=kv_heads, q_tokens=q_tokens,
                     k_tokens=k_tokens, dim=dim, dtype=dtype, causal=rng.random() < 0.75,
                     window=-1 if rng.random() < 0.35 else _spread(rng, 1, blocks), block=block,
                     sinks=0 if rng.random() < 0.4 else _spread(rng, 1, max(1, k_tokens // 4)),
                     ragged=rng.random() < 0.4, token_major=rng.random() < 0.5)
    page = rng.choice([16, 32, 48, 64, 128, 256])
    if kind == "append":
        new = _spread(rng, 1, 12480)
        batch = _spread(rng, 1, max(1, min(128, 24960 // new)))
        return _append(batch=batch, kv_heads=rng.randint(1, 10), new=new,
                       length=min(12480, new + _spread(rng, 1, max(1, min(4000, 200_000 // batch)))), page=page, dim=dim,
                       dtype=dtype, rotate=rng.random() < 0.7, interleaved=rng.random() < 0.5, **_draw_pairs(rng, dim))
    kv_heads, share = rng.randint(1, 10), rng.choice([1, 1, 2, 4, 5, 8, 16])
    length = _spread(rng, 1, 32768)
    batch = _spread(rng, 1, max(1, min(64, 1_000_000 // (kv_heads * length))))
    return _decode(batch=batch, q_heads=kv_heads * share, kv_heads=kv_heads, length=length, page=page, dim=dim,
                   dtype=dtype, window=-1 if rng.random() < 0.5 else _spread(rng, 1, length),
                   sinks=0 if rng.random() < 0.5 else _spread(rng, 1, 256),
                   block=1 if rng.random() < 0.8 else rng.randint(2, 300))


# ------------------------------------------------------------------------------ inputs


def _lengths(c, n, salt):
    """Sequence lengths of a batch: all n, or (ragged) from n down to about half of it, the first one full."""
    if not c["ragged"]:
        return [n] * c["batch"]
    return [n - (b * (7919 + salt)) % (n // 2 + 1) for b in range(c["batch"])]


def _table(c):
    """cos and sin of the three axes' angles, [frames*pf + grid_h*ph + grid_w*pw, 2], the way a program keeps them."""
    rows = []
    for n, pairs in ((c["frames"], c["pf"]), (c["grid_h"], c["ph"]), (c["grid_w"], c["pw"])):
        freq = 10000.0 ** (-torch.arange(pairs, device=DEV, dtype=torch.float64) / pairs)
        rows.append((torch.arange(n, device=DEV, dtype=torch.float64)[:, None] * freq).reshape(-1))
    a = torch.cat(rows)
    return torch.stack([a.cos(), a.sin()], 1).float()


def _randn(g, *shape, dtype, token_major=False):
    """[batch, heads, tokens, dim] values; token_major: the same as a view of [batch, tokens, heads, dim]."""
    if token_major:
        b, h, t, d = shape
        return torch.randn(b, t, h, d, generator=g, device=DEV, dtype=torch.float32).to(dtype).transpose(1, 2)
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _orders(c):
    """Half the heads frame-major, half anchor-first temporal-major, as the video workloads have them."""
    return [0 if h < (c["heads"] + 1) // 2 else 1 for h in range(c["heads"])]


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt = TYPES[c["dtype"]]
    s = dict(case=c)
    if c["op"] == "rotary":
        whole = c["frames"] * c["grid_h"] * c["grid_w"]
        t = c["tokens"] or whole
        s["x"] = _randn(g, c["batch"], c["heads"], t, c["dim"], dtype=dt, token_major=c["token_major"])
        s["table"] = _table(c)
        s["positions"] = None
        if c["tokens"]:
            first = torch.randint(0, whole - t + 1, (c["batch"], 1), generator=g, device=DEV)
            s["positions"] = (first + torch.arange(t, device=DEV)).int()
        s["y"] = torch.empty(c["batch"], c["heads"], t, c["dim"], dtype=dt, device=DEV)
    elif c["op"] in ("fwd", "bwd"):
        tm = c["token_major"]
        s["q"] = _randn(g, c["batch"], c["q_heads"], c["q_tokens"], c["dim"], dtype=dt, token_major=tm)
        s["k"] = _randn(g, c["batch"], c["kv_heads"], c["k_tokens"], c["dim"], dtype=dt, token_major=tm)
        s["v"] = _randn(g, c["batch"], c["kv_heads"], c["k_tokens"], c["dim"], dtype=dt, token_major=tm)
        s["o"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(c["batch"], c["q_heads"], c["q_tokens"], device=DEV)
        s["q_lens"] = s["k_lens"] = None
        if c["ragged"]:
            s["q_lens"] = torch.tensor(_lengths(c, c["q_tokens"], 0), dtype=torch.int32, device=DEV)
            s["k_lens"] = torch.tensor(_lengths(c, c["k_tokens"], 1), dtype=torch.int32, device=DEV)
        if c["op"] == "bwd":
            s["o"], s["lse"] = _attention(s)
            s["do"] = _randn(g, c["batch"], c["q_heads"], c["q_tokens"], c["dim"], dtype=dt, token_major=tm)
            s["dq"], s["dk"], s["dv"] = (torch.zeros_like(s[n]) for n in "qkv")
    else:
        need = -(-c["length"] // c["page"])
        pages = c["batch"] * need + 3
        lens = _lengths(c, c["length"], 1) if c["op"] == "decode" else [c["length"]] * c["batch"]
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["page_table"] = torch.randperm(pages, generator=g, device=DEV)[:c["batch"] * need].int().view(c["batch"], need)
        shape = (pages, c["kv_heads"], c["page"], c["dim"])
        s["k_pages"], s["v_pages"] = _randn(g, *shape, dtype=dt), _randn(g, *shape, dtype=dt)
        if c["op"] == "append":
            shape = (c["batch"], c["kv_heads"], c["new"], c["dim"])
            s["k"], s["v"] = (_randn(g, *shape, dtype=dt, token_major=True) for _ in range(2))
            s["table"] = _table(c) if c["rotate"] else None
        else:
            s["q"] = _randn(g, c["batch"], c["q_heads"], c["dim"], dtype=dt)
            s["o"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(c["batch"], c["q_heads"], device=DEV)
    if own:
        from block_sparse_spatio_attn_b200 import svga  # the program's own plan of its calls
        if c["op"] == "rotary" or (c["op"] == "append" and c["rotate"]):
            s["rotary"] = svga.RotarySpec(c["frames"], c["grid_h"], c["grid_w"], (c["pf"], c["ph"], c["pw"]),
                                          c["interleaved"], _orders(c) if c.get("ordered") else None)
        if c["op"] in ("fwd", "bwd", "decode"):
            s["mask"] = svga.WindowMask(c.get("causal", True), c["window"], c["sinks"], c["block"])
    return s


# ------------------------------------------------------------------------ the plain forms


def _angles(c, table, token):
    """cos and sin [..., pairs] of the tokens' (frame, row, column) places."""
    hw = c["grid_h"] * c["grid_w"]
    f, r, w = token // hw, token % hw // c["grid_w"], token % c["grid_w"]
    a, b = c["frames"] * c["pf"], c["frames"] * c["pf"] + c["grid_h"] * c["ph"]
    tf, th, tw = table[:a].view(-1, c["pf"], 2), table[a:b].view(-1, c["ph"], 2), table[b:].view(-1, c["pw"], 2)
    cs = torch.cat([tf[f], th[r], tw[w]], -2)
    return cs[..., 0], cs[..., 1]


def _turn(x, cos, sin, interleaved, inverse):
    """x [..., dim] in 32 bits with its first 2 * pairs values rotated."""
    n = cos.shape[-1]
    if inverse:
        sin = -sin
    a, rest = x[..., :2 * n], x[..., 2 * n:]
    if interleaved:
        x0, x1 = a[..., 0::2], a[..., 1::2]
        y = torch.stack([x0 * cos - x1 * sin, x1 * cos + x0 * sin], -1).flatten(-2)
    else:
        x0, x1 = a[..., :n], a[..., n:]
        y = torch.cat([x0 * cos - x1 * sin, x1 * cos + x0 * sin], -1)
    return torch.cat([y, rest], -1)


def _token_at(c, device):
    """[heads, tokens]: the frame-major token at each position of a head's order."""
    F, S = c["frames"], c["grid_h"] * c["grid_w"]
    pos = torch.arange(F * S, device=device)
    u = (pos - S).clamp(min=0)
    temporal = torch.where(pos < S, pos, (1 + u % max(1, F - 1)) * S + u // max(1, F - 1))
    return torch.where(torch.tensor(_orders(c), device=device)[:, None] == 1, temporal, pos)


def _rotary_plain(s):
    c, x = s["case"], s["x"]
    if s["positions"] is not None:
        cos, sin = (v[:, None] for v in _angles(c, s["table"], s["positions"].long()))
    else:
        cos, sin = _angles(c, s["table"], torch.arange(x.shape[2], device=x.device))
    if not c["ordered"]:
        return _turn(x.float(), cos, sin, c["interleaved"], c["inverse"]).to(x.dtype)
    at = _token_at(c, x.device)[None, :, :, None].expand(x.shape)
    if c["inverse"]:
        y = torch.empty_like(x, dtype=torch.float32).scatter_(2, at, x.float())
        return _turn(y, cos, sin, c["interleaved"], True).to(x.dtype)
    return _turn(x.float(), cos, sin, c["interleaved"], False).gather(2, at).to(x.dtype)


def _kept(c, q_len, k_len, n_q, n_k, device):
    """[batch, 1, n_q, n_k] truth values of the mask; q_len and k_len: [batch, 1]."""
    p = torch.arange(n_q, device=device) + (k_len - q_len)                   # [batch, n_q]
    bp = torch.div(p, c["block"], rounding_mode="floor")[:, :, None]
    j = torch.arange(n_k, device=device)
    bj = (j // c["block"])[None, None]
    keep = (j < k_len)[:, None, :]
    if c.get("causal", True):
        keep = keep & (bj <= bp)
    if c["window"] >= 0:
        keep = keep & (((bp - bj).abs() <= c["window"]) | (j < c["sinks"]))
    return keep[:, None]


def _lens_of(s):
    c, dev = s["case"], s["q"].device
    if s["q_lens"] is None:
        return (torch.full((c["batch"], 1), c[n], device=dev) for n in ("q_tokens", "k_tokens"))
    return s["q_lens"].long()[:, None], s["k_lens"].long()[:, None]


def _shared(x, q_heads):
    return x.float().repeat_interleave(q_heads // x.shape[1], 1)


def _attention(s):
    """The forward pass: o and lse, rows past a sequence's end as they were."""
    c, q = s["case"], s["q"]
    q_len, k_len = _lens_of(s)
    x = (q.float() / math.sqrt(c["dim"])) @ _shared(s["k"], c["q_heads"]).transpose(2, 3)
    x = x.masked_fill_(~_kept(c, q_len, k_len, c["q_tokens"], c["k_tokens"], q.device), -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p @ _shared(s["v"], c["q_heads"])) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (m + total.log())[..., 0]
    there = (torch.arange(c["q_tokens"], device=q.device) < q_len)[:, None]   # [batch, 1, q_tokens]
    return torch.where(there[..., None], o.to(q.dtype), s["o"]), torch.where(there, lse, s["lse"])


def _attention_backward(s):
    c, q, dt = s["case"], s["q"], s["q"].dtype
    scale = 1 / math.sqrt(c["dim"])
    q_len, k_len = _lens_of(s)
    there = (torch.arange(c["q_tokens"], device=q.device) < q_len)[:, None, :, None]
    keep = _kept(c, q_len, k_len, c["q_tokens"], c["k_tokens"], q.device) & there
    k, v = _shared(s["k"], c["q_heads"]), _shared(s["v"], c["q_heads"])
    lse = torch.where(s["lse"] == -math.inf, torch.zeros_like(s["lse"]), s["lse"])[..., None]
    p = ((q.float() * scale) @ k.transpose(2, 3)).sub_(lse).masked_fill_(~keep, -math.inf).exp_()
    do = s["do"].float()
    by_kv = (c["batch"], c["kv_heads"], c["q_heads"] // c["kv_heads"], c["k_tokens"], c["dim"])
    dv = (p.transpose(2, 3) @ do).view(by_kv).sum(2)
    ds = (do @ v.transpose(2, 3)).sub_((do * s["o"].float()).sum(-1, keepdim=True)).mul_(p)
    dq = (ds @ k) * scale
    dk = (ds.transpose(2, 3) @ q.float()).view(by_kv).sum(2) * scale
    k_there = (torch.arange(c["k_tokens"], device=q.device) < k_len)[:, None, :, None]
    return (torch.where(there, dq.to(dt), s["dq"]), torch.where(k_there, dk.to(dt), s["dk"]),
            torch.where(k_there, dv.to(dt), s["dv"]))


def _append_plain(s):
    c = s["case"]
    p = s["lens"].long()[:, None] - c["new"] + torch.arange(c["new"], device=DEV)
    k = s["k"].float()
    if c["rotate"]:
        cos, sin = (v[:, None] for v in _angles(c, s["table"], p))
        k = _turn(k, cos, sin, c["interleaved"], False)
    page, row = s["page_table"].long().gather(1, p // c["page"]), p % c["page"]
    s["k_pages"][page, :, row] = k.transpose(1, 2).to(s["k"].dtype)
    s["v_pages"][page, :, row] = s["v"].transpose(1, 2)
    return s["k_pages"], s["v_pages"]


def _decode_plain(s):
    c = s["case"]
    share = c["q_heads"] // c["kv_heads"]

    def keys(pages):
        x = pages[s["page_table"].long()]                                   # [batch, pages, heads, page, dim]
        return x.transpose(1, 2).flatten(2, 3)[:, :, :c["length"]].float()

    q = s["q"].float().view(c["batch"], c["kv_heads"], share, c["dim"]) / math.sqrt(c["dim"])
    length = s["lens"].long()[:, None]
    x = q @ keys(s["k_pages"]).transpose(2, 3)
    x = x.masked_fill_(~_kept(c, torch.ones_like(length), length, 1, c["length"], q.device), -math.inf)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p @ keys(s["v_pages"])) / total
    return o.view(c["batch"], c["q_heads"], c["dim"]).to(s["q"].dtype), (m + total.log()).view(c["batch"], -1)


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"rotary": _rotary_plain, "fwd": _attention, "bwd": _attention_backward, "append": _append_plain,
                "decode": _decode_plain}[c["op"]](s)
    from block_sparse_spatio_attn_b200 import svga
    scale = 1 / math.sqrt(c["dim"])
    if c["op"] == "rotary":
        return svga.svga_rotary(s["x"], s["y"], s["rotary"], s["table"], s["positions"], inverse=c["inverse"])
    if c["op"] == "fwd":
        svga.svga_window_attention_fwd(s["q"], s["k"], s["v"], s["o"], s["lse"], s["mask"], scale, s["q_lens"],
                                       s["k_lens"])
        return s["o"], s["lse"]
    if c["op"] == "bwd":
        return svga.svga_window_attention_bwd(s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], s["dq"], s["dk"],
                                              s["dv"], s["mask"], scale, s["q_lens"], s["k_lens"])
    if c["op"] == "append":
        svga.svga_cache_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["page_table"], s["lens"],
                               rotary=s.get("rotary"), table=s["table"])
        return s["k_pages"], s["v_pages"]
    svga.svga_cache_decode(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["lens"], s["o"], s["lse"],
                           s["mask"], scale)
    return s["o"], s["lse"]


# ---------------------------------------------------------------------------- the work


def _pairs(c, q_len, k_len):
    """Kept (query, key) pairs of one sequence and the keys that some query sees."""
    pairs, q = 0, torch.arange(q_len, dtype=torch.int64)
    b = torch.div(q + k_len - q_len, c["block"], rounding_mode="floor")
    top = ((b + 1) * c["block"]).clamp(0, k_len) if c.get("causal", True) else torch.full_like(b, k_len)
    if c["window"] < 0:
        return int(top.sum()), int(top.max()) if q_len else 0
    hi = torch.minimum(((b + c["window"] + 1) * c["block"]).clamp(0, k_len), top)
    lo = torch.minimum(((b - c["window"]) * c["block"]).clamp(0, k_len), hi)
    sink = torch.minimum(top.clamp(max=c["sinks"]), lo)                     # sinks below the window
    late = (top.clamp(max=c["sinks"]) - torch.maximum(hi, lo)).clamp(min=0)  # and above it (not causal)
    pairs = int((hi - lo + sink + late).sum())
    if not q_len:
        return 0, 0
    seen = int(torch.maximum(hi.max(), torch.minimum(top.max(), torch.tensor(c["sinks"])))) - max(0, int(lo.min()) - c["sinks"])
    return pairs, max(0, seen)


def work(case):
    c = case
    e = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "rotary":
        t = c["tokens"] or c["frames"] * c["grid_h"] * c["grid_w"]
        n = c["batch"] * c["heads"] * t
        return {"bytes": 2 * n * c["dim"] * e, "flops": 6 * n * (c["pf"] + c["ph"] + c["pw"])}
    if c["op"] == "append":
        n = c["batch"] * c["kv_heads"] * c["new"]
        return {"bytes": 4 * n * c["dim"] * e, "flops": 6 * n * (c["pf"] + c["ph"] + c["pw"]) if c["rotate"] else 0}
    if c["op"] == "decode":
        seen = [_pairs(c, 1, n) for n in _lengths(c, c["length"], 1)]
        keys = sum(k for k, _ in seen)
        return {"bytes": 2 * keys * c["kv_heads"] * c["dim"] * e + c["batch"] * c["q_heads"] * (2 * c["dim"] * e + 4),
                "flops": 4 * keys * c["q_heads"] * c["dim"]}
    lens = list(zip(_lengths(c, c["q_tokens"], 0), _lengths(c, c["k_tokens"], 1)))
    seen = [_pairs(c, a, b) for a, b in lens]
    q_rows, k_rows = c["q_heads"] * sum(a for a, _ in lens), c["kv_heads"] * sum(k for _, k in seen)
    pairs = c["q_heads"] * sum(p for p, _ in seen)
    if c["op"] == "fwd":
        return {"bytes": 2 * (q_rows + k_rows) * c["dim"] * e + 4 * q_rows, "flops": 4 * pairs * c["dim"]}
    return {"bytes": 4 * (q_rows + k_rows) * c["dim"] * e + 4 * q_rows, "flops": 10 * pairs * c["dim"]}


# ------------------------------------------------------------- the definitions, in 64 bits


def _exact_turn(c, x, place, inverse):
    """x [tokens, dim] in 64 bits, each token turned by its place's angles as complex numbers."""
    f, r, w = place // (c["grid_h"] * c["grid_w"]), place // c["grid_w"] % c["grid_h"], place % c["grid_w"]
    angle = torch.cat([pos.double()[:, None] * torch.pow(torch.tensor(10000.0, dtype=torch.float64, device=DEV),
                                                         -torch.arange(n, device=DEV).double() / n)
                       for pos, n in ((f, c["pf"]), (r, c["ph"]), (w, c["pw"]))], 1)
    z = torch.polar(torch.ones_like(angle), -angle if inverse else angle)
    n = angle.shape[1]
    i0 = torch.arange(n, device=DEV) * 2 if c["interleaved"] else torch.arange(n, device=DEV)
    i1 = i0 + 1 if c["interleaved"] else i0 + n
    t = torch.complex(x[:, i0], x[:, i1]) * z
    y = x.clone()
    y[:, i0], y[:, i1] = t.real, t.imag
    return y


def _exact_rows(c, q_len, k_len):
    """[q_len, k_len] truth values, straight from the definition."""
    p = torch.arange(q_len, device=DEV)[:, None] + (k_len - q_len)
    j = torch.arange(k_len, device=DEV)[None]
    bp, bj = torch.floor_divide(p, c["block"]), torch.floor_divide(j, c["block"])
    near = torch.ones(q_len, k_len, dtype=torch.bool, device=DEV)
    if c["window"] >= 0:
        near = (bp - bj <= c["window"]) & (bj - bp <= c["window"]) | (j < c["sinks"])
    return near & (bj <= bp) if c.get("causal", True) else near


def _exact_softmax(c, q, k, keep):
    """The kept softmax weights and the log of their sum, in 64 bits; a row that keeps nothing has weights 0."""
    x = torch.where(keep, q @ k.T / math.sqrt(c["dim"]), torch.tensor(-math.inf, dtype=torch.float64, device=DEV))
    lse = torch.logsumexp(x, 1)
    return torch.exp(x - torch.where(lse.isinf(), torch.zeros_like(lse), lse)[:, None]), lse


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "rotary":
        x, out = s["x"], torch.empty(s["x"].shape, dtype=torch.float64, device=DEV)
        whole = torch.arange(x.shape[2], device=DEV)
        F, S = c["frames"], c["grid_h"] * c["grid_w"]
        f, i = whole // S, whole % S
        at = torch.where(f == 0, i, S + i * (F - 1) + f - 1)                # a token's position in a temporal head
        for b in range(c["batch"]):
            place = whole if s["positions"] is None else s["positions"][b].long()
            for h in range(c["heads"]):
                to = at if c["ordered"] and _orders(c)[h] == 1 else whole
                if c["inverse"]:
                    out[b, h] = _exact_turn(c, x[b, h].double()[to], place, True)
                else:
                    out[b, h, to] = _exact_turn(c, x[b, h].double(), place, False)
        return out
    if c["op"] == "append":
        kp, vp = s["k_pages"].double(), s["v_pages"].double()
        for b in range(c["batch"]):
            place = torch.arange(c["length"] - c["new"], c["length"], device=DEV)
            page, row = s["page_table"][b].long()[place // c["page"]], place % c["page"]
            for h in range(c["kv_heads"]):
                k = s["k"][b, h].double()
                kp[page, h, row] = _exact_turn(c, k, place, False) if c["rotate"] else k
                vp[page, h, row] = s["v"][b, h].double()
        return kp, vp
    if c["op"] == "decode":
        o = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
        lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device=DEV)
        share = c["q_heads"] // c["kv_heads"]
        for b, n in enumerate(_lengths(c, c["length"], 1)):
            at = torch.arange(n, device=DEV)
            page, row = s["page_table"][b].long()[at // c["page"]], at % c["page"]
            keep = _exact_rows(c, 1, n)
            for h in range(c["kv_heads"]):
                mine = slice(h * share, (h + 1) * share)
                p, z = _exact_softmax(c, s["q"][b, mine].double(), s["k_pages"][page, h, row].double(), keep)
                o[b, mine], lse[b, mine] = p @ s["v_pages"][page, h, row].double(), z
        return o, lse
    names = ("o", "lse") if c["op"] == "fwd" else ("dq", "dk", "dv")
    out = {n: torch.zeros(s[n].shape, dtype=torch.float64, device=DEV) for n in names}
    share, scale = c["q_heads"] // c["kv_heads"], 1 / math.sqrt(c["dim"])
    for b, (nq, nk) in enumerate(zip(_lengths(c, c["q_tokens"], 0), _lengths(c, c["k_tokens"], 1))):
        keep = _exact_rows(c, nq, nk)
        for h in range(c["q_heads"]):
            g = h // share
            q, k, v = s["q"][b, h, :nq].double(), s["k"][b, g, :nk].double(), s["v"][b, g, :nk].double()
            p, z = _exact_softmax(c, q, k, keep)
            if c["op"] == "fwd":
                out["o"][b, h, :nq], out["lse"][b, h, :nq] = p @ v, z
                continue
            do = s["do"][b, h, :nq].double()
            out["dv"][b, g, :nk] += p.T @ do
            dp = do @ v.T
            ds = p * (dp - (p * dp).sum(1, keepdim=True)) * scale
            out["dq"][b, h, :nq] = ds @ k
            out["dk"][b, g, :nk] += ds.T @ q
    return tuple(out[n] for n in names)
