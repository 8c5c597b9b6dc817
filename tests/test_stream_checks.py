"""Refusals of the streaming attention calls, on the host: the C entry points with bad
arguments (any pointer will do, nothing is launched) and the binding's own checks."""
import ctypes

import pytest
import torch

from block_sparse_spatio_attn_b200 import svga

OK, ARG, SHAPE, ALIGN, UNSUP, WORK = 0, 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def lib():
    from block_sparse_spatio_attn_b200 import build
    build.build()
    return svga.load()


def refused(rc, status, words, lib):
    assert rc == status, (rc, lib.svga_last_error())
    assert words in lib.svga_last_error().decode(), lib.svga_last_error()


A, Z = 1 << 20, 1 << 30  # addresses that are never touched


def view(data=A, sb=6400, sh=640, st=64):
    return svga.View(data, sb, sh, st)


def rotary(lib, src=None, dst=None, shape=(2, 10, 10, 64), dtype=0, spec=None, table=A, positions=None, first=0,
           inverse=0, status=None):
    spec = svga.RotarySpec(10, 2, 5, (10, 11, 11)) if spec is None else spec
    return lib.svga_rotary(ctypes.byref(src or view()), ctypes.byref(dst or view(Z)), *shape, dtype,
                           ctypes.byref(spec.c), table, positions, first, inverse, status, None)


@pytest.mark.parametrize("kw,status,words", [
    (dict(dtype=3), UNSUP, "dtype"), (dict(shape=(2, 10, 10, 96)), UNSUP, "head_dim"),
    (dict(shape=(-1, 10, 10, 64)), SHAPE, "batch"), (dict(shape=(2, 0, 10, 64)), SHAPE, "heads"),
    (dict(shape=(2, 10, (1 << 24) + 1, 64)), SHAPE, "tokens"),
    (dict(src=view(0)), ARG, "src has no data"), (dict(src=view(A + 8)), ALIGN, "src is not 16-byte"),
    (dict(dst=view(Z, st=68)), ALIGN, "dst: stride of 68"), (dict(src=view(st=-64)), SHAPE, "src: stride -64"),
    (dict(src=view(st=56)), SHAPE, "below the 64 values"), (dict(dst=view(Z, sh=0)), ARG, "rows overlap"),
    (dict(dst=view(Z, sb=6392)), ARG, "rows overlap"),
    (dict(spec=svga.RotarySpec(10, 2, 5, (20, 11, 11))), SHAPE, "42 pairs do not fit"),
    (dict(spec=svga.RotarySpec(10, 2, 5, (-1, 11, 11))), SHAPE, "pairs[0]"),
    (dict(spec=svga.RotarySpec(0, 2, 5, (1, 1, 1))), SHAPE, "grid of 0 frames"),
    (dict(table=None), ARG, "table is NULL"), (dict(table=A + 4), ALIGN, "table is not"),
    (dict(first=91), SHAPE, "pass the grid"), (dict(first=-1), SHAPE, "pass the grid"),
    (dict(inverse=2), ARG, "inverse"), (dict(positions=A + 2), ALIGN, "positions"),
    (dict(dst=view(A + 64)), ARG, "overlap"), (dict(dst=view(A, sb=12800)), ARG, "overlap"),
    (dict(spec=svga.RotarySpec(10, 2, 5, (1, 1, 1), order=[0] * 10)), ARG, "every token"),
    (dict(spec=svga.RotarySpec(5, 1, 2, (1, 1, 1), order=[0] * 9 + [3])), ARG, "order 3"),
    (dict(spec=svga.RotarySpec(5, 1, 2, (1, 1, 1), order=[0] * 10), dst=view(A)), ARG, "overlap"),
])
def test_rotary_refusals(lib, kw, status, words):
    refused(rotary(lib, **kw), status, words, lib)


def test_rotary_table_refusals(lib):
    spec = svga.RotarySpec(10, 2, 5, (10, 11, 11))
    for theta in (1.0, 0.0, float("nan"), 1e19):
        refused(lib.svga_rotary_table(ctypes.byref(spec.c), theta, A, None), ARG, "theta", lib)
    assert svga.svga_rotary_table_size(spec) == 8 * (100 + 22 + 55)
    big = svga.RotarySpec(1 << 30, 1, 1, (64, 0, 0))
    refused(lib.svga_rotary_table_size(ctypes.byref(big.c), None), SHAPE, "table of", lib)


def cache(**kw):
    d = dict(k_pages=A, v_pages=A, pages=4, kv_heads=2, page_size=16, head_dim=64, dtype=0, batch=2, max_pages=2,
             page_table=A, lens=A, status=None)
    d.update(kw)
    return svga.PagedCacheC(*d.values())


BAD_CACHES = [
    (dict(page_size=8), UNSUP, "page_size"), (dict(page_size=24), UNSUP, "page_size"),
    (dict(page_size=2048), UNSUP, "page_size"), (dict(head_dim=32), UNSUP, "head_dim"),
    (dict(dtype=2), UNSUP, "dtype"), (dict(pages=-1), SHAPE, "out of range"),
    (dict(pages=1 << 27), SHAPE, "out of range"), (dict(max_pages=1 << 21), SHAPE, "out of range"),
    (dict(kv_heads=0), SHAPE, "out of range"), (dict(batch=65536), SHAPE, "out of range"),
    (dict(lens=None), ARG, "must be given"), (dict(page_table=None), ARG, "must be given"),
    (dict(k_pages=None), ARG, "must be given"), (dict(v_pages=A + 8), ALIGN, "16-byte"),
    (dict(lens=A + 2), ALIGN, "lens"), (dict(status=A + 1), ALIGN, "status"),
]


@pytest.mark.parametrize("kw,status,words", BAD_CACHES)
def test_cache_refusals(lib, kw, status, words):
    c, m = cache(**kw), svga.WindowMask()
    v = view()
    refused(lib.svga_cache_append(ctypes.byref(v), ctypes.byref(v), 3, None, ctypes.byref(c), None, None, None),
            status, words, lib)
    refused(lib.svga_cache_decode(ctypes.byref(v), ctypes.byref(v), None, 4, ctypes.byref(c), ctypes.byref(m.c), 0.1,
                                  None), status, words, lib)


def test_append_refusals(lib):
    def call(k=None, v=None, tokens=3, new=None, spec=None, table=None):
        return lib.svga_cache_append(ctypes.byref(k or view()), ctypes.byref(v or view()), tokens, new,
                                     ctypes.byref(cache()), None if spec is None else ctypes.byref(spec.c), table,
                                     None)
    refused(call(tokens=-1), SHAPE, "tokens", lib)
    refused(call(k=view(A + 4)), ALIGN, "k is not", lib)
    refused(call(v=view(0)), ARG, "v has no data", lib)
    refused(call(new=A + 1), ALIGN, "new_lens", lib)
    refused(call(table=A), ARG, "without a spec", lib)
    refused(call(spec=svga.RotarySpec(2, 2, 2, (1, 1, 1))), ARG, "table is NULL", lib)
    refused(call(spec=svga.RotarySpec(2, 2, 2, (1, 1, 1), order=[0, 0]), table=A), ARG, "order", lib)
    assert call(tokens=0) == OK


@pytest.mark.parametrize("mask,words", [
    (svga.WindowMask(window=-2), "window -2"), (svga.WindowMask(sinks=-1), "sinks -1"),
    (svga.WindowMask(block=0), "block 0"), (svga.WindowMask(block=(1 << 24) + 1), "block"),
    (svga.WindowMask(causal=2), "causal")])
def test_decode_refusals(lib, mask, words):
    def call(q=None, o=None, heads=4, m=svga.WindowMask(), scale=0.1, lse=None):
        return lib.svga_cache_decode(ctypes.byref(q or view()), ctypes.byref(o or view()), lse, heads,
                                     ctypes.byref(cache()), ctypes.byref(m.c), scale, None)
    refused(call(m=mask), ARG, words, lib)
    refused(call(heads=3), SHAPE, "multiple of kv_heads", lib)
    refused(call(scale=0.0), ARG, "scale", lib)
    refused(call(scale=float("nan")), ARG, "scale", lib)
    refused(call(q=view(A, sh=4)), ALIGN, "q: stride", lib)
    refused(call(o=view(A, sh=32)), ARG, "rows overlap", lib)
    refused(call(lse=A + 2), ALIGN, "lse", lib)


def rejected(fn, status, words):
    with pytest.raises(svga.SvgaError) as e:
        fn()
    assert e.value.status == status and words in str(e.value), str(e.value)


def test_specs_and_masks_cannot_fall_behind_their_fields():
    import dataclasses
    for x, name in ((svga.RotarySpec(1, 2, 5, (10, 11, 11)), "num_frames"), (svga.WindowMask(), "window")):
        with pytest.raises(dataclasses.FrozenInstanceError):
            setattr(x, name, 3)
    assert dataclasses.replace(svga.WindowMask(sinks=2), window=5).c.window == 5
    rejected(lambda: svga.RotarySpec(1, 2, 5, (10, 11)), 2, "2 axes")


def test_binding_checks():
    spec = svga.RotarySpec(1, 2, 5, (10, 11, 11))
    x, t = torch.zeros(1, 2, 10, 64, dtype=torch.bfloat16), torch.zeros(spec.table_shape)
    rejected(lambda: svga.svga_rotary(x[0], x, spec, t), 2, "src must be a tensor of 4")
    rejected(lambda: svga.svga_rotary(x.double(), x, spec, t), 1, "src must be bf16")
    rejected(lambda: svga.svga_rotary(x, x.half(), spec, t), 1, "dst must be")
    rejected(lambda: svga.svga_rotary(x, x[:, :1], spec, t), 2, "dst has shape")
    rejected(lambda: svga.svga_rotary(x, x, spec, t[1:]), 2, "table has shape")
    rejected(lambda: svga.svga_rotary(x, x, spec, t, torch.zeros(1, 10)), 1, "positions must be")
    rejected(lambda: svga.svga_rotary(x.transpose(2, 3), x, spec, t), 1, "src: the values of a row")
    y = torch.zeros(1, 2, 64, 10, dtype=torch.bfloat16).transpose(2, 3)
    rejected(lambda: svga.svga_rotary(x, y, spec, t), 1, "values of a row")
    rejected(lambda: svga.svga_rotary(x, x, spec, t), 1, "CUDA device")
    od = svga.RotarySpec(1, 2, 5, (10, 11, 11), order=[0])
    rejected(lambda: svga.svga_rotary(x, x, od, t), 2, "order names 1 heads")
    pages, table = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(1, 2, dtype=torch.int32)
    lens, q = torch.zeros(1, dtype=torch.int32), torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    m = svga.WindowMask()
    rejected(lambda: svga.svga_cache_decode(q, pages, pages, table, lens, q, None, m, 0.1), 1, "CUDA device")
    rejected(lambda: svga.svga_cache_decode(q.half(), pages, pages, table, lens, q, None, m, 0.1), 1, "q must be")
    rejected(lambda: svga.svga_cache_decode(q, pages, pages[:3], table, lens, q, None, m, 0.1), 2, "v_pages has shape")
    rejected(lambda: svga.svga_cache_decode(q, pages, pages, table[0], lens, q, None, m, 0.1), 2, "page_table")
    rejected(lambda: svga.svga_cache_decode(q, pages, pages, table, lens.long(), q, None, m, 0.1), 1, "lens must be")
    rejected(lambda: svga.svga_cache_append(x[:, :, :3], x, pages, pages, table, lens), 2, "v has shape")
    rejected(lambda: svga.svga_cache_append(x[:, :1], x, pages, pages, table, lens), 2, "k has shape")
    rejected(lambda: svga.svga_cache_append(x, x, pages, pages, table, lens, table=t), 1, "without a RotarySpec")


def problem(**kw):
    d = dict(batch=2, q_heads=4, kv_heads=2, q_tokens=300, k_tokens=300, head_dim=64, dtype=0,
             mask=svga.WindowMask().c, q_lens=None, k_lens=None, status=None)
    d.update(kw)
    return svga.WindowProblemC(*d.values())


def window_calls(lib, p, scale=0.1, ws=A, n=1 << 40, lse=A, **views):
    """Both passes with each view good unless given."""
    def v(name, heads, tokens):
        return ctypes.byref(views.get(name) or view(A, heads * tokens * 64, tokens * 64, 64))
    q = {x: v(x, 4, 300) for x in ("d_o", "q", "o", "dq")}
    k = {x: v(x, 2, 300) for x in ("k", "v", "dk", "dv")}
    fwd = lambda: lib.svga_window_attention_fwd(q["q"], k["k"], k["v"], q["o"], lse, ctypes.byref(p), scale, ws, n, None)  # noqa: E731
    bwd = lambda: lib.svga_window_attention_bwd(q["d_o"], q["q"], k["k"], k["v"], q["o"], lse, q["dq"], k["dk"], k["dv"],  # noqa: E731
                                                ctypes.byref(p), scale, ws, n, None)
    return fwd, bwd


@pytest.mark.parametrize("kw,status,words", [
    (dict(batch=-1), SHAPE, "batch -1"), (dict(batch=65536), SHAPE, "batch"), (dict(q_heads=5), SHAPE, "kv_heads 2"),
    (dict(kv_heads=0), SHAPE, "kv_heads 0"), (dict(q_tokens=-1), SHAPE, "q_tokens -1"),
    (dict(k_tokens=(1 << 24) + 1), SHAPE, "k_tokens"), (dict(head_dim=256), UNSUP, "head_dim"),
    (dict(dtype=2), UNSUP, "dtype"), (dict(q_lens=A + 2), ALIGN, "q_lens"), (dict(k_lens=A + 1), ALIGN, "k_lens"),
    (dict(status=A + 2), ALIGN, "status"), (dict(mask=svga.WindowMask(window=-2).c), ARG, "window -2"),
    (dict(batch=60000, q_heads=4096, kv_heads=1), SHAPE, "do not fit one launch")])
def test_window_problem_refusals(lib, kw, status, words):
    p = problem(**kw)
    for call in window_calls(lib, p):
        refused(call(), status, words, lib)
    refused(lib.svga_window_attention_size(ctypes.byref(p), None, None), status, words, lib)


@pytest.mark.parametrize("name", ["d_o", "q", "k", "v", "o", "dq", "dk", "dv"])
def test_window_view_refusals(lib, name):
    fwd_too = name in ("q", "k", "v", "o")
    for bad, status, words in ((view(0), ARG, "has no data"), (view(A + 8), ALIGN, "16-byte"),
                               (view(A, 38400, 19200, 68), ALIGN, "stride of 68"),
                               (view(A, 38400, 19200, 56), SHAPE, "below the 64 values"),
                               (view(A, 38400, 19200, 0), SHAPE, "below the 64 values"),
                               (view(A, -64, 19200, 64), SHAPE, "stride -64")):
        fwd, bwd = window_calls(lib, problem(), **{name: bad})
        refused(bwd(), status, f"{name}", lib)
        refused(bwd(), status, words, lib)
        if fwd_too:
            refused(fwd(), status, words, lib)
    fwd, bwd = window_calls(lib, problem(), **{name: view(A, 38400, 0, 64)})  # one head for all
    if name in ("dq", "dk", "dv"):
        refused(bwd(), ARG, "rows overlap", lib)
    if name == "o":
        refused(fwd(), ARG, "rows overlap", lib)


def test_window_scale_lse_and_workspace_refusals(lib):
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        for call in window_calls(lib, problem(), scale=scale):
            refused(call(), ARG, "scale", lib)
    for call in window_calls(lib, problem(), lse=A + 2):
        refused(call(), ALIGN, "lse", lib)
    refused(window_calls(lib, problem(), lse=None)[1](), ARG, "lse is NULL", lib)
    n = [ctypes.c_size_t() for _ in range(2)]
    p = problem(k_tokens=100_000, batch=1, q_tokens=300)
    assert lib.svga_window_attention_size(ctypes.byref(p), *map(ctypes.byref, n)) == OK
    fwd, bwd = n[0].value, n[1].value
    assert fwd > 0 and bwd > 0
    long = {x: view(A, 1 << 30, 100_000 * 64, 64) for x in ("k", "v", "dk", "dv")}
    for have, ws in ((fwd - 1, A), (fwd, None), (fwd, A + 128)):
        refused(window_calls(lib, p, ws=ws, n=have, **long)[0](), WORK, "workspace", lib)
    for have, ws in ((bwd - 1, A), (bwd, None), (bwd, A + 128)):
        refused(window_calls(lib, p, ws=ws, n=have, **long)[1](), WORK, "workspace", lib)
    # an output that starts where an input does
    good = {x: view(A + i * (1 << 24), 300 * 64 * (4 if x in ("d_o", "q", "o", "dq") else 2), 300 * 64, 64)
            for i, x in enumerate(("d_o", "q", "k", "v", "o", "dq", "dk", "dv"))}
    for name in ("q", "k", "v"):
        same = svga.View(good[name].data, good["o"].stride_batch, good["o"].stride_head, 64)
        fwd = window_calls(lib, problem(), **{**good, "o": same})[0]
        refused(fwd(), ARG, "o starts where", lib)
    for name in ("dq", "dk", "dv"):
        for other in ("d_o", "q", "k", "v", "o"):
            same = svga.View(good[other].data, good[name].stride_batch, good[name].stride_head, 64)
            refused(window_calls(lib, problem(), **{**good, name: same})[1](), ARG, f"{name} starts where {other}", lib)
    # nothing to do: accepted without a launch, pointers not looked at
    empty = problem(batch=0)
    for call in window_calls(lib, empty, ws=None, n=0, lse=None):
        assert call() == OK, lib.svga_last_error()


def test_window_binding_checks():
    q, k = torch.zeros(1, 4, 10, 64, dtype=torch.bfloat16), torch.zeros(1, 2, 10, 64, dtype=torch.bfloat16)
    lse, m = torch.zeros(1, 4, 10), svga.WindowMask()
    fwd, bwd = svga.svga_window_attention_fwd, svga.svga_window_attention_bwd
    rejected(lambda: fwd(q[0], k, k, q, lse, m, 0.1), 2, "q must be a tensor of 4")
    rejected(lambda: fwd(q.float(), k, k, q, lse, m, 0.1), 1, "q must be bf16 or fp16")
    rejected(lambda: fwd(q, k.half(), k, q, lse, m, 0.1), 1, "k must be torch.bfloat16")
    rejected(lambda: fwd(q, k, k[:, :1], q, lse, m, 0.1), 2, "v has shape")
    rejected(lambda: fwd(q, k, k, q[:, :2], lse, m, 0.1), 2, "o has shape")
    rejected(lambda: fwd(q, k, k, q, lse[:, :2], m, 0.1), 2, "lse has shape")
    rejected(lambda: fwd(q, k, k, q, lse, m, 0.1, torch.zeros(2, dtype=torch.int32)), 2, "q_lens has shape")
    rejected(lambda: fwd(q, k, k, q, lse, m, 0.1, None, torch.zeros(1)), 1, "k_lens must be")
    rejected(lambda: fwd(q, k, k, q, None, m, 0.1), 1, "CUDA device")
    rejected(lambda: bwd(q, q, k, k, q, None, q, k, k, m, 0.1), 1, "lse must be a torch.Tensor")
    rejected(lambda: bwd(q, q, k, k, q, lse, q, k, k[:, :1], m, 0.1), 2, "dv has shape")
    rejected(lambda: bwd(q, q, k, k, q, lse, k, k, k, m, 0.1), 2, "dq has shape")
    rejected(lambda: bwd(q, q, k, k, q, lse, q, k, k, m, 0.1), 1, "CUDA device")


def test_outputs_that_start_together_are_refused(lib):
    good = {x: view(A + i * (1 << 24), 300 * 64 * (4 if x in ("d_o", "q", "o", "dq") else 2), 300 * 64, 64)
            for i, x in enumerate(("d_o", "q", "k", "v", "o", "dq", "dk", "dv"))}
    for name, other in (("dq", "dk"), ("dk", "dv"), ("dq", "dv")):
        both = {**good, other: svga.View(good[name].data, good[other].stride_batch, good[other].stride_head, 64)}
        refused(window_calls(lib, problem(), **both)[1](), ARG, f"{name} starts where {other}", lib)
    c, m = cache(k_pages=Z, v_pages=2 * Z), svga.WindowMask()
    for o in (A, Z, 2 * Z):
        refused(lib.svga_cache_decode(ctypes.byref(view(A)), ctypes.byref(view(o)), None, 4, ctypes.byref(c),
                                      ctypes.byref(m.c), 0.1, None), ARG, "o starts where", lib)


def test_numbers_that_32_bits_cannot_hold_are_refused():
    # ctypes would make 2^32 a window of 0
    for kw in (dict(window=2**32), dict(sinks=2**31), dict(block=2**32 + 1), dict(window=-2**31 - 1)):
        rejected(lambda: svga.WindowMask(**kw), 2, "does not fit 32 bits")
    rejected(lambda: svga.RotarySpec(2**32 + 1, 2, 5, (1, 1, 1)), 2, "does not fit 32 bits")
    rejected(lambda: svga.RotarySpec(1, 2, 5, (1, 2**33, 1)), 2, "does not fit 32 bits")
    rejected(lambda: svga.RotarySpec(1, 2, 5, (1, 1, 1), order=[0, 2**32]), 2, "does not fit 32 bits")


def test_workspace_size_names_its_types():
    q, k = torch.zeros(1, 4, 10, 64), torch.zeros(1, 2, 10, 64)
    rejected(lambda: svga.svga_window_attention_size(q, k, svga.WindowMask()), 4, "dtype")
    n = svga.svga_window_attention_size(q.half(), k.half(), svga.WindowMask())
    assert n["bwd_bytes"] > 0
