"""Attention under a causal window with sinks, forward, against 64 bits: lengths around the
128-row tiles, masks that leave rows empty, shared heads, strides, padded batches, split key
lists."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from block_sparse_spatio_attn_b200 import svga  # noqa: E402
from tests.stream_reference import attention, within  # noqa: E402

BF, FP = torch.bfloat16, torch.float16
M = svga.WindowMask


def values(*shape, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype)


def forward(q, k, v, mask, scale, q_lens=None, k_lens=None, **kw):
    """CPU tensors in; o and lse back, both 9 where nothing was written."""
    o = torch.full(q.shape, 9.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:3], 9.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = [None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")
            for x in (q_lens, k_lens)]
    svga.svga_window_attention_fwd(q.cuda(), k.cuda(), v.cuda(), o, lse, mask, scale, *lens,
                                   status=status, **kw)
    assert status.item() == 0
    return o.cpu(), lse.cpu()


def check(q, k, v, mask, scale, o, lse, q_lens=None, k_lens=None):
    B, H = q.shape[:2]
    share = H // k.shape[1]
    for b in range(B):
        nq = q.shape[2] if q_lens is None else q_lens[b]
        nk = k.shape[2] if k_lens is None else k_lens[b]
        for h in range(H):
            want, z, tol, z_tol = attention(q[b, h, :nq], k[b, h // share, :nk],
                                            v[b, h // share, :nk], mask, scale)
            what = f"batch {b} head {h}, {nq} queries, {nk} keys, {mask}"
            within(o[b, h, :nq], want, tol, "o, " + what)
            within(lse[b, h, :nq], z, z_tol, "lse, " + what)
            assert (o[b, h, nq:] == 9).all() and (lse[b, h, nq:] == 9).all(), what


MASKS = [M(), M(causal=False), M(window=0), M(window=1), M(window=100), M(window=130, sinks=5),
         M(window=40, sinks=300), M(window=1, block=96), M(window=0, block=200, sinks=200),
         M(causal=False, window=70, sinks=10), M(causal=False, window=2, block=33, sinks=33),
         M(causal=True, window=1 << 24, sinks=1 << 24, block=1 << 24)]


@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (FP, 64), (FP, 128)])
@pytest.mark.parametrize("mask", MASKS, ids=str)
def test_masks(mask, dtype, d):
    q, k, v = (values(1, 2, 530, d, dtype=dtype, seed=s) for s in (1, 2, 3))
    scale = 1 / math.sqrt(d)
    check(q, k, v, mask, scale, *forward(q, k, v, mask, scale))


@pytest.mark.parametrize("nq,nk", [(1, 1), (1, 2), (2, 1), (1, 127), (1, 128), (1, 129), (127, 1),
                                   (128, 128), (129, 129), (255, 257), (256, 256), (257, 256),
                                   (300, 100), (100, 300), (5, 1000), (1000, 5), (640, 640)])
def test_lengths(nq, nk):
    for mask in (M(), M(window=30, sinks=3), M(causal=False, window=1, block=50)):
        q = values(1, 2, nq, 64, dtype=BF, seed=nq)
        k, v = (values(1, 1, nk, 64, dtype=BF, seed=nk + s) for s in (1, 2))
        check(q, k, v, mask, 0.125, *forward(q, k, v, mask, 0.125))


def test_no_keys_and_no_queries():
    q, e = values(2, 2, 130, 128, dtype=BF), torch.empty(2, 1, 0, 128, dtype=BF)
    o, lse = forward(q, e, e, M(), 0.1)
    assert (o == 0).all() and (lse == -math.inf).all()
    k = values(2, 1, 50, 128, dtype=BF)
    o, lse = forward(q[:, :, :0], k, k, M(), 0.1)
    assert o.numel() == 0
    forward(q[:0], k[:0], k[:0], M(), 0.1)


@pytest.mark.parametrize("share", [1, 2, 5, 8])
def test_shared_heads_and_strides(share):
    """q, k, v as views of one [batch, tokens, heads, d] projection, o into another."""
    B, T, G, d = 2, 300, 2, 64
    H = G * share
    qkv = values(B, T, H + 2 * G, d, dtype=FP, seed=share)
    q, k, v = (x.transpose(1, 2) for x in qkv.split([H, G, G], 2))
    dev = qkv.cuda()
    dq, dk, dv = (x.transpose(1, 2) for x in dev.split([H, G, G], 2))
    wide = torch.full((B, T, H + 1, d), 9.0, dtype=FP, device="cuda")
    o, lse = wide[:, :, :H].transpose(1, 2), torch.empty(B, H, T, device="cuda")
    mask = M(window=64, sinks=2)
    svga.svga_window_attention_fwd(dq, dk, dv, o, lse, mask, 0.125)
    check(q, k, v, mask, 0.125, o.cpu(), lse.cpu())
    assert (wide[:, :, H] == 9).all()


def test_broadcast_inputs():
    q = values(1, 1, 140, 64, dtype=BF).expand(3, 4, 140, 64)
    k = values(3, 1, 140, 64, dtype=BF, seed=1).expand(3, 2, 140, 64)
    v = values(1, 2, 140, 64, dtype=BF, seed=2).expand(3, 2, 140, 64)
    o, lse = torch.empty(3, 4, 140, 64, dtype=BF, device="cuda"), torch.empty(3, 4, 140, device="cuda")
    dq = q[:1, :1].cuda().expand(3, 4, 140, 64)
    dk = k[:, :1].cuda().expand(3, 2, 140, 64)
    dv = v[:1].cuda().expand(3, 2, 140, 64)
    svga.svga_window_attention_fwd(dq, dk, dv, o, lse, M(), 0.125)
    check(q, k, v, M(), 0.125, o.cpu(), lse.cpu())


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("d", [64, 128])
def test_padded_batch_with_garbage_past_the_lengths(dtype, d):
    """Rows past a sequence's lengths hold NaN and infinities: they change nothing, and the
    rows of o and lse there stay as they were."""
    q_lens, k_lens = [300, 0, 1, 129, 257, 300, 40], [300, 100, 200, 129, 0, 131, 255]
    q = values(7, 4, 300, d, dtype=dtype)
    k, v = (values(7, 2, 300, d, dtype=dtype, seed=s) for s in (1, 2))
    for b in range(7):
        q[b, :, q_lens[b]:] = math.nan
        k[b, :, k_lens[b]:] = math.inf
        v[b, :, k_lens[b]:] = math.nan
    for mask in (M(), M(causal=False), M(window=50, sinks=7), M(window=1, block=64, sinks=64)):
        o, lse = forward(q, k, v, mask, 0.1, q_lens, k_lens)
        check(q, k, v, mask, 0.1, o, lse, q_lens, k_lens)


def test_lengths_are_clamped():
    q, k = values(2, 1, 200, 64, dtype=BF), values(2, 1, 200, 64, dtype=BF, seed=1)
    o, lse = forward(q, k, k, M(), 0.1, [-5, 999], [100, 1 << 30])
    check(q, k, k, M(), 0.1, o, lse, [0, 200], [100, 200])


@pytest.mark.parametrize("B,H,G,nq,nk", [(1, 1, 1, 1, 20_000), (1, 8, 2, 100, 9000),
                                         (2, 4, 4, 300, 5001), (3, 16, 1, 17, 4096),
                                         (1, 74, 1, 3, 3000)])
def test_split_key_lists(B, H, G, nq, nk):
    q = values(B, H, nq, 64, dtype=BF, seed=nq)
    k, v = (values(B, G, nk, 64, dtype=BF, seed=s) for s in (1, 2))
    for mask in (M(), M(window=2500, sinks=500)):
        size = svga.svga_window_attention_size(q, k, mask)["fwd_bytes"]
        q_lens = [nq - b for b in range(B)]
        k_lens = [nk - 700 * b for b in range(B)]
        o, lse = forward(q, k, v, mask, 0.125, q_lens, k_lens)
        check(q, k, v, mask, 0.125, o, lse, q_lens, k_lens)
        assert size > 0
    need = svga.svga_window_attention_size(q, k, M())["fwd_bytes"]
    small = torch.empty(max(need - 1, 0), dtype=torch.uint8, device="cuda")
    with pytest.raises(svga.SvgaError) as e:
        forward(q, k, v, M(), 0.125, workspace=small)
    assert e.value.status == 5


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,G,nq,nk", [(1, 1, 1, 700), (8, 1, 1, 2000), (3, 1, 200, 1000), (1, 1, 256, 4097),
                                       (2, 2, 1500, 1500), (6, 3, 700, 1400), (1, 1, 600, 500), (16, 8, 90, 2100)])
def test_short_launches_split_into_small_parts(H, G, nq, nk, d):
    """Parts of a chunk or two: some have no key for one of a CTA's two query blocks, or for
    either, and padded sequences leave parts empty."""
    q = values(2, H, nq, d, dtype=BF, seed=nq)
    k, v = (values(2, G, nk, d, dtype=BF, seed=s) for s in (1, 2))
    assert svga.svga_window_attention_size(q, k, M())["fwd_bytes"] > 0 or nk <= 512  # (four chunks: whole)
    for mask in (M(), M(window=300, sinks=200), M(causal=False, window=0, block=400)):
        for k_lens in (None, [nk, max(nk // 7, 1)]):
            o, lse = forward(q, k, v, mask, 0.1, None, k_lens)
            check(q, k, v, mask, 0.1, o, lse, None, k_lens)


@pytest.mark.parametrize("mask,dtype,split", [(M(window=1800, sinks=100), BF, True), (M(window=700, sinks=100), BF, False), (M(), FP, False)],
                         ids=str)
def test_launches_split_in_part(mask, dtype, split):
    """160 items for 148 SMs: the last ones split where lists are of one length and long, none where
    they are short or under a causal mask without a window.  Three heads are compared."""
    q = values(1, 10, 4000, 64, dtype=dtype)
    k, v = (values(1, 5, 4000, 64, dtype=dtype, seed=s) for s in (1, 2))
    assert (svga.svga_window_attention_size(q, k, mask)["fwd_bytes"] > 0) == split
    o, lse = forward(q, k, v, mask, 0.125)
    for h in (0, 5, 9):
        g = h // 2
        check(q[:, h:h + 1], k[:, g:g + 1], v[:, g:g + 1], mask, 0.125, o[:, h:h + 1], lse[:, h:h + 1])


def test_scores_far_apart():
    """Scores up to +-2000 whose maximum moves from tile to tile: the reference maximum is
    raised again and again, in both types."""
    for dtype in (BF, FP):
        q, k, v = (values(1, 1, 700, 64, dtype=dtype, seed=s) for s in (1, 2, 3))
        k = k * torch.linspace(0.1, 30, 700)[:, None].to(dtype)
        for mask in (M(), M(window=200, sinks=1)):
            o, lse = forward(q, k, v, mask, 1.0)
            check(q, k, v, mask, 1.0, o, lse)


def test_same_bits_again_captured_and_on_another_stream():
    q, k, v = (values(2, 4, 700, 128, dtype=BF, seed=s).cuda() for s in (1, 2, 3))
    o, lse = torch.empty_like(q), torch.empty(2, 4, 700, device="cuda")
    mask = M(window=300, sinks=4)
    svga.svga_window_attention_fwd(q, k, v, o, lse, mask, 0.09)
    torch.cuda.synchronize()
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    side = torch.cuda.Stream()
    svga.svga_window_attention_fwd(q, k, v, o2, lse2, mask, 0.09, stream=side)
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        svga.svga_window_attention_fwd(q, k, v, o2, lse2, mask, 0.09)
    o2.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_agrees_with_the_spatial_heads_of_the_sparse_kernel():
    """Not causal, block = a frame, sinks = the anchor frame: the mask of a spatial head."""
    from block_sparse_spatio_attn_b200 import configs as C
    wl = C.tiny()
    H, N, S = 2, wl.tokens, wl.tokens_per_frame
    prob = svga.ProblemSpec(H, wl.frames, wl.grid_h, wl.grid_w, 64, [0, 0], [1, 1], [0, 0], 1, 64, 64)
    q, k, v = (values(H, N, 64, dtype=BF, seed=s).cuda() for s in (1, 2, 3))
    o, lse = torch.empty_like(q), torch.empty(H, N, device="cuda")
    svga.svga_sparse_attention_fwd(q, k, v, o, lse, prob, svga.build_block_map(prob), 0.125)
    mask = M(causal=False, window=1, sinks=S, block=S)
    got, got_lse = torch.empty_like(q)[None], torch.empty(1, H, N, device="cuda")
    svga.svga_window_attention_fwd(q[None], k[None], v[None], got, got_lse, mask, 0.125)
    check(q[None].cpu(), k[None].cpu(), v[None].cpu(), mask, 0.125, got.cpu(), got_lse.cpu())
    check(q[None].cpu(), k[None].cpu(), v[None].cpu(), mask, 0.125, o[None].cpu(), lse[None].cpu())
