"""The gradients of windowed attention against the formulas in 64 bits and against differences:
lengths around the tiles, empty rows, shared heads, strides, padded batches."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from block_sparse_spatio_attn_b200 import svga  # noqa: E402
from tests.stream_reference import gradients, kept, rotate, within  # noqa: E402

BF, FP = torch.bfloat16, torch.float16
M = svga.WindowMask


def values(*shape, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype)


def both_passes(q, k, v, do, mask, scale, q_lens=None, k_lens=None, **kw):
    """Device tensors in: o, lse and the gradients, 9 where nothing was written."""
    o = torch.full(q.shape, 9.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:3], 9.0, device="cuda")
    grads = [torch.full(x.shape, 9.0, dtype=q.dtype, device="cuda") for x in (q, k, v)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = [None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")
            for x in (q_lens, k_lens)]
    svga.svga_window_attention_fwd(q, k, v, o, lse, mask, scale, *lens, status=status)
    svga.svga_window_attention_bwd(do, q, k, v, o, lse, *grads, mask, scale, *lens,
                                   status=status, **kw)
    assert status.item() == 0
    return o, lse, grads


def check(q, k, v, do, mask, scale, grads, q_lens=None, k_lens=None):
    dq, dk, dv = (x.cpu() for x in grads)
    B, H = q.shape[:2]
    G = k.shape[1]
    for b in range(B):
        nq = q.shape[2] if q_lens is None else q_lens[b]
        nk = k.shape[2] if k_lens is None else k_lens[b]
        for g in range(G):
            want = [torch.zeros(nk, q.shape[3], dtype=torch.float64) for _ in range(4)]
            for h in range(g * (H // G), (g + 1) * (H // G)):
                w = gradients(q[b, h, :nq], k[b, g, :nk], v[b, g, :nk], do[b, h, :nq], mask, scale)
                what = f"batch {b} head {h}, {nq} queries, {nk} keys, {mask}"
                within(dq[b, h, :nq], w[0], w[3], "dq, " + what)
                assert (dq[b, h, nq:] == 9).all(), what
                for x, y in zip(want, (w[1], w[2], w[4], w[5])):
                    x += y
            within(dk[b, g, :nk], want[0], want[2], f"dk, batch {b} head {g}, {mask}")
            within(dv[b, g, :nk], want[1], want[3], f"dv, batch {b} head {g}, {mask}")
            assert (dk[b, g, nk:] == 9).all() and (dv[b, g, nk:] == 9).all()


def run(q, k, v, do, mask, scale, q_lens=None, k_lens=None):
    _, _, grads = both_passes(q.cuda(), k.cuda(), v.cuda(), do.cuda(), mask, scale, q_lens, k_lens)
    check(q, k, v, do, mask, scale, grads, q_lens, k_lens)
    return grads


MASKS = [M(), M(causal=False), M(window=0), M(window=100), M(window=130, sinks=5),
         M(window=40, sinks=300), M(window=1, block=96), M(window=0, block=200, sinks=200),
         M(causal=False, window=70, sinks=10), M(causal=False, window=2, block=33, sinks=33),
         M(window=1 << 24, sinks=1 << 24, block=1 << 24)]


@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (FP, 64), (FP, 128)])
@pytest.mark.parametrize("mask", MASKS, ids=str)
def test_masks(mask, dtype, d):
    q, k, v, do = (values(1, 2, 530, d, dtype=dtype, seed=s) for s in (1, 2, 3, 4))
    run(q, k, v, do, mask, 1 / math.sqrt(d))


@pytest.mark.parametrize("nq,nk", [(1, 1), (1, 2), (2, 1), (1, 127), (1, 128), (1, 129), (127, 1),
                                   (128, 128), (129, 129), (255, 257), (257, 256), (300, 100),
                                   (100, 300), (5, 1000), (1000, 5), (640, 640)])
def test_lengths(nq, nk):
    for mask in (M(), M(window=30, sinks=3), M(causal=False, window=1, block=50)):
        q, do = (values(1, 2, nq, 64, dtype=BF, seed=nq + s) for s in (0, 9))
        k, v = (values(1, 1, nk, 64, dtype=BF, seed=nk + s) for s in (1, 2))
        run(q, k, v, do, mask, 0.125)


def test_nothing_to_see():
    q, e = values(2, 2, 130, 128, dtype=BF), torch.empty(2, 1, 0, 128, dtype=BF)
    dq, dk, dv = run(q, e, e, q, M(), 0.1)
    assert (dq == 0).all()
    k, e = values(2, 1, 130, 128, dtype=BF), torch.empty(2, 2, 0, 128, dtype=BF)
    dq, dk, dv = run(e, k, k, e, M(), 0.1)
    assert (dk == 0).all() and (dv == 0).all()
    run(e[:0], k[:0], k[:0], e[:0], M(), 0.1)


@pytest.mark.parametrize("share", [1, 2, 5, 8])
def test_shared_heads_and_strides(share):
    B, T, G, d = 2, 300, 2, 64
    H = G * share
    qkv, do = values(B, T, H + 2 * G, d, dtype=FP, seed=share), values(B, T, H, d, dtype=FP)
    q, k, v = (x.transpose(1, 2) for x in qkv.split([H, G, G], 2))
    dev, ddo = qkv.cuda(), do.cuda().transpose(1, 2)
    parts = [x.transpose(1, 2) for x in dev.split([H, G, G], 2)]
    mask = M(window=64, sinks=2)
    o, lse, _ = both_passes(*parts, ddo, mask, 0.125)
    grad = torch.full((B, T, H + 2 * G + 1, d), 9.0, dtype=FP, device="cuda")
    outs = [x.transpose(1, 2) for x in grad[:, :, :-1].split([H, G, G], 2)]
    svga.svga_window_attention_bwd(ddo, *parts, o, lse, *outs, mask, 0.125)
    check(q, k, v, do.transpose(1, 2), mask, 0.125, outs)
    assert (grad[:, :, -1] == 9).all()


def test_broadcast_inputs_and_output_gradient():
    """Heads of k that are one tensor expanded get a gradient each; an expanded dO is read."""
    q = values(2, 4, 200, 64, dtype=BF)
    k, v = (values(2, 1, 200, 64, dtype=BF, seed=s) for s in (1, 2))
    do = values(2, 1, 200, 64, dtype=BF, seed=3)
    dev = [q.cuda(), k.cuda().expand(2, 2, 200, 64), v.cuda().expand(2, 2, 200, 64),
           do.cuda().expand(2, 4, 200, 64)]
    _, _, grads = both_passes(*dev, M(window=90), 0.125)
    check(q, k.expand(2, 2, 200, 64), v.expand(2, 2, 200, 64), do.expand(2, 4, 200, 64),
          M(window=90), 0.125, grads)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("d", [64, 128])
def test_padded_batch_with_garbage_past_the_lengths(dtype, d):
    q_lens, k_lens = [300, 0, 1, 129, 257, 300, 40], [300, 100, 200, 129, 0, 131, 255]
    q, do = (values(7, 4, 300, d, dtype=dtype, seed=s) for s in (0, 5))
    k, v = (values(7, 2, 300, d, dtype=dtype, seed=s) for s in (1, 2))
    for b in range(7):
        q[b, :, q_lens[b]:] = math.nan
        do[b, :, q_lens[b]:] = math.inf
        k[b, :, k_lens[b]:] = math.inf
        v[b, :, k_lens[b]:] = math.nan
    for mask in (M(), M(causal=False), M(window=50, sinks=7), M(window=1, block=64, sinks=64)):
        run(q, k, v, do, mask, 0.1, q_lens, k_lens)


def test_sinks_split_over_ctas():
    """Sink blocks of 60 steps beside others of a few, more items than one round of CTAs, a
    padded batch: the split and joined path with whole items beside it."""
    B, H, G, T = 2, 10, 5, 1500
    q, do = (values(B, H, T, 64, dtype=BF, seed=s) for s in (1, 2))
    k, v = (values(B, G, T, 64, dtype=BF, seed=s) for s in (3, 4))
    mask, q_lens, k_lens = M(window=100, sinks=130), [1500, 1111], [1500, 1300]
    dev = [x.cuda() for x in (q, k, v, do)]
    size = svga.svga_window_attention_size(dev[0], dev[1], mask)["bwd_bytes"]
    assert size > 4 * B * H * 12 * 256  # the rows' statistics and the parts
    _, _, grads = both_passes(*dev, mask, 0.125, q_lens, k_lens)
    for b in range(B):  # one key head of each sequence
        g, pair = 4 * b, slice(8 * b, 8 * b + 2)
        check(q[b:b + 1, pair], k[b:b + 1, g:g + 1], v[b:b + 1, g:g + 1], do[b:b + 1, pair], mask, 0.125,
              [grads[0][b:b + 1, pair], grads[1][b:b + 1, g:g + 1], grads[2][b:b + 1, g:g + 1]],
              q_lens[b:b + 1], k_lens[b:b + 1])


def test_gradients_are_the_differences_of_the_forward_pass():
    """d/dt <o(x + t u), g> at t = 0 in 64 bits, by a central difference of step 2^-12 (its
    error is below 1e-6 of values of order 1), against <gradient, u>."""
    n, d, mask, scale = 150, 64, M(window=60, sinks=4), 0.125
    q, k, v, do = (values(1, 1, n, d, dtype=BF, seed=s) for s in (1, 2, 3, 4))
    _, _, grads = both_passes(q.cuda(), k.cuda(), v.cuda(), do.cuda(), mask, scale)
    bounds = gradients(q[0, 0], k[0, 0], v[0, 0], do[0, 0], mask, scale)[3:]
    step = 2.0 ** -12
    for i, (grad, bound) in enumerate(zip(grads, bounds)):
        u = torch.randn(n, d, generator=torch.Generator().manual_seed(i), dtype=torch.float64)

        def value(t):
            x = [y[0, 0].double() for y in (q, k, v)]
            x[i] = x[i] + t * u
            s = torch.where(kept(mask, n, n), scale * x[0] @ x[1].T, -math.inf)
            return float(((torch.softmax(s, 1) @ x[2]) * do[0, 0].double()).sum())

        want = (value(step) - value(-step)) / (2 * step)
        got = float((grad[0, 0].double().cpu() * u).sum())
        assert abs(got - want) <= float((bound * u.abs()).sum()) + 1e-4


def test_same_bits_again_captured_and_with_a_workspace():
    q, k, v, do = (values(2, 4, 700, 128, dtype=BF, seed=s).cuda() for s in (1, 2, 3, 4))
    mask = M(window=300, sinks=4)
    o, lse, grads = both_passes(q, k, v, do, mask, 0.09)
    n = svga.svga_window_attention_size(q, k, mask)["bwd_bytes"]
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    again = [torch.zeros_like(x) for x in grads]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    svga.svga_window_attention_bwd(do, q, k, v, o, lse, *again, mask, 0.09, workspace=ws, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(grads, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        svga.svga_window_attention_bwd(do, q, k, v, o, lse, *again, mask, 0.09)
    for x in again:
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(grads, again))
    with pytest.raises(svga.SvgaError) as e:
        svga.svga_window_attention_bwd(do, q, k, v, o, lse, *again, mask, 0.09, workspace=ws[:n - 1])
    assert e.value.status == 5


def test_a_training_step_through_rotary_and_attention():
    """x -> rotary -> attention -> loss <o, g>, and back: the gradient of the unrotated q and k
    is the inverse rotation of the attention's."""
    B, H, G, d, T = 1, 4, 2, 64, 120
    spec = svga.RotarySpec(6, 4, 5, (10, 11, 11), False)
    table = svga.svga_rotary_table(spec, 1e4, torch.empty(spec.table_shape, device="cuda"))
    mask, scale = M(window=1, sinks=20, block=20), 0.125
    q = values(B, H, T, d, dtype=BF)
    k, v = (values(B, G, T, d, dtype=BF, seed=s) for s in (1, 2))
    do = values(B, H, T, d, dtype=BF, seed=3)
    tq, tk = (svga.svga_rotary(x.cuda(), torch.empty_like(x, device="cuda"), spec, table)
              for x in (q, k))
    _, _, (dq, dk, dv) = both_passes(tq, tk, v.cuda(), do.cuda(), mask, scale)
    check(tq.cpu(), tk.cpu(), v, do, mask, scale, (dq, dk, dv))
    for grad in (dq, dk):
        back = svga.svga_rotary(grad, torch.empty_like(grad), spec, table, inverse=True).cpu()
        for h in range(grad.shape[1]):
            within(back[0, h], *rotate(grad[0, h].cpu(), spec, 1e4, torch.arange(T), True))
