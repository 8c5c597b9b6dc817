"""fp16 has five bits of exponent: its smallest step is 2^-24 and its largest value 65504.  What the
attention calls hold in it on the way (P before its product with V) must lose nothing to that range: a
long tail of keys far below one key.

Bounds.  u = 2^-11, half a step relative.
  * P is held relative to 2^6 times the largest of the first tile in the forward call, so a value
    below fp16's normal range is off by at most 2^-25 / 2^6 = 2^-31 of the row's largest (decode: less)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from block_sparse_spatio_attn_b200 import svga  # noqa: E402
from tests.stream_reference import within  # noqa: E402

FP = torch.float16
U = 2.0 ** -11
M = svga.WindowMask


def values(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def tail(d, n, depth, seed=0):
    """One key `depth` (in nats) above n - 1 equal ones; its value row is 0, theirs are near 1."""
    q, k = torch.zeros(d), torch.zeros(n, d)
    q[0], k[0, 0] = 4.0, depth / 4
    v = 1 + 0.25 * values(n, d, seed=seed)
    v[0] = 0
    q, k, v = q.to(FP), k.to(FP), v.to(FP)
    p = torch.softmax(k.double() @ q.double(), 0)
    return q, k, v, p


def tail_bound(p, v):
    """P off by u, or 2^-31 of the largest; sums of 16 products each a step of 2^-23; the result's
    rounding."""
    v = v.double()
    o = p @ v
    return o, (p @ v.abs()) * (U + len(p) / 16 * 2.0 ** -23 + 2.0 ** -17) + 2.0 ** -31 * v.abs().sum(0) + U * o.abs() + 2.0 ** -25


# 17.6875 nats: each key has 2^-25.5 of the first one's weight, which fp16 would round to 0
@pytest.mark.parametrize("d,n,heads,rows", [(64, 16_384, 1, 1), (128, 16_384, 1, 1), (128, 20_000, 2, 130),
                                            (64, 16_384, 160, 256), (128, 5000, 4, 700)])
def test_forward_keeps_a_long_tail_far_below_one_key(d, n, heads, rows):
    q, k, v, p = tail(d, n, 17.6875)
    want, tol = tail_bound(p, v)
    assert want.min() > 4 * tol.max()
    dev_q = q.cuda().expand(1, heads, rows, d).contiguous()
    dev_k, dev_v = (x.cuda().expand(1, heads, n, d) for x in (k, v))
    for mask in (M(causal=False), M(causal=False, window=1, block=1 << 20, sinks=1)):
        o, lse = torch.empty_like(dev_q), torch.empty(1, heads, rows, device="cuda")
        svga.svga_window_attention_fwd(dev_q, dev_k, dev_v, o, lse, mask, 1.0)
        for h in (0, heads - 1):
            within(o[0, h], want.expand(rows, d), tol.expand(rows, d))
        assert (lse - torch.logsumexp(k.double() @ q.double(), 0).item()).abs().max() < 2.0 ** -15


@pytest.mark.parametrize("d,n,page", [(64, 16_384, 16), (128, 16_384, 64), (128, 3001, 48), (64, 32_768, 256)])
def test_decode_keeps_a_long_tail_far_below_one_key(d, n, page):
    q, k, v, p = tail(d, n, 17.6875)
    want, tol = tail_bound(p, v)
    assert want.min() > 2 * tol.max()
    need = -(-n // page)
    kp, vp = (torch.zeros(need * page, d, dtype=FP) for _ in range(2))
    kp[:n], vp[:n] = k, v
    kp, vp = (x.view(need, 1, page, d).expand(need, 2, page, d).contiguous().cuda() for x in (kp, vp))
    table = torch.arange(need, dtype=torch.int32, device="cuda").expand(3, need).contiguous()
    lens = torch.full((3,), n, dtype=torch.int32, device="cuda")
    dev_q = q.cuda().expand(3, 6, d).contiguous()
    o, lse = torch.empty_like(dev_q), torch.empty(3, 6, device="cuda")
    svga.svga_cache_decode(dev_q, kp, vp, table, lens, o, lse, M(), 1.0)
    within(o, want.expand(3, 6, d), tol.expand(3, 6, d))
    assert (lse - torch.logsumexp(k.double() @ q.double(), 0).item()).abs().max() < 2.0 ** -15
