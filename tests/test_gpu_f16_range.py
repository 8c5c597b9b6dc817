"""fp16 has five bits of exponent: its smallest step is 2^-24 and its largest value 65504.  What the
attention calls hold in it on the way (P before its products, dS) must lose nothing to that range: a
long tail of keys far below one key, key lists so long that each P is small, gradients of any size.

Bounds.  u = 2^-11, half a step relative.
  * P is held relative to 2^6 times the largest of the first tile in the forward call, so a value
    below fp16's normal range is off by at most 2^-25 / 2^6 = 2^-31 of the row's largest (2^3 and 2^-28
    where that tile keeps one key; decode: 2^15 and 2^-40);
  * in the backward call P and dS are held times powers of two that bring their bounds to 2^14, so
    only what is 2^-28 of that bound leaves the normal range, and each is off by u relative;
  * errors of roundings that fall independently add like their squares: a sum of n of them, each
    at most u |x_j|, has a standard deviation of at most u sqrt(sum x_j^2) / sqrt(3); four times
    u sqrt(sum x_j^2) is above six of them;
  * dS is P times the difference of two sums in fp32, dO V^T (d terms in the tensor cores: off by at
    most d 2^-23 sum |dO| |v|) and D (a few steps: 2^-20 sum |dO| |o|), whose errors stay where the
    difference is small: a row of one key has a dS of 0, and of values of 10^6 some 10^-2 are left.
    They differ from pair to pair and add like their squares too; D's, which a row's pairs have
    in common, meets the sum of P K.
The norm of a row's gradient is compared, against 64 bits."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from block_sparse_spatio_attn_b200 import svga  # noqa: E402
from tests.stream_reference import kept, within  # noqa: E402

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


def tail_bound(p, v, least=2.0 ** -31):
    """P off by u, or `least` of the largest; sums of 16 products each a step of 2^-23; the result's
    rounding."""
    v = v.double()
    o = p @ v
    return o, (p @ v.abs()) * (U + len(p) / 16 * 2.0 ** -23 + 2.0 ** -17) + least * v.abs().sum(0) + U * o.abs() + 2.0 ** -25


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


@pytest.mark.parametrize("d,n,heads,rows", [(64, 16_384, 2, 1), (128, 20_000, 1, 200), (64, 9000, 160, 300)])
def test_forward_keeps_the_tail_behind_a_single_sink(d, n, heads, rows):
    """The first chunk keeps the sink alone; the window starts some chunks later."""
    q, k, v, p = tail(d, n, 17.6875)
    gap = 640
    mask = M(window=n - rows - gap, sinks=1)   # the last row keeps keys gap + rows - 1 and up, the first gap
    dev_q = q.cuda().expand(1, heads, rows, d).contiguous()
    dev_k, dev_v = (x.cuda().expand(1, heads, n, d) for x in (k, v))
    o, lse = torch.empty_like(dev_q), torch.empty(1, heads, rows, device="cuda")
    svga.svga_window_attention_fwd(dev_q, dev_k, dev_v, o, lse, mask, 1.0)
    keep = kept(mask, rows, n)
    x = torch.where(keep, (k.double() @ q.double()).expand(rows, n), -math.inf)
    for r in {0, rows // 2, rows - 1}:
        assert keep[r, 0] and not keep[r, 1:gap].any()
        want, tol = tail_bound(torch.softmax(x[r], 0), torch.where(keep[r][:, None], v, torch.zeros_like(v)), 2.0 ** -28)
        assert want.max() > 4 * tol.max()
        for h in (0, heads - 1):
            within(o[0, h, r], want, tol)
    assert (lse[0].double().cpu() - torch.logsumexp(x, 1)).abs().max() < 2.0 ** -15


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


def backward(q, k, v, do, mask, scale):
    """[tokens, d] each, one head: o, lse and the gradients on the CPU."""
    q, k, v, do = (x.to(FP).cuda()[None, None] for x in (q, k, v, do))
    o, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    grads = [torch.empty_like(x) for x in (q, k, v)]
    svga.svga_window_attention_fwd(q, k, v, o, lse, mask, scale)
    svga.svga_window_attention_bwd(do, q, k, v, o, lse, *grads, mask, scale)
    return [x[0, 0].cpu() for x in (o, *grads)]


def exact(q, k, v, do, o, mask, scale):
    """P and dS in 64 bits from the inputs rounded to fp16 and the forward call's o (so that its
    rounding, which the backward call is given, is no error of this one); dS's absolute errors."""
    q, k, v, do = (x.to(FP).double() for x in (q, k, v, do))
    keep = kept(mask, q.shape[0], k.shape[0])
    x = torch.where(keep, scale * q @ k.T, -math.inf)
    p = torch.where(keep, torch.softmax(x, 1), 0.0)
    ds = p * (do @ v.T - (do * o.double()).sum(1, keepdim=True))
    d_err = 2.0 ** -20 * (do.abs() * o.double().abs()).sum(1, keepdim=True)
    return q, k, do, p, ds, p * (q.shape[1] * 2.0 ** -23 * do.abs() @ v.abs().T + d_err), d_err


def norms_within(got, want, squares, what, more=0.0):
    """Row norms of the difference: the roundings of the terms (squares: the sum of the squares of
    a row's terms), arithmetic in fp32 and the exponents (u more), the result's rounding, and
    what else there is."""
    err = (got.double() - want).norm(dim=-1)
    out = (U * want.abs()).clamp(min=2.0 ** -25).norm(dim=-1)
    tol = 4 * U * squares.sqrt() + U * want.norm(dim=-1) + U * squares.sqrt() + out + more
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} rows off, the worst by {(err / tol).nan_to_num(1e9).max():.3g} bounds"


def check_dq(dq, q, k, do, p, ds, e, d_err, scale, rows=slice(None)):
    k2 = (k ** 2).sum(1)
    more = scale * ((e ** 2 @ k2).sqrt() + d_err[:, 0] * (p @ k).norm(dim=1))
    norms_within(dq[rows], (scale * ds @ k)[rows], (scale ** 2 * ds ** 2 @ k2)[rows], "dq", more[rows])


def check_dk(dk, q, k, do, p, ds, e, d_err, scale, rows=slice(None)):
    q2 = (q ** 2).sum(1)
    more = scale * ((e ** 2).T @ q2).sqrt()
    norms_within(dk[rows], (scale * ds.T @ q)[rows], (scale ** 2 * (ds ** 2).T @ q2)[rows], "dk", more[rows])


def check_dv(dv, q, k, do, p, ds, e, d_err, scale, rows=slice(None)):
    norms_within(dv[rows], (p.T @ do)[rows], ((p ** 2).T @ (do ** 2).sum(1))[rows], "dv")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [1.0, 1e-2, 1e-3, 1e-4])
def test_small_output_gradients_over_many_keys(d, size):
    """dS is about size / keys; K (for dq) or Q (for dk) is large, so that the results are not."""
    nq, nk, scale, big = 130, 8192, d ** -0.5, 64.0
    q, k, v, do = values(nq, d, seed=1), values(nk, d, seed=2), values(nk, d, seed=3), size * values(nq, d, seed=4)
    mask = M(causal=False)
    o, dq, _, dv = backward(q / big, k * big, v, do, mask, scale)
    at = exact(q / big, k * big, v, do, o, mask, scale)
    check_dq(dq, *at, scale)
    o, _, dk, _ = backward(q * big, k / big, v, do, mask, scale)
    check_dk(dk, *exact(q * big, k / big, v, do, o, mask, scale), scale)


@pytest.mark.parametrize("d", [64, 128])
def test_large_output_gradients(d):
    """dS passes 65504 where dQ and dK do not."""
    n, scale, size = 200, d ** -0.5, 8192.0
    mask = M(window=4)
    q, k, v, do = values(n, d, seed=1) / 64, values(n, d, seed=2) / 64, 16 * values(n, d, seed=3), size * values(n, d, seed=4)
    o, dq, dk, dv = backward(q, k, v, do, mask, scale)
    at = exact(q, k, v, do, o, mask, scale)
    assert at[4].abs().max() > 4 * 65504
    assert (scale * at[4] @ at[1]).abs().max() < 60000 and (scale * at[4].T @ at[0]).abs().max() < 60000
    check_dq(dq, *at, scale)
    check_dk(dk, *at, scale)
    check_dv(dv, *at, scale)


@pytest.mark.parametrize("d", [64, 128])
def test_values_of_keys_that_every_query_weighs_little(d):
    """P is 2^-26 for all keys but one, and 8,192 queries make dV of it."""
    n, nk = 8192, 300
    q, k, v, p = tail(d, nk, 18.0)
    do = 1 + 0.25 * values(n, d, seed=5)
    q = q.double().expand(n, d)
    mask = M(causal=False)
    o, _, _, dv = backward(q, k, v, do, mask, 1.0)
    at = exact(q, k, v, do, o, mask, 1.0)
    # every query has the same P, so its rounding (and the exponent's) is the same in every term
    want = at[3].T @ at[2]
    assert want[1:].abs().min() > 2.0 ** -14
    within(dv, want, (2 * U + n / 16 * 2.0 ** -23 + 2.0 ** -17) * (at[3].T @ at[2].abs()) + 2.0 ** -25)


@pytest.mark.parametrize("d", [64, 128])
def test_gradients_of_very_different_sizes_in_one_call(d):
    """Tokens 0-127 with an output gradient near 1, the others near 2e-5: keys that only the others
    see keep the accuracy of their own size."""
    n, scale, big = 1000, d ** -0.5, 64.0
    q, k, v, do = (values(n, d, seed=s) for s in (1, 2, 3, 4))
    do[128:] *= 2e-5
    mask = M(window=100)
    o, dq, _, _ = backward(q / big, k * big, v, do, mask, scale)
    check_dq(dq, *exact(q / big, k * big, v, do, o, mask, scale), scale)
    o, _, dk, _ = backward(q * big, k / big, v, do, mask, scale)
    check_dk(dk, *exact(q * big, k / big, v, do, o, mask, scale), scale, slice(256, None))


def test_gradients_of_zero_and_the_smallest_ones():
    n, d, mask = 300, 64, M()
    q, k, v = (values(n, d, seed=s) for s in (1, 2, 3))
    for g in backward(q, k, v, torch.zeros(n, d), mask, 0.125)[1:]:
        assert (g == 0).all()
    for g in backward(q, k, torch.zeros(n, d), values(n, d), mask, 0.125)[1:3]:
        assert (g == 0).all()
    do = torch.full((n, d), 2.0 ** -24)
    o, dq, dk, dv = backward(q / 64, k * 64, v, do, mask, 0.125)
    at = exact(q / 64, k * 64, v, do, o, mask, 0.125)
    check_dq(dq, *at, 0.125)
    check_dk(dk, *at, 0.125)
    check_dv(dv, *at, 0.125)


@pytest.mark.parametrize("d", [64, 128])
def test_values_that_are_not_finite_stay_in_their_tiles(d):
    """A dO row of NaN and a V row of infinity reach the tiles that visit them and no others."""
    n, scale, mask = 900, d ** -0.5, M(window=100)
    q, k, v, do = (values(n, d, seed=s) for s in (1, 2, 3, 4))
    clean = exact(q, k, v, do, backward(q, k, v, do, mask, scale)[0], mask, scale)
    bad = do.clone()
    bad[50] = math.nan
    _, dq, dk, dv = backward(q, k, v, bad, mask, scale)
    check_dq(dq, *clean, scale, slice(128, None))
    check_dk(dk, *clean, scale, slice(128, None))
    check_dv(dv, *clean, scale, slice(128, None))
    bad = v.clone()
    bad[50] = math.inf
    _, dq, dk, dv = backward(q, k, bad, do, mask, scale)
    check_dq(dq, *clean, scale, slice(256, None))
    check_dk(dk, *clean, scale, slice(256, None))
    check_dv(dv, *clean, scale, slice(256, None))
