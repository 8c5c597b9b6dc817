"""Rotary positions on three axes against the formula in 64 bits, elementwise within the
rounding each value allows; the fused token order against the permutation call, bit for bit."""
import pytest
import torch

from block_sparse_spatio_attn_b200 import configs as C

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from block_sparse_spatio_attn_b200 import svga  # noqa: E402
from tests.stream_reference import rotate, within  # noqa: E402

TYPES = [torch.bfloat16, torch.float16, torch.float32]


def table_of(spec, theta=10000.0):
    return svga.svga_rotary_table(spec, theta, torch.empty(spec.table_shape, device="cuda"))


def values(*shape, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype)


def test_table_is_the_angles_in_64_bits_rounded_once():
    spec = svga.RotarySpec(70_000, 45, 80, (3, 21, 5))
    assert svga.svga_rotary_table_size(spec) == 8 * spec.table_shape[0]
    got = table_of(spec, 1e4).cpu().double()
    at = 0
    for n, pairs in ((70_000, 3), (45, 21), (80, 5)):
        a = (torch.arange(n).double()[:, None] *
             1e4 ** (-torch.arange(pairs).double() / pairs)).reshape(-1)
        # half a step of fp32, and the 64-bit angle's own rounding (up to 2^17 * 2^-53 each way)
        for x, want in zip(got[at:at + n * pairs].unbind(1), (a.cos(), a.sin())):
            assert ((x - want).abs() <= 2.0 ** -25 + 2.0 ** -24 * want.abs() / 2 + 2.0 ** -35).all()
        at += n * pairs


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,pairs,interleaved", [
    (64, (8, 12, 12), True), (64, (8, 12, 12), False), (128, (22, 21, 21), True),
    (128, (22, 21, 21), False), (128, (5, 0, 6), True), (128, (5, 0, 6), False),
    (128, (8, 4, 4), False), (64, (0, 0, 1), False), (64, (0, 0, 0), True), (64, (32, 0, 0), True)])
def test_matches_the_formula_forward_and_inverse(dtype, d, pairs, interleaved):
    B, H, F, gh, gw = 2, 5, 3, 5, 7
    spec = svga.RotarySpec(F, gh, gw, pairs, interleaved)
    T = F * gh * gw
    x = values(B, H, T, d, dtype=dtype)
    table = table_of(spec)
    for inverse in (False, True):
        y = svga.svga_rotary(x.cuda(), torch.empty_like(x, device="cuda"), spec, table,
                             inverse=inverse).cpu()
        for b in range(B):
            for h in range(H):
                want, tol = rotate(x[b, h], spec, 1e4, torch.arange(T), inverse)
                within(y[b, h], want, tol, f"{b} {h} inverse={inverse}")


@pytest.mark.parametrize("tokens", [1, 2, 33])
@pytest.mark.parametrize("heads", [1, 3, 40])
def test_positions_and_first_token(tokens, heads):
    spec = svga.RotarySpec(50_000, 4, 5, (10, 11, 11), False)
    table, B, d = table_of(spec), 3, 64
    x = values(B, heads, tokens, d, dtype=torch.bfloat16, seed=tokens)
    first = torch.tensor([0, 999_960, 77_777])
    pos = first[:, None] + torch.arange(tokens)
    y = svga.svga_rotary(x.cuda(), torch.empty_like(x, device="cuda"), spec, table, pos.int().cuda())
    z = svga.svga_rotary(x[1:2].cuda(), torch.empty_like(x[1:2], device="cuda"), spec, table,
                         first_token=999_960)
    assert torch.equal(y[1], z[0])
    for b in range(B):
        for h in range(heads):
            within(y[b, h], *rotate(x[b, h], spec, 1e4, pos[b]))


def test_strided_views_and_in_place():
    spec = svga.RotarySpec(3, 4, 5, (10, 11, 11))
    B, H, T, d = 2, 6, 60, 64
    qkv = values(B, T, 3, H, d, dtype=torch.float16).cuda()
    before = qkv.clone()
    table = table_of(spec)
    q, k = qkv[:, :, 0].transpose(1, 2), qkv[:, :, 1].transpose(1, 2)
    out = torch.empty(B, H, T, d, dtype=torch.float16, device="cuda")
    svga.svga_rotary(q, out, spec, table)
    dense = svga.svga_rotary(before[:, :, 0].transpose(1, 2).contiguous(), torch.empty_like(out),
                             spec, table)
    assert torch.equal(out, dense)
    svga.svga_rotary(k, k, spec, table)  # in place, in the middle of the projection's output
    want = svga.svga_rotary(before[:, :, 1].transpose(1, 2).contiguous(), torch.empty_like(out),
                            spec, table)
    assert torch.equal(k, want)
    assert torch.equal(qkv[:, :, 0], before[:, :, 0]) and torch.equal(qkv[:, :, 2], before[:, :, 2])
    one = before[:, :, 0].transpose(1, 2)[:, :1].expand(B, H, T, d)  # a broadcast head, read only
    assert torch.equal(svga.svga_rotary(one, out, spec, table),
                       svga.svga_rotary(one.contiguous(), torch.empty_like(out), spec, table))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [True, False])
def test_order_is_the_permutation_of_the_rotation(dtype, interleaved):
    wl = C.tiny()
    order = [C.ORDER_FRAME_MAJOR, C.ORDER_TEMPORAL_MAJOR, C.ORDER_TEMPORAL_MAJOR_STRICT]
    H, T, d = 3, wl.tokens, 64
    plain = svga.RotarySpec(wl.frames, wl.grid_h, wl.grid_w, (8, 12, 12), interleaved)
    spec = svga.RotarySpec(wl.frames, wl.grid_h, wl.grid_w, (8, 12, 12), interleaved, order)
    table = table_of(spec)
    x = values(2, H, T, d, dtype=dtype).cuda()
    turned = svga.svga_rotary(x, torch.empty_like(x), plain, table)
    got = svga.svga_rotary(x, torch.empty_like(x), spec, table)
    if dtype == torch.bfloat16:
        prob = svga.ProblemSpec(H, wl.frames, wl.grid_h, wl.grid_w, d, [0, 1, 1], [1, 8, 8], order)
        for b in range(2):
            want = svga.svga_permute_tokens(turned[b], torch.empty_like(turned[b]), prob)
            assert torch.equal(got[b], want)
    F, S = wl.frames, wl.tokens_per_frame
    for h, od in enumerate(order):
        for t in range(T):
            f, s = divmod(t, S)
            pos = t if od == 0 else (s * F + f if od == 2 else
                                     (s if f == 0 else S + s * (F - 1) + f - 1))
            assert torch.equal(got[:, h, pos], turned[:, h, t])
    # the inverse comes back to frame-major at the plain inverse's values
    back = svga.svga_rotary(got, torch.empty_like(x), spec, table, inverse=True)
    assert torch.equal(back, svga.svga_rotary(turned, torch.empty_like(x), plain, table, inverse=True))


def test_single_frame_orders_and_bad_positions():
    spec = svga.RotarySpec(1, 3, 4, (1, 1, 1), order=[0, 1, 2])
    table = table_of(spec)
    x = values(1, 3, 12, 64, dtype=torch.bfloat16).cuda()
    got = svga.svga_rotary(x, torch.empty_like(x), spec, table)
    plain = svga.RotarySpec(1, 3, 4, (1, 1, 1))
    assert torch.equal(got, svga.svga_rotary(x, torch.empty_like(x), plain, table))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = torch.full_like(x, 7.0)
    pos = torch.tensor([[0, 12, -1] + list(range(9))], dtype=torch.int32, device="cuda")
    svga.svga_rotary(x, y, plain, table, pos, status=status)
    assert status.item() == 1
    assert (y[:, :, 1:3] == 7).all() and not (y[:, :, 3:] == 7).all()


def test_gradient_is_the_inverse():
    """The rotation is orthogonal, so <R x, g> = <x, R^-1 g>: the inverse call is the
    gradient.  fp32, sums of 2 * 60 * 64 products in 64 bits of values off by a few 2^-24."""
    spec = svga.RotarySpec(3, 4, 5, (10, 11, 11))
    table = table_of(spec)
    x, g = (values(1, 2, 60, 64, dtype=torch.float32, seed=s).cuda() for s in (1, 2))
    rx = svga.svga_rotary(x, torch.empty_like(x), spec, table).double()
    rg = svga.svga_rotary(g, torch.empty_like(x), spec, table, inverse=True).double()
    a, b = (rx * g.double()).sum(), (x.double() * rg).sum()
    size = (rx.abs() * g.double().abs()).sum() + (x.double().abs() * rg.abs()).sum()
    assert (a - b).abs() <= 8 * 2.0 ** -24 * size


def test_empty_and_captured():
    spec = svga.RotarySpec(3, 4, 5, (10, 11, 11))
    table = table_of(spec)
    e = torch.empty(2, 3, 0, 64, dtype=torch.bfloat16, device="cuda")
    svga.svga_rotary(e, torch.empty_like(e), spec, table)
    x = values(2, 3, 60, 64, dtype=torch.bfloat16).cuda()
    y, want = torch.empty_like(x), torch.empty_like(x)
    stream = torch.cuda.Stream()
    svga.svga_rotary(x, want, spec, table)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        svga.svga_rotary(x, y, spec, table)
    x.copy_(values(2, 3, 60, 64, dtype=torch.bfloat16, seed=5))
    graph.replay()
    svga.svga_rotary(x, want, spec, table)
    torch.cuda.synchronize()
    assert torch.equal(y, want)
