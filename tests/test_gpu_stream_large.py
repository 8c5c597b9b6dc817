"""Offsets past 32 bits: a rotation of 9 GB, attention with its gradients over heads 4 GB apart,
a cache of 10 GB whose sequence lives in its last pages."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from block_sparse_spatio_attn_b200 import svga  # noqa: E402
from tests.stream_reference import attention, gradients, rotate, within  # noqa: E402

BF = torch.bfloat16


def values(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(BF)


def test_rotation_of_nine_gigabytes():
    spec = svga.RotarySpec(1050, 10, 100, (22, 21, 21))  # 1,050,000 tokens
    table = svga.svga_rotary_table(spec, 1e4, torch.empty(spec.table_shape, device="cuda"))
    T, H = 1_050_000, 17
    x = torch.empty(2, H, T, 128, dtype=BF, device="cuda")
    rows = values(40, 128)
    spots = [(b, h, t) for b in (0, 1) for h in (0, 8, 16) for t in (0, 524_287, T - 1)]
    for i, (b, h, t) in enumerate(spots):
        x[b, h, t] = rows[i].cuda()
    svga.svga_rotary(x, x, spec, table)
    for i, (b, h, t) in enumerate(spots):
        want, tol = rotate(rows[i:i + 1], spec, 1e4, torch.tensor([t]))
        within(x[b, h, t][None], want, tol, f"{b} {h} {t}")


def test_attention_over_heads_four_gigabytes_apart():
    n, d, mask, scale = 300, 64, svga.WindowMask(window=100, sinks=3), 0.125
    big = torch.empty((1 << 32) + (1 << 24), dtype=BF, device="cuda")  # 8.6 GB
    step = (1 << 31) + 64                                              # elements: 4 GB and a bit

    def view(at):
        return big.as_strided((1, 2, n, d), (step * 2, step, d, 1), at * n * d)

    q, k, v, o, do, dq, dk, dv = (view(i) for i in range(8))
    host = [values(1, 2, n, d, seed=s) for s in range(4)]
    for x, y in zip((q, k, v, do), host):
        x.copy_(y)
    lse = torch.empty(1, 2, n, device="cuda")
    svga.svga_window_attention_fwd(q, k, v, o, lse, mask, scale)
    svga.svga_window_attention_bwd(do, q, k, v, o, lse, dq, dk, dv, mask, scale)
    for h in range(2):
        a = [x[0, h] for x in host]
        want, z, tol, z_tol = attention(a[0], a[1], a[2], mask, scale)
        within(o[0, h], want, tol)
        within(lse[0, h], z, z_tol)
        g = gradients(*a, mask, scale)
        for got, w, t in zip((dq, dk, dv), g[:3], g[3:]):
            within(got[0, h], w, t)


def test_cache_of_ten_gigabytes():
    pages, heads, page, d, n = 40_000, 8, 64, 128, 1000
    k_pages = torch.empty(pages, heads, page, d, dtype=BF, device="cuda")
    v_pages = torch.empty_like(k_pages)
    need = -(-n // page)
    table = (pages - 1 - 3 * torch.arange(need, dtype=torch.int32))[None].cuda()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    k, v = values(1, heads, n, d), values(1, heads, n, d, seed=1)
    svga.svga_cache_append(k.cuda(), v.cuda(), k_pages, v_pages, table, lens)
    q = values(1, heads, d, seed=2)
    o, lse = torch.empty(1, heads, d, dtype=BF, device="cuda"), torch.empty(1, heads, device="cuda")
    svga.svga_cache_decode(q.cuda(), k_pages, v_pages, table, lens, o, lse, svga.WindowMask(), 1 / math.sqrt(d))
    for h in range(heads):
        want, z, tol, z_tol = attention(q[0, h][None], k[0, h], v[0, h], svga.WindowMask(), 1 / math.sqrt(d))
        within(o[0, h], want[0], tol[0])
        within(lse[0, h], z[0], z_tol[0])
