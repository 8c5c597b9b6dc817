"""The paged key-value cache: appended rows bit for bit where the page table says, and one
token's attention over the pages against 64 bits."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from block_sparse_spatio_attn_b200 import svga  # noqa: E402
from tests.stream_reference import attention, rotate, within  # noqa: E402

BF, FP = torch.bfloat16, torch.float16


class Cache:
    """Pages in a shuffled order, every row NaN until written."""

    def __init__(self, lens, heads, page, d, dtype, spare=2, seed=0):
        self.g = torch.Generator().manual_seed(seed)
        self.lens, self.page, self.dtype = list(lens), page, dtype
        most = max(1, max(-(-n // page) for n in self.lens))
        B = len(self.lens)
        n = B * most + spare
        ids = torch.randperm(n, generator=self.g)[:B * most].view(B, most).int()
        for b, x in enumerate(self.lens):
            ids[b, -(-x // page):] = -1  # never read
        self.table = ids.cuda()
        self.k = torch.full((n, heads, page, d), math.nan, dtype=dtype, device="cuda")
        self.v = self.k.clone()
        self.dev_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.g).to(self.dtype)

    def fill(self):
        """Random rows below each length; returns them as [batch][heads, len, d]."""
        ks, vs = [], []
        for b, n in enumerate(self.lens):
            k, v = (self.randn(self.k.shape[1], n, self.k.shape[3]) for _ in range(2))
            for x in range(0, n, self.page):
                i = int(self.table[b, x // self.page])
                m = min(self.page, n - x)
                self.k[i, :, :m], self.v[i, :, :m] = k[:, x:x + m].cuda(), v[:, x:x + m].cuda()
            ks.append(k)
            vs.append(v)
        return ks, vs

    def rows(self, pages, b):
        """[heads, len, d] of sequence b."""
        ids = self.table[b, :-(-self.lens[b] // self.page)].long()
        return pages[ids].transpose(0, 1).flatten(1, 2)[:, :self.lens[b]].cpu()

    def args(self):
        return self.k, self.v, self.table, self.dev_lens


def decode(c, q, mask, scale, **kw):
    B, H, d = q.shape
    o = torch.full((B, H, d), 9.0, dtype=q.dtype, device="cuda")
    lse = torch.full((B, H), 9.0, device="cuda")
    svga.svga_cache_decode(q.cuda(), *c.args(), o, lse, mask, scale, status=c.status, **kw)
    return o, lse


def check_decode(c, q, ks, vs, mask, o, lse, scale):
    share = q.shape[1] // c.k.shape[1]
    for b, n in enumerate(c.lens):
        for h in range(q.shape[1]):
            k, v = ks[b][h // share], vs[b][h // share]
            want, z, tol, z_tol = attention(q[b, h][None], k, v, mask, scale)
            within(o[b, h], want[0], tol[0], f"o of sequence {b} (length {n}), head {h}")
            within(lse[b, h], z[0], z_tol[0], f"lse of sequence {b} (length {n}), head {h}")


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("share", [1, 3, 16, 17])
def test_decode_lengths(dtype, d, share):
    lens = [0, 1, 15, 16, 17, 63, 64, 65, 130, 1000]
    c = Cache(lens, 2, 16, d, dtype, seed=share)
    ks, vs = c.fill()
    q = c.randn(len(lens), 2 * share, d)
    mask, scale = svga.WindowMask(), 1 / math.sqrt(d)
    o, lse = decode(c, q, mask, scale)
    assert c.status.item() == 0
    check_decode(c, q, ks, vs, mask, o, lse, scale)
    assert (o[0] == 0).all() and (lse[0] == -math.inf).all()


@pytest.mark.parametrize("page", [16, 48, 64, 256])
@pytest.mark.parametrize("mask", [
    svga.WindowMask(window=0), svga.WindowMask(window=7, sinks=3),
    svga.WindowMask(window=100, sinks=70), svga.WindowMask(window=1, block=60, sinks=60),
    svga.WindowMask(causal=False, window=3, block=17), svga.WindowMask(window=5000, sinks=5000)],
    ids=str)
def test_decode_masks_and_pages(page, mask):
    lens = [1, 59, 60, 61, 199, 777]
    c = Cache(lens, 3, page, 128, BF, seed=page)
    ks, vs = c.fill()
    q = c.randn(len(lens), 6, 128)
    o, lse = decode(c, q, mask, 0.2)
    assert c.status.item() == 0
    check_decode(c, q, ks, vs, mask, o, lse, 0.2)


def test_decode_splits_long_sequences():
    """Every number of CTAs a sequence's keys can be split over, and one longer than a
    16-bit row count."""
    for B, heads, n in ((1, 1, 70_001), (3, 1, 9000), (5, 3, 5000), (20, 7, 700), (75, 2, 300)):
        c = Cache([n - 3 * b for b in range(B)], heads, 64, 64, BF, seed=B)
        ks, vs = c.fill()
        q = c.randn(B, heads * 2, 64)
        o, lse = decode(c, q, svga.WindowMask(), 0.125)
        check_decode(c, q, ks, vs, svga.WindowMask(), o, lse, 0.125)
        again, _ = decode(c, q, svga.WindowMask(), 0.125)
        assert torch.equal(o, again)


def test_decode_large_scores_and_strided_tensors():
    """Scores up to +-3000 (the softmax is then one or two keys), q and o as slices of wider
    tensors, o's neighbours untouched, lse left out."""
    c = Cache([300, 200], 2, 32, 64, BF)
    ks, vs = c.fill()
    q = 40 * c.randn(2, 4, 64)
    wide_q = torch.zeros(2, 4, 192, dtype=BF, device="cuda")
    wide_q[:, :, 64:128] = q.cuda()
    wide_o = torch.full((4, 2, 128), 5.0, dtype=BF, device="cuda")
    o = wide_o.transpose(0, 1)[:, :, 64:]
    svga.svga_cache_decode(wide_q[:, :, 64:128], *c.args(), o, None, svga.WindowMask(), 1.0)
    share = 2
    for b in range(2):
        for h in range(4):
            want, _, tol, _ = attention(q[b, h][None], ks[b][h // share], vs[b][h // share],
                                        svga.WindowMask(), 1.0)
            within(o[b, h], want[0], tol[0])
    assert (wide_o[:, :, :64] == 5).all()


def test_decode_reports_bad_pages_and_lengths():
    c = Cache([100, 100, 100], 2, 16, 64, BF)
    ks, vs = c.fill()
    q = c.randn(3, 2, 64)
    c.table[0, 2] = 10_000       # keys 32-47 of sequence 0 count as masked
    c.table[1, 6] = -5           # keys 96-99 of sequence 1
    o, lse = decode(c, q, svga.WindowMask(), 0.1)
    assert c.status.item() == 1
    for b, cut in ((0, slice(32, 48)), (1, slice(96, 100)), (2, slice(0, 0))):
        at = torch.ones(100, dtype=torch.bool)
        at[cut] = False
        for h in range(2):
            want, z, tol, z_tol = attention(q[b, h][None], ks[b][h][at], vs[b][h][at],
                                            svga.WindowMask(), 0.1)
            within(o[b, h], want[0], tol[0])
            within(lse[b, h], z[0], z_tol[0])
    c = Cache([100], 2, 16, 64, BF)
    c.fill()
    c.dev_lens.fill_(113)        # 7 pages hold 112 rows
    o, lse = decode(c, q[:1], svga.WindowMask(), 0.1)
    assert c.status.item() == 1 and (o == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("rotate_it", [False, True, "halves"])
def test_append_writes_the_rows_the_table_names(dtype, rotate_it):
    new = [0, 1, 5, 33, 40]
    lens = [10, 1, 64, 33, 131]
    c = Cache(lens, 3, 16, 64, dtype)
    T = 40
    k, v = (c.randn(5, T, 3, 64).transpose(1, 2) for _ in range(2))
    spec = table = None
    if rotate_it:
        spec = svga.RotarySpec(7, 4, 5, (10, 11, 11), rotate_it is True)
        table = svga.svga_rotary_table(spec, 1e4, torch.empty(spec.table_shape, device="cuda"))
    svga.svga_cache_append(k.cuda(), v.cuda(), *c.args(),
                           torch.tensor(new, dtype=torch.int32, device="cuda"), spec, table,
                           status=c.status)
    assert c.status.item() == 0
    written = 0
    for b, (n, m) in enumerate(zip(new, lens)):
        got_k, got_v = c.rows(c.k, b), c.rows(c.v, b)
        assert got_k[:, :m - n].isnan().all() and got_v[:, :m - n].isnan().all()
        assert torch.equal(got_v[:, m - n:], v[b, :, :n])
        for h in range(3):
            if rotate_it:
                within(got_k[h, m - n:], *rotate(k[b, h, :n], spec, 1e4, torch.arange(m - n, m)))
            else:
                assert torch.equal(got_k[h, m - n:], k[b, h, :n])
        written += 3 * 64 * n
    assert int((~c.k.isnan()).sum()) == written and int((~c.v.isnan()).sum()) == written


def test_append_reports_and_skips_bad_rows():
    c = Cache([20, 20], 1, 16, 64, BF)
    k, v = c.randn(2, 1, 4, 64).cuda(), c.randn(2, 1, 4, 64).cuda()
    c.table[0, 1] = -1
    svga.svga_cache_append(k, v, *c.args(), status=c.status)
    assert c.status.item() == 1
    assert c.rows(c.k, 1)[:, 16:].equal(k[1].cpu()) and int((~c.k.isnan()).sum()) == 4 * 64
    c = Cache([20, 2], 1, 16, 64, BF)   # 4 rows cannot end at length 2
    svga.svga_cache_append(k, v, *c.args(), status=c.status)
    assert c.status.item() == 1
    assert c.rows(c.k, 1).equal(k[1, :, 2:].cpu()) and c.rows(c.k, 0)[:, 16:].equal(k[0].cpu())
    spec = svga.RotarySpec(1, 4, 4, (1, 1, 1))  # positions 16-19 lie outside the grid
    table = svga.svga_rotary_table(spec, 1e4, torch.empty(spec.table_shape, device="cuda"))
    c = Cache([18], 1, 16, 64, BF)
    svga.svga_cache_append(k[:1], v[:1], *c.args(), None, spec, table, status=c.status)
    assert c.status.item() == 1 and int((~c.k.isnan()).sum()) == 2 * 64


def test_append_leaves_both_rows_of_a_position_outside_the_grid():
    spec = svga.RotarySpec(1, 4, 4, (1, 1, 1))  # 16 positions
    table = svga.svga_rotary_table(spec, 1e4, torch.empty(spec.table_shape, device="cuda"))
    c = Cache([18], 1, 16, 64, BF)
    k, v = c.randn(1, 1, 4, 64).cuda(), c.randn(1, 1, 4, 64).cuda()
    svga.svga_cache_append(k, v, *c.args(), None, spec, table, status=c.status)
    assert c.status.item() == 1
    written = c.rows(c.v, 0).isnan().logical_not().all(-1)[0].tolist()
    assert written == [False] * 14 + [True] * 2 + [False] * 2
    assert c.rows(c.k, 0).isnan().logical_not().all(-1)[0].tolist() == written


def test_a_stream_of_steps_as_a_generator_runs_them():
    """Prompt, then token by token: rotate q, append rotated k, attend with a window and
    sinks, captured once and replayed with the lengths moved on the device."""
    B, Hk, share, d, page = 2, 2, 4, 64, 16
    spec = svga.RotarySpec(20, 2, 5, (10, 11, 11))
    table = svga.svga_rotary_table(spec, 1e4, torch.empty(spec.table_shape, device="cuda"))
    mask, scale, prompt, steps = svga.WindowMask(window=20, sinks=10), 0.125, [37, 52], 30
    c = Cache([n + steps for n in prompt], Hk, page, d, BF)
    all_k, all_v = (c.randn(B, Hk, 100, d) for _ in range(2))
    all_q = c.randn(B, Hk * share, 100, d)
    lens, one = torch.tensor(prompt, dtype=torch.int32, device="cuda"), torch.ones(B, dtype=torch.int32, device="cuda")
    svga.svga_cache_append(all_k[:, :, :52].cuda(), all_v[:, :, :52].cuda(), c.k, c.v, c.table, lens, lens, spec, table)
    q, k, v = (torch.empty(B, h, 1, d, dtype=BF, device="cuda") for h in (Hk * share, Hk, Hk))
    o = torch.empty(B, Hk * share, d, dtype=BF, device="cuda")
    turned = torch.empty_like(q)

    def step():
        lens.add_(one)
        svga.svga_rotary(q, turned, spec, table, (lens - 1)[:, None].contiguous(), status=c.status)
        svga.svga_cache_append(k, v, c.k, c.v, c.table, lens, None, spec, table, status=c.status)
        svga.svga_cache_decode(turned[:, :, 0], c.k, c.v, c.table, lens, o, None, mask, scale, status=c.status)

    def load(i):
        for dst, src in ((q, all_q), (k, all_k), (v, all_v)):
            dst.copy_(torch.stack([src[b, :, prompt[b] + i] for b in range(B)])[:, :, None])

    load(0)
    step()                      # eager once, then undone, then captured
    lens.sub_(one)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(steps):
        load(i)
        graph.replay()
        got = o.cpu()
        for b in range(B):
            n = prompt[b] + i + 1
            for h in range(Hk * share):
                # the calls round the turned q and k to bf16: the reference starts from those
                tq = rotate(all_q[b, h, n - 1][None], spec, 1e4, torch.tensor([n - 1]))[0].to(BF)
                tk = c.rows(c.k, b)[h // share, :n]
                want, _, tol, _ = attention(tq, tk, all_v[b, h // share, :n], mask, scale)
                # the library's own rounding of a tied turned value may differ by one step
                within(got[b, h], want[0], tol[0] + 2.0 ** -8 * 0.05)
    assert c.status.item() == 0
    for b in range(B):
        for h in range(Hk):
            n = prompt[b] + steps
            within(c.rows(c.k, b)[h], *rotate(all_k[b, h, :n], spec, 1e4, torch.arange(n)))


def test_other_streams_and_the_current_device():
    c = Cache([300], 2, 16, 64, FP)
    ks, vs = c.fill()
    q = c.randn(1, 4, 64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = torch.empty(1, 4, 64, dtype=FP, device="cuda")
    lse = torch.empty(1, 4, device="cuda")
    qd = q.cuda()
    side.wait_stream(torch.cuda.current_stream())
    svga.svga_cache_decode(qd, *c.args(), o, lse, svga.WindowMask(), 0.125, stream=side)
    side.synchronize()
    check_decode(c, q, ks, vs, svga.WindowMask(), o, lse, 0.125)
