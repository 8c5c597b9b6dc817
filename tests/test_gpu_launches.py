"""Kernels of the streaming calls start while the one before them in the stream ends.  A chain of
calls, each reading what the one before it (or a torch kernel or a copy between them) wrote,
gives the bits that it gives with a synchronisation behind every step, eager and captured."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from block_sparse_spatio_attn_b200 import svga  # noqa: E402

BF = torch.bfloat16


class Chain:
    """A few heads of a generator: every step rotates, appends, decodes, attends with gradient, and
    writes the next step's inputs from the results, in the same buffers throughout."""

    def __init__(self, d, T, batch=2, H=4, G=2, page=16, steps=24, split=False):
        g = torch.Generator().manual_seed(d + T)
        rand = lambda *s: torch.randn(*s, generator=g).to(BF).cuda()  # noqa: E731
        self.steps, self.scale, self.d = steps, d ** -0.5, d
        self.q, self.k, self.v = rand(batch, H, T, d), rand(batch, G, T, d), rand(batch, G, T, d)
        self.qr, self.kr, self.o, self.dq = (torch.zeros_like(x) for x in (self.q, self.k, self.q, self.q))
        self.dk, self.dv = torch.zeros_like(self.k), torch.zeros_like(self.v)
        self.lse = torch.zeros(batch, H, T, device="cuda")
        self.spec = svga.RotarySpec(64, 4, 8, (d // 4, d // 8, d // 8))
        self.table = svga.svga_rotary_table(self.spec, 1e4, torch.empty(self.spec.table_shape, device="cuda"))
        pages = -(-(steps + 1) // page)
        self.kp = torch.zeros(batch * pages, G, page, d, dtype=BF, device="cuda")
        self.vp = torch.zeros_like(self.kp)
        self.pt = torch.arange(batch * pages, dtype=torch.int32, device="cuda").view(batch, pages)
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.lens_host = torch.zeros(batch, dtype=torch.int32).pin_memory()
        self.o1 = torch.zeros(batch, H, d, dtype=BF, device="cuda")
        self.mask = svga.WindowMask(window=T // 2, sinks=2) if not split else svga.WindowMask()
        self.lse1 = torch.zeros(batch, H, device="cuda")

    def step(self, wait):
        svga.svga_rotary(self.q, self.qr, self.spec, self.table)
        wait()
        svga.svga_rotary(self.k, self.kr, self.spec, self.table)
        wait()
        self.lens.add_(1)
        svga.svga_cache_append(self.kr[:, :, :1], self.v[:, :, :1], self.kp, self.vp, self.pt, self.lens,
                               rotary=self.spec, table=self.table)
        wait()
        svga.svga_cache_decode(self.qr[:, :, 0], self.kp, self.vp, self.pt, self.lens, self.o1, self.lse1, self.mask,
                               self.scale)
        wait()
        svga.svga_window_attention_fwd(self.qr, self.kr, self.v, self.o, self.lse, self.mask, self.scale)
        wait()
        svga.svga_window_attention_bwd(self.o, self.qr, self.kr, self.v, self.o, self.lse, self.dq, self.dk, self.dv,
                                       self.mask, self.scale)
        wait()
        svga.svga_rotary(self.dq, self.dq, self.spec, self.table, inverse=True)   # in place
        wait()
        svga.svga_rotary(self.dk, self.dk, self.spec, self.table, inverse=True)
        wait()
        # the next step's inputs: one from kernels, one from a copy, one from a rotation at once; all
        # stay of one size (sums of gradients alone would grow without end)
        self.q.add_(self.o).add_(self.dq).tanh_().mul_(2)
        self.q[:, :, 0].add_(self.o1)
        self.dv.add_(self.dk).tanh_()
        self.v.copy_(self.dv)
        svga.svga_rotary(self.kr, self.k, self.spec, self.table, first_token=7)
        wait()

    def state(self):
        return [x.clone() for x in (self.q, self.k, self.v, self.o, self.o1, self.lse, self.lse1, self.kp, self.vp,
                                    self.dq, self.dk, self.dv)]


def same(a, b):
    for x, y in zip(a, b):
        x, y = x.cpu(), y.cpu()
        assert x.view(torch.int16 if x.dtype == BF else torch.int32).equal(
            y.view(torch.int16 if y.dtype == BF else torch.int32))


@pytest.mark.parametrize("d,T,split", [(64, 70, False), (128, 33, False), (64, 300, False), (128, 700, True)])
def test_calls_back_to_back(d, T, split):
    slow, fast = Chain(d, T, split=split), Chain(d, T, split=split)
    for _ in range(slow.steps):
        slow.step(torch.cuda.synchronize)
    for _ in range(fast.steps):
        fast.step(lambda: None)
    same(slow.state(), fast.state())
    for x in (slow.o1, slow.q, slow.v, slow.dq):  # (NaN would equal NaN)
        assert x.float().isfinite().all() and x.float().abs().mean() > 1e-3


@pytest.mark.parametrize("d,T,split", [(128, 33, False), (64, 700, True)])
def test_captured_with_kernels_and_copies_between(d, T, split):
    slow, fast = Chain(d, T, split=split), Chain(d, T, split=split)
    fast.step(lambda: None)          # (everything is loaded before the capture)
    slow.step(torch.cuda.synchronize)
    graph = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        fast.step(lambda: None)
    for _ in range(10):
        slow.step(torch.cuda.synchronize)
        graph.replay()
    torch.cuda.synchronize()
    same(slow.state(), fast.state())


def test_lengths_copied_right_before_a_call():
    """The lengths arrive by a copy from pinned memory between two decodes that read them."""
    c = Chain(64, 20)
    c.kp.copy_(torch.randn(c.kp.shape, generator=torch.Generator().manual_seed(3)).to(BF))
    c.vp.copy_(torch.randn(c.vp.shape, generator=torch.Generator().manual_seed(4)).to(BF))
    lens = [torch.tensor([n, 25 - n], dtype=torch.int32).pin_memory() for n in range(26)]
    outs = {True: [], False: []}
    for wait in (True, False):
        got = [torch.zeros_like(c.o1) for _ in lens]
        for n, o in zip(lens, got):
            c.lens.copy_(n, non_blocking=True)
            if wait:
                torch.cuda.synchronize()
            svga.svga_cache_decode(c.q[:, :, 0], c.kp, c.vp, c.pt, c.lens, o, None, c.mask, c.scale)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        outs[wait] = got
    same(outs[True], outs[False])
    assert (outs[True][0][0] == 0).all() and (outs[True][25][1] == 0).all()


def test_two_streams_at_once():
    """Two chains interleaved on two streams keep out of each other's way."""
    alone = [Chain(64, 70), Chain(128, 33)]
    for c in alone:
        for _ in range(12):
            c.step(torch.cuda.synchronize)
    both = [Chain(64, 70), Chain(128, 33)]
    streams = [torch.cuda.Stream() for _ in both]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(12):
        for c, s in zip(both, streams):
            with torch.cuda.stream(s):
                c.step(lambda: None)
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        same(a.state(), b.state())


@pytest.mark.parametrize("d,T", [(64, 70), (128, 33)])
def test_one_chain_passed_between_two_streams(d, T):
    """Every call on the other stream than the one before it, joined by events only."""
    slow, fast = Chain(d, T), Chain(d, T)
    for _ in range(10):
        slow.step(torch.cuda.synchronize)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    at = [0]
    before = torch.cuda.current_stream()

    def turn():
        now, then = streams[at[0]], streams[1 - at[0]]
        then.wait_event(now.record_event())
        at[0] = 1 - at[0]
        torch.cuda.set_stream(then)

    torch.cuda.set_stream(streams[0])
    for _ in range(10):
        fast.step(turn)
    torch.cuda.synchronize()
    torch.cuda.set_stream(before)
    same(slow.state(), fast.state())
