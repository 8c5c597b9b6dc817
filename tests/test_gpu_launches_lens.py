"""The window calls with lengths and tensors that the kernels right before them in the stream write:
the backward call reads none of them before those kernels have ended.  Every step gives the bits
that it gives with a synchronisation behind every call."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from block_sparse_spatio_attn_b200 import svga  # noqa: E402

STEPS = 12


class Padded:
    """A padded batch whose lengths arrive by copies from pinned memory and whose Q, K, V and dO are
    written anew by torch kernels and rotations, all right before the calls that read them."""

    def __init__(self, d, T, dtype, G=2, H=4, B=3, window=None, lens=True, sinks=5):
        g = torch.Generator().manual_seed(d + T)
        rand = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()  # noqa: E731
        self.scale, self.lens = d ** -0.5, lens
        self.q, self.k, self.v, self.do = rand(B, H, T, d), rand(B, G, T, d), rand(B, G, T, d), rand(B, H, T, d)
        self.qr, self.kr, self.o, self.dq = (torch.zeros_like(x) for x in (self.q, self.k, self.q, self.q))
        self.dk, self.dv, self.dor = torch.zeros_like(self.k), torch.zeros_like(self.v), torch.zeros_like(self.do)
        self.lse = torch.zeros(B, H, T, device="cuda")
        self.spec = svga.RotarySpec(T, 1, 1, (d // 2, 0, 0))
        self.table = svga.svga_rotary_table(self.spec, 1e4, torch.empty(self.spec.table_shape, device="cuda"))
        self.ql, self.kl = (torch.full((B,), T, dtype=torch.int32, device="cuda") for _ in range(2))
        self.hosts = [tuple(torch.randint(0, T + 1, (B,), generator=g, dtype=torch.int32).pin_memory()
                            for _ in range(2)) for _ in range(STEPS)]
        self.mask = svga.WindowMask(window=T // 2 if window is None else window, sinks=sinks)

    def step(self, i, wait):
        if self.lens:
            self.ql.copy_(self.hosts[i][0], non_blocking=True)
            self.kl.copy_(self.hosts[i][1], non_blocking=True)
        lens = (self.ql, self.kl) if self.lens else (None, None)
        wait()
        svga.svga_rotary(self.q, self.qr, self.spec, self.table)
        wait()
        svga.svga_rotary(self.k, self.kr, self.spec, self.table)
        wait()
        svga.svga_window_attention_fwd(self.qr, self.kr, self.v, self.o, self.lse, self.mask, self.scale, *lens)
        wait()
        svga.svga_rotary(self.do, self.dor, self.spec, self.table)  # dO by the call right before
        wait()
        svga.svga_window_attention_bwd(self.dor, self.qr, self.kr, self.v, self.o, self.lse, self.dq, self.dk, self.dv,
                                       self.mask, self.scale, *lens)
        wait()
        # again with K, V and lengths written by the kernels right before, and the same statistics
        if self.lens:
            self.kl.copy_(self.kl.clamp(max=self.kl.max() // 2 + 1))
        self.v.copy_(self.dv.float().tanh())
        svga.svga_rotary(self.k, self.kr, self.spec, self.table)
        wait()
        svga.svga_window_attention_fwd(self.qr, self.kr, self.v, self.o, self.lse, self.mask, self.scale, *lens)
        wait()
        svga.svga_window_attention_bwd(self.o, self.qr, self.kr, self.v, self.o, self.lse, self.dq, self.dk, self.dv,
                                       self.mask, self.scale, *lens)
        wait()
        self.q.add_(self.o).add_(self.dq).tanh_().mul_(2)
        self.k.add_(self.dk).tanh_().mul_(2)
        self.do.add_(self.dq).tanh_()

    def state(self):
        return [x.clone() for x in (self.q, self.k, self.v, self.do, self.o, self.lse, self.dq, self.dk, self.dv)]


def same(a, b):
    for x, y in zip(a, b):
        x, y = x.cpu(), y.cpu()
        kind = torch.int32 if x.dtype == torch.float32 else torch.int16
        assert x.view(kind).equal(y.view(kind))


@pytest.mark.parametrize("lens", [True, False])
@pytest.mark.parametrize("d,T,dtype", [(64, 70, torch.bfloat16), (128, 33, torch.float16), (128, 300, torch.bfloat16),
                                       (64, 900, torch.float16)])
def test_backward_calls_right_behind_what_writes_their_inputs(d, T, dtype, lens):
    slow, fast = Padded(d, T, dtype, lens=lens), Padded(d, T, dtype, lens=lens)
    for i in range(STEPS):
        slow.step(i, torch.cuda.synchronize)
    for i in range(STEPS):
        fast.step(i, lambda: None)
    same(slow.state(), fast.state())
    assert slow.dq.float().isfinite().all() and slow.q.float().abs().mean() > 1e-3


def test_captured_with_lengths_that_change_between_replays():
    slow, fast = Padded(64, 300, torch.bfloat16), Padded(64, 300, torch.bfloat16)
    slow.step(0, torch.cuda.synchronize)
    fast.step(0, lambda: None)
    fast.hosts[1][0].copy_(slow.hosts[1][0])
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        fast.step(1, lambda: None)  # the copies read fast.hosts[1] at every replay
    for i in range(1, STEPS):
        for x, y in zip(fast.hosts[1], slow.hosts[i]):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        slow.step(i, torch.cuda.synchronize)
    same(slow.state(), fast.state())


def test_a_backward_call_without_queries_between_others():
    """Gradients of keys that no query sees are zeros, behind a kernel that wrote 7s there."""
    k = torch.ones(2, 2, 300, 64, dtype=torch.bfloat16, device="cuda")
    e = torch.empty(2, 4, 0, 64, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(2, 4, 0, device="cuda")
    dk, dv = torch.empty_like(k), torch.empty_like(k)
    for _ in range(20):
        dk.fill_(7.0)
        dv.fill_(7.0)
        svga.svga_window_attention_bwd(e, e, k, k, e, lse, e, dk, dv, svga.WindowMask(), 0.125)
        x, y = dk.clone(), dv.clone()
        assert (x == 0).all() and (y == 0).all()
