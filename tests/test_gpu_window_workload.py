"""The window calls at the size of the 75,600-token video workload (21 frames of 45 x 80), causal: a
spatial head's band of three frames with its anchor frame, and no window at all.  Forward, and the
gradients of two query heads that share a key head, against 64 bits: sampled queries' rows of O, lse
and dQ, sampled keys' rows of dK and dV (over every query of both heads).

Bounds as in stream_reference.py, and for sums this long: fp32 accumulators add 16 products at a
time, a step of 2^-23 of the sum of the magnitudes each; a softmax sum adds a tile of 128 at a time.
In fp16 a P of the forward call is off by 2^-31 of the row's largest, a dS by 2^-39 of its bound."""
import math

import pytest
import torch

from block_sparse_spatio_attn_b200 import configs as C

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from block_sparse_spatio_attn_b200 import svga  # noqa: E402
from tests.stream_reference import ARITH, HALF_STEP, within  # noqa: E402

WL = C.headline()
N, S, D = WL.tokens, WL.tokens_per_frame, WL.head_dim
SCALE = D ** -0.5
ROWS = [0, 1, 127, 128, S - 1, S, 2 * S + 77, 37_800, 65_536, N - 129, N - 1]


def mask_rows(mask, rows):
    """[rows, N] truth values, straight from the mask's definition."""
    p, j = rows[:, None], torch.arange(N, device="cuda")[None]
    bp, bj = p // mask.block, j // mask.block
    near = ((bp - bj).abs() <= mask.window) | (j < mask.sinks) if mask.window >= 0 else torch.ones_like(bp < bj)
    return near & (bj <= bp) if mask.causal else near


def exact_rows(q, k, v, do, mask, rows, u):
    """One head's quantities of some query rows in 64 bits with bounds: a dict of tensors."""
    keep = mask_rows(mask, rows)
    x = (SCALE * q[rows] @ k.T).masked_fill_(~keep, -math.inf)
    r = {"lse": torch.logsumexp(x, 1)}
    p = x.sub_(r["lse"][:, None]).exp_()
    n = keep.sum(1)
    r["keep"], r["p"], r["o"] = keep, p, p @ v
    pv = p @ v.abs()
    size = SCALE * q[rows].abs() @ k.abs().amax(0)             # of scale q k, at most
    dx = size * D * 2.0 ** -23
    small = 2.0 ** -31 * p.amax(1)[:, None] * (keep.double() @ v.abs()) + 2.0 ** -25 if u == 2.0 ** -11 else 0.0
    r["o_tol"] = (u + 2 * dx + ARITH + n / 16 * 2.0 ** -23)[:, None] * pv + u * r["o"].abs() + small
    r["lse_tol"] = dx + n / 128 * 2.0 ** -24 + 2.0 ** -19 * (1 + r["lse"].abs())
    g = do[rows]
    r["delta"] = (g * r["o"]).sum(1)
    r["delta_abs"] = (g.abs() * (u * r["o"].abs() + r["o_tol"])).sum(1) + 2.0 ** -20 * (g.abs() * r["o"].abs()).sum(1)
    r["p_rel"] = 2 * (dx + r["lse_tol"]) + ARITH
    r["least"] = 2.0 ** -39 * (g.norm(dim=1) * v.norm(dim=1).max() + r["delta"].abs()) if u == 2.0 ** -11 else 0 * dx
    return r


def ds_of(r, g, v_rows, p, u):
    """dS and its bound for the pairs of r's rows and some keys (p: their P)."""
    ds = p * (g @ v_rows.T - r["delta"][:, None])
    err = p * ((g.abs() @ v_rows.abs().T) * D * 2.0 ** -23 + r["delta_abs"][:, None])
    return ds, err + (r["p_rel"] + u + ARITH)[:, None] * ds.abs() + r["least"][:, None]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("mask", [svga.WindowMask(window=WL.band[0], sinks=S, block=S), svga.WindowMask()], ids=str)
def test_causal_form_of_the_workload(mask, dtype):
    u, H = HALF_STEP[dtype], 2
    gen = torch.Generator(device="cuda").manual_seed(7)
    q, k, v, do = (torch.randn(1, h, N, D, generator=gen, device="cuda").to(dtype) for h in (H, 1, 1, H))
    o, lse, status = torch.empty_like(q), torch.empty(1, H, N, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    dq, dk, dv = (torch.empty_like(x) for x in (q, k, v))
    svga.svga_window_attention_fwd(q, k, v, o, lse, mask, SCALE, status=status)
    svga.svga_window_attention_bwd(do, q, k, v, o, lse, dq, dk, dv, mask, SCALE, status=status)
    assert status.item() == 0
    k64, v64 = k[0, 0].double(), v[0, 0].double()
    rows = torch.tensor(ROWS, device="cuda")
    keys = torch.tensor([0, 5, 130, S - 1, S, 3 * S + 11, 40_000, N - S - 1, N - 1], device="cuda")
    sums = {x: torch.zeros(len(keys), D, dtype=torch.float64, device="cuda") for x in ("dk", "dv", "dk_tol", "dv_tol")}
    for h in range(H):
        q64, g64 = q[0, h].double(), do[0, h].double()
        r = exact_rows(q64, k64, v64, g64, mask, rows, u)
        what = f"{mask} {dtype} head {h}"
        within(o[0, h, rows], r["o"].cpu(), r["o_tol"].cpu(), "o, " + what)
        within(lse[0, h, rows], r["lse"].cpu(), r["lse_tol"].cpu(), "lse, " + what)
        ds, err = ds_of(r, g64[rows], v64, r["p"], u)
        err = torch.where(r["keep"], err, 0.0)
        want = SCALE * ds @ k64
        long = (r["keep"].sum(1) / 16 * 2.0 ** -23)[:, None]
        tol = SCALE * err @ k64.abs() + (u + ARITH) * want.abs() + (ARITH + long) * SCALE * ds.abs() @ k64.abs() + 2.0 ** -25
        within(dq[0, h, rows], want.cpu(), tol.cpu(), "dq, " + what)
        for first in range(0, N, 1800):  # every query, for the sampled keys
            at = torch.arange(first, min(first + 1800, N), device="cuda")
            r = exact_rows(q64, k64, v64, g64, mask, at, u)
            p, there = r["p"][:, keys], r["keep"][:, keys]
            ds, err = ds_of(r, g64[at], v64[keys], p, u)
            err = torch.where(there, err, 0.0)
            long = N * H / 16 * 2.0 ** -23
            sums["dv"] += p.T @ g64[at]
            sums["dv_tol"] += (p * (u + r["p_rel"] + ARITH + long)[:, None] + there * 2.0 ** -39).T @ g64[at].abs()
            sums["dk"] += SCALE * ds.T @ q64[at]
            sums["dk_tol"] += SCALE * (err + (ARITH + long) * ds.abs()).T @ q64[at].abs()
    for x, got in (("dk", dk), ("dv", dv)):
        tol = sums[x + "_tol"] + (u + ARITH) * sums[x].abs() + 2.0 ** -25
        within(got[0, 0, keys], sums[x].cpu(), tol.cpu(), f"{x}, {mask} {dtype}")
