"""Attention of whole prompts whose scores are as large as the interface allows (+-1e30):
rows that one token decides get its V, and nothing is infinite or not a number."""

import numpy as np
import pytest
import torch

from chunk_ref import assert_attention
from libpkv import ensure_built
from test_gpu_prompt import Prompts

pytestmark = pytest.mark.gpu
MASKS = [(0, 0), (40, 3), (300, 0)]


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def decided(p, window, sinks):
    """(rows that one token decides [T, hq], its V there [T, hq, d] fp64, the largest |V| in sight [T, hq, d]).

    A score in fp32 is off by at most d roundings (2^-24 each) of sums no larger than sum |q_i k_i|, its product
    with the scale by one more, and so is the other one that it is compared with: 2 (d + 2) 2^-24 times the largest
    such sum in sight. Where the first is ahead of the second by that and 30 more, all others weigh less than
    513 e^-30 < 2^-34 beside it."""
    ok, best, top, at = [], [], [], 0
    for n in p.new:
        q, k, v = (x[at:at + n].double() for x in (p.q, p.k, p.v))
        at += n
        t = torch.arange(n, device="cuda")
        hide = t > t[:, None]
        if window > 0:
            hide |= (t[:, None] - t >= window) & (t >= sinks)
        qg = q.view(n, p.hkv, -1, p.d)
        x = (torch.einsum("mhgd,thd->mhgt", qg, k) * p.d ** -0.5).masked_fill(hide[:, None, None], -float("inf"))
        size = (torch.einsum("mhgd,thd->mhgt", qg.abs(), k.abs()) * p.d ** -0.5).masked_fill(hide[:, None, None], 0.0)
        two = torch.topk(x, min(2, n), dim=-1).values
        gap = two[..., 0] - two[..., 1] if n > 1 else torch.full_like(two[..., 0], float("inf"))
        bound = 2 * (p.d + 2) * 2.0 ** -24 * size.amax(-1)
        ok.append((gap >= bound + 30).reshape(n, p.hq))
        j = x.argmax(-1)  # [m, hkv, g]
        h = torch.arange(p.hkv, device="cuda")[None, :, None].expand_as(j)
        best.append(v[j, h].reshape(n, p.hq, p.d))
        big = v.abs()[None].masked_fill(hide[:, :, None, None], 0.0).amax(1)
        top.append(big[:, :, None].expand(n, p.hkv, p.hq // p.hkv, p.d).reshape(n, p.hq, p.d))
    return tuple(torch.cat(a).cpu().numpy() for a in (ok, best, top))


def check(p, share):
    for window, sinks in MASKS:
        out = p.run(window, sinks)
        ok, best, top = decided(p, window, sinks)
        got = out[:p.T].double().cpu().numpy()
        assert np.isfinite(got).all(), (window, sinks)
        # weights of one sum, each off by 2^-8 at most, and the output's rounding
        assert (np.abs(got) <= top * (1 + 2.0 ** -8) * (1 + 2.0 ** -8) + 1e-30).all()
        assert ok.mean() >= share, ok.mean()
        assert_attention(torch.as_tensor(got[ok]), best[ok], np.abs(best[ok]), f"window {window}")
        assert p.lc.error_bits() == 0


@pytest.mark.parametrize("heads", [(4, 2, 64), (16, 8, 128)])
@pytest.mark.parametrize("e", [20, 26, 27, 28, 29, 30, 31, 32, 33, 40, 64, 95])
def test_scores_up_to_the_largest(heads, e):
    check(Prompts(11, [6, 1, 300, 131], heads, q_mult=2.0 ** e), 0.8)


@pytest.mark.parametrize("heads", [(8, 1, 64), (8, 2, 128)])
@pytest.mark.parametrize("falling", [False, True])
def test_scores_that_grow_along_the_prompt(heads, falling):
    """From token to token, past every size at which the weights' path changes, and within each warp's rows."""
    p = Prompts(13, [300, 20, 513], heads)
    at = 0
    for n in p.new:
        e = torch.arange(n, device="cuda") * 90 // n  # 0 .. 89
        p.k[at:at + n] *= (2.0 ** (e.flip(0) if falling else e).double()).to(torch.bfloat16)[:, None, None]
        at += n
    check(p, 0.4)


def test_rows_of_all_sizes_side_by_side():
    p = Prompts(17, [400, 77], (8, 2, 128))
    g = torch.Generator().manual_seed(5)
    e = torch.randint(-6, 96, (p.T, 8, 1), generator=g)
    p.q[:p.T] *= (2.0 ** e.double()).to(torch.bfloat16).cuda()
    check(p, 0.6)
