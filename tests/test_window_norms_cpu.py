"""The norm bounds of window_norms tell a kernel that keeps its weights' digits
from one that does not (mistakes planted in a plain evaluation; no GPU)."""
import pytest
import torch

import window_norms


def attend(w, v, keep):
    return keep(w) @ v / w.sum(-1, keepdim=True)


def bf16(x):
    return x.to(torch.bfloat16).double()


def truncated(x):
    return (x.float().view(torch.int32) & -65536).view(torch.float32).double()


@pytest.mark.parametrize("n", [1000, 8200])
def test_the_bounds_separate_the_forms(n):
    g = torch.Generator().manual_seed(n)
    q, k, v = (torch.randn(s, 128, generator=g).to(torch.bfloat16).double() for s in (16, n, n))
    s = q @ k.T * 128 ** -0.5
    w = torch.exp(s - s.amax(-1, keepdim=True))
    ref = w @ v / w.sum(-1, keepdim=True)
    two = lambda x: bf16(x) + bf16(x - bf16(x))  # noqa: E731
    three = lambda x: two(x) + bf16(x - two(x))  # noqa: E731
    cut = lambda x: truncated(x) + truncated(x - truncated(x))  # noqa: E731
    off = {f: window_norms.off(attend(w, v, f), ref) for f in (two, three, cut, bf16)}
    assert off[three] < window_norms.CLUSTER < off[two] < window_norms.FOLDED < window_norms.UNFOLDED < off[bf16]
    assert off[cut] > window_norms.FOLDED
