"""What the row-wise operators take and refuse at their edges (before any HIP
call, so without a GPU; the addresses are never dereferenced)."""
import pytest
import torch

from fp4_block_scaled_quantizer_amd import binding as B
from tests.test_row_ops import RAN, A


def test_rotary_takes_heads_of_whole_tokens():
    L = B.lib()

    def f(n=100, heads=3, dim=64, xt=64, xh=6400, y=A[3], yt=192, yh=64):
        return L.fp4_rotary(A[0], n, heads, dim, xt, xh, 1, A[1], 64, A[2], 64, 0, 0, 1.0, y, yt, yh, None)

    assert f() in RAN                                           # [heads, tokens, dim] to [tokens, heads, dim]
    assert f(yt=64, yh=6400) in RAN and f(yt=72, yh=8000) in RAN  # to itself, and with gaps
    assert f(xt=192, xh=64, yt=64, yh=6400) in RAN              # and back
    assert f(y=A[0], yt=64, yh=6400) in RAN                     # in place
    assert f(y=A[0]) == B.EINVAL                                # in place in another order
    assert f(xh=6399) == B.ESHAPE and f(yt=64, yh=6399) == B.ESHAPE  # a head's last token meets the next head
    assert f(xt=63, xh=6400) == B.ESHAPE and f(xt=0) == B.ESHAPE and f(xh=-6400) == B.ESHAPE
    assert f(n=0, xt=0) in (B.OK, B.ESHAPE) and f(heads=1, xt=64, xh=64) in RAN
