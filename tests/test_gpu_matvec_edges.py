"""Products of few rows with FP4 weights at the ends of what they take."""
import math

import pytest
import torch

from tests.gpu_common import B, announce, device
from tests.test_gpu_row_ops import Padded

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("alpha", [1.0, math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("m,n", [(1, 1), (5, 1031), (64, 37)])
def test_no_columns_give_zeros(alpha, m, n):
    """Whatever alpha is, as the GEMMs do, and nothing beside Y."""
    dev = device()
    announce(f"matvec {m} x {n} x 0, alpha {alpha}")
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=dev)  # noqa: E731
    x = torch.ones((m, 0), dtype=BF, device=dev)
    for out in (F32, BF):
        for call in (lambda **a: B.fp4_matvec_mx(x, u8(n, 0), u8(n, 0), **a),
                     lambda **a: B.fp4_matvec_mx_pack8(u8(m, 0), u8(m, 0), u8(n, 0), u8(n, 0), **a),
                     lambda **a: B.fp4_matvec_nv(x, u8(n, 0), u8(n, 0), torch.ones(1, device=dev), **a)):
            py = Padded(m, n, out, dev, 3, 1)
            py.view.fill_(5.0)
            call(alpha=alpha, y=py.view)
            assert bool((py.view == 0).all()) and py.untouched()


def test_no_columns_of_many_rows():
    """More rows of W than 16 to a workgroup of 64 threads allow in one launch (nothing else bounds them at K = 0)."""
    dev = device()
    n = (1 << 30) + 77
    announce(f"matvec 1 x {n} x 0")
    y = torch.full((1, n), 5.0, dtype=BF, device=dev)
    none = torch.zeros((n, 0), dtype=torch.uint8, device=dev)
    B.fp4_matvec_mx(torch.ones((1, 0), dtype=BF, device=dev), none, none, y=y)
    assert not bool(y.any())
