"""8-bit rows of more pieces than one launch of the unpacking takes (2^31)."""
import pytest
import torch

from tests import pack8_ref as P
from tests.gpu_common import B, announce, device

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def give_back():
    """Some 45 GB, which later tests neither need nor expect in torch's cache."""
    yield
    if torch.cuda.is_available():
        torch.cuda.empty_cache()


def test_unpack_in_more_than_one_part():
    """Rows of 2^13 pieces of four binary32 elements: 2^18 rows in the first part, three in the second."""
    dev = device()
    announce("unpack8 past 2^31 pieces")
    first, cols = 1 << 18, 1 << 15
    rows = first + 3
    codes = torch.zeros((rows, cols), dtype=torch.uint8, device=dev)
    scales = torch.full((rows, cols // 32), 127, dtype=torch.uint8, device=dev)
    at = [0, 1, first - 1, first, first + 1, rows - 1]
    g = torch.Generator(device=dev).manual_seed(1)
    codes[at] = torch.randint(0, 127, (len(at), cols), generator=g, device=dev, dtype=torch.uint8)
    scales[at] = torch.randint(100, 150, (len(at), cols // 32), generator=g, device=dev, dtype=torch.uint8)
    y = B.fp4_unpack8(codes, scales, out_dtype=torch.float32)
    want = torch.from_numpy(P.values(codes[at].cpu(), scales[at].cpu()))
    assert torch.equal(y[at].double().cpu(), want)
    assert not bool(y[2:first - 1].any()) and not bool(y[first + 2:-1].any())
