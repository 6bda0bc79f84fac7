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


def test_outputs_in_other_columns_of_an_inputs_buffer():
    """Matrices of one pitch whose columns do not meet do not overlap; with
    another pitch, or a column in common, they may."""
    L = B.lib()
    X, far = A[0], A[1]

    def dropout(y, x=X, rows=4, cols=100, ld=256, ldy=256, t=1, res=None):
        return L.fp4_dropout(x, rows, cols, ld, t, res, ld, 0.1, 1, 0, y, ldy, None)

    assert dropout(X + 200) in RAN and dropout(X + 312) in RAN       # columns 100 and 156 on, of 256
    assert dropout(X + 198) == B.EINVAL and dropout(X + 314) == B.EINVAL  # a column in common, on the right and (of the next row) the left
    assert dropout(X - 200) in RAN and dropout(X - 198) == B.EINVAL and dropout(X - 312) in RAN and dropout(X - 314) == B.EINVAL
    assert dropout(X + 200 + 512) in RAN                              # beside, and a row further on
    assert dropout(X + 200, ldy=255) == B.EINVAL                      # another pitch
    assert dropout(X + 400, t=0) in RAN and dropout(X + 396, t=0) == B.EINVAL
    assert dropout(X, res=X + 200) in RAN and dropout(X + 200, res=X + 200) in RAN and dropout(X + 200, res=X + 202) == B.EINVAL

    def norm(h, y, mean=None):
        return L.fp4_norm(X, 4, 100, 512, 1, far, 100, 0.1, 1, 0, h, 512, 0, None, None, 0, 1e-5, y, 512, mean, None, None,
                          None, 0, None)

    assert norm(X + 200, X + 400) in RAN and norm(X, X + 400) in RAN
    assert norm(X + 200, X + 398) == B.EINVAL and norm(X + 198, X + 400) == B.EINVAL and norm(X + 200, X + 200) == B.EINVAL
    assert norm(X + 200, X + 400, mean=X + 800) == B.EINVAL           # not a matrix of that pitch

    def grad(dh, dx, dy=X, h=X + 200):
        return L.fp4_norm_grad(dy, 4, 100, 512, 1, h, 512, None, 0, 1, None, 0, None, far, 0.1, 1, 0, dh, 512, dx, 512, None,
                               None, None, 0, None)

    assert grad(X + 400, X + 600) in RAN and grad(X, X + 200) in RAN and grad(X + 200, X + 400) in RAN
    assert grad(X + 400, X + 598) == B.EINVAL and grad(X + 398, X + 600) == B.EINVAL and grad(X + 400, X + 400) == B.EINVAL

    def swiglu(dc, h, c=X, dh=X + 256, ld=512):
        return L.fp4_swiglu_grad_bf16(dh, 512, c, 16, 64, 512, 32, dc, ld, h, 512, None)

    assert swiglu(X + 384, X + 640) in RAN and swiglu(X, X + 256) in RAN and swiglu(X + 384, None) in RAN
    assert swiglu(X + 240, None) == B.EINVAL and swiglu(X + 384, X + 624) == B.EINVAL and swiglu(X + 384, X + 112) == B.EINVAL
    assert swiglu(X + 384, None, ld=520) == B.EINVAL

    def rotary(y, xt=512, xh=64, yt=512, yh=64, n=50):
        return L.fp4_rotary(X, n, 3, 64, xt, xh, 1, far, 64, A[2], 64, 0, 0, 1.0, y, yt, yh, None)

    assert rotary(X + 384) in RAN and rotary(X + 640) in RAN and rotary(X + 382) == B.EINVAL and rotary(X + 642) == B.EINVAL
    assert rotary(X + 384, yt=520) == B.EINVAL
    apart = dict(xt=64, xh=8000, yt=64, yh=8000)                      # heads of 50 tokens at a pitch of 125
    assert rotary(X + 6400, **apart) in RAN and rotary(X + 6398, **apart) == B.EINVAL and rotary(X + 9600, **apart) in RAN
    assert rotary(X + 9602, **apart) == B.EINVAL


def test_refused_overlaps_are_those_that_share_bytes():
    """Every start of y around x, against the bytes themselves."""
    L = B.lib()
    x = A[0]
    for rows, cols, ld in ((1, 5, 9), (3, 4, 9), (4, 7, 7), (2, 3, 16)):
        own = {x + 2 * (r * ld + c) for r in range(rows) for c in range(cols)}
        for at in range(-2 * rows * ld, 2 * rows * ld + 1):
            y = x + 2 * at
            meets = any(y + 2 * (r * ld + c) in own for r in range(rows) for c in range(cols))
            got = L.fp4_dropout(x, rows, cols, ld, 1, None, 0, 0.1, 1, 0, y, ld, None)
            assert got in (RAN if not meets or at == 0 else (B.EINVAL,)), (rows, cols, ld, at)


@pytest.mark.parametrize("given", [{}, dict(mx=True), dict(mx=True, layout=B.LAYOUT_TILED),
                                   dict(codes=torch.zeros(4, dtype=torch.uint8))])
def test_norm_of_what_is_no_matrix(given):
    """The same refusal with the operand and without."""
    x = torch.zeros((4, 128), dtype=torch.bfloat16)
    for bad in (x[0], x[None], x.half()):
        with pytest.raises(ValueError):
            B.fp4_norm(bad, **given)
    for bad in (None, 3, x.numpy):
        with pytest.raises(ValueError, match="x must be a tensor"):
            B.fp4_norm(bad, **given)


@pytest.mark.parametrize("device", [None, 0, 1, "cpu", "cuda:0"])
def test_rotary_frequencies_go_to_the_device_asked_for(device, monkeypatch):
    """Index 0 is a device; only None is none."""
    asked = []
    to = torch.Tensor.to

    def record(self, *args, **kwargs):
        if args and args[0] is torch.float32:
            return to(self, *args, **kwargs)
        asked.append(args[0])
        return self

    monkeypatch.setattr(torch.Tensor, "to", record)
    B.rotary_frequencies(64, device=device)
    assert asked == ["cpu" if device is None else device]


def test_the_workspace_is_that_of_the_shape():
    """A larger matrix may need less, as the header says; a call takes what
    the query gave for its own shape, or more, and refuses less."""
    L = B.lib()
    need = L.fp4q_norm_grad_workspace_bytes
    assert need(500, 4096) == 0 and need(500, 3000) == 6_000_000
    assert need(2000, 32768) < need(2000, 16384)

    def f(rows, cols, given):
        return L.fp4_norm_grad(A[0], rows, cols, cols, 1, A[1], cols, None, 0, 0, None, 0, A[2], A[3], 0.0, 1, 0, A[4], cols,
                               None, 0, A[5], A[6], A[7] if given else None, given, None)

    for rows, cols in ((500, 4096), (500, 3000), (2000, 16384), (2000, 32768), (1, 1), (10 ** 5, 64), (800, 9000)):
        n = need(rows, cols)
        assert f(rows, cols, n) in RAN and f(rows, cols, n + 1000) in RAN
        assert n == 0 or f(rows, cols, n - 1) == B.EINVAL
    assert f(500, 3000, need(500, 4096)) == B.EINVAL


def test_the_header_says_that_the_workspace_is_that_of_the_shape():
    with open(B.HEADER) as f:
        text = " ".join(f.read().replace("*", " ").split())
    at = text.index("size_t fp4q_norm_grad_workspace_bytes")
    assert "a larger matrix may need less (500 x 4096: none, 500 x 3000: 6 MB)" in text[at - 400:at]


def test_the_workspace_serves_either_type():
    """Binary32 rows of 16 waves keep weight sums in the workspace from 641
    rows on, bf16 from 769 on; the query does not know the type."""
    L = B.lib()
    need = L.fp4q_norm_grad_workspace_bytes

    def f(rows, cols, t, given):
        return L.fp4_norm_grad(A[0], rows, cols, cols, t, A[1], cols, None, 0, 0, None, 0, A[2], A[3], 0.0, 1, 0, A[4], cols,
                               None, 0, A[5], A[6], A[7] if given else None, given, None)

    for rows, cols in ((641, 8192), (768, 8192), (700, 7700)):
        assert need(rows, cols) == 256 * 2 * cols * 4
        assert f(rows, cols, B.OUT_F32, need(rows, cols)) in RAN and f(rows, cols, B.OUT_BF16, need(rows, cols)) in RAN
        assert f(rows, cols, B.OUT_F32, 0) == B.EINVAL and f(rows, cols, B.OUT_BF16, 0) in RAN
    assert need(640, 8192) == 0 and need(768, 4096) == 0 and need(768, 7680) == 256 * 2 * 7680 * 4
    assert f(769, 8192, B.OUT_BF16, 0) == B.EINVAL
