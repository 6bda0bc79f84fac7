"""Products of few rows with FP4 weights over many steps of columns: every
kernel's loop and not its start alone, against binary64 products of the values
that the operands stand for."""
import pytest
import torch

from tests import pack8_ref as P
from tests.gpu_common import B, announce, device
from tests.test_gpu_row_ops import draw

pytestmark = pytest.mark.gpu

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
FORMATS = ["mx", "nv", "nv tile"]
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def products_on_the_gpu():
    """The oracle's products run on the GPU, and torch keeps the memory that its matrix library works in: made before
    there is a large block that it could be cut from, it lets go of those when they are free."""
    if torch.cuda.is_available():
        torch.cuda.empty_cache()
        one = torch.ones((8, 8), dtype=F64, device="cuda")
        assert float((one @ one.t()).sum()) == 512
    yield
    if torch.cuda.is_available():
        torch.cuda.empty_cache()


class Weights:
    """Random codes and scales (few binary orders apart, so that no product is lost in a sum), in a layout."""

    def __init__(self, fmt, n, k, tiled, dev, seed):
        g = torch.Generator(device=dev).manual_seed(seed)
        self.fmt, self.n, self.k, self.tiled = fmt, n, k, tiled
        block = 32 if fmt == "mx" else 16
        room = (n + 31) // 32 * 32 if tiled else n
        self.codes = torch.randint(0, 256, (room, k // 2), generator=g, device=dev, dtype=torch.uint8)
        low, high = (123, 130) if fmt == "mx" else (0x31, 0x49)  # 2^-4 .. 2^2, or E4M3's 0.5625 .. 4
        self.scales = torch.randint(low, high, (room, k // block), generator=g, device=dev, dtype=torch.uint8)
        self.ts = None
        if fmt != "mx":
            tiles = 1 if fmt == "nv" else (n + 127) // 128 * (k // 128)
            self.ts = torch.rand(tiles, generator=g, device=dev) + 0.5

    def call(self):
        """The call's tensors."""
        c, s, k = self.codes, self.scales, self.k
        if self.tiled and self.fmt == "mx":
            c = c.view(-1, 32, k // 64, 2, 16).permute(0, 2, 3, 1, 4).reshape(len(c), k // 2)
            s = s.view(len(s), k // 128, 4).transpose(0, 1).contiguous()
        elif self.tiled:
            c = c.view(-1, 32, k // 128, 64).transpose(1, 2).reshape(len(c), k // 2)
            s = s.view(-1, 32, k // 128, 8).transpose(1, 2).reshape(len(s), k // 16)
        return [c, s] if self.ts is None else [c, s, self.ts]

    def values(self, rows):
        """Binary64 values of a run of rows (a slice that starts on a tile)."""
        c, s = self.codes[rows].to(torch.int64), self.scales[rows]
        grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=F64, device=c.device)
        c = torch.stack((c & 15, c >> 4), -1).flatten(1)
        v = torch.where(c < 8, grid[c & 7], -grid[c & 7])
        unit = torch.exp2(s.to(F64) - 127) if self.fmt == "mx" else s.view(torch.float8_e4m3fn).to(F64)
        if self.fmt == "nv":
            unit = unit * self.ts.to(F64)
        elif self.fmt == "nv tile":
            ts = self.ts.to(F64).view(-1, self.k // 128)
            tile = torch.arange(rows.start, rows.start + len(c), device=c.device) // 128
            unit = unit * ts[tile].repeat_interleave(8, 1)
        return v * unit.repeat_interleave(self.k // unit.shape[1], 1)

    def check(self, y, x, what):
        """y against x (binary64) times the weights, within `pack8_ref.matvec_bound` and y's rounding."""
        one = torch.ones((1, self.k)).numpy()
        factor = float(P.matvec_bound(one, one)[0, 0]) / self.k  # of sum |x w|
        for at in range(0, self.n, 4096):
            rows = slice(at, min(at + 4096, self.n))
            w = self.values(rows)
            want = x @ w.t()
            off = (y[:, rows].to(F64) - want).abs()
            u = U if y.dtype == F32 else 2.0 ** -8
            room = factor * (1 + u) * (x.abs() @ w.abs().t()) + u * want.abs()
            bad = ~(off <= room)
            assert not bool(bad.any()), (what, at, int(bad.sum()), bad.nonzero()[0].tolist(), float((off / room).max()))


def product(w, x, args, x8=False, **more):
    more["layout"] = B.LAYOUT_TILED if w.tiled else B.LAYOUT_LINEAR
    if x8:
        return B.fp4_matvec_mx_pack8(*B.fp4_pack8(x), *args, n=w.n, **more)
    if w.fmt == "mx":
        return B.fp4_matvec_mx(x, *args, n=w.n, **more)
    return B.fp4_matvec_nv(x, *args, B.NV_GLOBAL if w.fmt == "nv" else B.NV_TILE128, n=w.n, **more)


def columns(each, tiled, odd):
    """Columns of which four waves get 11 or 12 steps, eight waves (where a unit has 16 rows of W, 20 to 23 with 16
    waves) five or six; in rows a step is 256 columns, or 128 where there is an odd number of those."""
    steps = 45 if each == 1 else 21
    return 128 * (steps if tiled or odd else 2 * steps)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tiled", [False, True])
@pytest.mark.parametrize("each", [1, 2, 3, 4, 5, 6, 7, 8])
def test_many_steps(fmt, tiled, each):
    """Every number of W's rows to a wave, and of x's, at least five steps of columns a wave (three where a workgroup has
    eight waves of more than 16 rows of W, each with one step in flight); a last workgroup that is short."""
    dev = device()
    units = torch.cuda.get_device_properties(dev).multi_processor_count
    n = 16 * units * each - 21
    for odd in ([False] if tiled else [False, True]):
        k = columns(each, tiled, odd)
        announce(f"matvec {fmt} tiled {tiled} many steps {n} x {k}")
        w = Weights(fmt, n, k, tiled, dev, each)
        args = w.call()
        for m in (3, 8, 16, 24, 32, 48, 64):
            x = draw((m, k), m, BF).to(dev)
            w.check(product(w, x, args), x.to(F64), f"{m} rows")
            if fmt == "mx":
                x = draw((m, k), m, BF, 5.0).to(dev)
                y = product(w, x, args, x8=True, out_dtype=BF)
                w.check(y, B.fp4_unpack8(*B.fp4_pack8(x)).to(F64), f"{m} 8-bit rows")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tiled", [False, True])
@pytest.mark.parametrize("n,k", [(9000, 2560), (28641, 4096)])
def test_same_bits_from_other_kernels(fmt, tiled, n, k):
    """Where a unit has more than 16 rows of W, few rows of x and up to 16 run in different kernels over many steps: a
    row's bits are those of the row alone."""
    dev = device()
    announce(f"matvec batched and alone {fmt} tiled {tiled} {n} x {k}")
    w = Weights(fmt, n, k, tiled, dev, 9)
    args = w.call()
    x = draw((16, k), 6, BF).to(dev)
    for x8 in (False, True) if fmt == "mx" else (False,):
        alone = torch.cat([product(w, x[i:i + 1], args, x8) for i in range(16)])
        for m in (2, 4, 5, 7, 8, 9, 13, 16):
            assert torch.equal(product(w, x[:m], args, x8), alone[:m]), (m, x8)


@pytest.mark.parametrize("tiled", [False, True])
@pytest.mark.parametrize("m,n,k", [(1, 4096, 14336), (17, 4096, 4096), (32, 4096, 4096), (64, 9000, 2560)])
def test_8_bit_rows_at_ordinary_sizes(tiled, m, n, k):
    """Against binary64, 8-bit rows and the same rows unpacked."""
    dev = device()
    announce(f"matvec of 8-bit rows tiled {tiled} {m} x {n} x {k}")
    w = Weights("mx", n, k, tiled, dev, m)
    args = w.call()
    x = draw((m, k), 3, BF, 5.0).to(dev)
    v = B.fp4_unpack8(*B.fp4_pack8(x))
    y = product(w, x, args, x8=True)
    w.check(y, v.to(F64), "8-bit rows")
    same = product(w, v, args)
    w.check(same, v.to(F64), "the rows unpacked")


@pytest.mark.parametrize("tiled", [False, True])
@pytest.mark.parametrize("n,k", [(2000, 4096), (4096, 4096), (8192, 2048), (9000, 2560), (28641, 4096)])
def test_8_bit_rows_have_the_bits_of_the_rows_unpacked(tiled, n, k):
    """The order of the sums does not depend on x's type."""
    dev = device()
    announce(f"matvec of 8-bit rows and of the rows unpacked, tiled {tiled} {n} x {k}")
    w = Weights("mx", n, k, tiled, dev, 5)
    args = w.call()
    x = draw((64, k), 3, BF, 5.0).to(dev)
    v = B.fp4_unpack8(*B.fp4_pack8(x))
    for m in (1, 3, 5, 8, 12, 16, 17, 24, 32, 40, 48, 64):
        assert torch.equal(product(w, x[:m], args, x8=True), product(w, v[:m], args)), m
