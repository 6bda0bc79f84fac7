"""What a call on a named `stream` makes -- outputs, the operand, workspaces --
is memory of that stream, and what it returns may be let go of on the caller's
stream without more ado."""
import pytest
import torch

from tests.gpu_common import B, announce, device

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
T = B.LAYOUT_TILED


def pool_of(address):
    """The stream whose memory holds `address`."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= address < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("no such memory")


def tensors(v):
    if isinstance(v, torch.Tensor):
        return [v]
    return [t for e in v or () for t in tensors(e)] if isinstance(v, (tuple, list)) else []


def calls(dev, rows=1200, cols=1024):
    """Every binding call that makes what it returns; inputs are made here."""
    g = torch.Generator().manual_seed(1)
    x, r, dy = (torch.randn((rows, cols), generator=g).to(BF).to(dev) for _ in range(3))
    c = torch.randn((rows, 2 * cols), generator=g).to(BF).to(dev)
    w = (1 + torch.randn((cols,), generator=g) / 8).to(dev)
    pos = torch.arange(rows, device=dev)
    freq = B.rotary_frequencies(64, device=dev)[0]
    f = B.fp4_norm(x, w, residual=r, save=True)
    q = B.fp4_quantize_mx(x, layout=T)
    up = B.fp4_quantize_mx(torch.randn((512, cols), generator=g).to(BF).to(dev), layout=T)
    nv = B.fp4_quantize_nv(x)
    size = dict(layout=T, m=rows)
    return {
        "dropout": lambda **s: B.fp4_dropout(x, 0.2, seed=3, residual=r, **s),
        "norm": lambda **s: B.fp4_norm(x, w, residual=r, p=0.2, seed=4, save=True, mx=True, **s),
        "norm_grad": lambda **s: B.fp4_norm_grad(dy, f.h, w, mean=f.mean, rstd=f.rstd, p=0.2, seed=4, **s),
        "norm_grad, few rows": lambda **s: B.fp4_norm_grad(dy[:100], f.h[:100], w, mean=f.mean[:100], rstd=f.rstd[:100], **s),
        "swiglu_grad": lambda **s: B.fp4_swiglu_grad_bf16(dy, c, want_h=True, **s),
        "rotary": lambda **s: B.fp4_rotary(x.view(rows, 8, 128), pos, freq, **s),
        "quantize_mx": lambda **s: B.fp4_quantize_mx(x, layout=T, **s),
        "quantize_mx_dual": lambda **s: B.fp4_quantize_mx_dual(x[:1152], layout=T, **s),
        "hadamard32_quantize": lambda **s: B.fp4_hadamard32_quantize(x[:1152], 5, layout=T, **s),
        "quantize_nv": lambda **s: B.fp4_quantize_nv(x, **s),
        "quantize_nv, hadamard": lambda **s: B.fp4_quantize_nv(x[:1152], axis=B.ALONG_COLS, hadamard_mask=5, **s),
        "quantize_nv_noalloc": lambda **s: B.fp4_quantize_nv_noalloc(x, **s),
        "gemm_mx": lambda **s: B.fp4_gemm_mx(*q, *up, n=512, **size, **s),
        "gemm_mx_quant": lambda **s: B.fp4_gemm_mx_quant(*q, *up, n=512, **size, **s),
        "gemm_mx_swiglu_quant": lambda **s: B.fp4_gemm_mx_swiglu_quant(*q, *up, n=512, **size, **s),
        "swiglu": lambda **s: B.fp4_swiglu_bf16(c, cols, **s),
        "gemm_nv": lambda **s: B.fp4_gemm_nv(*nv, *nv, **s),
    }


def test_outputs_are_the_named_streams_memory():
    dev = device()
    side = torch.cuda.Stream()
    for name, call in calls(dev).items():
        announce(f"{name} on a named stream")
        want = [t.clone() for t in tensors(call())]
        torch.cuda.synchronize()
        got = tensors(call(stream=side))
        side.synchronize()
        assert len(got) == len(want) > 0
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), (name, i)
            assert pool_of(a.data_ptr()) == side.cuda_stream, (name, i)


def test_given_outputs_stay_where_they_are():
    dev = device()
    announce("given outputs on a named stream")
    side = torch.cuda.Stream()
    x = torch.randn((64, 256), device=dev).to(BF)
    y = torch.empty_like(x)
    torch.cuda.synchronize()
    assert B.fp4_dropout(x, 0.1, seed=1, y=y, stream=side).data_ptr() == y.data_ptr()
    side.synchronize()
    assert torch.cuda.current_stream() == torch.cuda.default_stream()  # as before the call


@pytest.mark.parametrize("what", ["norm_grad", "quantize_nv"])
def test_workspace_is_the_named_streams_memory(what):
    """With every output given the workspace is all that a call makes: the
    caller's pool does not grow and the named stream's does."""
    dev = device()
    announce(f"{what}'s workspace on a named stream")
    side = torch.cuda.Stream()
    rows, cols = 4096, 8192
    x = torch.randn((rows, cols), device=dev).to(BF)
    if what == "norm_grad":
        need = B.lib().fp4q_norm_grad_workspace_bytes(rows, cols)
        one, w = torch.ones(rows, device=dev), [torch.empty(cols, device=dev) for _ in range(2)]
        dh = torch.empty_like(x)

        def call():
            return B.fp4_norm_grad(x, x, rstd=one, mean=one, dh=dh, dgamma=w[0], dbeta=w[1], stream=side)
    else:
        need = B.fp4q_nv_workspace_bytes(rows, cols, B.ALONG_ROWS, B.NV_GLOBAL)
        out = B.fp4_quantize_nv(x)

        def call():
            return B.fp4_quantize_nv(x, codes=out[0], scales=out[1], tensor_scale=out[2], stream=side)
    assert need > 0
    torch.cuda.synchronize()

    def held(stream):
        return sum(s["total_size"] for s in torch.cuda.memory_snapshot() if s["stream"] == stream)

    torch.cuda.empty_cache()
    here, there = held(0), held(side.cuda_stream)
    call()
    side.synchronize()
    assert held(0) == here and held(side.cuda_stream) >= there + need


def test_outputs_let_go_of_wait_for_the_callers_stream():
    """A result read on the caller's stream and let go of there is not given
    out again on its own stream before the caller's work is through."""
    dev = device()
    side = torch.cuda.Stream()
    x = torch.randn((512, 1024), device=dev).to(BF)
    r = x.clone()
    pos, freq = torch.arange(512, device=dev), B.rotary_frequencies(128, device=dev)[0]
    torch.cuda.synchronize()
    for name, call in (("dropout", lambda: B.fp4_dropout(x, 0.1, seed=1, stream=side)),
                       ("norm", lambda: B.fp4_norm(x, residual=r, stream=side).y),
                       ("rotary", lambda: B.fp4_rotary(x.view(512, 8, 128), pos, freq, stream=side)),
                       ("swiglu", lambda: B.fp4_swiglu_bf16(x, 512, stream=side)),
                       ("quantize_mx", lambda: B.fp4_quantize_mx(x, stream=side)[0])):
        announce(f"{name}: a result let go of on the caller's stream")
        y = call()
        size, at = y.numel() * y.element_size(), y.data_ptr()
        side.synchronize()
        torch.cuda._sleep(200_000_000)  # the caller's stream is at work for a while
        busy = torch.cuda.Event()
        busy.record()
        del y
        with torch.cuda.stream(side):
            again = [torch.empty((size,), dtype=torch.uint8, device=dev) for _ in range(8)]
        ended = busy.query()
        assert ended or all(not t.data_ptr() <= at < t.data_ptr() + size for t in again), name
        torch.cuda.synchronize()


def test_streams_of_a_handle_and_of_nothing():
    dev = device()
    announce("streams given as a handle, and what is none")
    x = torch.randn((64, 256), device=dev).to(BF)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()

    class Handle:
        cuda_stream = side.cuda_stream

    want = B.fp4_dropout(x, 0.2, seed=3), B.fp4_quantize_mx(x)
    torch.cuda.synchronize()
    got = B.fp4_dropout(x, 0.2, seed=3, stream=Handle()), B.fp4_quantize_mx(x, stream=Handle())
    side.synchronize()
    assert torch.equal(got[0], want[0]) and all(torch.equal(a, b) for a, b in zip(got[1], want[1]))
    for bad in (object(), 5):
        with pytest.raises((AttributeError, ValueError)):
            B.fp4_dropout(x, 0.2, seed=3, stream=bad)
        with pytest.raises((AttributeError, ValueError)):
            B.fp4_quantize_mx(x, stream=bad)
    assert torch.equal(B.fp4_dropout(x, 0.2, seed=3), want[0])
    torch.cuda.synchronize()


def test_named_streams_in_a_captured_graph():
    """Calls on a stream forked off the captured one: every replay as the eager
    calls on its inputs."""
    dev = device()
    announce("named streams in a captured graph")
    rows, cols = 1200, 1024  # the gradient needs a workspace
    g = torch.Generator().manual_seed(1)
    x, r = (torch.randn((rows, cols), generator=g).to(BF).to(dev) for _ in range(2))
    w = (1 + torch.randn((cols,), generator=g) / 8).to(dev)
    side = torch.cuda.Stream()

    def step(**s):
        f = B.fp4_norm(x, w, residual=r, p=0.1, seed=1, save=True, mx=True, layout=T, **s)
        d = B.fp4_norm_grad(f.y, f.h, w, mean=f.mean, rstd=f.rstd, p=0.1, seed=1, **s)
        c, e = B.fp4_quantize_mx(d.dx, layout=T, **s)
        return [f.y, f.codes, f.scales, d.dh, d.dgamma, d.dbeta, B.fp4_dropout(d.dh, 0.2, seed=2, **s), c, e]

    def forked():
        side.wait_stream(torch.cuda.current_stream())
        out = step(stream=side)
        torch.cuda.current_stream().wait_stream(side)
        return out

    forked()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = forked()
    for k in range(3):
        x.copy_(torch.randn((rows, cols), generator=g).to(BF))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), k
