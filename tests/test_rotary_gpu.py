"""Rotary positions on the GPU against the float64 rotation.  fp32: two products and a sum of values
within 2^-24 each, sines to 2^-23 and angles to 2^-32 turns (1.5e-9 radians): one value is off by at
most 5 * 2^-24 * |x| < 4e-7 |x| (|x| the pair's length).  bf16: one rounding, half a step 2^-8 of the
value, on top."""
import numpy as np
import pytest
import torch

from hybrid_softmax_linear_chunked_b200 import binding as rb
from oracle import sequence_oracle as SO

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from hybrid_softmax_linear_chunked_b200 import build
    build.build()
    rb.load()
    return torch.device("cuda", 0)


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def check(got, x, positions, freq, scale, interleaved, inverse, what):
    """positions [B, n, R/2]"""
    x, y = f64(x), f64(got)
    R = 2 * freq.numel()
    for b in range(x.shape[0]):
        want = SO.rotary(x[b], positions[b], f64(freq), scale, interleaved, inverse)
        i1 = np.arange(0, R, 2) if interleaved else np.arange(R // 2)
        i2 = i1 + 1 if interleaved else i1 + R // 2
        size = np.abs(want)
        pair = np.hypot(x[b][..., i1], x[b][..., i2]) * abs(scale)
        size[..., i1] = size[..., i2] = pair
        tol = 4e-7 * size + (2.0 ** -8 * np.abs(want) if got.dtype == torch.bfloat16 else 0)
        assert (np.abs(y[b] - want) <= tol).all(), what
        assert (y[b][..., R:] == x[b][..., R:]).all(), what + ": dimensions past R"


def rows(g, dev, dtype, B, heads, n, D, layout):
    x = torch.randn(B, heads, n, D, generator=g).to(dtype).to(dev)
    if layout == "bnhd":
        return x.transpose(1, 2).contiguous().transpose(1, 2)
    if layout == "odd":  # rows at odd element offsets
        pad = torch.zeros(B, heads, n, D + 3, dtype=dtype, device=dev)
        pad[..., 1:D + 1] = x
        return pad[..., 1:D + 1]
    return x


CASES = [  # dtype, B, H, Hk, n, D, R, layout, interleaved, far
    (torch.bfloat16, 1, 1, 1, 1, 128, 128, "bhnd", False, 0),
    (torch.bfloat16, 8, 12, 12, 1, 128, 128, "bhnd", True, 5000),
    (torch.bfloat16, 2, 6, 2, 77, 64, 32, "bnhd", False, 1 << 20),
    (torch.bfloat16, 1, 3, 1, 130, 96, 48, "bhnd", True, (1 << 31) - 200),
    (torch.float32, 1, 2, 2, 513, 128, 128, "bhnd", False, 1 << 24),
    (torch.float32, 2, 5, 3, 33, 64, 32, "bnhd", True, 1 << 20),
    (torch.float32, 1, 2, 1, 9, 10, 6, "bhnd", False, 100),
    (torch.bfloat16, 2, 2, 1, 5, 24, 20, "odd", True, 3000),
    (torch.float32, 1, 40, 1, 3, 64, 64, "odd", False, 3000),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_rotation_and_gradient(dev, case):
    dt, B, H, Hk, n, D, R, layout, inter, far = case
    g = torch.Generator().manual_seed(n)
    q, k = rows(g, dev, dt, B, H, n, D, layout), rows(g, dev, dt, B, Hk, n, D, layout)
    freq, scale = rb.rotary_frequencies(R, scaling="yarn", factor=4.0, original_length=512,
                                        device=dev)
    pos = torch.randint(0, far + 1, (B, n), generator=g)
    want = f64(pos)[..., None].repeat(R // 2, -1)
    q0 = q.clone()
    for dtype in (torch.int32, torch.int64):
        for inverse in (False, True):
            a, b = rb.rotary(q, k, freq, positions=pos.to(dev, dtype), scale=scale,
                             interleaved=inter, inverse=inverse)
            rb.sync_status(dev)
            check(a, q, want, freq, scale, inter, inverse, "q")
            check(b, k, want, freq, scale, inter, inverse, "k")
    assert torch.equal(q, q0)
    # q alone, in place, from a start: the same values
    i = torch.arange(n) + 17
    want = np.broadcast_to(f64(i)[None, :, None], (B, n, R // 2))
    fresh = rb.rotary(q, None, freq, start=17, scale=scale, interleaved=inter)
    check(fresh, q, want, freq, scale, inter, False, "start")
    from_tensor = rb.rotary(q, None, freq, start=torch.full((B,), 17, device=dev), scale=scale,
                            interleaved=inter)
    assert torch.equal(from_tensor, fresh)
    assert rb.rotary(q, None, freq, start=17, scale=scale, interleaved=inter, q_out=q) is q
    assert torch.equal(q, fresh)


def test_video_axes_and_negative_positions(dev):
    T, fh, fw, R, B = 3, 4, 5, 32, 2
    n = T * fh * fw
    g = torch.Generator().manual_seed(1)
    q, k = (rows(g, dev, torch.float32, B, h, n, 48, "bhnd") for h in (3, 2))
    freq, _ = rb.rotary_frequencies(R, device=dev)
    axis = rb.rotary_axes((6, 5, 5), device=dev)
    pos = rb.video_positions(T, fh, fw, first_frame=-2, device=dev).expand(3, B, n)
    a, b = rb.rotary(q, k, freq, positions=pos, axis=axis)
    want = np.stack([f64(pos)[ax] for ax in axis.tolist()], -1)
    assert want.min() == -2
    check(a, q, want, freq, 1.0, False, False, "q")
    check(b, k, want, freq, 1.0, False, False, "k")


def test_gradient_is_the_transpose(dev):
    """<dy, J dx> = <J^T dy, dx>: the call is linear, so its inverse-turn form is its gradient."""
    g = torch.Generator().manual_seed(3)
    x, y = (torch.randn(1, 2, 40, 64, generator=g).to(dev) for _ in range(2))
    freq, _ = rb.rotary_frequencies(64, device=dev)
    fwd = rb.rotary(x, None, freq, start=1000, scale=1.3)
    bwd = rb.rotary(y, None, freq, start=1000, scale=1.3, inverse=True)
    lhs, rhs = ((y.double() * fwd.double()).sum(), (bwd.double() * x.double()).sum())
    assert abs(float(lhs - rhs)) <= 1e-6 * float(x.double().norm() * y.double().norm())


def test_graph_and_stream(dev):
    g = torch.Generator().manual_seed(4)
    q = torch.randn(4, 3, 1, 64, generator=g).to(dev)
    freq, _ = rb.rotary_frequencies(64, device=dev)
    start = torch.tensor([3, 9, 0, 70000], device=dev)
    want = rb.rotary(q, None, freq, start=start)
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        other = rb.rotary(q, None, freq, start=start)
    torch.cuda.current_stream(dev).wait_stream(side)
    assert torch.equal(other, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = rb.rotary(q, None, freq, start=start)
    start.add_(1)
    graph.replay()
    assert torch.equal(out, rb.rotary(q, None, freq, start=start))


def test_empty_and_refusals(dev):
    q = torch.zeros(2, 3, 0, 64, device=dev)
    freq, _ = rb.rotary_frequencies(64, device=dev)
    assert rb.rotary(q, None, freq).shape == q.shape
    q = torch.zeros(2, 3, 5, 64, device=dev)
    zeros = lambda *s, **k: torch.zeros(*s, device=dev, **k)  # noqa: E731
    for exc, kw in [
            (TypeError, dict(freq=freq.float())), (ValueError, dict(freq=freq.cpu())),
            (TypeError, dict(positions=zeros(2, 5))), (TypeError, dict(k=q.bfloat16())),
            (ValueError, dict(positions=zeros(2, 4, dtype=torch.int32))),
            (ValueError, dict(k=q[:, :, :4])), (ValueError, dict(start=zeros(3).int())),
            (ValueError, dict(axis=zeros(31, dtype=torch.uint8))),
            (ValueError, dict(positions=zeros(2, 5).int(), start=zeros(2).int())),
            (rb.RehyatError, dict(freq=zeros(33, dtype=torch.float64))),
            (rb.RehyatError, dict(positions=zeros(5, 2, 5).int())),
            (rb.RehyatError, dict(q_out=q.as_strided((2, 3, 5, 64), (960, 64, 192, 1))))]:
        with pytest.raises(exc):
            rb.rotary(**dict(dict(q=q, k=None, freq=freq), **kw))
