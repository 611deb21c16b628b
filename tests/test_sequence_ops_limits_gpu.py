"""Sequence operators at the limits: offsets past 32 bits, the checking build, a head's NaN and
infinities staying where they are, states in place, and odd batches of single tokens.

Tolerances as derived in test_decay_gpu: bf16 5e-3 (four roundings), fp32 states of bf16 rows 1e-5."""
import math

import numpy as np
import pytest
import torch

from hybrid_softmax_linear_chunked_b200 import binding as rb
from hybrid_softmax_linear_chunked_b200 import build
from oracle import sequence_oracle as SO

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    rb.load()
    return torch.device("cuda", 0)


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def rel(got, want):
    return float(np.linalg.norm(f64(got) - want) / np.linalg.norm(want))


def test_offsets_past_32_bits(dev):
    """Two heads more than 2^31 elements apart (and a state pool past 2^31 elements)."""
    n, D, far = 200, 128, (1 << 31) + 1024
    big = torch.empty(far + 4 * n * D, dtype=torch.bfloat16, device=dev)
    g = torch.Generator().manual_seed(1)
    views = []
    for i in range(4):  # q, k, v and the output, each with its two heads far apart
        t = big.as_strided((1, 2, n, D), (0, far, D, 1), i * n * D)
        if i < 3:
            t.copy_(torch.randn(1, 2, n, D, generator=g).to(torch.bfloat16))
        views.append(t)
    q, k, v, out = views
    decay = torch.tensor([-0.1, -0.01], device=dev)
    _, last = rb.decay_forward(q, k, v, decay, scale=0.1, final_state=True, out=out)
    grads = rb.decay_backward(q, k, v, decay, q, scale=0.1)
    freq, _ = rb.rotary_frequencies(D, device=dev)
    turned = rb.rotary(q, None, freq, start=3)
    for h in range(2):
        want, S = SO.decay_forward(f64(q[0, h]), f64(k[0, h]), f64(v[0, h]), float(decay[h]),
                                   scale=0.1)
        assert rel(out[0, h], want) <= 5e-3 and rel(last[0, h], S) <= 1e-5
        dq, dk, dv, _ = SO.decay_backward(f64(q[0, h]), f64(k[0, h]), f64(v[0, h]),
                                          float(decay[h]), f64(q[0, h]), scale=0.1)
        for name, w in (("dq", dq), ("dk", dk), ("dv", dv)):
            assert rel(grads[name][0, h], w) <= 5e-3
        want = SO.rotary(f64(q[0, h]), np.arange(n) + 3, f64(freq))
        assert rel(turned[0, h], want) <= 2.0 ** -8
    del big, views, q, k, v, out, turned, grads
    torch.cuda.empty_cache()
    pool, D = (1 << 31) // (128 * 128) + 2, 128  # the last two states lie past 2^31 elements
    state = torch.empty(pool, 1, D, D, device=dev)
    x = torch.randn(2, 1, 1, D, generator=g).to(dev)
    state[-2:] = 0
    slots = torch.tensor([pool - 1, pool - 2], dtype=torch.int32, device=dev)
    o = rb.decay_step(x, x, x, decay[:1], state, slots=slots)
    for b in range(2):
        want, S = SO.decay_forward(f64(x[b, 0]), f64(x[b, 0]), f64(x[b, 0]), -0.1)
        assert rel(o[b, 0], want) <= 5e-6 and rel(state[pool - 1 - b, 0], S) <= 5e-6


def calls(dev):
    g = torch.Generator().manual_seed(2)
    B, H, Hk, N, D = 2, 4, 2, 700, 72
    q, do = (torch.randn(B, N, H, D, generator=g).to(torch.bfloat16).to(dev).transpose(1, 2)
             for _ in range(2))
    k, v = (torch.randn(B, N, Hk, D, generator=g).to(torch.bfloat16).to(dev).transpose(1, 2)
            for _ in range(2))
    decay = torch.tensor([-0.5, -0.1, -0.01, 0.0], device=dev)
    L = torch.tensor([700, 333], dtype=torch.int32, device=dev)
    S = torch.randn(B, H, D, D, generator=g).to(dev)
    out, last = rb.decay_forward(q, k, v, decay, scale=0.1, lengths=L, state=S, final_state=True)
    grads = rb.decay_backward(q, k, v, decay, do, scale=0.1, lengths=L, state=S, dfinal=last)
    plain = rb.decay_forward(q[:, :, :130], k[:, :, :130], v[:, :, :130], decay)
    one = rb.decay_step(q[:, :, :1], k[:, :, :1], v[:, :, :1], decay, last)
    freq, _ = rb.rotary_frequencies(64, device=dev)
    qr, kr = rb.rotary(q, k, freq, start=5)
    rb.sync_status(dev)  # raises on a failed check
    return [out, last, plain, one, qr, kr, *grads.values()]


def test_the_checking_build_agrees(dev):
    """The debug-bounds library checks every tile coordinate of the bf16 kernels: no check fails and
    the results are the normal build's, bit for bit."""
    want = calls(dev)
    rb.use_library(build.build(debug_bounds=True))
    try:
        got = calls(dev)
    finally:
        rb.use_library(build.build())
    for x, y in zip(got, want):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_bad_values_stay_in_their_head_and_after_their_row(dev, dtype):
    """NaN and infinity in one head's rows reach no other head and no earlier chunk of 128 rows, and
    are not lost from the rows after them; a NaN decay spoils its head alone."""
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(1, 3, 600, 64, generator=g).to(dtype).to(dev) for _ in range(3))
    decay = torch.tensor([-0.05, -0.05, -0.05], device=dev)
    clean = rb.decay_forward(q, k, v, decay)
    v[0, 1, 300, 5] = math.nan
    k[0, 1, 310, 7] = math.inf
    out = rb.decay_forward(q, k, v, decay)
    assert torch.equal(out[0, [0, 2]], clean[0, [0, 2]])
    assert torch.equal(out[0, 1, :256], clean[0, 1, :256])
    assert bool(torch.isnan(out[0, 1, 300:, 5]).all())
    decay[2] = math.nan
    out = rb.decay_forward(q, k, v, decay)
    assert torch.equal(out[0, 0], clean[0, 0]) and bool(torch.isnan(out[0, 2]).all())


def test_many_small_sequences(dev):
    """More sequences than SMs, all lengths from 0 to 130, in one padded batch."""
    B, N, D = 393, 131, 32
    g = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn(B, 1, N, D, generator=g).to(torch.bfloat16).to(dev) for _ in range(3))
    lengths = [(i * 37) % (N + 1) for i in range(B)]
    L = torch.tensor(lengths, dtype=torch.int32, device=dev)
    decay = torch.tensor([-0.03], device=dev)
    out, last = rb.decay_forward(q, k, v, decay, lengths=L, final_state=True)
    for b in range(0, B, 29):
        n = lengths[b]
        want, S = SO.decay_forward(f64(q[b, 0, :n]), f64(k[b, 0, :n]), f64(v[b, 0, :n]), -0.03)
        assert not out[b, 0, n:].any()
        if n:
            assert rel(out[b, 0, :n], want) <= 5e-3 and rel(last[b, 0], S) <= 1e-5
        else:
            assert not last[b].any()
