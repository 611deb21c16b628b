"""The sequence operators take no part in autograd, but a tensor that one of them writes to counts as
written: a graph that saved it for its backward pass refuses to run on the new values."""
import pytest
import torch

from hybrid_softmax_linear_chunked_b200 import binding as rb
from hybrid_softmax_linear_chunked_b200.streaming import DecayStream

pytestmark = pytest.mark.gpu

B, H, N, D = 2, 3, 5, 32


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from hybrid_softmax_linear_chunked_b200 import build
    build.build()
    rb.load()
    return torch.device("cuda", 0)


def writes(dev):
    """(name, shape, call that writes to a tensor of that shape)"""
    x = [torch.randn(B, H, N, D, device=dev) for _ in range(3)]
    one = [t[:, :, :1] for t in x]
    g = torch.full((H,), -0.1, device=dev)
    freq, _ = rb.rotary_frequencies(D, device=dev)
    rows, token, state = (B, H, N, D), (B, H, 1, D), (B, H, D, D)
    other = torch.zeros(state, device=dev)
    return [
        ("rotary in place", rows, lambda t: rb.rotary(t, None, freq, q_out=t)),
        ("rotary q_out", rows, lambda t: rb.rotary(x[0], x[1], freq, q_out=t)),
        ("rotary k_out", rows, lambda t: rb.rotary(x[0], x[1], freq, k_out=t)),
        ("prompt out", rows, lambda t: rb.decay_forward(*x, g, out=t)),
        ("prompt final state", state, lambda t: rb.decay_forward(*x, g, final_state=t)),
        ("prompt state in place", state,
         lambda t: rb.decay_forward(*x, g, state=t, final_state=t)),
        ("step state", state, lambda t: rb.decay_step(*one, g, t)),
        ("step out", token, lambda t: rb.decay_step(*one, g, other, out=t)),
    ]


def test_written_tensors_that_a_graph_saved(dev):
    silent = []
    for name, shape, call in writes(dev):
        leaf = torch.randn(shape, device=dev, requires_grad=True)
        saved = leaf * 1.0
        loss = (saved * saved).sum()  # keeps `saved`
        call(saved)
        try:
            loss.backward()
            silent.append(name)
        except RuntimeError as e:
            assert "modified by an inplace operation" in str(e)
    assert not silent


def test_inputs_are_not_written_and_inference_tensors_are_taken(dev):
    x = [torch.randn(B, H, N, D, device=dev) for _ in range(4)]
    g = torch.full((H,), -0.1, device=dev)
    S = torch.randn(B, H, D, D, device=dev)
    before = [t._version for t in (*x, g, S)]
    rb.decay_forward(*x[:3], g, state=S, final_state=True)
    rb.decay_backward(*x[:3], g, x[3], state=S)
    rb.rotary(x[0], x[1], rb.rotary_frequencies(D, device=dev)[0])
    assert [t._version for t in (*x, g, S)] == before
    with torch.inference_mode():
        sess = DecayStream(g, B=B, D=D)
        out = sess.prompt(*x[:3])
        one = sess.step(*(t[:, :, :1] for t in x[:3]))
        assert out.is_inference() and bool(torch.isfinite(one).all())
