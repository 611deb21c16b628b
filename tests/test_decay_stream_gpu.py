"""DecayStream: rotary positions, ragged prompts and single tokens run together as a session, against
the float64 oracle on each whole sequence; checkpoint and captured steps.

Tolerance: q and k are rounded to bf16 once more after their rotation, which adds two independent
roundings to the four of the attention itself: sqrt(6) * 2^-8 / sqrt(3) = 5.6e-3 in the mean square,
taken as 6e-3; the states see one of those two, 2^-8 / sqrt(3) = 2.3e-3.  fp32: 5e-6 for the
attention, 4e-7 for the rotation."""
import numpy as np
import pytest
import torch

from hybrid_softmax_linear_chunked_b200 import binding as rb
from hybrid_softmax_linear_chunked_b200.streaming import DecayStream
from oracle import sequence_oracle as SO

pytestmark = pytest.mark.gpu

B, H, HK, D, R = 3, 4, 2, 64, 32


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


def session(dev):
    g = torch.tensor([-0.7, -0.1, -0.01, 0.0], device=dev)
    freq, scale = rb.rotary_frequencies(R, scaling="ntk", factor=2.0, device=dev)
    return DecayStream(g, B=B, D=D, Hk=HK, freq=freq, rotary_scale=scale, interleaved=True)


def rows(g, dev, dtype, n):
    return [torch.randn(B, n, h, D, generator=g).to(dtype).to(dev).transpose(1, 2)
            for h in (H, HK, HK)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_session_matches_whole_sequences(dev, dtype):
    g = torch.Generator().manual_seed(0)
    sess = session(dev)
    seq = [[[] for _ in range(3)] for _ in range(B)]  # the rows each sequence has really seen
    outs = [[] for _ in range(B)]

    def keep(x, out, lengths):
        for b in range(B):
            for i in range(3):
                seq[b][i].append(f64(x[i][b, :, :lengths[b]]))
            outs[b].append(f64(out[b, :, :lengths[b]]))
            assert not out[b, :, lengths[b]:].any()

    for n, lengths in ((150, None), (70, [70, 0, 33])):
        x = rows(g, dev, dtype, n)
        L = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=dev)
        keep(x, sess.prompt(*x, lengths=L), lengths or [n] * B)
    for _ in range(5):
        x = rows(g, dev, dtype, 1)
        keep(x, sess.step(*x), [1] * B)
    rb.sync_status(dev)
    assert sess.seen.tolist() == [225, 155, 188]
    tol, tol_state = (6e-3, 2.3e-3) if dtype == torch.bfloat16 else (5.4e-6, 5.4e-6)
    for b in range(B):
        q, k, v = (np.concatenate(x, 1) for x in seq[b])
        got = np.concatenate(outs[b], 1)
        pos = np.arange(q.shape[1])
        q, k = (SO.rotary(x, pos, f64(sess.freq), sess.rotary_scale, True) for x in (q, k))
        for h in range(H):
            want, S = SO.decay_forward(q[h], k[h // 2], v[h // 2], float(sess.log_decay[h]),
                                       scale=D ** -0.5)
            assert np.linalg.norm(got[h] - want) <= tol * np.linalg.norm(want)
            assert np.linalg.norm(f64(sess.state[b, h]) - S) <= tol_state * np.linalg.norm(S)


def test_resume_and_captured_steps_give_the_same_bits(dev):
    g = torch.Generator().manual_seed(1)
    prompt, *steps = [rows(g, dev, torch.bfloat16, n) for n in (300, 1, 1, 1)]
    sess = session(dev)
    sess.prompt(*prompt)
    saved = sess.state_dict()
    want = [sess.step(*x).clone() for x in steps]
    again = session(dev)
    again.load_state_dict(saved)
    for x, y in zip(steps, want):
        assert torch.equal(again.step(*x), y)
    assert torch.equal(again.state, sess.state) and torch.equal(again.seen, sess.seen)
    # one captured step, replayed on new tokens
    token = [x.clone() for x in steps[0]]
    again.load_state_dict(saved)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = again.step(*token)
    again.load_state_dict(saved)
    for x, y in zip(steps, want):
        for t, s in zip(token, x):
            t.copy_(s)
        graph.replay()
        assert torch.equal(out, y)
    assert torch.equal(again.seen, sess.seen)
    again.reset()
    assert not again.state.any() and not again.seen.any()


def test_captured_prompt_beside_a_longer_one(dev):
    """A captured prompt writes only to memory it owns, also after a longer prompt of the session."""
    g = torch.Generator().manual_seed(3)
    short, other, long = [rows(g, dev, torch.bfloat16, n) for n in (300, 300, 2500)]
    sess, plain = session(dev), session(dev)
    sess.prompt(*short)
    x = [t.clone() for t in short]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = sess.prompt(*x)
    sess.prompt(*long)
    fill = [torch.full((1 << 18,), i, dtype=torch.int32, device=dev) for i in range(32)]
    for t, s in zip(x, other):
        t.copy_(s)
    graph.replay()
    want = [plain.prompt(*y) for y in (short, long, other)][-1]
    assert torch.equal(out, want) and torch.equal(sess.state, plain.state)
    assert torch.equal(sess.seen, plain.seen)
    assert all(bool((t == i).all()) for i, t in enumerate(fill))


def test_refuses(dev):
    g = torch.Generator().manual_seed(2)
    sess = session(dev)
    q, k, v = rows(g, dev, torch.bfloat16, 4)
    for bad in ((q[:2], k[:2], v[:2]), (q, q, q), (q, k, v[:, :, :3]), (q[0], k[0], v[0])):
        with pytest.raises(ValueError):
            sess.prompt(*bad)
    with pytest.raises(ValueError):
        sess.step(q, k, v)
    st = sess.state_dict()
    with pytest.raises(ValueError):
        DecayStream(sess.log_decay, B=B, D=D).load_state_dict(st)
