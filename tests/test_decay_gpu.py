"""Linear attention with a decay per head on the GPU: prompts, gradients and single tokens against
the float64 recurrence.

Tolerances (relative 2-norm), from the roundings each path makes:
 * bf16 outputs and gradients: at most four independent roundings to bf16 (weighted rows or scores,
   the state the rows read, the output), each within half a step 2^-8 and so 2^-8 / sqrt(3) in the
   mean square: sqrt(4) * 2^-8 / sqrt(3) = 4.5e-3, taken as 5e-3.
 * fp32 states of bf16 inputs: rows in two bf16 parts leave at most 2^-16 of a term, 2^-16 / sqrt(3)
   in the mean square = 8.8e-6, and the fp32 sums below: 1e-5.
 * fp32: K-term sums of fp32 products, errors growing as sqrt(K) 2^-24; K <= 2500 + 128 here gives
   3e-6, the powers of the decay add 1e-6: 5e-6.
One value may be off by 8 of those in units of the result's root mean square, or of itself."""
import math

import numpy as np
import pytest
import torch

from hybrid_softmax_linear_chunked_b200 import binding as rb
from oracle import sequence_oracle as SO

pytestmark = pytest.mark.gpu

REL = {torch.bfloat16: 5e-3, torch.float32: 5e-6}
REL_STATE = {torch.bfloat16: 1e-5, torch.float32: 5e-6}


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


def close(got, want, tol, what):
    got, want = f64(got) if isinstance(got, torch.Tensor) else got, np.asarray(want)
    assert got.shape == want.shape, what
    assert np.isfinite(got).all(), what + ": non-finite"
    norm = np.linalg.norm(want)
    if norm == 0:
        assert (got == 0).all(), what
        return
    rel = np.linalg.norm(got - want) / norm
    rms = norm / math.sqrt(want.size)
    big = (np.abs(got - want) / np.maximum(rms, np.abs(want))).max()
    assert rel <= tol and big <= 8 * tol, f"{what}: rel-L2 {rel:.3e}, largest {big:.3e} (tol {tol})"


def rows(g, dev, dtype, B, heads, N, D, layout="bhnd"):
    x = torch.randn(B, heads, N, D, generator=g).to(dtype)
    if layout == "bhnd":
        return x.to(dev)
    if layout == "bnhd":
        return x.transpose(1, 2).contiguous().to(dev).transpose(1, 2)
    pad = torch.full((B, heads + 1, N, D + 8), 7.0, dtype=dtype, device=dev)  # a slice of more
    pad[:, 1:, :, 8:] = x.to(dev)
    return pad[:, 1:, :, 8:]


def problem(dev, dtype, B=1, H=2, Hk=None, N=64, D=64, state=False, layout="bhnd", decays=None,
            seed=0):
    g = torch.Generator().manual_seed(seed)
    Hk = Hk or H
    p = dict(q=rows(g, dev, dtype, B, H, N, D, layout), k=rows(g, dev, dtype, B, Hk, N, D, layout),
             v=rows(g, dev, dtype, B, Hk, N, D, layout),
             dout=rows(g, dev, dtype, B, H, N, D, layout))
    p["S0"] = torch.randn(B, H, D, D, generator=g).to(dev) if state else None
    p["dS"] = torch.randn(B, H, D, D, generator=g).to(dev) if state else None
    if decays is None:
        decays = [math.log1p(-2.0 ** -(1 + 9 * h / max(H - 1, 1))) for h in range(H)]
    p["g"] = torch.tensor(decays, dtype=torch.float32, device=dev)
    return p


def head(p, name, b, h, n):
    t = p[name]
    return f64(t[b, h * t.shape[1] // p["q"].shape[1], :n])


def check_forward(p, out, last, scale, lengths=None, what=""):
    B, H, N, D = p["q"].shape
    want, wantS = np.zeros((B, H, N, D)), np.zeros((B, H, D, D))
    for b in range(B):
        n = N if lengths is None else lengths[b]
        for h in range(H):
            S0 = None if p["S0"] is None else f64(p["S0"][b, h])
            want[b, h, :n], wantS[b, h] = SO.decay_forward(
                head(p, "q", b, h, n), head(p, "k", b, h, n), head(p, "v", b, h, n),
                float(p["g"][h]), S0, scale)
    dt = p["q"].dtype
    close(out, want, REL[dt], what + " out")
    if last is not None:
        close(last, wantS, REL_STATE[dt], what + " state")


def check_backward(p, got, scale, lengths=None, what=""):
    B, H, N, D = p["q"].shape
    Hk = p["k"].shape[1]
    want = {"dq": np.zeros((B, H, N, D)), "dk": np.zeros((B, Hk, N, D)),
            "dv": np.zeros((B, Hk, N, D)), "dstate": np.zeros((B, H, D, D))}
    for b in range(B):
        n = N if lengths is None else lengths[b]
        for h in range(H):
            S0, dS = (None if p[x] is None else f64(p[x][b, h]) for x in ("S0", "dS"))
            r = SO.decay_backward(head(p, "q", b, h, n), head(p, "k", b, h, n),
                                  head(p, "v", b, h, n), float(p["g"][h]),
                                  head(p, "dout", b, h, n), S0, dS, scale)
            hk = h * Hk // H
            want["dq"][b, h, :n] = r[0]
            want["dk"][b, hk, :n] += r[1]
            want["dv"][b, hk, :n] += r[2]
            want["dstate"][b, h] = r[3]
    dt = p["q"].dtype
    assert ("dstate" in got) == (p["S0"] is not None)
    for n, x in got.items():
        close(x, want[n], REL_STATE[dt] if n == "dstate" else REL[dt], f"{what} {n}")


SHAPES = [  # dtype, B, H, Hk, N, D, state, layout
    (torch.float32, 1, 1, 1, 1, 8, False, "bhnd"),
    (torch.float32, 2, 4, 2, 65, 40, True, "bnhd"),
    (torch.float32, 1, 2, 1, 129, 128, True, "slice"),
    (torch.float32, 1, 3, 3, 1000, 96, False, "bhnd"),
    (torch.float32, 1, 1, 1, 2500, 32, True, "bhnd"),
    (torch.bfloat16, 1, 1, 1, 1, 128, False, "bhnd"),
    (torch.bfloat16, 1, 2, 2, 2, 128, True, "bhnd"),
    (torch.bfloat16, 2, 4, 1, 63, 64, True, "bnhd"),
    (torch.bfloat16, 1, 2, 2, 127, 128, False, "slice"),
    (torch.bfloat16, 1, 2, 2, 128, 128, True, "bhnd"),
    (torch.bfloat16, 3, 2, 1, 129, 128, True, "bnhd"),
    (torch.bfloat16, 1, 3, 3, 385, 72, True, "bhnd"),
    (torch.bfloat16, 1, 2, 2, 2500, 128, True, "bnhd"),
    (torch.bfloat16, 1, 1, 1, 640, 8, False, "bhnd"),
]


def ident(s):
    return "-".join(str(x).replace("torch.", "") for x in s)


@pytest.mark.parametrize("shape", SHAPES, ids=ident)
def test_prompt_and_gradients(dev, shape):
    dt, B, H, Hk, N, D, state, layout = shape
    p = problem(dev, dt, B, H, Hk, N, D, state, layout, seed=N)
    scale = D ** -0.5
    kw = dict(scale=scale, state=p["S0"])
    out, last = rb.decay_forward(p["q"], p["k"], p["v"], p["g"], final_state=True, **kw)
    only = rb.decay_forward(p["q"], p["k"], p["v"], p["g"], **kw)
    grads = rb.decay_backward(p["q"], p["k"], p["v"], p["g"], p["dout"], dfinal=p["dS"], **kw)
    rb.sync_status(dev)
    check_forward(p, out, last, scale)
    check_forward(p, only, None, scale, what="without the state")
    check_backward(p, grads, scale)


@pytest.mark.parametrize("dtype,H,N", [(torch.bfloat16, 150, 3100), (torch.bfloat16, 74, 4700),
                                       (torch.float32, 150, 1000)], ids=str)
def test_long_segments(dev, dtype, H, N):
    """So many heads that a segment is 18 to 25 chunks long; three heads checked."""
    heads = [0, H // 2, H - 1]
    decays = [0.0 if h == H // 2 else -2.0 ** (-1 - h * 10 / H) for h in range(H)]
    p = problem(dev, dtype, 1, H, H, N, 32, True, decays=decays, seed=19)
    kw = dict(scale=0.125, state=p["S0"])
    out, last = rb.decay_forward(p["q"], p["k"], p["v"], p["g"], final_state=True, **kw)
    g = rb.decay_backward(p["q"], p["k"], p["v"], p["g"], p["dout"], dfinal=p["dS"], **kw)
    no_state = rb.decay_backward(p["q"], p["k"], p["v"], p["g"], p["dout"], scale=0.125)
    rb.sync_status(dev)
    cut = {n: (x[heads] if n == "g" else x[:, heads]) for n, x in p.items()}
    check_forward(cut, out[:, heads], last[:, heads], 0.125)
    check_backward(cut, {n: x[:, heads] for n, x in g.items()}, 0.125)
    cut["S0"] = cut["dS"] = None
    check_backward(cut, {n: x[:, heads] for n, x in no_state.items()}, 0.125)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("N", [130, 700])
def test_padded_batch(dev, dtype, N):
    """Lengths of zero, one, a tile's border, past the tensor and below zero; NaN in the padding."""
    lengths = [0, 1, 128, N - 1, N + 50, -3]
    B = len(lengths)
    p = problem(dev, dtype, B, 4, 2, N, 128, True, seed=3)
    n = [min(max(x, 0), N) for x in lengths]
    for b in range(B):
        for name in ("q", "k", "v", "dout"):
            p[name][b, :, n[b]:] = math.nan
    L = torch.tensor(lengths, dtype=torch.int32, device=dev)
    kw = dict(scale=0.1, lengths=L, state=p["S0"])
    out, last = rb.decay_forward(p["q"], p["k"], p["v"], p["g"], final_state=True, **kw)
    g = rb.decay_backward(p["q"], p["k"], p["v"], p["g"], p["dout"], dfinal=p["dS"], **kw)
    rb.sync_status(dev)
    check_forward(p, out, last, 0.1, n)
    check_backward(p, g, 0.1, n)
    assert torch.equal(last[0], p["S0"][0])  # no rows: the state as it was


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_extreme_decays(dev, dtype):
    """L = 0 (each row sees itself alone), far below fp32's range, and 1 (plain linear attention)."""
    p = problem(dev, dtype, 1, 4, 4, 400, 64, True, decays=[-math.inf, -90.0, -3.0, 0.0], seed=5)
    out, last = rb.decay_forward(p["q"], p["k"], p["v"], p["g"], state=p["S0"], scale=0.125,
                                 final_state=True)
    g = rb.decay_backward(p["q"], p["k"], p["v"], p["g"], p["dout"], state=p["S0"],
                          dfinal=p["dS"], scale=0.125)
    check_forward(p, out, last, 0.125)
    check_backward(p, g, 0.125)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_no_rows(dev, dtype):
    p = problem(dev, dtype, 2, 2, 1, 0, 64, True)
    out, last = rb.decay_forward(p["q"], p["k"], p["v"], p["g"], state=p["S0"], final_state=True)
    g = rb.decay_backward(p["q"], p["k"], p["v"], p["g"], p["dout"], state=p["S0"],
                          dfinal=p["dS"])
    assert out.shape == (2, 2, 0, 64) and torch.equal(last, p["S0"])
    assert torch.equal(g["dstate"], p["dS"]) and g["dk"].shape == (2, 1, 0, 64)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_gradients_are_the_differences_of_the_prompt(dev, dtype):
    """The loss is linear in each argument, so the difference along a direction that the type holds
    exactly (a power of two on one row) has no truncation error, only the outputs' roundings."""
    p = problem(dev, torch.float32, 1, 2, 2, 150, 64, False, seed=9)
    p = {n: (x.to(dtype) if n in ("q", "k", "v", "dout") else x) for n, x in p.items()}

    def loss(**kw):
        a = dict(p, **kw)
        out = rb.decay_forward(a["q"], a["k"], a["v"], a["g"], scale=0.125)
        return float((out.double() * p["dout"].double()).sum())

    g = rb.decay_backward(p["q"], p["k"], p["v"], p["g"], p["dout"], scale=0.125)
    for n in ("q", "k", "v"):
        d = torch.zeros_like(p[n])
        d[0, 1, 40] = 64.0
        up, dn = loss(**{n: d}), loss(**{n: -d})
        got = float((g["d" + n].double() * d.double()).sum())
        size = float((g["d" + n][0, 1, 40].double() * 64).norm()) * math.sqrt(64)
        assert abs((up - dn) / 2 - got) <= 4 * REL[dtype] * size


@pytest.mark.parametrize("dtype,B,H,Hk,D", [
    (torch.bfloat16, 1, 12, 12, 128), (torch.bfloat16, 5, 4, 2, 64), (torch.float32, 3, 2, 1, 40),
    (torch.float32, 2, 3, 3, 128), (torch.bfloat16, 33, 1, 1, 8)], ids=str)
def test_steps_go_on_from_a_prompt(dev, dtype, B, H, Hk, D):
    """A prompt and then tokens one at a time give what the whole sequence gives."""
    N, n0 = 9, 5
    p = problem(dev, dtype, B, H, Hk, N, D, True, layout="bnhd", seed=11)
    cut = lambda a, b: [p[x][:, :, a:b] for x in "qkv"]  # noqa: E731
    S = p["S0"].clone()
    outs = [rb.decay_forward(*cut(0, n0), p["g"], state=S, final_state=S, scale=0.5)[0]]
    for i in range(n0, N):
        outs.append(rb.decay_step(*cut(i, i + 1), p["g"], S, scale=0.5))
    rb.sync_status(dev)
    check_forward(p, torch.cat(outs, 2), S, 0.5)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_step_slots(dev, dtype):
    """Slots in any order, idle entries, a slot listed three times, and one past the pool."""
    slots, pool, H, D = [4, -1, 2, 4, 0, 7, 4, -9], 6, 3, 64
    B = len(slots)
    p = problem(dev, dtype, B, H, H, 1, D, seed=13)
    g = torch.Generator().manual_seed(14)
    state = torch.randn(pool, H, D, D, generator=g).to(dev)
    want, before = f64(state), state.clone()
    out = torch.full((B, H, 1, D), math.nan, dtype=dtype, device=dev)
    wout = np.zeros(out.shape)
    for b, s in enumerate(slots):
        for h in range(H):
            if 0 <= s < pool:
                wout[b, h], want[s, h] = SO.decay_forward(
                    head(p, "q", b, h, 1), head(p, "k", b, h, 1), head(p, "v", b, h, 1),
                    float(p["g"][h]), want[s, h], 0.5)
    rb.decay_step(p["q"], p["k"], p["v"], p["g"], state, scale=0.5, out=out,
                  slots=torch.tensor(slots, dtype=torch.int32, device=dev))
    with pytest.raises(rb.RehyatError) as e:
        rb.sync_status(dev)
    assert e.value.status == -8 and "value 7" in str(e.value)
    rb.sync_status(dev)  # the report was taken
    close(out, wout, REL[dtype], "out")
    close(state, want, 5e-6, "states")
    for s in (1, 3, 5):
        assert torch.equal(state[s], before[s])
    for b in (1, 5, 7):
        assert not out[b].any()


def test_writes_stay_inside_the_output(dev):
    """A ragged last tile written through strides leaves the rows and columns around it alone."""
    N, D = 130, 72
    p = problem(dev, torch.bfloat16, 1, 2, 2, N, D, seed=15)
    room = torch.full((1, 4, N + 8, D + 16), 3.0, dtype=torch.bfloat16, device=dev)
    out = room[:, 1:3, 4:N + 4, 8:D + 8]
    assert rb.decay_forward(p["q"], p["k"], p["v"], p["g"], scale=0.1, out=out) is out
    check_forward(p, out, None, 0.1)
    kept = room.clone()
    kept[:, 1:3, 4:N + 4, 8:D + 8] = 3.0
    assert bool((kept == 3.0).all())


def test_calls_repeat_bit_for_bit_and_replay_from_graphs(dev):
    """Eager calls, another stream and replays of two captured graphs agree bit for bit, with the
    inputs changed between replays."""
    p = problem(dev, torch.bfloat16, 2, 4, 2, 700, 128, True, seed=17)
    lengths = torch.tensor([700, 333], dtype=torch.int32, device=dev)
    S = p["S0"].clone()
    size = rb.decay_workspace_size(2, 4, 2, 700, 128, True)
    ws = torch.empty(size, dtype=torch.uint8, device=dev)  # shared by every call below

    def step():
        S.copy_(p["S0"])
        out, _ = rb.decay_forward(p["q"], p["k"], p["v"], p["g"], scale=0.1, lengths=lengths,
                                  state=S, final_state=S, workspace=ws)
        g = rb.decay_backward(p["q"], p["k"], p["v"], p["g"], p["dout"], scale=0.1,
                              lengths=lengths, state=p["S0"], dfinal=S, workspace=ws)
        one = rb.decay_step(*(p[x][:, :, :1] for x in "qkv"), p["g"], S, scale=0.1)
        return [out, *g.values(), one, S]

    eager = [x.clone() for x in step()]
    again = [x.clone() for x in step()]
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        other = [x.clone() for x in step()]
    torch.cuda.current_stream(dev).wait_stream(side)
    torch.cuda.synchronize(dev)
    for x, y, z in zip(eager, again, other):
        assert torch.equal(x, y) and torch.equal(x, z)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = step()
        graphs.append((graph, res))
    for graph, res in graphs:
        graph.replay()
        torch.cuda.synchronize(dev)
        for x, y in zip(eager, res):
            assert torch.equal(x, y)
    p["q"].mul_(2.0)  # exact: outputs double, the state does not change
    lengths.copy_(torch.tensor([600, 1], dtype=torch.int32))
    want = [x.clone() for x in step()]
    for graph, res in graphs:
        graph.replay()
        torch.cuda.synchronize(dev)
        for x, y in zip(want, res):
            assert torch.equal(x, y)


def test_calls_at_once(dev):
    """Calls on three streams, not ordered to one another, give what they give one by one."""
    shapes = [(torch.bfloat16, 2, 6, 3, 2000, 128), (torch.bfloat16, 1, 3, 3, 3000, 64),
              (torch.float32, 2, 4, 2, 500, 64)]
    probs = [problem(dev, dt, B, H, Hk, N, D, True, seed=30 + i)
             for i, (dt, B, H, Hk, N, D) in enumerate(shapes)]
    lengths = [torch.tensor([N // 3, N][:B], dtype=torch.int32, device=dev)
               for _, B, _, _, N, _ in shapes]

    def calls(i):
        p, kw = probs[i], dict(scale=0.1, lengths=lengths[i])
        x = (p["q"], p["k"], p["v"], p["g"])
        out, S = rb.decay_forward(*x, state=p["S0"], final_state=True, **kw)
        return [out, S, *rb.decay_backward(*x, p["dout"], state=p["S0"], dfinal=S, **kw).values()]

    want = [calls(i) for i in range(3)]
    torch.cuda.synchronize(dev)
    streams = [torch.cuda.Stream(dev) for _ in shapes]
    got = [[] for _ in shapes]
    for _ in range(4):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(calls(i))
    torch.cuda.synchronize(dev)
    rb.sync_status(dev)
    for w, runs in zip(want, got):
        for run in runs:
            assert all(torch.equal(x, y) for x, y in zip(w, run))


def test_refuses(dev):
    p = problem(dev, torch.bfloat16, 2, 4, 2, 16, 64, True)
    q, k, v, g = (p[x] for x in ("q", "k", "v", "g"))
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev)  # noqa: E731
    for exc, kw in [
            (TypeError, dict(k=k.float())), (TypeError, dict(log_decay=g.double())),
            (ValueError, dict(v=v[:, :, :8])), (ValueError, dict(log_decay=g[:2])),
            (ValueError, dict(lengths=i32(3))), (TypeError, dict(lengths=i32(2).long())),
            (ValueError, dict(state=p["S0"][:1])), (ValueError, dict(v=v.cpu())),
            (ValueError, dict(q=q.transpose(2, 3).contiguous().transpose(2, 3))),
            (ValueError, dict(state=p["S0"].transpose(2, 3))),
            (ValueError, dict(workspace=torch.empty(1 << 20, device=dev))),
            (rb.RehyatError, dict(k=k[:, :1].expand(2, 2, 16, 64))),
            (rb.RehyatError, dict(q=torch.zeros(2, 4, 16 * 64 + 8, dtype=q.dtype, device=dev)[
                :, :, 4:-4].view(2, 4, 16, 64)))]:
        with pytest.raises(exc):
            rb.decay_forward(**dict(dict(q=q, k=k, v=v, log_decay=g), **kw))
    one = [x[:, :, :1] for x in (q, k, v)]
    for kw in (dict(state=p["S0"][:1]), dict(slots=i32(1)), dict(out=q)):
        with pytest.raises(ValueError):
            rb.decay_step(*one, g, **dict(dict(state=p["S0"]), **kw))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("B,H,Hk,N", [(33, 1, 1, 1000), (100, 2, 1, 500), (256, 1, 1, 300)], ids=str)
def test_padded_batches_of_many_sequences(dev, dtype, B, H, Hk, N):
    """As many sequences as one warp finds the segments of, several to a lane: long ones, runs of
    empty ones (the first 32 among them, and the last), one row, and a chunk's border."""
    lengths = [0] * 32 + [(N, 1, 128, 129, 64, 0, 0, 0, N - 1, 300)[i % 10] for i in range(B - 32)]
    if B > 64:
        lengths[60:100] = [0] * 40
        lengths[2], lengths[-1] = N, 0
    n = [min(x, N) for x in lengths]
    p = problem(dev, dtype, B, H, Hk, N, 32, True, seed=40 + B, decays=[-0.03, -0.2][:H])
    L = torch.tensor(lengths, dtype=torch.int32, device=dev)
    kw = dict(scale=0.2, lengths=L, state=p["S0"])
    out, last = rb.decay_forward(p["q"], p["k"], p["v"], p["g"], final_state=True, **kw)
    only = rb.decay_forward(p["q"], p["k"], p["v"], p["g"], **kw)
    g = rb.decay_backward(p["q"], p["k"], p["v"], p["g"], p["dout"], dfinal=p["dS"], **kw)
    rb.sync_status(dev)
    want = {x: [] for x in ("out", "dq", "dk", "dv", "last", "dstate")}
    for b in range(B):
        kv = [np.zeros((Hk, n[b], 32)) for _ in range(2)]
        for h in range(H):
            x = [head(p, c, b, h, n[b]) for c in ("q", "k", "v", "dout")]
            S0, dS, gh = f64(p["S0"][b, h]), f64(p["dS"][b, h]), float(p["g"][h])
            o, S = SO.decay_forward(*x[:3], gh, S0, 0.2)
            dq, dk, dv, d0 = SO.decay_backward(*x[:3], gh, x[3], S0, dS, 0.2)
            kv[0][h * Hk // H] += dk
            kv[1][h * Hk // H] += dv
            for name, w in (("out", o), ("dq", dq), ("last", S), ("dstate", d0)):
                want[name].append(w)
        want["dk"] += list(kv[0])
        want["dv"] += list(kv[1])
    for name, x in (("out", out), ("out", only), ("dq", g["dq"]), ("dk", g["dk"]), ("dv", g["dv"])):
        # padding is zero and left out: its zeros would shrink the root mean square that one value's
        # error is measured in (of 33,000 rows 1,000 are valid: by sqrt(33))
        assert not any(bool(x[b, :, n[b]:].any()) for b in range(B)), name
        rows_ = torch.cat([x[b, h, :n[b]] for b in range(B) for h in range(x.shape[1])])
        close(rows_, np.concatenate(want[name]), REL[dtype], name)
    for name, x in (("last", last), ("dstate", g["dstate"])):
        close(x, np.stack(want[name]).reshape(x.shape), REL_STATE[dtype], name)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("H,Hk,N", [(2, 1, 700), (2, 2, 50), (150, 150, 300)], ids=str)
@pytest.mark.parametrize("have", ["S0", "dS"])
def test_gradients_with_one_of_the_states(dev, dtype, H, Hk, N, have):
    """A state before without a gradient of the last, and the other way round: only one of the passes
    has something carried in (one segment a sequence, or several)."""
    p = problem(dev, dtype, 1, H, Hk, N, 64, True, seed=50 + N)
    for name in ("S0", "dS"):
        if name != have:
            p[name] = None
    g = rb.decay_backward(p["q"], p["k"], p["v"], p["g"], p["dout"], scale=0.125, state=p["S0"],
                          dfinal=p["dS"])
    rb.sync_status(dev)
    check_backward(p, g, 0.125)
