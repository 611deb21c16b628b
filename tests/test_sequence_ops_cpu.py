"""Sequence operators on the host: what the library and the binding refuse before anything is
enqueued, the rotary frequency tables, and the kernel's angle arithmetic."""
import ctypes
import math

import numpy as np
import pytest
import torch

from hybrid_softmax_linear_chunked_b200 import binding as rb
from hybrid_softmax_linear_chunked_b200 import build

FAKE = 0x10000  # 16-byte aligned, never dereferenced: checks come first
B, H, HK, N, D = 2, 4, 2, 40, 64


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return rb.load()


def rows(heads, p=FAKE, n=N, d=D):
    return (p, heads * n * d, n * d, d)


def decay(lib, call="forward", **kw):
    a = dict(B=B, H=H, Hk=HK, N=N, D=D, pool=B, dtype=rb.REHYAT_BF16, q=rows(H), k=rows(HK),
             v=rows(HK), out=rows(H), dout=rows(H), dq=rows(H), dk=rows(HK), dv=rows(HK), g=FAKE,
             lengths=0, S0=0, last=FAKE, dlast=0, dS0=0, state=FAKE, slots=0, ws=FAKE,
             ws_bytes=1 << 40, scale=1.0)
    a.update(kw)
    order = {"forward": "B H Hk N D dtype q k v out g lengths S0 last ws ws_bytes scale",
             "backward": "B H Hk N D dtype q k v dout dq dk dv g lengths S0 dlast dS0 ws ws_bytes "
                         "scale",
             "step": "B H Hk D pool dtype q k v out g state slots scale"}[call].split()
    flat = [y for n in order for y in (a[n] if isinstance(a[n], tuple) else (a[n],))]
    return getattr(lib, "rehyat_decay_" + call)(
        getattr(rb, "_DECAY_" + call.upper()).pack(*flat), None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), -1), (dict(Hk=3), -1), (dict(Hk=0), -1), (dict(N=-1), -1), (dict(D=0), -1),
    (dict(D=60), -2), (dict(D=136), -2), (dict(B=70000), -2), (dict(H=40000, Hk=40000), -2),
    (dict(scale=math.nan), -1), (dict(scale=math.inf), -1), (dict(dtype=7), -3),
    (dict(q=rows(H, 0)), -1), (dict(v=rows(HK, FAKE + 8)), -7), (dict(g=0), -1),
    (dict(S0=FAKE + 4), -7), (dict(last=FAKE + 8), -7),
    (dict(q=(FAKE, H * N * D, N * D, D - 8)), -1),     # rows overlap
    (dict(k=(FAKE, HK * N * D, 0, D)), -1),            # heads expanded
    (dict(k=(FAKE, HK * N * D + 4, N * D, D)), -7),    # 8-byte stride in bf16
    (dict(k=(FAKE, 1 << 40, N * D, D)), -1),
    (dict(ws_bytes=0), -4), (dict(ws=0), -4), (dict(ws=FAKE + 8), -7),
])
def test_decay_forward_refuses(lib, kw, status):
    assert decay(lib, **kw) == status
    assert lib.rehyat_last_error().decode()


@pytest.mark.parametrize("kw,status", [
    (dict(Hk=3), -1), (dict(D=12), -2), (dict(dout=rows(H, 0)), -1),
    (dict(dk=rows(HK, 0)), -1), (dict(dv=rows(HK, FAKE + 2)), -7), (dict(ws_bytes=64), -4),
])
def test_decay_backward_refuses(lib, kw, status):
    assert decay(lib, "backward", **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(state=0), -1), (dict(g=0), -1), (dict(pool=0), -1), (dict(pool=1), -1),
    (dict(state=FAKE + 8), -7), (dict(out=rows(H, 0)), -1), (dict(D=4), -2), (dict(dtype=2), -3),
])
def test_decay_step_refuses(lib, kw, status):
    assert decay(lib, "step", **kw) == status


def test_written_tensors_are_no_other_argument(lib):
    """Refused with the message that says so; out of the way of every input's own checks."""
    at = lambda heads, i: rows(heads, FAKE + (i << 16))  # noqa: E731
    apart = dict(q=at(H, 1), k=at(HK, 2), v=at(HK, 3), out=at(H, 4), dout=at(H, 5), dq=at(H, 6),
                 dk=at(HK, 7), dv=at(HK, 8), S0=FAKE + (9 << 16), dlast=FAKE + (10 << 16))
    for call, pairs in (("forward", ["out q", "out k", "out v"]),
                        ("step", ["out q", "out k", "out v"]),
                        ("backward", ["dq q", "dq dout", "dk k", "dk v", "dk dq", "dv v", "dv dk",
                                      "dS0 S0", "dS0 dlast"])):
        for pair in pairs:
            w, r = pair.split()
            kw = dict(apart, **{w: (apart[r][0],) + apart[w][1:] if w != "dS0" else apart[r]})
            assert decay(lib, call, **kw) == -1
            assert lib.rehyat_last_error().decode().endswith("may not be another argument"), pair


def rotary_status(lib, **kw):
    a = dict(B=B, n=N, Hq=H, Hk=HK, D=D, R=D, interleaved=0, inverse=0, axes=1, pos64=0,
             add_index=1, dtype=rb.REHYAT_BF16, pos_axis=0, pos_batch=0, pos_token=0, start=0,
             freq=FAKE, axis=0, pos=0, q=rows(H, FAKE), k=rows(HK, FAKE + (1 << 16)),
             q_out=rows(H, FAKE + (2 << 16)), k_out=rows(HK, FAKE + (3 << 16)), scale=1.0)
    a.update(kw)
    flat = [y for x in a.values() for y in (x if isinstance(x, tuple) else (x,))]
    return lib.rehyat_rotary(rb._ROTARY.pack(*flat), None)


@pytest.mark.parametrize("kw", [
    dict(q_out=rows(H, FAKE + (1 << 16))), dict(q_out=rows(H, FAKE + (3 << 16))),
    dict(k_out=rows(HK, FAKE)),
    dict(k_out=(FAKE + (3 << 16), HK * N * D, 0, D)),   # the output's heads expanded
    dict(q_out=(FAKE + (2 << 16), 0, N * D, D)),
    dict(k=(FAKE + (1 << 16), HK * N * D, 0, D),        # expanded and in place
         k_out=(FAKE + (1 << 16), HK * N * D, 0, D)),
])
def test_rotary_refuses_outputs_that_overlap(lib, kw):
    assert rotary_status(lib, **kw) == -1
    assert lib.rehyat_last_error().decode()


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), -1), (dict(n=-1), -1), (dict(Hq=0), -1), (dict(Hk=-1), -1), (dict(R=0), -2),
    (dict(R=7), -2), (dict(R=66), -2), (dict(axes=0), -1), (dict(axes=5), -1),
    (dict(scale=math.nan), -1), (dict(dtype=3), -3), (dict(q=rows(H, 0)), -1),
    (dict(freq=0), -1), (dict(k=rows(HK, 0)), -1), (dict(q_out=(FAKE, H * N * D, 8, D)), -1),
])
def test_rotary_refuses(lib, kw, status):
    a = dict(B=B, n=N, Hq=H, Hk=HK, D=D, R=D, interleaved=0, inverse=0, axes=1, pos64=0,
             add_index=1, dtype=rb.REHYAT_BF16, pos_axis=0, pos_batch=0, pos_token=0, start=0,
             freq=FAKE, axis=0, pos=0, q=rows(H), k=rows(HK), q_out=rows(H, FAKE + 1024),
             k_out=rows(HK), scale=1.0)
    a.update(kw)
    flat = [y for x in a.values() for y in (x if isinstance(x, tuple) else (x,))]
    assert lib.rehyat_rotary(rb._ROTARY.pack(*flat), None) == status
    assert lib.rehyat_last_error().decode()


def test_argument_blocks_match_the_header(lib):
    """The sizes that the library asserts for its argument blocks; a null block is refused."""
    assert [x.size for x in (rb._ROTARY, rb._DECAY_FORWARD, rb._DECAY_BACKWARD,
                             rb._DECAY_STEP)] == [240, 208, 312, 184]
    for name in ("rotary", "decay_forward", "decay_backward", "decay_step"):
        assert getattr(lib, "rehyat_" + name)(None, None) == -1


def test_workspace_grows_with_shared_heads_only_for_gradients(lib):
    size = lambda Hk, bwd: rb.decay_workspace_size(1, 4, Hk, 1000, 64, bwd)  # noqa: E731
    assert size(4, False) == size(2, False)
    assert size(2, True) - size(4, True) == 2 * 4 * 1000 * 64 * 4  # dk and dv of every query head
    assert rb.decay_workspace_size(1, 4, 4, 0, 64) > 0
    with pytest.raises(rb.RehyatError):
        rb.decay_workspace_size(1, 4, 3, 10, 64)


def x(heads=H, n=N, d=D, dtype=torch.bfloat16):
    return torch.zeros(B, heads, n, d, dtype=dtype)


def test_binding_refuses_shapes():
    g, S = torch.zeros(H), torch.zeros(B, H, D, D)
    with pytest.raises(ValueError, match="CUDA device"):
        rb.decay_forward(x(), x(HK), x(HK), g)
    for bad in (dict(q=x()[0]), dict(k=x(3)), dict(k=x(0))):
        with pytest.raises(ValueError, match="heads"):
            rb.decay_forward(**dict(dict(q=x(), k=x(HK), v=x(HK), log_decay=g), **bad))
    with pytest.raises(ValueError, match="one token"):
        rb.decay_step(x(), x(HK), x(HK), g, S)
    f = torch.zeros(D // 2, dtype=torch.float64)
    with pytest.raises(ValueError, match="CUDA device"):
        rb.rotary(x(), x(HK), f)
    with pytest.raises(TypeError, match="unsupported dtype"):
        rb.rotary(x(dtype=torch.float16), None, f)


def test_frequency_tables():
    f, m = rb.rotary_frequencies(64)
    assert m == 1.0 and f.dtype == torch.float64
    assert np.allclose(f.numpy(), [10000.0 ** (-2 * p / 64) for p in range(32)], rtol=1e-14)
    f4, _ = rb.rotary_frequencies(64, scaling="linear", factor=4.0)
    assert torch.equal(f4, f / 4)
    n, _ = rb.rotary_frequencies(64, scaling="ntk", factor=4.0)
    assert float(n[0]) == 1.0 and abs(float(n[-1] / f[-1]) - 0.25) < 1e-12
    y, m = rb.rotary_frequencies(64, scaling="yarn", factor=4.0, original_length=4096)
    assert abs(m - (0.1 * math.log(4) + 1)) < 1e-15
    rounds = 4096 * f / (2 * math.pi)
    assert torch.equal(y[rounds >= 34], f[rounds >= 34])         # fast pairs kept
    assert torch.allclose(y[rounds < 0.9], f[rounds < 0.9] / 4)  # slow pairs stretched
    ratio = y / f
    assert bool((ratio[1:] <= ratio[:-1] + 1e-15).all())
    for bad in (dict(R=7), dict(R=0), dict(R=8, factor=0.5), dict(R=8, scaling="no"),
                dict(R=8, scaling="yarn"), dict(R=2, scaling="ntk", factor=2.0),
                dict(R=8, base=1.0)):
        with pytest.raises(ValueError):
            rb.rotary_frequencies(**bad)
    assert rb.rotary_axes((2, 1, 3)).tolist() == [0, 0, 1, 2, 2, 2]
    p = rb.video_positions(2, 2, 3, first_frame=5)
    assert p.shape == (3, 1, 12)
    assert p[:, 0].T.tolist()[7] == [6, 0, 1]


def test_angle_arithmetic_wraps_exactly():
    """The kernel's angle: a frequency as a 64-bit fraction of a turn, times the position modulo
    2^64, its upper 32 bits as a signed fraction of half a turn.  Against exact integers it is
    within 2^-32 turns (the dropped bits) plus the 2^-53 relative rounding of freq / 2 pi, taken
    pos times."""
    for freq in (1.0, 0.7, 10000.0 ** (-126 / 128), 1e-6):
        t = freq * 0.15915494309189533577
        frac = int((t - math.floor(t)) * 2.0 ** 64)
        for pos in (0, 1, 4095, 1 << 20, (1 << 31) - 1, -1, -12345):
            wrapped = ctypes.c_int32(((pos * frac) & (2 ** 64 - 1)) >> 32).value / 2.0 ** 32
            want = math.fmod(pos * (freq / (2 * math.pi)), 1.0)
            diff = (wrapped - want + 0.5) % 1.0 - 0.5
            assert abs(diff) <= 2.0 ** -32 + abs(pos) * t * 2.0 ** -51
