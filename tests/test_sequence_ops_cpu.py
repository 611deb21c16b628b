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


def st(heads, n=N, d=D):
    return rb.Strides(heads * n * d, n * d, d)


def decay(lib, call="forward", dt=rb.REHYAT_BF16, ws_bytes=1 << 40, ws=FAKE, **kw):
    a = dict(B=B, H=H, Hk=HK, N=N, D=D, scale=1.0)
    ptr = dict(q=FAKE, k=FAKE, v=FAKE, out=FAKE, g=FAKE, S0=None, last=FAKE, dout=FAKE, dq=FAKE,
               dk=FAKE, dv=FAKE, state=FAKE, slots=None, pool=B)
    sq, sk = kw.pop("sq", st(H)), kw.pop("sk", st(HK))
    a.update({n: kw.pop(n) for n in list(kw) if n in a})
    ptr.update(kw)
    args = rb.DecayArgs(*a.values())
    rows = (ptr["q"], sq, ptr["k"], sk, ptr["v"], st(HK))
    if call == "forward":
        return lib.rehyat_decay_forward(args, dt, *rows, ptr["g"], None, ptr["S0"], ptr["out"],
                                        st(H), ptr["last"], ws, ws_bytes, None)
    if call == "backward":
        return lib.rehyat_decay_backward(args, dt, *rows, ptr["g"], None, ptr["S0"], ptr["dout"],
                                         st(H), None, ptr["dq"], st(H), ptr["dk"], st(HK),
                                         ptr["dv"], st(HK), None, ws, ws_bytes, None)
    return lib.rehyat_decay_step(args, dt, *rows, ptr["g"], ptr["state"], ptr["pool"],
                                 ptr["slots"], ptr["out"], st(H), None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), -1), (dict(Hk=3), -1), (dict(Hk=0), -1), (dict(N=-1), -1), (dict(D=0), -1),
    (dict(D=60), -2), (dict(D=136), -2), (dict(B=70000), -2), (dict(H=40000, Hk=40000), -2),
    (dict(scale=math.nan), -1), (dict(scale=math.inf), -1), (dict(dt=7), -3),
    (dict(q=None), -1), (dict(v=FAKE + 8), -7), (dict(g=None), -1), (dict(S0=FAKE + 4), -7),
    (dict(sq=rb.Strides(H * N * D, N * D, D - 8)), -1),     # rows overlap
    (dict(sk=rb.Strides(HK * N * D, 0, D)), -1),            # heads expanded
    (dict(sk=rb.Strides(HK * N * D + 4, N * D, D)), -7),    # 8-byte stride in bf16
    (dict(sk=rb.Strides(1 << 40, N * D, D)), -1),
    (dict(ws_bytes=0), -4), (dict(ws=None), -4), (dict(ws=FAKE + 8), -7),
])
def test_decay_forward_refuses(lib, kw, status):
    assert decay(lib, **kw) == status
    assert lib.rehyat_last_error().decode()


@pytest.mark.parametrize("kw,status", [
    (dict(Hk=3), -1), (dict(D=12), -2), (dict(dout=None), -1), (dict(dk=None), -1),
    (dict(dv=FAKE + 2), -7), (dict(ws_bytes=64), -4),
])
def test_decay_backward_refuses(lib, kw, status):
    assert decay(lib, "backward", **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(state=None), -1), (dict(g=None), -1), (dict(pool=0), -1), (dict(pool=1), -1),
    (dict(state=FAKE + 8), -7), (dict(out=None), -1), (dict(D=4), -2), (dict(dt=2), -3),
])
def test_decay_step_refuses(lib, kw, status):
    assert decay(lib, "step", **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), -1), (dict(n=-1), -1), (dict(Hq=0), -1), (dict(Hk=-1), -1), (dict(R=0), -2),
    (dict(R=7), -2), (dict(R=66), -2), (dict(axes=0), -1), (dict(axes=5), -1),
    (dict(scale=math.nan), -1), (dict(dt=3), -3), (dict(q=None), -1), (dict(freq=None), -1),
    (dict(k=None), -1), (dict(q_out=FAKE, sqo=st(H, N + 1)), -1),
])
def test_rotary_refuses(lib, kw, status):
    names = [f[0] for f in rb.RotaryArgs._fields_]
    a = dict(zip(names, (B, N, H, HK, D, D, 0, 0, 1, 0, 1, 0, 0, 0, 0, 1.0)))
    a.update({n: kw[n] for n in kw if n in a})
    g = lambda n, d: kw[n] if n in kw else d  # noqa: E731
    assert lib.rehyat_rotary(rb.RotaryArgs(*a.values()), g("dt", rb.REHYAT_BF16), g("q", FAKE),
                             st(H), g("k", FAKE), st(HK), g("freq", FAKE), None, None,
                             g("q_out", FAKE + 1024), g("sqo", st(H)), FAKE, st(HK),
                             None) == status
    assert lib.rehyat_last_error().decode()


def test_workspace_grows_with_shared_heads_only_for_gradients(lib):
    size = lambda Hk, bwd: rb.decay_workspace_size(  # noqa: E731
        rb.DecayArgs(1, 4, Hk, 1000, 64, 1.0), rb.REHYAT_BF16, bwd)
    assert size(4, False) == size(2, False)
    assert size(2, True) - size(4, True) == 4 * 1000 * 64 * 4
    assert rb.decay_workspace_size(rb.DecayArgs(1, 4, 4, 0, 64, 1.0), 0) > 0


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
