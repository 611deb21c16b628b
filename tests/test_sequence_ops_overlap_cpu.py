"""Written tensors of the sequence operators that overlap themselves or another argument are refused
before anything is enqueued; neighbours in one buffer are not.

No call here gets past the checks: what is accepted is shown by the last argument's refusal, a
workspace laid over k, whose check comes after all others."""
import random

import numpy as np
import pytest

from hybrid_softmax_linear_chunked_b200 import binding as rb
from hybrid_softmax_linear_chunked_b200 import build

AT = [(i + 1) << 32 for i in range(12)]  # addresses far apart, never dereferenced
B, H, HK, N, D = 2, 4, 2, 40, 64


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return rb.load()


def rows(heads, p, n=N, d=D):
    return (p, heads * n * d, n * d, d)


def call(lib, name, **kw):
    a = dict(B=B, H=H, Hk=HK, N=N, D=D, pool=B, dtype=rb.REHYAT_BF16, q=rows(H, AT[0]),
             k=rows(HK, AT[1]), v=rows(HK, AT[2]), out=rows(H, AT[3]), dout=rows(H, AT[4]),
             dq=rows(H, AT[5]), dk=rows(HK, AT[6]), dv=rows(HK, AT[7]), g=AT[8],
             lengths=AT[8] + 4096, S0=AT[9], last=AT[10], dlast=AT[9] + (1 << 24),
             dS0=AT[10] + (1 << 24), state=AT[9], slots=AT[8] + 4096, ws=AT[1] - 16,
             ws_bytes=1 << 31, scale=1.0)
    a.update(kw)
    order = {"forward": "B H Hk N D dtype q k v out g lengths S0 last ws ws_bytes scale",
             "backward": "B H Hk N D dtype q k v dout dq dk dv g lengths S0 dlast dS0 ws ws_bytes "
                         "scale",
             "step": "B H Hk D pool dtype q k v out g state slots scale"}[name].split()
    flat = [y for n in order for y in (a[n] if isinstance(a[n], tuple) else (a[n],))]
    status = getattr(lib, "rehyat_decay_" + name)(
        getattr(rb, "_DECAY_" + name.upper()).pack(*flat), None)
    return status, lib.rehyat_last_error().decode()


LAST = (-1, "workspace overlaps k")  # all other checks passed


def test_the_checks_end_with_the_workspace(lib):
    assert call(lib, "forward") == LAST and call(lib, "backward") == LAST


@pytest.mark.parametrize("name", ["forward", "backward"])
@pytest.mark.parametrize("strides", [
    (D, N * D, D),                # sequences over rows
    (N * D, N * D, D),            # sequences over heads
    (H * N * D, D, D),            # heads over rows
    (H * N * D, D, 2 * D),        # heads between rows, but four of them
    (H * N * D, N * D, 2 * D),    # rows past the next head's
])
def test_outputs_that_overlap_themselves(lib, name, strides):
    out = "out" if name == "forward" else "dq"
    status, msg = call(lib, name, **{out: (AT[3], *strides)})
    assert status == -1 and msg == f"{out}: its rows overlap one another"


@pytest.mark.parametrize("name,kw,msg", [
    ("forward", dict(out=rows(H, AT[0] + 16)), "out overlaps q"),
    ("forward", dict(out=rows(H, AT[0] - 16)), "out overlaps q"),
    ("forward", dict(out=rows(H, AT[1] + 2 * HK * N * D * 2 - 16)), "out overlaps k"),
    ("forward", dict(last=AT[9] + 64), "S_last overlaps S0"),
    ("forward", dict(last=AT[0] + 64), "S_last overlaps q"),
    ("forward", dict(last=AT[8] - 64), "S_last overlaps log_decay"),
    ("forward", dict(ws=AT[3] + 64), "workspace overlaps out"),
    ("forward", dict(ws=AT[10] - 64), "workspace overlaps S_last"),
    ("backward", dict(dq=rows(H, AT[4] + 128)), "dq overlaps dout"),
    ("backward", dict(dk=rows(HK, AT[2] + 128)), "dk overlaps v"),
    ("backward", dict(dv=rows(HK, AT[6] + 128)), "dv overlaps dk"),
    ("backward", dict(dS0=AT[9] + 128), "dS0 overlaps S0"),
    ("backward", dict(ws=AT[5] + 128), "workspace overlaps dq"),
    ("step", dict(out=(AT[0] + 128, H * D, D, D), q=(AT[0], H * D, D, D)), "out overlaps q"),
    ("step", dict(out=(AT[9] + 128, H * D, D, D)), "state overlaps out"),
    ("step", dict(q=(AT[9] + 128, H * D, D, D)), "state overlaps q"),
    ("step", dict(slots=AT[9] + 128), "state overlaps slots"),
])
def test_written_tensors_that_overlap_another(lib, name, kw, msg):
    status, got = call(lib, name, **kw)
    assert status == -1 and got == msg


def test_neighbours_in_one_buffer_are_accepted(lib):
    packed = [(AT[0] + 2 * D * i, N * 12 * D, D, 12 * D) for i in (0, 4, 6, 8)]  # [B, N, 12, D]
    assert call(lib, "forward", **dict(zip(("q", "k", "v", "out"), packed)), ws=AT[0] - 16)[
        1].startswith("workspace overlaps")
    between = (AT[0] + 2 * N * D, H * 2 * N * D, 2 * N * D, D)  # every second head's place
    assert call(lib, "forward", q=(AT[0], H * 2 * N * D, 2 * N * D, D), out=between) == LAST
    behind = rows(H, AT[0] + 2 * B * H * N * D)
    assert call(lib, "forward", out=behind) == LAST
    assert call(lib, "forward", last=AT[9]) == LAST  # S_last may be S0
    # a stride of a dimension of one is not looked at
    assert call(lib, "forward", B=1, out=(AT[3], D, N * D, D)) == LAST


def offsets(t, shape):
    p, *st = t
    grid = np.add.outer(np.add.outer(np.arange(shape[0]) * st[0], np.arange(shape[1]) * st[1]),
                        np.arange(shape[2]) * st[2])
    return p // 16 + grid.ravel() * 2 // 16  # D = 8: a row is one 16-byte unit


def test_layouts_against_their_bytes(lib):
    """Random layouts of q and out in one buffer: what is refused shares a byte, and of layouts with
    the same strides, or with one of them dense, everything that shares one is refused."""
    r = random.Random(7)
    refused = accepted = 0
    for _ in range(3000):
        b, h, n = r.randint(1, 3), r.randint(1, 3), r.randint(1, 4)

        def layout(pad):
            order, size, st, step = list(range(3)), (b, h, n), [0] * 3, 8
            r.shuffle(order)
            for i in order:
                st[i] = step
                step *= size[i]
                step += 8 * (r.randint(0, 3) if pad else 0)
            return tuple(st)

        kind = r.choice(["same", "dense"])
        sq = layout(True)
        so = sq if kind == "same" else layout(False)
        if r.random() < 0.5 and kind == "dense":
            sq, so = so, sq
        q, out = (AT[0], *sq), (AT[0] + 16 * r.randint(-60, 60), *so)
        units = [offsets(t, (b, h, n)) for t in (q, out)]
        shared = bool(np.intersect1d(*units).size)
        assert np.unique(units[1]).size == b * h * n
        status, msg = call(lib, "forward", B=b, H=h, Hk=h, N=n, D=8, q=q, out=out,
                           k=rows(h, AT[1], n, 8), v=rows(h, AT[2], n, 8))
        assert status == -1
        if shared:
            assert msg in ("out overlaps q", "out may not be another argument"), (q, out, b, h, n)
        else:
            assert (status, msg) == LAST, (q, out, b, h, n)
        refused, accepted = refused + shared, accepted + (not shared)
    assert min(refused, accepted) > 500


def rotary(lib, **kw):
    a = dict(B=B, n=N, Hq=H, Hk=HK, D=D, R=D, interleaved=0, inverse=0, axes=1, pos64=0,
             add_index=0, dtype=rb.REHYAT_BF16, pos_axis=0, pos_batch=N, pos_token=1, start=0,
             freq=AT[4], axis=AT[5], pos=AT[6], q=rows(H, AT[0]), k=rows(HK, AT[1]),
             q_out=rows(H, AT[2]), k_out=rows(HK, AT[3]), scale=1.0)
    a.update(kw)
    flat = [y for x in a.values() for y in (x if isinstance(x, tuple) else (x,))]
    return lib.rehyat_rotary(rb._ROTARY.pack(*flat), None), lib.rehyat_last_error().decode()


@pytest.mark.parametrize("kw,msg", [
    (dict(q_out=(AT[2], D, N * D, D)), "q_out: its rows overlap one another"),
    (dict(k_out=(AT[3], HK * N * D, D, D)), "k_out: its rows overlap one another"),
    (dict(q_out=rows(H, AT[0] + 2)), "q_out overlaps q"),
    (dict(q_out=rows(H, AT[1] - 2)), "q_out overlaps k"),
    (dict(k_out=rows(HK, AT[0] + 2 * D)), "k_out overlaps q"),
    (dict(k_out=rows(HK, AT[2] + 2 * D)), "k_out overlaps q_out"),
    (dict(k_out=rows(HK, AT[6] - 2)), "k_out overlaps pos"),
    (dict(q_out=rows(H, AT[4] + 8)), "q_out overlaps freq"),
    # an expanded input under an output
    (dict(q=(AT[2] + 2 * D, 0, 0, D)), "q_out overlaps q"),
    # in place in a packed buffer, whose other part another output shares in part
    (dict(q=(AT[0], N * 6 * D, D, 6 * D), q_out=(AT[0], N * 6 * D, D, 6 * D),
          k=(AT[0] + 8 * D, N * 6 * D, D, 6 * D), k_out=(AT[0] + 6 * D, N * 6 * D, D, 6 * D)),
     "k_out overlaps q_out"),
])
def test_rotary_outputs_that_overlap(lib, kw, msg):
    status, got = rotary(lib, **kw)
    assert status == -1 and got == msg
