"""bf16 decayed attention scales its results by nothing: rounding the weighted rows of the carried
state must average out, also where the decay is so slow that all weights of a chunk (or, times the
scale of a gradient, all weights of a pass) lie within one step of the type.

The measure is the projection of the result on the float64 one, <got, want> / <want, want> - 1.
Tolerance: independent roundings leave at most 4.5e-3 of each value in the mean square (four
roundings of half a step 2^-8, 2^-8 / sqrt(3) each); the projection averages them over at least the
D * D = 4,096 independent values of one state: 4.5e-3 / 64 = 7e-5, four standard deviations of
which are 2.8e-4, taken as 3e-4."""
import numpy as np
import pytest
import torch

from hybrid_softmax_linear_chunked_b200 import binding as rb
from oracle import sequence_oracle as SO

pytestmark = pytest.mark.gpu

N, D, TOL = 4096, 64, 3e-4
SLOW = [0.0, -1.2e-5, -1e-4]


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


@pytest.mark.parametrize("scale", [257 / 256, 1 / 3], ids=["257/256", "1/3"])
@pytest.mark.parametrize("H", [3, 148])  # segments of one chunk; one segment a sequence
def test_results_are_not_scaled(dev, H, scale):
    g = torch.Generator().manual_seed(21)
    q, k, v, do = (torch.randn(1, H, N, D, generator=g).to(torch.bfloat16).to(dev)
                   for _ in range(4))
    decay = torch.tensor((SLOW + [-0.05] * H)[:H], device=dev)
    out = rb.decay_forward(q, k, v, decay, scale=scale)
    grads = rb.decay_backward(q, k, v, decay, do, scale=scale)
    rb.sync_status(dev)
    off = {}
    for h, d in enumerate(float(decay[h]) for h in range(len(SLOW))):
        x = [f64(t[0, h]) for t in (q, k, v)]
        want = dict(zip(("dq", "dk", "dv"), SO.decay_backward(*x, d, f64(do[0, h]), scale=scale)))
        want["out"] = SO.decay_forward(*x, d, scale=scale)[0]
        for name, w in want.items():
            got = f64((out if name == "out" else grads[name])[0, h])
            off[name, SLOW[h]] = float((got * w).sum() / (w * w).sum()) - 1
    assert all(abs(x) <= TOL for x in off.values()), off
