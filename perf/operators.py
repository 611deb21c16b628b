"""Cases of the sequence operators: rotary positions, and linear attention with a decay per head
(prompt, training gradients, single tokens).

listed() and draw() describe calls, prepare() makes a call's inputs on the GPU, run() makes one
call: in its plain form (elementary torch operations in fp32, angles and powers in fp64) or, with
`own`, through the package's binding.  exact() gives the same outputs from the definitions in
fp64, row block by row block.

  rotary         (x1, x2) -> scale * (x1 cos a - x2 sin a, x2 cos a + x1 sin a), a = pos * freq
  decay_forward  o_i = scale * (sum_{j<=i} L^(i-j) (q_i.k_j) v_j + L^(i+1) q_i S_0),
                 S_n = L^n S_0 + sum_j L^(n-1-j) k_j v_j^T
  decay_backward gradients of both for q, k, v and S_0
  decay_step     S <- L S + k v^T, o = scale * q S, one token for each sequence
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def rotary_case(**kw):
    return dict(dict(op="rotary", B=1, H=12, Hk=12, n=1, D=128, R=128, dtype="bf16",
                     interleaved=False, inverse=False, axes=1, far=0, factor=1.0, rows_first=False),
                **kw)


def decay_case(op, **kw):
    c = dict(op=op, B=1, H=12, Hk=12, n=1, D=128, dtype="bf16", ragged=False, state=False,
             rows_first=False)
    if op == "decay_step":
        c = dict(op=op, B=1, H=12, Hk=12, D=128, dtype="bf16", slots=0)
    return dict(c, **kw)


def listed():
    return [
        # one decoding step of eight sequences, each at its own position: launch latency
        rotary_case(name="rotary: one token, 8 sequences", B=8, far=5000),
        # q and k of a 480x832 5 s latent video: 21 frames of 30 x 52 tokens, three axes
        rotary_case(name="rotary: 480x832 5 s video", n=32760, axes=3),
        # gradient of a partly rotated head in fp32, stretched context, rows before heads
        rotary_case(name="rotary: gradient, far positions", B=2, H=5, Hk=3, n=4097, D=64, R=32,
                    dtype="f32", interleaved=True, inverse=True, far=1000000, factor=4.0,
                    rows_first=True),
        # one frame of a 480x832 video, as a short prompt that starts a stream
        decay_case("decay_forward", name="prompt: one 1,560-token frame", n=1560),
        # the whole 480x832 5 s sequence
        decay_case("decay_forward", name="prompt: 480x832 5 s video", n=32760),
        # a padded batch of chunks that goes on from earlier states, shared key/value heads,
        # rows before heads as a projection leaves them
        decay_case("decay_forward", name="prompt: ragged batch, carried state", B=5, H=12, Hk=4,
                   n=4680, ragged=True, state=True, rows_first=True),
        # two 720x1280 5 s sequences: the largest
        decay_case("decay_forward", name="prompt: two 720x1280 5 s videos", B=2, n=75600),
        # a reference-precision run on a narrow head
        decay_case("decay_forward", name="prompt: fp32, narrow head", H=4, Hk=4, n=1999, D=64,
                   dtype="f32", state=True),
        # the training step of the 480x832 5 s sequence
        decay_case("decay_backward", name="gradient: 480x832 5 s video", n=32760),
        # a small fp32 training step on a padded batch with carried states and shared heads
        decay_case("decay_backward", name="gradient: fp32, ragged batch", B=3, H=4, Hk=2, n=777,
                   D=96, dtype="f32", ragged=True, state=True),
        # one token of one sequence: launch latency
        decay_case("decay_step", name="step: one sequence"),
        # a serving batch: 192 sequences of a pool of 256 states
        decay_case("decay_step", name="step: 192 of 256 slots", B=192, slots=256),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rotary", "decay_forward", "decay_forward", "decay_backward",
                       "decay_step"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    D = rng.choice([32, 64, 96, 128, 128, 128])
    Hk = rng.choice([1, 2, 3, 4, 6, 12])
    H = Hk * rng.choice([1, 1, 2, 4])
    if kind == "rotary":
        n = _log_int(rng, 1, 40000)
        B = _log_int(rng, 1, max(1, min(64, 40000 // n)))
        return rotary_case(B=B, H=H, Hk=Hk, n=n, D=D, R=rng.choice([D, D, D // 2]), dtype=dtype,
                           interleaved=rng.random() < 0.5, inverse=rng.random() < 0.3,
                           axes=rng.choice([1, 1, 3]), far=rng.choice([0, 4000, 1000000]),
                           factor=rng.choice([1.0, 1.0, 4.0, 16.0]),
                           rows_first=rng.random() < 0.5)
    if kind == "decay_step":
        B = _log_int(rng, 1, 256)
        return decay_case(kind, B=B, H=H, Hk=Hk, D=D, dtype=dtype,
                          slots=rng.choice([0, B + rng.randrange(64)]))
    rows = 12 * 75600 if dtype == "bf16" else 12 * 4680
    n = _log_int(rng, 1, min(75600 if kind == "decay_forward" else 32760, rows // H))
    B = _log_int(rng, 1, max(1, min(16, rows // (H * n))))
    return decay_case(kind, B=B, H=H, Hk=Hk, n=n, D=D, dtype=dtype, ragged=rng.random() < 0.4,
                      state=rng.random() < 0.5, rows_first=rng.random() < 0.5)


def lengths_of(case):
    """Valid rows of each sequence; a ragged batch has a full one, an empty one, others between."""
    B, n = case["B"], case["n"]
    if not case["ragged"]:
        return [n] * B
    r = random.Random(1000 * n + B)
    return [n if b == 0 else 0 if b == 3 else r.randint(min(1, n), n) for b in range(B)]


def work(case):
    el = 2 if case["dtype"] == "bf16" else 4
    B, H, Hk, D = case["B"], case["H"], case["Hk"], case["D"]
    if case["op"] == "rotary":
        rows = B * case["n"] * (H + Hk)
        return {"bytes": 2.0 * rows * D * el, "flops": 3.0 * rows * case["R"]}
    if case["op"] == "decay_step":
        states = B * H * D * D
        return {"bytes": 8.0 * states + B * (2 * H + 2 * Hk) * D * el, "flops": 5.0 * states}
    rows = sum(lengths_of(case))
    out_rows = B * case["n"]
    states = B * H * D * D * 4.0
    if case["op"] == "decay_forward":
        return {"bytes": (rows * (H + 2 * Hk) + out_rows * H) * D * el
                + states * (1 + case["state"]), "flops": 4.0 * rows * H * D * D}
    return {"bytes": (rows * (2 * H + 2 * Hk) + out_rows * (H + 2 * Hk)) * D * el
            + states * (3 * case["state"]), "flops": 10.0 * rows * H * D * D}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _frequencies(case):
    """Radians per position of each rotated pair, and the factor on the rotated values.  Each of
    `axes` sections of pairs has its own axis.  With factor > 1 the context is stretched: slow
    pairs are divided by the factor, fast ones kept, a ramp between (lengths counted in turns over
    a 4,096-token context)."""
    R, base, factor, context = case["R"], 10000.0, case["factor"], 4096
    f = base ** (-2.0 * torch.arange(R // 2, dtype=torch.float64) / R)
    if factor == 1.0:
        return f, 1.0
    at = [R * math.log(context / (t * 2 * math.pi)) / (2 * math.log(base)) for t in (32, 1)]
    lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), R - 1)
    keep = 1 - ((torch.arange(R // 2, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return f * keep + f / factor * (1 - keep), 0.1 * math.log(factor) + 1.0


def _tensor(case, g, B, H, n, D):
    dt = DTYPES[case["dtype"]]
    if case.get("rows_first"):
        return torch.randn(B, n, H, D, generator=g, device="cuda").to(dt).transpose(1, 2)
    return torch.randn(B, H, n, D, generator=g, device="cuda").to(dt)


def log_decays(H):
    """From halving at every token to a window of about 4,000 tokens."""
    return torch.tensor([math.log1p(-2.0 ** -(1 + 11.0 * h / max(H - 1, 1))) for h in range(H)],
                        dtype=torch.float32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, H, Hk, D = case["B"], case["H"], case["Hk"], case["D"]
    s = {"case": case}
    if case["op"] == "rotary":
        n, R = case["n"], case["R"]
        s["q"], s["k"] = _tensor(case, g, B, H, n, D), _tensor(case, g, B, Hk, n, D)
        freq, s["scale"] = _frequencies(case)
        s["freq"] = freq.cuda()
        s["axis"] = None
        if case["axes"] == 3:  # frame, row and column of a token, a third of the pairs each
            s["axis"] = (torch.arange(R // 2) * 3 // (R // 2)).to(torch.uint8).cuda()
            i = torch.arange(n)
            grid = torch.stack([i // 1560, i // 52 % 30, i % 52]).to(torch.int32)
            s["positions"] = grid[:, None, :].expand(3, B, n).contiguous().cuda()
        else:
            first = torch.randint(0, case["far"] + 1, (B, 1), generator=g, device="cuda")
            s["positions"] = (first + torch.arange(n, device="cuda"))[None].to(torch.int32)
        return s
    s["g"] = log_decays(H).cuda()
    s["scale"] = D ** -0.5
    if case["op"] == "decay_step":
        shape = dict(case, rows_first=False)
        s["q"], s["k"], s["v"] = (_tensor(shape, g, B, h, 1, D) for h in (H, Hk, Hk))
        pool = case["slots"] or B
        s["state"] = torch.randn(pool, H, D, D, generator=g, device="cuda")
        s["slots"] = None
        if case["slots"]:
            s["slots"] = torch.randperm(pool, generator=g, device="cuda")[:B].to(torch.int32)
        return s
    n = case["n"]
    s["q"], s["k"], s["v"] = (_tensor(case, g, B, h, n, D) for h in (H, Hk, Hk))
    s["lengths"] = None
    if case["ragged"]:
        s["lengths"] = torch.tensor(lengths_of(case), dtype=torch.int32, device="cuda")
    s["state"] = None
    if case["state"]:
        s["state"] = torch.randn(B, H, D, D, generator=g, device="cuda")
    if case["op"] == "decay_backward":
        s["dout"] = _tensor(case, g, B, H, n, D)
        s["dfinal"] = None
        if case["state"]:
            s["dfinal"] = torch.randn(B, H, D, D, generator=g, device="cuda")
    return s


# ---------------------------------------------------------------------------------------------
# one call
# ---------------------------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return _own(op, state)
    return {"rotary": _rotary, "decay_forward": _forward, "decay_backward": _backward,
            "decay_step": _step}[op](state)


def _own(op, s):
    from hybrid_softmax_linear_chunked_b200 import binding as rb
    c = s["case"]
    if op == "rotary":
        q, k = rb.rotary(s["q"], s["k"], s["freq"], positions=s["positions"], axis=s["axis"],
                         scale=s["scale"], interleaved=c["interleaved"], inverse=c["inverse"])
        return {"q": q, "k": k}
    if op == "decay_step":
        out = rb.decay_step(s["q"], s["k"], s["v"], s["g"], s["state"], scale=s["scale"],
                            slots=s["slots"])
        return {"out": out, "state": s["state"]}
    if op == "decay_forward":
        out, final = rb.decay_forward(s["q"], s["k"], s["v"], s["g"], scale=s["scale"],
                                      lengths=s["lengths"], state=s["state"], final_state=True)
        return {"out": out, "state": final}
    return rb.decay_backward(s["q"], s["k"], s["v"], s["g"], s["dout"], scale=s["scale"],
                             lengths=s["lengths"], state=s["state"], dfinal=s["dfinal"])


# ---- plain forms ----
def _rotary(s):
    c = s["case"]
    axis = s["axis"].long() if s["axis"] is not None else torch.zeros(
        c["R"] // 2, dtype=torch.long, device="cuda")
    angle = s["positions"].double()[axis].permute(1, 2, 0) * s["freq"]  # [B, n, R/2]
    cos, sin = (angle.cos() * s["scale"]).float()[:, None], (angle.sin() * s["scale"]).float()[:, None]
    if c["inverse"]:
        sin = -sin
    return {"q": _rotate(s["q"], cos, sin, c), "k": _rotate(s["k"], cos, sin, c)}


def _rotate(x, cos, sin, c):
    R = c["R"]
    y = x.float()
    rot = y[..., :R]
    if c["interleaved"]:
        a, b = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = rot[..., :R // 2], rot[..., R // 2:]
        rot = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((rot, y[..., R:]), dim=-1).to(x.dtype)


def _power(g, m):
    """exp(g[h] m): [H, *m.shape] in fp32, formed in fp64."""
    return torch.exp(g.double().view(-1, *[1] * m.dim()) * m.double()).float()


def _heads(x, H):
    return x.float().repeat_interleave(H // x.shape[1], dim=1)


def _valid(x, lengths):
    """Rows past a sequence's length as zeros, whatever they hold."""
    if lengths is None:
        return x
    keep = torch.arange(x.shape[2], device=x.device)[None] < lengths[:, None]
    return torch.where(keep[:, None, :, None], x, torch.zeros((), device=x.device))


def _past(q, k, v, g, S0, C=128):
    """sum_{j<=i} L^(i-j) (q_i.k_j) v_j + L^(i+1) q_i S_0, chunk by chunk of C rows."""
    B, H, n, D = q.shape
    nc = -(-n // C)
    q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, nc * C - n)).view(B, H, nc, C, -1)
               for x in (q, k, v))
    i = torch.arange(C, device=q.device)
    inside = torch.where(i[:, None] >= i, _power(g, (i[:, None] - i).clamp(min=0)), 0.0)
    o = (q @ k.transpose(-1, -2) * inside[:, None]) @ v
    add = (k * _power(g, C - 1 - i)[:, None, :, None]).transpose(-1, -2) @ v  # [B, H, nc, D, D]
    c = torch.arange(nc, device=q.device)
    before = torch.where(c[:, None] > c, _power(g, (C * (c[:, None] - 1 - c)).clamp(min=0)), 0.0)
    S = (before @ add.flatten(-2)).view_as(add)
    if S0 is not None:
        S = S + _power(g, C * c)[:, :, None, None] * S0[:, :, None]
    return (o + _power(g, i + 1)[:, None, :, None] * (q @ S)).view(B, H, nc * C, -1)[:, :, :n]


def _last(k, v, g, lengths, first):
    """sum_{j<n} L^(n-1-j+first) k_j v_j^T for the n = lengths rows of each sequence."""
    B, H, n, _ = k.shape
    m = (lengths[:, None] - 1 + first) - torch.arange(n, device=k.device)  # [B, n]
    return (k * _power(g, m.clamp(min=0)).transpose(0, 1)[..., None]).transpose(-1, -2) @ v


def _lengths(s):
    c = s["case"]
    return s["lengths"] if s["lengths"] is not None else torch.full((c["B"],), c["n"],
                                                                    device="cuda")


def _forward(s):
    H = s["case"]["H"]
    q, k, v = (_valid(_heads(s[x], H), s["lengths"]) for x in "qkv")
    n, g, S0 = _lengths(s), s["g"], s["state"]
    out = _valid(_past(q, k, v, g, S0) * s["scale"], s["lengths"])
    final = _last(k, v, g, n, 0)
    if S0 is not None:
        final = final + _power(g, n).transpose(0, 1)[:, :, None, None] * S0
    return {"out": out.to(s["q"].dtype), "state": final}


def _backward(s):
    c = s["case"]
    B, H, Hk, N = c["B"], c["H"], c["Hk"], c["n"]
    q, k, v, do = (_valid(_heads(s[x], H), s["lengths"]) for x in ("q", "k", "v", "dout"))
    n, g, S0, dS = _lengths(s), s["g"], s["state"], s["dfinal"]
    back = [x.flip(2) for x in (q, k, v, do)]
    dq = _past(do, v, k, g, None if S0 is None else S0.transpose(-1, -2)) * s["scale"]
    dk = _past(back[2], back[3], back[0], g, None).flip(2) * s["scale"]
    dv = _past(back[1], back[0], back[3], g, None).flip(2) * s["scale"]
    out = {}
    if S0 is not None:
        i = torch.arange(N, device="cuda")
        to_end = _power(g, (n[:, None] - 1 - i).clamp(min=0)).transpose(0, 1)[..., None]
        dk = dk + to_end * (v @ dS.transpose(-1, -2))
        dv = dv + to_end * (k @ dS)
        first = _power(g, i + 1)[None, ..., None]
        out["dstate"] = ((q * first).transpose(-1, -2) @ do) * s["scale"] \
            + _power(g, n).transpose(0, 1)[:, :, None, None] * dS
    dk, dv = (x.view(B, Hk, H // Hk, N, -1).sum(2) for x in (dk, dv))
    for name, x in (("dq", dq), ("dk", dk), ("dv", dv)):
        out[name] = _valid(x, s["lengths"]).to(s["q"].dtype)
    return out


def _step(s):
    H = s["case"]["H"]
    q, k, v = (_heads(s[x], H)[:, :, 0] for x in "qkv")
    at = s["slots"].long() if s["slots"] is not None else slice(None)
    S = s["state"][at] * torch.exp(s["g"].double()).float()[:, None, None]
    S = S + k[..., None] * v[:, :, None, :]
    s["state"][at] = S
    out = (q[:, :, None, :] @ S)[:, :, 0] * s["scale"]
    return {"out": out[:, :, None].to(s["q"].dtype), "state": s["state"]}


# ---------------------------------------------------------------------------------------------
# from the definitions, in fp64
# ---------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "decay_forward": _exact_forward,
            "decay_backward": _exact_backward, "decay_step": _exact_step}[case["op"]](case, s)


def _exact_rotary(case, s):
    R, pairs = case["R"], case["R"] // 2
    out = {}
    for name in "qk":
        x = s[name].double()
        y = x.clone()
        for p in range(pairs):
            a, b = (2 * p, 2 * p + 1) if case["interleaved"] else (p, p + pairs)
            ax = 0 if s["axis"] is None else int(s["axis"][p])
            t = s["positions"][ax].double() * float(s["freq"][p]) * (-1 if case["inverse"] else 1)
            z = torch.polar(torch.full_like(t, s["scale"]), t)[:, None]
            w = torch.complex(x[..., a], x[..., b]) * z
            y[..., a], y[..., b] = w.real, w.imag
        out[name] = y
    return out


def _rows(n, step=2048):
    return [(r, min(r + step, n)) for r in range(0, n, step)]


def _exact_forward(case, s):
    B, H, n, D, rep = case["B"], case["H"], case["n"], case["D"], case["H"] // case["Hk"]
    out = torch.zeros(B, H, n, D, dtype=torch.float64, device="cuda")
    state = torch.zeros(B, H, D, D, dtype=torch.float64, device="cuda")
    for b, length in enumerate(lengths_of(case)):
        for h in range(H):
            lam = float(s["g"][h])
            q, k, v = (x[:length].double() for x in (s["q"][b, h], s["k"][b, h // rep],
                                                     s["v"][b, h // rep]))
            t = torch.arange(length, dtype=torch.float64, device="cuda")
            S0 = s["state"][b, h].double() if s["state"] is not None else 0.0 * state[b, h]
            for r0, r1 in _rows(length):
                d = t[r0:r1, None] - t[None, :r1]
                w = torch.where(d >= 0, torch.exp(lam * d.clamp(min=0)), 0.0)
                o = (w * (q[r0:r1] @ k[:r1].T)) @ v[:r1]
                o += torch.exp(lam * (t[r0:r1, None] + 1)) * (q[r0:r1] @ S0)
                out[b, h, r0:r1] = o * s["scale"]
            state[b, h] = math.exp(lam * length) * S0 \
                + (torch.exp(lam * (length - 1 - t))[:, None] * k).T @ v
    return {"out": out, "state": state}


def _exact_backward(case, s):
    B, H, Hk, n, D = (case[x] for x in ("B", "H", "Hk", "n", "D"))
    rep = H // Hk
    new = lambda *sh: torch.zeros(*sh, dtype=torch.float64, device="cuda")  # noqa: E731
    g = {"dq": new(B, H, n, D), "dk": new(B, Hk, n, D), "dv": new(B, Hk, n, D)}
    carried = s["state"] is not None
    if carried:
        g["dstate"] = new(B, H, D, D)
    for b, length in enumerate(lengths_of(case)):
        for h in range(H):
            lam, hk, sc = float(s["g"][h]), h // rep, s["scale"]
            q, k, v, do = (x[:length].double() for x in (s["q"][b, h], s["k"][b, hk],
                                                         s["v"][b, hk], s["dout"][b, h]))
            t = torch.arange(length, dtype=torch.float64, device="cuda")
            dk, dv = new(length, D), new(length, D)
            for r0, r1 in _rows(length):
                d = t[r0:r1, None] - t[None, :r1]
                w = sc * torch.where(d >= 0, torch.exp(lam * d.clamp(min=0)), 0.0)
                dp = w * (do[r0:r1] @ v[:r1].T)
                g["dq"][b, h, r0:r1] = dp @ k[:r1]
                dk[:r1] += dp.T @ q[r0:r1]
                dv[:r1] += (w * (q[r0:r1] @ k[:r1].T)).T @ do[r0:r1]
            if carried:
                S0, dS = s["state"][b, h].double(), s["dfinal"][b, h].double()
                w = sc * torch.exp(lam * (t + 1))[:, None]
                g["dq"][b, h, :length] += w * (do @ S0.T)
                g["dstate"][b, h] = (w * q).T @ do + math.exp(lam * length) * dS
                w = torch.exp(lam * (length - 1 - t))[:, None]
                dk += w * (v @ dS.T)
                dv += w * (k @ dS)
            g["dk"][b, hk, :length] += dk
            g["dv"][b, hk, :length] += dv
    return g


def _exact_step(case, s):
    B, H, rep = case["B"], case["H"], case["H"] // case["Hk"]
    state = s["state"].double()
    out = torch.zeros(B, H, 1, case["D"], dtype=torch.float64, device="cuda")
    lam = torch.exp(s["g"].double())[:, None, None]
    for b in range(B):
        at = b if s["slots"] is None else int(s["slots"][b])
        k, v = (s[x][b, :, 0].double().repeat_interleave(rep, 0) for x in "kv")
        state[at] = lam * state[at] + torch.einsum("hd,he->hde", k, v)
        out[b, :, 0] = torch.einsum("hd,hde->he", s["q"][b, :, 0].double(), state[at]) * s["scale"]
    return {"out": out, "state": state}
