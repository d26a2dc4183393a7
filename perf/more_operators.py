"""Cases and plain forms of the operators that run a prompt through one layer: rotary positions with several axes, causal
attention over packed prompts, and the experts' matrix products grouped by expert.

`prepare` makes the inputs, `run` is one pass through an operator (plain torch operations, or the framework's call where
`own` is true), `exact` the definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False


# ------------------------------------------------------------------ cases
def listed():
    return [
        # The verify tokens of four sequences' draft trees before they are attended: latency counts.
        dict(name="rotate_verify", op="rotate", tokens=28, Hq=64, Hkv=4, D=128, R=128, axes=1, far=9000, layout="halves", inverse=False, dtype="bf16"),
        # A prompt of text and video frames: time, height and width positions.
        dict(name="rotate_video", op="rotate", tokens=8192, Hq=32, Hkv=8, D=128, R=128, axes=3, far=20000, layout="halves", inverse=False, dtype="bf16"),
        # The gradient of a rotation of half of each head, at far positions, in fp32.
        dict(name="rotate_back", op="rotate", tokens=3001, Hq=64, Hkv=8, D=64, R=32, axes=1, far=1000000, layout="pairs", inverse=True, dtype="f32"),
        # One short prompt: latency counts.
        dict(name="attend_short", op="attend", seqs=1, length=77, Hq=32, Hkv=8, D=128),
        # A serving batch's prompts, ragged, 16 query heads on a kv head.
        dict(name="attend_batch", op="attend", seqs=24, length=1500, Hq=64, Hkv=4, D=128),
        # An odd number of query heads on a kv head, narrow heads.
        dict(name="attend_narrow", op="attend", seqs=6, length=3001, Hq=14, Hkv=2, D=64),
        # Long documents: the matrix products count.
        dict(name="attend_long", op="attend", seqs=2, length=12001, Hq=32, Hkv=8, D=128),
        # The toy layer on a handful of tokens: latency counts.
        dict(name="gate_up_toy", op="gate_up", tokens=37, H=256, I=512, E=16, k=2, tiled=False),
        # A few tokens more than a verify step takes: nearly every expert, a dozen or two tokens each, the weights' bytes count.
        dict(name="gate_up_few", op="gate_up", tokens=300, H=4096, I=1536, E=128, k=8, tiled=True),
        # A long prompt through the wide layer: the matrix products count.
        dict(name="gate_up_prompt", op="gate_up", tokens=8192, H=4096, I=1536, E=128, k=8, tiled=True),
        # The second product of a layer whose sizes are not whole tiles.
        dict(name="down_odd", op="down", tokens=1501, H=2880, I=2880, E=128, k=4, tiled=False),
        # The second product of the long prompt and the weighted sum over each token's experts.
        dict(name="down_prompt", op="down", tokens=8192, H=4096, I=1536, E=128, k=8, tiled=True),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["rotate", "attend", "attend", "gate_up", "down"])
    if op == "rotate":
        D = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        layout = rng.choice(["halves", "pairs"])
        R = rng.choice([D, D, D // 2, D - 16])
        return dict(op=op, tokens=_log(rng, 1, 6000), Hq=Hkv * rng.choice([1, 3, 4, 7, 8]), Hkv=Hkv, D=D, R=R, axes=rng.choice([1, 2, 3, 4]),
                    far=_log(rng, 100, 2000000), layout=layout, inverse=rng.random() < 0.3, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "attend":
        Hkv, G, D = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16]), rng.choice([64, 128])
        Hkv = min(Hkv, max(1, 64 // G))
        length, seqs = _log(rng, 1, 12000), _log(rng, 1, 48)
        # No costlier than the largest listed one: a bound on the pairs of rows.
        seqs = max(1, min(seqs, int(4.0e9 / (length * length * G * Hkv))))
        return dict(op=op, seqs=seqs, length=length, Hq=G * Hkv, Hkv=Hkv, D=D)
    E = rng.choice([4, 16, 60, 128])
    k = rng.choice([1, 2, 4, 6, 8])
    H, I = 64 * _log(rng, 1, 64), 64 * _log(rng, 1, 32)
    k = min(k, E)
    tokens = max(1, min(_log(rng, 1, 8000), 65536 // k, int(1.5e12 / (4.0 * k * H * I))))
    return dict(op=op, tokens=tokens, H=H, I=I, E=E, k=k, tiled=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _freqs(c):
    """Angle per position of each pair, in 64 bits, and its axis: with several axes the first takes the fastest quarter,
    the others share the rest (one axis: all of them)."""
    n = c["R"] // 2
    f = [10000.0 ** (-i / n) for i in range(n)]
    if c["axes"] == 1:
        return f, [0] * n
    first = n // 4
    return f, [0 if i < first else 1 + (i - first) * (c["axes"] - 1) // (n - first) for i in range(n)]


def _lengths(c):
    """Tokens of each prompt: ragged, the first at its full length; fixed by the case."""
    r = random.Random(7919 * c["length"] + 31 * c["seqs"] + c["Hq"])
    n = [c["length"]] + [r.randint(max(1, c["length"] // 8), c["length"]) for _ in range(c["seqs"] - 1)]
    if c["seqs"] > 3:
        n[2] = 0  # a sequence without a prompt in this batch
        n[3] = 1
    return n


def _routing(c):
    """Experts of each token [tokens, k], distinct, some experts far more popular than others; fixed by the case."""
    r = np.random.default_rng(c["tokens"] * 131 + c["E"] * 7 + c["k"])
    score = r.gumbel(size=(c["tokens"], c["E"])).astype(np.float32) - (3.0 / c["E"]) * r.permutation(c["E"]).astype(np.float32)
    return np.argsort(-score, axis=1, kind="stable")[:, :c["k"]].astype(np.int32)


def _union(ids, E):
    """The union of the tokens' experts, as the framework's union call lays it out: groups by expert, tokens ascending."""
    T, k = ids.shape
    order = np.argsort(ids.reshape(-1), kind="stable").astype(np.int32)
    unique, counts = np.unique(ids, return_counts=True)
    cap = min(E, T * k)
    offsets = np.full(cap + 1, T * k, dtype=np.int32)
    offsets[:len(unique) + 1] = np.concatenate([[0], np.cumsum(counts)])
    inv = np.empty(T * k, dtype=np.int32)
    inv[order] = np.arange(T * k, dtype=np.int32)
    u = {"n_unique": np.array([len(unique)], dtype=np.int32), "unique": np.zeros(cap, dtype=np.int32), "offsets": offsets,
         "perm_token": order // k, "perm_slot": order % k, "inv": inv}
    u["unique"][:len(unique)] = unique
    return {n: torch.from_numpy(a).cuda() for n, a in u.items()}, unique.tolist(), offsets[:len(unique) + 1].tolist()


def _normal(shape, gen, std, dtype):
    """Normal values rounded to the type, made in parts (the weights are large)."""
    t = torch.empty(shape, dtype=dtype, device="cuda")
    for part in t.view(-1).split(1 << 28):
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda", dtype=dtype).mul_(std))
    return t


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    st = {"c": c}
    if c["op"] == "rotate":
        T, A, far = c["tokens"], c["axes"], c["far"]
        dtype = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
        # q and k as slices of one projection's output [tokens, Hq + 2 Hkv, D]
        qkv = torch.randn((T, c["Hq"] + 2 * c["Hkv"], c["D"]), generator=gen, device="cuda").to(dtype)
        st["q"], st["k"] = qkv[:, :c["Hq"]], qkv[:, c["Hq"]:c["Hq"] + c["Hkv"]]
        r = random.Random(int(seed))
        t = torch.arange(T, device="cuda", dtype=torch.int32) + r.randrange(far)
        if A == 1:
            st["pos"] = t
        else:  # frames of 16 x 24 patches after a text: time, height, width (and a second width)
            i = torch.arange(T, device="cuda", dtype=torch.int32)
            st["pos"] = torch.stack([t[:1] + i // 384, t[:1] + i // 24 % 16, t[:1] + i % 24, t[:1] + i % 7][:A]).contiguous()
        if own:
            import serving_router_softmax_gb300 as mv

            f, axis = _freqs(c)
            st["rot"] = mv.Rotary(f, c["D"], axes=axis, interleaved=c["layout"] == "pairs")
        return st
    if c["op"] == "attend":
        n = _lengths(c)
        st["lengths"] = n
        st["start"] = torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32, device="cuda")
        qkv = torch.randn((sum(n), c["Hq"] + 2 * c["Hkv"], c["D"]), generator=gen, device="cuda").to(torch.bfloat16)
        qkv[:, :c["Hq"]] *= 1.5
        st["q"], st["k"], st["v"] = qkv[:, :c["Hq"]], qkv[:, c["Hq"]:c["Hq"] + c["Hkv"]], qkv[:, c["Hq"] + c["Hkv"]:]
        st["scale"] = c["D"] ** -0.5
        return st
    T, H, I, E, k = c["tokens"], c["H"], c["I"], c["E"], c["k"]
    ids = _routing(c)
    st["union"], st["experts"], st["groups"] = _union(ids, E)
    down = c["op"] == "down"
    st["w"] = _normal((E, H, I) if down else (E, 2 * I, H), gen, 0.02, torch.bfloat16)
    if down:
        st["h"] = _normal((T * k, I), gen, 0.5, torch.bfloat16)
        p = torch.rand((T, k), generator=gen, device="cuda") + 0.05
        st["weights"] = p / p.sum(1, keepdim=True)
    else:
        st["x"] = _normal((T, H), gen, 1.0, torch.bfloat16)
    if own:
        import serving_router_softmax_gb300 as mv

        # The layer's other matrix, which the call does not read.
        other = torch.zeros((E, 2 * I, H) if down else (E, H, I), dtype=torch.bfloat16, device="cuda")
        layer = mv.ExpertLayer(other if down else st["w"], st["w"] if down else other, "bf16")
        st["layer"] = mv.pack_tiled(layer) if c["tiled"] else layer
    return st


# ------------------------------------------------------------------ plain forms
def _rotate(st):
    c = st["c"]
    R = c["R"]
    f, axis = _freqs(c)
    pos = st["pos"].view(c["axes"], -1).to(torch.float64)
    angle = pos[torch.tensor(axis, device=pos.device)].t() * torch.tensor(f, dtype=torch.float64, device=pos.device)  # [T, R/2]
    if c["inverse"]:
        angle = -angle
    cos, sin = torch.cos(angle).to(torch.float32)[:, None], torch.sin(angle).to(torch.float32)[:, None]
    outs = []
    for x in (st["q"], st["k"]):
        y = x.to(torch.float32, copy=True, memory_format=torch.contiguous_format)
        a, b = (y[..., 0:R:2], y[..., 1:R:2]) if c["layout"] == "pairs" else (y[..., :R // 2], y[..., R // 2:R])
        ra, rb = a * cos - b * sin, a * sin + b * cos
        a.copy_(ra)
        b.copy_(rb)
        outs.append(y.to(x.dtype))
    return outs


def _attend(st):
    c, q, k, v = st["c"], st["q"], st["k"], st["v"]
    Hkv, G, D = c["Hkv"], c["Hq"] // c["Hkv"], c["D"]
    out, lse = torch.empty(q.shape, dtype=q.dtype, device=q.device), torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    first = 0
    for n in st["lengths"]:
        step = max(1, (1 << 29) // (max(n, 1) * Hkv * G))  # query rows at once: scores of 2 GB at most
        kk = k[first:first + n].to(torch.float32).permute(1, 2, 0)       # [Hkv, D, n]
        vv = v[first:first + n].to(torch.float32).transpose(0, 1)        # [Hkv, n, D]
        for i in range(0, n, step):
            m = min(step, n - i)
            rows = q[first + i:first + i + m].to(torch.float32).unflatten(1, (Hkv, G)).permute(1, 2, 0, 3)  # [Hkv, G, m, D]
            seen = i + m
            s = torch.matmul(rows.flatten(1, 2), kk[:, :, :seen]).unflatten(1, (G, m)).mul_(st["scale"])
            later = torch.arange(seen, device=q.device) > torch.arange(i, seen, device=q.device)[:, None]
            s.masked_fill_(later, -math.inf)
            top = s.amax(3, keepdim=True)
            p = torch.exp_(s.sub_(top))
            total = p.sum(3, keepdim=True)
            o = torch.matmul(p.flatten(1, 2), vv[:, :seen]).unflatten(1, (G, m)) / total
            out[first + i:first + i + m] = o.permute(2, 0, 1, 3).flatten(1, 2).to(q.dtype)
            lse[first + i:first + i + m] = (torch.log(total) + top)[..., 0].permute(2, 0, 1).flatten(1, 2)
        first += n
    return out, lse


def _gate_up(st):
    c, u = st["c"], st["union"]
    I = c["I"]
    h = torch.empty((c["tokens"] * c["k"], I), dtype=torch.bfloat16, device="cuda")
    for e, a, b in zip(st["experts"], st["groups"], st["groups"][1:]):
        z = torch.matmul(st["x"][u["perm_token"][a:b].long()].to(torch.float32), st["w"][e].to(torch.float32).t())
        g = z[:, :I]
        h[a:b] = (g / (1.0 + torch.exp(-g)) * z[:, I:]).to(torch.bfloat16)
    return h


def _down(st):
    c, u = st["c"], st["union"]
    o = torch.empty((c["tokens"] * c["k"], c["H"]), dtype=torch.float32, device="cuda")
    for e, a, b in zip(st["experts"], st["groups"], st["groups"][1:]):
        o[a:b] = torch.matmul(st["h"][a:b].to(torch.float32), st["w"][e].to(torch.float32).t())
    inv = u["inv"].long().view(c["tokens"], c["k"])
    y = torch.zeros((c["tokens"], c["H"]), dtype=torch.float32, device="cuda")
    for j in range(c["k"]):
        y += st["weights"][:, j:j + 1] * o[inv[:, j]]
    return y.to(torch.bfloat16)


def run(state):
    st, c = state, state["c"]
    if own:
        import serving_router_softmax_gb300 as mv

        if c["op"] == "rotate":
            return mv.rotate(st["rot"], st["q"], st["k"], st["pos"], inverse=c["inverse"])
        if c["op"] == "attend":
            return mv.prompt_attend(st["q"], st["k"], st["v"], st["start"], scale=st["scale"])
        if c["op"] == "gate_up":
            return mv.group_gate_up(st["x"], st["layer"], st["union"], c["k"])
        return mv.group_down(st["h"], st["layer"], st["union"], st["weights"])
    return {"rotate": _rotate, "attend": _attend, "gate_up": _gate_up, "down": _down}[c["op"]](st)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "rotate":
        size = 4 if c["dtype"] == "f32" else 2
        n = c["tokens"] * (c["Hq"] + c["Hkv"])
        return {"bytes": 2 * size * n * c["D"] + 4 * c["axes"] * c["tokens"], "flops": 3 * n * c["R"]}
    if c["op"] == "attend":
        n = _lengths(c)
        T, pairs = sum(n), sum(t * (t + 1) // 2 for t in n)
        return {"bytes": T * (2 * c["D"] * (2 * c["Hq"] + 2 * c["Hkv"]) + 4 * c["Hq"]), "flops": 4 * c["D"] * c["Hq"] * pairs}
    U, rows = len(np.unique(_routing(c))), c["tokens"] * c["k"]
    H, I, T = c["H"], c["I"], c["tokens"]
    if c["op"] == "gate_up":
        return {"bytes": 4 * U * I * H + 2 * T * H + 2 * rows * I + 4 * rows, "flops": 4 * rows * H * I}
    return {"bytes": 2 * U * I * H + 2 * T * H + 2 * rows * I + 8 * rows, "flops": 2 * rows * H * I + 2 * rows * H}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    c = case
    st = prepare(c, seed)
    if c["op"] == "rotate":
        n = c["R"] // 2
        f, axis = _freqs(c)
        pos = st["pos"].view(c["axes"], -1)
        res = []
        for x in (st["q"], st["k"]):
            y = x.double()
            z = y.clone()
            for i in range(n):
                w = torch.polar(torch.ones(c["tokens"], dtype=torch.float64, device="cuda"),
                                pos[axis[i]].double() * (-f[i] if c["inverse"] else f[i]))[:, None]
                at = (2 * i, 2 * i + 1) if c["layout"] == "pairs" else (i, i + n)
                turned = torch.complex(y[:, :, at[0]], y[:, :, at[1]]) * w
                z[:, :, at[0]], z[:, :, at[1]] = turned.real, turned.imag
            res.append(z)
        return res
    if c["op"] == "attend":
        n = st["lengths"]
        G = c["Hq"] // c["Hkv"]
        out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.zeros(st["q"].shape[:2], dtype=torch.float64, device="cuda")
        first = 0
        for t in n:
            at = slice(first, first + t)
            for h in range(c["Hq"]):
                kk, vv = st["k"][at, h // G].double(), st["v"][at, h // G].double()
                for i in range(0, t, 2048):
                    e = min(i + 2048, t)
                    x = torch.einsum("id,jd->ij", st["q"][first + i:first + e, h].double(), kk[:e]) * st["scale"]
                    x = torch.where(torch.ones_like(x, dtype=torch.bool).tril(i), x, -math.inf)
                    z = torch.logsumexp(x, 1)
                    lse[first + i:first + e, h] = z
                    out[first + i:first + e, h] = (x - z[:, None]).exp() @ vv[:e]
            first += t
        return out, lse
    ids = torch.from_numpy(_routing(c)).cuda()
    T, k = ids.shape
    place = st["union"]["inv"].long().view(T, k)
    if c["op"] == "gate_up":
        h = torch.zeros((T * k, c["I"]), dtype=torch.float64, device="cuda")
        for e in range(c["E"]):
            t, j = torch.nonzero(ids == e, as_tuple=True)
            if len(t):
                x = st["x"][t].double()
                gate, up = (torch.einsum("th,ih->ti", x, part.double()) for part in st["w"][e].split(c["I"]))
                h[place[t, j]] = gate * torch.sigmoid(gate) * up
        return h
    y = torch.zeros((T, c["H"]), dtype=torch.float64, device="cuda")
    for e in range(c["E"]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if len(t):
            y[t] += st["weights"][t, j].double()[:, None] * torch.einsum("ti,hi->th", st["h"][place[t, j]].double(), st["w"][e].double())
    return y
