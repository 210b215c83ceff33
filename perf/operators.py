"""The work of the packed-document training operators: masked attention and its gradient, rotary
positions over several axes and their gradient, and the AdamW step with 8-bit states.

A case names an operator and its sizes; prepare() makes the inputs on the GPU from a seed; run()
makes one pass, in elementary torch operations (own = False) or through this repository's library
(own = True); exact() computes the same outputs in 64 bits.
"""
import math
import random

import torch

own = False

F32, F64, BF16 = torch.float32, torch.float64, torch.bfloat16


# ---------------------------------------------------------------------------------- the cases

def listed():
    return [
        # one short text: the smallest call, where the launches' latency counts
        dict(name="attn one short text", op="attn_fwd", T=77, docs=1, layout="packed", prefix=False, causal=True,
             H=12, Hkv=12, hd=64, cap=0.0, bias=False),
        # the 12-layer stack's batch (8 x 1024 tokens, 12 heads of 64) as texts packed end to end
        dict(name="attn packed texts", op="attn_train", T=8192, docs=23, layout="packed", prefix=False, causal=True,
             H=12, Hkv=12, hd=64, cap=0.0, bias=False),
        # prompts seen both ways with a distance bias, shared key heads, batch padded to one length
        dict(name="attn padded prompts", op="attn_train", T=4 * 1023, docs=4, layout="padded", prefix=True,
             causal=True, H=16, Hkv=4, hd=128, cap=0.0, bias=True),
        # capped scores over many short texts, wide heads
        dict(name="attn capped texts", op="attn_train", T=6000, docs=40, layout="packed", prefix=False, causal=True,
             H=8, Hkv=8, hd=128, cap=50.0, bias=False),
        # one long text with capped scores: the largest call
        dict(name="attn one long text", op="attn_fwd", T=16384, docs=1, layout="packed", prefix=False, causal=True,
             H=8, Hkv=2, hd=128, cap=30.0, bias=False),
        # image patches that see each other, several images in one row
        dict(name="attn images", op="attn_train", T=4900, docs=9, layout="packed", prefix=False, causal=False, H=12,
             Hkv=12, hd=64, cap=0.0, bias=False),
        # positions of one short prompt
        dict(name="rope one prompt", op="rope", T=33, H=24, hd=64, axes=3, dtype="bf16", per_axis=False, far=2000),
        # queries and keys of the 12-layer stack's batch, float32 storage, per-axis frequencies
        dict(name="rope stack batch", op="rope", T=8192, H=24, hd=64, axes=3, dtype="f32", per_axis=True, far=4000),
        # a long video: many tokens, far positions, shared key heads
        dict(name="rope long video", op="rope", T=50001, H=40, hd=128, axes=3, dtype="bf16", per_axis=False,
             far=1000000),
        # the float32 one-block model (B 4, S 256, d 256): few small tensors
        dict(name="adamw8 one block", op="adamw8", d=256, F=688, V=4096, layers=1, clip=1.0, shadow=False, step=10),
        # the 12-layer stack's width with a ragged vocabulary: clipped step that writes bf16 working weights
        dict(name="adamw8 stack", op="adamw8", d=768, F=2048, V=50257, layers=12, clip=1.0, shadow=True, step=1000),
        # an odd width, no clipping
        dict(name="adamw8 odd width", op="adamw8", d=1023, F=2731, V=8191, layers=6, clip=0.0, shadow=True, step=3),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn_fwd", "attn_train", "attn_train", "rope", "adamw8"])
    if op.startswith("attn"):
        # a text of one token has gradients of nought for its query and key: training cases have longer ones
        T = _log_int(rng, 1 if op == "attn_fwd" else 24, 12000)
        group, Hkv = rng.choice([1, 1, 2, 4]), rng.choice([1, 2, 3, 4, 6])
        while T * T * group * Hkv > 8192 * 8192 * 8:
            T = T * 2 // 3
        layout = rng.choice(["packed", "packed", "padded"])
        docs = min(T if op == "attn_fwd" else T // 12, _log_int(rng, 1, 64))
        if layout == "padded":
            T = max(1, T // docs) * docs
        causal = rng.random() < 0.8
        return dict(op=op, T=T, docs=docs, layout=layout, prefix=causal and rng.random() < 0.4, causal=causal,
                    H=group * Hkv, Hkv=Hkv, hd=rng.choice([64, 128]), cap=rng.choice([0.0, 0.0, 30.0, 50.0]),
                    bias=rng.random() < 0.35)
    if op == "rope":
        return dict(op=op, T=_log_int(rng, 1, 40000), H=rng.choice([1, 3, 8, 16, 24, 40]),
                    hd=rng.choice([32, 64, 80, 96, 128]), axes=rng.choice([1, 2, 3, 4]),
                    dtype=rng.choice(["bf16", "f32"]), per_axis=rng.random() < 0.5, far=_log_int(rng, 10, 1000000))
    return dict(op=op, d=_log_int(rng, 17, 1100), F=_log_int(rng, 50, 2800), V=_log_int(rng, 300, 50000),
                layers=rng.randint(1, 8), clip=rng.choice([0.0, 1.0, 1e6]), shadow=rng.random() < 0.5,
                step=_log_int(rng, 1, 20000))


# ---------------------------------------------------------------------------------- layouts

def _documents(case):
    """(offsets [docs + 1], valid lengths [docs], prefix lengths [docs]) of a case, as lists."""
    T, n = case["T"], case["docs"]
    rng = random.Random("%d %d %s" % (T, n, case["layout"]))
    if case["layout"] == "padded":
        span = T // n
        off = [i * span for i in range(n + 1)]
        lens = [rng.randint((span + 1) // 2, span) for _ in range(n)]
    else:
        off = [0] + sorted(rng.randint(0, T) for _ in range(n - 1)) + [T]
        lens = [off[i + 1] - off[i] for i in range(n)]
    pre = [rng.randint(0, (2 * m + 2) // 3) if case["prefix"] else 0 for m in lens]
    return off, lens, pre


def _visible_pairs(case):
    _, lens, pre = _documents(case)
    if not case["causal"]:
        return sum(m * m for m in lens)
    return sum(m * (m + 1) // 2 + min(p, m) * (min(p, m) - 1) // 2 for m, p in zip(lens, pre))


def _sections(hd, axes):
    """Pairs of each axis: half to the first where there are several, the rest shared out."""
    half = hd // 2
    if axes == 1:
        return [half]
    rest = half - half // 4
    cut = [rest // (axes - 1)] * (axes - 1)
    cut[-1] += rest - sum(cut)
    return [half // 4] + cut


def _tensor_sizes(case):
    d, F, V, L = case["d"], case["F"], case["V"], case["layers"]
    return [V * d, d] + [n for _ in range(L) for n in (d, d, 3 * d * d, d * d, d * F, F * d)]


def _places(case):
    """First element of each tensor in the flat buffers, and their length: whole blocks."""
    at, total = [], 0
    for n in _tensor_sizes(case):
        at.append(total)
        total += -(-n // BLOCK) * BLOCK
    return at, total


def _tensors(case, x):
    """The tensors (or their blocks' scales) in the flat buffer x."""
    at, total = _places(case)
    if x.numel() == total:
        return [x[a:a + n] for a, n in zip(at, _tensor_sizes(case))]
    return [x[a // BLOCK:a // BLOCK + -(-n // BLOCK)] for a, n in zip(at, _tensor_sizes(case))]


HYPER = dict(lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
GRAD_SCALE = 0.25  # four microbatches
BLOCK = 256        # elements that share a scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=F32)

    s = {"case": case}
    if case["op"].startswith("attn"):
        T, H, Hkv, hd = case["T"], case["H"], case["Hkv"], case["hd"]
        off, lens, pre = _documents(case)
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        s["off"], s["len"], s["prefix"] = ints(off), ints(lens), ints(pre)
        # query, key and value heads as the column blocks of one projection's output; scores of a few units, and
        # near the cap where there is one
        qkv = normal(T, (H + 2 * Hkv) * hd)
        qkv[:, :H * hd] *= 6.0 if case["cap"] > 0 else 1.5
        s["qkv"] = qkv.to(BF16)
        s["q"], s["k"], s["v"] = s["qkv"].split([H * hd, Hkv * hd, Hkv * hd], dim=1)
        s["slopes"] = None
        if case["bias"]:
            s["slopes"] = torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda", dtype=F32) / H)
        if case["op"] == "attn_train":
            s["do"] = normal(T, H * hd).to(BF16)
    elif case["op"] == "rope":
        T, H, hd = case["T"], case["H"], case["hd"]
        dt = BF16 if case["dtype"] == "bf16" else F32
        s["x"], s["dy"] = normal(T, H * hd).to(dt), normal(T, H * hd).to(dt)
        # positions that rise along the row from a start of the document's own, restarted now and then
        step = torch.randint(0, 3, (case["axes"], T), generator=g, device="cuda")
        start = torch.randint(0, case["far"], (case["axes"], 1), generator=g, device="cuda")
        s["pos"] = (start + step.cumsum(1) % max(1, case["far"])).to(torch.int32)
    else:
        # every state in one buffer, the tensors one behind another, each from a multiple of a block on
        at, total = _places(case)
        each = torch.repeat_interleave(torch.tensor([0.02, 0.001, 0.005] * len(at), device="cuda")[:len(at)],
                                       torch.tensor([b - a for a, b in zip(at, at[1:] + [total])], device="cuda"))
        used = torch.zeros(total, device="cuda", dtype=torch.bool)
        for start, n in zip(at, _tensor_sizes(case)):
            used[start:start + n] = True
        code = lambda lo, hi: torch.randint(lo, hi + 1, (total,), generator=g, device="cuda") * used  # noqa: E731
        scale = lambda top: (torch.rand(total // BLOCK, generator=g, device="cuda") + 0.5) * top  # noqa: E731
        flat = {"p": 0.02 * normal(total) * used, "g": normal(total) * each * used, "m8": code(-127, 127).to(torch.int8),
                "r8": code(1, 255).to(torch.uint8), "ms": scale(1e-3 / 127 ** 2), "rs": scale(4e-3 / 255 ** 2)}
        if case["shadow"]:
            flat["w"] = torch.zeros(total, dtype=BF16, device="cuda")
        s["flat"] = flat
        for name, x in flat.items():
            s[name] = _tensors(case, x)
    return s


def work(case):
    if case["op"].startswith("attn"):
        T, H, Hkv, hd = case["T"], case["H"], case["Hkv"], case["hd"]
        pairs = _visible_pairs(case) * H
        io = T * hd * 2
        if case["op"] == "attn_fwd":
            return {"bytes": io * (2 * H + 2 * Hkv) + T * H * 4, "flops": 4 * hd * pairs}
        # forward, then q, k, v, o, do and lse read and dq, dk, dv written
        return {"bytes": io * (2 * H + 2 * Hkv) + io * (4 * H + 4 * Hkv) + T * H * 8, "flops": 14 * hd * pairs}
    if case["op"] == "rope":
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 4 * case["T"] * case["H"] * case["hd"] * size + 8 * case["axes"] * case["T"],
                "flops": 6 * case["T"] * case["H"] * case["hd"]}
    n = sum(_tensor_sizes(case))
    # weights read and written, gradient (twice with clipping: its norm comes first), codes read and written,
    # the working copy, and the two moments as the values that the codes stand for
    per = 8 + 4 + (4 if case["clip"] > 0 else 0) + 4 + (2 if case["shadow"] else 0) + 2 + 8
    return {"bytes": n * per, "flops": 30 * n}


# ---------------------------------------------------------------------------------- run

def run(state):
    op = state["case"]["op"]
    if op.startswith("attn"):
        return _attention_own(state) if own else _attention_plain(state)
    if op == "rope":
        return _rope_own(state) if own else _rope_plain(state)
    return _adamw8_own(state) if own else _adamw8_plain(state)


def _mask(state, causal):
    """visible[i, j] of tokens i, j."""
    T = state["case"]["T"]
    t = torch.arange(T, device="cuda")
    doc = torch.searchsorted(state["off"][1:].long(), t, right=True).clamp(max=state["case"]["docs"] - 1)
    inner = t - state["off"].long()[doc]
    valid = inner < state["len"].long()[doc]
    see = (doc[:, None] == doc[None, :]) & valid[:, None] & valid[None, :]
    if causal:
        see &= (t[None, :] <= t[:, None]) | (inner < state["prefix"].long()[doc])[None, :]
    return see, valid


def _attention_plain(state):
    c = state["case"]
    T, H, Hkv, hd = c["T"], c["H"], c["Hkv"], c["hd"]
    G, scale = H // Hkv, 1.0 / math.sqrt(hd)
    see, valid = _mask(state, c["causal"])
    q = state["q"].float().view(T, Hkv, G, hd).permute(1, 2, 0, 3).reshape(Hkv, G * T, hd)
    k = state["k"].float().view(T, Hkv, hd).transpose(0, 1)
    v = state["v"].float().view(T, Hkv, hd).transpose(0, 1)
    a = torch.bmm(q, k.transpose(1, 2)).mul_(scale).view(Hkv, G, T, T)
    th = None
    if c["cap"] > 0:
        th = torch.tanh_(a.div_(c["cap"]))
        a = th * c["cap"]
    if c["bias"]:
        t = torch.arange(T, device="cuda", dtype=F32)
        a = a.sub_(state["slopes"].view(Hkv, G, 1, 1) * (t[:, None] - t[None, :]).abs())
    a.masked_fill_(~see, -math.inf)
    top = a.amax(-1, keepdim=True)
    e = a.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    total = e.sum(-1, keepdim=True)
    lse = (top + torch.log(total)).view(H, T)
    p = e.div_(total.masked_fill(total == 0, 1.0)).view(Hkv, G * T, T)
    o = torch.bmm(p, v)
    back = lambda x: x.view(Hkv, G, T, hd).permute(2, 0, 1, 3).reshape(T, H * hd).to(BF16)  # noqa: E731
    if c["op"] == "attn_fwd":
        return {"o": back(o), "lse": lse}
    do = state["do"].float().view(T, Hkv, G, hd).permute(1, 2, 0, 3).reshape(Hkv, G * T, hd)
    dv = torch.bmm(p.transpose(1, 2), do)
    ds = torch.bmm(do, v.transpose(1, 2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    if th is not None:
        ds = ds.view(Hkv, G, T, T).mul_(th.square_().neg_().add_(1.0)).view(Hkv, G * T, T)
    dq = torch.bmm(ds, k) * scale
    dk = torch.bmm(ds.transpose(1, 2), q) * scale
    cols = lambda x: x.transpose(0, 1).reshape(T, Hkv * hd).to(BF16)  # noqa: E731
    return {"o": back(o), "lse": lse, "dq": back(dq), "dk": cols(dk), "dv": cols(dv)}


def _attention_own(state):
    from transformer_fwd_bwd_gb300 import xt
    c = state["case"]
    T, H, Hkv, hd = c["T"], c["H"], c["Hkv"], c["hd"]
    if "plan" not in state:  # the buffers that a training program keeps over its steps
        state["plan"] = xt.attention_plan_buffer(T)
        state["o"] = torch.empty(T, H * hd, dtype=BF16, device="cuda")
        state["lse"] = torch.empty(H, T, dtype=F32, device="cuda")
        if c["op"] == "attn_train":
            state["dqkv"] = torch.empty_like(state["qkv"])
            state["ws"] = xt.attention_masked_workspace(T, H, Hkv, hd)
    q, k, v, o, lse, plan = (state[n] for n in ("q", "k", "v", "o", "lse", "plan"))
    xt.xt_attention_plan(plan, T, c["docs"], state["off"], state["len"], state["prefix"], causal=int(c["causal"]))
    xt.xt_attention_masked_fwd(q, k, v, o, lse, plan, H, Hkv, hd, cap=c["cap"], slopes=state["slopes"])
    if c["op"] == "attn_fwd":
        return {"o": o, "lse": lse}
    dq, dk, dv = state["dqkv"].split([H * hd, Hkv * hd, Hkv * hd], dim=1)
    xt.xt_attention_masked_bwd(q, k, v, o, state["do"], lse, dq, dk, dv, plan, H, Hkv, hd, cap=c["cap"],
                               slopes=state["slopes"], ws=state["ws"])
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


ROPE_BASE = 10000.0


def _rope_plain(state):
    c = state["case"]
    T, H, hd = c["T"], c["H"], c["hd"]
    half, sec = hd // 2, torch.tensor(_sections(c["hd"], c["axes"]), device="cuda")
    pair = torch.arange(half, device="cuda")
    ends = sec.cumsum(0)
    axis = torch.searchsorted(ends, pair, right=True)
    if c["per_axis"]:
        power = (pair - (ends - sec)[axis]).to(F64) / sec[axis].to(F64)
    else:
        power = pair.to(F64) / half
    # far positions: the angle in 64 bits
    angle = state["pos"][axis].t().to(F64) * torch.pow(torch.tensor(ROPE_BASE, dtype=F64, device="cuda"), -power)
    cos, sin = torch.cos(angle).to(F32)[:, None, :], torch.sin(angle).to(F32)[:, None, :]
    x = state["x"].float().view(T, H, 2, half)
    d = state["dy"].float().view(T, H, 2, half)
    y = torch.stack((x[:, :, 0] * cos - x[:, :, 1] * sin, x[:, :, 1] * cos + x[:, :, 0] * sin), 2)
    dx = torch.stack((d[:, :, 0] * cos + d[:, :, 1] * sin, d[:, :, 1] * cos - d[:, :, 0] * sin), 2)
    return {"y": y.view(T, H * hd).to(state["x"].dtype), "dx": dx.view(T, H * hd).to(state["x"].dtype)}


def _rope_own(state):
    from transformer_fwd_bwd_gb300 import xt
    c = state["case"]
    if "y" not in state:
        state["y"], state["dx"] = torch.empty_like(state["x"]), torch.empty_like(state["x"])
    sections = _sections(c["hd"], c["axes"])
    xt.xt_rope_axes_fwd(state["x"], state["y"], state["pos"], sections, c["H"], c["hd"], ROPE_BASE,
                        per_axis=int(c["per_axis"]))
    xt.xt_rope_axes_bwd(state["dy"], state["dx"], state["pos"], sections, c["H"], c["hd"], ROPE_BASE,
                        per_axis=int(c["per_axis"]))
    return {"y": state["y"], "dx": state["dx"]}


def _f(x):
    """The float32 value of a hyperparameter, as a Python number."""
    return float(torch.tensor(x, dtype=F32))


def _adamw8_plain(state):
    c, s = state["case"], state["flat"]
    lr, b1, b2, eps, wd = (HYPER[k] for k in ("lr", "beta1", "beta2", "eps", "weight_decay"))
    b1, b2 = _f(b1), _f(b2)
    bc1, bc2 = 1.0 - b1 ** c["step"], 1.0 - b2 ** c["step"]
    out, factor = {}, GRAD_SCALE
    if c["clip"] > 0:
        norm = s["g"].double().square().sum().sqrt() * GRAD_SCALE
        factor = (GRAD_SCALE * (c["clip"] / (norm + 1e-6)).clamp(max=1.0)).to(F32)
        out["norm"] = norm.to(F32)
    blocks = lambda x: x.view(-1, BLOCK)  # noqa: E731
    g = blocks(s["g"]) * factor
    cm, cr = blocks(s["m8"]).to(F32), blocks(s["r8"]).to(F32)
    m = cm * cm.abs() * s["ms"][:, None]
    r = cr * cr * s["rs"][:, None]
    # every operation of the held moments is rounded to float32 by itself: it settles their codes
    m = m * b1 + g * _f(1.0 - b1)
    v = (r * r) * b2 + (g * _f(1.0 - b2)) * g
    r = v.sqrt()
    s["p"].copy_((blocks(s["p"]) * (1.0 - lr * wd) - (lr / bc1) * m / (r * math.sqrt(1.0 / bc2) + eps)).view(-1))
    # divided by tensors: a division by a number multiplies by its rounded reciprocal
    top = torch.tensor([16129.0, 65025.0], device="cuda")
    ms = m.abs().amax(1, keepdim=True) / top[0]
    rs = r.amax(1, keepdim=True) / top[1]
    cm = (m.abs() / ms).sqrt().round().nan_to_num(0.0) * m.sign()
    cr = (r / rs).sqrt().round().nan_to_num(0.0)
    cr = torch.where(v > 0, cr.clamp(min=1.0), cr)
    for name, new in (("m8", cm), ("r8", cr), ("ms", ms), ("rs", rs)):
        s[name].copy_(new.view(-1))
    out["p"] = s["p"]
    if c["shadow"]:
        out["w"] = s["w"].copy_(s["p"])
    out["m"], r = (cm * cm.abs() * ms).view(-1), cr * cr * rs
    out["v"] = (r * r).view(-1)
    return out


def _adamw8_own(state):
    from transformer_fwd_bwd_gb300 import xt
    c, s = state["case"], state["flat"]
    if "ws" not in state:
        state["norm"] = torch.empty(1, dtype=F32, device="cuda") if c["clip"] > 0 else None
        state["ws"] = xt.adamw8_workspace([t.numel() for t in state["p"]])
        s["m"], s["v"] = torch.zeros_like(s["p"]), torch.zeros_like(s["p"])
        state["m"], state["v"] = _tensors(c, s["m"]), _tensors(c, s["v"])
    cfg = xt.adamw_config(HYPER["lr"], HYPER["beta1"], HYPER["beta2"], HYPER["eps"], HYPER["weight_decay"],
                          c["clip"], GRAD_SCALE, c["step"])
    xt.xt_adamw8_step(cfg, state["p"], state["g"], state["m8"], state["r8"], state["ms"], state["rs"],
                      shadows=state.get("w"), norm_out=state["norm"], ws=state["ws"])
    xt.xt_adamw8_decode(state["m8"], state["r8"], state["ms"], state["rs"], state["m"], state["v"])
    out = {name: s[name] for name in ("p", "m", "v")}
    if c["shadow"]:
        out["w"] = s["w"]
    if c["clip"] > 0:
        out["norm"] = state["norm"].view(())
    return out


# ---------------------------------------------------------------------------------- exact

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("attn"):
        return _attention_exact(case, s)
    if case["op"] == "rope":
        return _rope_exact(case, s)
    return _adamw8_exact(case, s)


def _attention_exact(case, s):
    """Head by head and document by document, from the definition of the softmax."""
    T, H, Hkv, hd = case["T"], case["H"], case["Hkv"], case["hd"]
    off, lens, pre = _documents(case)
    train = case["op"] == "attn_train"
    new = lambda n: torch.zeros(T, n, hd, dtype=F64, device="cuda")  # noqa: E731
    q, k, v = (s[n].double().view(T, -1, hd) for n in ("q", "k", "v"))
    o, lse = new(H), torch.full((H, T), -math.inf, dtype=F64, device="cuda")
    if train:
        do, dq, dk, dv = s["do"].double().view(T, H, hd), new(H), new(Hkv), new(Hkv)
    for b, m, pl in zip(off, lens, pre):
        if m == 0:
            continue
        at = slice(b, b + m)
        i = torch.arange(m, device="cuda")
        hidden = (i[None, :] > i[:, None]) & (i >= pl)[None, :] if case["causal"] else None
        for h in range(H):
            kh = h // (H // Hkv)
            Q, K, V = q[at, h], k[at, kh], v[at, kh]
            z = Q @ K.T / math.sqrt(hd)
            t = None
            if case["cap"] > 0:
                t = torch.tanh(z / case["cap"])
                z = case["cap"] * t
            if case["bias"]:
                z = z - float(s["slopes"][h]) * (i[:, None] - i[None, :]).abs()
            if hidden is not None:
                z = z.masked_fill(hidden, -math.inf)
            lse[h, at] = torch.logsumexp(z, 1)
            p = torch.exp(z - lse[h, at][:, None])
            o[at, h] = p @ V
            if train:
                G = do[at, h]
                dv[at, kh] += p.T @ G
                dp = G @ V.T
                ds = p * (dp - (p * dp).sum(1, keepdim=True))
                if t is not None:
                    ds = ds * (1 - t * t)
                dq[at, h] = ds @ K / math.sqrt(hd)
                dk[at, kh] += ds.T @ Q / math.sqrt(hd)
    flat = lambda x: x.reshape(T, -1)  # noqa: E731
    if not train:
        return {"o": flat(o), "lse": lse}
    return {"o": flat(o), "lse": lse, "dq": flat(dq), "dk": flat(dk), "dv": flat(dv)}


def _rope_exact(case, s):
    T, H, hd, half = case["T"], case["H"], case["hd"], case["hd"] // 2
    angle = torch.empty(T, half, dtype=F64, device="cuda")
    i = 0
    for a, n in enumerate(_sections(hd, case["axes"])):
        for k in range(n):
            f = ROPE_BASE ** (-(k / n if case["per_axis"] else 2 * i / hd))
            angle[:, i] = s["pos"][a].double() * f
            i += 1
    turn = torch.polar(torch.ones_like(angle), angle)[:, None, :]

    def rotate(x, by):
        x = x.double().view(T, H, hd)
        z = torch.complex(x[..., :half], x[..., half:]) * by
        return torch.cat((z.real, z.imag), -1).view(T, H * hd)
    return {"y": rotate(s["x"], turn), "dx": rotate(s["dy"], turn.conj())}


def _adamw8_exact(case, s):
    """Weights from moments in 64 bits. The held moments are float32 numbers put into codes: their
    values before that are rounded where the definition rounds them."""
    lr, eps, wd = HYPER["lr"], HYPER["eps"], HYPER["weight_decay"]
    b1, b2 = _f(HYPER["beta1"]), _f(HYPER["beta2"])
    c1, c2 = _f(1.0 - b1), _f(1.0 - b2)
    r32 = lambda x: x.to(F32).to(F64)  # noqa: E731
    norm = GRAD_SCALE * math.sqrt(math.fsum(float((g.double() ** 2).sum()) for g in s["g"]))
    f = _f(GRAD_SCALE * (min(1.0, case["clip"] / (norm + 1e-6)) if case["clip"] > 0 else 1.0))
    out = {name: torch.zeros_like(s["flat"]["p"], dtype=F64) for name in ("p", "m", "v")}
    P, M, V = (_tensors(case, out[name]) for name in ("p", "m", "v"))
    for i, (p, g, m8, r8, ms, rs) in enumerate(
            zip(s["p"], s["g"], s["m8"], s["r8"], s["ms"], s["rs"])):
        n = p.numel()
        rows = torch.arange(n, device="cuda") // BLOCK
        blocks = ms.numel()
        per = lambda x, rows=rows: x[rows]  # noqa: E731
        m0 = r32(m8.double() * m8.double().abs() * per(ms.double()))
        r0 = r32(r8.double() ** 2 * per(rs.double()))
        g64 = g.double() * f
        m64, v64 = b1 * m0 + (1 - b1) * g64, b2 * r0 * r0 + (1 - b2) * g64 ** 2
        step = (m64 / (1 - b1 ** case["step"])) / ((v64 / (1 - b2 ** case["step"])).sqrt() + eps)
        P[i].copy_(p.double() * (1 - lr * wd) - lr * step)
        g32 = r32(g64)
        m1 = r32(r32(b1 * m0) + r32(c1 * g32))
        v1 = r32(r32(b2 * r32(r0 * r0)) + r32(r32(c2 * g32) * g32))
        r1 = r32(v1.sqrt())
        top = lambda x, rows=rows, blocks=blocks: torch.zeros(blocks, dtype=F64, device="cuda").scatter_reduce(  # noqa: E731
            0, rows, x, "amax")
        ms1, rs1 = r32(top(m1.abs()) / 16129.0), r32(top(r1) / 65025.0)
        root = lambda x, d: torch.where(d > 0, r32(r32(x / d).sqrt()).round(), torch.zeros_like(x))  # noqa: E731
        cm = root(m1.abs(), per(ms1)) * m1.sign()
        cr = root(r1, per(rs1))
        cr = torch.where(v1 > 0, cr.clamp(min=1.0), cr)
        M[i].copy_(r32(cm * cm.abs() * per(ms1)))
        V[i].copy_(r32(r32(cr * cr * per(rs1)) ** 2))
    if case["clip"] > 0:
        out["norm"] = norm
    if case["shadow"]:
        out["w"] = out["p"]
    return out
