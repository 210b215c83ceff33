"""The work of the operators at both ends and in the middle of a training step: log probabilities of given
tokens with entropy, top alternatives and their gradient; embedding lookup with scaling and its gradient by
sorted tokens; the gated feed-forward block with its backward pass; the Muon step, which orthogonalises a
momentum by Newton-Schulz products.

A case names an operator and its sizes; prepare() makes the inputs on the GPU from a seed; run()
makes one pass, in elementary torch operations (own = False) or through this repository's library
(own = True); exact() computes the same outputs in 64 bits.
"""
import math

import torch

own = False

F32, F64, BF16 = torch.float32, torch.float64, torch.bfloat16
DTYPE = {"f32": F32, "bf16": BF16}


# ---------------------------------------------------------------------------------- the cases

def listed():
    return [
        # the next tokens of three texts scored, with five alternatives each: the smallest call
        dict(name="logprobs three tokens", op="logprobs", R=3, V=50257, dtype="bf16", top=5, train=False, scale=1.0,
             banned=0.0),
        # the 12-layer stack's batch: log probabilities and entropies that a policy loss differentiates
        dict(name="logprobs stack batch", op="logprobs", R=8192, V=50304, dtype="bf16", top=0, train=True, scale=1.0,
             banned=0.0),
        # a wide vocabulary with twenty alternatives per token, as a teacher's answers are recorded
        dict(name="logprobs wide vocabulary", op="logprobs", R=4096, V=128256, dtype="bf16", top=20, train=False,
             scale=1.0, banned=0.0),
        # float32 logits, an odd vocabulary with a tenth of it banned, a temperature
        dict(name="logprobs odd vocabulary", op="logprobs", R=777, V=50257, dtype="f32", top=8, train=True, scale=1.25,
             banned=0.1),
        # one short prompt
        dict(name="embed one prompt", op="embed", T=37, d=768, V=50304, dtype="bf16", grad="f32", acc=1, scale=1.0),
        # the 12-layer stack's batch, gradients added over microbatches
        dict(name="embed stack batch", op="embed", T=8192, d=768, V=50304, dtype="bf16", grad="f32", acc=1,
             scale=math.sqrt(768.0)),
        # a long batch over a wide vocabulary, the gradient written afresh
        dict(name="embed long batch", op="embed", T=131072, d=1024, V=128256, dtype="bf16", grad="f32", acc=0,
             scale=32.0),
        # one short prompt through the block
        dict(name="gated one prompt", op="gated", T=77, d=768, F=2048, act="silu", train=False),
        # the 12-layer stack's batch, forward and backward
        dict(name="gated stack batch", op="gated", T=8192, d=768, F=2048, act="silu", train=True),
        # a wide block with ragged sizes
        dict(name="gated wide block", op="gated", T=12001, d=2048, F=5464, act="gelu", train=True),
        # the one-block model's matrices
        dict(name="muon one block", op="muon", d=256, F=688, layers=1, shadow=False),
        # the 12-layer stack's width
        dict(name="muon stack", op="muon", d=768, F=2048, layers=12, shadow=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "embed", "gated", "muon"])
    if op == "logprobs":
        V = _log_int(rng, 300, 130000)
        train = rng.random() < 0.5
        return dict(op=op, R=_log_int(rng, 1, max(1, 8192 * 50304 // V if not train else 4096 * 50304 // V)), V=V,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), top=rng.choice([0, 1, 5, 8, 20, 32]), train=train,
                    scale=rng.choice([1.0, 1.0, 0.7, 1.25]), banned=rng.choice([0.0, 0.0, 0.1, 0.5]))
    if op == "embed":
        d = rng.choice([8 * _log_int(rng, 4, 256), _log_int(rng, 17, 1100)])
        return dict(op=op, T=_log_int(rng, 1, 60000), d=d, V=_log_int(rng, 300, 130000 * 1024 // max(d, 1024)),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), grad=rng.choice(["f32", "f32", "bf16"]),
                    acc=rng.randint(0, 1), scale=rng.choice([1.0, math.sqrt(d)]))
    if op == "gated":
        d, F = 8 * _log_int(rng, 4, 256), 8 * _log_int(rng, 6, 680)
        T = _log_int(rng, 1, 12000)
        return dict(op=op, T=T, d=d, F=F, act=rng.choice(["silu", "silu", "gelu"]), train=rng.random() < 0.6)
    d = _log_int(rng, 17, 800)
    return dict(op=op, d=d, F=_log_int(rng, 40, 2500), layers=rng.randint(1, 6), shadow=rng.random() < 0.5)


# ---------------------------------------------------------------------------------- inputs

MUON = dict(lr=0.02, momentum=0.95, weight_decay=0.1, rms=0.2, eps=1e-7, steps=5)
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
GRAD_SCALE = 0.25  # four microbatches


def _shapes(case):
    """The matrices of every layer: query-key-value, output, gate and up, down."""
    d, F = case["d"], case["F"]
    return [s for _ in range(case["layers"]) for s in ((d, 3 * d), (d, d), (d, 2 * F), (F, d))]


def _places(case):
    """First element of each matrix in the flat buffers, and their length: each from a multiple of 64 on."""
    at, total = [], 0
    for n, m in _shapes(case):
        at.append(total)
        total += -(-n * m // 64) * 64
    return at, total


def _matrices(case, x):
    """The matrices in the flat buffer x."""
    return [x[a:a + n * m].view(n, m) for a, (n, m) in zip(_places(case)[0], _shapes(case))]


def _token_weights(V):
    """Tokens by falling frequency."""
    return 1.0 / (torch.arange(V, device="cuda", dtype=F64) + 10.0)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 29)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=F32)

    s = {"case": case}
    if case["op"] == "logprobs":
        R, V = case["R"], case["V"]
        x = torch.empty(R, V, dtype=DTYPE[case["dtype"]], device="cuda")
        for r in range(0, R, 1024):
            n = min(1024, R - r)
            x[r:r + n] = 2.5 * normal(n, V)
        allowed = torch.arange(V, device="cuda")
        if case["banned"] > 0:
            keep = torch.rand(V, generator=g, device="cuda") >= case["banned"]
            keep[:64] = True
            x[:, ~keep] = -math.inf
            allowed = allowed[keep]
        s["logits"] = x
        s["tokens"] = allowed[torch.randint(0, allowed.numel(), (R,), generator=g, device="cuda")].to(torch.int32)
        if case["train"]:
            # advantages of the tokens, and the weight of an entropy bonus
            s["d_logp"], s["d_entropy"] = normal(R) / R, (0.01 + 0.01 * torch.rand(R, generator=g, device="cuda")) / R
    elif case["op"] == "embed":
        T, d, V, dt = case["T"], case["d"], case["V"], DTYPE[case["dtype"]]
        s["E"] = (0.02 * normal(V, d)).to(dt)
        s["ids"] = torch.multinomial(_token_weights(V), T, replacement=True, generator=g).to(torch.int32)
        s["dh"] = (1e-2 * normal(T, d)).to(dt)
        s["dE"] = (1e-2 * normal(V, d)).to(DTYPE[case["grad"]])  # what earlier microbatches left
    elif case["op"] == "gated":
        T, d, F = case["T"], case["d"], case["F"]
        s["x"] = normal(T, d).to(BF16)
        s["w_up"], s["w_down"] = (normal(d, 2 * F) * d ** -0.5).to(BF16), (normal(F, d) * F ** -0.5).to(BF16)
        if case["train"]:
            s["dy"] = normal(T, d).to(BF16)
    else:
        # gradients of a few strong directions and noise
        def matrix(n, m, size):
            r = min(16, n, m)
            return size * (normal(n, r) @ normal(r, m) / math.sqrt(r) + 0.3 * normal(n, m))
        # every state in one buffer, the matrices one behind another
        s["flat"] = {name: torch.zeros(_places(case)[1], device="cuda", dtype=F32) for name in ("p", "g", "buf")}
        if case["shadow"]:
            s["flat"]["w"] = torch.zeros_like(s["flat"]["p"], dtype=BF16)
        for name, x in s["flat"].items():
            s[name] = _matrices(case, x)
        for (n, m), p, grad, buf in zip(_shapes(case), s["p"], s["g"], s["buf"]):
            p.copy_(0.02 * normal(n, m))
            grad.copy_(matrix(n, m, 1e-3))
            buf.copy_(matrix(n, m, 2e-3))
    return s


def _distinct(T, V):
    """Expected number of distinct tokens among T."""
    w = [1.0 / (v + 10.0) for v in range(V)]
    total = sum(w)
    return sum(1.0 - math.exp(T * math.log1p(-x / total)) for x in w)


def work(case):
    if case["op"] == "logprobs":
        R, V, e = case["R"], case["V"], 2 if case["dtype"] == "bf16" else 4
        fwd = R * V * e + R * (4 + 8 + 8 * case["top"])
        # forward, then the logits and row values read and the gradient written
        return {"bytes": fwd + (2 * R * V * e + R * 20 if case["train"] else 0),
                "flops": R * V * (5 + (6 if case["train"] else 0))}
    if case["op"] == "embed":
        T, d, V = case["T"], case["d"], case["V"]
        e, eg, rows = (2 if case["dtype"] == "bf16" else 4), (2 if case["grad"] == "bf16" else 4), _distinct(T, V)
        grad = 2 * rows * d * eg if case["acc"] else V * d * eg
        return {"bytes": 8 * T + rows * d * e + 2 * T * d * e + grad, "flops": 2 * T * d}
    if case["op"] == "gated":
        T, d, F = case["T"], case["d"], case["F"]
        if not case["train"]:
            return {"bytes": 4 * T * d + 6 * d * F, "flops": 6 * T * d * F}
        return {"bytes": 8 * T * d + 12 * d * F, "flops": 18 * T * d * F}
    n = sum(a * b for a, b in _shapes(case))
    flops = 0
    for a, b in _shapes(case):
        k, m = min(a, b), max(a, b)
        flops += MUON["steps"] * (k * (k + 1) * m + k * k * (k + 1) + 2 * k * k * m)
    # gradient read, momentum and weights read and written, the working copy written
    return {"bytes": n * (4 + 8 + 8 + (2 if case["shadow"] else 0)), "flops": flops}


# ---------------------------------------------------------------------------------- run

def run(state):
    op = state["case"]["op"]
    if op == "logprobs":
        return _logprobs_own(state) if own else _logprobs_plain(state)
    if op == "embed":
        return _embed_own(state) if own else _embed_plain(state)
    if op == "gated":
        return _gated_own(state) if own else _gated_plain(state)
    return _muon_own(state) if own else _muon_plain(state)


def _top_ids(z, k):
    """Indexes of the k largest of each row of float32 z, ties to the lowest index."""
    bits = (z + 0.0).view(torch.int32)
    key = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long() << 32
    key += torch.arange(z.shape[1] - 1, -1, -1, device=z.device)
    return key.topk(k, dim=1).indices


def _logprobs_plain(s):
    c = s["case"]
    R, V, k, scale = c["R"], c["V"], c["top"], c["scale"]
    new = lambda *shape, dt=F32: torch.empty(*shape, dtype=dt, device="cuda")  # noqa: E731
    out = {"logp": new(R), "entropy": new(R)}
    if k:
        out["top_logp"], out["top_ids"] = new(R, k), new(R, k, dt=torch.int32)
    if c["train"]:
        out["dlogits"] = torch.empty_like(s["logits"])
    for r in range(0, R, 2048):
        at = slice(r, min(R, r + 2048))
        z = s["logits"][at].float() * scale
        tok = s["tokens"][at].long()[:, None]
        top = z.amax(1, keepdim=True)
        e = torch.exp(z - top)
        total = e.sum(1, keepdim=True)
        logp = z - (top + torch.log(total))
        p = e / total
        plogp = torch.where(p > 0, p * logp, torch.zeros_like(p))
        entropy = -plogp.sum(1, keepdim=True)
        out["logp"][at], out["entropy"][at] = logp.gather(1, tok)[:, 0], entropy[:, 0]
        if k:
            ids = _top_ids(s["logits"][at].float(), k)
            out["top_logp"][at], out["top_ids"][at] = logp.gather(1, ids), ids.to(torch.int32)
        if c["train"]:
            dlp, dh = s["d_logp"][at][:, None], s["d_entropy"][at][:, None]
            d = -p * dlp - dh * (plogp + p * entropy)
            d.scatter_add_(1, tok, dlp)
            out["dlogits"][at] = d * scale
    return out


def _logprobs_own(s):
    from transformer_fwd_bwd_gb300 import xt
    c = s["case"]
    R, k = c["R"], c["top"]
    if "logp" not in s:  # the buffers that a program keeps over its steps
        new = lambda *shape, dt=F32: torch.empty(*shape, dtype=dt, device="cuda")  # noqa: E731
        s["logp"], s["entropy"], s["stats"] = new(R), new(R), new(R, 2)
        s["top_logp"], s["top_ids"] = (new(R, k), new(R, k, dt=torch.int32)) if k else (None, None)
        if c["train"]:
            s["dlogits"] = torch.empty_like(s["logits"])
    xt.xt_token_logprobs_fwd(s["logits"], s["tokens"], s["logp"], s["entropy"], s["stats"], s["top_logp"],
                             s["top_ids"], scale=c["scale"])
    out = {"logp": s["logp"], "entropy": s["entropy"]}
    if k:
        out["top_logp"], out["top_ids"] = s["top_logp"], s["top_ids"]
    if c["train"]:
        xt.xt_token_logprobs_bwd(s["logits"], s["tokens"], s["stats"], s["entropy"], s["d_logp"], s["d_entropy"],
                                 s["dlogits"], scale=c["scale"])
        out["dlogits"] = s["dlogits"]
    return out


def _embed_plain(s):
    c = s["case"]
    ids = s["ids"].long()
    h = (s["E"][ids].float() * c["scale"]).to(s["E"].dtype)
    d = torch.zeros(c["V"], c["d"], dtype=F32, device="cuda")
    d.index_add_(0, ids, s["dh"].float())
    d *= c["scale"]
    if c["acc"]:
        d += s["dE"].float()
    s["dE"].copy_(d)
    return {"h": h, "dE": s["dE"]}


def _embed_own(s):
    from transformer_fwd_bwd_gb300 import xt
    c = s["case"]
    if "h" not in s:
        s["h"], s["plan"] = torch.empty_like(s["dh"]), xt.embedding_plan_buffer(c["T"])
        s["ws"] = xt.embedding_sorted_workspace(c["T"], c["d"])
    xt.xt_embedding_lookup_fwd(s["ids"], s["E"], s["h"], scale=c["scale"])
    xt.xt_embedding_plan(s["ids"], c["V"], s["plan"])
    xt.xt_embedding_sorted_bwd(s["plan"], s["dh"], s["dE"], scale=c["scale"], acc=c["acc"], ws=s["ws"])
    return {"h": s["h"], "dE": s["dE"]}


def _gate(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        sig = torch.sigmoid(g)
        return g * sig, sig * (1.0 + g * (1.0 - sig))
    cdf = 0.5 * torch.erfc(g * -math.sqrt(0.5))
    return g * cdf, cdf + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)


def _gated_plain(s):
    c = s["case"]
    x, wu, wd = s["x"].float(), s["w_up"].float(), s["w_down"].float()
    gu = x @ wu
    g, u = gu[:, :c["F"]], gu[:, c["F"]:]
    a, da = _gate(g, c["act"])
    h = a * u
    out = {"y": (h @ wd).to(BF16)}
    if c["train"]:
        dy = s["dy"].float()
        dh = dy @ wd.T
        dgu = torch.cat((dh * u * da, dh * a), 1)
        out["dx"] = (dgu @ wu.T).to(BF16)
        out["dw_up"], out["dw_down"] = (x.T @ dgu).to(BF16), (h.T @ dy).to(BF16)
    return out


def _gated_own(s):
    from transformer_fwd_bwd_gb300 import xt
    c = s["case"]
    T, d, F = c["T"], c["d"], c["F"]
    act = {"silu": xt.XT_GATE_SILU, "gelu": xt.XT_GATE_GELU}[c["act"]]
    if "y" not in s:
        new = lambda *shape, dt=BF16: torch.empty(*shape, dtype=dt, device="cuda")  # noqa: E731
        s["h"], s["y"], s["gu"] = new(T, F), new(T, d), None
        s["ws"] = xt.gated_mlp_workspace(T, d, F)
        if c["train"]:
            s["gu"], s["dgu"], s["dx"] = new(T, 2 * F), new(T, 2 * F), new(T, d)
            s["dw_up"], s["dw_down"] = torch.empty_like(s["w_up"]), torch.empty_like(s["w_down"])
    xt.xt_gated_mlp_fwd(s["x"], s["w_up"], s["w_down"], s["gu"], s["h"], s["y"], act=act, ws=s["ws"])
    out = {"y": s["y"]}
    if c["train"]:
        xt.xt_gated_mlp_bwd(s["x"], s["w_up"], s["w_down"], s["gu"], s["h"], s["dy"], s["dgu"], s["dx"], s["dw_up"],
                            s["dw_down"], act=act, ws=s["ws"])
        out.update(dx=s["dx"], dw_up=s["dw_up"], dw_down=s["dw_down"])
    return out


def _muon_outputs(s):
    return {name: s["flat"][name] for name in ("p", "buf", "w") if name in s["flat"]}


def _muon_plain(s):
    a, b, c = COEFFICIENTS
    lr, mu, wd = MUON["lr"], MUON["momentum"], MUON["weight_decay"]
    for i, (p, g, buf) in enumerate(zip(s["p"], s["g"], s["buf"])):
        g = g * GRAD_SCALE
        buf.mul_(mu).add_(g)
        u = g + mu * buf
        x = u / (u.square().sum().sqrt() + MUON["eps"])
        tall = x.shape[0] > x.shape[1]
        if tall:
            x = x.T
        for _ in range(MUON["steps"]):
            A = x @ x.T
            x = a * x + (b * A + c * (A @ A)) @ x
        if tall:
            x = x.T
        p.mul_(1.0 - lr * wd).sub_(x * (lr * MUON["rms"] * math.sqrt(max(p.shape))))
        if s["case"]["shadow"]:
            s["w"][i].copy_(p)
    return _muon_outputs(s)


def _muon_own(s):
    from transformer_fwd_bwd_gb300 import xt
    if "ws" not in s:
        s["ws"] = xt.muon_workspace([tuple(p.shape) for p in s["p"]])
    cfg = xt.muon_config(MUON["lr"], MUON["momentum"], MUON["weight_decay"], rms=MUON["rms"], eps=MUON["eps"],
                         steps=MUON["steps"], grad_scale=GRAD_SCALE)
    xt.xt_muon_step(cfg, s["p"], s["g"], s["buf"], shadows=s.get("w"), ws=s["ws"])
    return _muon_outputs(s)


# ---------------------------------------------------------------------------------- exact

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "logprobs":
        return _logprobs_exact(case, s)
    if case["op"] == "embed":
        dE = s["dE"].double() if case["acc"] else torch.zeros(case["V"], case["d"], dtype=F64, device="cuda")
        dE.index_add_(0, s["ids"].long(), s["dh"].double(), alpha=case["scale"])
        return {"h": s["E"].double()[s["ids"].long()] * case["scale"], "dE": dE}
    if case["op"] == "gated":
        return _gated_exact(case, s)
    return _muon_exact(case, s)


def _logprobs_exact(case, s):
    """A few rows at a time, from the definition of the distribution."""
    R, V, k = case["R"], case["V"], case["top"]
    rows = {name: [] for name in ("logp", "entropy", "top_logp", "top_ids", "dlogits")}
    for r in range(0, R, 256):
        lp = torch.log_softmax(s["logits"][r:r + 256].double() * case["scale"], 1)
        n = lp.shape[0]
        tok = s["tokens"][r:r + n].long()
        p = lp.exp()
        mass = torch.special.entr(p)  # -p log p, 0 at p = 0
        H = mass.sum(1)
        rows["logp"].append(lp[torch.arange(n), tok])
        rows["entropy"].append(H)
        if k:
            ids = torch.sort(s["logits"][r:r + n].double(), dim=1, descending=True, stable=True).indices[:, :k]
            rows["top_ids"].append(ids.to(torch.int32))
            rows["top_logp"].append(lp.gather(1, ids))
        if case["train"]:
            dl, dh = s["d_logp"][r:r + n].double(), s["d_entropy"][r:r + n].double()
            d = (mass - p * H[:, None]) * dh[:, None] - p * dl[:, None]
            d[torch.arange(n), tok] += dl
            rows["dlogits"].append(d * case["scale"])
    return {name: torch.cat(parts) for name, parts in rows.items() if parts}


def _gated_exact(case, s):
    F = case["F"]
    x, wg, wu, wd = (t.double() for t in (s["x"], s["w_up"][:, :F], s["w_up"][:, F:], s["w_down"]))
    g, u = x @ wg, x @ wu
    if case["act"] == "silu":
        q = 1.0 / (1.0 + torch.exp(-g))
        a, slope = g * q, q + g * q * (1.0 - q)
    else:
        q = torch.special.ndtr(g)
        a, slope = g * q, q + g * torch.exp(-g * g / 2.0) * (2.0 * math.pi) ** -0.5
    out = {"y": (a * u) @ wd}
    if case["train"]:
        dy = s["dy"].double()
        dh = dy @ wd.T
        dg, du = dh * u * slope, dh * a
        out["dx"] = dg @ wg.T + du @ wu.T
        out["dw_up"] = torch.cat((x.T @ dg, x.T @ du), 1)
        out["dw_down"] = (a * u).T @ dy
    return out


def _muon_exact(case, s):
    """The polynomial acts on the singular values alone, as products of the matrix itself."""
    a, b, c = COEFFICIENTS
    out = {name: torch.zeros_like(s["flat"]["p"], dtype=F64) for name in ("p", "buf")}
    P, M = _matrices(case, out["p"]), _matrices(case, out["buf"])
    for i, (p, g, buf) in enumerate(zip(s["p"], s["g"], s["buf"])):
        G = g.double() * GRAD_SCALE
        M[i].copy_(MUON["momentum"] * buf.double() + G)
        u = G + MUON["momentum"] * M[i]
        x = u / (torch.linalg.matrix_norm(u) + MUON["eps"])
        left = x.shape[0] <= x.shape[1]
        eye = torch.eye(min(x.shape), dtype=F64, device="cuda")
        for _ in range(MUON["steps"]):
            S = x @ x.mT if left else x.mT @ x
            poly = a * eye + S @ (b * eye + c * S)
            x = poly @ x if left else x @ poly
        P[i].copy_(p.double() * (1.0 - MUON["lr"] * MUON["weight_decay"]) -
                   MUON["lr"] * MUON["rms"] * max(p.shape) ** 0.5 * x)
    if case["shadow"]:
        out["w"] = out["p"]
    return out
