"""Measured cases of the parts of a transformer block between its products.

What a training loop, or a program that generates tokens, computes around the
weights that the Muon step updates, on one GPU:

  rotary    queries and keys turned by their positions (halves or interleaved
            pairs, all of the head or its first part, frequencies scaled for
            long contexts), and their gradients
  resnorm   r' = a r + gate * N(y) and N(r'): the norm after a block, its gate,
            the residual sum and the norm before the next block, and their
            gradients
  mlp       act(x Wg^T) * (x Wu^T): the projections, activation and product of a
            gated feed-forward block, and the gradients of x and both weights

``run`` computes them in plain torch where ``own`` is false, and calls the
package where it is true. Shapes are those of the parameter sets this
repository's benchmark runs (Llama-1B-, Llama-3-8B- and GPT-2-small-shaped) or
generic ones.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # 64 sequences that each generate one token far into a long context: interleaved pairs of
        # half of the head, positions of their own; latency is all
        {"name": "rotary_tokens", "op": "rotary", "batch": 64, "seq": 1, "heads": 32, "kv": 8, "dim": 128, "part": 64,
         "layout": "pairs", "type": "bf16", "scaled": "parts", "far": 100_000, "train": False},
        # one sequence of 8192 of the Llama-3-8B-shaped model, both ways
        {"name": "rotary_8b", "op": "rotary", "batch": 1, "seq": 8192, "heads": 32, "kv": 8, "dim": 128, "part": 128,
         "layout": "halves", "type": "bf16", "scaled": "no", "far": 0, "train": True},
        # a float32 batch with heads of an odd width, evenly scaled positions, both ways
        {"name": "rotary_ragged_f32", "op": "rotary", "batch": 3, "seq": 1001, "heads": 10, "kv": 5, "dim": 90, "part": 70,
         "layout": "halves", "type": "f32", "scaled": "evenly", "far": 5000, "train": True},
        # 64 sequences that each generate one token, Llama-3-8B-shaped; latency is all
        {"name": "resnorm_tokens", "op": "resnorm", "rows": 64, "groups": 0, "dim": 4096, "res": "bf16", "type": "bf16",
         "post": False, "a": 1.0, "train": False},
        # one sequence of 8192, Llama-3-8B-shaped, norms on both sides of the block
        {"name": "resnorm_8b", "op": "resnorm", "rows": 8192, "groups": 0, "dim": 4096, "res": "bf16", "type": "bf16",
         "post": True, "a": 1.0, "train": False},
        # 8 sequences of 2048, Llama-1B-shaped, a gate for each sequence and channel, a residual stream in
        # float32 with a scale, both ways
        {"name": "resnorm_llama_1b_train", "op": "resnorm", "rows": 16384, "groups": 8, "dim": 2048, "res": "f32", "type": "bf16",
         "post": True, "a": 0.8, "train": True},
        # odd rows in float32, one gate, both ways
        {"name": "resnorm_ragged_f32", "op": "resnorm", "rows": 777, "groups": 1, "dim": 1003, "res": "f32", "type": "f32",
         "post": True, "a": 0.5, "train": True},
        # one token through the Llama-3-8B-shaped block
        {"name": "mlp_token_8b", "op": "mlp", "tokens": 1, "dim": 4096, "hidden": 14336, "type": "bf16", "act": "silu", "train": False},
        # 8 sequences of 1024 through a Llama-1B-shaped block
        {"name": "mlp_llama_1b", "op": "mlp", "tokens": 8192, "dim": 2048, "hidden": 8192, "type": "bf16", "act": "silu", "train": False},
        # one sequence of 8192, Llama-3-8B-shaped, both ways
        {"name": "mlp_8b_train", "op": "mlp", "tokens": 8192, "dim": 4096, "hidden": 14336, "type": "bf16", "act": "silu", "train": True},
        # one sequence of 1000 through a block of the GPT-2-small-shaped width, both ways
        {"name": "mlp_gpt2_train", "op": "mlp", "tokens": 1000, "dim": 768, "hidden": 2048, "type": "bf16", "act": "gelu", "train": True},
        # odd sizes in float32, both ways
        {"name": "mlp_ragged_f32", "op": "mlp", "tokens": 1201, "dim": 515, "hidden": 1365, "type": "f32", "act": "gelu_tanh", "train": True},
    ]


def _log(rng, lo, hi):
    hi = max(lo, hi)
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "resnorm", "mlp", "mlp"])
    if op == "rotary":
        dim = rng.choice([32, 64, 80, 90, 96, 128, 128, 192, 256])
        part = dim if rng.random() < 0.5 else 2 * rng.randint(1, dim // 2)
        kv = rng.choice([1, 2, 4, 5, 8])
        heads = kv * rng.choice([1, 2, 3, 4, 8])
        batch = _log(rng, 1, 64)
        seq = _log(rng, 1, max(1, 8192 * 40 * 128 // (batch * (heads + kv) * dim)))
        return {"op": op, "batch": batch, "seq": seq, "heads": heads, "kv": kv, "dim": dim, "part": part,
                "layout": rng.choice(["halves", "pairs"]), "type": rng.choice(["bf16", "bf16", "f32"]),
                "scaled": rng.choice(["no", "evenly", "parts"]), "far": rng.choice([0, 0, _log(rng, 10, 1_000_000)]),
                "train": rng.random() < 0.6}
    if op == "resnorm":
        dim = rng.choice([64, 100, 513, 768, 1000, 1280, 2048, 2050, 4096, 5120, 8192, 9001])
        groups = rng.choice([0, 0, 1, rng.randint(2, 16)])
        rows = _log(rng, 1, max(1, 16384 * 2048 // dim))
        rows = max(1, rows // groups) * groups if groups else rows
        kind = rng.choice(["bf16", "bf16", "f32"])
        return {"op": op, "rows": rows, "groups": groups, "dim": dim, "res": rng.choice([kind, "f32"]), "type": kind,
                "post": rng.random() < 0.6, "a": rng.choice([1.0, 0.7]), "train": rng.random() < 0.6}
    kind = rng.choice(["bf16", "bf16", "bf16", "f32"])
    train = rng.random() < 0.6
    dim = rng.choice([64, 100, 256, 513, 768, 1000, 1600, 2048, 4096])
    hidden = rng.choice([dim * 2, dim * 3 + 1, dim * 7 // 2, dim * 8 // 3, _log(rng, 64, 14336)])
    hidden = min(hidden, 14336)
    most = 8192 * 4096 * 14336 / (16 if kind == "f32" else 1)
    tokens = _log(rng, 1, min(16384, int(most / (dim * hidden))))
    return {"op": op, "tokens": tokens, "dim": dim, "hidden": hidden, "type": kind,
            "act": rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu"]), "train": train}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

BASE, FACTOR, CONTEXT, LOW, HIGH = 500000.0, 8.0, 8192, 1.0, 4.0
EPS = 1e-6


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(shape, gen, std, dtype):
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat = out.view(-1)
    step = 1 << 26
    for i in range(0, flat.numel(), step):
        part = flat[i:i + step]
        part.copy_(torch.randn(part.numel(), generator=gen, device=DEV).mul_(std))
    return out


def _gain(case):
    """What the turned part is multiplied by in a scaled context."""
    return 0.1 * math.log(FACTOR) + 1.0 if case["scaled"] == "parts" else 1.0


def prepare(case, seed):
    gen = _gen(seed)
    st = {"case": case}
    op, train = case["op"], case["train"]
    t = TYPES[case["type"]]
    if op == "rotary":
        b, s, hq, hk, d = case["batch"], case["seq"], case["heads"], case["kv"], case["dim"]
        # queries and keys are column ranges of one projection's output, as a model has them
        qkv = _normal((b, s, hq + 2 * hk, d), gen, 1.0, t)
        st["q"], st["k"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hk]
        st["pos"] = None
        if case["far"]:   # each sequence somewhere in a long context
            start = torch.randint(0, case["far"], (b, 1), generator=gen, device=DEV)
            st["pos"] = start + torch.arange(s, device=DEV)[None]
        if train:
            st["q"], st["k"] = st["q"].requires_grad_(), st["k"].requires_grad_()
            st["dq"] = _normal((b, s, hq, d), gen, 1e-2, t)
            st["dk"] = _normal((b, s, hk, d), gen, 1e-2, t)
        if own:
            import newton_schulz_orthogonalized_amd as nso
            kw = {"no": {}, "evenly": {"factor": FACTOR},
                  "parts": {"factor": FACTOR, "original_length": CONTEXT, "low": LOW, "high": HIGH}}[case["scaled"]]
            st["freqs"] = nso.rotary_frequencies(case["part"], base=BASE, device=DEV, **kw)
    elif op == "resnorm":
        n, d, r = case["rows"], case["dim"], TYPES[case["res"]]
        st["r"], st["y"] = _normal((n, d), gen, 3.0, r), _normal((n, d), gen, 0.3, t)
        st["w_pre"] = (_normal((d,), gen, 0.1, torch.float32) + 1).to(t)
        st["w_post"] = (_normal((d,), gen, 0.1, torch.float32) + 0.5).to(t) if case["post"] else None
        st["gate"] = _normal((case["groups"], d), gen, 0.5, t) if case["groups"] else None
        if train:
            for name in ("r", "y", "w_pre", "w_post", "gate"):
                if st[name] is not None:
                    st[name].requires_grad_()
            st["dr"], st["dn"] = _normal((n, d), gen, 1e-3, r), _normal((n, d), gen, 1e-3, t)
    else:
        n, d, f = case["tokens"], case["dim"], case["hidden"]
        st["x"] = _normal((n, d), gen, 1.0, t)
        st["wg"], st["wu"] = _normal((f, d), gen, d ** -0.5, t), _normal((f, d), gen, d ** -0.5, t)
        if train:
            for name in ("x", "wg", "wu"):
                st[name].requires_grad_()
            st["dh"] = _normal((n, f), gen, 1e-2, t)
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    import newton_schulz_orthogonalized_amd as nso
    case = st["case"]
    op, train = case["op"], case["train"]
    if op == "rotary":
        q, k = nso.rotary(st["q"], st["k"], freqs=st["freqs"], positions=st["pos"], interleaved=case["layout"] == "pairs",
                          scale=_gain(case))
        if not train:
            return {"q": q, "k": k}
        dq, dk = torch.autograd.grad((q, k), (st["q"], st["k"]), (st["dq"], st["dk"]))
        return {"q": q.detach(), "k": k.detach(), "dq": dq, "dk": dk}
    if op == "resnorm":
        r, n = nso.residual_norm(st["r"], st["y"], residual_scale=case["a"], gate=st["gate"], post_weight=st["w_post"],
                                 pre_weight=st["w_pre"], eps=EPS)
        if not train:
            return {"r": r, "n": n}
        names = [x for x in ("r", "y", "w_pre", "w_post", "gate") if st[x] is not None]
        grads = torch.autograd.grad((r, n), [st[x] for x in names], (st["dr"], st["dn"]))
        return {"r": r.detach(), "n": n.detach(), **{"d" + x: g for x, g in zip(names, grads)}}
    h = nso.gated_mlp(st["x"], st["wg"], st["wu"], activation=case["act"])
    if not train:
        return {"h": h}
    dx, dwg, dwu = torch.autograd.grad(h, (st["x"], st["wg"], st["wu"]), st["dh"])
    return {"h": h.detach(), "dx": dx, "dwg": dwg, "dwu": dwu}


def _angles(st):
    """cos and sin [batch or 1, seq, 1, part / 2], the angles in 64 bits."""
    case = st["case"]
    i = torch.arange(0, case["part"], 2, device=DEV, dtype=torch.float64)
    f = BASE ** (-i / case["part"])
    if case["scaled"] == "evenly":
        f = f / FACTOR
    elif case["scaled"] == "parts":
        keep = ((CONTEXT * f / (2 * math.pi) - LOW) / (HIGH - LOW)).clamp(0, 1)
        f = f * keep + f / FACTOR * (1 - keep)
    pos = st["pos"] if st["pos"] is not None else torch.arange(case["seq"], device=DEV)[None]
    a = pos.double()[:, :, None, None] * f
    gain = _gain(case)
    return (a.cos() * gain).float(), (a.sin() * gain).float()


def _turn(x, cos, sin, case):
    part = case["part"]
    y = x.float()
    if case["layout"] == "pairs":
        a, b = y[..., 0:part:2], y[..., 1:part:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = y[..., :part // 2], y[..., part // 2:part]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, y[..., part:]), -1).to(x.dtype)


def _act(g, kind):
    """(activation, its derivative) in 32 bits."""
    if kind == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    if kind == "gelu":
        c = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * c, c + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (g + 0.044715 * g * g * g))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)
    up = (g > 0).float()
    return g * up, up


@torch.no_grad()
def _run_plain(st):
    case = st["case"]
    op, train = case["op"], case["train"]
    t = TYPES[case["type"]]
    if op == "rotary":
        cos, sin = _angles(st)
        out = {"q": _turn(st["q"], cos, sin, case), "k": _turn(st["k"], cos, sin, case)}
        if train:
            out.update(dq=_turn(st["dq"], cos, -sin, case), dk=_turn(st["dk"], cos, -sin, case))
        return out
    if op == "resnorm":
        y = st["y"].float()
        s1 = torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)
        p = y * s1 * st["w_post"].float() if case["post"] else y
        groups, d = case["groups"], case["dim"]
        gate = st["gate"].float()[:, None, :] if groups else None
        add = (p.view(groups, -1, d) * gate).view(-1, d) if groups else p
        r = st["r"].float() * case["a"] + add
        s2 = torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS)
        w = st["w_pre"].float()
        out = {"r": r.to(st["r"].dtype), "n": (r * s2 * w).to(t)}
        if train:
            dn = st["dn"].float()
            v = dn * w
            dr = st["dr"].float() + s2 * (v - r * s2.square() * (v * r).mean(-1, keepdim=True))
            u = (dr.view(groups, -1, d) * gate).view(-1, d) if groups else dr
            if case["post"]:
                v = u * st["w_post"].float()
                dy = s1 * (v - y * s1.square() * (v * y).mean(-1, keepdim=True))
            else:
                dy = u
            out.update(dr=(dr * case["a"]).to(st["r"].dtype), dy=dy.to(t), dw_pre=(dn * r * s2).sum(0).to(t))
            if case["post"]:
                out["dw_post"] = (u * y * s1).sum(0).to(t)
            if groups:
                out["dgate"] = (dr * p).view(groups, -1, d).sum(1).to(t)
        return out
    x, wg, wu = st["x"].float(), st["wg"].float(), st["wu"].float()
    g, u = x @ wg.t(), x @ wu.t()
    a, slope = _act(g, case["act"])
    out = {"h": (a * u).to(t)}
    if train:
        dh = st["dh"].float()
        dg, du = dh * u * slope, dh * a
        out.update(dx=(dg @ wg + du @ wu).to(t), dwg=(dg.t() @ x).to(t), dwu=(du.t() @ x).to(t))
    return out


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def _size(name):
    return 2 if name == "bf16" else 4


def work(case):
    e = _size(case["type"])
    ways = 2 if case["train"] else 1
    if case["op"] == "rotary":
        rows = case["batch"] * case["seq"]
        cells = rows * (case["heads"] + case["kv"])
        pos = 8 * rows if case["far"] else 0
        return {"bytes": ways * (2 * cells * case["dim"] * e + pos), "flops": ways * 3 * cells * case["part"]}
    if case["op"] == "resnorm":
        n = case["rows"] * case["dim"]
        r = _size(case["res"])
        byt = n * (2 * r + 2 * e)
        if case["train"]:   # r', y, dr', dn in; dr, dy out (r' was written by the pass before)
            byt += n * (3 * r + 3 * e)
        return {"bytes": byt, "flops": n * (26 if case["train"] else 9)}
    n, d, f = case["tokens"], case["dim"], case["hidden"]
    byt = (n * d + 2 * d * f + n * f) * e
    if case["train"]:   # x, dh and the weights in; dx and the weights' gradients out
        byt += (2 * n * d + 4 * d * f + n * f) * e
    return {"bytes": byt, "flops": (3 if case["train"] else 1) * 4.0 * n * d * f}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _leaf(x):
    return x.detach().double().requires_grad_()


def exact(case, seed):
    st = prepare(case, seed)
    op, train = case["op"], case["train"]
    if op == "rotary":
        part, dim = case["part"], case["dim"]
        f = torch.exp(torch.arange(part // 2, device=DEV, dtype=torch.float64) * (-2.0 * math.log(BASE) / part))
        if case["scaled"] == "evenly":
            f = f / FACTOR
        elif case["scaled"] == "parts":   # turns over the context: few, slowed down; many, kept; between, in parts
            turns = CONTEXT * f / (2 * math.pi)
            between = (turns - LOW) / (HIGH - LOW)
            f = torch.where(turns < LOW, f / FACTOR, torch.where(turns > HIGH, f, between * f + (1 - between) * f / FACTOR))
        pos = torch.arange(case["seq"], device=DEV).expand(case["batch"], -1) if st["pos"] is None else st["pos"]
        angle = torch.outer(pos.reshape(-1).double(), f).view(case["batch"], case["seq"], 1, part // 2)
        unit = torch.polar(torch.full_like(angle, _gain(case)), angle)

        def turn(x, z):
            x = x.detach().double()
            head = x[..., :part]
            if case["layout"] == "pairs":
                c = torch.view_as_complex(head.reshape(*head.shape[:-1], part // 2, 2).contiguous()) * z
                head = torch.view_as_real(c).reshape(*head.shape)
            else:
                c = torch.complex(head[..., :part // 2].contiguous(), head[..., part // 2:].contiguous()) * z
                head = torch.cat((c.real, c.imag), -1)
            return head if part == dim else torch.cat((head, x[..., part:]), -1)

        out = {"q": turn(st["q"], unit), "k": turn(st["k"], unit)}
        if train:
            out.update(dq=turn(st["dq"], unit.conj()), dk=turn(st["dk"], unit.conj()))
        return out
    if op == "resnorm":
        leaves = {x: _leaf(st[x]) for x in ("r", "y", "w_pre", "w_post", "gate") if st[x] is not None}

        def norm(v, w):
            return v / (v.pow(2).sum(-1, keepdim=True) / v.shape[-1] + EPS).sqrt() * w

        with torch.enable_grad():
            p = norm(leaves["y"], leaves["w_post"]) if case["post"] else leaves["y"]
            if case["groups"]:
                p = p * leaves["gate"].repeat_interleave(case["rows"] // case["groups"], 0)
            r = case["a"] * leaves["r"] + p
            n = norm(r, leaves["w_pre"])
        out = {"r": r.detach(), "n": n.detach()}
        if train:
            grads = torch.autograd.grad((r, n), list(leaves.values()), (st["dr"].double(), st["dn"].double()))
            out.update({"d" + x: g for x, g in zip(leaves, grads)})
        return out
    x, wg, wu = _leaf(st["x"]), _leaf(st["wg"]), _leaf(st["wu"])
    with torch.enable_grad():
        g = torch.nn.functional.linear(x, wg)
        if case["act"] == "silu":
            a = g * torch.sigmoid(g)
        elif case["act"] == "gelu":
            a = g * torch.special.ndtr(g)
        elif case["act"] == "gelu_tanh":
            a = g * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))
        else:
            a = torch.relu(g)
        h = a * torch.nn.functional.linear(x, wu)
    out = {"h": h.detach()}
    if train:
        out.update(zip(("dx", "dwg", "dwu"), torch.autograd.grad(h, (x, wg, wu), st["dh"].double())))
    return out
