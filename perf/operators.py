"""Measured cases of the operators that feed the optimizer step.

What a training loop does around the Muon + AdamW step, on one GPU:

  norm      the global 2-norm of a list of gradients
  clip      that norm, and the gradients scaled to a bound on it (from float32
            accumulation buffers into gradients of the weights' type, or within one type)
  lookup    embedding rows of a batch of tokens, times a factor
  rowgrad   the embedding's dense gradient from the rows' gradients: the sum over
            each token's positions
  maxlogit  the largest attention logit magnitude of each query head, which QK-Clip reads

``run`` computes them in plain torch where ``own`` is false, and calls the
package where it is true. Shapes are those of the parameter sets this
repository's benchmark runs (Llama-1B-, Llama-3-8B- and GPT-2-small-shaped, and
the float32 128 x 256 set) or generic ones.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6   # added to the norm before the division


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the smallest set of the benchmark: one float32 matrix and one vector, where latency is all
        {"name": "norm_f32_128x256", "op": "norm", "tensors": "128x256,256", "types": "f32"},
        # every gradient of the Llama-1B-shaped set (24 layers, 195 tensors, 1.3e9 elements)
        {"name": "norm_llama_1b", "op": "norm", "tensors": llama_1b(24, 2), "types": "bf16"},
        # four layers and the embedding of the same model: float32 accumulation buffers
        # into the bfloat16 gradients that the step takes
        {"name": "clip_llama_1b_stage", "op": "clip", "tensors": llama_1b(4, 1), "types": "f32", "out": "bf16",
         "max_norm": 1.0},
        # a small model of odd sizes whose float32 norms and bfloat16 weights share a list;
        # buffers start at odd elements of a flat allocation
        {"name": "clip_ragged", "op": "clip", "tensors": ragged(40, 7, 300_000), "types": "mixed", "out": "same",
         "max_norm": 0.5, "shift": 1},
        # one sequence of the GPT-2-small-shaped model
        {"name": "lookup_gpt2", "op": "lookup", "vocab": 50304, "dim": 768, "tokens": 1024, "type": "bf16", "scale": 1.0},
        # two sequences of 8192 in the Llama-3-8B-shaped model, scaled by sqrt(dim), 32-bit tokens
        {"name": "lookup_8b_scaled", "op": "lookup", "vocab": 128256, "dim": 4096, "tokens": 16384, "type": "bf16",
         "scale": 64.0, "index": 32},
        # eight sequences of 1024, GPT-2-small-shaped
        {"name": "rowgrad_gpt2", "op": "rowgrad", "vocab": 50304, "dim": 768, "tokens": 8192, "type": "bf16",
         "out": "bf16", "scale": 1.0, "padding": 0.0},
        # one sequence of 8192, Llama-3-8B-shaped: most of the gradient is rows that no token touched
        {"name": "rowgrad_8b", "op": "rowgrad", "vocab": 128256, "dim": 4096, "tokens": 8192, "type": "bf16",
         "out": "bf16", "scale": 1.0, "padding": 0.0},
        # a padded batch of 32768 tokens, Llama-1B-shaped, into float32
        {"name": "rowgrad_llama_1b_f32", "op": "rowgrad", "vocab": 32768, "dim": 2048, "tokens": 32768, "type": "bf16",
         "out": "f32", "scale": 0.5, "padding": 0.15},
        # one float32 sequence of the GPT-2-small-shaped model
        {"name": "maxlogit_gpt2_f32", "op": "maxlogit", "batch": 1, "seq": 1024, "heads": 12, "kv": 12, "dim": 64,
         "type": "f32", "causal": True},
        # one sequence of 8192 of the Llama-3-8B-shaped model: 32 query heads on 8 key heads
        {"name": "maxlogit_8b", "op": "maxlogit", "batch": 1, "seq": 8192, "heads": 32, "kv": 8, "dim": 128,
         "type": "bf16", "causal": True},
        # 23 documents of ragged lengths packed into 16384 tokens, 16 heads of 128
        {"name": "maxlogit_packed", "op": "maxlogit", "batch": 1, "seq": 16384, "heads": 16, "kv": 16, "dim": 128,
         "type": "bf16", "causal": True, "docs": 23, "split": 5},
    ]


def llama_1b(layers, heads_and_tails):
    """Shapes of the Llama-1B-shaped set: `layers` layers, and 1 or 2 of embedding and unembedding."""
    per = ["2048x2048"] * 4 + ["8192x2048", "2048x8192"]
    return ",".join(per * layers + ["2048"] * (2 * layers + 1) + ["32768x2048"] * heads_and_tails)


def ragged(count, seed, largest):
    """`count` sizes between 1 and `largest`, spread over their logarithm."""
    r = np.random.RandomState(seed)
    return ",".join(str(max(1, int(round(math.exp(r.uniform(0, math.log(largest))))))) for _ in range(count))


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "clip", "lookup", "rowgrad", "maxlogit"])
    if op in ("norm", "clip"):
        case = {"op": op, "tensors": ragged(rng.randint(1, 60 if op == "clip" else 300), rng.randint(0, 10 ** 6),
                                            _log(rng, 2, 30_000_000)),
                "types": rng.choice(["f32", "bf16", "mixed"]), "shift": rng.choice([0, 0, 1, 3])}
        if op == "clip":
            case.update(out=rng.choice(["same", "bf16", "f32"]), max_norm=rng.choice([0.01, 0.5, 100.0]))
        return case
    if op in ("lookup", "rowgrad"):
        dim = rng.choice([64, 100, 256, 513, 768, 1000, 1280, 2048, 2050, 4096])
        vocab = min(_log(rng, 100, 130_000), 128256 * 4096 // dim)
        case = {"op": op, "vocab": vocab, "dim": dim, "tokens": _log(rng, 1, 32768) if dim <= 2048 else _log(rng, 1, 16384),
                "type": rng.choice(["bf16", "bf16", "f32"]), "scale": rng.choice([1.0, 0.5, 22.6]), "index": rng.choice([32, 64])}
        if op == "rowgrad":
            case.update(out=rng.choice(["bf16", "f32"]) if dim * vocab < 10 ** 8 else "bf16", padding=rng.choice([0.0, 0.0, 0.3]))
        return case
    kind = rng.choice(["bf16", "bf16", "f32"])
    dim = rng.choice([16, 40, 64, 80, 96, 128, 192, 256])
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 2, 3, 4, 8])
    docs = rng.choice([0, 0, rng.randint(2, 40)])
    batch = 1 if docs else rng.randint(1, 8)
    most = 32 * 128 * 8192 ** 2 / (16 if kind == "f32" else 1)
    seq = min(_log(rng, 1, 16384), int(math.sqrt(most / (heads * dim * batch))))
    seq = max(seq, docs)
    case = {"op": op, "batch": batch, "seq": seq, "heads": heads, "kv": kv, "dim": dim, "type": kind,
            "causal": rng.random() < 0.75}
    if docs:
        case.update(docs=docs, split=rng.randint(0, 10 ** 6))
    elif rng.random() < 0.5:
        case.update(padded=True, split=rng.randint(0, 10 ** 6))   # batch rows of unlike lengths
    return case


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

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


def _shapes(case):
    return [tuple(int(x) for x in t.split("x")) for t in case["tensors"].split(",")]


def _list_types(case, n):
    if case["types"] == "mixed":
        return [torch.float32 if i % 3 == 0 else torch.bfloat16 for i in range(n)]
    return [TYPES[case["types"]]] * n


def _views(shapes, types, shift):
    """Tensors of one allocation each, or (shift > 0) views that start `shift` elements into one."""
    out = []
    for s, t in zip(shapes, types):
        n = math.prod(s)
        out.append(torch.empty(n + shift, dtype=t, device=DEV)[shift:].view(s))
    return out


def _zipf(count, vocab, gen):
    """Tokens whose frequency falls as 1 / rank, the ranks spread over the ids."""
    u = torch.rand(count, generator=gen, device=DEV, dtype=torch.float64)
    rank = (torch.exp(u * math.log(vocab + 1)) - 1).long().clamp_(0, vocab - 1)
    step = 7919
    while math.gcd(step, vocab) != 1:
        step += 2
    return (rank * step + 12345) % vocab


def _lengths(case):
    """Lengths of the sequences: of packed documents, or of the rows of a padded batch."""
    if case.get("docs"):
        r = np.random.RandomState(case["split"])
        cuts = np.sort(r.choice(np.arange(1, case["seq"]), case["docs"] - 1, replace=False)) if case["docs"] > 1 else []
        return np.diff(np.concatenate([[0], cuts, [case["seq"]]]).astype(np.int64)).tolist()
    if case.get("padded"):
        r = np.random.RandomState(case["split"])
        return [int(x) for x in r.randint(0, case["seq"] + 1, case["batch"])]
    return [case["seq"]] * case["batch"]


def prepare(case, seed):
    gen = _gen(seed)
    st = {"case": case}
    op = case["op"]
    if op in ("norm", "clip"):
        shapes = _shapes(case)
        types = _list_types(case, len(shapes))
        st["grads"] = _views(shapes, types, case.get("shift", 0))
        for t in st["grads"]:
            t.copy_(_normal(tuple(t.shape), gen, 1e-3, t.dtype))
        if op == "clip":
            outs = types if case["out"] == "same" else [TYPES[case["out"]]] * len(shapes)
            st["outs"] = _views(shapes, outs, case.get("shift", 0))
            for t in st["outs"]:
                t.zero_()
    elif op in ("lookup", "rowgrad"):
        tok = _zipf(case["tokens"], case["vocab"], gen)
        st["padding"] = None
        if case.get("padding"):   # the last part of the batch is padding
            st["padding"] = 3 % case["vocab"]
            tok[int(case["tokens"] * (1 - case["padding"])):] = st["padding"]
        st["tokens"] = tok.int() if case.get("index") == 32 else tok
        if op == "lookup":
            st["weight"] = _normal((case["vocab"], case["dim"]), gen, 0.02, TYPES[case["type"]])
        else:
            st["rows"] = _normal((case["tokens"], case["dim"]), gen, 1e-3, TYPES[case["type"]])
    else:
        b, s, hq, hk, d = case["batch"], case["seq"], case["heads"], case["kv"], case["dim"]
        # queries and keys are column ranges of one projection's output, as a model has them
        qkv = _normal((b, s, hq + 2 * hk, d), gen, 1.0, TYPES[case["type"]])
        gain = torch.rand(hq + 2 * hk, 1, generator=gen, device=DEV) * 4 + 0.5   # heads of unlike sizes
        qkv.mul_(gain.to(qkv.dtype))
        st["q"], st["k"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hk]
        st["lengths"] = st["cu"] = None
        lens = _lengths(case)
        st["host_lengths"] = lens
        if case.get("docs"):
            st["q"], st["k"] = st["q"][0], st["k"][0]
            st["cu"] = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=DEV)
        elif case.get("padded"):
            st["lengths"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    import newton_schulz_orthogonalized_amd as nso
    case = st["case"]
    op = case["op"]
    if op == "norm":
        return nso.grad_norm(st["grads"])
    if op == "clip":
        norm = nso.clip_grads(st["grads"], case["max_norm"], outs=st["outs"])
        return {"norm": norm, "grads": st["outs"]}
    if op == "lookup":
        return nso.embedding(st["tokens"], st["weight"], scale=case["scale"])
    if op == "rowgrad":
        return nso.embedding_grad(st["tokens"], st["rows"], case["vocab"], scale=case["scale"],
                                  padding_idx=st["padding"], dtype=TYPES[case["out"]])
    return nso.qk_max_logits(st["q"], st["k"], causal=case["causal"], lengths=st["lengths"], cu_seqlens=st["cu"])


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op in ("norm", "clip"):
        # squares in 32 bits, their long sum in 64
        norm = torch.stack([g.float().square().sum(dtype=torch.float64) for g in st["grads"]]).sum().sqrt()
        if op == "norm":
            return norm.float()
        coef = (case["max_norm"] / (norm + EPS)).clamp(max=1.0).float()
        for g, o in zip(st["grads"], st["outs"]):
            o.copy_(g.float() * coef)
        return {"norm": norm.float(), "grads": st["outs"]}
    if op == "lookup":
        w = st["weight"]
        return (w[st["tokens"].long()].float() * case["scale"]).to(w.dtype)
    if op == "rowgrad":
        tok = st["tokens"].long()
        rows = st["rows"].float()
        if st["padding"] is not None:
            rows = rows * (tok != st["padding"]).float()[:, None]
        dense = torch.zeros(case["vocab"], case["dim"], device=DEV)
        dense.index_add_(0, tok, rows)
        return (dense * case["scale"]).to(TYPES[case["out"]])
    q, k, lens = st["q"], st["k"], st["host_lengths"]
    hq, hk, d = case["heads"], case["kv"], case["dim"]
    best = torch.zeros(hq, device=DEV)
    start = 0
    for b, n in enumerate(lens):
        if case.get("docs"):
            qs, ks = q[start:start + n], k[start:start + n]
            start += n
        else:
            qs, ks = q[b, :n], k[b, :n]
        if n == 0:
            continue
        for h in range(hq):
            logits = (qs[:, h].float() @ ks[:, h * hk // hq].float().t()).abs()
            if case["causal"]:
                i = torch.arange(n, device=DEV)
                logits = logits.masked_fill(i[None, :] > i[:, None], 0.0)
            best[h] = torch.maximum(best[h], logits.max())
    return best / math.sqrt(d)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def _size(name):
    return 2 if name == "bf16" else 4


def _distinct(count, vocab):
    """Expected number of distinct tokens among `count` of the distribution above."""
    r = np.arange(vocab, dtype=np.float64)
    p = np.log((r + 2) / (r + 1)) / math.log(vocab + 1)
    return float(np.sum(-np.expm1(count * np.log1p(-p))))


def work(case):
    op = case["op"]
    if op in ("norm", "clip"):
        n = [math.prod(s) for s in _shapes(case)]
        types = _list_types(case, len(n))
        ins = [2 if t is torch.bfloat16 else 4 for t in types]
        byt = sum(a * b for a, b in zip(n, ins))
        if op == "norm":
            return {"bytes": byt + 4, "flops": 2 * sum(n)}
        outs = ins if case["out"] == "same" else [_size(case["out"])] * len(n)
        return {"bytes": byt + 4 + sum(a * b for a, b in zip(n, outs)), "flops": 3 * sum(n)}
    if op in ("lookup", "rowgrad"):
        t, v, d = case["tokens"], case["vocab"], case["dim"]
        idx = t * (4 if case.get("index") == 32 else 8)
        if op == "lookup":
            return {"bytes": idx + (t + _distinct(t, v)) * d * _size(case["type"]), "flops": t * d}
        return {"bytes": idx + t * d * _size(case["type"]) + v * d * _size(case["out"]), "flops": t * d}
    hq, hk, d = case["heads"], case["kv"], case["dim"]
    lens = _lengths(case)
    pairs = sum(n * (n + 1) / 2 if case["causal"] else n * n for n in lens)
    return {"bytes": sum(lens) * (hq + hk) * d * _size(case["type"]) + 4 * hq, "flops": 2.0 * pairs * hq * d}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "clip"):
        total = torch.zeros((), dtype=torch.float64, device=DEV)
        for g in st["grads"]:
            v = g.reshape(-1)
            for i in range(0, v.numel(), 1 << 25):
                x = v[i:i + (1 << 25)].double()
                total += torch.dot(x, x)
        norm = torch.sqrt(total)
        if op == "norm":
            return norm
        factor = min(1.0, case["max_norm"] / (float(norm) + EPS))
        return {"norm": norm, "grads": [g.double() * factor for g in st["grads"]]}
    if op == "lookup":
        return torch.index_select(st["weight"], 0, st["tokens"].long()).double() * case["scale"]
    if op == "rowgrad":
        # runs of equal tokens in sorted order; each run's sum goes to its row
        tok, order = torch.sort(st["tokens"].long(), stable=True)
        ids, counts = torch.unique_consecutive(tok, return_counts=True)
        run_of = torch.repeat_interleave(torch.arange(ids.numel(), device=DEV), counts)
        sums = torch.zeros(ids.numel(), case["dim"], dtype=torch.float64, device=DEV)
        sums.index_add_(0, run_of, st["rows"][order].double())
        out = torch.zeros(case["vocab"], case["dim"], dtype=torch.float64, device=DEV)
        out[ids] = sums * case["scale"]
        if st["padding"] is not None:
            out[st["padding"]] = 0
        return out
    q, k = st["q"], st["k"]
    hq, hk, d = case["heads"], case["kv"], case["dim"]
    if case.get("docs"):
        edges = np.concatenate([[0], np.cumsum(st["host_lengths"])]).tolist()
        seqs = [(q[a:b], k[a:b]) for a, b in zip(edges[:-1], edges[1:])]
    else:
        seqs = [(q[b, :n], k[b, :n]) for b, n in enumerate(st["host_lengths"])]
    best = [0.0] * hq
    group = hq // hk
    for qs, ks in seqs:
        n = qs.shape[0]
        for h in range(hq):
            kh = ks[:, h // group].double().t().contiguous()
            for i in range(0, n, 2048):   # rows i .. i + 2047 see the keys up to their own
                rows = qs[i:i + 2048, h].double()
                last = min(n, i + rows.shape[0]) if case["causal"] else n
                s = rows @ kh[:, :last]
                if case["causal"]:
                    s = torch.tril(s, diagonal=i)
                best[h] = max(best[h], float(s.abs().max()))
    return torch.tensor([b / math.sqrt(d) for b in best], dtype=torch.float64)
