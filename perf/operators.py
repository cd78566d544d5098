"""Workloads of the operators on logits and gradients, and their plain forms.

Three kinds of case:

  sample   one token a row of logits (temperature, top-k, top-p, min-p) from given random numbers
  logprob  the log-probability of given tokens, and its gradient with respect to the logits
  clip     the global norm of many gradient tensors, and the clipped gradients

`run` makes the library's calls where `own` is true, and computes the same results with elementary torch operations
otherwise.  `exact` computes them from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

LOG2E = 1.4426950408889634
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"fp32": 4, "fp16": 2, "bf16": 2}


# ---- cases

def listed():
    return [
        # one answer of an interactive session: a single row, the usual filters; latency is all that counts
        dict(name="sample_one", kind="sample", rows=1, vocab=32768, dtype="fp32", temperature=0.8, top_k=50, top_p=0.95,
             min_p=0.0, per_row=False, masked=0.0),
        # a small batch of a server: every request has its own settings (some greedy), an odd vocabulary
        dict(name="sample_server", kind="sample", rows=48, vocab=50001, dtype="bf16", temperature=1.0, top_k=0, top_p=1.0,
             min_p=0.0, per_row=True, masked=0.0),
        # constrained decoding: most of the vocabulary is masked with -inf, a nucleus of the rest
        dict(name="sample_nucleus", kind="sample", rows=256, vocab=131072, dtype="bf16", temperature=1.0, top_k=0, top_p=0.9,
             min_p=0.0, per_row=False, masked=0.6),
        # a rollout batch: plain sampling at temperature 1 from fp32 logits
        dict(name="sample_rollout", kind="sample", rows=512, vocab=131072, dtype="fp32", temperature=1.0, top_k=0, top_p=1.0,
             min_p=0.0, per_row=False, masked=0.0),
        # scoring the candidates of one request
        dict(name="logprob_few", kind="logprob", rows=7, vocab=32768, dtype="fp16", grad=False, lse=False),
        # scoring a batch of sequences
        dict(name="logprob_score", kind="logprob", rows=4096, vocab=50001, dtype="bf16", grad=False, lse=False),
        # a training step whose weights are known beforehand: loss and gradient in one call, odd vocabulary
        dict(name="logprob_grad_odd", kind="logprob", rows=1000, vocab=50001, dtype="bf16", grad=True, lse=False),
        # the backward pass of a step that scored first (ratios of new to old probabilities), fp32 logits
        dict(name="logprob_backward", kind="logprob", rows=2048, vocab=32768, dtype="fp32", grad=True, lse=True),
        # a large training batch at a large vocabulary
        dict(name="logprob_grad_large", kind="logprob", rows=8192, vocab=131072, dtype="bf16", grad=True, lse=False),
        # a small policy's gradients: a dozen tensors, latency counts
        dict(name="clip_small", kind="clip", hidden=64, layers=1, vocab=256, dtype="fp32", out="fp32", scale=1.0, clip=True),
        # monitoring: the norm alone of a mid-size model with odd widths
        dict(name="norm_ragged", kind="clip", hidden=1001, layers=24, vocab=20011, dtype="bf16", out="bf16", scale=1.0,
             clip=False),
        # mixed precision: scaled fp16 gradients to clipped fp32 ones
        dict(name="clip_mixed", kind="clip", hidden=2048, layers=16, vocab=65536, dtype="fp16", out="fp32",
             scale=1.0 / 1024.0, clip=True),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["sample", "logprob", "clip"])
    if kind == "clip":
        hidden = _log_uniform(rng, 24, 2048)
        if _ffn(hidden) == 3072:
            hidden += 1
        dtype = rng.choice(sorted(DTYPES))
        return dict(kind=kind, hidden=hidden, layers=rng.randint(1, 16), vocab=_log_uniform(rng, 100, 65536), dtype=dtype,
                    out=rng.choice([dtype, "fp32"]), scale=rng.choice([1.0, 1.0 / 1024.0]), clip=rng.random() < 0.7)
    vocab = _log_uniform(rng, 500, 131072)
    vocab += vocab == 3072
    if kind == "sample":
        return dict(kind=kind, rows=_log_uniform(rng, 1, 512), vocab=vocab, dtype=rng.choice(sorted(DTYPES)),
                    temperature=round(rng.uniform(0.3, 1.5), 3), top_k=rng.choice([0, 0, 1, 20, 64, 500]),
                    top_p=rng.choice([1.0, 0.99, 0.9, 0.5]), min_p=rng.choice([0.0, 0.0, 0.02]),
                    per_row=rng.random() < 0.4, masked=rng.choice([0.0, 0.0, 0.5, 0.95]))
    grad = rng.random() < 0.7
    rows = _log_uniform(rng, 1, 8192)
    rows += rows == 3072
    dtype = rng.choice(sorted(DTYPES))
    if rows * vocab * BYTES[dtype] > 8192 * 131072 * 2:
        dtype = "bf16"
    return dict(kind=kind, rows=rows, vocab=vocab, dtype=dtype, grad=grad, lse=grad and rng.random() < 0.5)


def _ffn(hidden):
    return hidden * 8 // 3


def _shapes(case):
    """The gradients of a stack of layers: square and wide matrices, vectors, two tables."""
    h, f, v = case["hidden"], _ffn(case["hidden"]), case["vocab"]
    layer = [(h, h)] * 4 + [(h, f)] * 2 + [(f, h), (h,), (h,), (f,)]
    return [(v, h), (h, v)] + layer * case["layers"] + [(h,), (1,)]


def _numbers(case):
    return sum(math.prod(s) for s in _shapes(case))


# ---- inputs

def _logits(case, g):
    """Logits as a language model gives them: probabilities that fall like a power of the rank, with noise."""
    shape = (case["rows"], case["vocab"])
    x = torch.empty(shape, device="cuda").exponential_(1.0, generator=g).mul_(1.3)
    x += torch.randn(shape, device="cuda", generator=g) * 0.7
    masked = case.get("masked", 0.0)
    if masked:
        x.masked_fill_(torch.rand(shape, device="cuda", generator=g) < masked, -math.inf)
    return x.to(DTYPES[case["dtype"]])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["kind"] == "sample":
        r = case["rows"]
        s = dict(case=case, logits=_logits(case, g), u=torch.rand(r, device="cuda", generator=g))
        if case["per_row"]:
            # requests of their own kinds: greedy, top-k, nucleus, min-p, plain
            kind = torch.randint(0, 5, (r,), device="cuda", generator=g)
            t = torch.rand(r, device="cuda", generator=g) * 1.2 + 0.3
            s["temperature"] = torch.where(kind == 0, 0.0, t)
            s["top_k"] = torch.where(kind == 1, torch.randint(1, 200, (r,), device="cuda", generator=g), 0).int()
            s["top_p"] = torch.where(kind <= 2, torch.rand(r, device="cuda", generator=g) * 0.6 + 0.4, 1.0)
            s["min_p"] = torch.where(kind == 3, 0.05, 0.0)
        else:
            s.update({k: case[k] for k in ("temperature", "top_k", "top_p", "min_p")})
        return s
    if case["kind"] == "logprob":
        r, v = case["rows"], case["vocab"]
        x = _logits(case, g)
        t = torch.randint(0, v, (r,), device="cuda", generator=g)
        unused = torch.rand(r, device="cuda", generator=g) < 0.05  # padding
        s = dict(case=case, logits=x, tokens=torch.where(unused, -100, t))
        if case["grad"]:
            s["dlogp"] = torch.randn(r, device="cuda", generator=g)
        if case["lse"]:
            s["lse"] = torch.logsumexp(x.float(), dim=1)
        return s
    rng = random.Random(seed)
    grads = [(torch.randn(sh, device="cuda", generator=g) * 10.0 ** rng.uniform(-3, -1) / case["scale"] ** 0.5)
             .to(DTYPES[case["dtype"]]) for sh in _shapes(case)]
    s = dict(case=case, grads=grads, max_norm=1.0)
    if case["clip"]:
        s["outs"] = [torch.empty(x.shape, device="cuda", dtype=DTYPES[case["out"]]) for x in grads]
    if own:
        import parity_binade_chunked_gb300 as sq
        s["list"] = sq.TensorList(grads, s.get("outs"))  # the handle that a training program keeps
    return s


# ---- one pass

def run(s):
    kind = s["case"]["kind"]
    if own:
        import parity_binade_chunked_gb300 as sq
        if kind == "sample":
            tokens, logp = sq.sample_tokens(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"],
                                            top_p=s["top_p"], min_p=s["min_p"])
            return {"tokens": tokens, "logp": logp}
        if kind == "logprob":
            if not s["case"]["grad"]:
                logp, lse = sq.token_logprob(s["logits"], s["tokens"])
                return {"logp": logp, "lse": lse}
            if s["case"]["lse"]:
                return {"dlogits": sq.token_logprob_backward(s["logits"], s["tokens"], s["dlogp"], s["lse"])}
            dlogits, logp, lse = sq.token_logprob_grad(s["logits"], s["tokens"], s["dlogp"])
            return {"dlogits": dlogits, "logp": logp, "lse": lse}
        if not s["case"]["clip"]:
            return {"norm": s["list"].norm(scale=s["case"]["scale"])}
        return {"norm": s["list"].clip(s["max_norm"], scale=s["case"]["scale"]), "grads": _some(s["outs"])}
    if kind == "sample":
        return _sample_plain(s)
    if kind == "logprob":
        return _logprob_plain(s)
    return _clip_plain(s)


def _some(outs):
    """At most 60 of the tensors: the two tables, the first layers', the last ones (all are computed)."""
    return outs if len(outs) <= 60 else outs[:56] + outs[-4:]


# ---- the plain forms

def _per_row(v, r, dtype):
    v = v if isinstance(v, torch.Tensor) else torch.full((r,), v, device="cuda", dtype=dtype)
    return v.to(dtype)[:, None]


def _share(part, whole):
    """floor(part * whole / 2^32) for part <= 2^32 and whole < 2^55, in 64-bit integers."""
    hi, lo = whole >> 26, whole & ((1 << 26) - 1)
    return (part * hi + ((part * lo) >> 26)) >> 6


def _sample_rows(x, s, scaled, exp2):
    """The definition: weights in fixed point, then integers throughout.  Returns tokens, scaled logits, the kept sum."""
    r, v = x.shape
    temperature = _per_row(s["temperature"], r, torch.float32)
    top_k = _per_row(s["top_k"], r, torch.int64)
    top_p = _per_row(s["top_p"], r, torch.float32)
    min_p = _per_row(s["min_p"], r, torch.float32)
    x = torch.where(torch.isnan(x), -math.inf, x)
    m = x.max(dim=1, keepdim=True).values
    greedy = temperature <= 0
    d = torch.where(x == m, 0.0, scaled(x, m, torch.where(greedy, 1.0, temperature)))
    w = torch.round(exp2(d) * 2.0 ** 31).long()
    index = torch.arange(v, device=x.device)[None]
    d, order = torch.sort(d, dim=1, descending=True, stable=True)
    ws = w.gather(1, order)
    ws = torch.where((top_k <= 0) | (index < top_k), ws, 0)
    before = ws.cumsum(1) - ws
    cut = _share((top_p.double() * 2.0 ** 32).clamp(0, 2.0 ** 32).long(), ws.sum(1, keepdim=True))
    keep = (top_p >= 1) | (before < cut) | (index == 0)
    keep = keep & (ws >= torch.round(min_p.double() * 2.0 ** 31).long())
    kept = torch.zeros_like(w).scatter_(1, order, torch.where(keep, ws, 0))
    up_to = kept.cumsum(1)
    z = up_to[:, -1:]
    u = (s["u"].double() * 2.0 ** 32).clamp(0, 2.0 ** 32 - 1).long()[:, None]
    token = (up_to <= _share(u, z)).sum(1, keepdim=True)
    first = torch.where(x == m, index, v).min(dim=1, keepdim=True).values
    token = torch.where(greedy, first, token)
    nothing = m == -math.inf
    return torch.where(nothing, -1, token), greedy, nothing, m, torch.where(greedy, 1.0, temperature), z, x


def _sample_plain(s):
    x = s["logits"].float()
    token, greedy, nothing, m, t, z, x = _sample_rows(
        x, s, lambda x, m, t: (x - m) * (torch.full_like(t, LOG2E) / t), torch.exp2)
    c = torch.full_like(t, LOG2E) / t
    at = x.gather(1, token.clamp(min=0))
    d = torch.where(at == m, 0.0, (at - m) * c)
    logp = (d - torch.log2(z.float() * 2.0 ** -31)) * math.log(2.0)
    logp = torch.where(greedy, 0.0, logp)
    logp = torch.where(nothing, -math.inf, logp)
    return {"tokens": token[:, 0], "logp": logp[:, 0]}


def _logprob_plain(s):
    x, t = s["logits"].float(), s["tokens"][:, None]
    v = x.shape[1]
    used = (t >= 0) & (t < v)
    if "lse" in s:
        lse = s["lse"][:, None]
    else:
        m = x.max(dim=1, keepdim=True).values
        lse = m + torch.log(torch.exp(x - m).sum(1, keepdim=True))
    at = t.clamp(0, v - 1)
    logp = torch.where(used, x.gather(1, at) - lse, 0.0)
    if not s["case"]["grad"]:
        return {"logp": logp[:, 0], "lse": lse[:, 0]}
    a = torch.where(used, s["dlogp"][:, None], 0.0)
    d = torch.exp(x - lse).mul_(-a)
    d = d.scatter_add_(1, at, a).to(s["logits"].dtype)
    return {"dlogits": d} if "lse" in s else {"dlogits": d, "logp": logp[:, 0], "lse": lse[:, 0]}


def _clip_plain(s):
    scale = s["case"]["scale"]
    norm = torch.stack([g.float().square().sum() for g in s["grads"]]).sum().sqrt().mul(scale).reshape(1)
    if not s["case"]["clip"]:
        return {"norm": norm}
    f = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0) * scale
    outs = [o.copy_(g.float() * f) for g, o in zip(s["grads"], s["outs"])]
    return {"norm": norm, "grads": _some(outs)}


# ---- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "sample":
        x = s["logits"].double()
        token, greedy, nothing, m, t, z, x = _sample_exact(x, s)
        logp = torch.where(greedy, 0.0, (x.gather(1, token.clamp(min=0)) - m) / t - torch.log(z))
        return {"tokens": None, "logp": torch.where(nothing, -math.inf, logp)[:, 0]}
    if case["kind"] == "logprob":
        x, t = s["logits"].double(), s["tokens"]
        lse = s["lse"].double() if case["lse"] else torch.logsumexp(x, dim=1)
        r = torch.arange(len(t), device=x.device)
        used = (t >= 0) & (t < x.shape[1])
        at = torch.where(used, t, 0)
        logp = torch.where(used, x[r, at] - lse, 0.0)
        if not case["grad"]:
            return {"logp": logp, "lse": lse}
        a = torch.where(used, s["dlogp"].double(), 0.0)
        d = x.sub_(lse[:, None]).exp_().mul_(-a[:, None])
        d[r, at] += a
        return {"dlogits": d} if case["lse"] else {"dlogits": d, "logp": logp, "lse": lse}
    total = math.fsum(float(torch.linalg.vector_norm(g.double())) ** 2 for g in s["grads"])
    norm = math.sqrt(total) * case["scale"]
    out = {"norm": torch.tensor([norm], dtype=torch.float64)}
    if case["clip"]:
        f = case["scale"] * min(1.0, s["max_norm"] / (norm + 1e-6))
        out["grads"] = _some([g.double() * f for g in s["grads"]])
    return out


def _sample_exact(x, s):
    """The kept set from sorted 64-bit probabilities; the draw where their running sum passes u."""
    r, v = x.shape
    temperature = _per_row(s["temperature"], r, torch.float64)
    top_k = _per_row(s["top_k"], r, torch.int64)
    top_p = _per_row(s["top_p"], r, torch.float64)
    min_p = _per_row(s["min_p"], r, torch.float64)
    greedy = temperature <= 0
    t = torch.where(greedy, 1.0, temperature)
    m = x.max(dim=1, keepdim=True).values
    e, order = torch.exp((x - m) / t).sort(dim=1, descending=True, stable=True)
    rank = torch.arange(v, device=x.device)[None]
    e = torch.where((top_k > 0) & (rank >= top_k), 0.0, e)
    before = e.cumsum(1) - e
    keep = ((top_p >= 1) | (before < top_p * e.sum(1, keepdim=True)) | (rank == 0)) & (e >= min_p)
    kept = torch.zeros_like(e).scatter_(1, order, torch.where(keep, e, 0.0))
    up_to = kept.cumsum(1)
    z = up_to[:, -1:].clone()
    token = torch.where(greedy, order[:, :1], (up_to <= s["u"].double()[:, None] * z).sum(1, keepdim=True).clamp(max=v - 1))
    nothing = m == -math.inf
    return token, greedy, nothing, m, t, z, x


# ---- what a pass cannot do without

def work(case):
    if case["kind"] == "sample":
        n = case["rows"] * case["vocab"]
        settings = 16 if case["per_row"] else 0
        return {"bytes": n * BYTES[case["dtype"]] + case["rows"] * (4 + 12 + settings), "flops": 4 * n}
    if case["kind"] == "logprob":
        n = case["rows"] * case["vocab"]
        rows = case["rows"] * (8 + (4 if case["grad"] else 0) + (4 if case["lse"] else 8))
        return {"bytes": n * BYTES[case["dtype"]] * (2 if case["grad"] else 1) + rows, "flops": (7 if case["grad"] else 4) * n}
    n = _numbers(case)
    return {"bytes": n * (BYTES[case["dtype"]] + (BYTES[case["out"]] if case["clip"] else 0)) + 4,
            "flops": (3 if case["clip"] else 2) * n}
