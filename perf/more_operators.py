"""Measured cases of the two ends of a language model in the sharded step: the
token embedding with its gradient, and the distillation loss of the head.

* ``distill``: the loss of a linear head against a teacher's top logits,
  tau^2 KL(teacher || student) at temperature tau over the entries that the
  teacher kept, with or without the gradients of the last hidden states and of
  the head's weight.
* ``embed``: rows of the embedding table times a factor.
* ``embed_grad``: the table's gradient, the rows of each token added up, written
  whole or added to the gradient that a tied head left there.

With ``own`` false, run() computes them from elementary torch operations in
32 bits; with ``own`` true, through the package's entry points. exact() has
the same results in 64 bits.
"""
import math
from types import SimpleNamespace

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
INTS = {32: torch.int32, 64: torch.int64}
DEV = "cuda"
IGNORE = -100  # a token of the padding
UNUSED = -1    # an entry that the teacher did not keep


def listed():
    return [
        # one token scored against its teacher: the latency of a single row
        {"name": "distill one token", "op": "distill", "tokens": 1, "vocab": 50257, "dim": 768, "top": 64,
         "dtype": "bf16", "teacher": "f32", "ids": 64, "grad": False, "scale": 1.0, "tau": 1.0, "short": 0.0,
         "empty": 0.0},
        # evaluation of a batch: losses only
        {"name": "distill evaluation", "op": "distill", "tokens": 2048, "vocab": 32000, "dim": 5120, "top": 32,
         "dtype": "bf16", "teacher": "bf16", "ids": 32, "grad": False, "scale": 1.0, "tau": 2.0, "short": 0.25,
         "empty": 0.1},
        # training on one ragged sequence with a padded tail
        {"name": "distill training ragged", "op": "distill", "tokens": 1021, "vocab": 50257, "dim": 768, "top": 64,
         "dtype": "bf16", "teacher": "f32", "ids": 64, "grad": True, "scale": 1.0, "tau": 1.0, "short": 0.5,
         "empty": 0.2},
        # fp16 training under a static loss scale, an odd number of entries
        {"name": "distill training f16", "op": "distill", "tokens": 4096, "vocab": 50257, "dim": 1280, "top": 101,
         "dtype": "f16", "teacher": "f16", "ids": 32, "grad": True, "scale": 1024.0, "tau": 2.0, "short": 0.0,
         "empty": 0.0},
        # training in fp32 throughout
        {"name": "distill training f32", "op": "distill", "tokens": 512, "vocab": 32000, "dim": 1280, "top": 50,
         "dtype": "f32", "teacher": "f32", "ids": 64, "grad": True, "scale": 1.0, "tau": 4.0, "short": 0.0,
         "empty": 0.1},
        # the widest head: a large vocabulary on a hidden size of 8192, many entries
        {"name": "distill training wide", "op": "distill", "tokens": 4096, "vocab": 128000, "dim": 8192, "top": 256,
         "dtype": "bf16", "teacher": "bf16", "ids": 32, "grad": True, "scale": 1.0, "tau": 1.0, "short": 0.25,
         "empty": 0.05},
        # one token decoded: launch latency
        {"name": "embed one token", "op": "embed", "tokens": 1, "vocab": 50257, "dim": 768, "dtype": "bf16",
         "factor": 1.0, "ignored": 0.0},
        # a batch of long sequences on the widest table, scaled by sqrt(dim)
        {"name": "embed batch wide", "op": "embed", "tokens": 16384, "vocab": 128000, "dim": 8192, "dtype": "bf16",
         "factor": math.sqrt(8192.0), "ignored": 0.05},
        # one ragged sequence: most rows of the gradient are zeros
        {"name": "embed gradient ragged", "op": "embed_grad", "tokens": 1021, "vocab": 50257, "dim": 768,
         "dtype": "bf16", "factor": 1.0, "ignored": 0.2, "add": False},
        # a table tied to the head, whose gradient is there already
        {"name": "embed gradient tied", "op": "embed_grad", "tokens": 8192, "vocab": 50257, "dim": 1280,
         "dtype": "f16", "factor": 1.0, "ignored": 0.0, "add": True},
        # fp32, a width that no vector load divides
        {"name": "embed gradient f32 odd", "op": "embed_grad", "tokens": 4099, "vocab": 32000, "dim": 1283,
         "dtype": "f32", "factor": math.sqrt(1283.0), "ignored": 0.1, "add": False},
        # long sequences on the widest table
        {"name": "embed gradient wide", "op": "embed_grad", "tokens": 32768, "vocab": 128000, "dim": 8192,
         "dtype": "bf16", "factor": 1.0, "ignored": 0.05, "add": False},
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng):
    dim = _log_between(rng, 64, 8192)
    return max(64, dim // 64 * 64) if rng.random() < 0.75 else dim  # most models have round sizes, some do not


def draw(rng):
    op = rng.choice(["distill", "distill", "embed", "embed_grad", "embed_grad"])
    if op == "distill":
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        while True:
            tokens, vocab, dim = _log_between(rng, 1, 8192), _log_between(rng, 1000, 131072), _width(rng)
            # an fp32 head counts six times: its products are as exact as fp32's
            if 6.0 * tokens * vocab * dim * (6 if dtype == "f32" else 1) <= 2.5e13:
                break
        return {"op": op, "tokens": tokens, "vocab": vocab, "dim": dim, "top": _log_between(rng, 1, 256),
                "dtype": dtype, "teacher": rng.choice(["f32", dtype]), "ids": rng.choice([32, 64]),
                "grad": rng.random() < 0.7, "scale": 1024.0 if dtype == "f16" else 1.0,
                "tau": rng.choice([1.0, 1.0, 0.7, 2.0, 4.0]), "short": rng.choice([0.0, 0.25, 0.5]),
                "empty": rng.choice([0.0, 0.1, 0.5])}
    while True:
        tokens, vocab, dim = _log_between(rng, 1, 65536), _log_between(rng, 1000, 262144), _width(rng)
        if tokens * dim <= 2.7e8 and vocab * dim <= 1.05e9:
            break
    case = {"op": op, "tokens": tokens, "vocab": vocab, "dim": dim, "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]),
            "factor": rng.choice([1.0, math.sqrt(dim)]), "ignored": rng.choice([0.0, 0.1, 0.5])}
    if op == "embed_grad":
        case["add"] = rng.random() < 0.4
    return case


# ---------------------------------------------------------------- inputs


def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _prepare_distill(c, seed):
    g = _generator(seed)
    T, V, D, K, dt = c["tokens"], c["vocab"], c["dim"], c["top"], DTYPES[c["dtype"]]
    # the teacher's entries: one token of each of K parts of the vocabulary, in
    # the order of their logits, as a top-k leaves them
    part = torch.arange(K, device=DEV, dtype=torch.float64)
    ids = ((part + torch.rand(T, K, device=DEV, dtype=torch.float64, generator=g)) * (V / K)).long().clamp_(max=V - 1)
    ids = ids.gather(1, torch.rand(T, K, device=DEV, generator=g).argsort(1))
    teacher = torch.empty(T, K, device=DEV).normal_(0.0, 3.0, generator=g).sort(1, descending=True).values + 8.0
    # a head initialised at 0.02 and hidden states of unit size behind a norm,
    # which lean towards the teacher's first token by up to ten
    weight = torch.empty(V, D, device=DEV, dtype=torch.float32).normal_(0.0, 0.02, generator=g).to(dt)
    hidden = torch.empty(T, D, device=DEV, dtype=torch.float32).normal_(0.0, 1.0, generator=g)
    lift = torch.rand(T, 1, device=DEV, generator=g) * 12.0 - 2.0
    toward = weight[ids[:, 0]].float()
    hidden += lift.clamp_min_(0.0) * toward / toward.square().sum(1, keepdim=True)
    # rows of which the teacher kept fewer entries, and a padded tail without any
    kept = torch.randint(1, K + 1, (T,), device=DEV, generator=g)
    kept[torch.rand(T, device=DEV, generator=g) >= c["short"]] = K
    kept[T - int(T * c["empty"]):] = 0
    ids[torch.arange(K, device=DEV) >= kept[:, None]] = UNUSED
    s = SimpleNamespace(op="distill", case=c, hidden=hidden.to(dt), weight=weight,
                        teacher=teacher.to(DTYPES[c["teacher"]]), ids=ids.to(INTS[c["ids"]]))
    if own:
        import sharded_fsdp_reduce_gb300 as F
        s.head = F.HeadDistill(V, D, dt, max_tokens=T, top=K, temperature=c["tau"], grad=c["grad"], device=DEV)
        s.loss = torch.empty((), dtype=torch.float32, device=DEV)
        s.token_loss = torch.empty(T, dtype=torch.float32, device=DEV)
        if c["grad"]:
            s.d_hidden = torch.empty(T, D, dtype=dt, device=DEV)
            s.d_weight = torch.empty(V, D, dtype=dt, device=DEV)
    return s


def _tokens(c, g):
    """Tokens as frequent as a language's: the k-th most common about 1/k as often as the first."""
    T, V = c["tokens"], c["vocab"]
    u = torch.rand(T, device=DEV, dtype=torch.float64, generator=g)
    tokens = (torch.exp(u * math.log(V + 1.0)).long() - 1).clamp_(0, V - 1)
    tokens[T - int(T * c["ignored"]):] = IGNORE  # a padded tail
    return tokens


def _used(c):
    """How many rows of the table such tokens are expected to use."""
    n = c["tokens"] - int(c["tokens"] * c["ignored"])
    v = torch.arange(1, c["vocab"] + 1, dtype=torch.float64)
    p = torch.log1p(1.0 / v) / math.log(c["vocab"] + 1.0)
    return float(-torch.expm1(n * torch.log1p(-p)).sum())


def _prepare_embed(c, seed):
    g = _generator(seed)
    T, V, D, dt = c["tokens"], c["vocab"], c["dim"], DTYPES[c["dtype"]]
    s = SimpleNamespace(op=c["op"], case=c, tokens=_tokens(c, g))
    if c["op"] == "embed":
        s.weight = torch.empty(V, D, device=DEV, dtype=torch.float32).normal_(0.0, 0.02, generator=g).to(dt)
        s.out = torch.empty(T, D, dtype=dt, device=DEV)
    else:
        s.d_out = torch.empty(T, D, device=DEV, dtype=torch.float32).normal_(0.0, 1e-2, generator=g).to(dt)
        s.d_weight = torch.empty(V, D, dtype=dt, device=DEV)
        if c["add"]:
            s.d_weight.normal_(0.0, 1e-2, generator=g)
    if own:
        import sharded_fsdp_reduce_gb300 as F
        s.table = F.Embedding(V, D, dt, max_tokens=T, scale=c["factor"], grad=c["op"] == "embed_grad", device=DEV)
    return s


def prepare(case, seed):
    return (_prepare_distill if case["op"] == "distill" else _prepare_embed)(case, seed)


# ---------------------------------------------------------------- one pass


def _plain_distill(s):
    c, tau = s.case, s.case["tau"]
    x, w = s.hidden.float(), s.weight.float()
    # the teacher's distribution over its entries
    ids, a = s.ids.long(), s.teacher.float() / tau
    live = (ids >= 0) & (a > -math.inf)
    row = live.any(1)
    a = torch.where(live, a, -math.inf)
    a = a - torch.where(row, a.max(1).values, 0.0).unsqueeze(1)
    sum_p = torch.exp(a).sum(1, keepdim=True)
    p = torch.where(live, torch.exp(a) / sum_p, 0.0)
    at = torch.where(live, ids, 0)
    # the student's over the vocabulary
    z = (x @ w.t()).div_(tau)
    top = z.max(1, keepdim=True).values
    at_ids = z.gather(1, at)
    e = torch.exp(z.sub_(top))
    total = e.sum(1, keepdim=True)
    kl = torch.where(live, p * ((a - torch.log(sum_p)) - (at_ids - top - torch.log(total))), 0.0).sum(1)
    token_loss = torch.where(row, tau * tau * kl, 0.0)
    count = row.sum().clamp(min=1).float()
    loss = token_loss.sum() / count
    if not c["grad"]:
        return loss, token_loss
    del z
    d = e.div_(total)
    d.scatter_add_(1, at, -p)
    d.mul_((row.float() * (c["scale"] * tau / count)).unsqueeze(1))
    return loss, token_loss, (d @ w).to(s.hidden.dtype), (d.t() @ x).to(s.weight.dtype)


def _own_distill(s):
    if not s.case["grad"]:
        return s.head.forward(s.hidden, s.weight, s.teacher, s.ids, loss=s.loss, token_loss=s.token_loss)
    loss, token_loss = s.head.forward_backward(s.hidden, s.weight, s.teacher, s.ids, s.d_hidden, s.d_weight,
                                               grad_scale=s.case["scale"], loss=s.loss, token_loss=s.token_loss)
    return loss, token_loss, s.d_hidden, s.d_weight


def _plain_embed(s):
    live = s.tokens != IGNORE
    rows = s.weight[torch.where(live, s.tokens, 0)].float() * s.case["factor"]
    s.out.copy_(torch.where(live.unsqueeze(1), rows, 0.0))
    return s.out


def _plain_embed_grad(s):
    live = s.tokens != IGNORE
    rows = torch.where(live.unsqueeze(1), s.d_out.float(), 0.0)
    total = torch.zeros(s.d_weight.shape, dtype=torch.float32, device=DEV)
    total.index_add_(0, torch.where(live, s.tokens, 0), rows)
    total.mul_(s.case["factor"])
    s.d_weight.copy_(s.d_weight.float() + total if s.case["add"] else total)
    return s.d_weight


def run(state):
    if state.op == "distill":
        return _own_distill(state) if own else _plain_distill(state)
    if state.op == "embed":
        return state.table.forward(state.tokens, state.weight, out=state.out) if own else _plain_embed(state)
    if own:
        return state.table.backward(state.tokens, state.d_out, state.d_weight, accumulate=state.case["add"])
    return _plain_embed_grad(state)


# ---------------------------------------------------------------- what a pass has to do


def work(case):
    c = case
    e = 4 if c["dtype"] == "f32" else 2
    T, V, D = c["tokens"], c["vocab"], c["dim"]
    if c["op"] == "distill":
        both = 2 if c["grad"] else 1  # the inputs, and their gradients
        entry = (4 if c["teacher"] == "f32" else 2) + c["ids"] // 8
        return {"bytes": float(both * e * (T + V) * D + entry * T * c["top"] + 4 * T),
                "flops": (6.0 if c["grad"] else 2.0) * T * V * D}
    if c["op"] == "embed":
        return {"bytes": 8.0 * T + e * D * (_used(c) + T), "flops": float(T) * D}
    rows = T - int(T * c["ignored"])
    table = 2.0 * _used(c) if c["add"] else float(V)
    return {"bytes": 8.0 * T + e * D * (rows + table), "flops": float(rows) * D}


# ---------------------------------------------------------------- in 64 bits


def _exact_distill(c, s):
    if 6.0 * c["tokens"] * c["vocab"] * c["dim"] > 4e12:
        return None
    T, tau = c["tokens"], c["tau"]
    w = s.weight.double()
    token_loss = torch.zeros(T, dtype=torch.float64, device=DEV)
    dx = torch.zeros(T, c["dim"], dtype=torch.float64, device=DEV)
    dw = torch.zeros_like(w)
    keep = (s.ids >= 0) & torch.isfinite(s.teacher)
    rows = keep.any(1).nonzero().flatten()
    g = c["scale"] * tau / max(1, rows.numel())
    for part in rows.split(512):
        x = s.hidden[part].double()
        log_q = torch.log_softmax((x @ w.t()) / tau, 1)
        i, k = keep[part].nonzero(as_tuple=True)
        v = s.ids[part][i, k].long()
        log_p = torch.full((part.numel(), c["top"]), -math.inf, dtype=torch.float64, device=DEV)
        log_p[i, k] = s.teacher[part][i, k].double() / tau
        log_p = torch.log_softmax(log_p, 1)[i, k]
        p = torch.exp(log_p)
        token_loss.index_put_((part[i],), tau * tau * p * (log_p - log_q[i, v]), accumulate=True)
        if c["grad"]:
            d = torch.exp(log_q)
            d.index_put_((i, v), -p, accumulate=True)
            dx[part] = g * (d @ w)
            dw += g * (d.t() @ x)
    loss = token_loss.sum() / max(1, rows.numel())
    return (loss, token_loss, dx, dw) if c["grad"] else (loss, token_loss)


def _exact_embed(c, s):
    keep = (s.tokens != IGNORE).nonzero().flatten()
    if c["op"] == "embed":
        out = torch.zeros(c["tokens"], c["dim"], dtype=torch.float64, device=DEV)
        out[keep] = s.weight[s.tokens[keep]].double() * c["factor"]
        return out
    d_weight = s.d_weight.double() if c["add"] else torch.zeros(s.d_weight.shape, dtype=torch.float64, device=DEV)
    return d_weight.index_put_((s.tokens[keep],), s.d_out[keep].double() * c["factor"], accumulate=True)


def exact(case, seed):
    s = prepare(case, seed)
    return (_exact_distill if case["op"] == "distill" else _exact_embed)(case, s)
