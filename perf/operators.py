"""Measured cases of the head loss, the gradient clipping and the clipped model step.

Three operators around the sharded optimizer step:

* ``loss``: softmax cross entropy of a linear head over a large vocabulary,
  from the last hidden states and the head's weight, with or without the
  gradients of both.
* ``clip``: the global L2 norm over many gradient tensors and their scaling
  to a largest norm, written into a flat gradient buffer.
* ``step``: the model step of FSDP units with the averaged gradient's global
  norm clipped between the reduce-scatter and AdamW.

With ``own`` false, run() computes them from elementary torch operations in
32 bits; with ``own`` true, through the package's entry points. exact() has
the same results in 64 bits.
"""
import math
from types import SimpleNamespace

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
DEV = "cuda"
IGNORE = -100
CLIP_EPS = 1e-6  # added to the norm under the clipping quotient

# AdamW's scalars of every measured step
LR, BETA1, BETA2, EPS, DECAY, STEP = 1e-3, 0.9, 0.95, 1e-8, 0.1, 100


def listed():
    return [
        # one token scored: the latency of a single row against the whole vocabulary
        {"name": "loss one token", "op": "loss", "tokens": 1, "vocab": 50257, "dim": 768, "dtype": "bf16",
         "grad": False, "scale": 1.0, "ignored": 0.0},
        # evaluation of a batch: losses only
        {"name": "loss evaluation", "op": "loss", "tokens": 2048, "vocab": 32000, "dim": 5120, "dtype": "bf16",
         "grad": False, "scale": 1.0, "ignored": 0.1},
        # training on one ragged sequence with a padded tail
        {"name": "loss training ragged", "op": "loss", "tokens": 1021, "vocab": 50257, "dim": 768, "dtype": "bf16",
         "grad": True, "scale": 1.0, "ignored": 0.2},
        # fp16 training under a static loss scale
        {"name": "loss training f16", "op": "loss", "tokens": 4096, "vocab": 50257, "dim": 1280, "dtype": "f16",
         "grad": True, "scale": 1024.0, "ignored": 0.0},
        # training in fp32 throughout
        {"name": "loss training f32", "op": "loss", "tokens": 512, "vocab": 32000, "dim": 1280, "dtype": "f32",
         "grad": True, "scale": 1.0, "ignored": 0.1},
        # the widest head: a large vocabulary on a hidden size of 8192
        {"name": "loss training wide", "op": "loss", "tokens": 4096, "vocab": 128000, "dim": 8192, "dtype": "bf16",
         "grad": True, "scale": 1.0, "ignored": 0.05},
        # a few small odd tensors: launch latency
        {"name": "clip few small", "op": "clip", "tensors": 15, "numel": 52_361, "dtype": "f32", "sigma": 1e-2},
        # the leaves of a whole model of some 700 M parameters
        {"name": "clip many", "op": "clip", "tensors": 433, "numel": 708_390_403, "dtype": "bf16", "sigma": 1e-3},
        # a model of small units: launch latency of the whole clipped step
        {"name": "step small units", "op": "step", "units": 15, "numel": 750_015, "world": 8, "grad_dtype": "bf16",
         "out_dtype": "bf16", "scale": 1.0, "sigma": 1e-3},
        # the twelve blocks of GPT-2 small
        {"name": "step gpt2 small", "op": "step", "units": 12, "numel": 12 * 7_087_872, "world": 8,
         "grad_dtype": "bf16", "out_dtype": "bf16", "scale": 1.0, "sigma": 1e-3},
        # GPT-2 Large blocks, fp16 under a loss scale, two ranks
        {"name": "step gpt2 large f16", "op": "step", "units": 8, "numel": 8 * 19_677_440, "world": 2,
         "grad_dtype": "f16", "out_dtype": "f16", "scale": 1024.0, "sigma": 1e-3},
        # one GPT-3 13B block over eight ranks
        {"name": "step gpt3 13b", "op": "step", "units": 1, "numel": 314_639_360, "world": 8, "grad_dtype": "bf16",
         "out_dtype": "bf16", "scale": 1.0, "sigma": 1e-4},
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["loss", "loss", "clip", "step"])
    if op == "loss":
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        grad = rng.random() < 0.7
        while True:
            tokens, vocab = _log_between(rng, 1, 8192), _log_between(rng, 1000, 131072)
            dim = _log_between(rng, 64, 8192)
            if rng.random() < 0.75:
                dim = max(64, dim // 64 * 64)  # most heads have round sizes, some do not
            # an fp32 head counts six times: its products are as exact as fp32's
            if 6.0 * tokens * vocab * dim * (6 if dtype == "f32" else 1) <= 2.5e13:
                break
        return {"op": op, "tokens": tokens, "vocab": vocab, "dim": dim, "dtype": dtype, "grad": grad,
                "scale": 1024.0 if dtype == "f16" else 1.0, "ignored": rng.choice([0.0, 0.1, 0.5])}
    if op == "clip":
        tensors = _log_between(rng, 1, 500)
        return {"op": op, "tensors": tensors, "numel": tensors + _log_between(rng, 1000, 700_000_000),
                "dtype": rng.choice(["bf16", "f16", "f32"]), "sigma": rng.choice([1e-4, 1e-3, 1e-2])}
    units = rng.randint(1, 15)
    grad_dtype = rng.choice(["bf16", "f16", "f32"])
    scale = 1024.0 if grad_dtype == "f16" else 1.0
    out_dtype = rng.choice(["bf16", "f16"]) if grad_dtype == "f32" else grad_dtype
    return {"op": op, "units": units, "numel": units + _log_between(rng, 10_000, 150_000_000),
            "world": rng.choice([1, 2, 3, 4, 8, 8]), "grad_dtype": grad_dtype, "out_dtype": out_dtype,
            "scale": scale, "sigma": rng.choice([1e-4, 1e-3])}


# ---------------------------------------------------------------- inputs


def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _prepare_loss(c, seed):
    g = _generator(seed)
    T, V, D, dt = c["tokens"], c["vocab"], c["dim"], DTYPES[c["dtype"]]
    # a head initialised at 0.02 and hidden states of unit size behind a norm,
    # which lean towards the target by up to ten, as a trained model's do
    weight = torch.empty(V, D, device=DEV, dtype=torch.float32).normal_(0.0, 0.02, generator=g).to(dt)
    targets = torch.randint(0, V, (T,), device=DEV, generator=g)
    hidden = torch.empty(T, D, device=DEV, dtype=torch.float32).normal_(0.0, 1.0, generator=g)
    lift = torch.rand(T, 1, device=DEV, generator=g) * 12.0 - 2.0
    toward = weight[targets].float()
    hidden += lift.clamp_min_(0.0) * toward / toward.square().sum(1, keepdim=True)
    n_ignored = int(T * c["ignored"])
    if n_ignored:
        targets[T - n_ignored:] = IGNORE  # a padded tail
    s = SimpleNamespace(op="loss", case=c, hidden=hidden.to(dt), weight=weight, targets=targets)
    if own:
        import sharded_fsdp_reduce_gb300 as F
        s.head = F.HeadLoss(V, D, dt, max_tokens=T, grad=c["grad"], device=DEV)
        s.loss = torch.empty((), dtype=torch.float32, device=DEV)
        s.token_loss = torch.empty(T, dtype=torch.float32, device=DEV)
        if c["grad"]:
            s.d_hidden = torch.empty(T, D, dtype=dt, device=DEV)
            s.d_weight = torch.empty(V, D, dtype=dt, device=DEV)
    return s


def _clip_sizes(c):
    """Tensor sizes that add up to numel: matrices and their small vectors."""
    n, total = c["tensors"], c["numel"]
    shares = [(1.0, 0.002, 0.35, 0.001)[k % 4] * (1.0 + 0.1 * (k % 7)) for k in range(n)]
    left = total - n
    sizes = [1 + int(left * x / sum(shares)) for x in shares]
    sizes[0] += total - sum(sizes)
    return sizes


def _prepare_clip(c, seed):
    g = _generator(seed)
    dt = DTYPES[c["dtype"]]
    sizes = _clip_sizes(c)
    flat = torch.empty(c["numel"], device=DEV, dtype=dt).normal_(0.0, c["sigma"], generator=g)
    out = torch.empty(c["numel"], device=DEV, dtype=dt)
    s = SimpleNamespace(op="clip", case=c, tensors=list(flat.split(sizes)), out=out, outs=list(out.split(sizes)),
                        max_norm=0.5 * c["sigma"] * math.sqrt(c["numel"]))
    if own:
        import sharded_fsdp_reduce_gb300 as F
        s.clip = F.GradClip(s.tensors, out=s.outs)
    return s


def _unit_sizes(c):
    n, total = c["units"], c["numel"]
    if n * (total // n) == total and total % n == 0 and total // n > 1_000_000:
        return [total // n] * n  # equal blocks
    shares = [1.0 + 0.13 * (k % 5) for k in range(n)]
    sizes = [1 + int((total - n) * x / sum(shares)) for x in shares]
    sizes[0] += total - sum(sizes)
    return sizes


def _prepare_step(c, seed):
    g = _generator(seed)
    N, gdt, odt = c["world"], DTYPES[c["grad_dtype"]], DTYPES[c["out_dtype"]]
    sizes = _unit_sizes(c)
    if own:
        import sharded_fsdp_reduce_gb300 as F
        units = [F.FlatParamUnit([("w", (p,))], N, gdt, odt, device=DEV, n_full=1) for p in sizes]
    else:
        units = []
        for p in sizes:
            pad = -(-p // N) * N
            empty = lambda dt: torch.empty(pad, dtype=dt, device=DEV)  # noqa: E731
            units.append(SimpleNamespace(numel=p, grads=[empty(gdt) for _ in range(N)], master=empty(torch.float32),
                                         exp_avg=empty(torch.float32), exp_avg_sq=empty(torch.float32),
                                         full=[empty(odt)]))
    for u in units:
        for x in u.grads:
            x.normal_(0.0, c["sigma"] * c["scale"], generator=g)
        u.master.uniform_(-0.1, 0.1, generator=g)
        u.exp_avg.normal_(0.0, 0.3 * c["sigma"], generator=g)
        u.exp_avg_sq.uniform_(0.2 * c["sigma"] ** 2, c["sigma"] ** 2, generator=g)
        for x in [*u.grads, u.master, u.exp_avg, u.exp_avg_sq]:
            x[u.numel:] = 0  # the padding
    # a norm about twice the largest one allowed
    s = SimpleNamespace(op="step", case=c, units=units,
                        max_norm=0.5 * c["sigma"] * math.sqrt(c["numel"] / N))
    if own:
        s.model = F.UnitSequence(units)
        s.hp = F.AdamWHParams(LR, BETA1, BETA2, EPS, DECAY, STEP, c["scale"])
        s.norm = torch.empty((), dtype=torch.float32, device=DEV)
    return s


def prepare(case, seed):
    return {"loss": _prepare_loss, "clip": _prepare_clip, "step": _prepare_step}[case["op"]](case, seed)


# ---------------------------------------------------------------- one pass


def _plain_loss(s):
    c = s.case
    x, w = s.hidden.float(), s.weight.float()
    valid = s.targets != IGNORE
    at = torch.where(valid, s.targets, 0).unsqueeze(1)
    logits = x @ w.t()
    top = logits.max(1, keepdim=True).values
    e = torch.exp(logits - top)
    total = e.sum(1, keepdim=True)
    token_loss = torch.where(valid, (torch.log(total) + top - logits.gather(1, at)).squeeze(1), 0.0)
    count = valid.sum().clamp(min=1).float()
    loss = token_loss.sum() / count
    if not c["grad"]:
        return loss, token_loss
    del logits
    d = e.div_(total)
    d.scatter_add_(1, at, torch.full_like(at, -1.0, dtype=torch.float32))
    d.mul_((valid.float() * (c["scale"] / count)).unsqueeze(1))
    return loss, token_loss, (d @ w).to(s.hidden.dtype), (d.t() @ x).to(s.weight.dtype)


def _own_loss(s):
    if not s.case["grad"]:
        return s.head.forward(s.hidden, s.weight, s.targets, loss=s.loss, token_loss=s.token_loss)
    loss, token_loss = s.head.forward_backward(s.hidden, s.weight, s.targets, s.d_hidden, s.d_weight,
                                               grad_scale=s.case["scale"], loss=s.loss, token_loss=s.token_loss)
    return loss, token_loss, s.d_hidden, s.d_weight


def _coefficient(norm, max_norm):
    return (max_norm / (norm + CLIP_EPS)).clamp(max=1.0)


def _plain_clip(s):
    norm = torch.stack([x.float().square().sum() for x in s.tensors]).sum().sqrt()
    coef = _coefficient(norm, s.max_norm)
    _ = [y.copy_(x.float() * coef) for x, y in zip(s.tensors, s.outs)]
    return norm, s.out


def _own_clip(s):
    return s.clip.clip(s.max_norm), s.out


def _plain_update(u, g, coef):
    g = g * coef
    u.master.mul_(1.0 - LR * DECAY)
    u.exp_avg.mul_(BETA1).add_(g, alpha=1.0 - BETA1)
    u.exp_avg_sq.mul_(BETA2).add_(g * g, alpha=1.0 - BETA2)
    denom = u.exp_avg_sq.sqrt().div_(math.sqrt(1.0 - BETA2 ** STEP)).add_(EPS)
    u.master.sub_((u.exp_avg / denom).mul_(LR / (1.0 - BETA1 ** STEP)))
    u.full[0].copy_(u.master)
    return [u.master, u.exp_avg, u.exp_avg_sq, u.full[0]]


def _plain_step(s):
    c = s.case
    mean = [sum(x.float() for x in u.grads).mul_(1.0 / (c["world"] * c["scale"])) for u in s.units]
    norm = torch.stack([g.square().sum() for g in mean]).sum().sqrt()
    coef = _coefficient(norm, s.max_norm)
    return [norm] + [_plain_update(u, g, coef) for u, g in zip(s.units, mean)]


def _own_step(s):
    s.model.clip_step(s.hp, s.max_norm, gathers=1, norm=s.norm)
    return [s.norm] + [[u.master, u.exp_avg, u.exp_avg_sq, u.full[0]] for u in s.units]


def run(state):
    if own:
        return {"loss": _own_loss, "clip": _own_clip, "step": _own_step}[state.op](state)
    return {"loss": _plain_loss, "clip": _plain_clip, "step": _plain_step}[state.op](state)


# ---------------------------------------------------------------- what a pass has to do


def work(case):
    c = case
    size = lambda name: 4 if c[name] == "f32" else 2  # noqa: E731
    if c["op"] == "loss":
        T, V, D, e = c["tokens"], c["vocab"], c["dim"], size("dtype")
        both = 2 if c["grad"] else 1  # the inputs, and their gradients
        return {"bytes": both * e * (T + V) * D + 8 * T + 4 * T, "flops": (6.0 if c["grad"] else 2.0) * T * V * D}
    if c["op"] == "clip":
        return {"bytes": 2.0 * c["numel"] * size("dtype"), "flops": 3.0 * c["numel"]}
    per = c["world"] * size("grad_dtype") + 24 + 2 * size("out_dtype")  # the shard and one gathered buffer
    return {"bytes": float(c["numel"]) * per, "flops": float(c["numel"]) * (c["world"] + 17)}


# ---------------------------------------------------------------- in 64 bits


def _exact_loss(c, s):
    if 6.0 * c["tokens"] * c["vocab"] * c["dim"] > 4e12:
        return None
    w = s.weight.double()
    T = c["tokens"]
    token_loss = torch.zeros(T, dtype=torch.float64, device=DEV)
    dx = torch.zeros(T, c["dim"], dtype=torch.float64, device=DEV)
    dw = torch.zeros_like(w)
    rows = (s.targets != IGNORE).nonzero().flatten()
    g = c["scale"] / max(1, rows.numel())
    for part in rows.split(512):
        x = s.hidden[part].double()
        z = x @ w.t()
        lse = torch.logsumexp(z, 1)
        y = s.targets[part]
        k = torch.arange(part.numel(), device=DEV)
        token_loss[part] = lse - z[k, y]
        if c["grad"]:
            p = torch.exp(z - lse[:, None])
            p[k, y] -= 1.0
            dx[part] = g * (p @ w)
            dw += g * (p.t() @ x)
    loss = token_loss.sum() / max(1, rows.numel())
    return (loss, token_loss, dx, dw) if c["grad"] else (loss, token_loss)


def _exact_clip(c, s):
    x = torch.cat([t.reshape(-1) for t in s.tensors]).double()
    norm = math.sqrt(float(torch.dot(x, x)))
    return norm, x * min(1.0, s.max_norm / (norm + CLIP_EPS))


def _exact_step(c, s):
    total, grads = 0.0, []
    for u in s.units:
        g = torch.zeros(u.master.numel(), dtype=torch.float64, device=DEV)
        for x in u.grads:
            g += x.double()
        g /= c["world"] * c["scale"]
        total += float(torch.dot(g, g))
        grads.append(g)
    norm = math.sqrt(total)
    coef = min(1.0, s.max_norm / (norm + CLIP_EPS))
    out = [norm]
    for u, g in zip(s.units, grads):
        g = g * coef
        m = BETA1 * u.exp_avg.double() + (1.0 - BETA1) * g
        v = BETA2 * u.exp_avg_sq.double() + (1.0 - BETA2) * g ** 2
        step = (m / (1.0 - BETA1 ** STEP)) / (torch.sqrt(v / (1.0 - BETA2 ** STEP)) + EPS)
        p = u.master.double() * (1.0 - LR * DECAY) - LR * step
        out.append([p, m, v, p])
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"loss": _exact_loss, "clip": _exact_clip, "step": _exact_step}[case["op"]](case, s)
