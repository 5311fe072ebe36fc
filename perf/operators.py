"""The training-step operators around main_grad, as measured cases.

Four operators, each reached through the package's public functions:

  logprobs       token_logprobs: log probability of a given token in every row of logits,
                 with the row's entropy, its log of the sum of exponentials and its
                 top alternatives
  logprobs_grad  token_logprobs_backward: the gradient of log probability and entropy
                 with respect to the logits
  ortho          orthogonalize_update: five Newton-Schulz steps on a matrix or a batch
  muon           muon_step: momentum from main_grad, orthogonalised, applied to the weight

`own` chooses between the plain forms below (elementary torch operations in 32 bits,
rounded once at the end) and the package's kernels.
"""
import math

import torch

own = False

DEVICE = "cuda"
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # one token of one sequence, as a decode step scores it with five alternatives
        {"name": "logprobs_1x32000_bf16_k5", "op": "logprobs", "rows": 1, "vocab": 32000, "dtype": "bf16",
         "top_k": 5, "temperature": 1.0, "mask": False},
        # a decode batch with 20 alternatives; constrained rows hold -inf for tokens not allowed
        {"name": "logprobs_48x129280_fp32_k20", "op": "logprobs", "rows": 48, "vocab": 129280, "dtype": "fp32",
         "top_k": 20, "temperature": 0.7, "mask": True},
        # scoring of given answers over an odd vocabulary (rows start at any 2-byte boundary)
        {"name": "logprobs_2047x32003_bf16_k8", "op": "logprobs", "rows": 2047, "vocab": 32003, "dtype": "bf16",
         "top_k": 8, "temperature": 1.0, "mask": False},
        # the loss of a training micro-batch of 8192 tokens
        {"name": "logprobs_8192x129280_bf16", "op": "logprobs", "rows": 8192, "vocab": 129280, "dtype": "bf16",
         "top_k": 0, "temperature": 1.0, "mask": False},
        # the gradient of a few scored tokens
        {"name": "logprobs_grad_37x512_fp32", "op": "logprobs_grad", "rows": 37, "vocab": 512, "dtype": "fp32",
         "temperature": 1.0, "entropy": True},
        # policy training: an entropy bonus beside the log probability, an odd vocabulary, fp32
        {"name": "logprobs_grad_2047x32003_fp32", "op": "logprobs_grad", "rows": 2047, "vocab": 32003,
         "dtype": "fp32", "temperature": 0.9, "entropy": True},
        # the gradient of the 8192-token micro-batch's loss
        {"name": "logprobs_grad_8192x129280_bf16", "op": "logprobs_grad", "rows": 8192, "vocab": 129280,
         "dtype": "bf16", "temperature": 1.0, "entropy": False},
        # a small square matrix: launch latency counts
        {"name": "ortho_1x128x128_fp32", "op": "ortho", "batch": 1, "m": 128, "n": 128, "dtype": "fp32"},
        # stacked tall matrices of odd sizes, one call for all
        {"name": "ortho_12x1023x389_bf16", "op": "ortho", "batch": 12, "m": 1023, "n": 389, "dtype": "bf16"},
        # a projection between the hidden sizes of the embedding workloads
        {"name": "ortho_1x4096x7168_bf16", "op": "ortho", "batch": 1, "m": 4096, "n": 7168, "dtype": "bf16"},
        # the whole optimiser step of a mid-sized matrix with bf16 weights
        {"name": "muon_1x1024x4096_bf16", "op": "muon", "batch": 1, "m": 1024, "n": 4096, "dtype": "fp32",
         "weight": "bf16", "nesterov": True},
        # the largest: a square matrix of the headline hidden size, fp32 master weights
        {"name": "muon_1x7168x7168_fp32", "op": "muon", "batch": 1, "m": 7168, "n": 7168, "dtype": "fp32",
         "weight": "fp32", "nesterov": True},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs_grad", "ortho", "muon"])
    dtype = rng.choice(["bf16", "fp32"])
    if op in ("logprobs", "logprobs_grad"):
        most = 8192 * 129280 * 2 // SIZE[dtype]
        vocab = _spread(rng, 512, 129280)
        rows = _spread(rng, 1, min(8192, most // vocab))
        case = {"op": op, "rows": rows, "vocab": vocab, "dtype": dtype, "temperature": rng.choice([1.0, 1.0, 0.7, 1.3])}
        if op == "logprobs":
            case.update(top_k=rng.choice([0, 1, 5, 8, 20]) if rows * vocab < 1 << 28 else 0, mask=rng.random() < 0.3)
        else:
            case.update(entropy=rng.random() < 0.5)
        return case
    m, n = _spread(rng, 64, 7168), _spread(rng, 64, 7168)
    k, long = min(m, n), max(m, n)
    fits = max(1, int(2.1e12 / (STEPS * k * k * (3 * long + k))))
    batch = _spread(rng, 1, min(fits, 32)) if op == "ortho" else _spread(rng, 1, min(fits, 4))
    if op == "ortho":
        return {"op": op, "batch": batch, "m": m, "n": n, "dtype": dtype}
    return {"op": op, "batch": batch, "m": m, "n": n, "dtype": dtype, "weight": rng.choice(["bf16", "fp32"]),
            "nesterov": rng.random() < 0.7}


# ---- inputs ------------------------------------------------------------------

def _logits(case, g):
    """Rows of N(0, 2) logits with one favoured token each, and the tokens asked for: the
    favoured one in six rows of ten, else any; a sixteenth of the rows asks for none."""
    rows, vocab = case["rows"], case["vocab"]
    x = torch.randn(rows, vocab, generator=g, device=DEVICE, dtype=DTYPES[case["dtype"]])
    x *= 2.0
    hot = torch.randint(0, vocab, (rows,), generator=g, device=DEVICE)
    at = torch.arange(rows, device=DEVICE)
    lift = 6 + 8 * torch.rand(rows, generator=g, device=DEVICE)
    x[at, hot] = lift.to(x.dtype)
    if case.get("mask"):
        # every second row is constrained: to a third of the tokens, or to about one in a hundred;
        # the favoured token stays allowed
        token = torch.arange(vocab, device=DEVICE)
        x[1::4, token % 3 != 0] = -math.inf
        x[3::4, token % 97 != 5] = -math.inf
        x[at, hot] = lift.to(x.dtype)
    other = torch.randint(0, vocab, (rows,), generator=g, device=DEVICE)
    pick = torch.rand(rows, generator=g, device=DEVICE)
    targets = torch.where(pick < 0.6, hot, other)
    targets = torch.where(pick > 15 / 16, torch.full_like(targets, -100), targets)
    return x, targets


def _gradient(batch, m, n, g, scale):
    """Matrices as gradients are: a few strong directions over noise."""
    r = max(1, min(m, n) // 16)
    a = torch.randn(batch, m, r, generator=g, device=DEVICE)
    b = torch.randn(batch, r, n, generator=g, device=DEVICE)
    u = torch.matmul(a, b) / math.sqrt(r)
    u += 0.5 * torch.randn(batch, m, n, generator=g, device=DEVICE)
    return u * scale


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    op = case["op"]
    if op == "logprobs":
        logits, targets = _logits(case, g)
        return {"case": case, "logits": logits, "targets": targets}
    if op == "logprobs_grad":
        logits, targets = _logits(case, g)
        rows = case["rows"]
        gl = -torch.rand(rows, generator=g, device=DEVICE) / rows
        gh = -0.01 * torch.rand(rows, generator=g, device=DEVICE) / rows if case["entropy"] else None
        # what the forward pass left
        fwd = _plain_logprobs(logits, targets, 0, case["temperature"])
        return {"case": case, "logits": logits, "targets": targets, "logsumexp": fwd["logsumexp"],
                "entropy": fwd["entropy"], "grad_logprobs": gl, "grad_entropy": gh, "out": torch.empty_like(logits)}
    shape = (case["batch"], case["m"], case["n"])
    if op == "ortho":
        return {"case": case, "update": _gradient(*shape, g, 1e-3).to(DTYPES[case["dtype"]])}
    main_grad = _gradient(*shape, g, 1e-3).to(DTYPES[case["dtype"]])
    momentum = _gradient(*shape, g, 4e-3)
    weight = (0.02 * torch.randn(shape, generator=g, device=DEVICE)).to(DTYPES[case["weight"]])
    return {"case": case, "main_grad": main_grad, "momentum": momentum, "weight": weight,
            "new_momentum": torch.empty_like(momentum), "new_weight": torch.empty_like(weight),
            "lr": 3e-4, "beta": 0.95, "weight_decay": 0.1, "scale": 0.2 * math.sqrt(max(case["m"], case["n"]))}


# ---- the plain forms ---------------------------------------------------------

def _plain_top(logits, x, lse, top_k):
    """The top_k largest logits of a row by value, equal ones by the lowest index first; -1
    where fewer are above -inf, or where the row has no probabilities (a NaN or +inf)."""
    index = torch.arange(logits.shape[1], device=logits.device)
    bits = (logits.float() + 0.0).view(torch.int32).to(torch.int64)
    ordered = torch.where(bits >= 0, bits, bits ^ 0x7FFFFFFF)
    key = ordered * (1 << 32) + (0xFFFFFFFF - index)  # no two alike
    ids = 0xFFFFFFFF - (key.topk(top_k, dim=1).values & 0xFFFFFFFF)
    top = x.gather(1, ids) - lse[:, None]
    none = (x.gather(1, ids) == -math.inf) | torch.isnan(lse)[:, None]
    return torch.where(none & ~torch.isnan(lse)[:, None], torch.full_like(top, -math.inf), top), ids.masked_fill(none, -1)


def _plain_logprobs(logits, targets, top_k, temperature):
    vocab = logits.shape[1]
    x = logits.float() / temperature
    m = x.amax(1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    d = x - m
    e = torch.exp(d)
    s = e.sum(1)
    log_s = torch.log(s)
    weighted = (e * torch.where(e == 0, torch.zeros_like(d), d)).sum(1)
    lse = m[:, 0] + log_s
    entropy = torch.where(s == 0, torch.zeros_like(s), log_s - weighted / s)
    asked = d.gather(1, targets.long().clamp(0, vocab - 1)[:, None])[:, 0] - torch.where(s == 0, torch.zeros_like(s), log_s)
    asked = torch.where(targets < 0, torch.zeros_like(asked), asked)
    asked = torch.where(targets >= vocab, torch.full_like(asked, math.nan), asked)
    out = {"logprobs": asked, "entropy": entropy, "logsumexp": lse}
    if top_k:
        out["top_logprobs"], out["top_ids"] = _plain_top(logits, x, lse, top_k)
    return out


def _plain_logprobs_grad(logits, targets, lse, entropy, grad_logprobs, grad_entropy, temperature):
    vocab = logits.shape[1]
    empty = (lse == -math.inf)[:, None]
    logp = logits.float() / temperature - torch.where(empty, torch.zeros_like(lse)[:, None], lse[:, None])
    p = torch.exp(logp)
    g = torch.where(targets < 0, torch.zeros_like(grad_logprobs), grad_logprobs)
    g = torch.where(targets >= vocab, torch.full_like(g, math.nan), g)[:, None]
    grad = -g * p
    if grad_entropy is not None:
        grad = grad - grad_entropy[:, None] * p * (torch.where(p == 0, torch.zeros_like(p), logp) + entropy[:, None])
    grad.scatter_add_(1, targets.long().clamp(0, vocab - 1)[:, None], torch.where(empty, torch.zeros_like(g), g))
    return (grad / temperature).to(logits.dtype)


def _plain_newton_schulz(update):
    u = update.float()
    tall = u.shape[-2] > u.shape[-1]
    x = u.mT if tall else u
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + EPS)
    a, b, c = COEFFICIENTS
    for _ in range(STEPS):
        gram = torch.matmul(x, x.mT)
        x = a * x + torch.matmul(b * gram + c * torch.matmul(gram, gram), x)
    return x.mT.contiguous() if tall else x


def _plain_muon(s):
    g = s["main_grad"].float()
    momentum = s["beta"] * s["momentum"] + g
    update = g + s["beta"] * momentum if s["case"]["nesterov"] else momentum
    o = _plain_newton_schulz(update)
    weight = s["weight"].float() * (1 - s["lr"] * s["weight_decay"]) - (s["lr"] * s["scale"]) * o
    return {"weight": weight.to(s["weight"].dtype), "momentum": momentum}


# ---- one pass ----------------------------------------------------------------

def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import sparse_embedding_weight_amd as ewg

        if op == "logprobs":
            r = ewg.token_logprobs(state["logits"], state["targets"], top_k=case["top_k"], temperature=case["temperature"])
            out = {"logprobs": r.logprobs, "entropy": r.entropy, "logsumexp": r.logsumexp}
            if case["top_k"]:
                out.update(top_logprobs=r.top_logprobs, top_ids=r.top_ids)
            return out
        if op == "logprobs_grad":
            return ewg.token_logprobs_backward(state["logits"], state["targets"], state["logsumexp"], state["entropy"],
                                               state["grad_logprobs"], state["grad_entropy"],
                                               temperature=case["temperature"], out=state["out"])
        if op == "ortho":
            return ewg.orthogonalize_update(state["update"], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS)
        ewg.muon_step(state["weight"], state["main_grad"], state["momentum"], lr=state["lr"], beta=state["beta"],
                      nesterov=case["nesterov"], weight_decay=state["weight_decay"], scale=state["scale"], steps=STEPS,
                      coefficients=COEFFICIENTS, eps=EPS, out_weight=state["new_weight"],
                      out_momentum=state["new_momentum"])
        return {"weight": state["new_weight"], "momentum": state["new_momentum"]}
    if op == "logprobs":
        return _plain_logprobs(state["logits"], state["targets"], case["top_k"], case["temperature"])
    if op == "logprobs_grad":
        return _plain_logprobs_grad(state["logits"], state["targets"], state["logsumexp"], state["entropy"],
                                    state["grad_logprobs"], state["grad_entropy"], case["temperature"])
    if op == "ortho":
        return _plain_newton_schulz(state["update"]).to(torch.bfloat16)
    return _plain_muon(state)


# ---- what a pass cannot do without -------------------------------------------

def work(case):
    if case["op"] in ("logprobs", "logprobs_grad"):
        rows, cells = case["rows"], case["rows"] * case["vocab"]
        if case["op"] == "logprobs":
            # logits and targets in; three numbers and the alternatives out; scale, subtract, exp, two sums
            return {"bytes": cells * SIZE[case["dtype"]] + rows * (8 + 12 + 12 * case["top_k"]), "flops": 6 * cells}
        # logits in, gradient out; scale, subtract, exp, a linear factor
        return {"bytes": 2 * cells * SIZE[case["dtype"]] + rows * (8 + 12 + 4 * case["entropy"]), "flops": 6 * cells}
    k, long = min(case["m"], case["n"]), max(case["m"], case["n"])
    # a step: the Gram matrix and its square, half of each since both are symmetric, and one full product
    flops = case["batch"] * STEPS * (k * k * long + k * k * k + 2 * k * k * long)
    cells = case["batch"] * case["m"] * case["n"]
    if case["op"] == "ortho":
        return {"bytes": cells * (SIZE[case["dtype"]] + 2), "flops": flops}
    return {"bytes": cells * (SIZE[case["dtype"]] + 8 + 2 * SIZE[case["weight"]]), "flops": flops}


# ---- the definitions in 64 bits ----------------------------------------------

def _exact_rows(case, logits, targets):
    """Log probabilities by the definition, some rows at a time."""
    rows, vocab = logits.shape
    step = max(1, (1 << 27) // vocab)
    parts = []
    for r in range(0, rows, step):
        raw = logits[r:r + step].double()
        x = raw / case["temperature"]
        lse = torch.logsumexp(x, 1)
        logp = x - lse[:, None]
        entropy = -torch.xlogy(logp.exp(), logp.exp()).sum(1)
        t = targets[r:r + step].long()
        asked = logp.gather(1, t.clamp(min=0)[:, None])[:, 0].masked_fill(t < 0, 0.0)
        part = {"logprobs": asked, "entropy": entropy, "logsumexp": lse}
        if case["top_k"]:
            value, ids = torch.sort(raw, dim=1, descending=True, stable=True)
            value, ids = value[:, :case["top_k"]], ids[:, :case["top_k"]]
            part["top_logprobs"] = value / case["temperature"] - lse[:, None]
            part["top_ids"] = torch.where(value == -math.inf, torch.full_like(ids, -1), ids)
        parts.append(part)
    return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}


def _exact_polynomial(update):
    u = update.double()
    if u.shape[-2] > u.shape[-1]:
        return _exact_polynomial(update.transpose(-2, -1)).transpose(-2, -1).contiguous()
    x = u / (torch.linalg.matrix_norm(u)[..., None, None] + EPS)
    a, b, c = COEFFICIENTS
    for _ in range(STEPS):
        y = x @ x.transpose(-2, -1)
        x = a * x + b * (y @ x) + c * (y @ (y @ x))
    return x


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "logprobs":
        return _exact_rows(case, s["logits"], s["targets"])
    if op == "logprobs_grad":
        rows, vocab = s["logits"].shape
        step = max(1, (1 << 27) // vocab)
        parts = []
        for r in range(0, rows, step):
            cut = slice(r, r + step)
            logp = s["logits"][cut].double() / case["temperature"] - s["logsumexp"][cut].double()[:, None]
            t = s["targets"][cut].long()
            one = torch.zeros_like(logp)
            asked = t >= 0
            one[asked.nonzero()[:, 0], t[asked]] = 1.0
            g = s["grad_logprobs"][cut].double() * asked
            d = g[:, None] * (one - logp.exp())
            if case["entropy"]:
                d -= s["grad_entropy"][cut].double()[:, None] * logp.exp() * (logp + s["entropy"][cut].double()[:, None])
            parts.append(d / case["temperature"])
        return torch.cat(parts)
    if op == "ortho":
        return _exact_polynomial(s["update"])
    g = s["main_grad"].double()
    momentum = s["beta"] * s["momentum"].double() + g
    o = _exact_polynomial(g + s["beta"] * momentum if case["nesterov"] else momentum)
    weight = s["weight"].double() * (1 - s["lr"] * s["weight_decay"]) - s["lr"] * s["scale"] * o
    return {"weight": weight, "momentum": momentum}
