"""The end of a language model on FP8 rows and a gathered FP8 head, as cases that can be measured.

A rank that trains with FP8 parameters multiplies its last norm's FP8 rows with the
vocabulary's weight, and takes the loss of the logits.  The cases are the loss and
its gradients, without the logits ever being kept:

* ce / ce_grad: softmax cross entropy of each token's target (a target outside the
  vocabulary, as padding has, counts nothing), and the gradients of the rows and of
  the weight;
* distill / distill_grad: the divergence from a teacher of which each token's top
  logits are known, and its gradients.

`own` chooses between the plain form (elementary torch operations in 32 bits) and
the calls of block_quant_gb300.
"""

import math

import torch

own = False

GROUP = 128  # values of a row that share a scale; rows and columns of a weight's tile
TOP = 448.0  # largest finite E4M3 value
MOST = 8192 * 128256 * 4096  # products of the largest forward case; a gradient's has half


def listed():
    return [
        # a toy vocabulary, one token scored: latency only
        dict(name="ce_toy", op="ce", n=1, rows=1000, cols=512, ids=64, scale=1.0),
        # one token of a generated text scored against a full vocabulary: the weight's bytes
        dict(name="ce_token", op="ce", n=1, rows=128256, cols=4096, ids=64, scale=1.0),
        # perplexity of a short prompt, 2880-wide model, odd vocabulary
        dict(name="ce_ragged", op="ce", n=333, rows=50001, cols=2880, ids=32, scale=1.0),
        # the loss of one rank's tokens of a training step
        dict(name="ce_batch", op="ce", n=8192, rows=128256, cols=4096, ids=64, scale=1.0),
        # the gradients of the example's small model
        dict(name="ce_grad_small", op="ce_grad", n=2048, rows=1000, cols=512, ids=64, scale=1.0),
        # a few tokens fine-tuned: the weight's gradient is written whole for the pack
        dict(name="ce_grad_few", op="ce_grad", n=16, rows=128256, cols=4096, ids=64, scale=1.0),
        # a ragged micro-batch of a 2880-wide model
        dict(name="ce_grad_ragged", op="ce_grad", n=1025, rows=50001, cols=2880, ids=32, scale=1.0),
        # a micro-batch of a training step
        dict(name="ce_grad_batch", op="ce_grad", n=4096, rows=128256, cols=4096, ids=64, scale=1.0),
        # a few tokens distilled at temperature 2 from eight stored logits each
        dict(name="distill_few", op="distill", n=17, rows=32001, cols=2048, ids=32, scale=0.5, k=8, teacher="fp32"),
        # a micro-batch with 64 stored logits a token
        dict(name="distill_batch", op="distill", n=4096, rows=128256, cols=4096, ids=32, scale=1.0, k=64, teacher="bf16"),
        # gradients of a ragged one, 201088-word vocabulary
        dict(name="distill_grad_ragged", op="distill_grad", n=777, rows=201088, cols=2880, ids=64, scale=0.5, k=32,
             teacher="fp32"),
        # gradients of a whole one
        dict(name="distill_grad_batch", op="distill_grad", n=2048, rows=128256, cols=4096, ids=32, scale=1.0, k=64,
             teacher="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ce", "ce_grad", "distill", "distill_grad"])
    n, rows, cols = _log(rng, 1, 8192), _log(rng, 500, 201088), 16 * _log(rng, 8, 512)
    while n * rows * cols > MOST // (2 if op.endswith("grad") else 1):
        n = max(1, n // 2)
    case = dict(op=op, n=n, rows=rows, cols=cols, ids=rng.choice([32, 64]), scale=rng.choice([1.0, 1.0, 0.5]))
    if op.startswith("distill"):
        case["k"], case["teacher"] = _log(rng, 1, 128), rng.choice(["bf16", "fp32"])
    return case


def work(case):
    n, r, c = case["n"], case["rows"], case["cols"]
    g = -(-c // GROUP)
    read = n * (c + 4 * g) + r * c + 4 * g * -(-r // GROUP)
    if case["op"].startswith("distill"):
        pairs = n * case["k"]
        read += pairs * (case["ids"] // 8 + (2 if case["teacher"] == "bf16" else 4))
        both = 8 * n + 4 * pairs  # loss, lse and the student's log-probabilities
    else:
        read += n * case["ids"] // 8
        both = 8 * n
    if case["op"].endswith("grad"):
        # the logits again, and the products with the weight and with the rows
        return {"bytes": read + both + 4 * n + 2 * n * c + 2 * r * c, "flops": 6 * n * r * c}
    return {"bytes": read + both, "flops": 2 * n * r * c}


# ----------------------------------------------------------------------------- inputs


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _rand(gen, *shape):
    return torch.rand(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _to_codes(x, amax):
    """E4M3 codes and scale of values that share the maximum `amax`."""
    scale = amax / TOP
    y = torch.where(scale > 0, x * (TOP / amax), torch.zeros_like(x))
    return y.to(torch.float8_e4m3fn), scale


def _quant_rows(x):
    """fp32 [n, c] -> codes [n, c], scales [groups, n] (one per 128 values of a row)."""
    n, c = x.shape
    g = -(-c // GROUP)
    p = torch.nn.functional.pad(x, (0, g * GROUP - c)).view(n, g, GROUP)
    codes, scale = _to_codes(p, p.abs().amax(-1, keepdim=True))
    return codes.view(n, g * GROUP)[:, :c].contiguous(), scale.view(n, g).t().contiguous()


def _weight(gen, rows, cols):
    """FP8 weight as the optimizer step leaves it: codes [rows, cols], scales of its 128 x 128 tiles."""
    a, b = -(-rows // GROUP), -(-cols // GROUP)
    w = _randn(gen, rows, cols) * (0.02 * torch.exp(0.3 * _randn(gen, 1, cols)))
    p = torch.nn.functional.pad(w, (0, b * GROUP - cols, 0, a * GROUP - rows)).view(a, GROUP, b, GROUP)
    codes, scale = _to_codes(p, p.abs().amax(dim=(1, 3), keepdim=True))
    return codes.view(a * GROUP, b * GROUP)[:rows, :cols].contiguous(), scale.view(a, b).contiguous()


def _words(gen, n, rows):
    """Token ids with a count inversely proportional to their rank."""
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    rank = torch.exp(u * math.log(rows + 1)).long().clamp(1, rows) - 1
    return (rank * 7919 + 13) % rows


def _rows_towards(gen, words, w, w_scale):
    """FP8 rows of a last norm: noise, and as much of each word's own direction as a model has
    learned (none of it for some tokens, nearly all for others)."""
    n, c = words.shape[0], w.shape[1]
    tile = torch.arange(c, device="cuda") // GROUP
    to = w[words].float() * w_scale[words // GROUP][:, tile]
    to = to * torch.rsqrt(to.square().mean(1, keepdim=True) + 1e-20)
    x = _randn(gen, n, c) + 20 * c ** -0.5 * _rand(gen, n, 1) * to
    loud = (torch.rand(c, generator=gen, device="cuda") < 0.01).float() * 3 + 1
    return _quant_rows(x * torch.rsqrt(x.square().mean(1, keepdim=True)) * loud)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    n, r, c = case["n"], case["rows"], case["cols"]
    kind = torch.int64 if case["ids"] == 64 else torch.int32
    s = {"case": dict(case)}
    s["w"], s["w_scale"] = _weight(gen, r, c)
    words = _words(gen, n, r)
    s["codes"], s["code_scale"] = _rows_towards(gen, words, s["w"], s["w_scale"])
    padding = _rand(gen, n) < (0.03 if n > 1 else 0.0)
    f32 = dict(device="cuda", dtype=torch.float32)
    if case["op"].startswith("ce"):
        s["targets"] = torch.where(padding, torch.full_like(words, -100), words).to(kind)
        s["loss"], s["lse"] = torch.empty(n, **f32), torch.empty(n, **f32)
    else:
        # the word the student leans to and k - 1 others (each once), falling logits; padding tokens
        # know none, and some tokens fewer than k
        k = case["k"]
        step = 1 + (_rand(gen, n, 1) * max(1, (r - 1) // k)).long().clamp(max=max(0, (r - 1) // k - 1))
        ids = (words[:, None] + torch.arange(k, device="cuda") * step) % r
        known = k - (_rand(gen, n, 1) * k * 0.5).long() * (_rand(gen, n, 1) < 0.1).long()
        gone = padding[:, None] | (torch.arange(k, device="cuda") >= known)
        s["ids"] = torch.where(gone, torch.full_like(ids, -1), ids).to(kind).contiguous()
        fall = -torch.cumsum(-torch.log(1 - _rand(gen, n, k) * 0.999), 1) * (4.0 / math.sqrt(k))
        s["teacher"] = (18 + 2 * _randn(gen, n, 1) + fall).to(torch.bfloat16 if case["teacher"] == "bf16" else torch.float32)
        s["loss"], s["lse"], s["logp"] = torch.empty(n, **f32), torch.empty(n, **f32), torch.empty(n, k, **f32)
    if case["op"].endswith("grad"):
        # what the forward pass has left
        for name, value in _plain_forward(s).items():
            s[name] = value
        s["dloss"] = (0.5 + _rand(gen, n)) / n
        s["dx"] = torch.empty(n, c, device="cuda", dtype=torch.bfloat16)
        s["dw"] = torch.empty(r, c, device="cuda", dtype=torch.bfloat16)
    return s


# ----------------------------------------------------------------------------- one pass


def run(s):
    return _own_pass(s) if own else _plain_pass(s)


def _own_pass(s):
    import block_quant_gb300 as bq

    case = s["case"]
    op, scale = case["op"], case["scale"]
    ws = s.get("ws")
    if ws is None:
        size = bq.loss_fp8_grad_workspace if op.endswith("grad") else bq.loss_fp8_workspace
        ws = s["ws"] = torch.zeros(size(case["n"], case["rows"], case["cols"]), device="cuda", dtype=torch.uint8)
    head = s["codes"], s["code_scale"], s["w"], s["w_scale"]
    if op == "ce":
        bq.cross_entropy_fp8(*head, s["targets"], s["loss"], s["lse"], ws, scale=scale)
        return {"loss": s["loss"], "lse": s["lse"]}
    if op == "distill":
        bq.distill_fp8(*head, s["ids"], s["teacher"], s["loss"], s["lse"], s["logp"], ws, scale=scale)
        return {"loss": s["loss"], "lse": s["lse"], "logp": s["logp"]}
    if op == "ce_grad":
        bq.cross_entropy_fp8_grad(*head, s["targets"], s["loss"], s["lse"], s["dloss"], s["dx"], s["dw"], ws, scale=scale)
    else:
        bq.distill_fp8_grad(*head, s["ids"], s["teacher"], s["lse"], s["logp"], s["dloss"], s["dx"], s["dw"], ws,
                            scale=scale)
    return {"dx": s["dx"], "dw": s["dw"]}


def _plain_head(s):
    """The rows and the weight in fp32."""
    r, c = s["w"].shape
    x = s["codes"].float() * s["code_scale"].t().repeat_interleave(GROUP, 1)[:, :c]
    w = s["w"].float() * s["w_scale"].repeat_interleave(GROUP, 0).repeat_interleave(GROUP, 1)[:r, :c]
    return x, w


def _teacher(s):
    """(which pairs count, their ids with 0 for the others, the teacher's probabilities with 0 for them)."""
    r, ids = s["case"]["rows"], s["ids"].long()
    z = s["teacher"].float() * s["case"]["scale"]
    kept = (ids >= 0) & (ids < r) & (z != -math.inf)
    z = torch.where(kept, z, torch.full_like(z, -math.inf))
    top = z.amax(1, keepdim=True)
    e = torch.where(kept, torch.exp(z - torch.where(torch.isfinite(top), top, torch.zeros_like(top))), torch.zeros_like(z))
    total = e.sum(1, keepdim=True)
    return kept, torch.where(kept, ids, torch.zeros_like(ids)), e / torch.where(total > 0, total, torch.ones_like(total))


def _plain_forward(s):
    case = s["case"]
    x, w = _plain_head(s)
    z = x @ w.t()
    if case["scale"] != 1.0:
        z = z * case["scale"]
    # the largest logit stays out of the sum: a sure prediction's loss is log(1 + the others'
    # sum), which 32 bits hold however small it is
    top, best = z.max(1, keepdim=True)
    if case["op"].startswith("ce"):
        y = s["targets"].long()
        kept = ((y >= 0) & (y < case["rows"]))[:, None]
        at = torch.where(kept[:, 0], y, torch.zeros_like(y))[:, None]
    else:
        kept, at, q = _teacher(s)
    behind = z.gather(1, at) - top
    more = torch.log1p(z.sub_(top).exp_().scatter_(1, best, 0.0).sum(1, keepdim=True))
    logp = torch.where(kept, behind - more, torch.zeros_like(behind))
    lse = (top + more)[:, 0]
    if case["op"].startswith("ce"):
        return {"loss": -logp[:, 0], "lse": lse}
    terms = q * (torch.log(torch.where(q > 0, q, torch.ones_like(q))) - logp)
    return {"loss": terms.sum(1), "lse": lse, "logp": logp}


def _plain_pass(s):
    case = s["case"]
    if not case["op"].endswith("grad"):
        return _plain_forward(s)
    x, w = _plain_head(s)
    z = x @ w.t()
    if case["scale"] != 1.0:
        z = z * case["scale"]
    p = z.sub_(s["lse"][:, None]).exp_()
    # where the target has weight, p - weight by the forward pass's own log-probability
    if case["op"] == "ce_grad":
        y = s["targets"].long()
        seen = (y >= 0) & (y < case["rows"])
        at, less = torch.where(seen, y, torch.zeros_like(y))[:, None], torch.expm1(-s["loss"])[:, None]
    else:
        kept, at, q = _teacher(s)
        seen = kept.any(1)
        same = ((at[:, :, None] == at[:, None, :]) & kept[:, None, :]).float()
        less = torch.expm1(s["logp"]) + (1 - (same * q[:, None, :]).sum(2))
        first = kept.float().argmax(1, keepdim=True)  # pairs that do not count repeat one that does
        at, less = torch.where(kept, at, at.gather(1, first)), torch.where(kept, less, less.gather(1, first))
    p.scatter_(1, at, less)
    p *= (s["dloss"] * case["scale"])[:, None]
    p = torch.where(seen[:, None], p, torch.zeros_like(p))
    return {"dx": (p @ w).bfloat16(), "dw": (p.t() @ x).bfloat16()}


# ----------------------------------------------------------------------------- the definition in 64 bits


def _head_64(s):
    x, w = s["codes"].double(), s["w"].double()
    for j in range(s["code_scale"].shape[0]):
        x[:, j * GROUP:(j + 1) * GROUP] *= s["code_scale"][j].double()[:, None]
    rows = torch.arange(w.shape[0], device="cuda") // GROUP
    for j in range(s["w_scale"].shape[1]):
        w[:, j * GROUP:(j + 1) * GROUP] *= s["w_scale"].double()[rows, j][:, None]
    return x, w


def exact(case, seed):
    s = prepare(case, seed)
    n, r, f = case["n"], case["rows"], case["scale"]
    grad, many = case["op"].endswith("grad"), case["op"].startswith("distill")
    x, w = _head_64(s)
    rows = {}
    dw = torch.zeros(r, case["cols"], device="cuda", dtype=torch.float64) if grad else None
    for t0 in range(0, n, 1024):
        part = slice(t0, min(n, t0 + 1024))
        z = f * (x[part] @ w.t())
        if many:
            ids, logits = s["ids"][part].long(), f * s["teacher"][part].double()
            kept = (ids >= 0) & (ids < r) & ~torch.isneginf(logits)
            q = torch.softmax(logits.masked_fill(~kept, -math.inf), 1).masked_fill(~kept, 0.0)
        else:
            ids = s["targets"][part].long()[:, None]
            kept = (ids >= 0) & (ids < r)
            q = kept.double()
        some, at = kept.any(1), ids.clamp(0, r - 1)
        if grad:
            u = torch.exp(z - s["lse"][part].double()[:, None])
            known = s["logp"][part].double() if many else -s["loss"][part].double()[:, None]
            i, j = torch.nonzero(kept, as_tuple=True)
            u[i, at[i, j]] = torch.exp(known[i, j])
            u.index_put_((i, at[i, j]), -q[i, j], accumulate=True)
            u = (u * (f * s["dloss"][part].double())[:, None]).masked_fill(~some[:, None], 0.0)
            rows.setdefault("dx", []).append(u @ w)
            dw += u.t() @ x[part]
            continue
        lse = torch.logsumexp(z, 1)
        logp = (z.gather(1, at) - lse[:, None]).masked_fill(~kept, 0.0)
        rows.setdefault("lse", []).append(lse)
        if many:
            rows.setdefault("logp", []).append(logp)
            rows.setdefault("loss", []).append((torch.xlogy(q, q) - q * logp).sum(1))
        else:
            rows.setdefault("loss", []).append(-logp[:, 0])
    got = {name: torch.cat(v) for name, v in rows.items()}
    if grad:
        got["dw"] = dw
    return got
