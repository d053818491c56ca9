"""The operators around the DBuffer step, as cases that can be measured.

A rank that trains with FP8 parameters gathers E4M3 codes and 128 x 128 tile
scales, runs its layers on them and hands bf16 gradients to the pack.  The cases
below are the operators of that path:

* embed / embed_grad: rows of the token table (bf16, or the gathered FP8 codes)
  times a factor, and the table's gradient, summed over equal tokens;
* norm / norm_grad: the residual's addition, root-mean-square norm and an E4M3
  output with one scale per 128 values of a row, and the gradients of both;
* linear / linear_dx / linear_dw: the product of such an output with an FP8
  weight as gathered, and its gradients to the input and to the weight.

`own` chooses between the plain form (elementary torch operations in 32 bits)
and the calls of block_quant_gb300.
"""

import math

import torch

own = False

EPS = 1e-5
GROUP = 128  # values of a row that share a scale; rows and columns of a weight's tile
TOP = 448.0  # largest finite E4M3 value


def listed():
    return [
        # one token looked up in the gathered FP8 table of a 2880-wide model: latency only
        dict(name="embed_token", op="embed", n=1, rows=201088, cols=2880, table="fp8", ids=32),
        # one rank's tokens of a training step, bf16 table of a 128256-word vocabulary
        dict(name="embed_batch", op="embed", n=8192, rows=128256, cols=4096, table="bf16", ids=64),
        # that step's table gradient, written whole for the pack
        dict(name="embed_grad_batch", op="embed_grad", n=8192, rows=128256, cols=4096, out="bf16", ids=64),
        # a short micro-batch on an odd-sized table, gradient kept in fp32
        dict(name="embed_grad_ragged", op="embed_grad", n=1025, rows=50001, cols=2880, out="fp32", ids=32),
        # one generated token, 8192-wide residual stream: latency only
        dict(name="norm_token", op="norm", n=1, cols=8192, residual=True),
        # the norm before a layer's projections in training
        dict(name="norm_batch", op="norm", n=8192, cols=4096, residual=True),
        # its backward pass, ragged token count, wider stream
        dict(name="norm_grad_ragged", op="norm_grad", n=4099, cols=8192, residual=True),
        # one generated token through an 8192 x 8192 projection: the weight's bytes
        dict(name="linear_token", op="linear", n=1, rows=8192, cols=8192),
        # a short prompt through the narrow projection of a 2880-wide model
        dict(name="linear_ragged", op="linear", n=333, rows=2880, cols=4096),
        # the widest projection of a 4096-wide layer in training
        dict(name="linear_batch", op="linear", n=8192, rows=14336, cols=4096),
        # its gradients to the input and to the weight
        dict(name="linear_dx_batch", op="linear_dx", n=8192, rows=14336, cols=4096),
        dict(name="linear_dw_batch", op="linear_dw", n=8192, rows=14336, cols=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "norm", "norm_grad", "linear", "linear_dx", "linear_dw"])
    n = _log(rng, 1, 8192)
    if op in ("embed", "embed_grad"):
        cols = 8 * _log(rng, 16, 512)
        case = dict(op=op, n=n, rows=_log(rng, 1000, 128256), cols=cols, ids=rng.choice([32, 64]))
        if op == "embed":
            case["table"] = rng.choice(["bf16", "fp8"])
        else:
            case["out"] = rng.choice(["bf16", "fp32"])
        return case
    if op in ("norm", "norm_grad"):
        # widths of ordinary models, and now and then one that no vector of 8 divides
        cols = 8 * _log(rng, 16, 1024) if rng.random() < 0.75 else _log(rng, 128, 8192)
        return dict(op=op, n=n, cols=cols, residual=rng.random() < 0.75)
    rows, cols = _log(rng, 256, 14336), 16 * _log(rng, 16, 896)
    while n * rows * cols > 8192 * 14336 * 4096:
        n = max(1, n // 2)
    return dict(op=op, n=n, rows=rows, cols=cols)


def work(case):
    n, c = case["n"], case["cols"]
    g = -(-c // GROUP)
    op = case["op"]
    if op == "embed":
        return {"bytes": n * (c * (1 if case["table"] == "fp8" else 2) + 2 * c + case["ids"] // 8), "flops": n * c}
    if op == "embed_grad":
        out = case["rows"] * c * (2 if case["out"] == "bf16" else 4)
        return {"bytes": n * (2 * c + case["ids"] // 8) + out, "flops": n * c}
    if op == "norm":
        return {"bytes": n * (c * (7 if case["residual"] else 3) + 4 * g + 4) + 2 * c, "flops": 8 * n * c}
    if op == "norm_grad":
        return {"bytes": n * (c * (8 if case["residual"] else 6) + 4) + 6 * c, "flops": 10 * n * c}
    r = case["rows"]
    tiles = g * -(-r // GROUP)
    flops = 2 * n * r * c
    if op == "linear":
        return {"bytes": n * (c + 4 * g) + r * c + 4 * tiles + 2 * n * r, "flops": flops}
    if op == "linear_dx":
        return {"bytes": 2 * n * r + r * c + 4 * tiles + 2 * n * c, "flops": flops}
    return {"bytes": 2 * n * r + n * (c + 4 * g) + 2 * r * c, "flops": flops}


# ----------------------------------------------------------------------------- inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _stream_rows(gen, n, c):
    """Rows of a residual stream: a magnitude per token and a few loud channels."""
    x = _randn(gen, n, c) * torch.exp(0.5 * _randn(gen, n, 1))
    loud = (torch.rand(c, generator=gen, device="cuda") < 0.01).float() * 15 + 1
    return (x * loud).bfloat16()


def _tokens(gen, n, rows, bits):
    """Token ids with a count inversely proportional to their rank, 2% padding (-1)."""
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    rank = torch.exp(u * math.log(rows + 1)).long().clamp(1, rows) - 1
    ids = (rank * 7919 + 13) % rows
    ids = torch.where(torch.rand(n, generator=gen, device="cuda") < 0.02, torch.full_like(ids, -1), ids)
    return ids if bits == 64 else ids.int()


def _to_codes(x, amax):
    """E4M3 codes and scale of values that share the maximum `amax`."""
    scale = amax / TOP
    back = TOP / amax
    y = torch.where(torch.isinf(back), x / scale, x * back)
    y = torch.where(scale > 0, y, torch.zeros_like(x))
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


def prepare(case, seed):
    gen = _gen(seed)
    op, n, c = case["op"], case["n"], case["cols"]
    g = -(-c // GROUP)
    s = {"case": dict(case)}
    if op == "embed":
        if case["table"] == "fp8":
            s["table"], s["table_scale"] = _weight(gen, case["rows"], c)
        else:
            s["table"] = (_randn(gen, case["rows"], c) * 0.02).bfloat16()
        s["ids"] = _tokens(gen, n, case["rows"], case["ids"])
        s["factor"] = float(math.sqrt(c))
        s["out"] = torch.empty(n, c, device="cuda", dtype=torch.bfloat16)
    elif op == "embed_grad":
        s["dy"] = (_randn(gen, n, c) * 1e-3).bfloat16()
        s["ids"] = _tokens(gen, n, case["rows"], case["ids"])
        s["factor"] = float(math.sqrt(c))
        s["out"] = torch.empty(case["rows"], c, device="cuda", dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32)
    elif op in ("norm", "norm_grad"):
        s["x"] = _stream_rows(gen, n, c)
        s["weight"] = (1 + 0.1 * _randn(gen, c)).bfloat16()
        if op == "norm":
            s["residual"] = _stream_rows(gen, n, c) if case["residual"] else None
            s["h"] = torch.empty_like(s["x"])
            s["codes"] = torch.empty(n, c, device="cuda", dtype=torch.float8_e4m3fn)
            s["code_scale"] = torch.empty(g, n, device="cuda", dtype=torch.float32)
            s["rstd"] = torch.empty(n, device="cuda", dtype=torch.float32)
        else:
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(-1) + EPS)
            s["dy"] = (_randn(gen, n, c) * 1e-3).bfloat16()
            s["dh"] = (_randn(gen, n, c) * 1e-3).bfloat16() if case["residual"] else None
            s["dx"] = torch.empty_like(s["x"])
            s["dw"] = torch.empty(c, device="cuda", dtype=torch.float32)
    else:
        r = case["rows"]
        if op != "linear_dw":
            s["w"], s["w_scale"] = _weight(gen, r, c)
        if op != "linear_dx":
            s["codes"], s["code_scale"] = _quant_rows(_stream_rows(gen, n, c).float())
        if op != "linear":
            s["dy"] = (_randn(gen, n, r) * 1e-3 * torch.exp(_randn(gen, n, 1))).bfloat16()
        shape = {"linear": (n, r), "linear_dx": (n, c), "linear_dw": (r, c)}[op]
        s["out"] = torch.empty(*shape, device="cuda", dtype=torch.bfloat16)
    return s


# ----------------------------------------------------------------------------- one pass


def run(s):
    return _own_pass(s) if own else _plain_pass(s)


def _workspace(s, size):
    if "ws" not in s:
        s["ws"] = torch.zeros(size, device="cuda", dtype=torch.uint8)
    return s["ws"]


def _own_pass(s):
    import block_quant_gb300 as bq

    case = s["case"]
    op = case["op"]
    if op == "embed":
        bq.embed(s["table"], s["ids"], s["out"], scale=s["factor"], table_scale=s.get("table_scale"))
        return s["out"]
    if op == "embed_grad":
        ws = s.get("ws")
        if ws is None:
            ws = _workspace(s, bq.embed_grad_workspace(case["n"], case["rows"], case["cols"]))
        bq.embed_grad(s["dy"], s["ids"], s["out"], ws, scale=s["factor"])
        return s["out"]
    if op == "norm":
        bq.rmsnorm(s["x"], s["weight"], EPS, residual=s["residual"], h=s["h"] if case["residual"] else None,
                   codes=s["codes"], code_scale=s["code_scale"], rstd=s["rstd"])
        got = {"codes": s["codes"], "scale": s["code_scale"], "rstd": s["rstd"]}
        if case["residual"]:
            got["h"] = s["h"]
        return got
    if op == "norm_grad":
        ws = s.get("ws")
        if ws is None:
            ws = _workspace(s, bq.rmsnorm_grad_workspace(case["n"], case["cols"]))
        bq.rmsnorm_grad(s["dy"], s["x"], s["weight"], s["rstd"], s["dx"], s["dw"], ws, dh=s["dh"])
        return {"dx": s["dx"], "dw": s["dw"]}
    ws = s.get("ws")
    if ws is None:
        ws = _workspace(s, bq.linear_fp8_workspace(case["n"], case["rows"], case["cols"]))
    if op == "linear":
        bq.linear_fp8(s["codes"], s["code_scale"], s["w"], s["w_scale"], s["out"], ws)
    elif op == "linear_dx":
        bq.linear_fp8_dx(s["dy"], s["w"], s["w_scale"], s["out"], ws)
    else:
        bq.linear_fp8_dw(s["dy"], s["codes"], s["code_scale"], s["out"], ws)
    return s["out"]


def _spread_rows(scale, c):
    """Scales [groups, n] -> [n, c], one for each value."""
    return scale.t().repeat_interleave(GROUP, 1)[:, :c]


def _spread_tiles(scale, rows, cols):
    return scale.repeat_interleave(GROUP, 0).repeat_interleave(GROUP, 1)[:rows, :cols]


def _plain_pass(s):
    case = s["case"]
    op, c = case["op"], case["cols"]
    if op == "embed":
        ids = s["ids"].long()
        seen = (ids >= 0) & (ids < case["rows"])
        at = torch.where(seen, ids, torch.zeros_like(ids))
        y = s["table"][at].float()
        if case["table"] == "fp8":
            y = y * s["table_scale"][at // GROUP].repeat_interleave(GROUP, 1)[:, :c]
        return (y * s["factor"] * seen[:, None]).bfloat16()
    if op == "embed_grad":
        ids = s["ids"].long()
        seen = (ids >= 0) & (ids < case["rows"])
        at = torch.where(seen, ids, torch.zeros_like(ids))
        total = torch.zeros(case["rows"], c, device="cuda", dtype=torch.float32)
        total.index_add_(0, at, s["dy"].float() * seen[:, None])
        return (total * s["factor"]).to(s["out"].dtype)
    if op == "norm":
        h = s["x"]
        if case["residual"]:
            h = (h.float() + s["residual"].float()).bfloat16()
        f = h.float()
        rstd = torch.rsqrt(f.square().mean(-1) + EPS)
        codes, scale = _quant_rows(f * rstd[:, None] * s["weight"].float())
        got = {"codes": codes, "scale": scale, "rstd": rstd}
        if case["residual"]:
            got["h"] = h
        return got
    if op == "norm_grad":
        f, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
        unit = f * rstd
        t = dy * s["weight"].float()
        dx = rstd * (t - unit * (t * unit).mean(-1, keepdim=True))
        if case["residual"]:
            dx = dx + s["dh"].float()
        return {"dx": dx.bfloat16(), "dw": (dy * unit).sum(0)}
    if op == "linear":
        x = s["codes"].float() * _spread_rows(s["code_scale"], c)
        w = s["w"].float() * _spread_tiles(s["w_scale"], case["rows"], c)
        return (x @ w.t()).bfloat16()
    if op == "linear_dx":
        codes, scale = _quant_rows(s["dy"].float())
        dy = codes.float() * _spread_rows(scale, case["rows"])
        w = s["w"].float() * _spread_tiles(s["w_scale"], case["rows"], c)
        return (dy @ w).bfloat16()
    x = s["codes"].float() * _spread_rows(s["code_scale"], c)
    return (s["dy"].float().t() @ x).bfloat16()


# ----------------------------------------------------------------------------- the definition in 64 bits


def _e4m3_64(v):
    """The E4M3 value nearest to each fp64 value (ties to the even mantissa, +-448 at most)."""
    _, e = torch.frexp(v.abs().clamp(min=2.0 ** -20))
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-TOP, TOP)


def _blocks_64(v, amax):
    scale = amax / TOP
    return _e4m3_64(torch.where(scale > 0, v / torch.where(scale > 0, scale, torch.ones_like(scale)), torch.zeros_like(v))), scale


def _rows_64(v):
    n, c = v.shape
    codes, scales = torch.empty_like(v), []
    for j in range(0, c, GROUP):
        part = v[:, j:j + GROUP]
        codes[:, j:j + GROUP], scale = _blocks_64(part, part.abs().max(1, keepdim=True).values)
        scales.append(scale[:, 0])
    return codes, torch.stack(scales)


def _times_rows_64(codes, scale):
    v = codes.double()
    for j in range(scale.shape[0]):
        v[:, j * GROUP:(j + 1) * GROUP] *= scale[j].double()[:, None]
    return v


def _times_tiles_64(codes, scale):
    v = codes.double()
    for i in range(scale.shape[0]):
        band = v[i * GROUP:(i + 1) * GROUP]
        for j in range(scale.shape[1]):
            band[:, j * GROUP:(j + 1) * GROUP] *= float(scale[i, j])
    return v


def exact(case, seed):
    s = prepare(case, seed)
    op, c = case["op"], case["cols"]
    if op in ("embed", "embed_grad"):
        ids = s["ids"].long()
        seen = torch.nonzero((ids >= 0) & (ids < case["rows"]))[:, 0]
        at = ids[seen]
        if op == "embed":
            out = torch.zeros(case["n"], c, device="cuda", dtype=torch.float64)
            rows = s["table"][at].double()
            if case["table"] == "fp8":
                tile = torch.arange(c, device="cuda") // GROUP
                rows = rows * s["table_scale"].double()[at // GROUP][:, tile]
            out[seen] = rows * s["factor"]
            return out
        out = torch.zeros(case["rows"], c, device="cuda", dtype=torch.float64)
        return out.index_put_((at,), s["dy"][seen].double() * s["factor"], accumulate=True)
    if op == "norm":
        h = s["x"].double()
        if case["residual"]:
            h = (h + s["residual"].double()).bfloat16().double()
        rstd = 1 / torch.sqrt((h * h).sum(1) / c + EPS)
        codes, scale = _rows_64(h * rstd[:, None] * s["weight"].double())
        got = {"codes": codes, "scale": scale, "rstd": rstd}
        if case["residual"]:
            got["h"] = h
        return got
    if op == "norm_grad":
        h, dy, w, r = s["x"].double(), s["dy"].double(), s["weight"].double(), s["rstd"].double()[:, None]
        dot = (dy * w * h).sum(1, keepdim=True)
        dx = r * dy * w - r ** 3 * h * dot / c
        if case["residual"]:
            dx = dx + s["dh"].double()
        return {"dx": dx, "dw": (dy * h * r).sum(0)}
    if op == "linear":
        return _times_rows_64(s["codes"], s["code_scale"]) @ _times_tiles_64(s["w"], s["w_scale"]).t()
    if op == "linear_dx":
        codes, scale = _rows_64(s["dy"].double())
        return _times_rows_64(codes, scale) @ _times_tiles_64(s["w"], s["w_scale"])
    return s["dy"].double().t() @ _times_rows_64(s["codes"], s["code_scale"])
