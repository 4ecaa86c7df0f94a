"""Measured cases of the 8-bit LM head and of the token log-probabilities.

Operators (``op`` of a case):
  quant     rows to 8-bit integers with one scale a row
  matmul    product of 8-bit token rows with 8-bit channel rows, scaled
  head      LM head over the active 8-bit rows of each sequence, with top-k
  logprobs  log-probabilities of given tokens, entropy, top alternatives
  grad      gradient of the log-probabilities, entropy and log-sum-exp

``run`` computes each in plain torch operations where ``own`` is false and
through the package's binding where it is true.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}
LARGEST = 4096 * 128256 * 4096          # products of the largest listed matmul
WHOLE = 4096 * 128256                   # elements of the largest listed logits


def _pitch(d):
    """Bytes of one 8-bit row: d rounded up to 128, the rest zero."""
    return -(-d // 128) * 128


def listed():
    return [
        # the hidden rows of one draft step, quantised before the product
        dict(name="quant_hidden", op="quant", rows=8, d=4096, ld=4096, dtype="bf16"),
        # a whole output matrix, quantised when the weights are loaded
        dict(name="quant_weights", op="quant", rows=128256, d=4096, ld=4096, dtype="bf16"),
        # a small head, where latency is all
        dict(name="matmul_tiny", op="matmul", m=4, n=2048, d=256, out="fp32"),
        # the full-vocabulary head for one step's hidden rows
        dict(name="matmul_step", op="matmul", m=8, n=128256, d=4096, out="fp32"),
        # the full-vocabulary head over a whole draft tree of 60 nodes
        dict(name="matmul_tree", op="matmul", m=60, n=151936, d=3584, out="bf16"),
        # the logits of every position of a prompt
        dict(name="matmul_prompt", op="matmul", m=4096, n=128256, d=4096, out="bf16"),
        # one sequence's draft head over about 1000 active rows
        dict(name="head_step", op="head", b=1, m=8, k=8, n_max=2048, live=1000, v=128256, d=4096, dtype="bf16", logits=False),
        # a long window, wide tree level
        dict(name="head_window", op="head", b=1, m=64, k=16, n_max=16384, live=15500, v=151936, d=4096, dtype="bf16", logits=False),
        # log-probabilities of a draft step's children under the target
        dict(name="logprobs_step", op="logprobs", rows=8, v=128256, ld=128256, dtype="fp32", tokens=8, k=8, temp=1.0, masked=0.0, empty=False),
        # log-probabilities of a prompt's own tokens
        dict(name="logprobs_prompt", op="logprobs", rows=4096, v=128256, ld=128256, dtype="bf16", tokens=1, k=4, temp=1.0, masked=0.0, empty=False),
        # one short training sequence over an odd vocabulary, part of it masked
        dict(name="grad_odd", op="grad", rows=129, v=50257, ld=50257, dtype="fp32", tokens=1, temp=0.7, masked=0.25, empty=True),
        # a training batch over the whole vocabulary
        dict(name="grad_batch", op="grad", rows=4096, v=128256, ld=128256, dtype="bf16", tokens=1, temp=1.0, masked=0.0, empty=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("quant", "matmul", "head", "logprobs", "grad"))
    dtype = rng.choice(("bf16", "fp16", "fp32"))
    if op == "quant":
        d = _log(rng, 1, 16384)
        rows = _log(rng, 1, max(1, min(131072, WHOLE // (2 * d))))
        return dict(op=op, rows=rows, d=d, ld=d + rng.choice((0, 0, 3, 64)), dtype=dtype)
    if op == "matmul":
        d = _log(rng, 16, 16384)
        m = _log(rng, 1, 4096)
        n = _log(rng, 1, max(1, min(152000, LARGEST // (2 * m * d), WHOLE // m)))
        return dict(op=op, m=m, n=n, d=d, out=dtype)
    if op == "head":
        d = 8 * _log(rng, 2, 1024)
        b = _log(rng, 1, 64)
        m = rng.randint(1, 64)
        n_max = _log(rng, 16, max(16, min(16384, (1 << 27) // (b * d))))
        logits = rng.random() < 0.3
        live = n_max if logits else rng.randint(1, n_max)
        v = _log(rng, max(n_max, 2048), 152000)
        return dict(op=op, b=b, m=m, k=rng.randint(1, 64), n_max=n_max, live=live, v=v, d=d, dtype=dtype, logits=logits)
    rows = _log(rng, 1, 4096)
    v = _log(rng, 64, max(64, min(152000, WHOLE // (2 * rows))))
    c = dict(op=op, rows=rows, v=v, ld=v + rng.choice((0, 0, 1, 24)), dtype=dtype, tokens=rng.randint(1, 8),
             temp=rng.choice((1.0, 1.0, 0.7, 1.5)), masked=rng.choice((0.0, 0.0, 0.5)), empty=rng.random() < 0.3)
    if op == "logprobs":
        c["k"] = rng.choice((0, 1, 4, 8, 20, 64))
    return c


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rows8(g, n, d):
    """n rows of d 8-bit values as a row-wise quantiser leaves them, padded with zeros to their pitch."""
    q = torch.zeros((n, _pitch(d)), dtype=torch.int8, device="cuda")
    q[:, :d] = torch.randn((n, d), generator=g, device="cuda", dtype=torch.bfloat16).mul_(32).round_().clamp_(-127, 127)
    return q


def _scales(g, n, size):
    return size * torch.exp(0.3 * torch.randn(n, generator=g, device="cuda"))


def prepare(case, seed):
    g = _generator(seed)
    s = {"case": case}
    op = case["op"]
    if op == "quant":
        x = torch.randn((case["rows"], case["ld"]), generator=g, device="cuda", dtype=torch.float32 if case["dtype"] == "fp32" else torch.bfloat16)
        s["x"] = x.to(DTYPES[case["dtype"]])
    elif op == "matmul":
        s["xq"], s["xs"] = _rows8(g, case["m"], case["d"]), _scales(g, case["m"], 0.03)
        s["wq"], s["ws"] = _rows8(g, case["n"], case["d"]), _scales(g, case["n"], 0.0006)
    elif op == "head":
        b, n_max, v = case["b"], case["n_max"], case["v"]
        s["wq"], s["ws"] = _rows8(g, v, case["d"]), _scales(g, v, 0.0006)
        s["h"] = torch.randn((b, case["m"], case["d"]), generator=g, device="cuda").to(DTYPES[case["dtype"]])
        ids = torch.rand((b, v), generator=g, device="cuda").argsort(1)[:, :n_max]
        # the active ids ascend; what lies behind the last one is no row
        live = torch.arange(n_max, device="cuda") < case["live"]
        ids = torch.where(live, ids, v).sort(1).values
        s["ids"] = torch.where(live, ids, -1).to(torch.int32).contiguous()
        s["n"] = torch.full((b,), case["live"], dtype=torch.int32, device="cuda")
    else:
        rows, v = case["rows"], case["v"]
        z = torch.randn((rows, case["ld"]), generator=g, device="cuda", dtype=torch.float32 if case["dtype"] == "fp32" else torch.bfloat16).mul_(3)
        tokens = torch.randint(0, v, (rows, case["tokens"]), generator=g, device="cuda")
        # the tokens that text goes on with are likely ones
        likely = 12 + 2 * torch.randn((rows, case["tokens"]), generator=g, device="cuda")
        z.scatter_reduce_(1, tokens, likely.to(z.dtype), "amax")
        if case["masked"]:
            banned = torch.rand((v,), generator=g, device="cuda") < case["masked"]
            banned[0] = False
            z[:, :v].masked_fill_(banned, -math.inf)
        if case["empty"]:
            # a row that a grammar leaves without any token
            z[rows // 2, :v] = -math.inf
        s["z"] = z.to(DTYPES[case["dtype"]])
        s["tokens"] = tokens.to(torch.int32)
        if op == "grad":
            s["g_logprob"] = torch.randn((rows, case["tokens"]), generator=g, device="cuda")
            s["g_entropy"] = 0.1 * torch.randn((rows,), generator=g, device="cuda")
            s["g_lse"] = 0.01 * torch.randn((rows,), generator=g, device="cuda")
            # what the forward pass left
            s["lse"], s["entropy"] = _statistics(s["z"][:, :v], 1.0 / case["temp"])
    return s


def _statistics(z, inv_temp):
    """Log-sum-exp and entropy of each row of scaled logits, in 32 bits."""
    z = z.float() * inv_temp
    top = z.max(1, keepdim=True).values
    z = z - torch.where(top == -math.inf, 0.0, top)
    e = torch.exp(z)
    total = e.sum(1)
    weighted = torch.where(e > 0, e * z, 0.0).sum(1)
    lse = torch.log(total) + top[:, 0]
    # a row without a finite logit has no probabilities: -inf and 0
    return lse, torch.where(total > 0, torch.log(total) - weighted / total, 0.0)


def _best(values, k):
    """The places of the k largest of each row, ties to the lowest place."""
    bits = (values + 0.0).view(torch.int32)
    order = bits ^ ((bits >> 31) & 0x7FFFFFFF)
    place = torch.arange(values.shape[-1], device=values.device)
    return torch.topk((order.long() << 32) + (0xFFFFFFFF - place), k, dim=-1).indices


def _quantised(x):
    """Rows to 8-bit integers; in 64 bits, for values next to a border between two integers."""
    x = x.double()
    top = x.abs().amax(-1, keepdim=True)
    q = torch.where(top > 0, torch.round(127 * x / torch.where(top > 0, top, 1.0)), 0.0)
    return q, (top[..., 0] / 127).float()


def _plain_quant(s):
    c = s["case"]
    q, scale = _quantised(s["x"][:, :c["d"]])
    return {"q": torch.nn.functional.pad(q.to(torch.int8), (0, _pitch(c["d"]) - c["d"])), "scale": scale}


def _plain_matmul(s):
    # sums of products of 8-bit integers pass 2^24: 64 bits hold them
    total = s["xq"].double() @ s["wq"].double().t()
    scale = s["xs"][:, None] * s["ws"]
    return {"out": (total.float() * scale).to(DTYPES[s["case"]["out"]])}


def _plain_head(s):
    c = s["case"]
    q, scale = _quantised(s["h"])
    at = s["ids"].long().clamp(min=0)
    rows = s["wq"][:, :c["d"]][at].double()
    total = (rows @ q.transpose(1, 2).contiguous()).transpose(1, 2)
    logits = total.float() * (scale[:, :, None] * s["ws"][at][:, None, :])
    live = torch.arange(c["n_max"], device="cuda") < s["n"][:, None]
    k = min(c["k"], c["n_max"])
    masked = torch.where(live[:, None, :], logits, -math.inf)
    best = _best(masked, k)
    values = masked.gather(2, best)
    ids = s["ids"][:, None, :].expand(-1, c["m"], -1).gather(2, best)
    pad = (0, c["k"] - k)
    r = {"ids": torch.nn.functional.pad(ids, pad, value=-1), "values": torch.nn.functional.pad(values, pad, value=-math.inf)}
    if c["logits"]:
        r["logits"] = logits
    return r


def _plain_logprobs(s):
    c = s["case"]
    z = s["z"][:, :c["v"]].float()
    inv_temp = 1.0 / c["temp"]
    lse, entropy = _statistics(z, inv_temp)
    shift = torch.where(lse == -math.inf, 0.0, lse)[:, None]
    r = {"logprob": z.gather(1, s["tokens"].long()) * inv_temp - shift, "lse": lse, "entropy": entropy}
    if c["k"]:
        best = _best(z, c["k"])
        r["top_ids"], r["top_logprobs"] = best.to(torch.int32), z.gather(1, best) * inv_temp - shift
    return r


def _plain_grad(s):
    c = s["case"]
    inv_temp = 1.0 / c["temp"]
    logp = s["z"][:, :c["v"]].float() * inv_temp - torch.where(s["lse"] == -math.inf, 0.0, s["lse"])[:, None]
    p = torch.exp(logp)
    inner = torch.where(p > 0, s["g_entropy"][:, None] * (logp + s["entropy"][:, None]), 0.0)
    dz = p * ((s["g_lse"] - s["g_logprob"].sum(1))[:, None] - inner)
    dz.scatter_add_(1, s["tokens"].long(), s["g_logprob"])
    dz = torch.where(s["lse"][:, None] == -math.inf, 0.0, dz)
    return {"dlogits": (dz * inv_temp).to(s["z"].dtype)}


def _own(s):
    from dynamic_vocab_draft_amd import nanospec as ns
    c = s["case"]
    op = c["op"]
    keep = s.setdefault("keep", {})
    new = not keep
    if op == "quant":
        if new:
            keep["q"] = torch.empty((c["rows"], _pitch(c["d"])), dtype=torch.int8, device="cuda")
            keep["scale"] = torch.empty((c["rows"],), dtype=torch.float32, device="cuda")
        ns.nanospec_quant_rows(s["x"][:, :c["d"]], keep["q"], keep["scale"])
        return {"q": keep["q"], "scale": keep["scale"]}
    if op == "matmul":
        if new:
            keep["out"] = torch.empty((c["m"], c["n"]), dtype=DTYPES[c["out"]], device="cuda")
        ns.nanospec_quant_matmul(s["xq"], s["xs"], s["wq"], s["ws"], c["d"], keep["out"])
        return {"out": keep["out"]}
    if op == "head":
        if new:
            keep["ids"] = torch.empty((c["b"], c["m"], c["k"]), dtype=torch.int32, device="cuda")
            keep["values"] = torch.empty((c["b"], c["m"], c["k"]), dtype=torch.float32, device="cuda")
            if c["logits"]:
                keep["logits"] = torch.empty((c["b"], c["m"], c["n_max"]), dtype=torch.float32, device="cuda")
            keep["work"] = ns.alloc_quant_logits_workspace(c["b"], c["n_max"], c["m"], c["k"], c["d"])
        ns.nanospec_quant_logits_topk(s["wq"], s["ws"], s["ids"], s["n"], s["h"], c["k"], keep.get("logits"), keep["ids"], keep["values"], keep["work"])
        return {key: keep[key] for key in ("ids", "values", "logits") if key in keep}
    rows, k, inv_temp = c["rows"], c.get("k", 0), 1.0 / c["temp"]
    z = s["z"][:, :c["v"]]
    if op == "logprobs":
        if new:
            keep["logprob"] = torch.empty((rows, c["tokens"]), dtype=torch.float32, device="cuda")
            keep["lse"] = torch.empty((rows,), dtype=torch.float32, device="cuda")
            keep["entropy"] = torch.empty((rows,), dtype=torch.float32, device="cuda")
            if k:
                keep["top_ids"] = torch.empty((rows, k), dtype=torch.int32, device="cuda")
                keep["top_logprobs"] = torch.empty((rows, k), dtype=torch.float32, device="cuda")
            keep["work"] = ns.alloc_token_logprobs_workspace(rows, c["v"], k)
        ns.nanospec_token_logprobs(z, inv_temp, s["tokens"], keep["logprob"], keep["lse"], keep["entropy"], keep.get("top_ids"), keep.get("top_logprobs"),
                                   keep["work"])
        return {key: t for key, t in keep.items() if key != "work"}
    if new:
        keep["dlogits"] = torch.empty((rows, c["v"]), dtype=z.dtype, device="cuda")
    ns.nanospec_token_logprobs_grad(z, inv_temp, s["tokens"], s["lse"], s["entropy"], s["g_logprob"], s["g_entropy"], s["g_lse"], keep["dlogits"])
    return {"dlogits": keep["dlogits"]}


def run(state):
    if own:
        return _own(state)
    return {"quant": _plain_quant, "matmul": _plain_matmul, "head": _plain_head, "logprobs": _plain_logprobs,
            "grad": _plain_grad}[state["case"]["op"]](state)


def work(case):
    op = case["op"]
    if op == "quant":
        n = case["rows"] * case["d"]
        return {"bytes": n * (SIZES[case["dtype"]] + 1) + 4 * case["rows"], "flops": 4 * n}
    if op == "matmul":
        m, n, d = case["m"], case["n"], case["d"]
        return {"bytes": (m + n) * (d + 4) + m * n * SIZES[case["out"]], "flops": 2 * m * n * d}
    if op == "head":
        b, m, n, d, v = case["b"], case["m"], case["live"], case["d"], case["v"]
        # rows that several sequences hold are read once
        rows = v * (1 - (1 - n / v) ** b)
        size = rows * (d + 4) + b * n * 4 + b * m * d * SIZES[case["dtype"]] + b * m * case["k"] * 8
        return {"bytes": int(size + (4 * b * m * n if case["logits"] else 0)), "flops": 2 * b * m * n * d}
    n = case["rows"] * case["v"]
    if op == "logprobs":
        return {"bytes": n * SIZES[case["dtype"]] + case["rows"] * (8 * case["tokens"] + 8 * case["k"] + 8), "flops": 5 * n}
    return {"bytes": 2 * n * SIZES[case["dtype"]] + case["rows"] * (8 * case["tokens"] + 16), "flops": 7 * n}


def exact(case, seed):
    """The operators' definitions in 64 bits: whole rows of real numbers, no shared statistics or rounding of the plain form."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        x = s["x"][:, :case["d"]].to(torch.float64)
        return {"q": None, "scale": x.abs().max(1).values / 127.0}
    if op == "matmul":
        a = s["xq"].to(torch.float64).mul_(s["xs"].to(torch.float64).unsqueeze(1))
        b = s["wq"].to(torch.float64).mul_(s["ws"].to(torch.float64).unsqueeze(1))
        return {"out": torch.mm(a, b.t())}
    if op == "head":
        if case["b"] * case["n_max"] * case["d"] > 1 << 28:
            return None
        h = s["h"].to(torch.float64)
        most = h.abs().max(2, keepdim=True).values
        # the quantised rows as real numbers: whole multiples of a 127th of the largest, halves to even
        h = torch.round(h * 127.0 / most) * most / 127.0
        values, whole = [], []
        for b in range(case["b"]):
            ids = s["ids"][b, :case["live"]].long()
            w = s["wq"][ids][:, :case["d"]].to(torch.float64) * s["ws"][ids].to(torch.float64).unsqueeze(1)
            z = torch.mm(h[b], w.t().contiguous())
            found = z.sort(1, descending=True).values[:, :case["k"]]
            rest = torch.full((case["m"], case["k"] - found.shape[1]), -math.inf, dtype=torch.float64, device="cuda")
            values.append(torch.cat([found, rest], 1))
            whole.append(z)
        r = {"ids": None, "values": torch.stack(values)}
        if case["logits"]:
            r["logits"] = torch.stack(whole)
        return r
    z = s["z"][:, :case["v"]].to(torch.float64) / case["temp"]
    tokens = s["tokens"].long()
    empty = (z == -math.inf).all(1, keepdim=True)
    if op == "logprobs":
        logp = torch.where(empty, -math.inf, torch.log_softmax(z, 1))
        r = {"logprob": logp.gather(1, tokens), "lse": torch.logsumexp(z, 1), "entropy": -torch.special.xlogy(logp.exp(), logp.exp()).sum(1)}
        if case["k"]:
            r["top_ids"], r["top_logprobs"] = None, torch.topk(logp, case["k"], 1).values
        return r
    # d(sum of g * output): the softmax's own gradient of each part
    p = torch.softmax(z, 1)
    logp = torch.where(p > 0, torch.log_softmax(z, 1), 0.0)
    entropy = -(p * logp).sum(1, keepdim=True)
    total = s["g_logprob"].double().sum(1, keepdim=True)
    d = -total * p - s["g_entropy"].double()[:, None] * p * (logp + entropy) + s["g_lse"].double()[:, None] * p
    d = d.scatter_add(1, tokens, s["g_logprob"].double())
    return {"dlogits": torch.where(empty, 0.0, d / case["temp"])}
