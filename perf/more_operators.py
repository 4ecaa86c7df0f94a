"""Measured cases of the 4-bit LM head and of the clipped policy loss.

Operators (``op`` of a case):
  rows      rows to microscaled 4-bit floating point (blocks of 32 elements, a power of two each), and read back
  matmul    product of 4-bit token rows with 4-bit channel rows
  head      LM head over the active 4-bit rows of each sequence, with top-k
  policy    clipped policy loss with a KL term and an entropy bonus over full-vocabulary logits, alone or with its gradient

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
BLOCK = 32                              # elements that share a scale
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _pitch(d):
    """Bytes of one row's codes, two a byte: d rounded up to 256 elements, the rest zero.  A sixteenth of that are its scales."""
    return -(-d // 256) * 128


def listed():
    return [
        # the hidden rows of one draft step, quantised before the product
        dict(name="rows_hidden", op="rows", rows=8, d=4096, ld=4096, dtype="bf16"),
        # a whole output matrix, quantised when the weights are loaded
        dict(name="rows_weights", op="rows", rows=128256, d=4096, ld=4096, dtype="bf16"),
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
        # the loss of one step's tokens, without a gradient
        dict(name="policy_step", op="policy", rows=8, v=128256, ld=128256, dtype="fp32", grad=False, ref=True, temp=1.0, kl=0.02, ent=0.0, skip=0.0,
             masked=0.0, empty=False),
        # one short sequence over an odd vocabulary, its prompt and part of the vocabulary left out
        dict(name="policy_odd", op="policy", rows=129, v=50257, ld=50257, dtype="fp32", grad=True, ref=True, temp=0.7, kl=0.05, ent=0.01, skip=0.2,
             masked=0.25, empty=True),
        # a validation batch, half of it prompts
        dict(name="policy_check", op="policy", rows=2048, v=151936, ld=151936, dtype="fp16", grad=False, ref=True, temp=1.0, kl=0.02, ent=0.0, skip=0.5,
             masked=0.0, empty=False),
        # a training batch over the whole vocabulary
        dict(name="policy_batch", op="policy", rows=4096, v=128256, ld=128256, dtype="bf16", grad=True, ref=True, temp=1.0, kl=0.02, ent=0.0, skip=0.0,
             masked=0.0, empty=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rows", "matmul", "head", "policy"))
    dtype = rng.choice(("bf16", "fp16", "fp32"))
    if op == "rows":
        d = _log(rng, 1, 16384)
        rows = _log(rng, 1, max(1, min(131072, WHOLE // (2 * d))))
        return dict(op=op, rows=rows, d=d, ld=d + rng.choice((0, 0, 3, 64)), dtype=dtype)
    if op == "matmul":
        d = _log(rng, 16, 16384)
        m = _log(rng, 1, 4096)
        n = _log(rng, 1, max(1, min(152000, LARGEST // (2 * m * d), WHOLE // m)))
        return dict(op=op, m=m, n=n, d=d, out=dtype)
    if op == "head":
        d = _log(rng, 16, 8192)
        b = _log(rng, 1, 64)
        m = rng.randint(1, 64)
        n_max = _log(rng, 16, max(16, min(16384, (1 << 27) // (b * d))))
        logits = rng.random() < 0.3
        live = n_max if logits else rng.randint(1, n_max)
        v = _log(rng, max(n_max, 2048), 152000)
        return dict(op=op, b=b, m=m, k=rng.randint(1, 64), n_max=n_max, live=live, v=v, d=d, dtype=dtype, logits=logits)
    rows = _log(rng, 1, 4096)
    v = _log(rng, 64, max(64, min(152000, WHOLE // (2 * rows))))
    ref = rng.random() < 0.8
    return dict(op=op, rows=rows, v=v, ld=v + rng.choice((0, 0, 1, 24)), dtype=dtype, grad=rng.random() < 0.7, ref=ref,
                temp=rng.choice((1.0, 1.0, 0.7, 1.5)), kl=rng.choice((0.0, 0.02, 0.1)) if ref else 0.0, ent=rng.choice((0.0, 0.0, 0.01)), skip=rng.choice((0.0, 0.3)),
                masked=rng.choice((0.0, 0.0, 0.5)), empty=rows > 2 and rng.random() < 0.3)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _packed(x):
    """Rows as they are kept: codes [n, pitch] (element 2 i in the low half of byte i) and the blocks' exponents [n, pitch / 16], uint8."""
    value, exponent = _blocks(x)
    twice = (2 * value.abs()).to(torch.int32)
    code = torch.where(twice < 4, twice, torch.where(twice < 8, 2 + twice // 2, 4 + twice // 4)) + 8 * (value < 0).to(torch.int32)
    code = torch.nn.functional.pad(code.flatten(1), (0, 2 * _pitch(x.shape[1]) - code.flatten(1).shape[1])).to(torch.uint8)
    scale = torch.nn.functional.pad((exponent[..., 0] + 127).to(torch.uint8), (0, _pitch(x.shape[1]) // 16 - exponent.shape[1]))
    return code[:, ::2] | (code[:, 1::2] << 4), scale


def _rows4(g, n, d, size):
    """n rows of d weights, quantised a few at a time."""
    q = torch.empty((n, _pitch(d)), dtype=torch.uint8, device="cuda")
    scale = torch.empty((n, _pitch(d) // 16), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // d)
    for at in range(0, n, step):
        rows = min(step, n - at)
        x = torch.randn((rows, d), generator=g, device="cuda") * (size * torch.exp(0.3 * torch.randn((rows, 1), generator=g, device="cuda")))
        q[at:at + rows], scale[at:at + rows] = _packed(x)
    return q, scale


def prepare(case, seed):
    g = _generator(seed)
    s = {"case": case, "table": torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device="cuda")}
    op = case["op"]
    if op == "rows":
        x = torch.randn((case["rows"], case["ld"]), generator=g, device="cuda", dtype=torch.float32 if case["dtype"] == "fp32" else torch.bfloat16)
        s["x"] = x.to(DTYPES[case["dtype"]])
    elif op == "matmul":
        s["xq"], s["xs"] = _rows4(g, case["m"], case["d"], 1.0)
        s["wq"], s["ws"] = _rows4(g, case["n"], case["d"], 0.02)
    elif op == "head":
        b, n_max, v = case["b"], case["n_max"], case["v"]
        s["wq"], s["ws"] = _rows4(g, v, case["d"], 0.02)
        s["h"] = torch.randn((b, case["m"], case["d"]), generator=g, device="cuda").to(DTYPES[case["dtype"]])
        ids = torch.rand((b, v), generator=g, device="cuda").argsort(1)[:, :n_max]
        # the active ids ascend; what lies behind the last one is no row
        live = torch.arange(n_max, device="cuda") < case["live"]
        ids = torch.where(live, ids, v).sort(1).values
        s["ids"] = torch.where(live, ids, -1).to(torch.int32).contiguous()
        s["n"] = torch.full((b,), case["live"], dtype=torch.int32, device="cuda")
    else:
        _policy_inputs(s, g)
    return s


def _policy_inputs(s, g):
    case = s["case"]
    rows, v = case["rows"], case["v"]
    z = torch.randn((rows, case["ld"]), generator=g, device="cuda", dtype=torch.float32 if case["dtype"] == "fp32" else torch.bfloat16).mul_(3)
    tokens = torch.randint(0, v, (rows, 1), generator=g, device="cuda")
    # sampled tokens are likely ones
    z.scatter_reduce_(1, tokens, (12 + 2 * torch.randn((rows, 1), generator=g, device="cuda")).to(z.dtype), "amax")
    if case["masked"]:
        # what no sampler was allowed to take; it has taken the rows' tokens
        banned = torch.rand((v,), generator=g, device="cuda") < case["masked"]
        banned[tokens] = False
        z[:, :v].masked_fill_(banned, -math.inf)
    if case["empty"]:
        # a row that a grammar leaves without any token
        z[rows // 2, :v] = -math.inf
    s["z"] = z.to(DTYPES[case["dtype"]])
    s["tokens"] = tokens[:, 0].to(torch.int32)
    logp = torch.cat([_logp(part, at, 1.0 / case["temp"])[0] for part, at in zip(s["z"][:, :v].split(256), tokens.split(256))])
    logp = torch.where(torch.isfinite(logp), logp, -3.0)
    # How far the policy has moved since the tokens were drawn.  At a border of the clip the gradient jumps, and the
    # last digit of a log-probability would decide: none is drawn within a thousandth of one.
    moved = 0.25 * torch.randn((rows,), generator=g, device="cuda")
    for border in (math.log(1 - 0.2), math.log(1 + 0.28)):
        near = moved - border
        moved = torch.where(near.abs() < 1e-3, border + torch.where(near < 0, -1e-3, 1e-3), moved)
    s["old"] = (logp - moved).float()
    s["ref"] = (logp + 0.3 * torch.randn((rows,), generator=g, device="cuda")).float() if case["ref"] else None
    s["advantage"] = torch.randn((rows,), generator=g, device="cuda")
    taken = torch.rand((rows,), generator=g, device="cuda") >= case["skip"]
    taken[-1] = True
    s["weight"] = taken.float() / taken.sum()
    # what a step over several batches multiplies each loss by
    s["g_loss"] = torch.full((1,), 0.25, device="cuda")


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _blocks(x):
    """Values in units of the block's power of two [n, blocks, 32], and its exponent [n, blocks, 1]."""
    x = torch.nn.functional.pad(x.float(), (0, -x.shape[-1] % BLOCK)).unflatten(-1, (-1, BLOCK))
    top = x.abs().amax(-1, keepdim=True)
    exponent = torch.where(top > 0, torch.frexp(top).exponent - 3, -127).clamp(min=-127)
    y = torch.ldexp(x, -exponent)
    size = y.abs()
    step = torch.where(size < 2, 0.5, torch.where(size < 4, 1.0, 2.0))
    return torch.copysign((torch.round(size / step) * step).clamp(max=6.0), y), exponent


def _values(table, q, scale, d):
    """The values of packed rows [.., pitch], [.., pitch / 16], in 32 bits; table: those of the 16 codes."""
    codes = torch.stack([q & 15, q >> 4], -1).flatten(-2)
    size = torch.ldexp(torch.ones_like(scale, dtype=torch.float32), scale.int() - 127)
    return (table[codes.int()].unflatten(-1, (-1, BLOCK)) * size.unsqueeze(-1)).flatten(-2)[..., :d]


def _best(values, k):
    """The places of the k largest of each row, ties to the lowest place."""
    bits = (values + 0.0).view(torch.int32)
    order = bits ^ ((bits >> 31) & 0x7FFFFFFF)
    place = torch.arange(values.shape[-1], device=values.device)
    return torch.topk((order.long() << 32) + (0xFFFFFFFF - place), k, dim=-1).indices


def _plain_rows(s):
    c = s["case"]
    value, exponent = _blocks(s["x"][:, :c["d"]])
    return {"values": torch.ldexp(value, exponent).flatten(1)[:, :c["d"]].to(s["x"].dtype)}


def _plain_matmul(s):
    c = s["case"]
    # sums of products of these have few digits: 32 bits hold them
    return {"out": (_values(s["table"], s["xq"], s["xs"], c["d"]) @ _values(s["table"], s["wq"], s["ws"], c["d"]).t()).to(DTYPES[c["out"]])}


def _plain_head(s):
    c = s["case"]
    value, exponent = _blocks(s["h"].flatten(0, 1))
    h = torch.ldexp(value, exponent).flatten(1)[:, :c["d"]].unflatten(0, (c["b"], c["m"]))
    at = s["ids"].long().clamp(min=0)
    rows = _values(s["table"], s["wq"][at], s["ws"][at], c["d"])
    logits = (rows @ h.transpose(1, 2).contiguous()).transpose(1, 2)
    live = torch.arange(c["n_max"], device="cuda") < s["n"][:, None]
    k = min(c["k"], c["n_max"])
    masked = torch.where(live[:, None, :], logits, -math.inf)
    best = _best(masked, k)
    values = masked.gather(2, best)
    ids = s["ids"][:, None, :].expand(-1, c["m"], -1).gather(2, best)
    pad = (0, c["k"] - k)
    r = {"ids": torch.nn.functional.pad(ids, pad, value=-1), "values": torch.nn.functional.pad(values, pad, value=-math.inf)}
    if c["logits"]:
        r["logits"] = logits.contiguous()
    return r


def _logp(z, tokens, inv_temp):
    """Log-probabilities of one token a row in 64 bits, and the row's scaled logits, their exponentials (both from the
    maximum) and the exponentials' sum."""
    z = z.float()
    top = z.max(1, keepdim=True).values
    top = torch.where(top == -math.inf, 0.0, top)
    first = (z.gather(1, tokens).double() - top) * inv_temp
    z = (z - top) * inv_temp
    e = torch.exp(z)
    total = e.sum(1, keepdim=True)
    logp = first - torch.log(total.double())
    return torch.where(total > 0, logp, -math.inf)[:, 0], z, e, total


def _plain_policy(s):
    c = s["case"]
    inv_temp = 1.0 / c["temp"]
    tokens = s["tokens"].long()[:, None]
    logp, z, e, total = _logp(s["z"][:, :c["v"]], tokens, inv_temp)
    taken = s["weight"] != 0
    learns = taken & (logp > -math.inf)
    some = torch.where(learns, logp, s["old"])
    a = s["advantage"].double()
    ratio = torch.exp(some - s["old"])
    clipped = ratio.clamp(1 - 0.2, 1 + 0.28)
    delta = s["ref"].double() - some if c["ref"] else torch.zeros_like(some)
    kl = torch.expm1(delta) - delta
    # a row without a finite logit has no probabilities
    p = e / torch.where(total > 0, total, 1.0)
    entropy = torch.where(total[:, 0] > 0, torch.log(total[:, 0]) - (p * torch.where(p > 0, z, 0.0)).sum(1), 0.0)
    w = s["weight"].double() * learns
    loss = (w * (-torch.minimum(ratio * a, clipped * a) + c["kl"] * kl - c["ent"] * entropy)).sum()
    r = {"loss": loss.float()[None], "logprob": torch.where(taken, logp, 0.0).float(), "entropy": torch.where(taken, entropy, 0.0)}
    if c["ref"]:
        r["kl"] = (kl * learns).float()
    if c["grad"]:
        g = w * (torch.where(ratio * a <= clipped * a, -ratio * a, 0.0) + c["kl"] * (1 - torch.exp(delta)))
        factor = s["g_loss"] * inv_temp
        dz = p * (-g * factor).float()[:, None]
        if c["ent"]:
            dz += p * torch.where(p > 0, z - torch.log(total) + entropy[:, None], 0.0) * (w * c["ent"] * factor).float()[:, None]
        dz.scatter_add_(1, tokens, (g * factor).float()[:, None])
        r["dlogits"] = torch.where(learns[:, None], dz, 0.0).to(s["z"].dtype)
    return r


def _own(s):
    from dynamic_vocab_draft_amd import nanospec as ns
    c = s["case"]
    op = c["op"]
    keep = s.setdefault("keep", {})
    new = not keep
    if op == "rows":
        if new:
            keep["q"] = torch.empty((c["rows"], _pitch(c["d"])), dtype=torch.uint8, device="cuda")
            keep["scale"] = torch.empty((c["rows"], _pitch(c["d"]) // 16), dtype=torch.uint8, device="cuda")
            keep["values"] = torch.empty((c["rows"], c["d"]), dtype=s["x"].dtype, device="cuda")
        ns.nanospec_mx4_rows(s["x"][:, :c["d"]], keep["q"], keep["scale"])
        ns.nanospec_mx4_gather_rows(keep["q"], keep["scale"], None, None, keep["values"])
        return {"values": keep["values"]}
    if op == "matmul":
        if new:
            keep["out"] = torch.empty((c["m"], c["n"]), dtype=DTYPES[c["out"]], device="cuda")
        ns.nanospec_mx4_matmul(s["xq"], s["xs"], s["wq"], s["ws"], c["d"], keep["out"])
        return {"out": keep["out"]}
    if op == "head":
        if new:
            keep["ids"] = torch.empty((c["b"], c["m"], c["k"]), dtype=torch.int32, device="cuda")
            keep["values"] = torch.empty((c["b"], c["m"], c["k"]), dtype=torch.float32, device="cuda")
            if c["logits"]:
                keep["logits"] = torch.empty((c["b"], c["m"], c["n_max"]), dtype=torch.float32, device="cuda")
            keep["work"] = ns.alloc_mx4_logits_workspace(c["b"], c["n_max"], c["m"], c["k"], c["d"])
        ns.nanospec_mx4_logits_topk(s["wq"], s["ws"], s["ids"], s["n"], s["h"], c["k"], keep.get("logits"), keep["ids"], keep["values"], keep["work"])
        return {key: keep[key] for key in ("ids", "values", "logits") if key in keep}
    z = s["z"][:, :c["v"]]
    if new:
        keep["loss"] = torch.empty((1,), dtype=torch.float32, device="cuda")
        for key in ("logprob", "entropy") + (("kl",) if c["ref"] else ()):
            keep[key] = torch.empty((c["rows"],), dtype=torch.float32, device="cuda")
        if c["grad"]:
            keep["dlogits"] = torch.empty((c["rows"], c["v"]), dtype=z.dtype, device="cuda")
        keep["work"] = ns.alloc_policy_loss_workspace(c["rows"], c["v"])
    ns.nanospec_policy_loss(z, 1.0 / c["temp"], s["tokens"], s["old"], s["ref"], s["advantage"], s["weight"], 0.2, 0.28, c["kl"], c["ent"], keep["loss"],
                            keep["logprob"], keep.get("kl"), keep["entropy"], s["g_loss"], keep.get("dlogits"), keep["work"])
    return {key: t for key, t in keep.items() if key != "work"}


def run(state):
    if own:
        return _own(state)
    return {"rows": _plain_rows, "matmul": _plain_matmul, "head": _plain_head, "policy": _plain_policy}[state["case"]["op"]](state)


def work(case):
    op = case["op"]
    if op == "rows":
        # the rows, their codes and scales, and what these stand for
        n = case["rows"] * case["d"]
        return {"bytes": int(n * (2 * SIZES[case["dtype"]] + 0.5 + 1 / BLOCK)), "flops": 4 * n}
    if op == "matmul":
        m, n, d = case["m"], case["n"], case["d"]
        return {"bytes": int((m + n) * d * (0.5 + 1 / BLOCK)) + m * n * SIZES[case["out"]], "flops": 2 * m * n * d}
    if op == "head":
        b, m, n, d, v = case["b"], case["m"], case["live"], case["d"], case["v"]
        # rows that several sequences hold are read once
        rows = v * (1 - (1 - n / v) ** b)
        size = rows * d * (0.5 + 1 / BLOCK) + b * n * 4 + b * m * d * SIZES[case["dtype"]] + b * m * case["k"] * 8
        return {"bytes": int(size + (4 * b * m * n if case["logits"] else 0)), "flops": 2 * b * m * n * d}
    # rows without a weight are not looked at, but their gradient is written
    n = case["rows"] * case["v"]
    read = n * (1 - case["skip"])
    return {"bytes": int((read + n * case["grad"]) * SIZES[case["dtype"]]) + case["rows"] * 32, "flops": int(read * (8 if case["grad"] else 5))}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _nearest4(x):
    """Each element's nearest value of its block's grid, x [.., d] in 64 bits: by the borders between the grid's values."""
    d = x.shape[-1]
    grid = torch.tensor(MAGNITUDES, dtype=torch.float64, device=x.device)
    borders = (grid[1:] + grid[:-1]) / 2
    x = torch.nn.functional.pad(x, (0, -d % BLOCK))
    x = x.reshape(*x.shape[:-1], -1, BLOCK)
    top = x.abs().max(-1, keepdim=True).values
    # 2^floor(log2 top) from the bits of the double
    unit = (top.contiguous().view(torch.int64) & (0x7FF << 52)).view(torch.float64) / 4
    unit = unit.clamp(min=2.0 ** -127)
    size = x.abs() / unit
    at = torch.bucketize(size, borders, right=True)
    # on a border the value with an even code
    at = at - ((at > 0) & (size == borders[(at - 1).clamp(min=0)]) & (at % 2 == 1)).long()
    return (torch.sign(x) * grid[at] * unit).flatten(-2)[..., :d]


def _stored(q, scale, d):
    """Packed rows as real numbers, code by code: sign, exponent and mantissa bits."""
    code = torch.empty((*q.shape[:-1], 2 * q.shape[-1]), dtype=torch.int64, device=q.device)
    code[..., 0::2], code[..., 1::2] = q & 15, q >> 4
    e, m = (code >> 1) & 3, (code & 1).double()
    size = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.pow(2.0, (e - 1).double()))
    unit = torch.pow(2.0, scale.double() - 127.0).repeat_interleave(BLOCK, -1)
    return (torch.where(code >= 8, -size, size) * unit)[..., :d]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rows":
        step = max(1, (1 << 26) // case["d"])
        return {"values": torch.cat([_nearest4(part.double()) for part in s["x"][:, :case["d"]].split(step)])}
    if op == "matmul":
        x = _stored(s["xq"], s["xs"], case["d"])
        out = torch.empty((case["m"], case["n"]), dtype=torch.float64, device="cuda")
        step = max(1, (1 << 26) // case["d"])
        for at in range(0, case["n"], step):
            w = _stored(s["wq"][at:at + step], s["ws"][at:at + step], case["d"])
            out[:, at:at + step] = torch.mm(x, w.t())
        return {"out": out}
    if op == "head":
        if case["b"] * case["n_max"] * case["d"] > 1 << 28:
            return None
        h = _nearest4(s["h"].double())
        values, whole = [], []
        for b in range(case["b"]):
            ids = s["ids"][b, :case["live"]].long()
            z = torch.mm(h[b], _stored(s["wq"][ids], s["ws"][ids], case["d"]).t().contiguous())
            found = z.sort(1, descending=True).values[:, :case["k"]]
            rest = torch.full((case["m"], case["k"] - found.shape[1]), -math.inf, dtype=torch.float64, device="cuda")
            values.append(torch.cat([found, rest], 1))
            whole.append(z)
        r = {"ids": None, "values": torch.stack(values)}
        if case["logits"]:
            r["logits"] = torch.stack(whole)
        return r
    step = max(1, (1 << 26) // case["v"])
    parts = [_exact_policy(case, s, slice(at, at + step)) for at in range(0, case["rows"], step)]
    r = {key: torch.cat([p[key] for p in parts]) for key in parts[0]}
    r["loss"] = r["loss"].sum()[None]
    return r


def _exact_policy(case, s, rows):
    """Rows of the policy loss and its gradient, the gradient as the softmax's of each part of the loss."""
    z = s["z"][rows, :case["v"]].to(torch.float64) / case["temp"]
    tokens = s["tokens"][rows].long().unsqueeze(1)
    empty = (z == -math.inf).all(1, keepdim=True)
    every = torch.where(empty, -math.inf, torch.log_softmax(z, 1))
    logp = every.gather(1, tokens).squeeze(1)
    p = torch.where(empty, 0.0, every.exp())
    entropy = -torch.special.xlogy(p, p).sum(1)
    w = s["weight"][rows].double()
    taken = w > 0
    learns = taken & (logp > -math.inf)
    a, old = s["advantage"][rows].double(), s["old"][rows].double()
    r = torch.where(learns, torch.exp(logp - old), 1.0)
    over, under = (a > 0) & (r > 1.28), (a < 0) & (r < 0.8)
    gain = torch.where(over, 1.28 * a, torch.where(under, 0.8 * a, r * a))
    slope = torch.where(over | under, 0.0, r * a)
    back = torch.ones_like(r)
    kl = torch.zeros_like(r)
    if case["ref"]:
        ref = s["ref"][rows].double()
        back = torch.where(learns, torch.exp(ref - logp), 1.0)
        kl = torch.where(learns, back - 1.0 - (ref - logp), 0.0)
    w = torch.where(learns, w, 0.0)
    out = {"loss": w * (case["kl"] * kl - gain - case["ent"] * entropy), "logprob": torch.where(taken, logp, 0.0),
           "entropy": torch.where(taken, entropy, 0.0)}
    if case["ref"]:
        out["kl"] = kl
    if case["grad"]:
        one = torch.zeros_like(p).scatter_(1, tokens, 1.0)
        d = (w * (case["kl"] * (1.0 - back) - slope)).unsqueeze(1) * (one - p)
        d += (w * case["ent"]).unsqueeze(1) * p * (torch.where(p > 0, every, 0.0) + entropy.unsqueeze(1))
        out["dlogits"] = torch.where(learns.unsqueeze(1), d, 0.0) * (0.25 / case["temp"])
    return out
