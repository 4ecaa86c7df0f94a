"""nanospec_token_logprobs and its gradient against the formulas in float64.

Tolerances, with u = 2^-24 (half a float32 step, relative) and Z the largest
|inv_temp * z| among the logits of a row whose probability is not 0:
  * an exponent c z - E carries c's rounding and its own, at most 3 Z u in
    natural units; 2^y and the longest chain of additions (32 within a batch,
    63 batches, 6 lane steps, 64 parts) add at most 200 u to a sum; log2 and the last
    operations at most 20 u (a log2 below 20) and Z u.  So lse and
    log-probabilities are within u (8 Z + 300), absolutely, and 8 u of its
    own size for a token far below the rest;
  * entropy is a difference of log2 S and a weighted mean of exponents whose
    terms carry the same relative errors: u (8 Z + 400) (2 + H);
  * the gradient's p_j carry u (8 Z + 320) relatively through lse, its factors
    the errors of logp and H; the result is rounded once to its type
    (eps / 2), fp16 below its normal range to 2^-25.
"""
import math

import numpy as np
import pytest
import torch

from tests.gpu_common import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def ns():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from dynamic_vocab_draft_amd import nanospec
    return nanospec


def make_logits(L, V, dtype, seed, ld=None, scale=3.0, offset=0):
    """Rows of V logits ld apart that start `offset` elements into an allocation; the guard values are 1.5."""
    ld = ld or V
    rng = np.random.default_rng(seed)
    mem = torch.full((L * ld + offset + 8,), 1.5, dtype=DT[dtype], device="cuda")
    z = mem[offset:offset + L * ld].view(L, ld)[:, :V]
    z.copy_(torch.from_numpy((rng.standard_normal((L, V)) * scale).astype(np.float32)).to(DT[dtype]))
    return z, mem


def reference(z, it, tokens, k):
    """lse, logprob, entropy, top ids and log-probabilities in float64 (numpy)."""
    x = z.double().cpu().numpy()
    y = x * it
    L, V = y.shape
    with np.errstate(all="ignore"):
        bad = np.isnan(x).any(1) | (x == np.inf).any(1)
        top = y.max(1)
        none = ~bad & (top == -np.inf)
        s = np.exp(np.where((top == -np.inf)[:, None], -np.inf, y - top[:, None])).sum(1)
        lse = np.where(none, -np.inf, top + np.log(s))
        # relative to the top, so that logits at the type's lowest keep their differences
        logp = np.where((y == -np.inf) | none[:, None], -np.inf, (y - top[:, None]) - np.log(s)[:, None])
        p = np.exp(logp)
        H = -np.where(p > 0, p * logp, 0.0).sum(1)
    lse[bad] = np.nan
    H[bad] = np.nan
    logp[bad] = np.nan
    H[none] = 0.0
    ids = np.empty((L, k), np.int64)
    for i in range(L):
        order = np.lexsort((np.arange(V), -np.nan_to_num(x[i], nan=0.0, posinf=np.inf, neginf=-np.inf)))
        ids[i] = -1 if bad[i] else order[:k]
    tv = np.where(bad[:, None], np.nan, np.take_along_axis(logp, np.maximum(ids, 0), 1)) if k else np.zeros((L, 0))
    lp = np.zeros(tokens.shape)
    for i in range(L):
        for t in range(tokens.shape[1]):
            if 0 <= tokens[i, t] < V:
                lp[i, t] = logp[i, tokens[i, t]]
    fin = np.where(np.isfinite(y) & (p > 0), np.abs(y), 0.0).max(1)
    return dict(lse=lse, H=H, logp=logp, ids=ids, tv=tv, lp=lp, Z=fin)


def call(ns, z, it, tokens, k, entropy=True, stream=None, work=None):
    L, V = z.shape
    T = tokens.shape[1]
    tok = torch.as_tensor(tokens.astype(np.int32)).cuda() if T else None
    f = lambda *s: torch.full(s, 7.25, device="cuda")
    lp = f(L, T) if T else None
    lse, H = f(L), f(L) if entropy else None
    ti = torch.full((L, k), 77, dtype=torch.int32, device="cuda") if k else None
    tv = f(L, k) if k else None
    work = ns.alloc_token_logprobs_workspace(L, V, k) if work is None else work
    ns.nanospec_token_logprobs(z, it, tok, lp, lse, H, ti, tv, work, stream=stream)
    return dict(lp=lp, lse=lse, H=H, ids=ti, tv=tv, tok=tok)


def near(got, ref, tol, what):
    got = got.double().cpu().numpy()
    tol = np.broadcast_to(tol, ref.shape)
    fin = np.isfinite(ref)
    same = (np.isnan(got) & np.isnan(ref)) | (got == ref)
    assert same[~fin].all(), f"{what}: values that are not finite differ"
    bad = np.abs(got[fin] - ref[fin]) > tol[fin]
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off, worst " \
                          f"{np.max(np.abs(got[fin] - ref[fin]) / tol[fin]):.3g} of the tolerance"


def check(ns, z, it, tokens, k, what):
    say("token_logprobs", what)
    r = reference(z, it, tokens, k)
    o = call(ns, z, it, tokens, k)
    torch.cuda.synchronize()
    base = U * (8 * r["Z"] + 300)
    near(o["lse"], r["lse"], base, f"{what} lse")
    near(o["H"], r["H"], U * (8 * r["Z"] + 400) * (2 + np.nan_to_num(r["H"])), f"{what} entropy")
    if tokens.shape[1]:
        near(o["lp"], r["lp"], base[:, None] + 8 * U * np.abs(r["lp"]), f"{what} logprob")
    if k:
        assert np.array_equal(o["ids"].cpu().numpy(), r["ids"]), f"{what}: top ids"
        near(o["tv"], r["tv"], base[:, None] + 8 * U * np.abs(r["tv"]), f"{what} top")
    return r, o


def tokens_for(L, V, T, seed):
    return np.random.default_rng(seed).integers(0, V, (L, T))


CASES = [
    # L, V, dtype, ld, offset, T, k, inv_temp
    (1, 1, "fp32", 1, 0, 1, 1, 1.0),
    (3, 2, "bf16", 5, 1, 2, 2, 1.0),
    (2, 7, "bf16", 7, 3, 1, 7, 0.5),
    (5, 9, "fp16", 9, 0, 4, 3, 1.0),
    (4, 64, "fp32", 67, 1, 8, 64, 2.0),
    (1, 1000, "bf16", 1001, 0, 64, 64, 1.0),
    (129, 4097, "fp16", 4097, 1, 1, 20, 1.0),
    (7, 50257, "bf16", 50257, 0, 3, 4, 1.3),
    (1, 128256, "fp32", 128256, 0, 1, 8, 1.0),
    (60, 32000, "fp32", 32008, 2, 10, 1, 0.7),
    (2, 151936, "bf16", 151936, 0, 2, 64, 1.0),
    (2100, 515, "bf16", 515, 1, 1, 4, 1.0),
    (2049, 5000, "fp32", 5000, 0, 1, 33, 1.0),
    (300, 20011, "fp16", 20011, 0, 1, 0, 1.0),
    (2050, 2300, "fp16", 2304, 0, 0, 5, 3.0),
]


@pytest.mark.parametrize("c", CASES, ids=lambda c: "x".join(str(v) for v in c))
def test_against_float64(ns, c):
    L, V, dtype, ld, off, T, k, it = c
    z, mem = make_logits(L, V, dtype, 11 + V, ld, offset=off)
    before = mem.clone()
    check(ns, z, it, tokens_for(L, V, T, 5) if T else np.zeros((L, 0), np.int64), k, str(c))
    assert torch.equal(mem, before)


@pytest.mark.parametrize("V", [40, 1000, 6000, 30011])
@pytest.mark.parametrize("k", [1, 7, 64])
def test_ties_go_to_the_lowest_id(ns, V, k):
    k = min(k, V)
    for L in (3, 2100 if V <= 6000 else 5):
        for levels in (1, 2, 9):
            rng = np.random.default_rng(V + levels)
            z = torch.from_numpy(rng.integers(0, levels, (L, V)).astype(np.float32) - 1).cuda().bfloat16()
            z[0] = torch.where(z[0] == 0, torch.tensor(-0.0, device="cuda", dtype=z.dtype), z[0])
            check(ns, z, 1.0, tokens_for(L, V, 1, 3), k, f"ties V={V} k={k} L={L} levels={levels}")
        z = torch.arange(V, device="cuda", dtype=torch.float32).div(64).floor().repeat(L, 1)   # rising values
        check(ns, z, 1.0, tokens_for(L, V, 1, 3), k, f"rising V={V} k={k} L={L}")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("k", [1, 20, 64])
def test_many_equal_logits(ns, dtype, k):
    """Runs of equal logits, in rising and falling steps, among masked ones and alone: more reach the bound than fit."""
    V = 20011
    rng = np.random.default_rng(k)
    ids = np.arange(V)
    rows = [np.full(V, -np.inf), np.full(V, 7.0), ids // 600 * 0.25, -(ids // 600) * 0.25, ids // 70 % 3 * 1.0,
            np.where(rng.random(V) < 0.5, -np.inf, 1.0), np.where(ids < V - 40, -np.inf, 1.0),
            np.where(rng.random(V) < 0.002, 2.0, 1.0), np.where(ids % 8 == 7, 3.0, -1.0), np.where(ids % 512 < 100, 4.0, 4.25)]
    z = torch.from_numpy(np.stack(rows * 230 if k == 20 else rows).astype(np.float32)).to(DT[dtype]).cuda()
    check(ns, z, 1.0, tokens_for(z.shape[0], V, 2, 5), k, f"equal logits {dtype} k={k}")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("L", [6, 2104])
@pytest.mark.parametrize("V", [70, 4100, 9001])
def test_masks_and_extremes(ns, dtype, L, V):
    z, _ = make_logits(L, V, dtype, 3)
    low = torch.finfo(DT[dtype]).min
    z[0] = -math.inf                                     # nothing left
    z[1, :] = -math.inf
    z[1, V - 1] = 2.5                                    # one logit, the last
    z[2, : V // 2] = low                                 # the type's lowest as a mask
    z[3] = low                                           # nothing but the lowest: a uniform row
    z[4, 5:] = -math.inf
    z[5] = z[5] * 0 - 300.0                              # far below zero
    if L > 6:
        z[6, 3] = math.nan
        z[7, V - 1] = math.inf
        z[8, 0] = -math.inf
        z[9] = torch.linspace(-1, 1, V, device="cuda").to(z.dtype) * 60000     # far apart
        z[10, 1] = 900.0
        z[11] = math.nan
        z[12, 64:] = -math.inf
        z[13, : V - 1] = -math.inf
    tok = tokens_for(L, V, 3, 8)
    tok[:, 1] = -1
    tok[0, 2] = V
    tok[1, 0] = V - 1
    tok[1, 2] = 3
    check(ns, z, 1.0, tok, min(64, V), f"masks {dtype} L={L} V={V}")


def test_late_maximum_and_wide_temperatures(ns):
    for V in (5000, 70000):
        z, _ = make_logits(3, V, "fp32", 4)
        z[0, V - 3] = 90.0                               # the maximum comes last
        z[1, : V - 2000] = -math.inf                     # the first batches are empty
        z[2, V // 2:] += 70
        for it in (2.0 ** -20, 0.01, 1.0, 40.0):
            check(ns, z, it, tokens_for(3, V, 2, 9), 5, f"late V={V} it={it}")
    z, _ = make_logits(2, 3000, "fp32", 4, scale=1.0)
    # differences of float32 logits near 1e6 are exact, so probabilities are too; lse itself is not
    z += 1.0e6
    r = reference(z, 1.0, tokens_for(2, 3000, 1, 9), 4)
    o = call(ns, z, 1.0, tokens_for(2, 3000, 1, 9), 4)
    near(o["lp"], r["lp"], U * 400, "shifted logprob")
    near(o["H"], r["H"], U * 800 * 12, "shifted entropy")
    near(o["lse"], r["lse"], U * (8e6 + 300), "shifted lse")


def test_optional_outputs_and_streams(ns):
    z, _ = make_logits(9, 3001, "bf16", 2)
    tok = tokens_for(9, 3001, 2, 1)
    full = call(ns, z, 1.0, tok, 4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    part = call(ns, z, 1.0, tok, 0, entropy=False, stream=s)
    none = call(ns, z, 1.0, np.zeros((9, 0), np.int64), 4, stream=s)
    torch.cuda.synchronize()
    # without top alternatives the parts and sums are the same: equal bits
    for a, b in ((full["lp"], part["lp"]), (full["lse"], part["lse"]), (full["tv"], none["tv"]),
                 (full["ids"], none["ids"]), (full["H"], none["H"])):
        assert torch.equal(a, b)


def test_no_rows(ns):
    z = torch.empty((0, 100), device="cuda")
    e = torch.empty(0, device="cuda")
    ns.nanospec_token_logprobs(z, 1.0, None, None, e, None, None, None, ns.alloc_token_logprobs_workspace(0, 100, 0))
    ns.nanospec_token_logprobs_grad(z, 1.0, None, e, None, None, None, None, torch.empty_like(z))


# ---------------------------------------------------------------------------
# Gradient
# ---------------------------------------------------------------------------
def grad_reference(z, it, tokens, r, g, gH, gl):
    L, V = z.shape
    p = np.exp(r["logp"])
    G = gl - np.where((tokens >= 0) & (tokens < V), g, 0.0).sum(1)
    logp = np.where(p > 0, r["logp"], 0.0)
    inner = G[:, None] - gH[:, None] * (logp + r["H"][:, None])
    d = p * inner
    size = p * (np.abs(G)[:, None] + np.abs(gH)[:, None] * (np.abs(logp) + r["H"][:, None] + 3))
    for i in range(L):
        for t in range(tokens.shape[1]):
            if 0 <= tokens[i, t] < V:
                d[i, tokens[i, t]] += g[i, t]
                size[i, tokens[i, t]] += abs(g[i, t])
    none = r["lse"] == -np.inf
    d[none] = 0.0
    size[none] = 0.0
    return d * it, size * it


def run_grad(ns, z, it, tokens, lse, H, g, gH, gl, out):
    T = tokens.shape[1]
    f = lambda a: None if a is None else torch.from_numpy(np.asarray(a, np.float32)).cuda()
    tok = torch.as_tensor(tokens.astype(np.int32)).cuda() if T else None
    ns.nanospec_token_logprobs_grad(z, it, tok, lse, H, f(g) if T else None, f(gH), f(gl), out)


def check_grad(ns, z, it, tokens, what, use_H=True, use_l=True, inplace=False, ld_d=None, off=0):
    say("token_logprobs_grad", what)
    L, V = z.shape
    rng = np.random.default_rng(L + V)
    g = rng.standard_normal(tokens.shape).astype(np.float32)
    gH = rng.standard_normal(L).astype(np.float32) if use_H else np.zeros(L, np.float32)
    gl = rng.standard_normal(L).astype(np.float32) if use_l else np.zeros(L, np.float32)
    r = reference(z, it, tokens, 0)
    d, size = grad_reference(z, it, tokens, r, g.astype(np.float64), gH.astype(np.float64), gl.astype(np.float64))
    o = call(ns, z, it, tokens, 0)
    mem = None
    if inplace:
        out = z
    else:
        ld = ld_d or V
        mem = torch.full((L * ld + off + 8,), 1.5, dtype=z.dtype, device="cuda")
        out = mem[off:off + L * ld].view(L, ld)[:, :V]
    run_grad(ns, z, it, tokens, o["lse"], o["H"] if use_H else None, g, gH if use_H else None, gl if use_l else None, out)
    torch.cuda.synchronize()
    eps = torch.finfo(z.dtype).eps
    tiny = 2.0 ** -25 if z.dtype == torch.float16 else 2.0 ** -133 if z.dtype == torch.bfloat16 else 2.0 ** -126
    tol = size * U * (8 * r["Z"][:, None] + 400) * 2
    tol = tol + (np.abs(d) + tol) * eps / 2 + tiny
    near(out, d, tol, what)
    if mem is not None:
        keep = torch.ones_like(mem, dtype=torch.bool)
        keep[off:off + L * ld].view(L, ld)[:, :V] = False
        assert (mem[keep] == 1.5).all(), f"{what}: wrote between the rows"
    return out


GRADS = [
    # L, V, dtype, ld, offset, T, inv_temp, ld_d, off_d
    (1, 1, "fp32", 1, 0, 1, 1.0, 1, 0),
    (2, 3, "bf16", 4, 1, 2, 1.0, 5, 3),
    (5, 9, "fp16", 9, 1, 4, 0.5, 9, 0),
    (4, 70, "fp32", 70, 1, 64, 2.0, 71, 1),
    (129, 4097, "fp16", 4097, 1, 1, 1.0, 4097, 1),
    (7, 50257, "bf16", 50257, 0, 3, 1.3, 50257, 0),
    (33, 32000, "fp32", 32004, 0, 1, 0.7, 32000, 0),
    (3, 151936, "bf16", 151936, 0, 8, 1.0, 151936, 0),
]


@pytest.mark.parametrize("c", GRADS, ids=lambda c: "x".join(str(v) for v in c))
def test_grad_against_float64(ns, c):
    L, V, dtype, ld, off, T, it, ld_d, off_d = c
    z, _ = make_logits(L, V, dtype, 21 + V, ld, offset=off)
    tok = tokens_for(L, V, T, 6)
    tok[:, -1] = tok[:, 0]                               # a token named twice
    check_grad(ns, z, it, tok, str(c), ld_d=ld_d, off=off_d)


@pytest.mark.parametrize("use_H,use_l,T", [(False, False, 1), (True, False, 0), (False, True, 2)])
def test_grad_optional_inputs(ns, use_H, use_l, T):
    z, _ = make_logits(5, 3001, "fp32", 2)
    check_grad(ns, z, 1.0, tokens_for(5, 3001, T, 1) if T else np.zeros((5, 0), np.int64), f"{use_H} {use_l} {T}",
               use_H, use_l)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_grad_in_place(ns, dtype):
    for V, ld, off in ((9001, 9001, 0), (9001, 9005, 1), (16, 16, 0), (5, 6, 1)):
        z, _ = make_logits(6, V, dtype, 2, ld, offset=off)
        tok = tokens_for(6, V, 4, 1)
        tok[:, 2] = tok[:, 1]
        tok[0, 0] = V - 1
        tok[1, 0] = -1
        apart = check_grad(ns, z, 0.8, tok, f"apart {dtype} {V}")
        same = check_grad(ns, z, 0.8, tok, f"in place {dtype} {V}", inplace=True)
        assert torch.equal(apart, same)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_grad_masks(ns, dtype):
    V = 4100
    z, _ = make_logits(8, V, dtype, 3)
    z[0] = -math.inf
    z[1, :] = -math.inf
    z[1, V - 1] = 2.5
    z[2, : V // 2] = torch.finfo(z.dtype).min
    z[3, 5:] = -math.inf
    tok = tokens_for(8, V, 2, 8)
    tok[4] = -1
    tok[5, 0] = V
    tok[3, 0] = 2
    tok[2] = [V - 1, V // 2]
    check_grad(ns, z, 1.0, tok, f"masks {dtype}")
    # rows without a distribution: NaN through the whole row; a lse past float32's resolution: 0
    z[6, 3] = math.nan
    z[7] = torch.finfo(z.dtype).min
    o = call(ns, z, 1.0, tok, 0)
    out = torch.empty_like(z)
    run_grad(ns, z, 1.0, tok, o["lse"], o["H"], np.ones((8, 2)), np.ones(8), np.ones(8), out)
    assert torch.isnan(out[6]).all()
    assert torch.isfinite(out[:6]).all()
    if dtype != "fp16":                                  # fp16's lowest, -65504, is an ordinary float32
        assert (out[7] == 0).all()


def test_grad_against_differences(ns):
    """The directional derivative of g . logprob + g_H . H + g_l . lse (float64) against the kernel's gradient."""
    L, V, T, it = 3, 300, 2, 0.9
    z, _ = make_logits(L, V, "fp32", 5, scale=1.0)
    tok = tokens_for(L, V, T, 2)
    rng = np.random.default_rng(1)
    g, gH, gl = rng.standard_normal((L, T)), rng.standard_normal(L), rng.standard_normal(L)
    g, gH, gl = (a.astype(np.float32).astype(np.float64) for a in (g, gH, gl))
    o = call(ns, z, it, tok, 0)
    d = torch.empty_like(z)
    run_grad(ns, z, it, tok, o["lse"], o["H"], g, gH, gl, d)

    def value(x):
        r = reference(x, it, tok, 0)
        return (g * r["lp"]).sum() + (gH * r["H"]).sum() + (gl * r["lse"]).sum()

    for s in range(4):
        v = torch.from_numpy(np.random.default_rng(s).standard_normal((L, V))).cuda()
        h = 1e-4
        diff = (value(z.double() + h * v) - value(z.double() - h * v)) / (2 * h)
        # central differences: h^2 / 6 of the third derivative (about 1e-7 here); the gradient's own 1e-5
        assert abs(diff - float((d.double() * v).sum())) < 1e-4 * (1 + abs(diff))
