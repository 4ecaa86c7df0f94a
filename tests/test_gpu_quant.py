"""8-bit rows against their definitions in 64 bits.

Quantised integers and scales are defined exactly, so they are compared for
equality.  A product carries three float32 roundings (the sum, the scales'
product, their product): at most 3.01 * 2^-24 relatively, then half a step of
the output type; it is also compared bit for bit with those three roundings
done in numpy, so the head's ids can be compared for equality too.
"""
import math

import numpy as np
import pytest
import torch

from tests.gpu_common import say

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def ns():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from dynamic_vocab_draft_amd import nanospec
    return nanospec


def pitch(d):
    return -(-d // 128) * 128


def quantised(x):
    """q (float64 integers) and scale (float32) of float64 rows, from the definition."""
    a = np.abs(x).max(-1, keepdims=True)
    bad = ~np.isfinite(x).all(-1)
    with np.errstate(all="ignore"):
        q = np.where(a > 0, np.rint(127 * x / np.where(a > 0, a, 1)), 0.0)
    q[bad] = 0
    s = (a[..., 0] / 127).astype(np.float32)
    s[bad] = np.nan
    return q, s


def run_quant(ns, x):
    R, d = x.shape
    q = torch.full((R, pitch(d)), 99, dtype=torch.int8, device="cuda")
    s = torch.full((R,), 7.0, device="cuda")
    ns.nanospec_quant_rows(x, q, s)
    torch.cuda.synchronize()
    return q, s


def check_quant(ns, x, what):
    say("quant_rows", what)
    q, s = run_quant(ns, x)
    rq, rs = quantised(x.double().cpu().numpy())
    d = x.shape[1]
    assert np.array_equal(s.cpu().numpy(), rs, equal_nan=True), f"{what}: scales"
    q = q.cpu().numpy()
    assert (q[:, d:] == 0).all(), f"{what}: padding"
    assert np.array_equal(q[:, :d].astype(np.float64), rq), f"{what}: {int((q[:, :d] != rq).sum())} integers differ"


QUANT = [(1, 1, "fp32", 1, 0), (3, 2, "bf16", 3, 1), (5, 8, "fp16", 8, 0), (7, 127, "bf16", 127, 0),
         (4, 128, "fp32", 131, 1), (9, 129, "fp16", 129, 1), (8, 4096, "bf16", 4096, 0), (60, 3584, "bf16", 3600, 0),
         (33, 4096, "fp32", 4096, 0), (5, 4104, "fp16", 4104, 0), (2, 16384, "fp32", 16384, 0),
         (3, 16384, "bf16", 16384, 0), (3, 16383, "fp16", 16383, 1), (3001, 250, "bf16", 250, 0),
         (1000, 1000, "fp32", 1000, 0), (70, 8192, "bf16", 8200, 0)]


@pytest.mark.parametrize("c", QUANT, ids=lambda c: "x".join(str(v) for v in c))
def test_quant_rows(ns, c):
    R, d, dtype, ld, off = c
    rng = np.random.default_rng(R + d)
    mem = torch.zeros(R * ld + off + 8, dtype=DT[dtype], device="cuda")
    x = mem[off:off + R * ld].view(R, ld)[:, :d]
    x.copy_(torch.from_numpy(rng.standard_normal((R, d)).astype(np.float32)).to(DT[dtype]))
    check_quant(ns, x, str(c))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("d", [200, 4096])
def test_quant_borders(ns, dtype, d):
    """Halves, the float32 neighbours of halves, zeros, the largest, the smallest and values that are not finite."""
    R = 40
    rng = np.random.default_rng(d)
    x = rng.standard_normal((R, d))
    halves = (2 * rng.integers(0, 127, (R, d)) + 1) / 2.0            # n + 1/2
    x[:8] = (halves * np.where(rng.random((R, d)) < 0.5, -1, 1))[:8]
    x[:8, 0] = 127.0                                                 # scale 1: exact halves
    if dtype == "fp32":
        near = np.nextafter(halves.astype(np.float32), np.where(rng.random((R, d)) < 0.5, 0, 1e9).astype(np.float32))
        x[8:16] = near[8:16]
        x[8:16, 0] = 127.0
        x[16:20] = (halves * 3.3)[16:20]                             # next to halves after the division
        x[16:20, 0] = 127 * 3.3
    x[20] = 0
    x[21] = -0.0
    t = torch.from_numpy(x.astype(np.float32)).to(DT[dtype]).cuda()
    fi = torch.finfo(DT[dtype])
    t[22] *= fi.tiny                                                 # subnormal for the most part
    t[23] = 0
    t[23, 5] = fi.smallest_normal
    t[24] = 0
    t[24, d - 1] = -fi.smallest_normal / 4 if dtype != "bf16" else fi.smallest_normal
    t[25] = torch.where(t[25] > 0, fi.max, fi.min)
    t[26, 7] = fi.max
    t[27, 3] = math.nan
    t[28, d - 1] = math.inf
    t[29, 0] = -math.inf
    t[30] = math.nan
    t[31] = t[31, 0]
    check_quant(ns, t, f"borders {dtype} {d}")


# rows that 16 lanes, a wave or a block take, with every remainder of a vector
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("R,d", [(1, 3), (17, 9), (5000, 30), (33, 121), (1025, 255), (2000, 260), (50, 505), (1030, 511),
                                 (1100, 514), (40, 517), (1500, 1023), (1030, 4091), (20, 4090), (1100, 4100), (9, 10007)])
def test_quant_rows_in_parts(ns, R, d, dtype):
    rng = np.random.default_rng(d)
    x = torch.from_numpy(rng.standard_normal((R, d + 1)).astype(np.float32)).to(DT[dtype]).cuda()
    check_quant(ns, x[:, 1:], f"{R} x {d} {dtype}")


@pytest.mark.parametrize("d", [60, 512, 1000, 5000])
def test_quant_next_to_halves(ns, d):
    """float32 values at and beside (n + 1/2) a / 127 for maxima a of every size, down to subnormal ones."""
    R = 1200
    rng = np.random.default_rng(d)
    a = np.exp2(rng.uniform(-148, 127.9, (R, 1))).astype(np.float32)
    a[:400] = np.exp2(rng.uniform(-3, 3, (400, 1))).astype(np.float32)
    h = (2 * rng.integers(0, 127, (R, d)) + 1) / 254.0 * a.astype(np.float64)
    x = h.astype(np.float32)
    for _ in range(2):
        to = np.where(rng.random((R, d)) < 0.5, np.float32(0), np.float32(np.inf))
        x = np.where(rng.random((R, d)) < 0.4, np.nextafter(x, to), x)
    x = np.minimum(x, a) * np.where(rng.random((R, d)) < 0.5, np.float32(-1), np.float32(1))
    x[:, d // 2] = a[:, 0]
    check_quant(ns, torch.from_numpy(x.astype(np.float32)).cuda(), f"next to halves {d}")


def int8_rows(n, d, seed, extreme=False):
    rng = np.random.default_rng(seed)
    q = np.zeros((n, pitch(d)), np.int8)
    q[:, :d] = rng.choice([-128, 127], (n, d)) if extreme else np.clip(np.rint(rng.standard_normal((n, d)) * 40), -127, 127)
    return q


def replica(xq, xs, wq, ws):
    """The three float32 roundings of a product, in numpy."""
    acc = xq.astype(np.float64) @ wq.astype(np.float64).T
    return acc.astype(np.float32) * (xs.astype(np.float32)[:, None] * ws.astype(np.float32)[None])


def check_matmul(ns, M, N, d, out, ld=None, off=0, extreme=False, what=""):
    say("quant_matmul", M, N, d, out, ld, off, what)
    xq, wq = int8_rows(M, d, 1, extreme), int8_rows(N, d, 2, extreme)
    rng = np.random.default_rng(3)
    xs, ws = (np.exp(rng.standard_normal(n)).astype(np.float32) * 0.01 for n in (M, N))
    ld = ld or N
    mem = torch.full((M * ld + off + 8,), 1.5, dtype=DT[out], device="cuda")
    o = mem[off:off + M * ld].view(M, ld)[:, :N]
    dev = lambda a: torch.from_numpy(a).cuda()
    ns.nanospec_quant_matmul(dev(xq), dev(xs), dev(wq), dev(ws), d, o)
    torch.cuda.synchronize()
    ref = replica(xq, xs, wq, ws)
    want = torch.from_numpy(ref).to(DT[out])
    assert torch.equal(o.cpu(), want), f"{int((o.cpu() != want).sum())} of {M * N} differ"
    exact = (xq.astype(np.float64) @ wq.astype(np.float64).T) * xs.astype(np.float64)[:, None] * ws.astype(np.float64)
    tol = np.abs(exact) * 3.01 * 2.0 ** -24
    if out != "fp32":
        tol = tol + (np.abs(exact) + tol) * torch.finfo(DT[out]).eps / 2 + (2.0 ** -25 if out == "fp16" else 0)
    assert (np.abs(o.double().cpu().numpy() - exact) <= tol).all()
    keep = torch.ones_like(mem, dtype=torch.bool)
    keep[off:off + M * ld].view(M, ld)[:, :N] = False
    assert (mem[keep] == 1.5).all(), "wrote between the rows"


MATMUL = [(1, 1, 1, "fp32", None, 0), (1, 17, 130, "bf16", 20, 1), (3, 64, 128, "fp16", None, 0),
          (4, 2048, 256, "fp32", None, 0), (8, 5000, 4096, "fp32", None, 0), (16, 333, 3584, "bf16", 333, 1),
          (17, 1000, 512, "fp16", 1003, 1), (32, 4097, 640, "bf16", None, 0), (33, 257, 1000, "fp32", 260, 2),
          (60, 3000, 3584, "bf16", None, 0), (64, 129, 16384, "fp32", None, 0), (65, 130, 200, "bf16", None, 0),
          (100, 1000, 384, "fp16", None, 0), (128, 256, 128, "bf16", None, 0), (200, 4099, 1100, "bf16", 4099, 1),
          (255, 511, 4096, "fp32", None, 0), (257, 513, 129, "bf16", 515, 0), (513, 2049, 1280, "fp16", None, 0),
          (1000, 1536, 2048, "bf16", None, 0), (2049, 40, 777, "fp32", None, 0), (1, 70001, 300, "bf16", None, 0),
          # the stream of eight-row units and of taller ones, each token tile, ends inside a unit
          (9, 4097, 256, "bf16", 4099, 1), (20, 9001, 1000, "fp32", None, 0), (40, 16384, 384, "bf16", None, 0),
          (61, 5003, 129, "fp16", 5003, 1), (10, 16390, 512, "fp32", 16401, 3), (31, 17001, 300, "bf16", None, 0),
          (47, 20011, 128, "fp16", 20012, 0), (64, 33333, 640, "bf16", 33333, 1), (64, 16385, 2048, "fp32", None, 0),
          # up to 128 tokens over many channels
          (65, 65537, 128, "fp32", None, 0), (100, 70003, 384, "bf16", 70003, 1), (128, 66000, 256, "fp16", None, 0),
          # few channels: the sides change places
          (65, 1, 128, "fp32", None, 0), (300, 7, 200, "bf16", 9, 1), (1000, 64, 512, "fp32", 70, 1),
          (5000, 33, 384, "fp16", None, 0), (20000, 17, 256, "bf16", 17, 0)]


@pytest.mark.parametrize("c", MATMUL, ids=lambda c: "x".join(str(v) for v in c))
def test_quant_matmul(ns, c):
    check_matmul(ns, *c)


@pytest.mark.parametrize("M", [1, 40, 300])
def test_quant_matmul_largest_sums(ns, M):
    check_matmul(ns, M, 300, 16384, "fp32", extreme=True)


@pytest.mark.parametrize("M", [3, 150])
def test_quant_matmul_special_scales(ns, M):
    """NaN scales reach exactly their rows and columns; a type's overflow is infinite, as its own conversion gives."""
    N, d = 200, 256
    xq, wq = int8_rows(M, d, 1), int8_rows(N, d, 2)
    xs, ws = np.full(M, 0.5, np.float32), np.full(N, 0.25, np.float32)
    xs[1], ws[7], ws[9] = np.nan, np.nan, 1e6
    dev = lambda a: torch.from_numpy(a).cuda()
    for out in DT:
        o = torch.empty((M, N), dtype=DT[out], device="cuda")
        ns.nanospec_quant_matmul(dev(xq), dev(xs), dev(wq), dev(ws), d, o)
        want = torch.from_numpy(replica(xq, xs, wq, ws)).to(DT[out])
        torch.testing.assert_close(o.cpu(), want, rtol=0, atol=0, equal_nan=True)


# more than 64 tokens: groups of 64 for few channels (the last group of one
# token, or of 64), tiles of 128 and 256 tokens for more
GROUPS = [(65, 65, 128, "fp32", None, 0), (128, 100, 300, "bf16", 101, 1), (129, 2001, 130, "fp16", 2003, 1),
          (2305, 70, 200, "fp32", 75, 2), (8192, 80, 129, "bf16", None, 0), (321, 184, 9508, "bf16", 184, 1),
          (128, 5120, 256, "fp32", None, 0), (128, 5121, 256, "fp32", 5125, 1), (70, 6001, 1000, "bf16", 6001, 1),
          (127, 65535, 128, "fp16", None, 0), (640, 1030, 129, "fp32", 1033, 1), (129, 3905, 640, "bf16", None, 0),
          (8193, 81, 384, "fp16", None, 0), (20001, 65, 128, "bf16", 66, 1)]


# tiles of 64, 128 and 256 tokens, one a block and several, with sums of one, two, three and more stages
TILES = [(300, 70000, 128, "bf16", None, 0), (513, 33001, 100, "fp32", None, 0), (2049, 9000, 128, "fp16", 9001, 1),
         (1500, 12000, 256, "bf16", None, 0), (700, 20000, 384, "fp32", 20003, 3), (256, 16384, 128, "fp32", None, 0),
         (129, 20000, 300, "bf16", None, 0), (200, 60000, 200, "bf16", 60000, 0), (66, 17000, 640, "fp16", None, 0),
         (1000, 8000, 130, "fp32", None, 0), (4097, 4099, 64, "bf16", 4101, 1), (150, 150000, 128, "bf16", None, 0)]


@pytest.mark.parametrize("c", TILES, ids=lambda c: "x".join(str(v) for v in c))
def test_quant_matmul_rounds_of_tiles(ns, c):
    check_matmul(ns, *c)


@pytest.mark.parametrize("c", GROUPS, ids=lambda c: "x".join(str(v) for v in c))
def test_quant_matmul_groups_of_tokens(ns, c):
    check_matmul(ns, *c)


@pytest.mark.parametrize("M,N", [(100, 5500), (300, 4100)])
def test_quant_matmul_tiles_largest_sums_and_special_scales(ns, M, N):
    check_matmul(ns, M, N, 2048, "fp32", extreme=True)
    d = 200
    xq, wq = int8_rows(M, d, 1), int8_rows(N, d, 2)
    xs, ws = np.full(M, 0.5, np.float32), np.full(N, 0.25, np.float32)
    xs[1], xs[M - 1], ws[7], ws[N - 1], ws[9] = np.nan, np.inf, np.nan, 0.0, 1e6
    dev = lambda a: torch.from_numpy(a).cuda()
    with np.errstate(invalid="ignore", over="ignore"):
        want = torch.from_numpy(replica(xq, xs, wq, ws))
    for out in DT:
        o = torch.empty((M, N), dtype=DT[out], device="cuda")
        ns.nanospec_quant_matmul(dev(xq), dev(xs), dev(wq), dev(ws), d, o)
        torch.testing.assert_close(o.cpu(), want.to(DT[out]), rtol=0, atol=0, equal_nan=True)


def test_quant_no_rows(ns):
    z = lambda *s, t=torch.float32: torch.empty(s, dtype=t, device="cuda")
    ns.nanospec_quant_rows(z(0, 64), z(0, 128, t=torch.int8), z(0))
    ns.nanospec_quant_matmul(z(0, 128, t=torch.int8), z(0), z(5, 128, t=torch.int8), z(5), 64, z(0, 5))


# ---------------------------------------------------------------------------
# Restricted head
# ---------------------------------------------------------------------------
def head_case(B, n_max, M, d, V, dtype, seed, counts=None, holes=0.0, ids=True):
    rng = np.random.default_rng(seed)
    wq = int8_rows(V, d, seed)
    ws = (np.exp(0.3 * rng.standard_normal(V)) * 1e-3).astype(np.float32)
    h = torch.from_numpy(rng.standard_normal((B, M, d)).astype(np.float32)).to(DT[dtype])
    I = None
    if ids:
        I = np.stack([rng.permutation(V)[:n_max] for _ in range(B)]).astype(np.int32)
        I[rng.random(I.shape) < holes] = -1
        if holes:
            I[:, ::17] = V                                # past the vocabulary: holes too
    n = None if counts is None else np.asarray(counts, np.int32)
    return wq, ws, h, I, n


def check_head(ns, case, k, want_logits=True, work=None, what=""):
    wq, ws, h, I, n = case
    B, M, d = h.shape
    V = wq.shape[0]
    n_max = V if I is None else I.shape[1]
    say("quant_logits_topk", (B, M, d, V, n_max, k), what)
    dev = lambda a: None if a is None else torch.from_numpy(a).cuda()
    logits = torch.full((B, M, n_max), 1.5, device="cuda") if want_logits else None
    ids = torch.full((B, M, k), 77, dtype=torch.int32, device="cuda")
    vals = torch.full((B, M, k), 7.0, device="cuda")
    work = ns.alloc_quant_logits_workspace(B, n_max, M, k, d) if work is None else work
    ns.nanospec_quant_logits_topk(dev(wq), dev(ws), dev(I), dev(n), h.cuda(), k, logits, ids, vals, work)
    torch.cuda.synchronize()
    q, hs = quantised(h.double().numpy())
    for b in range(B):
        live = n_max if n is None else min(max(int(n[b]), 0), n_max)
        row = np.arange(n_max) if I is None else I[b]
        on = (np.arange(n_max) < live) & (row >= 0) & (row < V)
        z = replica(q[b], hs[b], wq[row[on]][:, :d], ws[row[on]])
        if want_logits:
            got = logits[b].cpu().numpy()
            assert np.array_equal(got[:, on], z, equal_nan=True), f"{what} b={b}: logits"
            assert (got[:, ~on] == 1.5).all(), f"{what} b={b}: wrote a dead column"
        for m in range(M):
            fine = ~np.isnan(z[m])
            v, g = z[m][fine], row[on][fine]
            order = np.lexsort((g, -(v + 0.0)))[:k]
            kk = len(order)
            gi, gv = ids[b, m].cpu().numpy(), vals[b, m].cpu().numpy()
            assert np.array_equal(gi[:kk], g[order]) and (gi[kk:] == -1).all(), f"{what} b={b} m={m}: ids"
            assert np.array_equal(gv[:kk], v[order]) and np.isneginf(gv[kk:]).all(), f"{what} b={b} m={m}: values"


HEADS = [
    # B, n_max, M, d, V, dtype, k, counts, holes, ids
    (1, 1, 1, 8, 5, "fp32", 1, None, 0.0, True),
    (1, 20, 3, 100, 50, "bf16", 5, [13], 0.0, True),
    (1, 16, 1, 64, 64, "fp16", 64, [0], 0.0, True),
    (1, 2048, 8, 4096, 5000, "bf16", 8, [1000], 0.0, True),
    (1, 1000, 60, 3584, 4000, "bf16", 10, [937], 0.1, True),
    (1, 1500, 17, 512, 3000, "fp32", 64, None, 0.3, True),
    (3, 700, 33, 264, 1000, "fp16", 20, [700, 1, 350], 0.0, True),
    (5, 130, 5, 1000, 400, "bf16", 7, [-3, 131, 64, 65, 999], 0.2, True),
    (1, 5000, 4, 256, 9000, "bf16", 16, [4999], 0.0, True),
    (1, 5000, 4, 256, 9000, "bf16", 16, [3000], 0.0, True),
    (2, 9000, 2, 128, 9000, "fp32", 64, [9000, 4097], 0.0, True),
    (1, 16384, 64, 640, 20000, "bf16", 16, [15500], 0.05, True),
    (1, 33000, 9, 192, 33000, "bf16", 3, None, 0.0, False),
    (20, 300, 8, 1024, 4000, "bf16", 8, list(range(100, 300, 10)), 0.0, True),
    (64, 96, 16, 384, 800, "fp16", 4, list(range(30, 94)), 0.0, True),
    (1, 64, 64, 16384, 100, "bf16", 8, [64], 0.0, True),
]


@pytest.mark.parametrize("c", HEADS, ids=lambda c: "x".join(str(v) if not isinstance(v, list) else "n" for v in c))
def test_quant_head(ns, c):
    B, n_max, M, d, V, dtype, k, counts, holes, ids = c
    case = head_case(B, n_max, M, d, V, dtype, 5, counts, holes, ids)
    check_head(ns, case, k, True, what=str(c))
    check_head(ns, case, k, False, what=str(c) + " no logits")


@pytest.mark.parametrize("n_max", [300, 6000])
def test_quant_head_ties_and_nan(ns, n_max):
    wq, ws, h, I, n = head_case(1, n_max, 6, 256, n_max + 10, "bf16", 7, [n_max])
    wq[:] = wq[0]                                         # every logit of a row ties
    ws[:] = 0.5
    ws[I[0, 5]] = np.nan                                  # but one that is no number
    h[0, 1] = 0
    h[0, 2, 3] = math.nan                                 # a hidden row that is none
    check_head(ns, (wq, ws, h, I, n), 20, what=f"ties n={n_max}")


@pytest.mark.parametrize("k", [33, 64])
@pytest.mark.parametrize("levels", [0, 3, 40])
def test_quant_head_many_candidates(ns, k, levels):
    """Counts around those where every logit is a candidate, where waves of them are merged, and where they no longer fit."""
    counts = [63, 64, 65, 100, 128, 129, 500, 513, 1000, 1008, 1009, 1023, 1024, 1025, 1100, 2000, 2200]
    wq, ws, h, I, n = head_case(len(counts), 2200, 3, 64, 2500, "bf16", 11, counts, holes=0.01)
    if levels:                                            # few different logits: many tie
        wq[:] = wq[np.arange(len(wq)) % levels]
        ws[:] = 0.5
    check_head(ns, (wq, ws, h, I, n), k, what=f"candidates k={k} levels={levels}")


def test_quant_head_reuses_a_workspace(ns):
    """A larger call's leavings in the workspace do not reach a smaller one."""
    big, small = head_case(1, 6000, 16, 512, 8000, "bf16", 1, [6000]), head_case(1, 40, 3, 128, 90, "bf16", 2, [33])
    work = ns.alloc_quant_logits_workspace(1, 6000, 16, 32, 512)
    work.fill_(0xFF)
    for case, k in ((big, 32), (small, 5), (big, 32)):
        check_head(ns, case, k, work=work, what="shared workspace")
