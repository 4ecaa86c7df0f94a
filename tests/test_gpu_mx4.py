"""4-bit rows against their definitions in 64 bits.

Scales, codes and the values read back are defined exactly and compared for
equality.  A product of two codes is a quarter of an integer, so where the
terms of a sum are multiples of a unit u and their magnitudes add up to less
than 2^24 u, float32 holds every partial sum and the product has to be the
exact sum rounded to the output type, whatever kernel took it; the tests of
equality check that of their inputs first.  Otherwise each matrix instruction
(128 elements) and each join of partial sums may be off by a step of float32's
24 bits and one more for the alignment of its terms, 2^-22 of the sum of the
magnitudes.
"""
import math

import numpy as np
import pytest
import torch

from tests.gpu_common import say

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
MAG = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


@pytest.fixture(scope="module")
def ns():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from dynamic_vocab_draft_amd import nanospec
    return nanospec


def pitch(d):
    return -(-d // 256) * 128


def blocks(x):
    x = np.pad(x, ((0, 0), (0, -x.shape[1] % 32)))
    return x.reshape(x.shape[0], -1, 32)


def quantised(x):
    """(codes [R, blocks, 32], scale bytes [R, blocks]) of float64 rows, from the definition."""
    b = blocks(x)
    bad = ~np.isfinite(b).all(-1)
    a = np.abs(np.where(bad[..., None], 0, b)).max(-1)
    e = np.maximum(np.frexp(a)[1] - 3, -127)
    e[a == 0] = -127
    y = np.abs(np.where(bad[..., None], 0, b)) / np.ldexp(1.0, e)[..., None]
    code = np.zeros(y.shape, int)
    best = np.abs(y - MAG[0])
    for c in range(1, 8):                             # the nearest, ties to the even code
        off = np.abs(y - MAG[c])
        better = (off < best) | ((off == best) & (c % 2 == 0))
        code, best = np.where(better, c, code), np.where(better, off, best)
    code[y >= 6] = 7
    code += 8 * (np.signbit(b) & ~bad[..., None])
    return code, np.where(bad, 255, e + 127)


def packed(code, scale, d):
    """Codes and scale bytes as they are stored."""
    q = np.zeros((len(code), 2 * pitch(d)), np.uint8)
    q[:, :code.shape[1] * 32] = code.reshape(len(code), -1)
    s = np.zeros((len(code), pitch(d) // 16), np.uint8)
    s[:, :scale.shape[1]] = scale
    return q[:, ::2] | q[:, 1::2] << 4, s


def values(q, s, d):
    """What stored rows stand for, in float64."""
    c = np.stack([q & 15, q >> 4], -1).reshape(len(q), -1).astype(int)
    v = np.where(c >= 8, -MAG[c & 7], MAG[c & 7]).reshape(len(q), -1, 32)
    unit = np.where(s == 255, np.nan, np.ldexp(1.0, s.astype(int) - 127))
    return (v * unit[..., None]).reshape(len(q), -1)[:, :d]


def run_rows(ns, x):
    R, d = x.shape
    q = torch.full((R, pitch(d)), 0x99, dtype=torch.uint8, device="cuda")
    s = torch.full((R, pitch(d) // 16), 7, dtype=torch.uint8, device="cuda")
    ns.nanospec_mx4_rows(x, q, s)
    return q, s


def positive_zeros(q):
    """Codes with -0 as +0: a negative element rounded to zero may keep its sign."""
    lo, hi = q & 15, q >> 4
    return np.where(lo == 8, 0, lo) | np.where(hi == 8, 0, hi) << 4


def check_rows(ns, x, what):
    say("mx4_rows", what)
    d = x.shape[1]
    q, s = run_rows(ns, x)
    rq, rs = packed(*quantised(x.double().cpu().numpy()), d)
    assert np.array_equal(s.cpu().numpy(), rs), f"{what}: {int((s.cpu().numpy() != rs).sum())} scales differ"
    got = q.cpu().numpy()
    assert np.array_equal(positive_zeros(got), positive_zeros(rq)), f"{what}: {int((got != rq).sum())} bytes differ"
    for name, t in DT.items():                         # read back, in each type
        out = torch.full((x.shape[0], d + 3), 5.0, dtype=t, device="cuda")
        ns.nanospec_mx4_gather_rows(q, s, None, None, out[:, :d])
        want = torch.from_numpy(values(rq, rs, d)).to(t)
        torch.cuda.synchronize()
        assert torch.equal(out[:, :d].cpu().nan_to_num(nan=12345.0), want.nan_to_num(nan=12345.0)), f"{what}: values as {name}"
        assert (out[:, d:] == 5).all(), f"{what}: elements between rows"


ROWS = [(1, 1, "fp32", 1, 0), (3, 2, "bf16", 3, 1), (5, 8, "fp16", 8, 0), (7, 31, "bf16", 33, 1), (4, 33, "fp32", 33, 0),
        (7, 127, "bf16", 127, 0), (4, 256, "fp32", 259, 1), (9, 257, "fp16", 257, 1), (8, 4096, "bf16", 4096, 0),
        (60, 3584, "bf16", 3600, 0), (33, 4096, "fp32", 4096, 0), (5, 4104, "fp16", 4104, 0), (2, 16384, "fp32", 16384, 0),
        (3, 16383, "fp16", 16383, 1), (3001, 250, "bf16", 250, 0), (1000, 1000, "fp32", 1000, 0), (70, 8191, "bf16", 8200, 0)]


@pytest.mark.parametrize("c", ROWS, ids=lambda c: "x".join(str(v) for v in c))
def test_rows(ns, c):
    R, d, dtype, ld, off = c
    rng = np.random.default_rng(R + d)
    mem = torch.zeros(R * ld + off + 8, dtype=DT[dtype], device="cuda")
    x = mem[off:off + R * ld].view(R, ld)[:, :d]
    x.copy_(torch.from_numpy(rng.standard_normal((R, d)).astype(np.float32)).to(DT[dtype]))
    check_rows(ns, x, str(c))


@pytest.mark.parametrize("dtype", DT)
def test_rows_at_borders(ns, dtype):
    """Every half step of the grid and its neighbours, at several scales; zeros, subnormal, largest, infinite and NaN blocks."""
    t = DT[dtype]
    top = {"bf16": 120, "fp16": 12, "fp32": 120}[dtype]
    low = {"bf16": -130, "fp16": -20, "fp32": -140}[dtype]
    rows = []
    for e in (low, low + 3, -3, 0, 1, 7, top):
        for first in (4.0, 6.0, 7.75):
            x = [first] + [k * 0.25 for k in range(31)]
            rows.append(torch.tensor(x, dtype=torch.float64) * 2.0 ** e)
    x = torch.stack(rows).to(t)
    nudged = [x, -x]
    bits = x.view(torch.int16 if x.element_size() == 2 else torch.int32)
    for step in (1, -1):
        n = bits + step
        n = torch.where(bits == 0, bits, n).view(t)
        n[:, 0] = x[:, 0]
        nudged.append(n)
    x = torch.cat(nudged, 0)
    x = torch.cat([x, x.roll(5, 0)], 1)
    big = torch.finfo(t).max
    extra = torch.zeros((9, 64), dtype=t)
    extra[1, 3], extra[2, 40], extra[3, 0], extra[4, 63] = math.inf, -math.inf, math.nan, -math.nan
    extra[5] = big
    extra[6, :32] = torch.finfo(t).smallest_normal
    extra[7] = torch.finfo(t).smallest_normal * torch.finfo(t).eps          # the smallest subnormal
    extra[8] = -0.0
    check_rows(ns, torch.cat([x, extra.to(t)], 0).cuda(), dtype)


def test_read_back_by_ids(ns):
    V, d, n = 50, 300, 40
    rng = np.random.default_rng(5)
    q, s = run_rows(ns, torch.from_numpy(rng.standard_normal((V, d)).astype(np.float32)).cuda())
    ids = rng.integers(0, V, n).astype(np.int32)
    ids[3], ids[7], ids[11] = -1, V, 2 ** 30
    whole = values(q.cpu().numpy(), s.cpu().numpy(), d)
    for live, kept in ((None, n), (25, 25), (0, 0), (-4, 0), (1000, n)):
        out = torch.full((n, d), 9.0, device="cuda")
        ns.nanospec_mx4_gather_rows(q, s, torch.from_numpy(ids).cuda(), None if live is None else torch.tensor([live], dtype=torch.int32, device="cuda"), out)
        want = np.full((n, d), 9.0)
        for j in range(kept):
            if 0 <= ids[j] < V:
                want[j] = whole[ids[j]]
        assert np.array_equal(out.cpu().numpy().astype(np.float64), want), live


# ---------------------------------------------------------------------------
# Product
# ---------------------------------------------------------------------------
def made(rng, n, d, spread=1):
    """Stored rows of n normal rows, blocks' scales up to 2^spread apart beside what the values need."""
    x = rng.standard_normal((n, d)) * np.exp(0.3 * rng.standard_normal((n, 1)))
    if spread > 1:
        x = x * np.repeat(2.0 ** rng.integers(0, spread, (n, -(-d // 32))), 32, 1)[:, :d]
    return packed(*quantised(x), d)


def on_gpu(*arrays):
    return [torch.from_numpy(a).cuda() for a in arrays]


def exact_in_float32(a, b, total):
    """Where float32 holds every partial sum of a product: a value's two bits end at a unit of its own, a block's terms are
    multiples of the units of its two halves, and the sum of those of the smallest."""
    def units(v):
        v = blocks(v)
        return np.min(np.where(v == 0, np.inf, np.ldexp(1.0, np.frexp(v)[1] - 2)), axis=2)
    ua, ub = units(a), units(b)
    with np.errstate(all="ignore"):
        unit = ua.min(1)[:, None] * ub.min(1)
        sure = (total == 0) | (total < 2.0 ** 24 * unit)
    if sure.all():
        return sure
    unit = np.full(total.shape, np.inf)
    for k in range(ua.shape[1]):
        np.minimum(unit, ua[:, k, None] * ub[:, k], out=unit)
    with np.errstate(all="ignore"):
        return (total == 0) | (total < 2.0 ** 24 * unit)


def check_product(ns, M, N, d, dtype, seed=0, ld=None, spread=1, exact=True):
    say("mx4_matmul", M, N, d, dtype)
    rng = np.random.default_rng(seed + M + N + d)
    (xq, xs), (wq, ws) = made(rng, M, d, spread), made(rng, N, d, spread)
    a, b = values(xq, xs, d), values(wq, ws, d)
    want, total = a @ b.T, np.abs(a) @ np.abs(b).T
    ld = ld or N
    mem = torch.full((M, ld), 3.0, dtype=DT[dtype], device="cuda")
    ns.nanospec_mx4_matmul(*on_gpu(xq, xs, wq, ws), d, mem[:, :N])
    torch.cuda.synchronize()
    assert (mem[:, N:] == 3).all(), "elements between rows"
    got = mem[:, :N].cpu()
    bound = (2 * -(-d // 256) + 8) * 2.0 ** -22 * total + torch.finfo(DT[dtype]).eps / 2 * np.abs(want)
    assert (np.abs(got.double().numpy() - want) <= bound).all()
    if exact:                                          # but for rows whose last block holds next to nothing
        at = torch.from_numpy(exact_in_float32(a, b, total))
        assert at.double().mean() > 0.9, "inputs that float32 does not sum exactly"
        assert torch.equal(got[at], torch.from_numpy(want).float().to(DT[dtype])[at])


PRODUCTS = [(1, 1, 1, "fp32"), (1, 5, 31, "bf16"), (2, 16, 33, "fp16"), (4, 2048, 256, "fp32"), (3, 17, 257, "fp32"),
            (16, 33, 512, "bf16"), (17, 100, 1000, "fp32"), (8, 5000, 4096, "fp32"), (33, 1000, 3584, "bf16"),
            (48, 16500, 300, "fp16"), (60, 4097, 1024, "bf16"), (64, 300, 16384, "fp32"), (65, 257, 700, "fp32"),
            (100, 40, 5000, "bf16"), (129, 1025, 640, "fp16"), (257, 700, 128, "fp32"), (300, 2049, 2000, "bf16"),
            (1000, 513, 96, "bf16"), (520, 1, 512, "fp32"), (1, 20001, 2048, "bf16")]


@pytest.mark.parametrize("c", PRODUCTS, ids=lambda c: "x".join(str(v) for v in c))
def test_product(ns, c):
    check_product(ns, *c)


@pytest.mark.parametrize("c", [(5, 40, 500), (20, 300, 4096), (70, 300, 3000), (200, 1000, 1500)], ids=lambda c: "x".join(str(v) for v in c))
def test_product_of_scales_far_apart(ns, c):
    check_product(ns, *c, "fp32", spread=40, exact=False)


@pytest.mark.parametrize("c", [(3, 70, 300, 71), (40, 900, 513, 1000), (130, 600, 512, 601)], ids=lambda c: "x".join(str(v) for v in c))
@pytest.mark.parametrize("dtype", DT)
def test_product_into_strided_rows(ns, c, dtype):
    check_product(ns, *c[:3], dtype, ld=c[3])


@pytest.mark.parametrize("M,N", [(3, 40), (60, 5000), (200, 600)])
def test_block_of_nan(ns, M, N):
    d = 700
    rng = np.random.default_rng(M)
    (xq, xs), (wq, ws) = made(rng, M, d), made(rng, N, d)
    xs[1, 5], ws[N - 2, 21] = 255, 255
    out = torch.zeros((M, N), device="cuda")
    ns.nanospec_mx4_matmul(*on_gpu(xq, xs, wq, ws), d, out)
    bad = np.zeros((M, N), bool)
    bad[1], bad[:, N - 2] = True, True
    assert np.array_equal(torch.isnan(out).cpu().numpy(), bad)


def test_smallest_and_largest_scales(ns):
    """Scales 2^-127 and 2^127 meet as 1; two of either leave float32's range at both ends."""
    d = 256
    one = np.full((1, d // 2), 0x22, np.uint8)             # 1.0 everywhere
    s = lambda v: np.full((1, 8), v, np.uint8)             # noqa: E731
    for a, b, want in ((0, 254, float(d)), (254, 0, float(d)), (254, 254, math.inf), (0, 0, 0.0), (127, 127, float(d)), (0, 127 + 40, d * 2.0 ** -87)):
        out = torch.full((1, 1), 3.0, device="cuda")
        ns.nanospec_mx4_matmul(*on_gpu(one, s(a), one, s(b)), d, out)
        assert out.item() == want, (a, b, out.item())


def test_nothing_to_do(ns):
    d = 64
    w = torch.zeros((4, pitch(d)), dtype=torch.uint8, device="cuda")
    ws = torch.zeros((4, pitch(d) // 16), dtype=torch.uint8, device="cuda")
    ns.nanospec_mx4_rows(torch.empty((0, d), device="cuda"), w[:0], ws[:0])
    ns.nanospec_mx4_matmul(w[:0], ws[:0], w, ws, d, torch.empty((0, 4), device="cuda"))
    ns.nanospec_mx4_gather_rows(w, ws, None, None, torch.empty((0, d), device="cuda"))
    torch.cuda.synchronize()


# ---------------------------------------------------------------------------
# Restricted head
# ---------------------------------------------------------------------------
def best_of(z, ids, k):
    """Top-k by (value desc, id asc), padded; NaN never selected."""
    oi, ov = np.full((len(z), k), -1), np.full((len(z), k), -np.inf)
    for m, row in enumerate(z):
        keep = ~np.isnan(row)
        order = np.lexsort((ids[keep], -row[keep]))[:k]
        oi[m, :len(order)], ov[m, :len(order)] = ids[keep][order], row[keep][order]
    return oi, ov


def check_head(ns, B, M, k, n_max, V, d, dtype, live=None, holes=0, all_rows=False, logits=True, seed=0):
    say("mx4_logits_topk", B, M, k, n_max, V, d, dtype)
    rng = np.random.default_rng(seed + B + M + k + n_max + d)
    wq, ws = made(rng, V, d)
    h = torch.from_numpy(rng.standard_normal((B, M, d)).astype(np.float32)).to(DT[dtype])
    if all_rows:
        ids = np.broadcast_to(np.arange(n_max), (B, n_max)).astype(np.int32)
    else:
        ids = np.stack([np.sort(rng.permutation(V)[:n_max]) for _ in range(B)]).astype(np.int32)
        for b in range(B):
            ids[b, rng.permutation(n_max)[:holes]] = rng.choice([-1, V, 2 ** 31 - 1], holes)
    n = np.full(B, n_max) if live is None else np.asarray(live)
    z = torch.full((B, M, n_max), 77.0, device="cuda") if logits else None
    oi = torch.full((B, M, k), -9, dtype=torch.int32, device="cuda")
    ov = torch.zeros((B, M, k), device="cuda")
    work = ns.alloc_mx4_logits_workspace(B, n_max, M, k, d)
    work.fill_(0xFF)
    gq, gs = on_gpu(wq, ws)
    ns.nanospec_mx4_logits_topk(gq, gs, None if all_rows else torch.from_numpy(ids).cuda(), None if live is None else torch.tensor(n, dtype=torch.int32, device="cuda"),
                                h.cuda(), k, z, oi, ov, work)
    torch.cuda.synchronize()
    w = values(wq, ws, d)
    for b in range(B):
        hq, hs = packed(*quantised(h[b].double().numpy()), d)
        x = values(hq, hs, d)
        nb = int(np.clip(n[b], 0, n_max))
        ok = np.flatnonzero((ids[b, :nb] >= 0) & (ids[b, :nb] < V))
        rows = w[ids[b, ok]]
        want, total = x @ rows.T, np.abs(x) @ np.abs(rows).T
        sure = exact_in_float32(x, rows, total) if len(ok) else np.ones(want.shape, bool)
        assert logits or sure.all()
        if logits:
            got = z[b].cpu().numpy()
            assert np.array_equal(got[:, ok][sure], want.astype(np.float32)[sure]), b
            assert sure.size == 0 or sure.mean() > 0.9
            bound = (2 * -(-d // 256) + 8) * 2.0 ** -22 * total + 2.0 ** -24 * np.abs(want)
            assert (np.abs(got[:, ok] - want) <= bound).all()
            want = np.where(sure, want, got[:, ok])        # the selection is held to the logits as they are
            rest = np.setdiff1d(np.arange(n_max), ok)
            assert (got[:, rest] == 77).all(), "columns that are no rows"
        ri, rv = best_of(want.astype(np.float32), ids[b, ok], k)
        assert np.array_equal(oi[b].cpu().numpy(), ri) and np.array_equal(ov[b].cpu().numpy(), rv.astype(np.float32)), b


HEADS = [(1, 1, 1, 1, 5, 32, "fp32"), (1, 8, 8, 1000, 3000, 256, "bf16"), (2, 3, 5, 37, 200, 100, "fp16"), (1, 17, 64, 500, 600, 264, "bf16"),
         (3, 64, 16, 300, 900, 1000, "fp32"), (1, 16, 8, 900, 1000, 4096, "bf16"), (1, 8, 8, 700, 1000, 4104, "fp16"), (1, 2, 8, 100, 300, 16384, "bf16"),
         (5, 40, 3, 2100, 3000, 128, "bf16"), (1, 64, 64, 9000, 12000, 300, "bf16"), (2, 16, 10, 20000, 21000, 64, "fp16"), (40, 4, 8, 450, 800, 512, "bf16")]


@pytest.mark.parametrize("c", HEADS, ids=lambda c: "x".join(str(v) for v in c))
def test_head(ns, c):
    check_head(ns, *c)


def test_head_live_counts_and_holes(ns):
    check_head(ns, 6, 8, 8, 400, 900, 512, "bf16", live=[0, 1, 399, -3, 10 ** 6, 17], holes=40)
    check_head(ns, 4, 33, 8, 3000, 4000, 300, "bf16", live=[0, 2999, 5, 16], holes=100, logits=False)


@pytest.mark.parametrize("M", [4, 50])
def test_head_over_all_rows(ns, M):
    check_head(ns, 1, M, 8, 2500, 2500, 300, "fp32", all_rows=True)
    check_head(ns, 2, M, 8, 100, 100, 300, "fp32", all_rows=True, logits=False)


def test_head_of_a_nan_hidden_row(ns):
    V, d, k = 100, 64, 4
    rng = np.random.default_rng(1)
    wq, ws = on_gpu(*made(rng, V, d))
    h = torch.randn((1, 3, d), device="cuda")
    h[0, 1, 40] = math.nan
    oi, ov = torch.zeros((1, 3, k), dtype=torch.int32, device="cuda"), torch.zeros((1, 3, k), device="cuda")
    ns.nanospec_mx4_logits_topk(wq, ws, None, None, h, k, None, oi, ov, ns.alloc_mx4_logits_workspace(1, V, 3, k, d))
    assert (oi[0, 1] == -1).all() and (ov[0, 1] == -math.inf).all() and (oi[0, ::2] >= 0).all()


def test_ties_go_to_the_lowest_id(ns):
    V, d, k = 5000, 256, 64
    wq, ws = run_rows(ns, torch.ones((V, d), device="cuda"))
    ids = torch.arange(V - 1, -1, -1, dtype=torch.int32, device="cuda")[None].contiguous()
    oi, ov = torch.zeros((1, 2, k), dtype=torch.int32, device="cuda"), torch.zeros((1, 2, k), device="cuda")
    ns.nanospec_mx4_logits_topk(wq, ws, ids, None, torch.ones((1, 2, d), device="cuda"), k, None, oi, ov, ns.alloc_mx4_logits_workspace(1, V, 2, k, d))
    assert (oi.cpu() == torch.arange(k)).all() and (ov == d).all()
