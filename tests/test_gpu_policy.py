"""The clipped policy loss and its gradient against the definition in float64.

Tolerances, with u = 2^-24 (half a step of float32).  A row's S is a float32
sum: terms that matter have |y| <= 24, so y's rounding costs at most ln2 24 u,
exp2 2 u, and the chain of additions (batches of 32, a lane's batches, lanes,
waves, parts) under 60 u: S is within 80 u, and so is a log-probability before
it is rounded (u of its size).  A ratio and exp(delta) are within that
relatively, losses and gradients follow by their formulas; W / S, at most some
24 + log2 V in size, costs the entropy twice as much of 1 + log V.
"""
import math

import numpy as np
import pytest
import torch

from tests.gpu_common import say

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = 2.0 ** -24


@pytest.fixture(scope="module")
def ns():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from dynamic_vocab_draft_amd import nanospec
    return nanospec


class Case:
    """Inputs of one call; everything a row has beside its logits in numpy."""

    def __init__(self, L, V, dtype="fp32", t=1.0, lo=0.2, hi=0.28, beta=0.05, ent=0.01, seed=0, scale=3.0, ld=None, off=0):
        rng = np.random.default_rng(seed + L + V)
        self.L, self.V, self.dtype, self.t, self.lo, self.hi, self.beta, self.ent = L, V, dtype, np.float32(t), lo, hi, beta, ent
        self.ld, self.off = ld or V, off
        self.tokens = rng.integers(0, V, L).astype(np.int32)
        z = scale * rng.standard_normal((L, V))
        z[np.arange(L), self.tokens] += 3 * scale
        self.z = torch.from_numpy(z).to(DT[dtype])
        self.advantage = rng.standard_normal(L).astype(np.float32)
        self.weight = (rng.random(L) / L + 0.1 / L).astype(np.float32)
        self.g_loss = np.float32(0.75)
        logp = self.logp()
        moved = 0.25 * rng.standard_normal(L)
        for border in (math.log(1 - lo) if lo < 1 else -1e9, math.log(1 + hi)):
            near = moved - border                      # at a border the gradient jumps
            moved = np.where(np.abs(near) < 1e-3, border + np.where(near < 0, -1e-3, 1e-3), moved)
        seen = np.where(np.isfinite(logp), logp, -2.0)
        self.old = (seen - moved).astype(np.float32)
        self.ref = (seen + 0.3 * rng.standard_normal(L)).astype(np.float32) if beta else None

    def rows(self):
        with np.errstate(all="ignore"):
            z = self.z.double().numpy() * float(self.t)
            top = z.max(1, keepdims=True)
            top = np.where(np.isfinite(top), top, 0.0)
            lse = np.log(np.exp(z - top).sum(1, keepdims=True)) + top
            every = np.where(np.isneginf(lse), -np.inf, z - lse)
        return every

    def logp(self):
        return self.rows()[np.arange(self.L), np.clip(self.tokens, 0, self.V - 1)]

    def want(self):
        """Outputs and tolerances."""
        L, V = self.L, self.V
        every = self.rows()
        w = np.ones(L) if self.weight is None else self.weight.astype(np.float64)
        taken = (self.tokens >= 0) & (self.tokens < V) & (w != 0)
        tok = np.clip(self.tokens, 0, V - 1)
        logp = every[np.arange(L), tok]
        bad = taken & ~(every <= 1e-6).all(1)
        learns = taken & ~bad & (logp > -104)
        with np.errstate(all="ignore"):
            p = np.exp(every)
            p = np.where(np.isnan(p) & ~bad[:, None], 0, p)
            H = -np.where(p > 0, p * every, 0).sum(1)
            A = np.where(learns, self.advantage, 0).astype(np.float64)
            r = np.exp(np.where(learns, logp - self.old, 0))
            over, under = (A > 0) & (r > 1 + np.float32(self.hi)), (A < 0) & (r < 1 - np.float32(self.lo))
            gain = np.where(over, (1 + float(np.float32(self.hi))) * A, np.where(under, (1 - float(np.float32(self.lo))) * A, r * A))
            slope = np.where(over | under, 0, r * A)
            back, kl = np.ones(L), np.zeros(L)
            if self.ref is not None:
                delta = np.where(learns, self.ref - logp, 0)
                back, kl = np.exp(delta), np.expm1(delta) - delta
        b, e = float(np.float32(self.beta)), float(np.float32(self.ent))
        wl = np.where(learns, w, 0)
        rows = wl * (-gain + b * kl - e * H)
        g = wl * (-slope + b * (1 - back))
        H = np.where(taken, H, 0)
        one = np.zeros((L, V))
        one[np.arange(L), tok] = 1
        up = float(self.g_loss) * float(self.t)
        with np.errstate(all="ignore"):
            inner = np.where(p > 0, every + H[:, None], 0)
            dz = up * (g[:, None] * (one - p) + (wl * e)[:, None] * p * inner)
        dz[~learns] = 0
        tl = 80 * U
        tH = 160 * U * (1 + math.log(V))
        trow = np.abs(wl) * (np.abs(slope) * tl * 1.01 + b * np.abs(back - 1) * tl * 1.01 + b * back * tl ** 2 + abs(e) * tH)
        tg = np.abs(wl) * (np.abs(slope) + b * back) * tl * 1.01 + 4 * U * np.abs(g)
        off = np.where(p > 0, np.abs(every), 0) * 2 * U + tl + 8 * U      # relative error of p_j: its own y and S
        tdz = up * (tg[:, None] * (one + p) + np.abs(g)[:, None] * p * off +
                    (wl * abs(e))[:, None] * p * (np.abs(inner) * off + tH + tl + 4 * U * np.abs(every, where=p > 0, out=np.zeros_like(p))))
        # the exponential instruction gives 0 for what lies below 2^-126, the smallest normal number: p_j is off by that much
        # at most there (S >= 1), and p_j |logp_j + H| by 2^-126 (126 ln2 + log V), since x |log x| falls with x
        tdz += up * (np.abs(g) + np.abs(wl * e) * 140)[:, None] * 2.0 ** -126
        t = DT[self.dtype]
        with np.errstate(all="ignore"):
            tdz = tdz * 1.1 + torch.finfo(t).eps / 2 * np.abs(dz) + torch.finfo(t).smallest_normal * torch.finfo(t).eps
        logp_out = np.where(taken, logp, 0)
        out = {"loss": (np.array([rows.sum()]), np.array([trow.sum() + U * abs(rows.sum()) * 2])),
               "logprob": (logp_out, np.where(np.isfinite(logp_out), tl + U * np.abs(logp_out), 0)),
               "entropy": (H, tH + U * H),
               "dlogits": (dz, tdz)}
        if self.ref is not None:
            out["kl"] = (np.where(learns, kl, 0), np.abs(back - 1) * tl * 1.01 + back * tl ** 2 + 2 * U * kl)
        for name, (v, tol) in out.items():
            if bad.any():
                if name == "loss":
                    v[:] = np.nan
                else:
                    v[bad] = np.nan
        return out

    def device_rows(self, dtype=None):
        mem = torch.full((self.L * self.ld + self.off + 8,), 9.0, dtype=DT[self.dtype], device="cuda")
        z = mem[self.off:self.off + self.L * self.ld].view(self.L, self.ld)[:, :self.V]
        z.copy_(self.z)
        return mem, z

    def arguments(self):
        c = lambda a: None if a is None else torch.from_numpy(a).cuda()   # noqa: E731
        return [c(self.tokens), c(self.old), c(self.ref), c(self.advantage), c(self.weight), self.lo, self.hi, self.beta, self.ent]

    def outputs(self):
        new = lambda: torch.full((self.L,), 55.0, device="cuda")   # noqa: E731
        return {"loss": torch.full((1,), 55.0, device="cuda"), "logprob": new(), "kl": new() if self.ref is not None else None, "entropy": new()}


def workspace(ns, L, V):
    work = ns.alloc_policy_loss_workspace(L, V)
    return work.fill_(0xFF)


def near(got, want, tol, what):
    got = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN"
    assert np.array_equal(np.isinf(got), np.isinf(want)) and (got[np.isinf(want)] == want[np.isinf(want)]).all(), f"{what}: infinities"
    fine = np.isfinite(want)
    off = np.abs(np.where(fine, got, 0) - np.where(fine, want, 0))
    tol = np.broadcast_to(tol, want.shape)
    worst = np.unravel_index(np.argmax(np.where(fine, off - tol, -1)), want.shape)
    assert (off[fine] <= tol[fine]).all(), f"{what}: {got[worst]} for {want[worst]} at {worst}, tolerance {tol[worst]}"


def check(ns, case, grad=True, inplace=False, what=""):
    say("policy_loss", case.L, case.V, case.dtype, what)
    want = case.want()
    mem, z = case.device_rows()
    out = case.outputs()
    dmem, dz = (mem, z) if inplace else case.device_rows()
    if not inplace:
        dmem.fill_(9.0)
    ns.nanospec_policy_loss(z, float(case.t), *case.arguments(), out["loss"], out["logprob"], out["kl"], out["entropy"],
                            torch.tensor([case.g_loss], device="cuda"), dz if grad else None, workspace(ns, case.L, case.V))
    torch.cuda.synchronize()
    for name in ("loss", "logprob", "kl", "entropy"):
        if out[name] is not None:
            near(out[name], *want[name], name)
    if grad:
        near(dz, *want["dlogits"], "dlogits")
        dz.fill_(9.0)
        assert (dmem == 9).all(), "elements between rows"
    return out


SHAPES = [(1, 1), (2, 2), (3, 7), (1, 8), (5, 9), (4, 64), (7, 1000), (3, 4097), (2, 50257), (70, 5003), (300, 2048), (1, 128256), (5, 151936), (1100, 600)]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_shapes(ns, shape, dtype):
    c = Case(*shape, dtype, t=0.7 if shape[1] % 2 else 1.0)
    check(ns, c)
    check(ns, c, grad=False)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("c", [(5, 1000, 1003, 1), (3, 4001, 4001, 3), (260, 513, 520, 0), (2, 70001, 70001, 1)], ids=lambda c: "x".join(map(str, c)))
def test_strides_and_in_place(ns, c, dtype):
    L, V, ld, off = c
    check(ns, Case(L, V, dtype, ld=ld, off=off), inplace=True)
    check(ns, Case(L, V, dtype, ld=ld, off=off, seed=3))


def test_terms_apart(ns):
    for beta, ent, lo, hi in ((0.0, 0.0, 0.2, 0.2), (0.3, 0.0, 0.2, 0.2), (0.0, 0.5, 0.2, 0.2), (0.1, -0.2, 0.0, 0.0), (0.1, 0.0, 1.0, math.inf)):
        check(ns, Case(40, 700, beta=beta, ent=ent, lo=lo, hi=hi), what=str((beta, ent, lo, hi)))
    c = Case(40, 700)
    c.weight = None
    check(ns, c, what="no weights")
    c = Case(6, 300)
    c.g_loss = np.float32(0)
    check(ns, c, what="g_loss 0")


def test_optional_outputs(ns):
    c = Case(30, 900)
    z = c.device_rows()[1]
    full, part = c.outputs(), c.outputs()
    ns.nanospec_policy_loss(z, 1.0, *c.arguments(), full["loss"], full["logprob"], full["kl"], full["entropy"], None, None, workspace(ns, 30, 900))
    ns.nanospec_policy_loss(z, 1.0, *c.arguments(), part["loss"], part["logprob"], None, None, None, None, workspace(ns, 30, 900))
    assert torch.equal(full["loss"], part["loss"]) and torch.equal(full["logprob"], part["logprob"])


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("shape", [(12, 900), (9, 40001)], ids=lambda s: "x".join(map(str, s)))
def test_masks_and_rows_left_out(ns, shape, dtype):
    L, V = shape
    c = Case(L, V, dtype)
    lowest = torch.finfo(DT[dtype]).min
    c.z[:, 1::3] = -math.inf
    c.z[:, 2::3] = lowest
    c.tokens[:] = c.tokens // 3 * 3
    c.z[np.arange(L), c.tokens] = 4.0
    c.tokens[1] = 1                            # a token that the mask rules out
    c.tokens[2] = 2                            # and one ruled out by the type's lowest value
    c.z[3] = -math.inf                         # a row that leaves nothing
    c.tokens[4], c.tokens[5] = -1, V           # padding
    c.z[4], c.z[5] = math.nan, math.inf        # whose logits may be anything
    c.weight[6] = 0
    c.z[6] = math.nan
    c.old[6], c.advantage[6] = math.nan, math.inf
    logp = c.logp()
    c.old = np.where(np.isfinite(logp) & (logp > -104), logp - 0.1, np.where(c.weight == 0, np.nan, -2)).astype(np.float32)
    c.ref = np.where(np.isfinite(logp) & (logp > -104), logp + 0.2, -2).astype(np.float32)
    check(ns, c)
    check(ns, c, inplace=True)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("V", [900, 30001])
def test_rows_without_a_distribution(ns, V, dtype):
    for what, value in (("nan", math.nan), ("inf", math.inf)):
        c = Case(5, V, dtype)
        c.z[2, V - 1] = value
        c.z[3, 0] = value
        check(ns, c, what=what)


@pytest.mark.parametrize("shift", [-3e4, 900.0, 3e4])
def test_shifted_logits(ns, shift):
    """Logits far from zero: multiples of 1/64, so that the shift takes none of their digits."""
    c = Case(6, 3000)
    z = torch.round(c.z.double() * 64) / 64
    c.z = (z + shift).float()
    assert torch.equal(c.z.double() - shift, z)
    logp = c.logp()
    c.old, c.ref = (logp - 0.1).astype(np.float32), (logp + 0.2).astype(np.float32)
    check(ns, c)


@pytest.mark.parametrize("t", [2.0 ** -20, 0.01, 30.0, 2.0 ** 20])
def test_temperatures(ns, t):
    c = Case(6, 3000, t=t)
    if t > 100:                                # p is 0 or 1 then: the token is the largest
        c.z[np.arange(6), c.tokens] = 40.0
    logp = c.logp()
    c.old, c.ref = (logp - 0.1).astype(np.float32), (logp + 0.2).astype(np.float32)
    check(ns, c)


def test_gradient_against_differences(ns):
    """Central differences of the definition's loss in float64."""
    c = Case(4, 40, beta=0.2, ent=0.3)
    c.tokens[2] = -1
    c.g_loss = np.float32(1)
    tol = c.want()["dlogits"][1]
    z = c.device_rows()[1]
    out, dz = c.outputs(), torch.zeros((4, 40), device="cuda")
    ns.nanospec_policy_loss(z, 1.0, *c.arguments(), out["loss"], out["logprob"], out["kl"], out["entropy"], None, dz, workspace(ns, 4, 40))
    got = dz.double().cpu().numpy()
    base, h = c.z.double(), 1e-5
    for i in range(4):
        for j in range(40):
            side = []
            for s in (h, -h):
                c.z = base.clone()
                c.z[i, j] += s
                side.append(c.want()["loss"][0][0])
            slope = (side[0] - side[1]) / (2 * h)
            # the difference's own error: h^2 / 6 of a third derivative of some units, and the sums' last digits over h
            assert abs(got[i, j] - slope) <= 1e-9 + tol[i, j], (i, j)


def test_same_bits_again(ns):
    for shape in ((3, 70000), (600, 3001)):
        c = Case(*shape, "bf16")
        z = c.device_rows()[1]
        got = []
        for _ in range(3):
            out, dz = c.outputs(), torch.empty(shape, dtype=torch.bfloat16, device="cuda")
            ns.nanospec_policy_loss(z, 1.0, *c.arguments(), out["loss"], out["logprob"], out["kl"], out["entropy"], None, dz, workspace(ns, *shape))
            got.append((out["loss"].item(), out["logprob"].clone(), dz))
        assert all(g[0] == got[0][0] and torch.equal(g[1], got[0][1]) and torch.equal(g[2], got[0][2]) for g in got)


def test_no_rows(ns):
    e = torch.empty((0,), device="cuda")
    loss = torch.full((1,), 5.0, device="cuda")
    ns.nanospec_policy_loss(torch.empty((0, 50), device="cuda"), 1.0, e.int(), e, None, e, None, 0.2, 0.2, 0.0, 0.0, loss, e, None, None, None, None,
                            workspace(ns, 0, 50))
    assert loss.item() == 0


def test_agrees_with_token_logprobs(ns):
    """With ratio 1, advantage 1, no KL term and no entropy the loss is -1 a row and its gradient that of -logprob."""
    L, V = 50, 4000
    c = Case(L, V, beta=0.0, ent=0.0)
    z = c.device_rows()[1]
    tok = torch.from_numpy(c.tokens).cuda()
    e = lambda *s: torch.zeros(s, device="cuda")   # noqa: E731
    lp, lse, H = e(L, 1), e(L), e(L)
    ns.nanospec_token_logprobs(z, 1.0, tok[:, None].contiguous(), lp, lse, H, None, None, ns.alloc_token_logprobs_workspace(L, V, 0))
    one = torch.ones(L, device="cuda")
    dz, dz2, loss, lp2, H2 = e(L, V), e(L, V), e(1), e(L), e(L)
    ns.nanospec_policy_loss(z, 1.0, tok, lp[:, 0].contiguous(), None, one, None, 0.2, 0.2, 0.0, 0.0, loss, lp2, None, H2, None, dz, workspace(ns, L, V))
    ns.nanospec_token_logprobs_grad(z, 1.0, tok[:, None].contiguous(), lse, H, -torch.ones((L, 1), device="cuda"), None, None, dz2)
    assert abs(loss.item() + L) < 1e-4 and torch.allclose(lp2, lp[:, 0], rtol=0, atol=2e-6) and torch.allclose(H, H2, rtol=0, atol=2e-5)
    assert torch.allclose(dz, dz2, rtol=2e-5, atol=2e-6)


# forms taken by size: rows in parts or whole, blocks of one, four and eight waves, a row a block or many, rows longer than
# a block's registers, every third row left out
@pytest.mark.parametrize("c", [(95, 3000, "bf16"), (96, 3000, "bf16"), (120, 2000, "fp32"), (130, 9000, "fp16"), (100, 20000, "fp32"), (97, 40000, "fp32"),
                               (100, 66000, "bf16"), (260, 70001, "fp32"), (2100, 66001, "bf16"), (270, 131073, "bf16"), (3000, 300, "fp32"), (700, 4099, "fp16")],
                         ids=lambda c: "x".join(map(str, c)))
def test_forms_by_size(ns, c):
    case = Case(*c)
    case.weight[::3] = 0
    case.weight[-1] = 0
    check(ns, case)
    check(ns, case, grad=False)


def test_no_row_taken(ns):
    for L, V in ((5, 1000), (300, 70000), (2100, 600)):
        case = Case(L, V, "bf16")
        case.weight[:] = 0
        check(ns, case)
        check(ns, case, grad=False)
