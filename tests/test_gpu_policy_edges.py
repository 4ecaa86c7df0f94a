"""Policy loss at the edges of its terms: log-probabilities far apart and past
float32's range, certain rows, unlikely tokens, outputs over inputs.
Definitions and tolerances are those of tests/test_gpu_policy.py."""
import math

import numpy as np
import pytest
import torch

from tests.gpu_common import say
from tests.test_gpu_policy import DT, U, Case, check, near, workspace

pytestmark = pytest.mark.gpu

# rows in parts, with one part and with many; whole rows of one wave and of sixteen
SHAPES = [(9, 900), (9, 40001), (120, 500), (100, 20001)]
shapes = pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))


@pytest.fixture(scope="module")
def ns():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from dynamic_vocab_draft_amd import nanospec
    return nanospec


@shapes
@pytest.mark.parametrize("dtype", DT)
def test_reference_far_below(ns, shape, dtype):
    """exp(delta) is 0 for a token that the reference masks, so the KL term's slope is kl_coef whatever fills the mask."""
    for ref in (-math.inf, -1e30, -1e9, -1e4, -300.0):
        c = Case(*shape, dtype, beta=0.3, ent=0.0)
        c.advantage[:] = 0
        c.ref[1::2] = ref
        check(ns, c, what=str(ref))
        check(ns, c, grad=False, what=str(ref))


@shapes
def test_reference_near_and_above(ns, shape):
    """Both forms of exp(delta) - 1 and where they meet."""
    c = Case(*shape, beta=0.3, ent=0.0)
    logp = c.logp()
    c.ref = (logp + np.resize([-20, -3, -0.6, -0.5, -0.4, -1e-3, 1e-3, 0.5, 0.6, 3, 20], shape[0])).astype(np.float32)
    check(ns, c)


def past_range(case, want):
    """The values that the output's type cannot hold, as infinities."""
    w = torch.from_numpy(want).float().to(DT[case.dtype]).double().numpy()
    return np.where(np.isinf(w), w, want)


def check_huge(ns, case, what):
    """As `check`, with values past the outputs' range."""
    say("policy_loss", case.L, case.V, case.dtype, what)
    with np.errstate(all="ignore"):
        want = case.want()
    z, dz, out = case.device_rows()[1], case.device_rows()[1], case.outputs()
    ns.nanospec_policy_loss(z, float(case.t), *case.arguments(), out["loss"], out["logprob"], out["kl"], out["entropy"],
                            torch.tensor([case.g_loss], device="cuda"), dz, workspace(ns, case.L, case.V))
    torch.cuda.synchronize()
    for name in ("loss", "logprob", "kl", "entropy"):
        if out[name] is not None:
            v, tol = want[name]
            with np.errstate(all="ignore"):
                v = torch.from_numpy(v).float().double().numpy()
            near(out[name], v, np.where(np.isfinite(tol), tol, 0) + U * np.abs(np.where(np.isfinite(v), v, 0)), name)
    v, tol = want["dlogits"]
    # where a row's slopes are past 2^100 the kernel takes them 2^k smaller and 2^y 2^k larger, k <= 150 here: the
    # exponent k + y then rounds by 2^-24 of up to 150 more
    near(dz, past_range(case, v), tol + 1.1 * 150 * U * np.abs(np.where(np.isfinite(v), v, 0)), "dlogits")


@shapes
@pytest.mark.parametrize("dtype", DT)
def test_ratios_past_float32(ns, shape, dtype):
    for what, ahead, advantage in (("no advantage", 100.0, 0.0), ("no advantage, far", 500.0, 0.0), ("clipped", 100.0, 1.5),
                                   ("not clipped", 100.0, -1.5), ("not clipped, far", 150.0, -0.5)):
        c = Case(*shape, dtype, lo=0.2, hi=0.28, ent=0.01)
        c.z[:, 2::3] = -math.inf                  # masked logits have no gradient whatever the slope
        c.z[np.arange(c.L), c.tokens] = 8.0
        logp = c.logp()
        c.ref = (logp + 0.1).astype(np.float32)
        c.old = np.where(np.arange(c.L) % 2, logp - ahead, logp - 0.05).astype(np.float32)
        c.advantage[1::2] = advantage
        check_huge(ns, c, what)


@shapes
def test_unbounded_clip_and_no_advantage(ns, shape):
    """Without an upper clip the ratio itself is past float32's range on both sides of the comparison."""
    c = Case(*shape, hi=math.inf, ent=0.0)
    c.old = np.where(np.arange(c.L) % 2, c.logp() - 200.0, c.old).astype(np.float32)
    c.advantage[1::2] = 0
    check_huge(ns, c, "no clip")


@shapes
def test_reference_far_above(ns, shape):
    """exp(delta) past float32's range."""
    c = Case(*shape, beta=0.3, ent=0.0)
    c.z[:, 2::3] = -math.inf
    c.z[np.arange(c.L), c.tokens] = 8.0
    c.ref = (c.logp() + np.where(np.arange(c.L) % 2, 100.0, 0.2)).astype(np.float32)
    c.old = (c.logp() - 0.1).astype(np.float32)
    check_huge(ns, c, "reference")


def badly_rounded_temperature(most):
    """An inverse temperature up to `most` whose product with log2(e) float32 rounds by more than 0.9 half steps."""
    for i in range(10000):
        t = np.float32(most - i * most * 1e-6)
        c = float(t) * 1.4426950408889634
        off = abs(c - float(np.float32(c))) / (2.0 ** math.floor(math.log2(c)) * U)
        if off > 0.9 and c / 2.0 ** math.floor(math.log2(c)) < 1.1:
            return float(t)


@pytest.mark.parametrize("L", [7, 120])
@pytest.mark.parametrize("sign", [1, -1])
def test_entropy_slope_of_a_certain_row(ns, L, sign):
    """A row whose largest logit is all of it has entropy 0 and an entropy slope of 0 there, however far the logits lie
    from zero.  In units of U = 2^-24: the exponential, and the logarithm of its sum, are off by 4 relative to p = 1, the
    quotient W / S by 2, and the slope A + B y is a sum of terms under 0.4, rounded at each of four steps: 8 in all; twice that is allowed."""
    t = badly_rounded_temperature(1.5)
    V = 700
    c = Case(L, V, t=t, beta=0.0, ent=1.0)
    top = sign * 460.0                            # |c z| of some 1000
    c.z[:] = top - 60.0
    best = (c.tokens + 1) % V
    c.z[np.arange(L), best] = top
    c.z[np.arange(L), c.tokens] = top - 40.0
    c.advantage[:] = 0
    c.weight[:] = 1
    c.g_loss = np.float32(1)
    c.old = c.logp().astype(np.float32)
    assert (c.logp() > -104).all()
    z, dz, out = c.device_rows()[1], c.device_rows()[1], c.outputs()
    ns.nanospec_policy_loss(z, float(c.t), *c.arguments(), out["loss"], out["logprob"], None, out["entropy"], None, dz, workspace(ns, L, V))
    want = c.want()["dlogits"][0]
    assert np.abs(want).max() < 1e-12
    worst = float(dz.abs().max())
    say("largest slope, in 2^-24", worst / U)
    assert worst <= 16 * U * float(c.t)


@shapes
@pytest.mark.parametrize("shift", [-930.0, 500.0, 900.0])
def test_entropy_of_shifted_logits(ns, shape, shift):
    c = Case(*shape, beta=0.1, ent=0.5, t=badly_rounded_temperature(0.75))
    z = torch.round(c.z.double() * 64) / 64
    c.z = (z + shift).float()
    assert torch.equal(c.z.double() - shift, z)
    logp = c.logp()
    c.old, c.ref = (logp - 0.1).astype(np.float32), (logp + 0.2).astype(np.float32)
    check(ns, c)


@shapes
def test_unlikely_tokens(ns, shape):
    """Down to a log-probability of -104 a token teaches as any other, below that nothing."""
    for below, learns in ((80.0, True), (95.0, True), (103.5, True), (104.5, False), (140.0, False)):
        c = Case(*shape, beta=0.2, ent=0.01)
        odd = np.arange(1, c.L, 2)
        c.z[odd, c.tokens[odd]] = -200.0
        others = torch.logsumexp(c.z[odd].double(), 1)
        c.z[odd, c.tokens[odd]] = (others - below).float()
        logp = c.logp()
        assert ((logp[odd] > -104) == learns).all()
        c.old, c.ref = (logp - 0.1).astype(np.float32), (logp + 0.3).astype(np.float32)
        check(ns, c, what=str(below))
        got = check(ns, c, grad=False, what=str(below))["kl"].cpu().numpy()[odd]
        assert (got > 0.04).all() if learns else (got == 0).all()


@pytest.mark.parametrize("shape", [(1, 300), (5, 1000), (3, 40001), (95, 3000), (40, 128256), (120, 2000), (300, 70001)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("grad", [True, False])
def test_outputs_over_a_row_s_inputs(ns, shape, grad):
    """logprob, kl and entropy may replace the row's inputs, the loss what it is multiplied by."""
    for turn in range(3):
        c = Case(*shape, "bf16", seed=turn, ent=0.02)
        c.weight[::4] = 0
        want, z, g = c.outputs(), c.device_rows()[1], torch.tensor([c.g_loss], device="cuda")
        dz = torch.empty_like(z) if grad else None
        ns.nanospec_policy_loss(z, 1.0, *c.arguments(), want["loss"], want["logprob"], want["kl"], want["entropy"], g, dz, workspace(ns, *shape))
        for over in ((1, 2, 3), (3, 4, 1)):       # old, ref and advantage; advantage, weight and old
            args = c.arguments()
            lp, kl, H = (args[i] for i in over)
            loss, dz2 = g.clone(), torch.empty_like(z) if grad else None
            ns.nanospec_policy_loss(z, 1.0, *args, loss, lp, kl, H, loss, dz2, workspace(ns, *shape))
            assert torch.equal(loss, want["loss"]) and torch.equal(lp, want["logprob"]) and torch.equal(kl, want["kl"])
            assert torch.equal(H, want["entropy"]) and (not grad or torch.equal(dz, dz2))


@pytest.mark.parametrize("grad", [True, False])
def test_infinite_old_log_probabilities(ns, grad):
    """A token that the old policy ruled out has a ratio past any range: 0 with no advantage, clipped with one, infinite against one."""
    for L in (8, 100):
        c = Case(L, 700, ent=0.0)
        z, got = c.device_rows()[1], []
        for old, advantage in ((-math.inf, (0.0, 1.0)), (-3e38, (0.0, 1.0)), (-300.0, (0.0, 1.0)), (-math.inf, (-1.0, 0.0))):
            c.old[:] = old
            c.advantage[:] = np.resize(advantage, L)
            out, dz = c.outputs(), torch.empty_like(z) if grad else None
            ns.nanospec_policy_loss(z, 1.0, *c.arguments(), out["loss"], out["logprob"], out["kl"], out["entropy"], None, dz, workspace(ns, L, 700))
            got.append((out["loss"], dz))
        assert torch.isfinite(got[0][0]) and all(torch.equal(g[0], got[0][0]) for g in got[1:3])
        assert got[3][0].item() == math.inf
        if grad:
            assert torch.isfinite(got[0][1]).all() and all(torch.equal(g[1], got[0][1]) for g in got[1:3])
            d = got[3][1].cpu()
            assert (d[np.arange(0, L, 2), c.tokens[::2]] == math.inf).all() and torch.isfinite(d[1::2]).all() and not d.isnan().any()


@shapes
@pytest.mark.parametrize("shift", [-715.0, 700.0, 709.0])
def test_logits_on_both_sides_of_the_exponents_limit(ns, shape, shift):
    """|c z| on both sides of 1024, where parts of a row are kept in two ways and joined."""
    c = Case(*shape, beta=0.1, ent=0.01)
    z = torch.round(c.z.double() * 64) / 64
    c.z = (z + shift).float()
    assert torch.equal(c.z.double() - shift, z)
    logp = c.logp()
    c.old, c.ref = (logp - 0.1).astype(np.float32), (logp + 0.2).astype(np.float32)
    check(ns, c)
    check(ns, c, grad=False)


@shapes
def test_ratios_past_float32_of_far_logits(ns, shape):
    """The two together: slopes past 2^100 in rows whose exponents are taken from their largest logit."""
    c = Case(*shape, ent=0.01)
    z = torch.round(c.z.double() * 64) / 64
    z[:, 2::3] = -math.inf
    z[np.arange(c.L), c.tokens] = 8.0
    c.z = (z + 3e4).float()
    logp = c.logp()
    c.ref = (logp + 0.1).astype(np.float32)
    c.old = np.where(np.arange(c.L) % 2, logp - 110.0, logp - 0.05).astype(np.float32)
    c.advantage[1::2] = -1.5
    check_huge(ns, c, "far")
