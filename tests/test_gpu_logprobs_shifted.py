"""The gradient of rows whose log-sum-exp is large: shifted logits, masks of fp16's lowest value, low temperatures.

lse itself is a float32, half a step of it is 2^-5 at 10^6 and 1/2 below 2^24, so probabilities cannot come from it there.
Tolerances, with u = 2^-24.  Relative to a reference next to lse differences of logits are exact wherever p is not 0, so an
exponent carries c's rounding and its own, 2 u |logp|, in the sum as well (weighted by p: at most 2 u 20); exp2 adds 2 u,
the longest chain of positive additions (32 within a batch, 63 batches, 6 lane steps, 4 waves) 110 u, log2 and the last
operations 20 u: p within u (4 |logp| + 400) relatively.  The entropy that the forward call wrote is within u 400 (2 + H)
likewise (no term in the logits' own size, which differences do not see), and twice all that is allowed.  The device's
2^y is 0 where it is below float32's normal range, so p is off by up to 2^-126 there, and the gradient by that times its
factor inv_temp (|G| + |g_H| (|logp| + H + 3)): a p of 2^-128 at inv_temp = 300 is lost whole."""
import numpy as np
import pytest
import torch

from tests.gpu_common import say
from tests.test_gpu_logprobs import DT, U, call, grad_reference, near, ns, reference, run_grad, tokens_for  # noqa: F401

pytestmark = pytest.mark.gpu


def rows(V, dtype, seed):
    """Rows with |lse| between 1024 and 2^24, among ordinary ones, an empty one and one without a distribution."""
    rng = np.random.default_rng(seed)
    n = rng.standard_normal((16, V)).astype(np.float32)
    z = n * 3
    if dtype == "fp32":
        z[0] = n[0] * 3 + 1.0e6
        z[1] = n[1] * 3 - 1.0e6
        z[2] = np.rint(n[2] * 2) + 1.6e7                 # just below 2^24
        z[3] = np.rint(n[3] * 2) - 1.6e7
        z[4] = n[4] * 3 + 1030
        z[5] = n[5] * 3 - 1.2e3 - np.log(V)
        z[6] = n[6] + 7.0e4
        z[6, V // 2] = 7.0e4 + 12
    else:
        step = 256.0 if dtype == "bf16" else 32.0        # of the type between 32768 and 65536
        z[0] = 50000 // step * step
        z[1] = -(50000 // step * step)
        z[2] = np.where(n[2] > 1, 2080, 2064)
        z[3] = np.where(n[3] > 1, -2080, -2064)
        z[4] = np.where(n[4] > 0, 1104, 1096)
        z[5] = -65504.0 if dtype == "fp16" else -65536.0  # fp16's lowest: nothing but masked logits
        z[6] = -65504.0 if dtype == "fp16" else -65536.0
        z[6, V // 2] = z[6, V // 2] / 2
    z[7, ::2] = z[0, ::2]                                # half of a row far above the other half
    z[8] = z[0]
    z[8, ::3] = -np.inf
    z[9] = -np.inf
    z[9, V - 1] = z[0, 0]                                # a single logit
    z[10] = -np.inf
    z[11] = z[0]
    z[11, 3 % V] = np.nan
    return torch.from_numpy(z).to(DT[dtype]).cuda()


def check(ns, z, it, T, what, use_H=True):  # noqa: F811
    say("gradient, shifted", what)
    L, V = z.shape
    rng = np.random.default_rng(V + T)
    tok = tokens_for(L, V, T, 3)
    if T > 2:
        tok[:, 2] = tok[:, 1]                            # a token named twice
        tok[1, 0] = -1
        tok[2, 0] = V
        tok[3, 0] = V - 1
    g = rng.standard_normal(tok.shape).astype(np.float32)
    gH, gl = (rng.standard_normal(L).astype(np.float32) for _ in range(2))
    if not use_H:
        gH[:] = 0
    r = reference(z, it, tok, 0)
    with np.errstate(invalid="ignore"):
        d, size = grad_reference(z, it, tok, r, g.astype(np.float64), gH.astype(np.float64), gl.astype(np.float64))
    o = call(ns, z, it, tok, 0)
    out = torch.full((L, V + 3), 1.5, dtype=z.dtype, device="cuda")
    args = (it, tok, o["lse"], o["H"] if use_H else None, g, gH if use_H else None, gl)
    run_grad(ns, z, *args, out[:, :V])
    same = z.clone()
    run_grad(ns, same, *args, same)                      # in place
    torch.cuda.synchronize()
    assert (out[:, V:] == 1.5).all(), f"{what}: wrote between the rows"
    assert torch.equal(torch.nan_to_num(out[:, :V], nan=99.0), torch.nan_to_num(same, nan=99.0)), f"{what}: in place"
    with np.errstate(invalid="ignore"):
        logp = np.where(np.isfinite(r["logp"]), np.abs(r["logp"]), 0.0)
        tol = 2 * size * U * (4 * logp + 800)
        wide = (np.abs(r["lse"]) > 1024) & (np.abs(r["lse"]) < 2.0 ** 24)
        # the other rows: probabilities from the rounded lse, 8 Z u
        tol = np.where(wide[:, None], tol, tol + 2 * size * U * 8 * r["Z"][:, None])
        G = gl - np.where((tok >= 0) & (tok < V), g, 0).sum(1)
        factor = it * (np.abs(G)[:, None] + np.abs(gH)[:, None] * (logp + np.abs(r["H"])[:, None] + 3))
        tiny = factor * 2.0 ** -126 + (2.0 ** -25 if z.dtype == torch.float16 else 2.0 ** -133 if z.dtype == torch.bfloat16
                                       else 2.0 ** -126)
        tol = tol + (np.abs(d) + tol) * torch.finfo(z.dtype).eps / 2 + tiny
    d[np.isnan(r["lse"])] = np.nan
    d[np.abs(r["lse"]) > 2.0 ** 24] = 0                  # what is promised beyond
    near(out[:, :V], d, tol, what)
    return wide


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("V", [5, 70, 4099, 9000])
@pytest.mark.parametrize("T", [0, 1, 5])
def test_shifted_rows(ns, V, dtype, T):  # noqa: F811
    wide = check(ns, rows(V, dtype, V), 1.0, T, f"V={V} {dtype} T={T}")
    assert wide[:9].all() and not wide[10:].any()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_shifted_rows_of_many_parts(ns, dtype):  # noqa: F811
    check(ns, rows(50257, dtype, 1), 1.0, 3, f"V=50257 {dtype}")
    check(ns, rows(50257, dtype, 2), 1.0, 3, f"V=50257 {dtype} without entropy", use_H=False)


@pytest.mark.parametrize("it", [2.0 ** -9, 0.3, 7.0, 300.0])
def test_shifted_rows_at_temperatures(ns, it):  # noqa: F811
    for V in (300, 5003):
        n = np.random.default_rng(V).standard_normal((4, V))
        z = np.stack([n[0] + 1.0e5, n[1] - 3.0e4, n[2] + 4000 / it, n[3] - 2000 / it])
        check(ns, torch.from_numpy(z.astype(np.float32)).cuda(), it, 3, f"V={V} it={it}")
