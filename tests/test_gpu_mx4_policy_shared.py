"""The step of tests/test_gpu_mx4_policy.py: its gradient against float64, and
captured graphs whose workspaces are shared."""
import numpy as np
import pytest
import torch

from tests.test_gpu_mx4_policy import L, V, Step, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ns():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from dynamic_vocab_draft_amd import nanospec
    return nanospec


def gradient(s, old):
    """(dlogits, tolerance) of a step whose tokens were scored `old`: the derivative of the definition's loss in float64.
    With u = 2^-24 a row's log-probability, its ratio and exp(delta), relatively, are within 80 u, and each p_j within
    its own exponential's error beside that, 2 u |logp_j| + 8 u; the row's slope g is a difference of two such terms; the output is rounded to bf16."""
    z, t = s.z.double().cpu(), s.tokens.long().cpu()
    z.requires_grad_()
    every = torch.log_softmax(z, 1)
    lp = every.gather(1, t)[:, 0]
    a, w, old = s.adv.double().cpu(), s.weight.double().cpu(), old[:, 0].double().cpu()
    ratio, delta = torch.exp(lp - old), old - lp
    lo, hi, beta = 1 - float(np.float32(0.2)), 1 + float(np.float32(0.2)), float(np.float32(0.05))
    near = ((ratio - lo).abs() < 1e-4) | ((ratio - hi).abs() < 1e-4)       # where the slope jumps
    assert not near[w != 0].any()
    (w * (-torch.minimum(ratio * a, ratio.clamp(lo, hi) * a) + beta * (torch.expm1(delta) - delta))).sum().backward()
    with torch.no_grad():
        u = 2.0 ** -24
        p = every.exp()
        one = torch.zeros_like(p).scatter_(1, t, 1.0)
        slope = w * (ratio * a.abs() + beta * (1 + delta.exp()))           # a sum of magnitudes
        tol = slope[:, None] * 84 * u * (one + p) + slope[:, None] * p * (every.abs() * 2 + 88) * u
        return z.grad, 1.1 * tol + 2.0 ** -8 * z.grad.abs() + 2.0 ** -133


def test_gradient_of_the_step(ns):
    for seed in (11, 12):
        s = Step(ns, seed)
        s.run()
        old, dz = s.old.clone(), s.dz.clone()
        want, tol = gradient(s, old)
        off = (dz.double().cpu() - want).abs()
        assert (off <= tol).all(), float((off - tol).max())
        assert (want[10:].abs().sum(1) > 0).sum() > L // 2 and (dz[:10] == 0).all()


def test_graphs_that_share_workspaces(ns):
    """Two steps with outputs of their own and one workspace of each kind, captured and replayed in order, both ways round."""
    a, b = Step(ns, 13), Step(ns, 14)
    for name in ("head_ws", "lp_ws", "p_ws"):
        setattr(b, name, getattr(a, name))
    a.run()
    first = a.results()
    b.run()
    want = [first, b.results()]
    assert not same(*want)
    graphs = []
    for s in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run(torch.cuda.current_stream())
        graphs.append(g)
    for turn in range(4):
        a.spoil(), b.spoil()
        for ws in (a.head_ws, a.lp_ws, a.p_ws):
            ws.fill_(0xFF)
        order = (0, 1) if turn % 2 else (1, 0)
        for i in order:                               # one behind the other on one stream, nothing between
            graphs[i].replay()
        assert same(a.results(), want[0]) and same(b.results(), want[1]), turn
        b.spoil()
        b.run()                                       # an eager step over the same workspaces
        assert same(b.results(), want[1]), turn
    loss = torch.zeros(1, device="cuda")
    s = a                                             # a policy loss of another size in the same workspace
    ns.nanospec_policy_loss(s.z[:7], 1.0, s.tokens[:7, 0].contiguous(), s.old[:7, 0].contiguous(), None, s.adv[:7].contiguous(), None, 0.2, 0.2, 0.0, 0.0,
                            loss, torch.empty(7, device="cuda"), None, None, None, torch.empty((7, V), dtype=torch.bfloat16, device="cuda"), s.p_ws)
    graphs[0].replay()
    assert same(a.results(), want[0])
