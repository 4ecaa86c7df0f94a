"""4-bit rows and the policy loss as they are used: a draft with the 4-bit
head, tokens scored by the 4-bit rows, a training step against the
full-precision logits; in captured graphs, on streams of their own, and with
calls of the 8-bit rows and the log-probabilities between them."""
import numpy as np
import pytest
import torch

from tests.gpu_common import say

pytestmark = pytest.mark.gpu

V, D, L = 6000, 512, 96


@pytest.fixture(scope="module")
def ns():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from dynamic_vocab_draft_amd import nanospec
    return nanospec


def e(*s, t=torch.float32):
    return torch.full(s, 3, dtype=t, device="cuda")


class Step:
    """One step of drafting and training: all buffers in hand, `run` only enqueues."""

    def __init__(self, ns, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, device="cuda")   # noqa: E731
        self.ns = ns
        self.w = (0.05 * r(V, D)).to(torch.bfloat16)
        self.h = r(L, D).to(torch.bfloat16)
        p = ns.nanospec_mx4_pitch(D)
        u8 = torch.uint8
        self.wq, self.ws = e(V, p, t=u8), e(V, p // 16, t=u8)
        self.hq, self.hs = e(L, p, t=u8), e(L, p // 16, t=u8)
        self.ids = torch.arange(0, V, 7, dtype=torch.int32, device="cuda")[None].contiguous()
        n = self.ids.shape[1]
        self.n = torch.tensor([n - 3], dtype=torch.int32, device="cuda")
        self.oi, self.ov = e(1, 8, 4, t=torch.int32), e(1, 8, 4)
        self.head_ws = ns.alloc_mx4_logits_workspace(1, n, 8, 4, D)
        self.packed = e(n, D, t=torch.bfloat16)
        self.z4 = e(L, V)
        self.tokens = torch.randint(0, V, (L, 1), generator=g, device="cuda").to(torch.int32)
        self.old, self.lse = e(L, 1), e(L)
        self.lp_ws = ns.alloc_token_logprobs_workspace(L, V, 0)
        self.z = (self.h.float() @ self.w.float().t()).to(torch.bfloat16)
        self.adv = r(L)
        self.weight = torch.full((L,), 1 / L, device="cuda")
        self.weight[:10] = 0
        self.loss, self.logp, self.kl = e(1), e(L), e(L)
        self.dz = e(L, V, t=torch.bfloat16)
        self.p_ws = ns.alloc_policy_loss_workspace(L, V)

    def run(self, stream=None):
        ns = self.ns
        ns.nanospec_mx4_rows(self.w, self.wq, self.ws, stream)
        ns.nanospec_mx4_gather_rows(self.wq, self.ws, self.ids[0], self.n, self.packed, stream)
        ns.nanospec_mx4_logits_topk(self.wq, self.ws, self.ids, self.n, self.h[:8][None], 4, None, self.oi, self.ov, self.head_ws, stream)
        ns.nanospec_mx4_rows(self.h, self.hq, self.hs, stream)
        ns.nanospec_mx4_matmul(self.hq, self.hs, self.wq, self.ws, D, self.z4, stream)
        ns.nanospec_token_logprobs(self.z4, 1.0, self.tokens, self.old, self.lse, None, None, None, self.lp_ws, stream)
        ns.nanospec_policy_loss(self.z, 1.0, self.tokens[:, 0].contiguous() if stream is None else self.tokens.view(L), self.old.view(L), self.old.view(L),
                                self.adv, self.weight, 0.2, 0.2, 0.05, 0.0, self.loss, self.logp, self.kl, None, None, self.dz, self.p_ws, stream)

    def results(self):
        torch.cuda.synchronize()
        return [t.clone() for t in (self.packed, self.oi, self.ov, self.z4, self.old, self.loss, self.logp, self.kl, self.dz)]

    def spoil(self):
        for t in (self.wq, self.ws, self.hq, self.hs, self.oi, self.ov, self.z4, self.old, self.loss, self.logp, self.kl, self.dz, self.head_ws, self.p_ws, self.lp_ws):
            t.zero_()
        self.packed.fill_(3)


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_step_against_plain_form(ns):
    s = Step(ns, 1)
    s.run()
    packed, oi, ov, z4, old, loss, logp, kl, dz = s.results()
    n = int(s.n.item())
    w4 = e(V, D)
    ns.nanospec_mx4_gather_rows(s.wq, s.ws, None, None, w4)
    h4 = e(L, D)
    ns.nanospec_mx4_gather_rows(s.hq, s.hs, None, None, h4)
    w4, h4 = w4.double().cpu(), h4.double().cpu()
    assert torch.equal(packed[:n].double().cpu(), w4[s.ids[0, :n].long().cpu()]) and (packed[n:] == 3).all()
    full = h4 @ w4.t()
    assert torch.equal(z4.cpu(), full.float())
    rows = s.ids[0, :n].long().cpu()
    best = full[:8][:, rows].sort(dim=1, descending=True, stable=True)
    assert torch.equal(ov[0].cpu(), best.values[:, :4].float()) and torch.equal(oi[0].cpu().long(), rows[best.indices[:, :4]])
    # the rows are off by what four bits take: half a step is an eighth of a value, and less from a block's top down
    err = (full - s.h.double().cpu() @ s.w.double().cpu().t()).norm() / full.norm()
    say("4-bit logits off by", float(err))
    assert err < 0.25
    z = s.z.double().cpu()
    t = s.tokens.long().cpu()
    lp = torch.log_softmax(z, 1).gather(1, t)[:, 0]
    want_old = torch.log_softmax(full, 1).gather(1, t)[:, 0]
    assert torch.allclose(old[:, 0].double().cpu(), want_old, rtol=0, atol=1e-5)
    ratio = torch.exp(lp - old[:, 0].double().cpu())
    a, wt = s.adv.double().cpu(), s.weight.double().cpu()
    delta = old[:, 0].double().cpu() - lp
    want = (wt * (-torch.minimum(ratio * a, ratio.clamp(float(np.float32(1) - np.float32(0.2)), 1.2) * a) + 0.05 * (torch.expm1(delta) - delta))).sum()
    assert abs(loss.double().item() - want.item()) < 1e-5 * (wt * (ratio * a).abs()).sum().item() + 1e-7
    assert (dz[:10] == 0).all() and (logp[:10] == 0).all() and (dz[10:].float().abs().sum(1) >= 0).all()


def test_captured_and_replayed(ns):
    """Two graphs of steps with buffers of their own, replayed in turn with eager work and 8-bit calls between."""
    a, b = Step(ns, 2), Step(ns, 3)
    a.run(), b.run()
    want = [a.results(), b.results()]
    graphs = []
    for s in (a, b):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            s.run(side)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run(torch.cuda.current_stream())
        graphs.append(g)
    q, sc = e(V, D, t=torch.int8), e(V)
    for turn in range(4):
        for s, g, w in zip((a, b), graphs, want):
            s.spoil()
            g.replay()
            assert same(s.results(), w), turn
        ns.nanospec_quant_rows(a.w, q, sc)
        b.spoil()
        b.run()
        assert same(b.results(), want[1]), turn


def test_two_streams_at_once(ns):
    a, b = Step(ns, 4), Step(ns, 5)
    a.run(), b.run()
    want = [a.results(), b.results()]
    a.spoil(), b.spoil()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for s, st in zip((a, b), streams):
            s.run(st)
    assert same(a.results(), want[0]) and same(b.results(), want[1])


def test_packed_rows_feed_the_full_precision_head(ns):
    """Rows read back in bf16 are a PACKED buffer of nanospec_draft_logits_topk."""
    s = Step(ns, 6)
    s.run()
    n_max = s.ids.shape[1]
    lg, ti, tv = e(8, n_max), e(8, 4, t=torch.int32), e(8, 4)
    ns.nanospec_draft_logits_topk(s.packed, ns.NS_PACKED, s.ids[0], s.n, n_max, V, D, ns.NS_BF16, s.h[:8].contiguous(), 8, 4, lg, ti, tv,
                                  ns.alloc_workspace(n_max, 8, 4, D))
    torch.cuda.synchronize()
    n = int(s.n.item())
    want = s.h[:8].double().cpu() @ s.packed[:n].double().cpu().t()
    assert (lg[:, :n].double().cpu() - want).abs().max() < 1e-2
