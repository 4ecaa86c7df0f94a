"""The 8-bit head and the token log-probabilities as a serving loop uses them,
beside the calls they stand next to: a prompt (logits of every position, its
candidates, its tokens' log-probabilities), decode steps over the active set,
verification of the children under the full-vocabulary head, and the gradient.
Eager, captured and replayed, on other streams, with workspaces that two
graphs share, and with rows past 4 GB."""
import numpy as np
import pytest
import torch

import oracle.nanospec_oracle as O
from tests.gpu_common import dev_i32, say
from tests.test_gpu_logprobs import U, near, reference
from tests.test_gpu_quant import pitch, quantised, replica

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ns():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from dynamic_vocab_draft_amd import nanospec
    return nanospec


class Target:
    """Everything a loop keeps: 8-bit rows, window state, buffers, workspaces."""

    def __init__(self, ns, V, d, L, M, k, w_max, seed):
        self.ns, self.V, self.d, self.L, self.M, self.k, self.w_max = ns, V, d, L, M, k, w_max
        g = torch.Generator(device="cuda").manual_seed(seed)
        e = lambda *s, t=torch.float32: torch.zeros(s, dtype=t, device="cuda")
        i32, i8 = torch.int32, torch.int8
        W = torch.randn((V, d), generator=g, device="cuda").mul_(0.05).bfloat16()
        self.wq, self.ws = e(V, pitch(d), t=i8), e(V)
        ns.nanospec_quant_rows(W, self.wq, self.ws)
        self.W = W
        self.st = ns.NanoSpecState(V, w_max)
        self.ids, self.n = e(w_max, t=i32), e(1, t=i32)
        # prompt
        self.hp, self.prompt = e(L, d, t=torch.bfloat16), e(L, t=i32)
        self.hq, self.hs, self.z = e(L, pitch(d), t=i8), e(L), e(L, V, t=torch.bfloat16)
        self.pid, self.pval = e(L, 4, t=i32), e(L, 4)
        self.plp, self.plse, self.pH = e(L, 1), e(L), e(L)
        self.pwork = ns.alloc_token_logprobs_workspace(L, V, 0)
        # decode step
        self.h = e(1, M, d, t=torch.bfloat16)
        self.tree, self.ver = e(6, t=i32), e(2, t=i32)
        self.tid, self.tval = e(1, M, k, t=i32), e(1, M, k)
        self.work = ns.alloc_quant_logits_workspace(1, w_max, M, k, d)
        self.vq, self.vs, self.vz = e(M, pitch(d), t=i8), e(M), e(M, V)
        self.lp, self.lse, self.H = e(M, k), e(M), e(M)
        self.top, self.toplp = e(M, 3, t=i32), e(M, 3)
        self.lwork = ns.alloc_token_logprobs_workspace(M, V, 3)
        self.glp, self.gH, self.dz = torch.ones((M, k), device="cuda"), torch.full((M,), 0.1, device="cuda"), e(M, V)
        self.fidx, self.fval, self.fid = e(1, 5, t=i32), e(1, 5), e(1, 5, t=i32)

    def run_prompt(self):
        ns = self.ns
        ns.nanospec_quant_rows(self.hp, self.hq, self.hs)
        ns.nanospec_quant_matmul(self.hq, self.hs, self.wq, self.ws, self.d, self.z)
        ns.nanospec_prefill_topk(self.z, self.L, self.V, ns.NS_BF16, 4, self.pid, self.pval)
        ns.nanospec_stream_append(self.st, self.prompt, self.L, 0)
        ns.nanospec_stream_append(self.st, self.pid, self.L * 4, 1)
        ns.nanospec_token_logprobs(self.z, 1.0, self.prompt.view(-1, 1), self.plp, self.plse, self.pH, None, None,
                                   self.pwork)

    def run_step(self):
        ns, M, k = self.ns, self.M, self.k
        ns.nanospec_step_update(self.st, self.tree, 6, self.ver, 2, self.ids, self.n)
        ns.nanospec_quant_logits_topk(self.wq, self.ws, self.ids.view(1, -1), self.n, self.h, k, None, self.tid,
                                      self.tval, self.work)
        ns.nanospec_tree_select(self.tval, self.tid, M * k, 1, 5, self.fidx, self.fval, self.fid)
        # the target's view of the same rows' children
        ns.nanospec_quant_rows(self.h[0], self.vq, self.vs)
        ns.nanospec_quant_matmul(self.vq, self.vs, self.wq, self.ws, self.d, self.vz)
        ns.nanospec_token_logprobs(self.vz, 1.0, self.tid[0], self.lp, self.lse, self.H, self.top, self.toplp,
                                   self.lwork)
        ns.nanospec_token_logprobs_grad(self.vz, 1.0, self.tid[0], self.lse, self.H, self.glp, self.gH, None, self.dz)

    OUT = ("ids", "n", "tid", "tval", "fidx", "fval", "fid", "vz", "lp", "lse", "H", "top", "toplp", "dz")

    def feed(self, t):
        g = torch.Generator(device="cuda").manual_seed(1000 + t)
        self.h.copy_(torch.randn(self.h.shape, generator=g, device="cuda"))
        self.tree.copy_(torch.randint(0, self.V, (6,), generator=g, device="cuda"))
        self.ver.copy_(torch.randint(0, self.V, (2,), generator=g, device="cuda"))

    def results(self):
        n = int(self.n.item())
        return {k: (self.ids[:n] if k == "ids" else getattr(self, k)).clone() for k in self.OUT}


def make(ns, seed=1, L=40):
    t = Target(ns, 5003, 520, L, 8, 6, 1024, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 50)
    t.hp.copy_(torch.randn(t.hp.shape, generator=g, device="cuda"))
    t.prompt.copy_(torch.randint(0, t.V, (L,), generator=g, device="cuda"))
    return t


def test_prompt_and_steps_against_definitions(ns):
    t = make(ns)
    t.run_prompt()
    torch.cuda.synchronize()
    rq, rs = quantised(t.W.double().cpu().numpy())
    hq, hs = quantised(t.hp.double().cpu().numpy())
    want = torch.from_numpy(replica(hq, hs, rq, rs)).bfloat16()
    assert torch.equal(t.z.cpu(), want)
    p_ids, _ = O.prefill_topk(t.z.view(torch.int16).cpu().numpy().view(np.uint16), 4, "bf16")
    assert np.array_equal(t.pid.cpu().numpy(), p_ids)
    r = reference(t.z, 1.0, t.prompt.cpu().numpy().astype(np.int64)[:, None], 0)
    near(t.plp, r["lp"], (U * (8 * r["Z"] + 300))[:, None] + 8 * U * np.abs(r["lp"]), "prompt logprob")
    near(t.pH, r["H"], U * (8 * r["Z"] + 400) * (2 + r["H"]), "prompt entropy")

    seq = O.Sequence_(t.w_max)
    seq.append_prompt(t.prompt.cpu().numpy())
    seen = list(dict.fromkeys(p_ids.reshape(-1).tolist()))
    seq.append_prompt(np.asarray(seen))                    # tuple(): each id once, at its first place
    for step in range(3):
        say("target step", step)
        t.feed(step)
        t.run_step()
        torch.cuda.synchronize()
        seq.step(t.tree.cpu().numpy(), t.ver.cpu().numpy())
        I = seq.active()
        assert np.array_equal(t.ids[:int(t.n.item())].cpu().numpy(), I)
        q, s = quantised(t.h[0].double().cpu().numpy())
        z = replica(q, s, rq[I], rs[I])
        order = np.lexsort((np.broadcast_to(I, z.shape), -(z + 0.0)), axis=1)[:, :t.k]
        assert np.array_equal(t.tid[0].cpu().numpy(), I[order])
        assert np.array_equal(t.tval[0].cpu().numpy(), np.take_along_axis(z, order, 1))
        full = replica(q, s, rq, rs)
        assert np.array_equal(t.vz.cpu().numpy(), full)
        r = reference(t.vz, 1.0, t.tid[0].cpu().numpy().astype(np.int64), 3)
        near(t.lp, r["lp"], (U * (8 * r["Z"] + 300))[:, None] + 8 * U * np.abs(r["lp"]), "children")
        assert np.array_equal(t.top.cpu().numpy(), r["ids"])
        # the gradient of sum(lp) + 0.1 H: every row of sum_j dz_j is 0 up to rounding
        p = np.exp(r["logp"])
        d = p * (-t.k - np.float64(np.float32(0.1)) * (r["logp"] + r["H"][:, None]))
        for m in range(t.M):
            np.add.at(d[m], t.tid[0, m].cpu().numpy(), 1.0)
        size = p * (t.k + 0.1 * (np.abs(r["logp"]) + r["H"][:, None] + 3)) + (d > 0)
        near(t.dz, d, size * U * (8 * r["Z"][:, None] + 400) * 2 + np.abs(d) * U + 2.0 ** -126, "gradient")


def test_graph_replays_match_eager(ns):
    a, b = make(ns, 3), make(ns, 3)
    for t in (a, b):
        t.run_prompt()
        t.feed(0)
        t.run_step()                                       # the first calls, before the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.run_step()
    torch.cuda.synchronize()
    for step in range(1, 6):
        say("target replay", step)
        a.feed(step)
        g.replay()
        torch.cuda.synchronize()
        b.feed(step)
        b.run_step()
        torch.cuda.synchronize()
        x, y = a.results(), b.results()
        for k in x:
            assert torch.equal(x[k], y[k]), f"replay {step}: {k}"


def test_two_graphs_share_workspaces_in_order(ns):
    """Two captured products of different sizes on one workspace each, replayed in turn."""
    V, d = 6000, 256
    g0 = torch.Generator(device="cuda").manual_seed(2)
    wq = torch.randint(-127, 128, (V, d), generator=g0, device="cuda", dtype=torch.int32).to(torch.int8)
    ws = torch.rand(V, generator=g0, device="cuda")
    work = ns.alloc_quant_logits_workspace(1, V, 32, 16, d)
    lwork = ns.alloc_token_logprobs_workspace(32, V, 16)
    work.fill_(0xFF)
    lwork.fill_(0xFF)

    def side(M, k):
        h = torch.randn((1, M, d), generator=g0, device="cuda").bfloat16()
        ti, tv = torch.zeros((1, M, k), dtype=torch.int32, device="cuda"), torch.zeros((1, M, k), device="cuda")
        z = torch.zeros((1, M, V), device="cuda")
        lse, ids, lp = torch.zeros(M, device="cuda"), ti[0].clone(), tv[0].clone()

        def run():
            ns.nanospec_quant_logits_topk(wq, ws, None, None, h, k, z, ti, tv, work)
            ns.nanospec_token_logprobs(z[0], 0.01, None, None, lse, None, ids, lp, lwork)
        return run, (ti, tv, z, lse, ids, lp)
    sides = [side(32, 16), side(3, 5)]
    want = []
    for run, out in sides:
        run()
        torch.cuda.synchronize()
        want.append([o.clone() for o in out])
    graphs = []
    for run, out in sides:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        graphs.append(g)
    for turn in range(4):
        for o in [o for _, out in sides for o in out]:
            o.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for (_, out), w in zip(sides, want):
            for o, x in zip(out, w):
                assert torch.equal(o, x), f"turn {turn}"


def test_calls_on_two_streams_at_once(ns):
    """Independent calls (buffers and workspaces of their own) on two streams, against the same on one."""
    sides = [make(ns, 7), make(ns, 8)]
    for t in sides:
        t.run_prompt()
        t.feed(1)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sides]
    for t, s in zip(sides, streams):
        with torch.cuda.stream(s):
            t.run_step()
    torch.cuda.synchronize()
    for seed, t in zip((7, 8), sides):
        u = make(ns, seed)
        u.run_prompt()
        u.feed(1)
        u.run_step()
        torch.cuda.synchronize()
        x, y = t.results(), u.results()
        for k in x:
            assert torch.equal(x[k], y[k]), k


# ---------------------------------------------------------------------------
# Addresses past 32 bits
# ---------------------------------------------------------------------------
def test_rows_past_four_gigabytes(ns):
    V, d, M = 1 << 20, 4200, 3                             # 4.4 GB of 8-bit rows
    p = pitch(d)
    wq = torch.zeros((V, p), dtype=torch.int8, device="cuda")
    for i in range(0, V, 1 << 17):
        wq[i:i + (1 << 17), :d] = torch.randint(-127, 128, (1 << 17, d), device="cuda", dtype=torch.int8)
    ws = torch.rand(V, device="cuda")
    h = torch.randn((1, M, d), device="cuda").bfloat16()
    q, s = torch.zeros((M, p), dtype=torch.int8, device="cuda"), torch.zeros(M, device="cuda")
    ns.nanospec_quant_rows(h[0], q, s)
    out = torch.zeros((M, V), device="cuda")
    ns.nanospec_quant_matmul(q, s, wq, ws, d, out)
    look = torch.tensor([0, 1, V // 2, V - 4097, V - 2, V - 1], device="cuda")
    rows = wq[look].cpu().numpy()
    want = replica(q.cpu().numpy(), s.cpu().numpy(), rows, ws[look].cpu().numpy())
    assert np.array_equal(out[:, look].cpu().numpy(), want)
    # more than 64 tokens
    x = q[torch.arange(70, device="cuda") % M].contiguous()
    xs = s[torch.arange(70, device="cuda") % M].contiguous()
    big = torch.zeros((70, V), dtype=torch.bfloat16, device="cuda")
    ns.nanospec_quant_matmul(x, xs, wq, ws, d, big)
    assert torch.equal(big[69 % M][look].cpu(), torch.from_numpy(want[69 % M]).bfloat16())
    assert torch.equal(big[69][look].cpu(), torch.from_numpy(want[0]).bfloat16())
    # the restricted head, few rows and many
    for n in (50, 20000):
        ids = torch.arange(V - n, V, device="cuda", dtype=torch.int32).view(1, -1)
        ti, tv = torch.zeros((1, M, 4), dtype=torch.int32, device="cuda"), torch.zeros((1, M, 4), device="cuda")
        ns.nanospec_quant_logits_topk(wq, ws, ids, None, h, 4, None, ti, tv, ns.alloc_quant_logits_workspace(1, n, M, 4, d))
        best = torch.topk(out[:, V - n:], 4)
        assert torch.equal(tv[0], best.values)
        assert torch.equal(ti[0], (best.indices + V - n).int())


def test_logits_past_four_gigabytes(ns):
    L, V = 17000, 128256                                   # 4.4 GB of bf16 logits
    z = torch.zeros((L, V), dtype=torch.bfloat16, device="cuda")
    last = torch.randn((3, V), device="cuda").mul_(3).bfloat16()
    z[L - 3:] = last
    tok = torch.full((L, 1), V - 1, dtype=torch.int32, device="cuda")
    lp, lse, H = torch.zeros((L, 1), device="cuda"), torch.zeros(L, device="cuda"), torch.zeros(L, device="cuda")
    ti, tv = torch.zeros((L, 2), dtype=torch.int32, device="cuda"), torch.zeros((L, 2), device="cuda")
    ns.nanospec_token_logprobs(z, 1.0, tok, lp, lse, H, ti, tv, ns.alloc_token_logprobs_workspace(L, V, 2))
    r = reference(last, 1.0, np.full((3, 1), V - 1), 2)
    near(lse[L - 3:], r["lse"], U * (8 * r["Z"] + 300), "last rows")
    assert np.array_equal(ti[L - 3:].cpu().numpy(), r["ids"])
    assert (ti[:L - 3].cpu() == torch.tensor([0, 1], dtype=torch.int32)).all()
    near(lse[:L - 3], np.full(L - 3, np.log(V)), np.full(L - 3, U * 300), "zero rows")
    g = torch.ones((L, 1), device="cuda")
    ns.nanospec_token_logprobs_grad(z, 1.0, tok, lse, None, g, None, None, z)      # in place
    p = np.exp(r["logp"])
    d = -p
    d[:, V - 1] += 1
    near(z[L - 3:], d, p * U * (8 * r["Z"][:, None] + 400) * 2 + np.abs(d) * 2.0 ** -8 + 2.0 ** -133, "last gradients")
