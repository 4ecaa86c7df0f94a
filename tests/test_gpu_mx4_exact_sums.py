"""The bound within which a 4-bit product is exact in every form: blocks whose
scales (x's and w's together) lie within 2^s of one another and 144 d 2^s <= 2^24,
at the largest magnitudes, all of one sign."""
import numpy as np
import pytest
import torch

from tests.test_gpu_mx4 import on_gpu, packed, pitch, values


@pytest.fixture(scope="module")
def ns():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from dynamic_vocab_draft_amd import nanospec
    return nanospec


def spread_of(d):
    """The largest s of 144 d 2^s <= 2^24."""
    return int(np.floor(np.log2(2.0 ** 24 / (144 * d))))


def rows(rng, n, d, spread):
    """Stored rows: three quarters of the elements 6, the rest the smallest, a half; scales `spread` apart at random, both ends taken."""
    blocks = -(-d // 32)
    code = np.where(rng.random((n, blocks, 32)) < 0.75, 7, 1)
    code.reshape(n, -1)[:, d:] = 0
    scale = 120 + rng.integers(0, spread + 1, (n, blocks))
    scale[:, 0], scale[:, -1] = 120, 120 + spread
    return packed(code, scale, d)


def test_bound():
    """In float32 alone: any order within the bound, not at a spread of 2^10."""
    rng = np.random.default_rng(0)
    d = 4096
    assert spread_of(d) == 4 and spread_of(16384) == 2
    for s, exact in ((4, True), (10, False)):
        x = np.where(np.arange(d) < d // 2, 36.0 * 2 ** s, 0.25).astype(np.float32)
        sums = set()
        for order in (np.arange(d), np.arange(d)[::-1], rng.permutation(d)):
            sums.add(float(np.cumsum(x[order], dtype=np.float32)[-1]))
        assert (sums == {float(x.astype(np.float64).sum())}) == exact


# the kernel for few rows, streams of every unit height, tiles
@pytest.mark.gpu
@pytest.mark.parametrize("c", [(3, 40, 4096), (60, 300, 16384), (8, 17000, 4096), (30, 9000, 4096), (30, 17000, 1024), (64, 17000, 1024), (100, 9000, 4096),
                               (300, 2000, 16384), (70, 300, 4000), (1030, 9000, 300)], ids=lambda c: "x".join(map(str, c)))
def test_products(ns, c):
    M, N, d = c
    rng = np.random.default_rng(M + N + d)
    s = spread_of(d)
    (xq, xs), (wq, ws) = rows(rng, M, d, s // 2), rows(rng, N, d, s - s // 2)
    want = torch.from_numpy(values(xq, xs, d)).float() @ torch.from_numpy(values(wq, ws, d)).float().t()
    picked = rng.integers(0, N, 50)                  # the host's float32 sums are exact by the same bound; some of them in float64 as well
    assert np.array_equal(want[:, picked].double().numpy(), values(xq, xs, d) @ values(wq[picked], ws[picked], d).T)
    out = torch.zeros((M, N), device="cuda")
    ns.nanospec_mx4_matmul(*on_gpu(xq, xs, wq, ws), d, out)
    assert torch.equal(out.cpu(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("c", [(1, 8, 1000, 4096), (1, 8, 17000, 4096), (2, 40, 300, 4096), (1, 40, 9000, 4096), (8, 20, 4096, 1024)],
                         ids=lambda c: "x".join(map(str, c)))
def test_heads(ns, c):
    """Logits do not depend on how many columns are live, nor on the other sequences."""
    B, M, n, d = c
    rng = np.random.default_rng(n + d)
    s = spread_of(d)
    wq, ws = rows(rng, n, d, s - s // 2)
    xq, xs = rows(rng, B * M, d, s // 2)
    x = values(xq, xs, d)                            # quantises to itself: each block's largest is 6
    h = torch.from_numpy(x.reshape(B, M, d)).float().cuda()
    want = (torch.from_numpy(x).float() @ torch.from_numpy(values(wq, ws, d)).float().t()).view(B, M, n)
    picked = rng.integers(0, n, 50)
    assert np.array_equal(want.reshape(B * M, n)[:, picked].double().numpy(), x @ values(wq[picked], ws[picked], d).T)
    ids = torch.arange(n, dtype=torch.int32).repeat(B, 1).cuda()
    gq, gs = on_gpu(wq, ws)
    work = ns.alloc_mx4_logits_workspace(B, n, M, 2, d)
    for live in (n, n // 2 + 1, 5):
        z = torch.full((B, M, n), 7.0, device="cuda")
        oi, ov = torch.zeros((B, M, 2), dtype=torch.int32, device="cuda"), torch.zeros((B, M, 2), device="cuda")
        ns.nanospec_mx4_logits_topk(gq, gs, ids, torch.full((B,), live, dtype=torch.int32, device="cuda"), h, 2, z, oi, ov, work)
        assert torch.equal(z[..., :live].cpu(), want[..., :live]) and (z[..., live:] == 7).all()
        assert torch.equal(ov.cpu(), want[..., :live].sort(2, descending=True).values[..., :2])


def test_rows_are_stored_as_they_are_meant():
    q, s = rows(np.random.default_rng(1), 3, 70, 2)
    assert q.shape == (3, pitch(70)) and (values(q, s, 70) > 0).all() and set(s[:, :3].ravel()) <= {120, 121, 122}
