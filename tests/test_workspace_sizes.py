"""A workspace that fits the largest call of a loop fits its smaller ones: the size queries never fall as a dimension
grows, though fewer rows are split into more parts each."""
import pytest


@pytest.fixture(scope="module")
def ns():
    from dynamic_vocab_draft_amd import nanospec
    return nanospec


def rising(sizes):
    return all(0 < a <= b for a, b in zip(sizes, sizes[1:]))


def test_token_logprobs(ns):
    size = ns.nanospec_token_logprobs_workspace_bytes
    Ls = list(range(0, 3200)) + [4095, 4096, 10000, 1 << 20]
    Vs = sorted({v + o for v in (64, 256, 512, 1024, 4096, 8192, 65536, 128256, 151936) for o in (-1, 0, 1)}) + [1 << 20]
    for k in (0, 1, 16, 33):
        for V in (64, 300, 1025, 5000, 20011, 50257, 128256, 1 << 20):
            assert rising([size(L, V, k) for L in Ls]), (V, k)
        for L in (1, 3, 47, 511, 512, 767, 1535, 1536, 5000):
            assert rising([size(L, V, k) for V in Vs]), (L, k)
    for L, V in ((1, 128256), (1535, 5000), (3000, 151936)):
        assert rising([size(L, V, k) for k in range(65)]), (L, V)


def test_quant_head(ns):
    size = ns.nanospec_quant_logits_workspace_bytes
    edges = sorted({v + o for v in (1, 64, 4096, 8192, 16384, 32768, 262144) for o in (0, 1, 2)}) + [1 << 20]
    for M in (1, 17, 64):
        for k in (1, 64):
            assert rising([size(2, n, M, k, 4096) for n in edges])
            assert rising([size(B, 5000, M, k, 512) for B in (1, 2, 3, 128, 129, 4096)])
            assert rising([size(1, 20000, M, k, d) for d in (1, 127, 128, 129, 4096, 16384)])
    assert rising([size(1, 20000, M, 8, 512) for M in range(1, 65)])
    assert rising([size(1, 20000, 8, k, 512) for k in range(1, 65)])


@pytest.mark.gpu
def test_one_workspace_for_every_batch(ns):
    import torch
    L, V, k = 1536, 5000, 8
    work = ns.alloc_token_logprobs_workspace(L, V, k)
    z = torch.randn((L, V), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    for n in (1536, 1535, 1000, 511, 60, 1):
        e = lambda *s, t=torch.float32: torch.zeros(s, dtype=t, device="cuda")
        a, b = ((e(n), e(n, k, t=torch.int32), e(n, k)) for _ in range(2))
        ns.nanospec_token_logprobs(z[:n], 1.0, None, None, a[0], None, a[1], a[2], work)
        ns.nanospec_token_logprobs(z[:n], 1.0, None, None, b[0], None, b[1], b[2], ns.alloc_token_logprobs_workspace(n, V, k))
        assert all(torch.equal(x, y) for x, y in zip(a, b)), n
        # within u (8 Z + 300) of float64, Z below 5
        assert (a[2].double() - torch.log_softmax(z[:n].double(), 1).topk(k, 1).values).abs().max() < 340 * 2.0 ** -24, n
