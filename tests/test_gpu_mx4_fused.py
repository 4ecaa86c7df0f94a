"""The 4-bit head that quantises its hidden rows in the product's launch, beside
the sizes where it is taken, and the product over few rows with every number of
chunks that may be left to a wave."""
import pytest
import torch

from tests.test_gpu_mx4 import check_head, check_product

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ns():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from dynamic_vocab_draft_amd import nanospec
    return nanospec


# M, n_max, d: groups of eight hidden rows by chunks a wave, one to four of them and one more
HEADS = [(1, 100, 8), (2, 33, 257), (8, 700, 2048), (8, 300, 2049), (9, 300, 2041), (16, 200, 4096), (17, 300, 2047), (24, 1000, 1000), (25, 500, 130),
         (32, 400, 2048), (33, 400, 256), (3, 90, 8192), (7, 120, 8001), (8, 130, 8193), (16, 100, 4100), (24, 80, 2050)]


@pytest.mark.parametrize("c", HEADS, ids=lambda c: "x".join(str(v) for v in c))
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_heads(ns, c, dtype):
    M, n, d = c
    check_head(ns, 1, M, min(5, n), n, n + 50, d, dtype)


@pytest.mark.parametrize("c", [(2, 8, 4096, 256), (1, 8, 16400, 40), (1, 8, 8192, 264), (1, 16, 8200, 64), (5, 20, 1000, 90), (40, 32, 100, 72)],
                         ids=lambda c: "x".join(str(v) for v in c))
def test_heads_of_many_rows(ns, c):
    B, M, n, d = c
    live = [n - 3 * (b % 2) if b != 1 else 5 for b in range(B)]
    check_head(ns, B, M, 3, n, n + 70, d, "bf16", live=live, holes=4, logits=False)
    check_head(ns, B, M, 3, n, n + 70, d, "fp32", live=live, logits=B < 10)


@pytest.mark.parametrize("d", [1792, 2048, 2816, 4096, 6144, 8192, 10240, 12544, 16384])
def test_products_of_few_rows(ns, d):
    for M, N in ((3, 100), (20, 70), (40, 50), (64, 33)):
        check_product(ns, M, N, d, "fp32", exact=False)
    check_product(ns, 9, 8192 if d == 1792 else 40, d, "bf16", exact=False)
