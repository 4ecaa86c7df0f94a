"""The 4-bit head that quantises its hidden rows in the product's launch, beside
the sizes where it is taken, the product over few rows with every number of
chunks that may be left to a wave, and streams of eight-row units beside it."""
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


@pytest.mark.parametrize("M", [17, 32, 40, 48, 50, 64])
def test_streams_of_eight_row_units(ns, M):
    for n, d, dtype in ((8193, 300, "fp32"), (9001, 256, "bf16"), (16384, 1300, "fp16")):
        check_product(ns, M, n, d, dtype)
    check_head(ns, 1, M, 5, 9000, 10000, 300, "bf16")
    check_head(ns, 3, M, 5, 4500, 5500, 128, "fp16", live=[4500, 7, 0], holes=9)


@pytest.mark.parametrize("c", [(5, 16400, 4100), (40, 8200, 8300), (64, 8193, 9000)], ids=lambda c: "x".join(str(v) for v in c))
def test_streams_of_long_rows(ns, c):
    check_product(ns, *c, "fp32")


@pytest.mark.parametrize("c", [(8, 16400, 2100), (30, 8200, 4500), (40, 8200, 3000)], ids=lambda c: "x".join(str(v) for v in c))
def test_head_streams_of_long_rows(ns, c):
    M, n, d = c
    check_head(ns, 1, M, 5, n, n + 1000, d, "bf16")


@pytest.mark.parametrize("c", [(8, 16384, 300), (16, 9000, 700), (64, 8192, 520), (100, 4000, 700), (1000, 300, 520), (520, 1024, 40)],
                         ids=lambda c: "x".join(str(v) for v in c))
def test_products_of_few_rows_over_many_blocks(ns, c):
    check_product(ns, *c, "bf16")


@pytest.mark.parametrize("c", [(1, 8, 16000, 4100), (1, 64, 8000, 520), (3, 40, 2500, 4100), (1, 40, 300, 16384)],
                         ids=lambda c: "x".join(str(v) for v in c))
def test_heads_over_few_rows(ns, c):
    B, M, n, d = c
    check_head(ns, B, M, 5, n, n + 100, d, "bf16")
