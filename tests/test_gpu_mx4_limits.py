"""The 4-bit product beside the limits of its kernel for few rows: the most
blocks of it for a number of tokens and a row length, and one more."""
import pytest
import torch

from tests.test_gpu_mx4 import check_product

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ns():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from dynamic_vocab_draft_amd import nanospec
    return nanospec


# tokens, row length, blocks of 16 channels (by groups of 64 tokens)
LIMITS = [(7, 1000, 768), (16, 1020, 1024), (17, 300, 512), (48, 200, 512), (49, 700, 256), (64, 1000, 512), (64, 4300, 256), (65, 1700, 256), (65, 2040, 512),
          (500, 256, 256), (500, 1800, 512), (2048, 2040, 512), (2049, 2040, 256), (4000, 100, 256)]


@pytest.mark.parametrize("c", LIMITS, ids=lambda c: "x".join(map(str, c)))
def test_limits(ns, c):
    M, d, blocks = c
    most = blocks // -(-M // 64) * 16
    check_product(ns, M, most, d, "bf16")
    check_product(ns, M, most + 1, d, "fp32")
