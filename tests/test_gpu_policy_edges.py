"""Policy loss at the edges of its terms: reference log-probabilities far from the
policy's.  Definitions and tolerances are those of tests/test_gpu_policy.py."""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_policy import DT, Case, check

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
