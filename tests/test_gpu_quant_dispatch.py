"""The forms of the restricted 8-bit head and of the 8-bit product that are taken by size, each against the definition:
the streamed head of eight-row units (8192 to 65536 columns over all sequences) and of taller ones (more), for each number
of token tiles, with ids and without; the selection's join of many chunks; and products whose output rows lie so far apart
that 31 bits do not reach them.  Integers, ids and values are compared for equality (see test_gpu_quant.py)."""
import numpy as np
import pytest
import torch

from tests.gpu_common import say
from tests.test_gpu_quant import DT, check_head, head_case, int8_rows, ns, replica  # noqa: F401

pytestmark = pytest.mark.gpu


def ragged(B, n_max, seed):
    """Live counts: none, one, all, past the end, and ones that end inside a unit of 8, 16 and 32 rows."""
    rng = np.random.default_rng(seed)
    n = rng.integers(0, n_max + 1, B)
    n[:7] = [0, n_max, 1, n_max + 5, n_max - 1, -1, n_max // 32 * 32 - 15][:B]
    return n.tolist()


STREAMS = [
    # B, n_max, M, d, V, dtype, k, holes
    # eight-row units
    (10, 1000, 20, 264, 1500, "bf16", 8, 0.05), (6, 2000, 40, 136, 2500, "fp16", 16, 0.1),
    (129, 70, 3, 320, 200, "bf16", 5, 0.0), (257, 40, 33, 72, 100, "fp32", 40, 0.1), (300, 64, 64, 128, 70, "bf16", 4, 0.0),
    (52, 1000, 48, 96, 1300, "bf16", 10, 0.2), (1, 9000, 32, 640, 9500, "fp32", 20, 0.05),
    # taller units
    (33, 2048, 9, 392, 3000, "bf16", 8, 0.05), (40, 1700, 20, 264, 2000, "bf16", 64, 0.0),
    (33, 2048, 40, 136, 2100, "fp16", 7, 0.1), (64, 2048, 64, 72, 2500, "bf16", 8, 0.05),
    (260, 300, 16, 200, 400, "fp32", 3, 0.3), (520, 128, 33, 64, 140, "bf16", 8, 0.1), (5, 14000, 17, 128, 15000, "bf16", 33, 0.02),
    (2, 40000, 49, 64, 41000, "bf16", 9, 0.0),
    # and with more stages a row than the ring holds
    (33, 2048, 8, 1100, 2300, "bf16", 8, 0.05), (36, 1900, 30, 904, 2000, "bf16", 6, 0.0),
    (33, 2048, 45, 1000, 2100, "fp16", 5, 0.05), (33, 2040, 60, 1000, 2100, "bf16", 16, 0.0),
]


@pytest.mark.parametrize("c", STREAMS, ids=lambda c: "x".join(str(v) for v in c))
def test_streamed_head(ns, c):  # noqa: F811
    B, n_max, M, d, V, dtype, k, holes = c
    case = head_case(B, n_max, M, d, V, dtype, 3, ragged(B, n_max, 4), holes)
    check_head(ns, case, k, True, what=str(c))
    check_head(ns, case[:4] + (None,), k, False, what=str(c) + " all live")


@pytest.mark.parametrize("B,V,M,d,counts", [(1, 70001, 9, 192, None), (1, 70001, 17, 64, [69999]), (1, 66000, 40, 72, None),
                                            (1, 65600, 64, 128, None), (1, 20000, 33, 128, None), (4, 18000, 12, 64, [18000, 0, 17, 9001]),
                                            (12, 900, 20, 128, None), (3, 128256, 3, 64, [128256, 100000, 3])])
def test_streamed_head_over_the_whole_vocabulary(ns, B, V, M, d, counts):  # noqa: F811
    check_head(ns, head_case(B, V, M, d, V, "bf16", 6, counts, ids=False), 8, True, what=f"full {B} {V} {M} {d}")


@pytest.mark.parametrize("V,M,k,counts", [(270001, 2, 64, [270001]), (270001, 2, 64, [262145]), (270001, 3, 64, [16385]),
                                          (270001, 2, 61, [16384]), (1 << 20, 1, 64, None)])
def test_selection_of_many_chunks(ns, V, M, k, counts):  # noqa: F811
    """More than 1024 keys of chunks to join, up to the 4096 of the largest vocabulary; counts that leave one chunk."""
    check_head(ns, head_case(1, V, M, 8, V, "bf16", 6, counts, ids=False), k, False, what=f"chunks {V} {k} {counts}")


def test_selection_of_many_chunks_that_tie(ns):  # noqa: F811
    wq, ws, h, I, n = head_case(1, 280000, 2, 8, 280000, "bf16", 6, [279999], ids=False)
    wq[:] = wq[np.arange(len(wq)) % 3]
    ws[:] = 0.5
    check_head(ns, (wq, ws, h, I, n), 64, False, what="many chunks, ties")


@pytest.mark.parametrize("M,N,out", [(3, 5000, "fp32"), (20, 4100, "bf16"), (64, 16400, "fp16"), (100, 66000, "bf16"), (128, 65537, "fp32"),
                                       (5000, 7, "bf16"), (70, 64, "fp32")])
def test_outputs_past_31_bits(ns, M, N, out):  # noqa: F811
    say("quant_matmul past 31 bits", M, N, out)
    d = 130
    size = torch.finfo(DT[out]).bits // 8
    ld = (1 << 31) // (size * (M - 1)) + 77               # the last row begins past 2 GiB
    assert ((M - 1) * ld + N) * size >= 1 << 31
    xq, wq = int8_rows(M, d, 1), int8_rows(N, d, 2)
    rng = np.random.default_rng(3)
    xs, ws = (np.exp(rng.standard_normal(n)).astype(np.float32) * 0.01 for n in (M, N))
    mem = torch.full((M * ld,), 1.5, dtype=DT[out], device="cuda")
    o = mem.view(M, ld)
    dev = lambda a: torch.from_numpy(a).cuda()
    ns.nanospec_quant_matmul(dev(xq), dev(xs), dev(wq), dev(ws), d, o[:, :N])
    torch.cuda.synchronize()
    assert torch.equal(o[:, :N].cpu(), torch.from_numpy(replica(xq, xs, wq, ws)).to(DT[out]))
    assert bool((o[:, N:] == 1.5).all()), "wrote between the rows"
