"""Forms of the 4-bit product and head that are taken by size: tiles of every
height over several rounds, the streams of every unit height and number of token
operands, rows past 2 GB and outputs past 31 bits, the fused head, long rows."""
import numpy as np
import pytest
import torch

from tests.gpu_common import say
from tests.test_gpu_mx4 import check_head, check_product, made, on_gpu, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ns():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from dynamic_vocab_draft_amd import nanospec
    return nanospec


# tiles: 256 tokens (several tiles a block), 128 and 64; one chunk a row, two, an odd number of them
TILES = [(1030, 20000, 256, "bf16"), (520, 40000, 300, "fp32"), (2050, 9000, 700, "fp16"), (300, 12000, 1100, "bf16"), (140, 70000, 256, "fp16"),
         (130, 5000, 600, "fp32"), (400, 2500, 3000, "bf16"), (1000, 1000, 16384, "bf16"), (65, 5000, 31, "fp32")]


@pytest.mark.parametrize("c", TILES, ids=lambda c: "x".join(str(v) for v in c))
def test_tiles(ns, c):
    check_product(ns, *c)


# streams: eight-row units (N <= 16384, or up to 16 tokens), 16 and 32 rows; rounds of passes; one chunk a row
STREAMS = [(m, n, d, t) for m in (3, 16, 17, 32, 40, 48, 50, 64) for n, d, t in ((5001, 300, "fp32"), (40003, 256, "bf16"), (33000, 1300, "fp16"))]


@pytest.mark.parametrize("c", STREAMS, ids=lambda c: "x".join(str(v) for v in c))
def test_streams(ns, c):
    check_product(ns, *c)


@pytest.mark.parametrize("c", [(5, 5000, 16384), (33, 4500, 16384), (64, 4500, 16300), (40, 17000, 8300)], ids=lambda c: "x".join(str(v) for v in c))
def test_streams_of_long_rows(ns, c):
    check_product(ns, *c, "fp32")


HEADS = [(m, n, d) for m in (7, 16, 20, 33, 48, 64) for n, d in ((6000, 300), (20000, 128))] + \
        [(8, 6000, 9000), (30, 5000, 9000), (33, 5000, 9000), (16, 2000, 4097), (12, 300, 4096), (16, 4096, 40)]


@pytest.mark.parametrize("c", HEADS, ids=lambda c: "x".join(str(v) for v in c))
def test_heads(ns, c):
    M, n, d = c
    check_head(ns, 1, M, 5, n, n + 1000, d, "bf16")
    if d < 500:
        check_head(ns, 3, M, 5, n, n + 1000, d, "fp16", live=[n, 7, 0], holes=9)


def test_many_sequences(ns):
    check_head(ns, 300, 2, 3, 40, 400, 64, "bf16", logits=False)
    check_head(ns, 130, 17, 3, 200, 400, 64, "fp32", logits=False)


def test_stored_rows_past_31_bits(ns):
    """A product and a head over more than 2 GB of rows, and rows read back from their end."""
    d, N = 16384, 290000
    p = ns.nanospec_mx4_pitch(d)
    rng = np.random.default_rng(3)
    (xq, xs), (tq, ts) = made(rng, 4, d), made(rng, 50, d)
    q = torch.zeros((N, p), dtype=torch.uint8, device="cuda")
    s = torch.full((N, p // 16), 127, dtype=torch.uint8, device="cuda")
    at = torch.from_numpy(np.sort(rng.permutation(N)[:50]))
    at[-1] = N - 1
    q[at.cuda()], s[at.cuda()] = on_gpu(tq, ts)
    want = (values(xq, xs, d) @ values(tq, ts, d).T).astype(np.float32)
    for M in (4, 70):
        say("rows past 2 GB", M)
        gx, gs = on_gpu(np.tile(xq, (M // 4 + 1, 1))[:M], np.tile(xs, (M // 4 + 1, 1))[:M])
        out = torch.zeros((M, N), device="cuda")
        ns.nanospec_mx4_matmul(gx, gs, q, s, d, out)
        got = out[:, at.cuda()].cpu().numpy()
        assert np.array_equal(got, np.tile(want, (M // 4 + 1, 1))[:M])
        assert int((out != 0).sum()) == int((got != 0).sum())
        del out
    back = torch.zeros((50, d), device="cuda")
    ns.nanospec_mx4_gather_rows(q, s, at.to(torch.int32).cuda(), None, back)
    assert np.array_equal(back.double().cpu().numpy(), values(tq, ts, d))
    h = torch.from_numpy(values(xq, xs, d).astype(np.float32))[None].cuda()      # quantises to itself
    oi, ov = torch.zeros((1, 4, 1), dtype=torch.int32, device="cuda"), torch.zeros((1, 4, 1), device="cuda")
    ids = torch.arange(0, N, 29, dtype=torch.int32)
    ids = torch.cat([ids, at.to(torch.int32)]).unique()[None].contiguous()
    ns.nanospec_mx4_logits_topk(q, s, ids.cuda(), None, h, 1, None, oi, ov, ns.alloc_mx4_logits_workspace(1, ids.shape[1], 4, 1, d))
    assert np.array_equal(ov[0, :, 0].cpu().numpy(), want.max(1)) and np.array_equal(oi[0, :, 0].cpu().numpy(), at.numpy()[want.argmax(1)])


def test_outputs_past_31_bits(ns):
    """Rows of outputs far apart, for the kernels with 31-bit output offsets and those with more."""
    d = 64
    rng = np.random.default_rng(4)
    for M, N, ld in ((3, 5000, 1 << 29), (70, 5000, 1 << 24)):
        say("outputs past 31 bits", M, N, ld)
        (xq, xs), (wq, ws) = made(rng, M, d), made(rng, N, d)
        mem = torch.zeros(((M - 1) * ld + N,), dtype=torch.bfloat16, device="cuda")
        out = mem.as_strided((M, N), (ld, 1))
        ns.nanospec_mx4_matmul(*on_gpu(xq, xs, wq, ws), d, out)
        want = torch.from_numpy(values(xq, xs, d) @ values(wq, ws, d).T).float().bfloat16()
        assert torch.equal(out.cpu(), want)
        del mem, out
