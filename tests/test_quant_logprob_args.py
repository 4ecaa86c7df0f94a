"""Argument checks of the 8-bit rows and the token log-probabilities that need
no GPU: the C entry points refuse before anything is enqueued, and the binding
refuses tensors whose device, type, shape or strides do not fit (it would
otherwise hand the kernels addresses they may not read)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def ns():
    from dynamic_vocab_draft_amd import nanospec
    return nanospec


FAKE = ctypes.c_void_p(0x10000)          # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10001)


def refused(call, base, **cases):
    for name, value in cases.items():
        for v in value if isinstance(value, list) else [value]:
            yield name, v, call(**dict(base, **{name: v}))


def test_quant_rows_and_matmul(ns):
    L = ns._lib
    assert [L.nanospec_quant_pitch(d) for d in (-1, 0, 1, 128, 129, 4096, 16384, 16385)] == \
        [0, 0, 128, 128, 256, 4096, 16384, 0]
    big = ns.NS_MAX_ROWS + 1

    def rows(x, ld, R, d, dtype, q, s):
        return L.nanospec_quant_rows(x, ld, R, d, dtype, q, s, None)
    base = dict(x=FAKE, ld=64, R=2, d=64, dtype=0, q=FAKE, s=FAKE)
    for name, v, rc in refused(rows, base, x=[None, ODD], ld=[63, 2 ** 41], R=[-1, big], d=[0, -5, 16385], q=[None, ODD], s=None):
        assert rc == ns.NS_EINVAL, (name, v)
    assert rows(**dict(base, dtype=3)) == ns.NS_EDTYPE
    assert rows(**dict(base, R=0, x=None)) == ns.NS_OK

    def mm(xq, xs, M, wq, ws, N, d, out, ld, dtype):
        return L.nanospec_quant_matmul(xq, xs, M, wq, ws, N, d, out, ld, dtype, None)
    base = dict(xq=FAKE, xs=FAKE, M=2, wq=FAKE, ws=FAKE, N=8, d=64, out=FAKE, ld=8, dtype=0)
    for name, v, rc in refused(mm, base, xq=[None, ODD], xs=None, M=[-1, big], wq=[None, ODD], ws=None,
                               N=[0, -1, ns.NS_MAX_V + 1], d=[0, 16385], out=[None, ODD], ld=[7, 2 ** 41]):
        assert rc == ns.NS_EINVAL, (name, v)
    assert mm(**dict(base, dtype=-1)) == ns.NS_EDTYPE
    assert mm(**dict(base, M=0, xq=None)) == ns.NS_OK


def test_quant_head(ns):
    L = ns._lib
    size = L.nanospec_quant_logits_workspace_bytes
    need = size(1, 100, 8, 8, 64)
    assert need > 0 and need % 256 == 0
    for bad in ((0, 100, 8, 8, 64), (ns.NS_MAX_BATCH + 1, 100, 8, 8, 64), (1, 0, 8, 8, 64),
                (1, ns.NS_MAX_V + 1, 8, 8, 64), (1, 100, 0, 8, 64), (1, 100, 65, 8, 64), (1, 100, 8, 0, 64),
                (1, 100, 8, 65, 64), (1, 100, 8, 8, 0), (1, 100, 8, 8, 16385)):
        assert size(*bad) == 0, bad

    def head(wq, sc, ids, n, n_max, B, V, d, h, dtype, M, k, lg, ti, tv, ws, wb):
        return L.nanospec_quant_logits_topk(wq, sc, ids, n, n_max, B, V, d, h, dtype, M, k, lg, ti, tv, ws, wb, None)
    base = dict(wq=FAKE, sc=FAKE, ids=FAKE, n=FAKE, n_max=100, B=1, V=200, d=64, h=FAKE, dtype=0, M=8, k=8, lg=None,
                ti=FAKE, tv=FAKE, ws=FAKE, wb=need)
    for name, v, rc in refused(head, base, wq=[None, ODD], sc=None, n_max=[0, ns.NS_MAX_V + 1], B=[0, 5000],
                               V=[0, ns.NS_MAX_V + 1], d=[0, 16385], h=[None, ODD], M=[0, 65], k=[0, 65], ti=None,
                               tv=None, ws=[None, ctypes.c_void_p(0x10010)]):
        assert rc == ns.NS_EINVAL, (name, v)
    assert head(**dict(base, ids=None, V=99)) == ns.NS_EINVAL           # n_max rows of a smaller vocabulary
    assert head(**dict(base, dtype=9)) == ns.NS_EDTYPE
    assert head(**dict(base, wb=need - 1)) == ns.NS_ECAPACITY


def test_token_logprobs(ns):
    L = ns._lib
    size = L.nanospec_token_logprobs_workspace_bytes
    need = size(4, 100, 8)
    assert need > 0 and size(0, 100, 0) > 0
    for bad in ((-1, 100, 8), (ns.NS_MAX_ROWS + 1, 100, 8), (4, 0, 0), (4, ns.NS_MAX_V + 1, 8), (4, 100, -1),
                (4, 100, 65), (4, 7, 8)):
        assert size(*bad) == 0, bad
    nan, inf = float("nan"), float("inf")

    def fwd(z, ld, R, V, dtype, it, tok, T, k, lp, lse, H, ti, tv, ws, wb):
        return L.nanospec_token_logprobs(z, ld, R, V, dtype, it, tok, T, k, lp, lse, H, ti, tv, ws, wb, None)
    base = dict(z=FAKE, ld=100, R=4, V=100, dtype=0, it=1.0, tok=FAKE, T=2, k=8, lp=FAKE, lse=FAKE, H=FAKE, ti=FAKE,
                tv=FAKE, ws=FAKE, wb=need)
    for name, v, rc in refused(fwd, base, z=[None, ODD], ld=[99, 2 ** 41], R=[-1, ns.NS_MAX_ROWS + 1], V=[0, ns.NS_MAX_V + 1],
                               it=[0.0, -1.0, nan, inf, 2.0 ** -21, 2.0 ** 21], tok=None, T=[-1, 65], k=[-1, 65],
                               lp=None, lse=None, ti=None, tv=None, ws=[None, ctypes.c_void_p(0x10010)]):
        assert rc == ns.NS_EINVAL, (name, v)
    assert fwd(**dict(base, V=7)) == ns.NS_EINVAL                       # k > V
    assert fwd(**dict(base, dtype=3)) == ns.NS_EDTYPE
    assert fwd(**dict(base, wb=need - 512)) == ns.NS_ECAPACITY
    assert fwd(**dict(base, R=0, z=None)) == ns.NS_OK

    def bwd(z, ld, R, V, dtype, it, tok, T, lse, H, g, gH, gl, d, ldd):
        return L.nanospec_token_logprobs_grad(z, ld, R, V, dtype, it, tok, T, lse, H, g, gH, gl, d, ldd, None)
    out = ctypes.c_void_p(0x20000)
    base = dict(z=FAKE, ld=100, R=4, V=100, dtype=0, it=1.0, tok=FAKE, T=2, lse=FAKE, H=FAKE, g=FAKE, gH=FAKE, gl=FAKE,
                d=out, ldd=100)
    for name, v, rc in refused(bwd, base, z=[None, ODD], ld=99, R=-1, V=0, it=[0.0, nan, inf], tok=None, T=[-1, 65],
                               lse=None, H=None, g=None, d=[None, ODD], ldd=[99, 2 ** 41]):
        assert rc == ns.NS_EINVAL, (name, v)
    assert bwd(**dict(base, d=FAKE, ldd=101)) == ns.NS_EINVAL           # in place with another stride
    assert bwd(**dict(base, dtype=3)) == ns.NS_EDTYPE
    assert bwd(**dict(base, R=0)) == ns.NS_OK


def test_binding_refuses_host_tensors(ns):
    f = torch.zeros
    i8, i32 = torch.int8, torch.int32
    calls = [
        lambda: ns.nanospec_quant_rows(f(2, 64), f(2, 128, dtype=i8), f(2)),
        lambda: ns.nanospec_quant_matmul(f(2, 128, dtype=i8), f(2), f(3, 128, dtype=i8), f(3), 64, f(2, 3)),
        lambda: ns.nanospec_quant_logits_topk(f(9, 128, dtype=i8), f(9), None, None, f(1, 2, 64), 2, None,
                                              f(1, 2, 2, dtype=i32), f(1, 2, 2), f(4096, dtype=torch.uint8)),
        lambda: ns.nanospec_token_logprobs(f(2, 64), 1.0, None, None, f(2), None, None, None,
                                           f(4096, dtype=torch.uint8)),
        lambda: ns.nanospec_token_logprobs_grad(f(2, 64), 1.0, None, f(2), None, None, None, None, f(2, 64)),
    ]
    for c in calls:
        with pytest.raises(ns.NanoSpecError) as e:
            c()
        assert e.value.code == ns.NS_EINVAL


@pytest.mark.gpu
def test_binding_refuses_misfits(ns):
    f = lambda *s, t=torch.float32: torch.zeros(s, dtype=t, device="cuda")
    i8, i32, u8 = torch.int8, torch.int32, torch.uint8

    def fails(fn, code=ns.NS_EINVAL):
        with pytest.raises(ns.NanoSpecError) as e:
            fn()
        assert e.value.code == code

    q = ns.nanospec_quant_rows
    fails(lambda: q(f(2, 64), f(2, 64, t=i8), f(2)))                       # no pitch
    fails(lambda: q(f(2, 64), f(2, 128, t=i8), f(3)))
    fails(lambda: q(f(64, 2).t(), f(2, 128, t=i8), f(2)))                  # columns contiguous
    fails(lambda: q(f(1, 64).expand(2, 64), f(2, 128, t=i8), f(2)))        # the same row twice
    fails(lambda: q(f(2, 64), f(2, 128, t=u8), f(2)), ns.NS_EDTYPE)
    fails(lambda: q(f(2, 64, t=torch.float64), f(2, 128, t=i8), f(2)), ns.NS_EDTYPE)
    fails(lambda: q(f(2, 64), f(2, 128, t=i8), torch.zeros(2)))            # a host tensor among them
    m = ns.nanospec_quant_matmul
    fails(lambda: m(f(2, 128, t=i8), f(2), f(3, 256, t=i8), f(3), 64, f(2, 3)))
    fails(lambda: m(f(2, 128, t=i8), f(2), f(3, 128, t=i8), f(3), 64, f(3, 2).t()))
    fails(lambda: m(f(2, 128, t=i8), f(2), f(3, 128, t=i8), f(3), 64, f(2, 3, t=i32)), ns.NS_EDTYPE)
    h = ns.nanospec_quant_logits_topk
    work = ns.alloc_quant_logits_workspace(1, 9, 2, 2, 64)
    args = [f(9, 128, t=i8), f(9), f(1, 9, t=i32), f(1, t=i32), f(1, 2, 64), 2, None, f(1, 2, 2, t=i32), f(1, 2, 2), work]
    h(*args)
    for at, bad in ((0, f(9, 64, t=i8)), (1, f(8)), (2, f(9, t=i32)), (3, f(2, t=i32)), (4, f(2, 64)), (5, 3),
                    (6, f(1, 2, 8)), (7, f(1, 2, 3, t=i32)), (8, f(2, 2)), (9, work[128:])):
        fails(lambda: h(*(args[:at] + [bad] + args[at + 1:])))
    fails(lambda: h(*(args[:9] + [work[:256]])), ns.NS_ECAPACITY)
    p = ns.nanospec_token_logprobs
    work = ns.alloc_token_logprobs_workspace(2, 64, 3)
    args = [f(2, 64), 1.0, f(2, 1, t=i32), f(2, 1), f(2), f(2), f(2, 3, t=i32), f(2, 3), work]
    p(*args)
    for at, bad in ((0, f(64)), (1, 0.0), (2, f(2, t=i32)), (2, None), (3, f(2, 2)), (4, f(3)), (5, f(2, 1)), (6, None),
                    (7, f(2, 4)), (8, work[128:])):
        fails(lambda: p(*(args[:at] + [bad] + args[at + 1:])))
    fails(lambda: p(*(args[:8] + [work[:256]])), ns.NS_ECAPACITY)
    g = ns.nanospec_token_logprobs_grad
    z = f(2, 64)
    args = [z, 1.0, f(2, 1, t=i32), f(2), f(2), f(2, 1), f(2), f(2), f(2, 64)]
    g(*args)
    for at, bad in ((3, f(1)), (4, None), (5, f(1, 2)), (5, None), (6, f(2, 2)), (7, f(5)), (8, f(2, 63)),
                    (8, f(64, 2).t())):
        fails(lambda: g(*(args[:at] + [bad] + args[at + 1:])))
    fails(lambda: g(*(args[:8] + [f(2, 64, t=torch.bfloat16)])), ns.NS_EDTYPE)
    torch.cuda.synchronize()
