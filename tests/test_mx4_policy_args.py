"""Argument checks of the 4-bit rows and of the policy loss that need no GPU:
the C entry points refuse before anything is enqueued, and the binding refuses
tensors whose device, type, shape or strides do not fit."""
import ctypes
import math
import os
import re

import pytest
import torch

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "nanospec.h")
FAKE = ctypes.c_void_p(0x10000)          # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10001)


@pytest.fixture(scope="module")
def ns():
    from dynamic_vocab_draft_amd import nanospec
    return nanospec


def refused(call, base, **cases):
    for name, value in cases.items():
        for v in value if isinstance(value, list) else [value]:
            yield name, v, call(**dict(base, **{name: v}))


def test_every_declared_name_is_exported_and_bound(ns):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(nanospec_[a-z0-9_]+)\s*\(", src))
    assert sum("mx4" in n for n in names) == 6 and "nanospec_policy_loss" in names
    for n in names:
        assert hasattr(ns._lib, n) and n in ns._SIGS, n


def test_rows_and_gather(ns):
    L = ns._lib
    assert [L.nanospec_mx4_pitch(d) for d in (-1, 0, 1, 256, 257, 4096, 16384, 16385)] == [0, 0, 128, 128, 256, 2048, 8192, 0]
    big = ns.NS_MAX_ROWS + 1

    def rows(x, ld, R, d, dtype, q, s):
        return L.nanospec_mx4_rows(x, ld, R, d, dtype, q, s, None)
    base = dict(x=FAKE, ld=64, R=2, d=64, dtype=0, q=FAKE, s=FAKE)
    for name, v, rc in refused(rows, base, x=[None, ODD], ld=[63, 2 ** 41], R=[-1, big], d=[0, -5, 16385],
                               q=[None, ctypes.c_void_p(0x10008)], s=[None, ctypes.c_void_p(0x10004)]):
        assert rc == ns.NS_EINVAL, (name, v)
    assert rows(**dict(base, dtype=3)) == ns.NS_EDTYPE
    assert rows(**dict(base, R=0, x=None)) == ns.NS_OK

    def gather(q, s, V, d, ids, n, n_max, out, ld, dtype):
        return L.nanospec_mx4_gather_rows(q, s, V, d, ids, n, n_max, out, ld, dtype, None)
    base = dict(q=FAKE, s=FAKE, V=10, d=64, ids=FAKE, n=None, n_max=20, out=FAKE, ld=64, dtype=1)
    for name, v, rc in refused(gather, base, q=[None, ODD], s=[None, ODD], V=[0, ns.NS_MAX_V + 1], d=[0, 16385], n_max=[-1, big],
                               out=[None, ODD], ld=[63, 2 ** 41], ids=None):
        assert rc == ns.NS_EINVAL, (name, v)
    assert gather(**dict(base, dtype=3)) == ns.NS_EDTYPE
    assert gather(**dict(base, n_max=0, q=None)) == ns.NS_OK


def test_matmul(ns):
    def mm(xq, xs, M, wq, ws, N, d, out, ld, dtype):
        return ns._lib.nanospec_mx4_matmul(xq, xs, M, wq, ws, N, d, out, ld, dtype, None)
    base = dict(xq=FAKE, xs=FAKE, M=2, wq=FAKE, ws=FAKE, N=8, d=64, out=FAKE, ld=8, dtype=0)
    for name, v, rc in refused(mm, base, xq=[None, ODD], xs=[None, ODD], M=[-1, ns.NS_MAX_ROWS + 1], wq=[None, ODD], ws=[None, ODD],
                               N=[0, -1, ns.NS_MAX_V + 1], d=[0, 16385], out=[None, ODD], ld=[7, 2 ** 41]):
        assert rc == ns.NS_EINVAL, (name, v)
    assert mm(**dict(base, dtype=-1)) == ns.NS_EDTYPE
    assert mm(**dict(base, M=0, xq=None)) == ns.NS_OK


def test_head(ns):
    L = ns._lib
    size = L.nanospec_mx4_logits_workspace_bytes
    need = size(1, 100, 8, 8, 64)
    assert need > 0 and need % 256 == 0
    for bad in ((0, 100, 8, 8, 64), (ns.NS_MAX_BATCH + 1, 100, 8, 8, 64), (1, 0, 8, 8, 64), (1, ns.NS_MAX_V + 1, 8, 8, 64),
                (1, 100, 0, 8, 64), (1, 100, 65, 8, 64), (1, 100, 8, 0, 64), (1, 100, 8, 65, 64), (1, 100, 8, 8, 0), (1, 100, 8, 8, 16385)):
        assert size(*bad) == 0, bad

    def head(wq, sc, ids, n, n_max, B, V, d, h, dtype, M, k, lg, ti, tv, ws, wb):
        return L.nanospec_mx4_logits_topk(wq, sc, ids, n, n_max, B, V, d, h, dtype, M, k, lg, ti, tv, ws, wb, None)
    base = dict(wq=FAKE, sc=FAKE, ids=FAKE, n=FAKE, n_max=100, B=1, V=200, d=64, h=FAKE, dtype=0, M=8, k=8, lg=None, ti=FAKE, tv=FAKE, ws=FAKE, wb=need)
    for name, v, rc in refused(head, base, wq=[None, ODD], sc=[None, ODD], n_max=[0, ns.NS_MAX_V + 1], B=[0, 5000], V=[0, ns.NS_MAX_V + 1],
                               d=[0, 16385], h=[None, ODD], M=[0, 65], k=[0, 65], ti=None, tv=None, ws=[None, ctypes.c_void_p(0x10010)]):
        assert rc == ns.NS_EINVAL, (name, v)
    assert head(**dict(base, ids=None, V=99)) == ns.NS_EINVAL           # n_max rows of a smaller vocabulary
    assert head(**dict(base, dtype=9)) == ns.NS_EDTYPE
    assert head(**dict(base, wb=need - 1)) == ns.NS_ECAPACITY


def test_policy(ns):
    L = ns._lib
    size = L.nanospec_policy_loss_workspace_bytes
    need = size(4, 100)
    assert need > 0 and need % 256 == 0 and size(0, 1) > 0
    for bad in ((-1, 100), (ns.NS_MAX_ROWS + 1, 100), (4, 0), (4, ns.NS_MAX_V + 1)):
        assert size(*bad) == 0, bad
    for V in (1, 1000, 50257, 128256, 1 << 20):                        # never falls as rows or columns are added
        sizes = [size(n, V) for n in (0, 1, 2, 3, 7, 8, 9, 31, 64, 100, 255, 256, 257, 511, 512, 513, 1000, 2047, 2048, 4096, 1 << 20)]
        assert sizes == sorted(sizes), V
    for n in (1, 8, 300, 4096):
        sizes = [size(n, V) for V in (1, 7, 8, 1000, 4095, 4096, 4097, 50257, 128256, 1 << 20)]
        assert sizes == sorted(sizes), n

    def policy(z, ld, n, V, dtype, t, tok, old, ref, adv, w, lo, hi, beta, ent, loss, lp, kl, H, g, dz, ldd, ws, wb):
        return L.nanospec_policy_loss(z, ld, n, V, dtype, t, tok, old, ref, adv, w, lo, hi, beta, ent, loss, lp, kl, H, g, dz, ldd, ws, wb, None)
    base = dict(z=FAKE, ld=100, n=4, V=100, dtype=1, t=1.0, tok=FAKE, old=FAKE, ref=FAKE, adv=FAKE, w=None, lo=0.2, hi=0.2, beta=0.1, ent=0.0,
                loss=FAKE, lp=FAKE, kl=None, H=None, g=None, dz=None, ldd=0, ws=FAKE, wb=need)
    nan = math.nan
    for name, v, rc in refused(policy, base, z=[None, ODD], ld=[99, 2 ** 41], n=[-1, ns.NS_MAX_ROWS + 1], V=[0, ns.NS_MAX_V + 1],
                               t=[0.0, -1.0, nan, 2.0 ** -21, 2.0 ** 21], tok=None, old=None, ref=None, adv=None, lo=[-0.1, 1.1, nan],
                               hi=[-0.1, nan], beta=[nan, math.inf], ent=[nan, -math.inf], loss=None, lp=None,
                               ws=[None, ctypes.c_void_p(0x10010)], dz=[FAKE, ODD]):
        assert rc == ns.NS_EINVAL, (name, v)
    assert policy(**dict(base, ref=None, beta=0.0, kl=FAKE)) == ns.NS_EINVAL            # a KL value without a reference
    apart = ctypes.c_void_p(0x900000)
    for ldd in (99, 2 ** 41):
        assert policy(**dict(base, dz=apart, ldd=ldd)) == ns.NS_EINVAL
    assert policy(**dict(base, dz=FAKE, ldd=104)) == ns.NS_EINVAL                       # in place with another stride
    assert policy(**dict(base, dtype=3)) == ns.NS_EDTYPE
    assert policy(**dict(base, wb=need - 1)) == ns.NS_ECAPACITY


def test_binding_refuses_misfits(ns):
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)   # noqa: E731
    f = lambda *s: torch.zeros(s)                       # noqa: E731
    calls = [lambda: ns.nanospec_mx4_rows(f(2, 64), u8(2, 128), u8(2, 8)),
             lambda: ns.nanospec_mx4_rows([1.0], u8(2, 128), u8(2, 8)),
             lambda: ns.nanospec_mx4_gather_rows(u8(2, 128), u8(2, 8), None, None, f(2, 64)),
             lambda: ns.nanospec_mx4_matmul(u8(2, 128), u8(2, 8), u8(3, 128), u8(3, 8), 64, f(2, 3)),
             lambda: ns.nanospec_mx4_logits_topk(u8(2, 128), u8(2, 8), None, None, f(1, 2, 64), 1, None, None, None, None),
             lambda: ns.nanospec_mx4_logits_topk(u8(2, 128), u8(2, 8), None, None, None, 1, None, None, None, None),
             lambda: ns.nanospec_policy_loss(f(2, 8), 1.0, None, None, None, None, None, 0.2, 0.2, 0.0, 0.0, None, None, None, None, None, None, None),
             lambda: ns.nanospec_policy_loss(f(8), 1.0, None, None, None, None, None, 0.2, 0.2, 0.0, 0.0, None, None, None, None, None, None, None),
             lambda: ns.alloc_mx4_logits_workspace(1, 0, 1, 1, 64), lambda: ns.alloc_policy_loss_workspace(1, 0)]
    for i, call in enumerate(calls):
        with pytest.raises(ns.NanoSpecError) as e:
            call()
        assert e.value.code == ns.NS_EINVAL, i


@pytest.mark.gpu
def test_binding_refuses_misfits_on_the_gpu(ns):
    f = lambda *s, t=torch.float32: torch.zeros(s, dtype=t, device="cuda")   # noqa: E731
    i32, u8 = torch.int32, torch.uint8

    def fails(fn, code=ns.NS_EINVAL):
        with pytest.raises(ns.NanoSpecError) as e:
            fn()
        assert e.value.code == code

    q = ns.nanospec_mx4_rows
    q(f(2, 64), f(2, 128, t=u8), f(2, 8, t=u8))
    fails(lambda: q(f(2, 64), f(2, 64, t=u8), f(2, 8, t=u8)))                                # no pitch
    fails(lambda: q(f(2, 64), f(2, 128, t=u8), f(2, 4, t=u8)))
    fails(lambda: q(f(64, 2).t(), f(2, 128, t=u8), f(2, 8, t=u8)))                           # columns contiguous
    fails(lambda: q(f(2, 64), f(2, 128, t=torch.int8), f(2, 8, t=u8)), ns.NS_EDTYPE)
    fails(lambda: q(f(2, 64, t=torch.float64), f(2, 128, t=u8), f(2, 8, t=u8)), ns.NS_EDTYPE)
    fails(lambda: q(f(2, 64), f(2, 128, t=u8), torch.zeros((2, 8), dtype=u8)))               # a host tensor among them
    r = ns.nanospec_mx4_gather_rows
    args = [f(4, 128, t=u8), f(4, 8, t=u8), f(3, t=i32), f(1, t=i32), f(3, 64)]
    r(*args)
    for at, bad in ((0, f(128, t=u8)), (1, f(3, 8, t=u8)), (2, f(2, t=i32)), (3, f(2, t=i32)), (4, f(64, 3).t()), (4, f(3, 300))):
        fails(lambda: r(*(args[:at] + [bad] + args[at + 1:])))
    fails(lambda: r(args[0], args[1], None, None, f(5, 64)))                                 # more rows than there are
    m = ns.nanospec_mx4_matmul
    args = [f(2, 128, t=u8), f(2, 8, t=u8), f(3, 128, t=u8), f(3, 8, t=u8), 64, f(2, 3)]
    m(*args)
    for at, bad in ((0, f(3, 128, t=u8)), (1, f(2, 16, t=u8)), (2, f(3, 256, t=u8)), (3, f(2, 8, t=u8)), (4, 300), (4, 0), (5, f(3, 2).t())):
        fails(lambda: m(*(args[:at] + [bad] + args[at + 1:])))
    fails(lambda: m(*(args[:5] + [f(2, 3, t=i32)])), ns.NS_EDTYPE)
    h = ns.nanospec_mx4_logits_topk
    work = ns.alloc_mx4_logits_workspace(1, 9, 2, 2, 64)
    args = [f(9, 128, t=u8), f(9, 8, t=u8), f(1, 9, t=i32), f(1, t=i32), f(1, 2, 64), 2, None, f(1, 2, 2, t=i32), f(1, 2, 2), work]
    h(*args)
    for at, bad in ((0, f(9, 64, t=u8)), (1, f(8, 8, t=u8)), (2, f(9, t=i32)), (3, f(2, t=i32)), (4, f(2, 64)), (5, 3),
                    (6, f(1, 2, 8)), (7, f(1, 2, 3, t=i32)), (8, f(2, 2)), (9, work[128:])):
        fails(lambda: h(*(args[:at] + [bad] + args[at + 1:])))
    fails(lambda: h(*(args[:9] + [work[:256]])), ns.NS_ECAPACITY)
    p = ns.nanospec_policy_loss
    work = ns.alloc_policy_loss_workspace(300, 64)
    args = [f(300, 64), 1.0, f(300, t=i32), f(300), f(300), f(300), f(300), 0.2, 0.2, 0.1, 0.0, f(1), f(300), f(300), f(300), f(1), f(300, 64), work]
    p(*args)
    for at, bad in ((0, f(64)), (1, 0.0), (2, f(300, 1, t=i32)), (2, None), (3, f(2)), (4, f(3)), (4, None), (5, None), (6, f(2)), (7, 2.0), (8, -1.0),
                    (9, math.inf), (11, f(2)), (12, None), (13, f(2)), (14, f(300, 1)), (15, f(2)), (16, f(300, 63)), (16, f(64, 300).t()), (17, work[128:])):
        fails(lambda: p(*(args[:at] + [bad] + args[at + 1:])))
    fails(lambda: p(*(args[:16] + [f(300, 64, t=torch.bfloat16), work])), ns.NS_EDTYPE)
    fails(lambda: p(*(args[:17] + [work[:256]])), ns.NS_ECAPACITY)
    torch.cuda.synchronize()
