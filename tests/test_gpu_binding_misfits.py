"""What is no device tensor where the 8-bit and log-probability calls need one ends in the binding's own error, which
names the argument, whichever argument it is."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ns():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from dynamic_vocab_draft_amd import nanospec
    return nanospec


def f(*s, t=torch.float32):
    return torch.zeros(s, dtype=t, device="cuda")


def calls(ns):
    """(function, arguments, {place of a tensor that may not be missing: its name})"""
    i8, i32 = torch.int8, torch.int32
    yield ns.nanospec_quant_rows, [f(2, 64), f(2, 128, t=i8), f(2)], {0: "x", 1: "q", 2: "scale"}
    yield (ns.nanospec_quant_matmul, [f(2, 128, t=i8), f(2), f(3, 128, t=i8), f(3), 64, f(2, 3)],
           {0: "xq", 1: "xs", 2: "wq", 3: "ws", 5: "out"})
    yield (ns.nanospec_quant_logits_topk,
           [f(9, 128, t=i8), f(9), f(1, 9, t=i32), f(1, t=i32), f(1, 2, 64), 2, None, f(1, 2, 2, t=i32), f(1, 2, 2),
            ns.alloc_quant_logits_workspace(1, 9, 2, 2, 64)],
           {0: "wq", 1: "wscale", 4: "h", 7: "topk_ids", 8: "topk_vals", 9: "work"})
    yield (ns.nanospec_token_logprobs,
           [f(2, 64), 1.0, f(2, 1, t=i32), f(2, 1), f(2), f(2), f(2, 3, t=i32), f(2, 3),
            ns.alloc_token_logprobs_workspace(2, 64, 3)],
           {0: "logits", 4: "lse", 8: "work"})
    yield (ns.nanospec_token_logprobs_grad, [f(2, 64), 1.0, f(2, 1, t=i32), f(2), f(2), f(2, 1), f(2), f(2), f(2, 64)],
           {0: "logits", 3: "lse", 8: "dlogits"})


@pytest.mark.parametrize("bad", [None, [1.0], 0, "host"], ids=str)
def test_no_device_tensor(ns, bad):
    for fn, args, needed in calls(ns):
        fn(*args)
        for at, name in needed.items():
            wrong = args[at].cpu() if bad == "host" else bad
            with pytest.raises(ns.NanoSpecError, match=name) as e:
                fn(*(args[:at] + [wrong] + args[at + 1:]))
            assert e.value.code == ns.NS_EINVAL, (fn.__name__, name)
    torch.cuda.synchronize()
