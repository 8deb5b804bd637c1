"""Argument checks of the calls around the verify step (no GPU: nothing is launched)."""
import ctypes

import pytest

import speculative_decoding_tree_va_b200 as va
from speculative_decoding_tree_va_b200 import build as va_build

FAKE = 1 << 20  # aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    va_build.build()
    return va.load_library()


def fill(cls, ptrs, **kw):
    a = cls()
    for f in ptrs:
        setattr(a, f, FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def logprob_args(**kw):
    base = dict(dtype=va.VA_F32, R=4, V=100, ld=100, scale=1.0, G=2, K=3)
    return fill(va.VaLogprobArgs, ("logits", "tokens", "tok_lp", "top_ids", "lse"), **{**base, **kw})


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=2), 1), (dict(R=-1), 1), (dict(V=0), 1), (dict(ld=99), 1), (dict(K=17), 1),
    (dict(K=-1), 1), (dict(K=5, V=4), 1), (dict(G=-1), 1), (dict(G=65537), 1),
    (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(logits=None), 1), (dict(logits=FAKE + 2), 1),
    (dict(tokens=None), 1), (dict(tok_lp=None), 1), (dict(top_ids=None), 1),
    (dict(lse=FAKE + 2), 1), (dict(top_lp64=FAKE + 4), 1), (dict(K=0, top_lp=FAKE), 1),
    (dict(R=0x7fffffff), 2), (dict(V=0x7fffffff, ld=0x7fffffff), 2),
])
def test_logprob_checks(lib, bad, status):
    assert lib.va_token_logprobs(ctypes.byref(logprob_args(**bad)), None) == status


def key_weight_args(**kw):
    base = dict(dtype=va.VA_BF16, B=2, H=64, T=33, scale=0.07, num_pages=100, page_size=64,
                max_pages=50, decay=1.0, workspace=FAKE, workspace_bytes=1 << 40)
    return fill(va.VaKeyWeightArgs, ("q_nope", "q_pe", "c_kv", "k_pe", "page_table", "kv_len",
                                     "tree_mask", "lse", "weights"), **{**base, **kw})


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=7), 1), (dict(B=-1), 1), (dict(H=0), 1), (dict(T=0), 1), (dict(T=66), 1),
    (dict(page_size=32), 2), (dict(B=65536), 2), (dict(flags=2), 1), (dict(flags=8), 1),
    (dict(flags=4), 1), (dict(flags=4, kv_scale=float("inf")), 1), (dict(scale=float("nan")), 1),
    (dict(decay=float("inf")), 1), (dict(num_pages=0), 1), (dict(max_pages=0), 1),
    (dict(num_pages=1 << 26), 2), (dict(max_pages=1 << 26), 2), (dict(B=60000, T=65, H=600), 2),
    (dict(B=1, T=33, H=1 << 17), 2),
    (dict(q_nope=None), 1), (dict(c_kv=FAKE + 8), 1), (dict(lse=None), 1), (dict(weights=None), 1),
    (dict(tree_mask=FAKE + 4), 1), (dict(path=FAKE), 1), (dict(accept_len=FAKE), 1),
    (dict(weights_in=FAKE + 2), 1), (dict(req_status=FAKE + 1), 1),
    (dict(workspace=None), 1), (dict(workspace=FAKE + 128), 1), (dict(workspace_bytes=16), 1),
])
def test_key_weight_checks(lib, bad, status):
    a = key_weight_args(**bad)
    if "workspace" in bad or "workspace_bytes" in bad:  # a call that needs one
        a.B, a.max_pages, a.dtype = 1, 2, va.VA_F32
        assert lib.va_key_weights_workspace_bytes(ctypes.byref(a)) > 16
    assert lib.va_key_weights(ctypes.byref(a), None) == status
    if status != 1 or "workspace" not in str(bad):
        assert lib.va_key_weights_workspace_bytes(ctypes.byref(a)) == 0


def evict_args(**kw):
    base = dict(B=2, capacity=640, T=33, n_sink=4, n_recent=16)
    return fill(va.VaEvictArgs, ("weights", "kv_len", "budget", "path", "accept_len", "new_len",
                                 "from_slot"), **{**base, **kw})


@pytest.mark.parametrize("bad,status", [
    (dict(B=-1), 1), (dict(T=66), 1), (dict(T=-1), 1), (dict(n_sink=-1), 1), (dict(n_recent=-1), 1),
    (dict(capacity=0), 1), (dict(capacity=32), 1), (dict(B=65536), 2), (dict(weights=None), 1),
    (dict(from_slot=FAKE + 2), 1), (dict(path=None), 1), (dict(accept_len=None), 1), (dict(T=0), 1),
    (dict(pos_out=FAKE), 1), (dict(weights_out=FAKE + 1), 1), (dict(capacity=1 << 30), 2),
])
def test_evict_checks(lib, bad, status):
    assert lib.va_evict_plan(ctypes.byref(evict_args(**bad)), None) == status


@pytest.mark.parametrize("at,value,status", [
    (0, None, 1), (0, FAKE + 8, 1), (1, None, 1), (2, 3, 1), (3, 0, 1), (3, 1 << 26, 2), (4, 32, 2),
    (5, None, 1), (6, -1, 1), (6, 65536, 2), (7, 0, 1), (7, 1 << 26, 2), (8, None, 1), (9, None, 1),
    (10, FAKE + 2, 1),
])
def test_move_checks(lib, at, value, status):
    args = [FAKE, FAKE, 2, 100, 64, FAKE, 2, 50, FAKE, FAKE, None]
    args[at] = value
    assert lib.va_kv_move(*args, None) == status


def test_nothing_to_do(lib):
    assert lib.va_token_logprobs(ctypes.byref(logprob_args(R=0, logits=None)), None) == 0
    assert lib.va_key_weights(ctypes.byref(key_weight_args(B=0)), None) == 0
    assert lib.va_evict_plan(ctypes.byref(evict_args(B=0)), None) == 0
    assert lib.va_kv_move(None, None, 2, 1, 64, None, 0, 1, None, None, None, None) == 0
    for f in (lib.va_token_logprobs, lib.va_key_weights, lib.va_evict_plan):
        assert f(None, None) == 1


def test_binding_refuses_host_tensors():
    import torch
    with pytest.raises(va.VerifyAttnError):
        va.token_logprobs(torch.zeros(2, 10))
    f = lambda *s: torch.zeros(*s)  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(va.VerifyAttnError):
        va.key_weights(f(1, 1, 1, 512), f(1, 1, 1, 64), f(1, 64, 512), f(1, 64, 64), i(1, 1), i(1),
                       torch.zeros(1, 1, 1, dtype=torch.int64), f(1, 1, 1), scale=1.0)
    with pytest.raises(va.VerifyAttnError):
        va.evict_plan(f(1, 64), i(1), i(1))
    with pytest.raises(va.VerifyAttnError):
        va.kv_move(f(1, 64, 512), f(1, 64, 64), i(1, 1), i(1, 64), i(1))


@pytest.mark.parametrize("cache,table", [((64, 512), (2, 3)), ((), (2, 3)), ((4, 64, 512), (6,)),
                                         ((4, 64, 512), ()), ((4, 64, 512), (2, 3, 1))])
def test_binding_refuses_other_numbers_of_axes(cache, table):
    """A cache or page table with an axis more or less is refused by its name."""
    import torch
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    c, k, t = torch.zeros(cache), torch.zeros(4, 64, 64), i(*table) if table else i(1)[0]
    name = "c_kv has" if len(cache) != 3 else "page_table has"
    with pytest.raises(va.VerifyAttnError, match=name):
        va.kv_move(c, k, t, i(2, 192), i(2))
    q = torch.zeros(2, 1, 1, 512)
    with pytest.raises(va.VerifyAttnError, match=name):
        va.key_weights(q, q[..., :64], c, k, t, i(2), torch.zeros(2, 1, 1, dtype=torch.int64),
                       torch.zeros(2, 1, 1), scale=1.0)


@pytest.mark.parametrize("bad", [dict(flags=17), dict(flags=17, dtype=va.VA_F32),
                                 dict(flags=16, dtype=va.VA_F32, B=100, max_pages=100)])
def test_the_wait_hook_is_refused_on_cuda_cores(lib, bad):
    a = key_weight_args(**bad)
    assert lib.va_key_weights(ctypes.byref(a), None) == va.VA_ERR_INVALID_ARG
    assert lib.va_key_weights_workspace_bytes(ctypes.byref(a)) == 0
