"""Key weights of batches whose key tiles are shared by several CTA pairs: short paths, where
a request has fewer row blocks than the call plans parts for, and many requests a pair."""
import numpy as np
import pytest

import _around as ar
from test_gpu_key_weights import KINDS, Case, cu, near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def va():
    import speculative_decoding_tree_va_b200 as va
    va.load_library()
    return va


@pytest.mark.parametrize("dtype,kv", [("bf16", "bf16"), ("bf16", "fp8"), ("f32", "f32"), ("f32", "fp8")])
@pytest.mark.parametrize("B,H,T,prefix,accept", [
    (16, 64, 33, 500, 4), (28, 64, 33, 146, 1), (4, 64, 33, 1000, 4), (40, 16, 24, 400, 3),
    (9, 128, 17, 300, 2), (150, 20, 9, 60, 2), (7, 64, 65, 700, 0), (30, 40, 33, 300, 6),
])
def test_paths_shorter_than_the_plan(va, dtype, kv, B, H, T, prefix, accept):
    """Values, the same bits on every run, and no wait that runs into its bound."""
    import torch
    rng = np.random.default_rng(B + H)
    c = Case(B * 7 + T, B, H, T, rng.integers(1, prefix + 1, B), dtype, kv)
    c.alen = np.minimum(c.alen, rng.integers(0, accept + 1, B)).astype(np.int32)
    c.alen[B // 2] = min(accept, 1)
    before = va.device_timeouts()
    status = torch.zeros(B, dtype=torch.int32, device="cuda")
    kw = dict(scale=0.0721, kv_scale=c.kv_scale, path=cu(c.path), accept_len=cu(c.alen),
              req_status=status)
    first = c.run(va, req_status=status)
    near(first, c.ref())
    runs = [va.key_weights(**c.d, **kw) for _ in range(10)]
    torch.cuda.synchronize()
    assert all(torch.equal(r, runs[0]) for r in runs)
    assert not status.any()
    assert va.device_timeouts() == before


@pytest.mark.parametrize("dtype,kv,flags", KINDS)
@pytest.mark.parametrize("H", [3, 128])
def test_rows_that_add_nothing_meet_keys_that_are_no_numbers(va, dtype, kv, flags, H):
    """Counted nodes that are all absent, or whose rows are all empty: a NaN or infinity in the
    cache reaches nothing, and the old weights come back decayed."""
    import torch
    c = Case(31, 3, H, 9, (100, 300, 130), dtype, kv, absent=3)
    bad = ar.slots(c.table, 0, 109)[[5, 64, 99]].tolist() + ar.slots(c.table, 1, 309)[[0, 299]].tolist()
    for x in (c.d["c_kv"], c.d["k_pe"]):
        if kv == "fp8":
            x.view(torch.uint8).view(-1, x.shape[-1])[bad] = 0x7f
        else:
            x.view(-1, x.shape[-1])[bad] = torch.tensor([float("nan"), float("inf"), -float("inf"),
                                                         float("nan"), float("inf")],
                                                        device="cuda", dtype=x.dtype)[:, None]
    c.path[0, :3], c.alen[0] = (6, 7, 8), 3          # absent nodes
    c.path[1, :2], c.alen[1] = (0, 2), 2             # rows without a log-sum-exp
    c.lse[1] = -np.inf
    c.d["lse"].copy_(torch.from_numpy(c.lse))
    old = np.abs(c.rng.normal(size=(3, c.cap))).astype(np.float32)
    got = c.run(va, True, weights=cu(old), decay=0.5, flags=flags)
    used = np.arange(c.cap)[None] < c.kv_len[:, None]
    want = np.where(used, np.float32(0.5) * old, np.float32(0))
    assert np.array_equal(got.cpu().numpy()[:2], want[:2])
    near(got[2:], c.ref(True, old, 0.5)[2:])


@pytest.mark.parametrize("flags", [0, 1])
@pytest.mark.parametrize("H", [2, 64])
def test_largest_finite_numbers_are_numbers(va, flags, H):
    """fp32 elements past the largest bf16, in queries and in keys: their scores are the exact
    ones (the other side holds 2^-123, so that a product is 32)."""
    import torch
    c = Case(32, 2, H, 5, (200, 77), "f32")
    big, small = float(np.finfo(np.float32).max), 2.0 ** -123
    sign = lambda *s: torch.from_numpy(c.rng.choice([-1.0, 1.0], s)).float()  # noqa: E731
    n = c.c.shape[0]
    c.qn[..., 7], c.c[..., 7] = big * sign(2, 5, H), small * sign(n, 64)
    c.qn[..., 300], c.c[..., 300] = small * sign(2, 5, H), big * sign(n, 64)
    c.qp[..., 63], c.k[..., 63] = big * sign(2, 5, H), small * sign(n, 64)
    for b in range(2):
        q, keys = c.parts(b)
        c.lse[b] = ar.lse_ref(q, keys, c.see[b], c.prefix[b], ar.SCALE)
    c.d.update(q_nope=c.qn.cuda(), q_pe=c.qp.cuda(), c_kv=c.c.cuda(), k_pe=c.k.cuda(),
               lse=cu(c.lse))
    for path in (True, False):
        near(c.run(va, path, flags=flags), c.ref(path))


@pytest.mark.parametrize("dtype,kv", [("bf16", "bf16"), ("bf16", "fp8"), ("f32", "f32"), ("f32", "fp8")])
@pytest.mark.parametrize("spread", [1.0, 3.0])
def test_scores_are_neither_short_nor_long_on_average(va, dtype, kv, spread):
    """Over 32768 keys of one row, the error of ln w grows with the score by at most 2.4e-7 of
    it: 1e-7 for what the mean rounding of the sums varies by with the data, a half step of
    fp32 (6e-8) each for the scale and its product with the cache's, 1.3e-8 for log2 e.  The
    slope of the fit is good to 1e-8 (errors of 1.4e-6 a key, scores of 4)."""
    import torch
    c = Case(33, 1, 1, 1, 32767, dtype, kv)
    for name, x in (("q_nope", c.qn), ("q_pe", c.qp)):
        x.mul_(spread)
        c.d[name].copy_(x)
    c.d["lse"].zero_()
    w = c.run(va, False)[0].double().cpu().numpy()[:32768]
    q, keys = c.parts(0)
    s = ar.scores_ref(q, keys, np.float64(np.float32(ar.SCALE)))[0, 0]
    err = np.log(w) - s
    assert abs((err * s).sum() / (s * s).sum()) <= 2.4e-7
