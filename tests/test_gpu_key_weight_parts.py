"""Key weights of batches whose key tiles are shared by several CTA pairs: short paths, where
a request has fewer row blocks than the call plans parts for, and many requests a pair."""
import numpy as np
import pytest

from test_gpu_key_weights import Case, cu, near

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
