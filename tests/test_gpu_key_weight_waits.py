"""The key-weight kernel's bounded waits: with products that never come, every request is
flagged, nothing hangs, and the same context then runs a normal call.  The hook issues no
tensor-core work; the copies have long landed when the waits give up."""
import pytest

from test_gpu_key_weights import Case, near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def va():
    import speculative_decoding_tree_va_b200 as va
    va.load_library()
    return va


@pytest.mark.parametrize("dtype,kv", [("bf16", "bf16"), ("bf16", "fp8"), ("f32", "f32"), ("f32", "fp8")])
@pytest.mark.parametrize("B,H,T,prefix", [
    (2, 4, 5, (100, 300)),       # few rows stay in shared memory, one tile a request
    (1, 8, 9, 30000),            # more tiles than CTA pairs: the rings fill
    (3, 64, 33, (700, 20, 290)), # rows pass by, tiles in parts
])
def test_expired_waits_flag_requests_and_leave_the_context_usable(va, dtype, kv, B, H, T, prefix):
    import torch
    c = Case(B + H, B, H, T, prefix, dtype, kv)
    before = va.device_timeouts()
    status = torch.zeros(B, dtype=torch.int32, device="cuda")
    c.run(va, False, flags=va.VA_FLAG_TEST_STALL_KEY_WEIGHTS, req_status=status)
    torch.cuda.synchronize()
    assert status.cpu().tolist() == [va.VA_ERR_CUDA] * B
    after = va.device_timeouts()
    assert after > before
    status.zero_()
    near(c.run(va, False, req_status=status), c.ref(False))
    assert not status.any() and va.device_timeouts() == after
