"""Log probabilities of given tokens, entropy and top-k on the GPU against 64 bits."""
import numpy as np
import pytest

import _around as ar

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def va():
    import speculative_decoding_tree_va_b200 as va
    va.load_library()
    return va


def device_rows(x, dtype, pad=0, shift=0):
    """Rows of x on the GPU in rows of V + pad elements that start `shift` elements in;
    the padding holds NaN, which nothing may read."""
    import torch
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    R, V = x.shape
    flat = torch.full((R * (V + pad) + shift + 8,), float("nan"), dtype=dt, device="cuda")
    t = flat[shift:shift + R * (V + pad)].view(R, V + pad)[:, :V]
    t.copy_(torch.from_numpy(x).to(dt))
    return t


def check(va, t, tokens=None, k=0, scale=1.0, what=""):
    import torch
    x = t.double().cpu().numpy()
    R, V = x.shape
    status = torch.zeros(R, dtype=torch.int32, device="cuda")
    tk = None if tokens is None else torch.from_numpy(tokens).cuda()
    got = va.token_logprobs(t, tk, k=k, scale=scale, row_status=status)
    ref = ar.logprobs_ref(x, tokens, k, np.float64(np.float32(scale)))
    tol = ar.logprobs_tol(V, scale, x)

    def same(name, a, b, grow):
        a = a.double().cpu().numpy()
        with np.errstate(over="ignore"):  # what fp32 does not hold rounds to an infinity
            b = np.where(np.isinf(b.astype(np.float32)), b.astype(np.float32), b)
        assert np.array_equal(np.isnan(a), np.isnan(b)), (what, name)
        assert np.array_equal(np.isneginf(a), np.isneginf(b)), (what, name)
        f = np.isfinite(b)
        # one rounding of the stored result, and of scale * (x - m) before it
        bar = tol * grow + 3 * 2.0 ** -24 * np.abs(b[f])
        assert (np.abs(a[f] - b[f]) <= bar).all(), (what, name, np.abs(a[f] - b[f]).max(), tol)

    same("lse", got.lse, ref["lse"], 1.0)
    # S / Z: each y is off by three half steps and weighted by p, |y| <= 40; twice the lse's
    same("entropy", got.entropy, ref["entropy"], 40.0)
    if k:
        assert np.array_equal(got.top_ids.cpu().numpy(), ref["top_ids"]), what
        same("top_lp", got.top_lp, ref["top_lp"], 1.0)
    if tokens is not None:
        same("tok_lp", got.tok_lp, ref["tok_lp"], 1.0)
    assert np.array_equal(status.cpu().numpy() != 0, ref["bad"]), what
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R,V,pad,shift,k,G", [
    (1, 1, 0, 0, 1, 1), (3, 2, 1, 1, 2, 0), (2, 7, 0, 3, 5, 2), (5, 255, 2, 0, 16, 1),
    (1, 4096, 0, 0, 8, 0), (7, 4097, 0, 1, 16, 3), (300, 1000, 0, 0, 1, 1),
    (3, 8193, 5, 2, 0, 1), (2, 50257, 0, 0, 16, 4), (1, 200003, 1, 1, 16, 1),
    (40, 32771, 0, 0, 2, 1), (160, 20001, 3, 0, 11, 0),
])
def test_shapes(va, dtype, R, V, pad, shift, k, G):
    rng = np.random.default_rng(R * 1000 + V)
    x = rng.normal(0, 2.5, (R, V))
    tokens = rng.integers(-1, V, (R, G)).astype(np.int32) if G else None
    check(va, device_rows(x, dtype, pad, shift), tokens, k, what=f"{dtype} {R}x{V}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [5, 300, 9001, 40009])
def test_special_rows(va, dtype, V):
    """Ties, masks of -inf and of the lowest value, empty rows, NaN and +inf rows,
    rows that meet larger logits all the way, zeros of both signs."""
    import torch
    rng = np.random.default_rng(V)
    low = float(torch.finfo({"f32": torch.float32, "bf16": torch.bfloat16}[dtype]).min)
    n = rng.normal(0, 2, V)
    rows = [np.zeros(V), np.where(rng.random(V) < 0.5, 0.0, -0.0), np.full(V, -np.inf),
            np.full(V, low), np.where(rng.random(V) < 0.97, -np.inf, n),
            np.where(rng.random(V) < 0.97, low, n), np.sort(n), np.sort(n)[::-1],
            np.where(np.arange(V) == V // 2, 3.0, -np.inf), np.round(n),
            np.where(np.arange(V) == V - 1, np.nan, n), np.where(np.arange(V) == 0, np.inf, n),
            n * 1e4, n * 1e-6 + 100, np.where(np.arange(V) % 2 == 0, 80.0, -80.0)]
    x = np.stack(rows)
    tokens = np.stack([np.full(len(rows), V // 2), np.full(len(rows), -1)], 1).astype(np.int32)
    check(va, device_rows(x, dtype), tokens, min(V, 16), what=f"{dtype} V={V}")
    check(va, device_rows(x, dtype, pad=1), tokens, 1, what=f"{dtype} V={V} greedy")


@pytest.mark.parametrize("scale", [0.25, 1.0, 1.7, 10.0])
def test_temperature(va, scale):
    rng = np.random.default_rng(3)
    x = rng.normal(0, 2.5, (4, 9000))
    check(va, device_rows(x, "f32"), None, 4, scale=scale, what=f"scale {scale}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [0.7, 0.9, 1.0, 1.25, 1.3, 3.0, 1e-6, 1e9])
def test_threads_with_nothing_but_masks(va, dtype, scale):
    """Rows shorter than the threads of a block, masks of every usual value that fill
    whole threads, and rows that they fill, at temperatures other than one."""
    rng = np.random.default_rng(17)
    for V in (1, 50, 1000, 9001):
        n = rng.normal(0, 2, V)
        rows = [n]
        for fill in (-1e4, -1e9, -1e20, -1e30, -np.inf):
            rows += [np.full(V, fill), np.where(rng.random(V) < 0.97, fill, n),
                     np.where(np.arange(V) < V // 2, fill, n)]
        check(va, device_rows(np.stack(rows), dtype), None, min(V, 4), scale=scale,
              what=f"{dtype} V={V} scale {scale}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [0.9, 1.0, 1.3])
def test_large_logits(va, dtype, scale):
    rng = np.random.default_rng(18)
    for V in (3, 2000):
        n = rng.normal(0, 2, V)
        x = np.stack([sign * 10.0 ** e + n * 10.0 ** f for e in (3, 5, 6, 7, 8, 10, 12, 20, 28, 30, 37)
                      for sign in (1, -1) for f in (0, e - 3)])
        check(va, device_rows(x, dtype), None, min(V, 4), scale=scale, what=f"{dtype} V={V}")


def test_token_past_the_vocabulary_is_flagged(va):
    rng = np.random.default_rng(4)
    x = rng.normal(0, 2, (3, 100))
    tokens = np.array([[99, 5], [100, 5], [2 ** 30, -1]], np.int32)
    check(va, device_rows(x, "bf16"), tokens, 2, what="tokens")


def test_wide_top_k_feeds_the_builder(va):
    """[B, L, V] drafter logits: wide log probabilities are the float32 ones widened, and
    the tree they build is the oracle's on the same values."""
    import torch

    import oracle
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(3, 15, 4096, device="cuda", generator=g) * 2
    wide = va.token_logprobs(x, k=8, wide=True)
    slim = va.token_logprobs(x, k=8)
    assert wide.top_lp.dtype == torch.float64 and wide.top_lp.shape == (3, 15, 8)
    assert torch.equal(wide.top_lp, slim.top_lp.double()) and torch.equal(wide.top_ids, slim.top_ids)
    par, tok, _, n = va.build_tree(wide.top_lp, wide.top_ids, 32)
    ref = oracle.build_trees(wide.top_lp.cpu().numpy(), wide.top_ids.cpu().numpy(), 32)
    assert np.array_equal(par.cpu().numpy(), ref["parent"])
    assert np.array_equal(tok.cpu().numpy(), ref["token"])


def test_no_rows_and_outputs_left_out(va):
    import torch
    r = va.token_logprobs(torch.empty(0, 10, device="cuda"), k=2)
    assert r.lse.shape == (0,) and r.top_ids.shape == (0, 2)
    r = va.token_logprobs(torch.randn(10, device="cuda"))
    assert r.lse.shape == () and r.tok_lp is None and r.top_ids is None


def test_repeated_streams_and_graph(va):
    """The same bits on every run, on another stream, and replayed from a graph on new logits."""
    import torch
    x = torch.randn(20, 70001, device="cuda", dtype=torch.bfloat16)
    a = va.token_logprobs(x, k=16)
    b = va.token_logprobs(x, k=16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c = va.token_logprobs(x, k=16, stream=s)
    torch.cuda.synchronize()
    for o in (b, c):
        assert all(torch.equal(p, q) for p, q in zip(a, o) if p is not None)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = va.token_logprobs(x, k=16)
    x.copy_(torch.randn(20, 70001, device="cuda"))
    g.replay()
    torch.cuda.synchronize()
    want = va.token_logprobs(x, k=16)
    assert all(torch.equal(p, q) for p, q in zip(r, want) if p is not None)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [0.5, 1e-20, 1e-37, 3e-38])
def test_differences_past_the_range_of_fp32(va, dtype, scale):
    """Logits of both signs near the type's largest, with the type's lowest beside them: their
    difference is no fp32 number, but its scaled value is."""
    rng = np.random.default_rng(20)
    top = float(np.finfo(np.float32).max) if dtype == "f32" else 3.3895e38
    for V in (4, 300, 9001):
        u = rng.uniform(-1, 1, V) * top
        x = np.stack([u, np.where(np.arange(V) % 2 == 0, top, -top), np.full(V, top),
                      np.where(np.arange(V) == V // 2, 1e37, -top),
                      np.where(rng.random(V) < 0.5, -np.inf, u)])
        tokens = np.stack([np.arange(5) % V, np.full(5, V - 1)], 1).astype(np.int32)
        check(va, device_rows(x, dtype), tokens, min(V, 4), scale=scale, what=f"{dtype} V={V}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [0.9, 1.0, 1.3, 30.0, 1e-6, 1e-28, 1e-30, 1e-36])
def test_rows_next_to_the_lowest_logit_read_as_it_is(va, dtype, scale):
    """The kernel reads logits below -X as -X, with X the power of two that times the scale
    (and log2 e) is in [2^23, 2^24), or 2^100: rows whose largest logit lies from there to 300
    binary orders of weight above, and ordinary rows where 2^100 is close to them."""
    rng = np.random.default_rng(19)
    c = float(np.float32(scale)) * np.log2(np.e)
    X = 2.0 ** min(24 - np.frexp(c)[1], 100)
    low = float(np.finfo(np.float32).min) if dtype == "f32" else -3.3895e38
    for V in (10, 700, 9001):
        n = np.abs(rng.normal(0, 2, V)) / c
        n[V // 3] = 0.0
        hide = rng.random(V) < 0.9
        hide[V // 3] = False
        rows = []
        for above in (0.0, 0.5, 1.0, 8.0, 60.0, 150.0, 199.0, 201.0, 300.0):
            x = -X + above / c - n
            rows += [x, np.where(hide, -np.inf, x), np.where(hide, low, x),
                     np.where(np.arange(V) == V // 3, x, -np.inf)]
        rows += [-n, np.where(hide, -np.inf, -n), np.where(np.arange(V) == V // 3, 0.0, -np.inf)]
        x = np.maximum(np.stack(rows), np.where(np.isneginf(np.stack(rows)), -np.inf, low))
        check(va, device_rows(x, dtype), None, min(V, 4), scale=scale,
              what=f"{dtype} V={V} scale {scale}")
