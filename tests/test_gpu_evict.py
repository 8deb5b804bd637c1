"""Eviction plans and moves on the GPU against a slot-by-slot form (equal, not near)."""
import numpy as np
import pytest

import _around as ar

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def va():
    import speculative_decoding_tree_va_b200 as va
    va.load_library()
    return va


def cu(a):
    import torch
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def check_plan(va, w, kv_len, budget, T=0, path=None, alen=None, pos=None, n_sink=0, n_recent=0,
               in_place=False, what=""):
    import torch
    ref = ar.evict_ref(w, kv_len, budget, T, path, alen, pos, n_sink, n_recent)
    status = torch.zeros(w.shape[0], dtype=torch.int32, device="cuda")
    dw, dp = cu(w), cu(pos)
    kw = dict(weights_out=dw, pos_out=dp) if in_place else {}
    got = va.evict_plan(dw, cu(kv_len), cu(budget), path=cu(path), accept_len=cu(alen),
                        tree_len=T, pos=dp, n_sink=n_sink, n_recent=n_recent, req_status=status, **kw)
    torch.cuda.synchronize()
    assert np.array_equal(got.new_len.cpu().numpy(), ref[0]), what
    assert np.array_equal(got.from_slot.cpu().numpy(), ref[1]), what
    assert np.array_equal(got.weights.cpu().numpy(), ref[2], equal_nan=True), what
    if pos is not None:
        assert np.array_equal(got.pos.cpu().numpy(), ref[3]), what
    assert np.array_equal(status.cpu().numpy() != 0, ref[4]), what
    return got, ref


def make(rng, B, cap, T, zeros=0.1):
    kv_len = rng.integers(max(T, 1), cap + 1, B).astype(np.int32)
    kv_len[0] = cap
    w = np.exp(rng.normal(0, 2, (B, cap))).astype(np.float32)
    w[rng.random((B, cap)) < zeros] = 0.0
    path = alen = None
    if T:
        par = ar.random_tree(rng, B, T)
        path, alen = ar.random_path(rng, par, ar.ancestors(par))
    return w, kv_len, path, alen


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,cap,T,sink,recent,pos", [
    (1, 1, 0, 0, 0, False), (1, 1, 1, 0, 0, False), (3, 64, 5, 0, 0, False),
    (5, 191, 33, 2, 7, True), (2, 4096, 65, 4, 64, False), (3, 4097, 0, 0, 0, True),
    (2, 8200, 9, 4, 500, True), (1, 40001, 65, 16, 1024, True), (1, 131136, 33, 0, 0, False),
    (200, 500, 17, 1, 10, True),
])
def test_plans(va, B, cap, T, sink, recent, pos, in_place):
    rng = np.random.default_rng(cap + B)
    w, kv_len, path, alen = make(rng, B, cap, T)
    at = np.stack([rng.permutation(2 * cap)[:cap] for _ in range(B)]).astype(np.int32) if pos else None
    for share in (0.0, 0.3, 0.9, 2.0):
        budget = (share * kv_len).astype(np.int32)
        check_plan(va, w, kv_len, budget, T, path, alen, at, sink, recent, in_place,
                   what=f"cap {cap} share {share}")


@pytest.mark.parametrize("cap", [262144, 262145, 300003])
def test_longest_requests(va, cap):
    """Around the length whose keys no longer fit in the cluster's shared memory."""
    rng = np.random.default_rng(cap)
    w, kv_len, path, alen = make(rng, 1, cap, 33)
    w[0, ::3] = 1.0
    at = rng.permutation(2 * cap)[:cap].astype(np.int32)[None]
    check_plan(va, w, kv_len, np.array([cap // 3 + 5], np.int32), 33, path, alen, at, 7, 1000,
               in_place=True, what=f"cap {cap}")


@pytest.mark.parametrize("B,cap", [(80, 40000), (40, 70001), (76, 32768), (74, 9001), (30, 33000)])
@pytest.mark.parametrize("pos", [False, True])
def test_batches_of_long_requests(va, B, cap, pos):
    """Clusters of one, two and four, with keys held in shared memory and read again."""
    rng = np.random.default_rng(cap + pos)
    w, kv_len, path, alen = make(rng, B, cap, 20)
    w = np.round(w)  # many ties
    at = np.stack([rng.permutation(cap) for _ in range(B)]).astype(np.int32) if pos else None
    check_plan(va, w, kv_len, (rng.random(B) * kv_len).astype(np.int32), 20, path, alen, at, 4, 99,
               in_place=True, what=f"{B} x {cap}")


def test_ties_and_special_weights(va):
    """Equal weights go by slot; NaN ranks like -inf; +-0 are equal; infinities rank."""
    rng = np.random.default_rng(8)
    B, cap = 8, 9000
    w = np.ones((B, cap), np.float32)
    w[1] = 0.0
    w[2] = np.where(rng.random(cap) < 0.5, 0.0, -0.0)
    w[3] = np.nan
    w[4] = np.where(rng.random(cap) < 0.3, np.nan, np.where(rng.random(cap) < 0.3, -np.inf, 1.0))
    w[5] = np.where(rng.random(cap) < 0.1, np.inf, -rng.random(cap))
    w[6] = rng.integers(0, 3, cap)
    w[7] = np.float32(1.0) + rng.integers(0, 5, cap).astype(np.float32) * np.float32(2 ** -23)
    kv_len = np.full(B, cap, np.int32)
    for n in (0, 1, 4500, 8999, 9000):
        check_plan(va, w, kv_len, np.full(B, n, np.int32), what=f"budget {n}")
        check_plan(va, w, kv_len, np.full(B, n, np.int32), n_sink=4, n_recent=50, in_place=True,
                   what=f"budget {n}, protected")


def test_commit_of_the_accepted_path(va):
    """A budget above the candidates drops the rejected nodes and nothing else."""
    rng = np.random.default_rng(9)
    w, kv_len, path, alen = make(rng, 16, 700, 33)
    got, ref = check_plan(va, w, kv_len, np.full(16, 10 ** 6, np.int32), 33, path, alen)
    assert np.array_equal(ref[0], kv_len - 33 + alen)


def test_flagged_requests(va):
    rng = np.random.default_rng(10)
    w, kv_len, path, alen = make(rng, 8, 300, 9)
    kv_len[1], kv_len[2] = 8, 301
    alen[3], alen[4] = -1, 10
    path[5, :3], alen[5] = (0, 4, 4), 3
    path[6, :2], alen[6] = (0, 9), 2
    path[7, :2], alen[7] = (-1, 2), 2
    kv_len[3:] = rng.integers(9, 301, 5)
    _, ref = check_plan(va, w, kv_len, np.full(8, 50, np.int32), 9, path, alen)
    assert ref[4].tolist() == [False] + [True] * 7


def pools(rng, num, kind):
    import torch
    c, k = rng.normal(size=(num, 64, 512)), rng.normal(size=(num, 64, 64))
    dt = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}.get(kind)
    if kind == "u8":
        return (torch.from_numpy(rng.integers(0, 256, c.shape).astype(np.uint8)).cuda(),
                torch.from_numpy(rng.integers(0, 256, k.shape).astype(np.uint8)).cuda())
    return torch.from_numpy(c).to(dt).cuda(), torch.from_numpy(k).to(dt).cuda()


def raw(t):
    import torch
    return t.view(torch.uint8).cpu().numpy().copy()


@pytest.mark.parametrize("kind", ["f32", "bf16", "fp8", "u8"])
@pytest.mark.parametrize("B,cap,T", [(1, 60, 1), (3, 300, 9), (2, 2500, 65), (40, 130, 5)])
def test_moves(va, kind, B, cap, T):
    """Every kept key's row, bit for bit, in its new slot; all other slots of the pool as
    they were."""
    import torch
    rng = np.random.default_rng(cap + T)
    w, kv_len, path, alen = make(rng, B, cap, T)
    table, num = ar.paged(rng, B, kv_len)
    full = table.shape[1] * 64
    w = np.pad(w, ((0, 0), (0, full - cap)))
    budget = (0.4 * kv_len).astype(np.int32)
    plan = va.evict_plan(cu(w), cu(kv_len), cu(budget), path=cu(path), accept_len=cu(alen), tree_len=T)
    c, k = pools(rng, num, kind)
    before = raw(c).reshape(num * 64, -1), raw(k).reshape(num * 64, -1)
    status = torch.zeros(B, dtype=torch.int32, device="cuda")
    va.kv_move(c, k, cu(table), plan.from_slot, plan.new_len, req_status=status)
    after = raw(c).reshape(num * 64, -1), raw(k).reshape(num * 64, -1)
    new_len, src, _, _, _ = ar.evict_ref(w, kv_len, budget, T, path, alen)
    for x, y in zip(before, after):
        want = x.copy()
        for b in range(B):
            n = int(new_len[b])
            at = ar.slots(table, b, int(kv_len[b]))
            want[at[:n]] = x[at[src[b, :n]]]
        assert np.array_equal(want, y)
    assert not status.any()


def test_move_refuses_bad_plans(va):
    """A source inside the kept part, past the table, or on a page outside the pool is
    flagged and not moved; a bad length moves nothing."""
    import torch
    rng = np.random.default_rng(11)
    B, m = 6, 3
    table = np.arange(B * m, dtype=np.int32).reshape(B, m)
    table[3, 2] = B * m           # source page outside the pool
    table[4, 0] = -1              # destination page outside the pool
    src = np.full((B, 192), -1, np.int32)
    src[:, :100] = np.arange(100)
    src[:, 7] = 150               # slot 150 moves to 7
    src[1, 7] = 50
    src[2, 7] = 192
    n = np.array([100, 100, 100, 100, 100, 193], np.int32)
    c, k = pools(rng, B * m, "bf16")
    before = c.clone()
    status = torch.zeros(B, dtype=torch.int32, device="cuda")
    va.kv_move(c, k, cu(table), cu(src), cu(n), req_status=status)
    assert status.cpu().tolist() == [0, 1, 1, 1, 1, 1]
    want = before.clone()
    want[0, 7] = before[2, 150 - 128]
    assert torch.equal(c, want)


def test_streams_and_graph(va):
    """One plan for two layers, captured with its moves, replayed on new weights."""
    import torch
    rng = np.random.default_rng(12)
    B, T = 4, 17
    kv_len = np.array([900, 64, 333, 1000], np.int32)
    table, num = ar.paged(rng, B, kv_len)
    cap = table.shape[1] * 64
    w, _, path, alen = make(rng, B, cap, T)
    c, k = pools(rng, num, "bf16")
    c2, k2 = c.clone(), k.clone()
    d = [cu(x) for x in (w, kv_len, (kv_len // 2).astype(np.int32), path, alen, table)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        r = va.evict_plan(d[0], d[1], d[2], path=d[3], accept_len=d[4], tree_len=T)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = va.evict_plan(d[0], d[1], d[2], path=d[3], accept_len=d[4], tree_len=T)
        va.kv_move(c, k, d[5], r.from_slot, r.new_len)
        va.kv_move(c2, k2, d[5], r.from_slot, r.new_len)
    w2 = np.exp(rng.normal(0, 2, w.shape)).astype(np.float32)
    d[0].copy_(torch.from_numpy(w2))
    before = c.clone()
    g.replay()
    torch.cuda.synchronize()
    n, src, _, _, _ = ar.evict_ref(w2, kv_len, kv_len // 2, T, path, alen)
    assert np.array_equal(r.from_slot.cpu().numpy(), src)
    assert torch.equal(c, c2) and torch.equal(k, k2)
    flat, old = c.view(-1, 512), before.view(-1, 512)
    for b in range(B):
        at = torch.from_numpy(ar.slots(table, b, int(kv_len[b]))).cuda()
        assert torch.equal(flat[at[:n[b]]], old[at[torch.from_numpy(src[b, :n[b]]).long().cuda()]])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_weights_and_positions_through_two_steps(va, dtype):
    """Weights, plan, move; then the next tree behind the kept keys, weights on top of the
    plan's, and a second plan by the positions carried along: each key's weight and position
    stay its own, whatever slot it is in."""
    import torch

    from test_gpu_key_weights import Case, near
    B, H, T = 3, 4, 9
    c = Case(41, B, H, T, (150, 40, 280), dtype, spare=2)
    w1 = c.run(va, True)
    want1 = c.ref()
    pos = np.tile(np.arange(c.cap, dtype=np.int32), (B, 1))
    budget = np.array([70, 30, 200], np.int32)
    plan = va.evict_plan(w1, c.d["kv_len"], cu(budget), path=cu(c.path), accept_len=cu(c.alen),
                         tree_len=T, pos=cu(pos), n_sink=3, n_recent=10)
    n1, src, _, pos1, _ = ar.evict_ref(w1.cpu().numpy(), c.kv_len, budget, T, c.path, c.alen, pos, 3, 10)
    assert np.array_equal(plan.from_slot.cpu().numpy(), src)
    va.kv_move(c.d["c_kv"], c.d["k_pe"], c.d["page_table"], plan.from_slot, plan.new_len)
    old = np.zeros((B, c.cap))
    for b in range(B):
        old[b, :n1[b]] = want1[b, src[b, :n1[b]]]
    # the next tree: other nodes, queries and keys, behind the kept keys
    c.prefix, c.kv_len = [int(n) for n in n1], (n1 + T).astype(np.int32)
    c.c, c.k = c.d["c_kv"].cpu(), c.d["k_pe"].cpu()
    for x in (c.qn, c.qp):
        x.copy_(torch.from_numpy(c.rng.normal(size=tuple(x.shape))))
    for b in range(B):
        at = torch.from_numpy(ar.slots(c.table, b, int(c.kv_len[b]))[n1[b]:])
        for pool in (c.c, c.k):
            flat = pool.view(-1, pool.shape[-1])
            flat[at] = torch.from_numpy(c.rng.normal(size=(T, flat.shape[1]))).to(flat.dtype)
    c.par = ar.random_tree(c.rng, B, T)
    c.see = ar.ancestors(c.par)
    c.path, c.alen = ar.random_path(c.rng, c.par, c.see)
    for b in range(B):
        q, keys = c.parts(b)
        c.lse[b] = ar.lse_ref(q, keys, c.see[b], c.prefix[b], ar.SCALE)
    mask, _ = va.build_tree_mask(cu(c.par))
    c.d.update(q_nope=c.qn.cuda(), q_pe=c.qp.cuda(), c_kv=c.c.cuda(), k_pe=c.k.cuda(),
               kv_len=plan.new_len + T, tree_mask=mask, lse=cu(c.lse))
    w2 = c.run(va, True, weights=plan.weights, decay=0.5, out=plan.weights)
    want2 = c.ref()
    for b in range(B):
        want2[b, :c.kv_len[b]] += 0.5 * old[b, :c.kv_len[b]]
    near(w2, want2)
    pos2 = pos1.copy()
    for b in range(B):
        pos2[b, n1[b]:n1[b] + T] = 10 ** 6 + np.arange(T)
    check_plan(va, w2.cpu().numpy(), c.kv_len, (c.kv_len // 2).astype(np.int32), T, c.path, c.alen,
               pos2, 3, 10, in_place=True, what="second step")
