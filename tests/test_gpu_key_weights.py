"""Accumulated attention weights on the GPU against 64 bits, and the step they belong to."""
import numpy as np
import pytest

import _around as ar

pytestmark = pytest.mark.gpu

# An entry is a sum of positive terms exp(s - lse), so its relative error is at
# most that of its worst term.  s is a sum of 576 products; partial sums stay
# below 100 in q.k units (four standard deviations of 24), each fp32 addition
# rounds at most 2^-24 of that, and independent roundings grow like the square
# root of their count: 100 * 2^-24 * 24 = 1.4e-4 in q.k, 1.0e-5 after the scale
# of 1/13.86.  exp adds 2^-22, s - lse and its product with log2(e) 2^-23 of at
# most 20: 5e-6.  Sums of up to 8320 rows in chains of at most 160: 1e-5.
RTOL = 2.5e-5


@pytest.fixture(scope="module")
def va():
    import speculative_decoding_tree_va_b200 as va
    va.load_library()
    return va


def cu(a):
    import torch
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Case:
    """One batch: queries, paged cache, tree, log-sum-exp; float64 copies beside them."""

    def __init__(self, seed, B, H, T, prefix, dtype="bf16", kv=None, absent=0, stale="finite",
                 spare=1):
        import torch
        kv = kv or dtype
        rng = np.random.default_rng(seed)
        self.B, self.H, self.T, self.rng = B, H, T, rng
        self.prefix = [prefix] * B if np.isscalar(prefix) else list(prefix)
        self.kv_len = np.array([p + T for p in self.prefix], np.int32)
        self.par = ar.random_tree(rng, B, T, absent)
        self.see = ar.ancestors(self.par)
        self.path, self.alen = ar.random_path(rng, self.par, self.see)
        self.table, num = ar.paged(rng, B, self.kv_len, spare)
        dt = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
        val = lambda *s: torch.from_numpy(rng.normal(size=s).astype(np.float32)).to(dt)  # noqa: E731
        self.qn, self.qp = val(B, T, H, 512), val(B, T, H, 64)
        self.c, self.k = val(num, 64, 512), val(num, 64, 64)
        self.kv_scale = 1.0
        if kv == "fp8":
            self.kv_scale = float(np.float32(5 / 448))
            self.c, self.k = ((x.float() / self.kv_scale).clamp(-448, 448).to(torch.float8_e4m3fn)
                              for x in (self.c, self.k))
        used = np.zeros(num * 64, bool)
        for b in range(B):
            used[ar.slots(self.table, b, int(self.kv_len[b]))] = True
        if stale == "nan":
            junk = torch.from_numpy(~used).view(num, 64, 1)
            for x in (self.c, self.k):
                if kv == "fp8":
                    x.view(torch.uint8).masked_fill_(junk, 0x7f)
                else:
                    x.masked_fill_(junk, float("nan"))
        self.lse = np.zeros((B, T, H), np.float32)
        for b in range(B):
            q, keys = self.parts(b)
            self.lse[b] = ar.lse_ref(q, keys, self.see[b], self.prefix[b], ar.SCALE)
        words = np.zeros((B, T, (T + 63) // 64), np.uint64)
        for j in range(T):
            words[:, :, j >> 6] |= self.see[:, :, j].astype(np.uint64) << np.uint64(j & 63)
        self.d = dict(q_nope=self.qn.cuda(), q_pe=self.qp.cuda(), c_kv=self.c.cuda(),
                      k_pe=self.k.cuda(), page_table=cu(self.table), kv_len=cu(self.kv_len),
                      tree_mask=cu(words.view(np.int64)), lse=cu(self.lse))
        self.cap = self.table.shape[1] * 64

    def parts(self, b):
        import torch
        q = torch.cat([self.qn[b], self.qp[b]], -1).double().numpy()
        at = torch.from_numpy(ar.slots(self.table, b, int(self.kv_len[b])))
        c = self.c.view(-1, 512)[at].to(torch.float64)
        k = self.k.view(-1, 64)[at].to(torch.float64)
        return q, torch.cat([c, k], -1).numpy() * self.kv_scale

    def ref(self, path=True, old=None, decay=1.0, skip=()):
        out = np.zeros((self.B, self.cap))
        for b in range(self.B):
            n = int(self.kv_len[b])
            nodes = self.path[b, :self.alen[b]] if path else range(self.T)
            q, keys = self.parts(b)
            lse = self.lse[b].astype(np.float64)
            if b not in skip:
                out[b, :n] = ar.key_weights_ref(q, keys, self.see[b], lse, nodes, self.prefix[b],
                                                np.float64(np.float32(ar.SCALE)))
            if old is not None:
                out[b, :n] += float(np.float32(decay)) * old[b, :n].astype(np.float64)
        return out

    def run(self, va, path=True, **kw):
        if path:
            kw = dict(path=cu(self.path), accept_len=cu(self.alen), **kw)
        return va.key_weights(**self.d, scale=ar.SCALE, kv_scale=self.kv_scale, **kw)


def near(got, want, what=""):
    got = got.double().cpu().numpy()
    assert np.array_equal(got == 0, want == 0), what
    off = np.abs(got - want) / np.maximum(np.abs(want), 1e-30)
    assert off[want != 0].max(initial=0) <= RTOL, (what, off.max())


KINDS = [("f32", "f32", 0), ("f32", "fp8", 0), ("bf16", "bf16", 0), ("bf16", "fp8", 0),
         ("bf16", "bf16", 1), ("bf16", "fp8", 1), ("f32", "f32", 1), ("f32", "fp8", 1)]


@pytest.mark.parametrize("dtype,kv,flags", KINDS)
@pytest.mark.parametrize("B,H,T,prefix,absent", [
    (1, 1, 1, 0, 0), (1, 1, 1, 1, 0), (2, 3, 5, (0, 70), 0), (1, 16, 9, 119, 2),
    (3, 8, 33, (1, 640, 255), 3), (1, 64, 65, 300, 0), (2, 20, 65, (63, 64), 20),
    (1, 128, 65, 130, 1), (5, 1, 64, (10, 500, 20, 1, 127), 0),
])
def test_weights(va, dtype, kv, flags, B, H, T, prefix, absent):
    c = Case(B * 100 + H + T, B, H, T, prefix, dtype, kv, absent)
    for path in (True, False):
        near(c.run(va, path, flags=flags), c.ref(path), f"{dtype} {kv} path={path}")


@pytest.mark.parametrize("dtype,kv,flags", KINDS)
def test_accumulation_in_place_and_untouched_slots(va, dtype, kv, flags):
    """decay * old + new, in place or into another array; nothing from kv_len on is
    written, and NaN in unused slots of a page reaches nothing."""
    import torch
    c = Case(5, 3, 8, 17, (5, 200, 431), dtype, kv, stale="nan", spare=2)
    old = np.abs(c.rng.normal(size=(3, c.cap))).astype(np.float32)
    want = c.ref(True, old, 0.75)
    used = np.arange(c.cap)[None] < c.kv_len[:, None]
    out = torch.full((3, c.cap), -7.0, device="cuda")
    got = c.run(va, True, weights=cu(old), decay=0.75, out=out, flags=flags)
    assert got is out
    g = got.double().cpu().numpy()
    assert (g[~used] == -7).all()
    near(torch.from_numpy(np.where(used, g, 0)), want)
    both = cu(old)
    c.run(va, True, weights=both, decay=0.75, out=both, flags=flags)
    g2 = both.cpu().numpy()
    assert np.array_equal(g2[used], got.cpu().numpy()[used])
    assert np.array_equal(g2[~used], old[~used])


@pytest.mark.parametrize("dtype,kv,flags", KINDS)
def test_long_prefix_with_few_rows(va, dtype, kv, flags):
    c = Case(6, 1, 4, 9, 9000, dtype, kv)
    near(c.run(va, flags=flags), c.ref())


@pytest.mark.parametrize("dtype,kv,flags", KINDS)
def test_flagged_requests(va, dtype, kv, flags):
    """Bad lengths, pages, path entries and accept lengths are flagged and contained."""
    import torch
    c = Case(7, 7, 4, 9, (100, 150, 90, 80, 200, 64, 70), dtype, kv)
    old = np.ones((7, c.cap), np.float32)
    want = c.ref(True, old, 1.0, skip=(3, 4))
    c.d["kv_len"][0] = 8                      # shorter than the tree
    c.d["kv_len"][1] = c.cap + 1
    c.d["page_table"][2, 1] = -1              # keys 64 .. 98 of request 2
    want[2, 64:99] = 1.0
    want[0], want[1] = -7, -7                 # not written
    alen = c.alen.copy()
    alen[3], alen[4] = -1, 10
    path = c.path.copy()
    path[5, 0] = 9                            # the root's entry is bad: that node is left out
    q, keys = c.parts(5)
    want[5, :73] = 1.0 + ar.key_weights_ref(q, keys, c.see[5], c.lse[5].astype(np.float64),
                                            c.path[5, 1:c.alen[5]], 64, np.float64(np.float32(ar.SCALE)))
    status = torch.zeros(7, dtype=torch.int32, device="cuda")
    out = torch.full((7, c.cap), -7.0, device="cuda")
    got = va.key_weights(**c.d, scale=ar.SCALE, kv_scale=c.kv_scale, path=cu(path),
                         accept_len=cu(alen), weights=cu(old), out=out, req_status=status, flags=flags)
    torch.cuda.synchronize()
    assert status.cpu().tolist() == [1, 1, 1, 1, 1, 1, 0]
    used = np.arange(c.cap)[None] < c.kv_len[:, None]
    want = np.where(used, want, -7)
    off = np.abs(got.double().cpu().numpy() - want) / np.abs(want)
    assert off.max() <= RTOL


@pytest.mark.parametrize("flags", [0, 1])
def test_many_short_requests(va, flags):
    """More requests than the kernel has threads: its ranges begin inside a thread's share."""
    rng = np.random.default_rng(21)
    c = Case(22, 1100, 2, 3, rng.integers(0, 40, 1100), "bf16")
    near(c.run(va, flags=flags), c.ref())


def test_empty_counts(va):
    """No accepted node, and a path that lists a node twice."""
    c = Case(8, 2, 4, 9, (100, 30))
    c.path[1, :3], c.alen[:] = (0, 0, 0), (0, 3)
    near(c.run(va), c.ref())


@pytest.mark.parametrize("dtype,kv,flags", [("bf16", "bf16", 0), ("bf16", "fp8", 0),
                                            ("f32", "f32", 0), ("f32", "f32", 1)])
@pytest.mark.parametrize("B,H,T,prefix", [(2, 5, 33, 700), (3, 64, 40, 300), (1, 16, 65, 2100),
                                          (80, 8, 24, 200)])
def test_lists_longer_than_any_path(va, dtype, kv, flags, B, H, T, prefix):
    """T entries in any order, some more than once and some not at all: more rows than
    the deepest path has, and than the sizes let the host expect."""
    c = Case(B + T, B, H, T, prefix, dtype, kv)
    c.path = c.rng.integers(0, T, (B, T)).astype(np.int32)
    c.alen = np.full(B, T, np.int32)
    c.alen[B // 2] = T - 1
    near(c.run(va, flags=flags), c.ref())


def test_same_bits_on_every_run_stream_and_replay(va):
    import torch
    c = Case(9, 2, 64, 33, (500, 77))
    a = c.run(va, False)
    assert torch.equal(a, c.run(va, False))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = c.run(va, False, stream=s)
    s.synchronize()
    assert torch.equal(a, other)
    path, alen = cu(c.path), cu(c.alen)
    kw = dict(scale=ar.SCALE, path=path, accept_len=alen)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        r1 = va.key_weights(**c.d, **kw)
    with torch.cuda.graph(g2):
        r2 = va.key_weights(**c.d, **kw)
    alen.fill_(1)
    c.alen[:] = 1
    for g in (g1, g2, g1):
        g.replay()
    torch.cuda.synchronize()
    near(r1, c.ref())
    assert torch.equal(r1, r2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_step_with_eviction(va, dtype):
    """Drafter logits -> tree -> mask -> verify -> target logits -> accept -> key weights ->
    plan -> move, each stage on the one before; then a verify over what stayed, with the
    kept keys' rows as 64 bits see them."""
    import torch

    import oracle
    B, H, L, V, budget = 3, 8, 8, 2000, 16
    T = budget + 1
    g = torch.Generator(device="cuda").manual_seed(13)
    draft = torch.randn(B, L, V, device="cuda", generator=g) * 2
    top = va.token_logprobs(draft, k=4, wide=True)
    par, tok, _, _ = va.build_tree(top.top_lp, top.top_ids, budget)
    mask, _ = va.build_tree_mask(par)
    c = Case(14, B, H, T, (300, 41, 130), dtype)
    c.par = par.cpu().numpy()
    c.see = ar.ancestors(c.par)
    c.d["tree_mask"] = mask
    d = {k: c.d[k] for k in ("q_nope", "q_pe", "c_kv", "k_pe", "page_table", "kv_len", "tree_mask")}
    _, lse = va.verify_attn(**d, scale=ar.SCALE)
    # a target that agrees with the first child of every node
    target = torch.randn(B, T, V, device="cuda", generator=g)
    p_h, t_h = c.par, tok.cpu().numpy()
    for b in range(B):
        for i in range(T - 1, 0, -1):
            if p_h[b, i] >= 0:
                target[b, p_h[b, i]] += torch.nn.functional.one_hot(
                    torch.tensor(int(t_h[b, i])), V).cuda() * (40.0 + T - i)
    greedy = va.token_logprobs(target, tok, k=1)
    assert torch.equal(greedy.top_ids[..., 0], target.argmax(-1).int())
    path, alen, _ = va.tree_accept(par, tok, greedy.top_ids[..., 0].contiguous())
    ref_path = oracle.tree_accept(p_h, t_h, greedy.top_ids[..., 0].cpu().numpy())
    assert np.array_equal(path.cpu().numpy(), ref_path[0]) and int(alen.max()) > 1
    c.path, c.alen, c.lse = path.cpu().numpy(), alen.cpu().numpy(), lse.cpu().numpy()
    c.d["lse"] = lse
    w = c.run(va, True)
    near(w, c.ref())
    plan = va.evict_plan(w, d["kv_len"], (d["kv_len"] // 2).int(), path=path, accept_len=alen,
                         tree_len=T, n_sink=2, n_recent=8)
    ref = ar.evict_ref(w.cpu().numpy(), c.kv_len, c.kv_len // 2, T, c.path, c.alen, None, 2, 8)
    assert np.array_equal(plan.from_slot.cpu().numpy(), ref[1])
    kept = []
    for b in range(B):
        _, keys = c.parts(b)
        kept.append(keys[ref[1][b, :ref[0][b]]])
    va.kv_move(d["c_kv"], d["k_pe"], d["page_table"], plan.from_slot, plan.new_len)
    # every kept key is now prefix; the next root is appended behind it (one node)
    q_n, q_p = d["q_nope"][:, :1].contiguous(), d["q_pe"][:, :1].contiguous()
    one = torch.ones(B, 1, 1, dtype=torch.int64, device="cuda")
    out, lse = va.verify_attn(q_n, q_p, d["c_kv"], d["k_pe"], d["page_table"], plan.new_len, one,
                              scale=ar.SCALE)
    for b in range(B):
        q = torch.cat([q_n[b], q_p[b]], -1).double().cpu().numpy()
        s = ar.scores_ref(q, kept[b], ar.SCALE)[0]
        p = np.exp(s - s.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        tol = 1e-5 if dtype == "f32" else 1e-2
        assert np.abs(out[b, 0].double().cpu().numpy() - p @ kept[b][:, :512]).max() <= tol
