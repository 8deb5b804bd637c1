"""Cases for timing and checking the operators around the tree-verify step.

Three operators, each reached through the package's public calls:

* ``token_logprobs``: log-sum-exp, entropy, log probabilities of given tokens
  and the top alternatives of each row of logits -- the drafter's per-depth
  top-k that the tree builder reads, and the target's greedy tokens that the
  accept walk reads;
* ``key_weights``: the attention weight each cached key received from the
  tree's (accepted) nodes, recomputed from the verify call's log-sum-exp and
  accumulated per slot;
* ``evict``: ``evict_plan`` chooses which slots of the paged cache stay and
  ``kv_move`` fills the holes in place.

``run`` computes them from elementary torch operations, or with ``own`` set
through the package.  ``exact`` computes the same values in 64 bits, one
request at a time, from the definitions.
"""
import math
import random

import numpy as np
import torch

own = False

DC, DR, PAGE = 512, 64, 64
SCALE = 1.0 / math.sqrt(192.0)
KV_SCALE = float(np.float32(5.0 / 448.0))   # FP8 cache: 5 standard deviations at the largest code
DEPTH = 15


# ------------------------------------------------------------------ the cases

def _lp(name, R, V, dtype, k, G, pad=0, masked=0.0):
    return dict(name=name, op="token_logprobs", R=R, V=V, dtype=dtype, k=k, G=G, pad=pad,
                masked=masked)


def _kw(name, B, H, T, P, dtype, kv, rows, accept, ragged=False):
    return dict(name=name, op="key_weights", B=B, H=H, T=T, P=P, dtype=dtype, kv=kv, rows=rows,
                accept=accept, ragged=ragged)


def _ev(name, B, T, P, kv, keep, sink, recent, accept, with_pos, ragged=False):
    return dict(name=name, op="evict", B=B, T=T, P=P, kv=kv, keep=keep, sink=sink, recent=recent,
                accept=accept, with_pos=with_pos, ragged=ragged)


def listed():
    return [
        # one request's drafter: 15 depths, top 8 of 4096 fp32 logits (the smallest call)
        _lp("lp-draft-b1", 15, 4096, "f32", 8, 0),
        # 64 requests' drafters at once
        _lp("lp-draft-b64", 960, 4096, "f32", 8, 0),
        # the target's greedy token and the draft token's log probability, 64 trees of 33 nodes
        _lp("lp-target-b64", 2112, 131072, "bf16", 1, 1),
        # one tree with alternatives to report; a vocabulary that is no multiple of a vector,
        # a third of the tokens masked out
        _lp("lp-masked-odd", 65, 50257, "bf16", 16, 3, pad=2, masked=0.33),
        # one short request, a few heads on this GPU, accepted nodes only (latency)
        _kw("kw-b1-short", 1, 16, 9, 700, "bf16", "bf16", "path", 3),
        # the batch of the default benchmark: ragged prefixes, accepted nodes
        _kw("kw-b64-ragged", 64, 64, 33, 8192, "bf16", "bf16", "path", 5, ragged=True),
        # every node of deep trees counts: dense tensor work
        _kw("kw-b16-all-nodes", 16, 64, 65, 4096, "bf16", "bf16", "all", 8),
        # FP8 cache, heads split over GPUs, accepted nodes
        _kw("kw-b16-fp8", 16, 16, 65, 16384, "bf16", "fp8", "path", 4),
        # fp32 queries on an fp32 cache
        _kw("kw-f32-page", 1, 64, 33, 2048, "f32", "f32", "all", 4),
        # one short request gives back its rejected nodes and a few keys (latency)
        _ev("ev-b1-short", 1, 9, 700, "f32", 0.9, 4, 64, 3, False),
        # a ragged batch cut to half
        _ev("ev-b64-half", 64, 33, 8192, "bf16", 0.5, 4, 128, 4, True, ragged=True),
        # four long prefixes cut to a quarter
        _ev("ev-b4-long", 4, 65, 131072, "bf16", 0.25, 16, 1024, 6, True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("token_logprobs", "key_weights", "evict"))
    if kind == "token_logprobs":
        V = _log_int(rng, 1000, 160000)
        R = _log_int(rng, 1, min(2112, 2112 * 131072 // V))
        return dict(op=kind, R=R, V=V, dtype=rng.choice(("f32", "bf16")) if R * V < 1.3e8 else "bf16",
                    k=rng.choice((0, 1, 1, 2, 5, 8, 11, 16)), G=rng.choice((0, 1, 1, 3)),
                    pad=rng.choice((0, 0, 1, 8, 33)), masked=rng.choice((0.0, 0.0, 0.1, 0.9)))
    B = _log_int(rng, 1, 64)
    T = rng.choice((1, 9, 17, 33, 47, 64, 65))
    accept = rng.randint(1, min(T, 8))
    if kind == "key_weights":
        H = rng.choice((1, 3, 8, 16, 20, 64, 128))
        dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
        kv = rng.choice((dtype, dtype, "fp8"))
        rows = rng.choice(("path", "path", "all"))
        n = accept if rows == "path" else T
        most = (2.8e8 if dtype == "bf16" else 1e7) / (B * n * H)   # score elements of a pass
        P = _log_int(rng, 16, int(max(32, min(16384, 5e5 / B, most))))
        return dict(op=kind, B=B, H=H, T=T, P=P, dtype=dtype, kv=kv, rows=rows, accept=accept,
                    ragged=rng.random() < 0.5)
    P = _log_int(rng, 64, min(131072, 500000 // B))
    return dict(op=kind, B=B, T=T, P=P, kv=rng.choice(("bf16", "bf16", "fp8", "f32")) if B * P < 2.5e5
                else "bf16", keep=rng.choice((0.1, 0.25, 0.5, 0.75, 0.95)), sink=rng.choice((0, 4)),
                recent=rng.choice((0, 32, 257)), accept=accept, with_pos=rng.random() < 0.5,
                ragged=rng.random() < 0.5)


def _lens(case):
    """Prefix length and accepted length of every request: part of the case, not of the seed."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    B, P, T = case["B"], case["P"], case["T"]
    pre = [r.randint(max(1, P // 16), P) if case["ragged"] else P for _ in range(B)]
    if case["ragged"]:
        pre[r.randrange(B)] = P
    # between one (only the root) and twice the mean less one, at most the tree
    acc = [r.randint(1, max(1, min(T, DEPTH + 1, 2 * case["accept"] - 1))) for _ in range(B)]
    return pre, acc


_EB = {"f32": 4, "bf16": 2, "fp8": 1}


def work(case):
    if case["op"] == "token_logprobs":
        R, V = case["R"], case["V"]
        return {"bytes": R * V * _EB[case["dtype"]] + R * (8 + 8 * case["G"] + 8 * case["k"]),
                "flops": 6.0 * R * V}
    pre, acc = _lens(case)
    T = case["T"]
    if case["op"] == "key_weights":
        H, e, eq = case["H"], _EB[case["kv"]], _EB[case["dtype"]]
        nodes = [a if case["rows"] == "path" else T for a in acc]
        keys = [p + T for p in pre]
        return {"bytes": sum(n * H * (576 * eq + 4) + k * (576 * e + 8) for n, k in zip(nodes, keys)),
                "flops": 2.0 * 576 * H * sum(n * k for n, k in zip(nodes, keys))}
    # kept slots above the new length move down: of the kept, the share that lies above it
    b = 0.0
    for p, a in zip(pre, acc):
        n = p + a
        m = max(1, min(n, int(case["keep"] * p)))
        extra = 8 * (p + T + m) if case["with_pos"] else 0
        b += 8 * p + 4 * m + extra + 2.0 * m * (n - m) / n * 576 * _EB[case["kv"]]
    return {"bytes": b, "flops": 0}


# ---------------------------------------------------------------- the inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _trees(case, rng, acc):
    """Random draft trees of T nodes with an accepted chain of the case's length:
    parents [B, T] (-1: root or absent), path [B, T] (-1 past the end)."""
    B, T = case["B"], case["T"]
    parents = np.full((B, T), -1, np.int32)
    path = np.full((B, T), -1, np.int32)
    for b in range(B):
        chain = [0] + sorted(int(x) for x in rng.choice(np.arange(1, T), acc[b] - 1, replace=False)) \
            if T > 1 else [0]
        on = dict(zip(chain[1:], chain[:-1]))
        depth = [0] * T
        absent_from = T - int(rng.integers(0, 3)) if T > 8 else T   # underfull trees end early
        for i in range(1, T):
            if i in on:
                p = on[i]
            elif i >= absent_from:
                depth[i] = DEPTH
                continue
            else:
                p = int(rng.integers(0, i))
                while depth[p] >= DEPTH or (p > 0 and parents[b, p] < 0):
                    p = int(rng.integers(0, i))
            parents[b, i], depth[i] = p, depth[p] + 1
        path[b, :len(chain)] = chain
    return parents, path


def _ancestors(parents):
    """bool [B, T, T]: node j is node i or one of its ancestors; absent nodes see nothing."""
    B, T = parents.shape
    see = np.zeros((B, T, T), bool)
    for b in range(B):
        see[b, 0, 0] = True
        for i in range(1, T):
            if parents[b, i] >= 0:
                see[b, i] = see[b, parents[b, i]]
                see[b, i, i] = True
    return see


def _mask_words(see):
    B, T, _ = see.shape
    W = (T + 63) // 64
    m = np.zeros((B, T, W), np.uint64)
    for j in range(T):
        m[:, :, j >> 6] |= see[:, :, j].astype(np.uint64) << np.uint64(j & 63)
    return m.view(np.int64)


def _cache(case, kv_len, gen, rng):
    """A page pool with the requests' pages scattered over it."""
    pages = [(k + PAGE - 1) // PAGE for k in kv_len]
    num = sum(pages) + 3
    perm = rng.permutation(num).astype(np.int32)
    table = np.zeros((case["B"], max(pages) + 1), np.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n
    kv = case["kv"]
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}.get(kv, torch.bfloat16)
    c = torch.empty(num, PAGE, DC, device="cuda", dtype=dt).normal_(generator=gen)
    k = torch.empty(num, PAGE, DR, device="cuda", dtype=dt).normal_(generator=gen)
    # one key in fifty is longer than the others: the heavy hitters
    big = torch.where(torch.rand(num, PAGE, 1, device="cuda", generator=gen) < 0.02, 2.0, 1.0).to(dt)
    c *= big
    k *= big
    if kv == "fp8":
        c = (c.float() / KV_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn)
        k = (k.float() / KV_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn)
    return c, k, torch.from_numpy(table).cuda()


def prepare(case, seed):
    gen, rng = _gen(seed), np.random.default_rng(seed)
    if case["op"] == "token_logprobs":
        R, V, G = case["R"], case["V"], case["G"]
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        buf = torch.empty(R, V + case["pad"], device="cuda", dtype=dt)
        buf.normal_(0.0, 2.5, generator=gen)
        if case["masked"]:
            for r0 in range(0, R, 64):
                part = buf[r0:r0 + 64]
                part.masked_fill_(torch.rand(part.shape, device="cuda", generator=gen)
                                  < case["masked"], float("-inf"))
        tok = None
        if G:
            tok = torch.randint(0, V, (R, G), device="cuda", dtype=torch.int32, generator=gen)
            tok[::7, 0] = -1           # absent nodes have no token
        return dict(case=case, logits=buf[:, :V], tokens=tok)

    pre, acc = _lens(case)
    B, T = case["B"], case["T"]
    parents, path = _trees(case, rng, acc)
    kv_len = [p + T for p in pre]
    c, k, table = _cache(case, kv_len, gen, rng)
    cap = table.shape[1] * PAGE
    s = dict(case=case, c_kv=c, k_pe=k, page_table=table, parents=parents, amax=max(acc),
             kv_len=torch.tensor(kv_len, dtype=torch.int32, device="cuda"),
             path=torch.from_numpy(path).cuda(),
             accept_len=torch.tensor(acc, dtype=torch.int32, device="cuda"))
    slot = torch.arange(cap, device="cuda")
    used = slot[None, :] < s["kv_len"][:, None]
    if case["op"] == "evict":
        # what a prefix has collected: few heavy keys, many light ones, some untouched
        w = torch.empty(B, cap, device="cuda").normal_(0.0, 3.0, generator=gen).exp_()
        w = torch.where(torch.rand(B, cap, device="cuda", generator=gen) < 0.05, 0.0, w)
        s["weights"] = torch.where(used, w, 0.0)
        s["budget"] = torch.tensor([max(1, int(case["keep"] * p)) for p in pre],
                                   dtype=torch.int32, device="cuda")
        s["pos"] = None
        if case["with_pos"]:       # an earlier eviction left gaps and another order
            pos = torch.full((B, cap), -1, dtype=torch.int32, device="cuda")
            for b, p in enumerate(pre):
                x = rng.choice(2 * p + 1, p, replace=False).astype(np.int32)
                pos[b, :p] = torch.from_numpy(x).cuda()
                d = [0] * T
                for i in range(1, T):
                    d[i] = d[parents[b, i]] + 1 if parents[b, i] >= 0 else 0
                pos[b, p:p + T] = 2 * p + 1 + torch.tensor(d, dtype=torch.int32, device="cuda")
            s["pos"] = pos
        return s

    H = case["H"]
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    s["q_nope"] = torch.empty(B, T, H, DC, device="cuda", dtype=dt).normal_(generator=gen)
    s["q_pe"] = torch.empty(B, T, H, DR, device="cuda", dtype=dt).normal_(generator=gen)
    see = _ancestors(parents)
    s["mask"] = torch.from_numpy(_mask_words(see)).cuda()
    # the log-sum-exp that the verify call has returned for every row
    lse = torch.empty(B, T, H, device="cuda")
    for b in range(B):
        z = _request_scores(s, b, torch.float32)
        seen = torch.ones(T, kv_len[b], dtype=torch.bool, device="cuda")
        seen[:, pre[b]:] = torch.from_numpy(see[b]).cuda()
        seen &= torch.from_numpy(see[b].any(-1)).cuda()[:, None]     # absent nodes: empty rows
        z.masked_fill_(~seen[:, None, :], float("-inf"))
        lse[b] = torch.logsumexp(z, -1)
        del z
    s["lse"] = lse
    s["weights"] = torch.where(used, torch.rand(B, cap, device="cuda", generator=gen) * 4.0, 0.0)
    s["decay"] = 0.9
    s["out"] = torch.zeros(B, cap, device="cuda")
    if case["rows"] == "all":
        s["path"] = s["accept_len"] = None
    return s


def _request_scores(s, b, dt):
    """scale * q.k of one request, [T, H, kv_len], in the given type."""
    n = int(s["kv_len"][b])
    rows = (s["page_table"][b].long()[:, None] * PAGE + torch.arange(PAGE, device="cuda")).reshape(-1)[:n]
    unit = KV_SCALE if s["case"]["kv"] == "fp8" else 1.0
    k = torch.cat([s["c_kv"].view(-1, DC)[rows].to(dt), s["k_pe"].view(-1, DR)[rows].to(dt)], -1) * unit
    q = torch.cat([s["q_nope"][b].to(dt), s["q_pe"][b].to(dt)], -1)
    return torch.matmul(q, k.t()) * SCALE


# ------------------------------------------------------------- the plain forms

def _orderable(x):
    """fp32 values as int64 that compare alike (NaN as -inf, -0 as 0)."""
    x = torch.where(torch.isnan(x), float("-inf"), x) + 0.0
    i = x.view(torch.int32).long()
    return torch.where(i >= 0, i, -(i & 0x7FFFFFFF))


def _plain_logprobs(s):
    x0, tok, k = s["logits"], s["tokens"], s["case"]["k"]
    x = x0.float()
    V = x.shape[1]
    m = x.max(-1, keepdim=True).values
    e = torch.exp(x - m)
    z = e.sum(-1)
    lse = m[:, 0] + torch.log(z)
    d = torch.where(e > 0, x - m, 0.0)
    out = {"lse": lse, "entropy": torch.log(z) - (e * d).sum(-1) / z}
    if tok is not None:
        at = torch.gather(x, 1, tok.clamp(min=0).long()) - lse[:, None]
        out["tok_lp"] = torch.where(tok >= 0, at, float("-inf"))
    if k:
        key = (_orderable(x) << 32) + (V - 1 - torch.arange(V, device=x.device))
        ids = V - 1 - (torch.topk(key, k, dim=-1).values & 0xFFFFFFFF)
        out["top_ids"] = ids.int()
        out["top_lp"] = torch.gather(x, 1, ids) - lse[:, None]
    return out


def _plain_key_weights(s):
    case = s["case"]
    B, T, H = case["B"], case["T"], case["H"]
    dev = s["c_kv"].device
    cap = s["page_table"].shape[1] * PAGE
    rows = (s["page_table"].long()[:, :, None] * PAGE + torch.arange(PAGE, device=dev)).reshape(B, cap)
    unit = KV_SCALE if case["kv"] == "fp8" else 1.0
    k = torch.cat([s["c_kv"].float().view(-1, DC)[rows], s["k_pe"].float().view(-1, DR)[rows]], -1)
    if s["path"] is None:
        node = torch.arange(T, device=dev).expand(B, T)
        counts = torch.ones(B, T, dtype=torch.bool, device=dev)
    else:
        node = s["path"][:, :s["amax"]].long().clamp(min=0)
        counts = torch.arange(s["amax"], device=dev)[None, :] < s["accept_len"][:, None]
    A = node.shape[1]
    bi = torch.arange(B, device=dev)[:, None]
    q = torch.cat([s["q_nope"][bi, node].float(), s["q_pe"][bi, node].float()], -1)
    lse = s["lse"][bi, node].reshape(B, A * H, 1)
    z = torch.bmm(q.view(B, A * H, DC + DR), k.transpose(1, 2)) * (SCALE * unit)
    p = torch.exp(z - lse)                                            # [B, A H, cap]
    # which keys each node sees: the prefix, and the tail slots of its mask
    slot = torch.arange(cap, device=dev)
    nd = slot[None, :] - (s["kv_len"].long() - T)[:, None]            # [B, cap]
    words = s["mask"][bi, node]                                       # [B, A, W]
    at = nd.clamp(0, T - 1)[:, None, :].expand(B, A, cap)
    bit = (torch.gather(words, 2, at >> 6) >> (at & 63)) & 1
    self_bit = (torch.gather(words, 2, (node >> 6)[:, :, None])[:, :, 0] >> (node & 63)) & 1
    sees = (nd < 0)[:, None, :] | ((nd < T)[:, None, :] & (bit == 1))
    sees &= (counts & (self_bit == 1))[:, :, None]
    w = torch.where(sees[:, :, None, :], p.view(B, A, H, cap), 0.0).sum((1, 2))
    used = slot[None, :] < s["kv_len"][:, None]
    return {"weights": torch.where(used, s["decay"] * s["weights"] + w, 0.0)}


def _plain_evict(s):
    case = s["case"]
    B, T = case["B"], case["T"]
    w, dev = s["weights"], s["weights"].device
    cap = w.shape[1]
    slot = torch.arange(cap, device=dev).expand(B, cap)
    P = (s["kv_len"].long() - T)[:, None]
    bi = torch.arange(B, device=dev)[:, None]
    taken = torch.arange(T, device=dev)[None, :] < s["accept_len"][:, None]
    at = torch.where(taken, P + s["path"].long().clamp(min=0), cap)
    accepted = torch.zeros(B, cap + 1, dtype=torch.bool, device=dev)
    accepted[bi, at] = True
    accepted = accepted[:, :cap]
    cand = (slot < P) | accepted
    pos = slot if s["pos"] is None else s["pos"].long()
    newest = torch.where(cand, pos, -1).max(1, keepdim=True).values
    prot = accepted | (cand & ((pos < case["sink"]) | (newest - pos < case["recent"])))
    group = cand.long() + prot.long()                                  # 2 protected, 1 other, 0 dropped
    key = torch.where(group == 1, _orderable(w), 0) + (group << 34)
    order = torch.sort(key, dim=1, descending=True, stable=True).indices
    n_prot = prot.sum(1, keepdim=True)
    n = torch.maximum(torch.minimum(s["budget"].long()[:, None], cand.sum(1, keepdim=True)), n_prot)
    keep = torch.zeros(B, cap, dtype=torch.bool, device=dev)
    keep[bi, order] = slot < n
    hole = ~keep & (slot < n)
    mover = keep & (slot >= n)
    src = torch.where(slot < n, slot, -1)
    hb, hs = hole.nonzero(as_tuple=True)
    mb, ms = mover.nonzero(as_tuple=True)
    src[hb, hs] = ms                                                   # both in request, slot order
    live = src >= 0
    out = {"new_len": n[:, 0].int(), "from_slot": src.int(),
           "weights": torch.where(live, torch.gather(w, 1, src.clamp(min=0)), 0.0)}
    if s["pos"] is not None:
        out["pos"] = torch.where(live, torch.gather(s["pos"], 1, src.clamp(min=0)), -1)
    rows = (s["page_table"].long()[:, :, None] * PAGE + torch.arange(PAGE, device=dev)).reshape(B, cap)
    to, frm = rows[hb, hs], rows[mb, ms]
    for name, d in (("c_kv", DC), ("k_pe", DR)):
        pool = s[name]
        flat = (pool.view(torch.uint8) if case["kv"] == "fp8" else pool).view(-1, d)
        flat[to] = flat[frm]
        out[name] = pool
    return out


# ------------------------------------------------------- the package's own calls

def _own_logprobs(s):
    import speculative_decoding_tree_va_b200 as va
    case = s["case"]
    r = va.token_logprobs(s["logits"], s["tokens"], k=case["k"])
    out = {"lse": r.lse, "entropy": r.entropy}
    if case["G"]:
        out["tok_lp"] = r.tok_lp
    if case["k"]:
        out["top_ids"], out["top_lp"] = r.top_ids, r.top_lp
    return out


def _own_key_weights(s):
    import speculative_decoding_tree_va_b200 as va
    w = va.key_weights(s["q_nope"], s["q_pe"], s["c_kv"], s["k_pe"], s["page_table"], s["kv_len"],
                       s["mask"], s["lse"], scale=SCALE, path=s["path"], accept_len=s["accept_len"],
                       weights=s["weights"], decay=s["decay"], out=s["out"], kv_scale=KV_SCALE)
    return {"weights": w}


def _own_evict(s):
    import speculative_decoding_tree_va_b200 as va
    case = s["case"]
    r = va.evict_plan(s["weights"], s["kv_len"], s["budget"], pos=s["pos"], path=s["path"],
                      accept_len=s["accept_len"], tree_len=case["T"], n_sink=case["sink"],
                      n_recent=case["recent"])
    va.kv_move(s["c_kv"], s["k_pe"], s["page_table"], r.from_slot, r.new_len)
    out = {"new_len": r.new_len, "from_slot": r.from_slot, "weights": r.weights}
    if s["pos"] is not None:
        out["pos"] = r.pos
    out["c_kv"], out["k_pe"] = s["c_kv"], s["k_pe"]
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"token_logprobs": _own_logprobs, "key_weights": _own_key_weights,
                "evict": _own_evict}[op](state)
    return {"token_logprobs": _plain_logprobs, "key_weights": _plain_key_weights,
            "evict": _plain_evict}[op](state)


# ------------------------------------------------- the definitions, in 64 bits

def _exact_logprobs(s):
    case, R = s["case"], s["case"]["R"]
    lse = torch.empty(R, dtype=torch.float64, device="cuda")
    ent = torch.empty_like(lse)
    tlp = torch.full((R, case["G"]), float("-inf"), dtype=torch.float64, device="cuda")
    ids = torch.empty(R, case["k"], dtype=torch.int32, device="cuda")
    klp = torch.empty(R, case["k"], dtype=torch.float64, device="cuda")
    for r0 in range(0, R, 32):
        x = s["logits"][r0:r0 + 32].double()
        at = slice(r0, r0 + x.shape[0])
        lse[at] = torch.logsumexp(x, -1)
        lp = x - lse[at, None]
        ent[at] = torch.special.entr(lp.exp()).sum(-1)
        if case["G"]:
            t = s["tokens"][at].long()
            got = torch.gather(lp, 1, t.clamp(min=0))
            tlp[at] = torch.where(t < 0, torch.full_like(got, float("-inf")), got)
        if case["k"]:
            # every index that may be among the first k, lowest first, then a stable sort
            low = torch.topk(x, case["k"], dim=-1).values[:, -1:]
            for i in range(x.shape[0]):
                c = (x[i] >= low[i]).nonzero()[:, 0]
                o = c[torch.sort(x[i][c], descending=True, stable=True).indices[:case["k"]]]
                ids[r0 + i], klp[r0 + i] = o.int(), lp[i][o]
    out = {"lse": lse, "entropy": ent}
    if case["G"]:
        out["tok_lp"] = tlp
    if case["k"]:
        out["top_ids"], out["top_lp"] = ids, klp
    return out


def _exact_key_weights(s):
    case = s["case"]
    B, T = case["B"], case["T"]
    see = _ancestors(s["parents"])
    out = torch.zeros(s["weights"].shape, dtype=torch.float64, device="cuda")
    for b in range(B):
        n = int(s["kv_len"][b])
        nodes = list(range(T)) if s["path"] is None else \
            s["path"][b, :int(s["accept_len"][b])].tolist()
        z = _request_scores(s, b, torch.float64)
        acc = s["decay"] * s["weights"][b, :n].double()
        for i in nodes:
            if see[b, i, i]:
                w = torch.exp(z[i] - s["lse"][b, i].double()[:, None]).sum(0)
                w[n - T:] *= torch.from_numpy(see[b, i]).cuda()
                acc += w
        out[b, :n] = acc
    return {"weights": out}


def _exact_evict(s):
    case = s["case"]
    B, T = case["B"], case["T"]
    w = s["weights"].double().cpu().numpy()
    cap = w.shape[1]
    table = s["page_table"].cpu().numpy()
    pos_all = None if s["pos"] is None else s["pos"].cpu().numpy()
    path, acc = s["path"].cpu().numpy(), s["accept_len"].cpu().numpy()
    kv_len, budget = s["kv_len"].cpu().numpy(), s["budget"].cpu().numpy()
    new_len = np.zeros(B, np.int32)
    src = np.full((B, cap), -1, np.int32)
    wo = np.zeros((B, cap))
    po = np.full((B, cap), -1, np.int32)
    moved_to, moved_from = [], []
    for b in range(B):
        P = int(kv_len[b]) - T
        taken = P + path[b, :acc[b]]
        cand = np.concatenate([np.arange(P), taken])
        pos = cand if pos_all is None else pos_all[b, cand]
        safe = (cand >= P) | (pos < case["sink"]) | (pos.max() - pos < case["recent"])
        ranked = np.lexsort((cand, -w[b, cand], ~safe))
        n = max(min(int(budget[b]), len(cand)), int(safe.sum()))
        kept = np.sort(cand[ranked[:n]])
        stay, move = kept[kept < n], kept[kept >= n]
        holes = np.setdiff1d(np.arange(n), stay)
        src[b, stay], src[b, holes] = stay, move
        new_len[b] = n
        wo[b, :n] = w[b, src[b, :n]]
        if pos_all is not None:
            po[b, :n] = pos_all[b, src[b, :n]]
        phys = lambda j: table[b, j // PAGE].astype(np.int64) * PAGE + j % PAGE  # noqa: E731
        moved_to.append(phys(holes))
        moved_from.append(phys(move))
    out = {"new_len": torch.from_numpy(new_len), "from_slot": torch.from_numpy(src),
           "weights": torch.from_numpy(wo)}
    if pos_all is not None:
        out["pos"] = torch.from_numpy(po)
    to = torch.from_numpy(np.concatenate(moved_to)).cuda()
    frm = torch.from_numpy(np.concatenate(moved_from)).cuda()
    for name, d in (("c_kv", DC), ("k_pe", DR)):
        pool = s[name].float().view(-1, d)
        pool[to] = pool[frm]
        out[name] = pool.view(s[name].shape)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"token_logprobs": _exact_logprobs, "key_weights": _exact_key_weights,
            "evict": _exact_evict}[case["op"]](s)
