"""Plain 64-bit forms of the calls around the verify step, and small inputs for them."""
from __future__ import annotations

import math

import numpy as np

SCALE = 1.0 / math.sqrt(192.0)
PAGE = 64


# ------------------------------------------------------------------ logits

def logprobs_ref(x, tokens=None, k=0, scale=1.0):
    """x float64 [R, V] holding the stored logits; one row at a time."""
    R, V = x.shape
    out = dict(lse=np.full(R, np.nan), entropy=np.full(R, np.nan), bad=np.zeros(R, bool),
               top_ids=np.full((R, k), -1, np.int32), top_lp=np.full((R, k), np.nan))
    if tokens is not None:
        out["tok_lp"] = np.full(tokens.shape, np.nan)
    for r in range(R):
        z = x[r] * scale
        if np.isnan(z).any() or np.isposinf(z).any():
            out["bad"][r] = True
            continue
        order = np.lexsort((np.arange(V), -(x[r] + 0.0)))[:k]
        out["top_ids"][r] = order
        m = z.max()
        if m == -np.inf:
            lp = np.full(V, -np.inf)
            out["lse"][r], out["entropy"][r] = -np.inf, 0.0
        else:
            ln_z = math.log(np.exp(z - m).sum())
            lp = (z - m) - ln_z
            out["lse"][r] = m + ln_z
            p = np.exp(lp)
            out["entropy"][r] = -(p[p > 0] * lp[p > 0]).sum()
        out["top_lp"][r] = lp[order]
        if tokens is not None:
            for g, t in enumerate(tokens[r]):
                if t < V:
                    out["tok_lp"][r, g] = lp[t] if t >= 0 else -np.inf
                else:
                    out["bad"][r] = True
    return out


def logprobs_tol(V, scale, x):
    """Absolute error allowed to a fp32 log-sum-exp over V logits, from the arithmetic.

    Each exponent y = (x - m) c is off by at most three half steps of |y| (the
    difference, the product, the rounded constant); its exponential by 2^-22
    (the hardware's 2 units); and a thread adds at most V / 256 + 33 terms in
    a row, then 18 partial sums, each addition off by half a step of a sum of
    positive terms.  Terms beyond |y| = 40 no longer count, so |y| <= 40."""
    steps = 3 * 40 * math.log(2) + 4 + V / 256 + 33 + 18
    return steps * 2.0 ** -24


# ------------------------------------------------------------- trees and caches

def random_tree(rng, B, T, absent=0):
    """parents int32 [B, T] with parent < child; the last `absent` nodes absent."""
    par = np.full((B, T), -1, np.int32)
    for b in range(B):
        for i in range(1, T - absent):
            par[b, i] = rng.integers(max(0, i - 6), i)
    return par


def ancestors(par):
    B, T = par.shape
    see = np.zeros((B, T, T), bool)
    for b in range(B):
        see[b, 0, 0] = True
        for i in range(1, T):
            if par[b, i] >= 0:
                see[b, i] = see[b, par[b, i]]
                see[b, i, i] = True
    return see


def random_path(rng, par, see):
    """A root-to-node path per request: path [B, T] (-1 past the end), length [B]."""
    B, T = par.shape
    path, n = np.full((B, T), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        present = np.flatnonzero(see[b, np.arange(T), np.arange(T)])
        nodes = np.flatnonzero(see[b, rng.choice(present)])
        path[b, :len(nodes)], n[b] = nodes, len(nodes)
    return path, n


def paged(rng, B, kv_len, spare_pages=1):
    """page_table int32 [B, max_pages] over a shuffled pool, and the pool's page count."""
    pages = [-(-int(k) // PAGE) for k in kv_len]
    m = max(pages + [1]) + spare_pages
    num = sum(pages) + 2
    perm = rng.permutation(num).astype(np.int32)
    table = np.zeros((B, m), np.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, num


def slots(table, b, n):
    j = np.arange(n)
    return table[b, j // PAGE].astype(np.int64) * PAGE + j % PAGE


def scores_ref(q, keys, scale):
    """float64 scores [T, H, n] of one request: q [T, H, 576], keys [n, 576]."""
    return np.einsum("thd,nd->thn", q, keys) * scale


def lse_ref(q, keys, see, P, scale):
    """float64 log-sum-exp [T, H] of one request's rows (-inf for absent nodes)."""
    s = scores_ref(q, keys, scale)
    T = q.shape[0]
    vis = np.ones((T, keys.shape[0]), bool)
    vis[:, P:] = see
    vis &= see[np.arange(T), np.arange(T)][:, None]
    s = np.where(vis[:, None, :], s, -np.inf)
    m = np.where(np.isneginf(s.max(-1)), 0.0, s.max(-1))
    with np.errstate(divide="ignore"):
        return m + np.log(np.exp(s - m[..., None]).sum(-1))


def key_weights_ref(q, keys, see, lse, nodes, P, scale):
    """float64 weight of each key of one request from the counted nodes."""
    s = scores_ref(q, keys, scale)
    w = np.zeros(keys.shape[0])
    for i in nodes:
        if not see[i, i]:
            continue
        live = ~np.isneginf(lse[i])
        e = np.exp(s[i][live] - lse[i][live][:, None]).sum(0)
        e[P:] = np.where(see[i], e[P:], 0.0)
        w += e
    return w


# ------------------------------------------------------------------ eviction

def evict_ref(w, kv_len, budget, T=0, path=None, alen=None, pos=None, n_sink=0, n_recent=0):
    """(new_len, from_slot, weights, pos, flagged) of a whole batch, slot by slot."""
    B, cap = w.shape
    new_len = np.zeros(B, np.int32)
    src = np.full((B, cap), -1, np.int32)
    wo = np.zeros((B, cap), np.float32)
    po = np.full((B, cap), -1, np.int32)
    flagged = np.zeros(B, bool)
    for b in range(B):
        n_all = int(kv_len[b])
        if not T <= n_all <= cap:
            flagged[b] = True
            continue
        P = n_all - T
        nodes = []
        if T:
            a = int(alen[b])
            ok = 0 <= a <= T
            nodes = [int(x) for x in path[b, :a]] if ok else []
            ok = ok and all(0 <= x < T for x in nodes) and nodes == sorted(set(nodes))
            if not ok:
                flagged[b] = True
                new_len[b] = n_all
                src[b, :n_all] = np.arange(n_all)
                wo[b, :n_all] = w[b, :n_all]
                if pos is not None:
                    po[b, :n_all] = pos[b, :n_all]
                continue
        cand = list(range(P)) + [P + x for x in nodes]
        where = {j: (j if pos is None else int(pos[b, j])) for j in cand}
        newest = max(where.values()) if cand else 0
        safe = [j for j in cand if j >= P or where[j] < n_sink or newest - where[j] < n_recent]
        held = set(safe)
        rest = [j for j in cand if j not in held]
        key = lambda j: -np.inf if np.isnan(w[b, j]) else float(w[b, j])  # noqa: E731
        rest.sort(key=lambda j: (-key(j), j))
        n = max(min(max(int(budget[b]), 0), len(cand)), len(safe))
        kept = sorted(safe + rest[:n - len(safe)])
        new_len[b] = n
        stay = set(j for j in kept if j < n)
        movers = [j for j in kept if j >= n]
        holes = [d for d in range(n) if d not in stay]
        for d in stay:
            src[b, d] = d
        for d, j in zip(holes, movers):
            src[b, d] = j
        for d in range(n):
            wo[b, d] = w[b, src[b, d]]
            if pos is not None:
                po[b, d] = pos[b, src[b, d]]
    return new_len, src, wo, po, flagged
