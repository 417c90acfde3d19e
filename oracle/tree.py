"""Oracle for the operators on drafted trees -- test infrastructure only.

Only the tests and ``__graft_entry__.smoke()`` may import this module. It shares no code with the
product library: plain loops and numpy in float64, straight from the definitions in the header.

A tree: node 0 is the root, parents[i] < i or -1. A node sees itself, its ancestors and the
context, within the window; the context keys come first in the cache, then the nodes' in order.

Pinning: ``tests/test_oracle_tree_pins.py`` checks the closed forms (chains against causal blocks, one key, uniform
scores, brute-force ancestor sets, acceptance over every token pattern of a tiny tree, moves
against a list).
"""
from __future__ import annotations

import math

import numpy as np


def chain_up(parents, i):
    """[i, its parent, ..., the root]"""
    out = [int(i)]
    while parents[out[-1]] >= 0:
        out.append(int(parents[out[-1]]))
    return out


def visible(parents, n, ctx, window):
    """Truth values [n, ctx + n]: which keys each node sees."""
    vis = np.zeros((n, ctx + n), dtype=bool)
    for i in range(n):
        up = chain_up(parents, i)
        pos = ctx + len(up) - 1
        for j in range(ctx):
            vis[i, j] = window == 0 or j > pos - window
        for step, a in enumerate(up):
            vis[i, ctx + a] = window == 0 or pos - step > pos - window
    return vis


def tree_attn(q, keys, values, parents, ctx, window, scale):
    """One request: q [n, Hq, D], keys and values [ctx + n, Hkv, D] float64. Returns out [n, Hq, D],
    lse [n, Hq], spread [n, Hq, D] (sum_j p_j |v_j|) and size [n, Hq] (the largest
    scale * sum_d |q_d k_d| over the visible keys): the quantities that error bounds are made of."""
    n, hq, d = q.shape
    hkv = keys.shape[1]
    vis = visible(parents, n, ctx, window)
    out, spread = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    lse, size = np.zeros((n, hq)), np.zeros((n, hq))
    for h in range(hq):
        g = h // (hq // hkv)
        for i in range(n):
            k, v = keys[vis[i], g], values[vis[i], g]
            s = scale * (k @ q[i, h])
            m = s.max()
            e = np.exp(s - m)
            p = e / e.sum()
            out[i, h], spread[i, h] = p @ v, p @ np.abs(v)
            lse[i, h] = m + math.log(e.sum())
            size[i, h] = scale * (np.abs(k) @ np.abs(q[i, h])).max()
    return out, lse, spread, size


def token_logprobs(logits, tokens, top_k, temperature):
    """Rows of float64 logits [R, V], tokens [R, m] (or None). Returns token_logp, entropy, log_z, top, top_logp."""
    R, V = logits.shape
    logp = np.full((R, V), -np.inf)
    log_z, entropy = np.full(R, -np.inf), np.zeros(R)
    for r in range(R):
        x = logits[r] / temperature
        m = x.max()
        if m == -np.inf:
            continue
        ln_s = math.log(np.exp(x - m).sum())
        log_z[r] = m + ln_s
        logp[r] = (x - m) - ln_s  # about the maximum: rows of the type's lowest value lose ln_s beside m
        live = logp[r] > -np.inf
        entropy[r] = -(np.exp(logp[r][live]) * logp[r][live]).sum()
    given = None
    if tokens is not None:
        given = np.full(tokens.shape, -np.inf)
        for r in range(R):
            for j, t in enumerate(tokens[r]):
                if 0 <= t < V:
                    given[r, j] = logp[r, t]
    # largest first, of equal values the smaller id
    top = np.argsort(-logits, axis=1, kind="stable")[:, :top_k]
    return given, entropy, log_z, top, np.take_along_axis(logp, top, axis=1)


def tree_accept(logits, tokens, parents, num_nodes):
    """logits [B, T, V] float64. Returns accepted [B], path [B, T], next token [B], argmax [B, T]."""
    B, T, _ = logits.shape
    acc, path = np.zeros(B, dtype=np.int64), np.full((B, T), -1, dtype=np.int64)
    nxt, best = np.full(B, -1, dtype=np.int64), np.full((B, T), -1, dtype=np.int64)
    for b in range(B):
        n = int(num_nodes[b])
        if n == 0:
            continue
        best[b, :n] = logits[b, :n].argmax(axis=1)
        at = 0
        path[b, 0] = 0
        while True:
            child = [i for i in range(n) if parents[b, i] == at and tokens[b, i] == best[b, at]]
            if not child:
                break
            at = child[0]
            acc[b] += 1
            path[b, acc[b]] = at
        nxt[b] = best[b, at]
    return acc, path, nxt, best


def tree_commit(cache, page_table, seq_lens, path, accepted, num_nodes):
    """cache [layers, pages, page_size, Hkv, D]: a changed copy, and the new lengths."""
    P = cache.shape[2]
    new = cache.copy()
    lens = np.array(seq_lens, dtype=np.int64)
    for b in range(len(lens)):
        if num_nodes[b] == 0:
            continue
        ctx = int(seq_lens[b] - num_nodes[b])
        for s in range(1, int(accepted[b]) + 1):
            src, dst = ctx + int(path[b, s]), ctx + s
            new[:, page_table[b, dst // P], dst % P] = cache[:, page_table[b, src // P], src % P]
        lens[b] = ctx + accepted[b] + 1
    return new, lens
