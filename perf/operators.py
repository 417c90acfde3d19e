"""What is measured of the operators for drafted token trees: cases, inputs, plain forms.

Four operators, in the order in which a serving loop runs them:

  token_logprobs  log probabilities of given tokens, entropy and the top alternatives of rows of
                  logits: a drafter's candidates for the next level of the tree, and what a server
                  answers when a user asks for log probabilities
  tree_attn       attention of a tree of drafted tokens over the paged cache: a node sees its
                  request's context and its own ancestors
  tree_accept     the target's token at every node and the longest accepted path from the root
  tree_commit     the accepted nodes' keys and values moved to consecutive positions of the cache

With ``own`` false ``run`` computes them in elementary torch operations in 32 bits; with ``own``
true it makes the calls of this package.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------- cases


def listed():
    return [
        # One drafted token on a short context: the cost of the call itself.
        dict(name="attn_one_token", op="tree_attn", batch=1, nodes=1, hq=32, hkv=8, dim=128, page=16, lo=1003,
             hi=1003, window=0, dtype="bf16"),
        # A verify step of one request at the framework's global layer (32/4 heads of 512, 8k keys):
        # few rows on a long axis that has to be split.
        dict(name="attn_global_8k", op="tree_attn", batch=1, nodes=24, hq=32, hkv=4, dim=512, page=16, lo=8192,
             hi=8192, window=0, dtype="bf16"),
        # Sliding-window layers of four long requests (the framework's 32/16 heads of 256, window 1024).
        dict(name="attn_sliding", op="tree_attn", batch=4, nodes=16, hq=32, hkv=16, dim=256, page=16, lo=30001,
             hi=32768, window=1024, dtype="bf16"),
        # A batch of ragged requests with trees of up to 64 nodes: 256 query rows per KV head.
        dict(name="attn_batch_ragged", op="tree_attn", batch=8, nodes=64, hq=32, hkv=8, dim=128, page=32, lo=1024,
             hi=32768, window=0, dtype="bf16"),
        # Long contexts: the K/V stream is everything.
        dict(name="attn_long_128k", op="tree_attn", batch=4, nodes=32, hq=32, hkv=8, dim=128, page=64, lo=120001,
             hi=131072, window=0, dtype="bf16"),
        # 32-bit caches: a small model, or a check of a 16-bit one.
        dict(name="attn_fp32", op="tree_attn", batch=2, nodes=12, hq=8, hkv=2, dim=64, page=16, lo=1501, hi=2500,
             window=0, dtype="fp32"),
        # The log probability of one sampled token, with eight alternatives, some tokens ruled out.
        dict(name="logprobs_one_row", op="token_logprobs", rows=1, vocab=32000, given=1, top=8, temperature=1.0,
             dtype="bf16", masked=True),
        # Scoring a prompt with 32-bit logits, or 64 candidates a slot for a large batch.
        dict(name="logprobs_prompt", op="token_logprobs", rows=1000, vocab=151937, given=3, top=64, temperature=0.7,
             dtype="fp32", masked=False),
        # Acceptance of one small tree.
        dict(name="accept_one", op="tree_accept", batch=1, nodes=16, vocab=32000, dtype="bf16"),
        # Acceptance of a batch of trees of up to 64 nodes: every node's row of logits is read.
        dict(name="accept_batch", op="tree_accept", batch=8, nodes=64, vocab=262144, dtype="bf16"),
        # Moving one request's accepted nodes in one layer's cache.
        dict(name="commit_one", op="tree_commit", batch=1, nodes=16, layers=1, hkv=4, dim=512, page=16, lo=1001,
             hi=1001, accepted=4, dtype="bf16"),
        # Moving the accepted nodes of a batch in every layer's cache with one call.
        dict(name="commit_layers", op="tree_commit", batch=32, nodes=64, layers=32, hkv=8, dim=128, page=16, lo=201,
             hi=400, accepted=6, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: any operator, sizes over the whole range (their logarithm)."""
    op = rng.choice(["tree_attn", "tree_attn", "tree_attn", "token_logprobs", "tree_accept", "tree_commit"])
    if op == "tree_attn":
        dtype = "fp32" if rng.random() < 0.2 else "bf16"
        hq, hkv, dim = rng.choice([(32, 8, 128), (32, 4, 512), (32, 16, 256), (32, 8, 64), (8, 8, 128), (16, 2, 64),
                                   (28, 4, 128), (8, 1, 256), (12, 2, 96), (20, 4, 192), (6, 3, 80)])
        nodes = _log_int(rng, 1, 128)
        case = dict(op=op, batch=_log_int(rng, 1, 12), nodes=nodes, hq=hq, hkv=hkv, dim=dim,
                    page=rng.choice([16, 16, 32, 64, 8, 48]), window=rng.choice([0, 0, 0, 512, 1000]), dtype=dtype)
        hi = _log_int(rng, nodes + 30, 131072 if dtype == "bf16" else 8192)
        case["hi"] = hi
        case["lo"] = max(nodes, int(hi * rng.uniform(0.1, 1.0)))
        limit = work([c for c in listed() if c["name"] == "attn_long_128k"][0])
        while case["batch"] > 1 and (work(case)["bytes"] > limit["bytes"] or work(case)["flops"] > limit["flops"]):
            case["batch"] -= 1
        while work(case)["bytes"] > limit["bytes"] or work(case)["flops"] > limit["flops"]:
            case["hi"] = case["hi"] * 3 // 4
            case["lo"] = max(nodes, min(case["lo"], case["hi"]))
        return case
    if op == "token_logprobs":
        vocab = rng.choice([32000, 50257, 151936, 262144, _log_int(rng, 1000, 262144)])
        dtype = rng.choice(["bf16", "fp32"])
        most = 1000 * 151937 * 4 // (vocab * (2 if dtype == "bf16" else 4))
        return dict(op=op, rows=_log_int(rng, 1, min(4000, most)), vocab=vocab, given=rng.randint(0, 8),
                    top=rng.choice([0, 1, 5, 20, 64, rng.randint(1, 64)]),
                    temperature=rng.choice([1.0, 1.0, 0.7, 1.3]), dtype=dtype, masked=rng.random() < 0.4)
    if op == "tree_accept":
        vocab = rng.choice([32000, 50257, 151936, 262144, _log_int(rng, 1000, 262144)])
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        nodes = _log_int(rng, 1, 128)
        most = 8 * 64 * 262144 * 2 // (nodes * vocab * (2 if dtype == "bf16" else 4))
        return dict(op=op, batch=_log_int(rng, 1, max(1, min(64, most))), nodes=nodes, vocab=vocab, dtype=dtype)
    hkv, dim = rng.choice([(8, 128), (4, 512), (16, 256), (2, 64), (1, 80)])
    nodes = _log_int(rng, 4, 128)
    lo = rng.randint(nodes, nodes + 300)
    return dict(op=op, batch=_log_int(rng, 1, 32), nodes=nodes, layers=_log_int(rng, 1, 32), hkv=hkv, dim=dim,
                page=rng.choice([16, 32, 64]), lo=lo, hi=lo + rng.randint(0, 300),
                accepted=rng.randint(0, min(6, nodes // 2)), dtype=rng.choice(["bf16", "bf16", "fp32"]))


def _nodes_of(case):
    """Nodes of each request's tree: from the widest down to three quarters of it."""
    n = case["nodes"]
    return [n - (7 * b) % (n // 4 + 1) for b in range(case["batch"])]


def _lens_of(case):
    """Keys of each request, its tree's own among them: spread from lo to hi, the longest not last."""
    B, lo, hi = case["batch"], case["lo"], case["hi"]
    if B == 1:
        return [hi]
    return [lo + (hi - lo) * ((5 * b + B - 1) % B) // (B - 1) for b in range(B)]


def _accepted_of(case):
    return [case["accepted"] - b % (case["accepted"] + 1) for b in range(case["batch"])]


def _elem(case):
    return 2 if case["dtype"] == "bf16" else 4


def work(case):
    e = _elem(case)
    if case["op"] == "tree_attn":
        hq, hkv, d = case["hq"], case["hkv"], case["dim"]
        nbytes = flops = 0
        for n, length in zip(_nodes_of(case), _lens_of(case)):
            ctx = length - n
            # the keys that some node sees, and about half of its own tree on average
            keys = n + (min(ctx, case["window"]) if case["window"] else ctx)
            nbytes += keys * hkv * d * 2 * e + n * hq * (2 * d * e + 4)
            flops += 4 * n * hq * d * (keys - n + (n + 1) // 2)
        return dict(bytes=nbytes, flops=flops)
    if case["op"] == "token_logprobs":
        r, v = case["rows"], case["vocab"]
        return dict(bytes=r * (v * e + 8 * case["given"] + 8 * case["top"] + 8), flops=5 * r * v)
    if case["op"] == "tree_accept":
        rows = sum(_nodes_of(case))
        return dict(bytes=rows * (case["vocab"] * e + 16), flops=rows * case["vocab"])
    moved = sum(_accepted_of(case)) * case["layers"] * case["hkv"] * case["dim"] * 2
    return dict(bytes=2 * moved * e + case["batch"] * case["nodes"] * 4, flops=0)


# ------------------------------------------------------------------------------------ inputs


def _trees(gen, nodes, width):
    """Parents [B, width] int32 of random trees: node 0 is the root, every other node hangs on one
    of the nodes before it, mostly on one of the last few; -1 in the padding."""
    dev = gen.device
    B = len(nodes)
    reach = torch.rand((B, width), generator=gen, device=dev) ** 2
    i = torch.arange(width, device=dev)
    parents = (i - 1 - (reach * torch.clamp(i, max=12)).long()).clamp(min=0)
    parents = torch.where(i == 0, -torch.ones_like(parents), parents)
    n = torch.tensor(nodes, device=dev)
    return torch.where(i[None, :] < n[:, None], parents, -torch.ones_like(parents)).to(torch.int32)


def _pages(gen, lens, page):
    """A page table over a shuffled pool a quarter larger than needed, and the pool's pages."""
    need = [(x + page - 1) // page for x in lens]
    total = sum(need)
    pool = total + total // 4 + 1
    perm = torch.randperm(pool, generator=gen, device=gen.device).to(torch.int32)
    table = torch.zeros((len(lens), max(need)), dtype=torch.int32, device=gen.device)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = perm[at:at + k]
        at += k
    return table, pool


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _logits(gen, rows, vocab, dtype):
    """Logits with a few likely tokens a row over a broad background."""
    x = torch.randn((rows, vocab), generator=gen, device="cuda") * 2.0
    hot = torch.randint(0, vocab, (rows, 16), generator=gen, device="cuda")
    x.scatter_add_(1, hot, torch.rand((rows, 16), generator=gen, device="cuda") * 12.0)
    return x.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    st = dict(case=case)
    if case["op"] == "tree_attn":
        B, T = case["batch"], case["nodes"]
        nodes, lens = _nodes_of(case), _lens_of(case)
        table, pool = _pages(gen, lens, case["page"])
        shape = (pool, case["page"], case["hkv"], case["dim"])
        st["k"] = torch.randn(shape, generator=gen, device="cuda", dtype=dt)
        st["v"] = torch.randn(shape, generator=gen, device="cuda", dtype=dt)
        st["q"] = torch.randn((B * T, case["hq"], case["dim"]), generator=gen, device="cuda", dtype=dt)
        st["table"], st["lens"], st["nodes"] = table, _ints(lens), _ints(nodes)
        st["parents"] = _trees(gen, nodes, T)
        st["lens_host"], st["nodes_host"] = lens, nodes
        # padding rows of the outputs are not written: they keep these zeros
        st["out"] = torch.zeros_like(st["q"])
        st["lse"] = torch.zeros((B * T, case["hq"]), device="cuda")
    elif case["op"] == "token_logprobs":
        R, V, m = case["rows"], case["vocab"], case["given"]
        st["logits"] = _logits(gen, R, V, dt)
        if case["masked"]:
            # tokens that a grammar rules out
            out = torch.rand((R, V), generator=gen, device="cuda") < 0.2
            st["logits"].masked_fill_(out, -math.inf)
        st["tokens"] = torch.randint(0, V, (R, m), generator=gen, device="cuda", dtype=torch.int32) if m else None
    elif case["op"] == "tree_accept":
        B, T, V = case["batch"], case["nodes"], case["vocab"]
        nodes = _nodes_of(case)
        st["logits"] = _logits(gen, B * T, V, dt).view(B, T, V)
        st["parents"], st["nodes"] = _trees(gen, nodes, T), _ints(nodes)
        # a node holds its parent's most likely token seven times in ten (siblings may agree)
        best = st["logits"].float().argmax(dim=2)
        good = best.gather(1, st["parents"].long().clamp(min=0))
        other = torch.randint(0, V, (B, T), generator=gen, device="cuda")
        pick = torch.rand((B, T), generator=gen, device="cuda") < 0.7
        st["tokens"] = torch.where(pick, good, other).to(torch.int32)
    else:
        B, T = case["batch"], case["nodes"]
        nodes, lens, acc = _nodes_of(case), _lens_of(case), _accepted_of(case)
        table, pool = _pages(gen, lens, case["page"])
        shape = (case["layers"], pool, case["page"], case["hkv"], case["dim"])
        st["k"] = torch.randn(shape, generator=gen, device="cuda", dtype=dt)
        st["v"] = torch.randn(shape, generator=gen, device="cuda", dtype=dt)
        st["table"], st["lens"], st["nodes"] = table, _ints(lens), _ints(nodes)
        # accepted nodes among the later ones, as of a tree numbered level by level
        path = torch.full((B, T), -1, dtype=torch.int32, device="cuda")
        path[:, 0] = 0
        for b in range(B):
            a = acc[b] = min(acc[b], max(0, nodes[b] - 1 - acc[b]))
            late = torch.randperm(nodes[b] - 1 - a, generator=gen, device="cuda")[:a] + a + 1
            path[b, 1:1 + a] = late.sort().values.to(torch.int32)
        st["path"], st["accepted"] = path, _ints(acc)
    if own:
        import speculative_decoding_block_dflash_gb300 as dfl

        st["lib"] = dfl
    return st


# --------------------------------------------------------------------------------- plain forms


def _ancestors(parents):
    """[B, T, T] truth values: column j is row i's node itself or one of its ancestors."""
    B, T = parents.shape
    up = torch.zeros((B, T, T), device=parents.device)
    up.scatter_(2, parents.long().clamp(min=0)[:, :, None], (parents >= 0).float()[:, :, None])
    reach = up + torch.eye(T, device=parents.device)
    steps = 1
    while steps < T:
        reach = (torch.bmm(reach, reach) > 0).float()
        steps *= 2
    return reach > 0


def _plain_attn(st):
    case = st["case"]
    T, hq, hkv, d, W = case["nodes"], case["hq"], case["hkv"], case["dim"], case["window"]
    G = hq // hkv
    seen = _ancestors(st["parents"])
    depth = seen.sum(dim=2) - 1
    out = torch.zeros((case["batch"], T, hq, d), device="cuda")
    lse = torch.zeros((case["batch"], T, hq), device="cuda")
    q = st["q"].view(case["batch"], T, hkv, G, d)
    for b, (n, length) in enumerate(zip(st["nodes_host"], st["lens_host"])):
        ctx = length - n
        first = max(0, ctx - W + 1) if W else 0  # no node sees a key before this one
        p0 = first // case["page"]
        rows = st["table"][b, p0:(length + case["page"] - 1) // case["page"]].long()
        lo, hi = p0 * case["page"], length
        k = st["k"][rows].view(-1, hkv, d)[:hi - lo].float()
        v = st["v"][rows].view(-1, hkv, d)[:hi - lo].float()
        qb = q[b, :n].float().permute(1, 0, 2, 3).reshape(hkv, n * G, d)
        s = torch.bmm(qb, k.permute(1, 2, 0)) / math.sqrt(d)  # [hkv, n*G, keys]
        pos = torch.arange(lo, hi, device="cuda")
        vis = torch.ones((n, hi - lo), dtype=torch.bool, device="cuda")
        vis[:, ctx - lo:] = seen[b, :n, :n]
        if W:
            # a key of the context sits at its own position, a node at ctx + its depth
            at = torch.cat([pos[:ctx - lo], ctx + depth[b, :n]])
            vis &= at[None, :] > (ctx + depth[b, :n])[:, None] - W
        s = s.view(hkv, n, G, hi - lo).masked_fill(~vis[None, :, None, :], -math.inf)
        m = s.amax(dim=3, keepdim=True)
        e = (s - m).exp()
        z = e.sum(dim=3, keepdim=True)
        o = torch.bmm((e / z).view(hkv, n * G, hi - lo), v.permute(1, 0, 2))
        out[b, :n] = o.view(hkv, n, G, d).permute(1, 0, 2, 3).reshape(n, hq, d)
        lse[b, :n] = (m + z.log())[..., 0].permute(1, 0, 2).reshape(n, hq)
    return out.view(-1, hq, d).to(st["q"].dtype), lse.view(-1, hq)


def _order_keys(x):
    """int64 keys of float32 values: larger value first, then the lower index (all distinct)."""
    bits = (x + 0.0).view(torch.int32)
    bits = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    return (bits << 32) | (0xFFFFFFFF - torch.arange(x.shape[-1], device=x.device))


def _plain_logprobs(st):
    case = st["case"]
    raw = st["logits"].float()
    x = raw / case["temperature"]
    m = x.amax(dim=1, keepdim=True)
    z = (x - m).exp().sum(dim=1, keepdim=True)
    log_z = m + z.log()
    logp = x - log_z
    entropy = -(logp.exp() * logp.masked_fill(logp == -math.inf, 0.0)).sum(dim=1)
    given = logp.gather(1, st["tokens"].long()) if case["given"] else None
    top = top_logp = None
    if case["top"]:
        keys = _order_keys(raw).topk(case["top"], dim=1, sorted=True).values
        idx = 0xFFFFFFFF - (keys & 0xFFFFFFFF)
        top, top_logp = idx.to(torch.int32), logp.gather(1, idx)
    return dict(given=given, entropy=entropy, log_z=log_z[:, 0], top=top, top_logp=top_logp)


def _plain_accept(st):
    case = st["case"]
    B, T = case["batch"], case["nodes"]
    best = (0xFFFFFFFF - (_order_keys(st["logits"].float()).amax(dim=2) & 0xFFFFFFFF))
    i = torch.arange(T, device="cuda")
    real = i[None, :] < st["nodes"][:, None]
    best = torch.where(real, best, -torch.ones_like(best))
    par = st["parents"].long()
    right = (st["tokens"].long() == best.gather(1, par.clamp(min=0))) & (par >= 0) & real
    # of the siblings that hold the target's token the first goes on
    twin = (par[:, :, None] == par[:, None, :]) & right[:, None, :] & (i[None, :] < i[:, None])[None]
    right &= ~twin.any(dim=2)
    right[:, 0] = True
    on = (_ancestors(st["parents"]) <= right[:, None, :]).all(dim=2) & real
    path = torch.where(on, i[None, :].expand(B, T), torch.full_like(par, T)).sort(dim=1).values
    length = on.sum(dim=1) - 1
    nxt = best.gather(1, path.gather(1, length[:, None]))[:, 0]
    path = torch.where(path == T, -torch.ones_like(path), path)
    return length.to(torch.int32), path.to(torch.int32), nxt.to(torch.int32), best.to(torch.int32)


def _plain_commit(st):
    page = st["case"]["page"]
    ctx = (st["lens"] - st["nodes"]).long()[:, None]
    T = st["path"].shape[1]
    s = torch.arange(T, device="cuda")[None, :]
    move = (s >= 1) & (s <= st["accepted"][:, None])
    src, dst = ctx + st["path"].long().clamp(min=0), (ctx + s).expand_as(move)
    b = torch.arange(src.shape[0], device="cuda")[:, None].expand_as(move)[move]
    src, dst = src[move], dst[move]
    sp, dp = st["table"][b, src // page].long(), st["table"][b, dst // page].long()
    for cache in (st["k"], st["v"]):
        cache[:, dp, dst % page] = cache[:, sp, src % page]
    return st["k"], st["v"], (ctx[:, 0] + 1 + st["accepted"]).to(torch.int32)


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"tree_attn": _plain_attn, "token_logprobs": _plain_logprobs, "tree_accept": _plain_accept,
                "tree_commit": _plain_commit}[op](state)
    dfl = state["lib"]
    case = state["case"]
    if op == "tree_attn":
        return dfl.tree_attn(state["q"], state["k"], state["v"], state["table"], state["lens"], state["parents"],
                             num_nodes=state["nodes"], window=case["window"], max_seq_len=case["hi"],
                             out=state["out"], lse=state["lse"])
    if op == "token_logprobs":
        given, entropy, log_z, top, top_logp = dfl.token_logprobs(state["logits"], state["tokens"],
                                                                  top_k=case["top"],
                                                                  temperature=case["temperature"])
        return dict(given=given, entropy=entropy, log_z=log_z, top=top, top_logp=top_logp)
    if op == "tree_accept":
        return dfl.tree_accept(state["logits"], state["tokens"], state["parents"], num_nodes=state["nodes"])
    new_lens = dfl.tree_commit(state["k"], state["v"], state["table"], state["lens"], state["path"],
                               state["accepted"], num_nodes=state["nodes"])
    return state["k"], state["v"], new_lens


# ------------------------------------------------------------------------------- in 64 bits


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "tree_attn":
        return _exact_attn(case, st)
    if case["op"] == "token_logprobs":
        return _exact_logprobs(case, st)
    if case["op"] == "tree_accept":
        return _exact_accept(case, st)
    return _exact_commit(case, st)


def _walk_up(parents, n):
    """Each node's ancestors and itself, by walking from node to node on the host."""
    chains = []
    for i in range(n):
        chain, j = [], i
        while j >= 0:
            chain.append(j)
            j = parents[j]
        chains.append(chain)
    return chains


def _exact_attn(case, st):
    B, T, hq, hkv, d, P, W = (case[x] for x in ("batch", "nodes", "hq", "hkv", "dim", "page", "window"))
    out = torch.zeros((B, T, hq, d), device="cuda", dtype=torch.float64)
    lse = torch.zeros((B, T, hq), device="cuda", dtype=torch.float64)
    q = st["q"].view(B, T, hq, d)
    for b in range(B):
        n, length = st["nodes_host"][b], st["lens_host"][b]
        ctx = length - n
        chains = _walk_up(st["parents"][b].tolist(), n)
        start = max(0, ctx - W) // P * P if W else 0
        j = torch.arange(start, length, device="cuda")
        phys = st["table"][b].long()[j // P]
        bias = torch.zeros((n, length - start), dtype=torch.float64)
        bias[:, ctx - start:] = -math.inf
        for i, chain in enumerate(chains):
            if W:
                bias[i, :max(0, min(ctx, ctx + len(chain) - 1 - W + 1) - start)] = -math.inf
            for up in chain[:W] if W else chain:
                bias[i, ctx - start + up] = 0.0
        bias = bias.cuda()
        for g in range(hkv):
            k = st["k"][phys, j % P, g].double()
            v = st["v"][phys, j % P, g].double()
            for h in range(g * hq // hkv, (g + 1) * hq // hkv):
                s = q[b, :n, h].double() @ k.T / math.sqrt(d) + bias
                lse[b, :n, h] = torch.logsumexp(s, dim=1)
                out[b, :n, h] = torch.softmax(s, dim=1) @ v
    return out.view(B * T, hq, d), lse.view(B * T, hq)


def _exact_logprobs(case, st):
    parts = []
    for r in range(0, case["rows"], 64):
        x = st["logits"][r:r + 64].double()
        logp = torch.log_softmax(x / case["temperature"], dim=1)
        p = logp.exp()
        row = [torch.gather(logp, 1, st["tokens"][r:r + 64].long()) if case["given"] else None,
               -torch.where(p > 0, p * logp, 0.0).sum(dim=1),
               torch.logsumexp(x / case["temperature"], dim=1)]
        if case["top"]:
            idx = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :case["top"]]
            row += [idx.to(torch.int32), torch.gather(logp, 1, idx)]
        else:
            row += [None, None]
        parts.append(row)
    cat = [None if c[0] is None else torch.cat(c) for c in zip(*parts)]
    return dict(zip(("given", "entropy", "log_z", "top", "top_logp"), cat))


def _exact_accept(case, st):
    B, T = case["batch"], case["nodes"]
    best = torch.full((B, T), -1, dtype=torch.int64)
    for b, n in enumerate(_nodes_of(case)):
        x = st["logits"][b, :n].double()
        at = torch.arange(case["vocab"], device="cuda")
        best[b, :n] = torch.where(x == x.amax(dim=1, keepdim=True), at, case["vocab"]).amin(dim=1).cpu()
    length, path, nxt = [], [], []
    for b, n in enumerate(_nodes_of(case)):
        parents, tokens = st["parents"][b].tolist(), st["tokens"][b].tolist()
        here = [0]
        while True:
            fits = [i for i in range(1, n) if parents[i] == here[-1] and tokens[i] == int(best[b, here[-1]])]
            if not fits:
                break
            here.append(fits[0])
        length.append(len(here) - 1)
        path.append(here + [-1] * (T - len(here)))
        nxt.append(int(best[b, here[-1]]))
    return _ints(length), _ints(path), _ints(nxt), best.to(torch.int32).cuda()


def _exact_commit(case, st):
    # what moves keeps its value: an element for element copy on the host's indices
    P = case["page"]
    table, lens, nodes = st["table"].tolist(), st["lens"].tolist(), st["nodes"].tolist()
    path, acc = st["path"].tolist(), st["accepted"].tolist()
    k, v = st["k"].clone(), st["v"].clone()
    for b in range(case["batch"]):
        base = lens[b] - nodes[b]
        for s in range(1, acc[b] + 1):
            src, dst = base + path[b][s], base + s
            for new, old in ((k, st["k"]), (v, st["v"])):
                new[:, table[b][dst // P], dst % P] = old[:, table[b][src // P], src % P]
    return k, v, _ints([lens[b] - nodes[b] + 1 + acc[b] for b in range(case["batch"])])
