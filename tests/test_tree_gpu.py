"""GPU checks of the operators on drafted trees against oracle/tree.py in float64.

Bounds, from the arithmetic (u = half a step of a type: bf16 2^-8, fp32 2^-24), with p the exact
probabilities, A = sum_j p_j |v_j| and S = the largest scale * sum_d |q_d k_d| of a row:
  * a score's fp32 sum of D products is off by at most (D + 2) u32 S, which changes every p by a
    factor within exp(+-2 ds), ds = (D + 2) u32 S + 2^-20: the exponential's own error (2 ulp, 2^-22),
    its argument's rounding (|argument| <= 2^7 or so, 2^-17 relative to 1 ulp of 2^-24 each: 2^-17 covers
    arguments whose p counts) and the joins' weights lie inside 2^-17, taken for ds' constant below;
  * on the tensor cores P is rounded to bf16 before the product with V, its sum is not: u16 A;
  * sums over n keys in fp32: n u32 A (and n u32 for the lse);
  * the output's own rounding: u |o|.
"""
import threading

import numpy as np
import pytest
import torch

import speculative_decoding_block_dflash_gb300 as dfl
from oracle import tree as ot
from speculative_decoding_block_dflash_gb300 import _binding as B
from speculative_decoding_block_dflash_gb300 import build as build_mod

pytestmark = pytest.mark.gpu

U16, U32 = 2.0 ** -8, 2.0 ** -24
GUARD = 1024
KERNELS16 = ("simt", "tc")


@pytest.fixture(scope="module", autouse=True)
def _built():
    build_mod.build()
    dfl.load_library()


def random_parents(rng, n, kind="tree"):
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "star":
        return [-1] + [0] * (n - 1)
    if kind == "forest":
        return [-1 if i % 4 == 0 else int(rng.integers(0, i)) for i in range(n)]
    return [-1] + [int(rng.integers(max(0, i - 6), i)) for i in range(1, n)]


class Tree:
    """Inputs of one call; what nobody may use (cache slots behind the keys and before the window, free
    pages, padding rows of q) holds NaN."""

    def __init__(self, nodes, lens, T=None, hq=4, hkv=2, d=64, page=16, window=0, dtype=torch.bfloat16, kind="tree",
                 seed=0, layout="nhd", poison=True):
        rng = np.random.default_rng(seed)
        self.nodes, self.lens, self.window, self.page, self.d = nodes, lens, window, page, d
        self.hq, self.hkv = hq, hkv
        nb = len(nodes)
        T = self.T = T or max(nodes)
        self.parents = np.full((nb, T), -1, dtype=np.int32)
        for b, n in enumerate(nodes):
            self.parents[b, :n] = random_parents(rng, n, kind)
        need = [-(-L // page) for L in lens]
        pool = sum(need) + 5
        perm = rng.permutation(pool)
        self.table = np.full((nb, max(max(need), 1) + 1), -7, dtype=np.int32)  # entries past the keys are never read
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = perm[at:at + k]
            at += k
        g = torch.Generator(device="cuda").manual_seed(seed)
        shape = {"nhd": (pool, page, hkv, d), "hnd": (pool, hkv, page, d), "padded": (pool, page, hkv + 1, d + 16)}[layout]
        fill = float("nan") if poison else 0.0
        caches = []
        for _ in range(2):
            c = torch.full(shape, fill, dtype=dtype, device="cuda")
            c = {"nhd": c, "hnd": c.permute(0, 2, 1, 3), "padded": c[:, :, :hkv, 8:8 + d] if layout == "padded" else c}[layout]
            for b, (n, L) in enumerate(zip(nodes, lens)):
                ctx = L - n
                first = max(0, ctx - window + 1) if window else 0
                if n == 0 or L <= first:
                    continue
                j = torch.arange(first, L)
                pg, sl = torch.from_numpy(self.table[b])[j // page].long().cuda(), (j % page).cuda()
                c[pg, sl] = torch.randn((L - first, hkv, d), generator=g, device="cuda").to(dtype)
            caches.append(c)
        self.k, self.v = caches
        self.q = torch.full((nb * T, hq, d), fill, dtype=dtype, device="cuda")
        for b, n in enumerate(nodes):
            self.q[b * T:b * T + n] = torch.randn((n, hq, d), generator=g, device="cuda").to(dtype)
        self.scale = float(np.float32(d ** -0.5))

    def call(self, kernel="auto", **kw):
        nb, T = self.parents.shape
        n = nb * T * self.hq * self.d
        buf = torch.full((n + 2 * GUARD,), 3.0e38, dtype=self.q.dtype, device="cuda")
        lbuf = torch.full((nb * T * self.hq + 2 * GUARD,), 3.0e38, device="cuda")
        out, lse = buf[GUARD:GUARD + n].view(nb * T, self.hq, self.d), lbuf[GUARD:-GUARD].view(nb * T, self.hq)
        args = dict(num_nodes=torch.tensor(self.nodes, dtype=torch.int32, device="cuda"), window=self.window,
                    scale=self.scale, out=out, lse=lse, kernel=kernel)
        args.update(kw)
        dims = dfl.make_dims(self.q, self.k, torch.from_numpy(self.table), T)
        self.ws = torch.zeros(dfl.tree_attn_workspace_bytes(dims, T), dtype=torch.uint8, device="cuda")
        args.setdefault("workspace", self.ws)
        dfl.tree_attn(self.q, self.k, self.v, torch.from_numpy(self.table).cuda(),
                      torch.tensor(self.lens, dtype=torch.int32, device="cuda"),
                      torch.from_numpy(self.parents).cuda(), **args)
        torch.cuda.synchronize()
        for x in (buf, lbuf):
            assert (x[:GUARD] == x[0]).all() and (x[-GUARD:] == x[0]).all(), "wrote outside the output"
        return out, lse

    def request(self, b):
        """(keys, values) [L, Hkv, D] of request b in float64, zeros where no node sees."""
        n, L = self.nodes[b], self.lens[b]
        j = np.arange(L)
        pg = self.table[b][j // self.page]
        out = []
        for c in (self.k, self.v):
            x = c[torch.from_numpy(pg).long().cuda(), torch.from_numpy(j % self.page).cuda()].double().cpu().numpy()
            out.append(np.nan_to_num(x))
        return out

    def check(self, out, lse, rounded_sum=False):
        nb, T = self.parents.shape
        bf16 = self.q.dtype == torch.bfloat16
        fresh = torch.full((1,), 3.0e38, dtype=self.q.dtype).double().item()
        for b in range(nb):
            n = self.nodes[b]
            rows = slice(b * T, b * T + n)
            pad = slice(b * T + n, (b + 1) * T)
            assert (out[pad].double() == fresh).all() and (lse[pad] == np.float32(3.0e38)).all(), "padding written"
            if n == 0:
                continue
            keys, values = self.request(b)
            o, l, spread, size = ot.tree_attn(self.q[rows].double().cpu().numpy(), keys, values, self.parents[b],
                                              self.lens[b] - n, self.window, self.scale)
            ds = (self.d + 2) * U32 * size + 2.0 ** -17
            tol = (U16 if bf16 else U32) * np.abs(o) + (2 * ds[..., None] + self.lens[b] * U32) * spread
            if bf16:
                tol = tol + U16 * spread
            if rounded_sum:  # the row sum is of bf16 probabilities: off by up to u16 of itself
                tol = tol + 1.01 * U16 * np.abs(o)
            err = np.abs(out[rows].double().cpu().numpy() - o)
            assert np.all(err <= tol), f"request {b}: off by {np.max(err / tol):.3g} bounds"
            lerr = np.abs(lse[rows].double().cpu().numpy() - l)
            ltol = ds + self.lens[b] * U32 + 2.0 ** -20 * (1 + np.abs(l)) + (1.01 * U16 if rounded_sum else 0)
            assert np.all(lerr <= ltol), f"request {b}: lse off by {np.max(lerr / ltol):.3g} bounds"

    def error(self):
        return dfl.read_error(self.ws)


BOTH = [("simt", torch.float32), ("simt", torch.bfloat16), ("tc", torch.bfloat16)]




@pytest.mark.parametrize("kernel,dtype", BOTH)
@pytest.mark.parametrize("d", [16, 64, 80, 96, 128, 192, 256, 320, 512])
def test_head_dims(kernel, dtype, d):
    t = Tree([7, 5], [150, 300], d=d, dtype=dtype, seed=d)
    t.check(*t.call(kernel))
    assert t.error() == 0


@pytest.mark.parametrize("kernel,dtype", BOTH)
@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (7, 1), (8, 1), (12, 2), (20, 4), (32, 8), (96, 2), (160, 1), (300, 1)])
def test_head_layouts(kernel, dtype, hq, hkv):
    t = Tree([9, 4, 1], [140, 20, 257], hq=hq, hkv=hkv, dtype=dtype, seed=hq)
    t.check(*t.call(kernel))


@pytest.mark.parametrize("kernel,dtype", BOTH)
@pytest.mark.parametrize("T,hq,hkv,d", [(1, 8, 2, 128), (2, 4, 4, 64), (33, 8, 2, 128), (64, 8, 1, 128), (65, 8, 2, 256),
                                        (128, 4, 1, 64), (200, 6, 2, 128), (256, 2, 1, 512), (256, 4, 2, 128),
                                        (90, 8, 2, 64), (95, 4, 1, 48), (157, 8, 2, 32)])
def test_tree_sizes(kernel, dtype, T, hq, hkv, d):
    nodes = [T, max(1, T // 2)]
    t = Tree(nodes, [nodes[0] + 200, nodes[1] + 1], T=T, hq=hq, hkv=hkv, d=d, dtype=dtype, seed=T)
    t.check(*t.call(kernel))


@pytest.mark.parametrize("kernel,dtype", BOTH)
@pytest.mark.parametrize("page", [8, 16, 24, 32, 48, 64, 128, 200, 256])
def test_page_sizes(kernel, dtype, page):
    t = Tree([6, 6, 3], [page * 2, page * 3 + 5, 700], page=page, dtype=dtype, seed=page)
    t.check(*t.call(kernel))
    assert t.error() == 0


@pytest.mark.parametrize("kernel,dtype", BOTH)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_lengths_around_tiles(kernel, dtype, d):
    lens = [5, 6, 63, 64, 65, 127, 128, 129, 130, 255, 256, 257, 384, 1000]
    nodes = [5, 1, 5, 3, 5, 4, 5, 5, 1, 5, 2, 5, 5, 3]
    t = Tree(nodes, lens, T=5, d=d, dtype=dtype, seed=11)
    t.check(*t.call(kernel))


@pytest.mark.parametrize("kernel,dtype", BOTH)
@pytest.mark.parametrize("window", [1, 2, 5, 40, 128, 300, 2 ** 31 - 1])
@pytest.mark.parametrize("kind", ["tree", "chain"])
def test_windows(kernel, dtype, window, kind):
    t = Tree([20, 12, 1], [500, 12, 290], window=window, kind=kind, dtype=dtype, d=128, seed=window % 1000)
    t.check(*t.call(kernel))
    assert t.error() == 0


@pytest.mark.parametrize("kernel,dtype", BOTH)
@pytest.mark.parametrize("kind", ["chain", "star", "forest"])
@pytest.mark.parametrize("d", [128, 256])
def test_tree_shapes(kernel, dtype, kind, d):
    t = Tree([40, 13], [41, 200], kind=kind, dtype=dtype, d=d, seed=5)
    t.check(*t.call(kernel))


@pytest.mark.parametrize("kernel,dtype", BOTH)
@pytest.mark.parametrize("layout", ["hnd", "padded"])
def test_cache_strides(kernel, dtype, layout):
    t = Tree([7, 9], [150, 333], layout=layout, dtype=dtype, d=128, seed=21)
    t.check(*t.call(kernel))


@pytest.mark.parametrize("kernel,dtype", BOTH)
def test_ragged_batch_of_many_requests_some_empty(kernel, dtype):
    rng = np.random.default_rng(4)
    nodes = [int(x) for x in rng.integers(0, 17, 70)]
    nodes[0] = nodes[33] = nodes[69] = 0
    lens = [n + int(rng.integers(0, 400)) for n in nodes]
    t = Tree(nodes, lens, T=16, dtype=dtype, seed=6)
    t.check(*t.call(kernel))
    assert t.error() == 0


@pytest.mark.parametrize("kernel,dtype", BOTH)
def test_all_requests_empty(kernel, dtype):
    t = Tree([0, 0], [0, 55], T=4, dtype=dtype)
    t.check(*t.call(kernel))


@pytest.mark.parametrize("kernel,dtype", BOTH)
@pytest.mark.parametrize("d,hq,hkv", [(128, 8, 2), (512, 16, 2), (64, 32, 4)])
def test_long_contexts_in_many_ranges(kernel, dtype, d, hq, hkv):
    t = Tree([10, 3], [6000, 9001], hq=hq, hkv=hkv, d=d, dtype=dtype, seed=8)
    t.check(*t.call(kernel))


@pytest.mark.parametrize("kernel,dtype", BOTH)
@pytest.mark.parametrize("d", [48, 128, 256, 512])
@pytest.mark.parametrize("nodes,hq,hkv", [(1, 1, 1), (3, 8, 2)])
def test_few_rows_in_many_ranges(kernel, dtype, d, nodes, hq, hkv):
    # up to a partial per CTA of the GPU for each row
    t = Tree([nodes], [31003], hq=hq, hkv=hkv, d=d, dtype=dtype, seed=55)
    t.check(*t.call(kernel))


@pytest.mark.parametrize("kernel,dtype", BOTH)
def test_scores_far_apart(kernel, dtype):
    # scores of some hundreds: later tiles raise the maximum and rescale the accumulators many times
    t = Tree([16, 16], [900, 1500], hq=8, hkv=2, d=128, dtype=dtype, seed=9)
    ramp = torch.linspace(0.2, 6.0, t.k.shape[0], device="cuda").to(dtype)
    t.k.mul_(ramp[:, None, None, None])
    t.q.mul_(4.0)
    t.check(*t.call(kernel))


def test_bad_lengths_and_sizes_give_zeros_and_an_error():
    for kernel, dtype in BOTH:
        t = Tree([5, 5, 5, 5], [60, 70, 80, 90], T=6, dtype=dtype, poison=False)
        t.lens = [4, 70, 10 ** 6, -3]
        out, lse = t.call(kernel)
        assert t.error() == B.DEVERR_SEQ_LEN
        for b in (0, 2, 3):
            assert (out[b * 6:b * 6 + 6] == 0).all() and (lse[b * 6:b * 6 + 6] == -np.inf).all()
        assert torch.isfinite(out[6:11].float()).all()
        t.lens, t.nodes = [60, 70, 80, 90], [5, 7, -1, 5]
        out, lse = t.call(kernel)
        assert t.error() == B.DEVERR_TREE
        for b in (1, 2):
            assert (out[b * 6:b * 6 + 6] == 0).all() and (lse[b * 6:b * 6 + 6] == -np.inf).all()


@pytest.mark.parametrize("kernel,dtype", BOTH)
def test_bad_parents_count_as_roots(kernel, dtype):
    t = Tree([8, 8], [100, 150], dtype=dtype, seed=3)
    good = t.parents.copy()
    t.parents[0, 3], t.parents[1, 5], t.parents[1, 6] = 3, 100, -9
    out, lse = t.call(kernel)
    assert t.error() == B.DEVERR_TREE
    good[0, 3] = good[1, 5] = good[1, 6] = -1
    t.parents = good
    t.check(out, lse)


@pytest.mark.parametrize("kernel,dtype", BOTH)
def test_bad_pages_read_as_zero_keys(kernel, dtype):
    t = Tree([4, 4], [100, 200], dtype=dtype, seed=2)
    page_of = t.table.copy()
    t.table[1, 3], t.table[1, 7] = -1, t.k.shape[0]
    out, lse = t.call(kernel)
    assert t.error() == B.DEVERR_PAGE_ID
    t.table = page_of
    for c in (t.k, t.v):
        c[int(page_of[1, 3])] = 0
        c[int(page_of[1, 7])] = 0
    t.check(out, lse)


@pytest.mark.parametrize("kernel,dtype", BOTH)
def test_no_num_nodes_no_lse_and_a_bound_on_the_lengths(kernel, dtype):
    t = Tree([6, 6], [100, 222], dtype=dtype, seed=12)
    out, lse = t.call(kernel, num_nodes=None, max_seq_len=222)
    t.check(out, lse)
    again, none = dfl.tree_attn(t.q, t.k, t.v, torch.from_numpy(t.table).cuda(),
                                torch.tensor(t.lens, dtype=torch.int32, device="cuda"),
                                torch.from_numpy(t.parents).cuda(), scale=t.scale, kernel=kernel, want_lse=False)
    assert none is None and dfl.tree_attn_error() == 0
    torch.testing.assert_close(again, out, rtol=0, atol=0)


@pytest.mark.parametrize("kernel,dtype", BOTH)
def test_chain_agrees_with_the_causal_block(kernel, dtype):
    t = Tree([9, 9], [300, 431], hq=8, hkv=2, d=128, kind="chain", dtype=dtype, seed=14)
    out, lse = t.call(kernel)
    bo, bl = dfl.block_attn(t.q, t.k, t.v, torch.from_numpy(t.table).clamp(min=0).cuda(),
                            torch.tensor(t.lens, dtype=torch.int32, device="cuda"), 9, causal=True, scale=t.scale)
    torch.cuda.synchronize()
    # each is within the bounds of the exact result (the block kernel's row sums are of rounded probabilities)
    t.check(bo, bl, rounded_sum=dtype == torch.bfloat16)
    t.check(out, lse)


@pytest.mark.parametrize("kernel,dtype", BOTH)
def test_same_bits_twice_on_streams_and_in_graphs(kernel, dtype):
    a = Tree([30, 9], [900, 2000], hq=8, hkv=2, d=128, dtype=dtype, seed=15)
    c = Tree([8, 16], [1500, 300], hq=8, hkv=2, d=128, dtype=dtype, seed=16)

    def go(t, stream=None, out=None, lse=None):
        return dfl.tree_attn(t.q, t.k, t.v, t.dev[0], t.dev[1], t.dev[2], num_nodes=t.dev[3], scale=t.scale,
                             kernel=kernel, stream=stream, out=out, lse=lse)

    for t in (a, c):
        t.dev = (torch.from_numpy(t.table).cuda(), torch.tensor(t.lens, dtype=torch.int32, device="cuda"),
                 torch.from_numpy(t.parents).cuda(), torch.tensor(t.nodes, dtype=torch.int32, device="cuda"))
    want = [go(a), go(c)]
    torch.cuda.synchronize()
    # two streams at once, each with its own workspace
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        got = [go(a, s1), go(c, s2.cuda_stream)]
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            torch.testing.assert_close(w, g, rtol=0, atol=0, equal_nan=True)
    # two graphs replayed on two streams
    outs, graphs = [], []
    for t in (a, c):
        o, l = torch.zeros_like(t.q), torch.zeros(t.q.shape[:2], device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            go(t, out=o, lse=l)
        outs.append((o, l))
        graphs.append(g)
    for _ in range(5):
        for o, l in outs:
            o.zero_()
            l.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, (s1, s2)):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for w, g in zip(want, outs):
            torch.testing.assert_close(w, g, rtol=0, atol=0, equal_nan=True)


@pytest.mark.parametrize("kernel,dtype", BOTH)
def test_threads_that_share_a_stream(kernel, dtype):
    # two threads' calls on one stream, whose workspace they share
    cases = [Tree([9, 4], [900, 1300], hq=8, hkv=2, d=128, dtype=dtype, seed=56),
             Tree([3], [2500], hq=8, hkv=2, d=64, dtype=dtype, seed=57)]
    calls = []
    for t in cases:
        args = (torch.from_numpy(t.table).cuda(), torch.tensor(t.lens, dtype=torch.int32, device="cuda"),
                torch.from_numpy(t.parents).cuda(), torch.tensor(t.nodes, dtype=torch.int32, device="cuda"))
        calls.append(lambda t=t, a=args: dfl.tree_attn(t.q, t.k, t.v, a[0], a[1], a[2], num_nodes=a[3], kernel=kernel))
    want = [c() for c in calls]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        for _ in range(100):
            got = [calls[i]() for _ in range(4)]
            bad.extend(i for g in got if not (torch.equal(g[0], want[i][0]) and torch.equal(g[1], want[i][1])))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not bad


@pytest.mark.parametrize("kernel", ["tc", "simt"])
def test_inputs_made_just_before(kernel):
    # the attention may set itself up while the work before it still runs: copies, fills and kernels of its own and of
    # another stream that write its inputs, eagerly and captured; and layers back to back that feed each other
    t = Tree([12, 5, 1], [700, 90, 33], hq=16, hkv=4, d=128, page=16, seed=43)
    dev = (torch.from_numpy(t.table).cuda(), torch.tensor(t.lens, dtype=torch.int32, device="cuda"),
           torch.from_numpy(t.parents).cuda(), torch.tensor(t.nodes, dtype=torch.int32, device="cuda"))

    def go(q, k, v, args):
        return dfl.tree_attn(q, k, v, args[0], args[1], args[2], num_nodes=args[3], kernel=kernel)

    ref = go(t.q, t.k, t.v, dev)[0]
    second = go(ref, t.k, t.v, dev)[0]
    torch.cuda.synchronize()
    q, k, v = (torch.zeros_like(x) for x in (t.q, t.k, t.v))
    args = [torch.zeros_like(x) for x in dev]
    big = torch.zeros(64 << 20, device="cuda")
    side = torch.cuda.Stream()

    def work():
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            big.add_(1.0)  # a few hundred microseconds before the inputs are there
            v.copy_(t.v)
            k.zero_()
            k.add_(t.k)
        big.mul_(0.5)
        for x, y in zip(args, dev):
            x.copy_(y)
        q.copy_(t.q)
        here.wait_stream(side)
        first = go(q, k, v, args)[0]
        return first, go(first, k, v, args)[0]

    def wipe():
        for x in [q, k, v] + args:
            x.zero_()
        torch.cuda.synchronize()

    for _ in range(3):
        wipe()
        got = work()
        torch.cuda.synchronize()
        assert torch.equal(got[0], ref) and torch.equal(got[1], second)
    wipe()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = work()
    for _ in range(3):
        wipe()
        for x in got:
            x.fill_(7.0)
        torch.cuda.synchronize()
        g.replay()
        g.replay()  # nothing waits between the two
        torch.cuda.synchronize()
        assert torch.equal(got[0], ref) and torch.equal(got[1], second)


def test_offsets_past_32_bits():
    # a pool of more than 2^31 elements, its pages used from the end
    page, hkv, d = 64, 8, 128
    pool = 2 ** 31 // (page * hkv * d) + 200
    k = torch.zeros((pool, page, hkv, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    t = Tree([9, 4], [1000, 500], hq=16, hkv=hkv, d=d, page=page, seed=17)
    far = torch.arange(pool - t.k.shape[0], pool, device="cuda")
    k[far], v[far] = t.k, t.v
    t.k, t.v = k, v
    t.table = np.where(t.table >= 0, t.table + (pool - far.numel()), -7).astype(np.int32)
    for kernel in KERNELS16:
        t.check(*t.call(kernel))


@pytest.mark.parametrize("T", [8, 24])  # one CTA per query tile, and pairs
def test_a_wait_that_runs_out_is_reported_and_the_workspace_recovers(T):
    # A limit of 1 us: the scores of the first tile (eight stages of keys at head_dim 512, out of DRAM as L2 holds
    # something else) take some 4 us to come, so the kernel gives up by itself, reports it and returns.
    t = Tree([T, T - 3], [6000, 7000], T=T, hq=16, hkv=2, d=512, seed=19)
    torch.empty(256 << 20, dtype=torch.uint8, device="cuda").zero_()
    t.call("tc", wait_limit_us=1)
    ws = t.ws
    assert t.error() & B.DEVERR_TIMEOUT
    out, lse = t.call("tc", workspace=ws)
    t.ws = ws
    assert t.error() == 0
    t.check(out, lse)


def test_wrapper_refusals_on_the_gpu():
    t = Tree([4, 4], [40, 50], d=64, seed=20)
    dev = (torch.from_numpy(t.table).cuda(), torch.tensor(t.lens, dtype=torch.int32, device="cuda"),
           torch.from_numpy(t.parents).cuda())
    for bad in (dict(q=t.q.float()), dict(q=t.q[:, :, ::2]), dict(parents=dev[2].long()), dict(parents=dev[2][:1]),
                dict(lens=dev[1].cpu()), dict(table=dev[0][:, ::2]), dict(out=torch.empty_like(t.q, dtype=torch.float32)),
                dict(lse=torch.empty(3, device="cuda")), dict(num_nodes=torch.zeros(3, dtype=torch.int32, device="cuda")),
                dict(v=t.v[:-1]), dict(workspace=torch.zeros(1 << 20, dtype=torch.uint8))):
        a = dict(q=t.q, k=t.k, v=t.v, table=dev[0], lens=dev[1], parents=dev[2])
        kw = {k: v for k, v in bad.items() if k not in a}
        a.update({k: v for k, v in bad.items() if k in a})
        with pytest.raises((ValueError, TypeError)):
            dfl.tree_attn(a["q"], a["k"], a["v"], a["table"], a["lens"], a["parents"], **kw)
    with pytest.raises(dfl.DflashError):
        dfl.tree_attn(t.q, t.k, t.v, *dev, workspace=torch.zeros(512, dtype=torch.uint8, device="cuda"))
    with pytest.raises(dfl.DflashError):
        dfl.tree_attn(t.q, t.k, t.v, *dev, out=t.q)
    x = torch.zeros((2, 9), device="cuda")
    for kw in (dict(top_k=10), dict(top_k=-1), dict(temperature=0.0), dict(temperature=float("nan"))):
        with pytest.raises(dfl.DflashError):
            dfl.token_logprobs(x, **kw)
    with pytest.raises(ValueError):
        dfl.token_logprobs(x, torch.zeros((2, 3), dtype=torch.int64, device="cuda"))
    with pytest.raises(TypeError):
        dfl.token_logprobs(x.half())


# ------------------------------------------------------------------------- log probabilities


def lp_check(logits, tokens, k, temperature, stats=True, **kw):
    given, ent, z, top, top_lp = dfl.token_logprobs(logits, tokens, top_k=k, temperature=temperature, **kw)
    torch.cuda.synchronize()
    V = logits.shape[-1]
    x = logits.double().cpu().numpy().reshape(-1, V)
    tok = None if tokens is None else tokens.cpu().numpy().reshape(x.shape[0], -1)
    # the kernel divides by the fp32 temperature
    e = ot.token_logprobs(x, tok, k, float(np.float32(temperature)))
    # x - m is one rounding (u32 |x - m|), its quotient another, the exponential 2^-22 and its argument's two
    # roundings relative to |y| <= 30 for terms that count (2^-18 in all); sums of V terms are taken by
    # 256 threads and joined: V / 256 + 40 roundings. ln and the final sums are a few roundings of their size.
    terms = 2.0 ** -18 + (V / 256 + 40) * U32
    live = np.where(np.isfinite(x), x, 0.0) / temperature
    size = np.abs(live).max(axis=1)

    def close(got, want, tol):
        got = got.double().cpu().numpy().reshape(want.shape)
        same = (got == want) | (np.isneginf(got) & np.isneginf(want))
        assert np.all(same | (np.abs(got - want) <= tol)), np.nanmax(np.abs(got - want) / tol)

    close(z, e[2], terms + 8 * U32 * (1 + size))
    # sum p y: |y| up to log(V) + a spread where p counts; 64 bounds |y| of terms above 2^-64 of the sum
    close(ent, e[1], 64 * terms)
    spread = 8 * U32 * (1 + 2 * size)[:, None]
    if tokens is not None:
        close(given, e[0], terms + spread)
    if k:
        assert (top.cpu().numpy().reshape(e[3].shape) == e[3]).all(), "top tokens"
        close(top_lp, e[4], terms + spread)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1, 2, 7, 64, 255, 1000, 4097, 8192, 32001, 100000])
@pytest.mark.parametrize("R", [1, 5])
def test_logprobs_sizes(dtype, V, R):
    g = torch.Generator(device="cuda").manual_seed(V + R)
    logits = (torch.randn((R, V), generator=g, device="cuda") * 4).to(dtype)
    tokens = torch.randint(0, V, (R, 3), generator=g, device="cuda", dtype=torch.int32)
    for k in (0, 1, min(V, 8), min(V, 64)):
        lp_check(logits, tokens, k, 1.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("offset,stride", [(0, 5003), (1, 5003), (3, 5008), (5, 5001)])
def test_logprobs_rows_off_16_byte_boundaries(dtype, offset, stride):
    g = torch.Generator(device="cuda").manual_seed(stride + offset)
    base = torch.full((9 * stride + offset,), float("nan"), device="cuda", dtype=dtype)
    rows = base[offset:offset + 9 * stride].view(9, stride)[:, :5000]
    rows.copy_(torch.randn((9, 5000), generator=g, device="cuda"))
    lp_check(rows, torch.randint(0, 5000, (9, 1), generator=g, device="cuda", dtype=torch.int32), 20, 0.6)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_logprobs_ties_take_the_smaller_id(dtype):
    V = 70000
    x = torch.zeros((5, V), device="cuda")
    x[1] = -0.0
    x[1, 1::2] = 0.0          # -0 and +0 are equal
    x[2, 40000:] = 1.0
    x[3, [69999, 3, 50001, 50000]] = 5.0
    x[4] = torch.arange(V, device="cuda") % 3
    lp_check(x.to(dtype), None, 64, 1.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [20000, 150000])
def test_logprobs_ordered_rows(dtype, V):
    # every element beats the ones before it (and the reverse), the worst for a running bound
    up = torch.linspace(-60, 60, V, device="cuda")
    lp_check(torch.stack([up, up.flip(0)]).to(dtype), None, 64, 1.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_logprobs_masked_tokens_and_rows(dtype):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((6, 30000), generator=g, device="cuda")
    x[0, ::2] = -np.inf
    x[1] = -np.inf
    x[2] = -np.inf
    x[2, 29999] = -3.0
    x[3, :29990] = -np.inf
    x[4] = torch.finfo(dtype).min
    x[5, 1:] = torch.finfo(dtype).min
    tokens = torch.tensor([[0, 1, -1], [5, 6, 7], [29999, 0, -5], [29995, 3, 9], [0, 1, 2], [0, 1, 2]], dtype=torch.int32,
                          device="cuda")
    lp_check(x.to(dtype), tokens, 20, 1.0)


@pytest.mark.parametrize("temperature", [1e-30, 0.01, 0.7, 30.0, 1e30])
def test_logprobs_temperatures(temperature):
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randint(-40, 40, (3, 9000), generator=g, device="cuda").float() / 8
    x[:, 77] = 6.0
    if temperature == 1e-30:
        given, ent, z, top, lp = dfl.token_logprobs(x, top_k=2, temperature=temperature)
        assert (top[:, 0] == 77).all() and (lp[:, 0] == 0).all() and (ent == 0).all() and (lp[:, 1] < -1e28).all()
        return
    lp_check(x, None, 4, temperature)


def test_logprobs_one_likely_token_keeps_its_small_entropy():
    x = torch.zeros((1, 1000), device="cuda")
    x[0, 7] = 25.0
    _, ent, _, _, _ = dfl.token_logprobs(x)
    p = 999 * np.exp(-25.0)
    want = p / (1 + p) * 25 + np.log1p(p)
    assert abs(ent.item() - want) <= 3 * U32 + 1e-5 * want


def test_logprobs_token_ids_and_empty_calls():
    x = torch.randn((2, 50), device="cuda")
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    tokens = torch.tensor([[0, -1], [49, -7]], dtype=torch.int32, device="cuda")
    given, *_ = dfl.token_logprobs(x, tokens, device_error=word)
    assert word.item() == 0 and (given[:, 1] == -np.inf).all() and torch.isfinite(given[:, 0]).all()
    tokens[1, 1] = 50
    given, *_ = dfl.token_logprobs(x, tokens, device_error=word)
    assert word.item() == B.DEVERR_TOKEN_ID and given[1, 1].item() == -np.inf
    given, ent, z, top, lp = dfl.token_logprobs(x[:0], tokens[:0], top_k=3)
    assert given.shape == (0, 2) and ent.shape == (0,) and top.shape == (0, 3)
    given, ent, z, top, lp = dfl.token_logprobs(x, tokens[:, :0], want_entropy=False)
    assert given.shape == (2, 0) and ent is None and top is None
    three = torch.randn((2, 3, 40), device="cuda")
    given, ent, z, top, lp = dfl.token_logprobs(three, top_k=2)
    assert z.shape == (2, 3) and top.shape == (2, 3, 2)
    one = dfl.token_logprobs(three[1, 2])[2]
    assert one.shape == () and one.item() == z[1, 2].item()


def test_logprobs_many_rows_match_torch():
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((3000, 3001), generator=g, device="cuda")
    tok = torch.randint(0, 3001, (3000, 2), generator=g, device="cuda", dtype=torch.int32)
    given, ent, z, top, lp = dfl.token_logprobs(x, tok, top_k=5)
    want = torch.log_softmax(x.double(), 1)
    tol = 2.0 ** -17
    assert ((given - want.gather(1, tok.long())).abs() <= tol).all()
    sv, si = want.sort(dim=1, descending=True, stable=True)
    assert (top == si[:, :5]).all() and ((lp - sv[:, :5]).abs() <= tol).all()
    assert ((ent + (want.exp() * want).sum(1)).abs() <= 32 * tol).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_logprobs_long_slices_of_equal_and_ordered_values(dtype):
    # enough rows for one slice each, of more than 16 steps: every group of equal values is read again
    R, V, k = 700, 70001, 64
    g = torch.Generator(device="cuda").manual_seed(54)
    x = torch.randn((R, V), generator=g, device="cuda").to(dtype)
    x[0::7] = 1.5
    x[1::7] = -torch.inf
    x[2::7] = torch.where(torch.arange(V, device="cuda") % 3 == 1, 2.0, -1.0).to(dtype)
    x[3::7] = torch.arange(V, device="cuda").to(dtype)
    x[4::7] = -torch.arange(V, device="cuda").to(dtype)
    x[5::7, 40000:] = 5.0
    _, _, z, top, lp = dfl.token_logprobs(x, top_k=k)
    assert torch.equal(z[0::7], torch.full_like(z[0::7], 1).fill_(z[0].item()))
    for r in list(range(14)) + [R - 1]:
        sv, si = x[r].double().sort(descending=True, stable=True)
        assert torch.equal(top[r].long(), si[:k]), r
        want = sv[:k] - torch.logsumexp(x[r].double(), 0) if torch.isfinite(sv[0]) else sv[:k]
        # values of up to 70000 less a maximum of their size, exact; ln s to a few roundings of values below 16
        assert ((lp[r].double() - want).nan_to_num(0.0).abs() <= 2.0 ** -17).all(), r


def test_logprobs_repeats_streams_and_graphs():
    # several slices a row, other sizes in between, and graphs whose workspaces are their own
    g = torch.Generator(device="cuda").manual_seed(51)
    cases = [(torch.randn((3, 90001), generator=g, device="cuda"), 20), (torch.randn((40, 7000), generator=g,
             device="cuda").bfloat16(), 64)]
    want = [dfl.token_logprobs(x, top_k=k) for x, k in cases]
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [dfl.token_logprobs(x, top_k=k, stream=st) for (x, k), st in zip(cases, s)]
        again = [dfl.token_logprobs(x, top_k=k, stream=s[0]) for x, k in cases]
        torch.cuda.synchronize()
        for w, o, u in zip(want, got, again):
            assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(w[1:], o[1:], u[1:]))
    graphs, outs = [], []
    for x, k in cases:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(dfl.token_logprobs(x, top_k=k))
        graphs.append(gr)
    for _ in range(4):
        for o in outs:
            for x in o[1:]:
                x.fill_(-9)
        torch.cuda.synchronize()
        for gr, st in zip(graphs, s):
            with torch.cuda.stream(st):
                gr.replay()
                gr.replay()
        torch.cuda.synchronize()
        for w, o in zip(want, outs):
            assert all(torch.equal(a, b) for a, b in zip(w[1:], o[1:]))


def test_largest_counts_of_rows_and_requests():
    g = torch.Generator(device="cuda").manual_seed(52)
    n = 65535
    x = torch.randn((n, 7), generator=g, device="cuda")
    _, ent, z, top, lp = dfl.token_logprobs(x, top_k=7)
    want = torch.log_softmax(x.double(), 1)
    sv, si = want.sort(dim=1, descending=True, stable=True)
    assert (top == si).all() and ((lp - sv).abs() <= 2.0 ** -18).all()
    # one-node trees and the largest trees
    for nb, T in ((n, 1), (255, 256)):
        logits = torch.randn((nb, T, 7), generator=g, device="cuda")
        parents = torch.arange(-1, T - 1, dtype=torch.int32, device="cuda").repeat(nb, 1)
        best = logits.argmax(2).int()
        tokens = torch.roll(best, 1, 1)  # every node continues its parent as the target does
        acc, path, nxt, arg = dfl.tree_accept(logits, tokens, parents)
        assert torch.equal(arg, best) and (acc == T - 1).all() and torch.equal(nxt, best[:, -1])
        assert torch.equal(path, torch.arange(T, dtype=torch.int32, device="cuda").repeat(nb, 1))
    # a batch of the largest size: request b attends to its own key and the page all of them share
    k = torch.zeros((2, 8, 1, 16), device="cuda")
    v = torch.randn((2, 8, 1, 16), generator=g, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        kd, vd = k.to(dtype), v.to(dtype)
        q = torch.randn((n, 1, 16), generator=g, device="cuda").to(dtype)
        lens = torch.randint(1, 17, (n,), generator=g, device="cuda", dtype=torch.int32)
        table = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda").repeat(n, 1)
        root = torch.full((n, 1), -1, dtype=torch.int32, device="cuda")
        out, lse = dfl.tree_attn(q, kd, vd, table, lens, root)
        # zero scores: the mean of the values, lse = log(count); P and the products are exact, the mean is rounded once
        mean = vd.double().view(16, 16).cumsum(0)[lens.long() - 1] / lens.double()[:, None]
        eps = torch.finfo(dtype).eps
        spread = vd.double().abs().view(16, 16).cumsum(0)[lens.long() - 1] / lens.double()[:, None]
        # fp32 sums of up to 16 values: 17 roundings of half a step of 2^-23, beside the output's own
        assert ((out[:, 0].double() - mean).abs() <= eps / 2 * mean.abs() + 17 * 2.0 ** -24 * spread).all()
        # the logarithm of at most 16 and its scaling to base e: a few roundings of values below 4
        assert ((lse[:, 0].double() - lens.double().log()).abs() <= 2.0 ** -19).all()


# ------------------------------------------------------------------------------- acceptance


def accept_case(nb, T, V, dtype, seed, nodes=None, kind="tree", agree=0.75):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = torch.randn((nb, T, V), generator=g, device="cuda").to(dtype)
    nodes = nodes or [int(x) for x in rng.integers(max(1, T // 2), T + 1, nb)]
    parents = np.full((nb, T), -1, dtype=np.int32)
    best = logits.double().cpu().numpy().argmax(axis=2)
    tokens = rng.integers(0, V, (nb, T)).astype(np.int32)
    for b, n in enumerate(nodes):
        parents[b, :n] = random_parents(rng, n, kind)
        for i in range(1, n):
            if parents[b, i] >= 0 and rng.random() < agree:
                tokens[b, i] = best[b, parents[b, i]]
    return logits, torch.from_numpy(tokens).cuda(), torch.from_numpy(parents).cuda(), nodes


def accept_check(logits, tokens, parents, nodes, **kw):
    nn = torch.tensor(nodes, dtype=torch.int32, device="cuda")
    got = dfl.tree_accept(logits, tokens, parents, num_nodes=nn, **kw)
    torch.cuda.synchronize()
    live = logits.double().cpu().numpy()
    want = ot.tree_accept(live, tokens.cpu().numpy(), parents.cpu().numpy(), nodes)
    for g, w in zip(got, want):
        np.testing.assert_array_equal(g.cpu().numpy(), w)
    return want


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("nb,T,V", [(1, 1, 1), (1, 1, 9), (2, 9, 1000), (5, 64, 4099), (1, 256, 333), (3, 17, 32001),
                                    (1, 2, 100000)])
def test_accept_matches_oracle(dtype, nb, T, V):
    accept_check(*accept_case(nb, T, V, dtype, seed=V + T))


def test_accept_shapes_of_trees_and_every_length():
    for kind in ("chain", "star", "forest"):
        accept_check(*accept_case(6, 20, 500, torch.float32, seed=4, kind=kind))
    # a chain of 256 that agrees all the way
    case = accept_case(2, 256, 64, torch.float32, seed=5, nodes=[256, 100], kind="chain", agree=1.1)
    want = accept_check(*case)
    assert want[0].tolist() == [255, 99]


def test_accept_empty_trees_padding_rows_and_bad_input():
    logits, tokens, parents, _ = accept_case(5, 8, 300, torch.bfloat16, seed=6, nodes=[8, 8, 8, 8, 8])
    logits[1, 3:] = float("nan")  # padding is not read
    accept_check(logits, tokens, parents, [8, 3, 0, 1, 8])
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    nn = torch.tensor([8, 3, -1, 9, 8], dtype=torch.int32, device="cuda")
    acc, path, nxt, arg = dfl.tree_accept(logits, tokens, parents, num_nodes=nn, device_error=word)
    assert word.item() == B.DEVERR_TREE
    for b in (2, 3):
        assert acc[b] == 0 and nxt[b] == -1 and (path[b] == -1).all() and (arg[b] == -1).all()
    # a parent out of range is a root: its node is on no path
    word.zero_()
    par = parents.clone()
    par[0, 5], par[4, 2] = 5, 77
    acc, path, nxt, arg = dfl.tree_accept(logits, tokens, par, device_error=word)
    fixed = par.clone()
    fixed[0, 5] = fixed[4, 2] = -1
    want = ot.tree_accept(np.nan_to_num(logits.double().cpu().numpy()), tokens.cpu().numpy(), fixed.cpu().numpy(), [8] * 5)
    assert word.item() == B.DEVERR_TREE
    for b in (0, 4):
        assert path[b].tolist() == want[1][b].tolist()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_accept_ties_signed_zeros_and_masks(dtype):
    V = 90000
    x = torch.full((1, 6, V), -5.0, device="cuda")
    x[0, 0, [88888, 12, 50000]] = 2.0
    x[0, 1] = -0.0
    x[0, 1, 7000:] = 0.0
    x[0, 2] = -np.inf
    x[0, 3] = -np.inf
    x[0, 3, 89999] = torch.finfo(dtype).min
    x[0, 4, 0] = 1.0
    x[0, 5, 89999] = 1.0
    parents = torch.tensor([[-1, 0, 1, 2, 3, 4]], dtype=torch.int32, device="cuda")
    tokens = torch.tensor([[0, 12, 0, 0, 89999, 0]], dtype=torch.int32, device="cuda")
    want = accept_check(x.to(dtype), tokens, parents, [6])
    assert want[3][0].tolist() == [12, 0, 0, 89999, 0, 89999] and want[0][0] == 5


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_accept_rows_off_16_byte_boundaries(dtype):
    g = torch.Generator(device="cuda").manual_seed(8)
    base = torch.randn((2, 5, 7003), generator=g, device="cuda").to(dtype)
    _, tokens, parents, nodes = accept_case(2, 5, 7001, dtype, seed=9)
    accept_check(base[:, :, 1:7002], tokens, parents, nodes)


def test_accept_repeats_streams_and_graphs():
    cases = [accept_case(4, 16, 30000, torch.bfloat16, seed=s) for s in (10, 11)]
    cases = [(l, t, p, torch.tensor(n, dtype=torch.int32, device="cuda")) for l, t, p, n in cases]
    want = [dfl.tree_accept(l, t, p, num_nodes=n) for l, t, p, n in cases]
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [dfl.tree_accept(l, t, p, num_nodes=n, stream=st) for (l, t, p, n), st in zip(cases, s)]
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            assert all(torch.equal(a, b) for a, b in zip(w, g))
    graphs, outs = [], []
    for l, t, p, n in cases:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(dfl.tree_accept(l, t, p, num_nodes=n))
        graphs.append(gr)
    for _ in range(4):
        for o in outs:
            for x in o:
                x.fill_(-9)
        torch.cuda.synchronize()
        for gr, st in zip(graphs, s):
            with torch.cuda.stream(st):
                gr.replay()
        torch.cuda.synchronize()
        for w, g in zip(want, outs):
            assert all(torch.equal(a, b) for a, b in zip(w, g))


# ------------------------------------------------------------------------------------ moves


def commit_case(nb, T, layers, hkv, d, page, dtype, seed, nodes=None, accepted=None, layout="nhd"):
    rng = np.random.default_rng(seed)
    nodes = nodes or [int(x) for x in rng.integers(1, T + 1, nb)]
    lens = [n + int(rng.integers(0, 60)) for n in nodes]
    need = [-(-L // page) for L in lens]
    pool = sum(need) + 3
    perm = rng.permutation(pool)
    table = np.full((nb, max(max(need), 1)), -3, dtype=np.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = perm[at:at + k]
        at += k
    acc = np.zeros(nb, dtype=np.int32)
    path = np.full((nb, T), -1, dtype=np.int32)
    for b, n in enumerate(nodes):
        if n == 0:
            continue
        acc[b] = accepted[b] if accepted else rng.integers(0, n)
        path[b, :acc[b] + 1] = [0] + sorted(rng.choice(np.arange(1, n), acc[b], replace=False))
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (layers, pool, hkv, page, d) if layout == "hnd" else (layers, pool, page, hkv, d)
    caches = []
    for _ in range(2):
        c = torch.randn(shape, generator=g, device="cuda").to(dtype)
        caches.append(c.permute(0, 1, 3, 2, 4) if layout == "hnd" else c)
    return caches[0], caches[1], table, lens, path, acc, nodes


def commit_check(k, v, table, lens, path, acc, nodes, squeeze=False, **kw):
    want = [ot.tree_commit(c.float().cpu().numpy(), table, lens, path, acc, nodes) for c in (k, v)]
    dev = [torch.from_numpy(np.asarray(x, dtype=np.int32)).cuda() for x in (table, lens, path, acc, nodes)]
    if squeeze:
        new = dfl.tree_commit(k[0], v[0], dev[0], dev[1], dev[2], dev[3], num_nodes=dev[4], **kw)
    else:
        new = dfl.tree_commit(k, v, dev[0], dev[1], dev[2], dev[3], num_nodes=dev[4], **kw)
    torch.cuda.synchronize()
    for c, (w, l) in zip((k, v), want):
        np.testing.assert_array_equal(c.float().cpu().numpy(), w)
        np.testing.assert_array_equal(new.cpu().numpy(), l)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("nb,T,layers,hkv,d,page", [(1, 1, 1, 1, 16, 8), (1, 16, 1, 4, 512, 16), (3, 40, 3, 2, 80, 24),
                                                    (9, 64, 2, 8, 128, 64), (1, 256, 1, 1, 64, 256), (40, 6, 1, 2, 64, 16)])
def test_commit_moves(dtype, layout, nb, T, layers, hkv, d, page):
    commit_check(*commit_case(nb, T, layers, hkv, d, page, dtype, seed=T + nb, layout=layout), squeeze=layers == 1)


def test_commit_long_overlapping_paths_and_empty_requests():
    # paths of every other node, of all nodes (nothing moves) and of all but the second
    nodes = [200, 30, 31, 0, 12]
    case = list(commit_case(5, 200, 2, 2, 64, 16, torch.bfloat16, seed=3, nodes=nodes, accepted=[99, 29, 29, 0, 0]))
    path = np.full((5, 200), -1, dtype=np.int32)
    path[0, :100] = np.arange(0, 200, 2)
    path[1, :30] = np.arange(30)
    path[2, :30] = [0] + list(range(2, 31))
    path[4, 0] = 0
    case[4] = path
    commit_check(*case)


def test_commit_lengths_in_place_and_bad_input():
    k, v, table, lens, path, acc, nodes = commit_case(7, 10, 1, 2, 64, 16, torch.bfloat16, seed=5, nodes=[10] * 7,
                                                       accepted=[3, 3, 3, 3, 3, 3, 3])
    before = k.clone()
    good = ot.tree_commit(k.float().cpu().numpy(), table, lens, path, acc, nodes)
    path[1, 2] = path[1, 1]      # not increasing
    path[2, 3] = 10              # no such node
    path[3, 0] = 1               # not from the root
    acc[4] = 10                  # longer than the tree
    bad_lens = list(lens)
    bad_lens[5] = 9              # shorter than the tree
    dev = [torch.from_numpy(np.asarray(x, dtype=np.int32)).cuda() for x in (table, bad_lens, path, acc, nodes)]
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    new = dfl.tree_commit(k[0], v[0], dev[0], dev[1], dev[2], dev[3], num_nodes=dev[4], new_lens=dev[1],
                          device_error=word)
    torch.cuda.synchronize()
    assert new.data_ptr() == dev[1].data_ptr()
    assert word.item() == B.DEVERR_TREE | B.DEVERR_SEQ_LEN
    assert new.tolist() == [good[1][0], lens[1], lens[2], lens[3], lens[4], 9, good[1][6]]
    got = k.float().cpu().numpy()
    for b in range(7):
        pages = table[b][table[b] >= 0]
        np.testing.assert_array_equal(got[:, pages], (good[0] if b in (0, 6) else before.float().cpu().numpy())[:, pages])
    # a page that does not exist: its moves alone are left out
    word.zero_()
    k, v, table, lens, path, acc, nodes = commit_case(1, 10, 1, 2, 64, 8, torch.float32, seed=6, nodes=[10], accepted=[2])
    ctx = lens[0] - 10
    path[0, :3] = [0, 8, 9]
    want = k.cpu().numpy().copy()
    bad = (ctx + 9) // 8
    for s, node in ((1, 8), (2, 9)):
        if (ctx + node) // 8 != bad:
            want[:, table[0, (ctx + s) // 8], (ctx + s) % 8] = k.cpu().numpy()[:, table[0, (ctx + node) // 8], (ctx + node) % 8]
    table[0, bad] = k.shape[1]
    dev = [torch.from_numpy(np.asarray(x, dtype=np.int32)).cuda() for x in (table, lens, path, acc, nodes)]
    dfl.tree_commit(k, v, dev[0], dev[1], dev[2], dev[3], num_nodes=dev[4], device_error=word)
    assert word.item() == B.DEVERR_PAGE_ID
    np.testing.assert_array_equal(k.cpu().numpy(), want)


# -------------------------------------------------------------------------- a run of them all


def test_a_serving_step_from_candidates_to_the_committed_cache():
    """Candidates -> a tree -> attention -> acceptance -> commit; attention of the next block over the committed
    cache equals attention over a cache that holds the accepted tokens' K/V from the start."""
    rng = np.random.default_rng(1)
    g = torch.Generator(device="cuda").manual_seed(30)
    nb, V, page, hkv, hq, d = 3, 5000, 16, 2, 8, 128
    T, width = 13, 3
    # the drafter's logits at two levels give the branches: 3 children of the root, 3 of each of these
    level1 = torch.randn((nb, V), generator=g, device="cuda").bfloat16()
    _, _, _, c1, lp1 = dfl.token_logprobs(level1, top_k=width)
    level2 = torch.randn((nb, width, V), generator=g, device="cuda").bfloat16()
    _, _, _, c2, lp2 = dfl.token_logprobs(level2, top_k=width)
    tokens = torch.cat([torch.zeros((nb, 1), dtype=torch.int32, device="cuda"), c1, c2.reshape(nb, -1)], dim=1)
    parents = torch.tensor([[-1, 0, 0, 0, 1, 1, 1, 2, 2, 2, 3, 3, 3]] * nb, dtype=torch.int32, device="cuda")
    # the scores have the selector's form
    assert c1.dtype == torch.int32 and lp1.dtype == torch.float32 and (lp1[:, 0] >= lp1[:, 1]).all()
    ctx = [50, 61, 130]
    lens = torch.tensor([c + T for c in ctx], dtype=torch.int32, device="cuda")
    table = torch.randperm(60, generator=g, device="cuda").int()[:33].view(nb, 11)
    k = torch.randn((2, 60, page, hkv, d), generator=g, device="cuda").bfloat16()
    v = torch.randn((2, 60, page, hkv, d), generator=g, device="cuda").bfloat16()
    q = torch.randn((nb * T, hq, d), generator=g, device="cuda").bfloat16()
    out, _ = dfl.tree_attn(q, k[0], v[0], table, lens, parents)
    assert torch.isfinite(out.float()).all()
    # the target's logits: request 0 takes the second child and its third, 1 nothing, 2 the first child
    logits = torch.randn((nb, T, V), generator=g, device="cuda").bfloat16()
    for b, i in ((0, 2), (0, 9), (2, 1)):
        logits[b, int(parents[b, i]), int(tokens[b, i])] = 30.0
    acc, path, nxt, best = dfl.tree_accept(logits, tokens, parents)
    assert acc.tolist()[0] >= 2 and path[0, :3].tolist() == [0, 2, 9] and path[2, :2].tolist() == [0, 1]
    # what each position holds before and after
    old_k, old_v = k.clone(), v.clone()
    new = dfl.tree_commit(k, v, table, lens, path, acc)
    for b in range(nb):
        a = int(acc[b])
        assert int(new[b]) == ctx[b] + a + 1
        keep = list(range(ctx[b])) + [ctx[b] + int(x) for x in path[b, :a + 1]]
        for cache, old in ((k, old_k), (v, old_v)):
            for pos, src in enumerate(keep):
                assert torch.equal(cache[:, table[b, pos // page], pos % page], old[:, table[b, src // page], src % page])
    # the next block of one query over each committed request
    q1 = torch.randn((nb, hq, d), generator=g, device="cuda").bfloat16()
    o1, l1 = dfl.block_attn(q1, k[1], v[1], table, new, 1)
    o2, l2 = dfl.tree_attn(q1, k[1], v[1], table, new, torch.full((nb, 1), -1, dtype=torch.int32, device="cuda"))
    # the block kernel's row sums are of bf16 probabilities (u16), both products with V are (u16 of sum p |v| <= 5
    # each, |v| < 5 in this draw) and both outputs are rounded
    assert v.abs().max() < 5.5
    torch.testing.assert_close(l1, l2, rtol=1e-5, atol=1.01 * U16)
    torch.testing.assert_close(o1.float(), o2.float(), rtol=4 * U16, atol=2 * 5.5 * U16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_captured_step_serves_other_lengths_and_trees(dtype):
    """One graph of all four calls, replayed for lengths, trees and logits that it was not captured with."""
    g = torch.Generator(device="cuda").manual_seed(53)
    rng = np.random.default_rng(53)
    nb, T, V, page, hkv, hq, d, layers = 4, 21, 3001, 16, 2, 8, 64, 3
    k = torch.zeros((layers, 80, page, hkv, d), dtype=dtype, device="cuda")
    v, q = torch.zeros_like(k), torch.zeros((nb * T, hq, d), dtype=dtype, device="cuda")
    logits = torch.zeros((nb, T, V), dtype=dtype, device="cuda")
    tokens, parents = (torch.zeros((nb, T), dtype=torch.int32, device="cuda") for _ in range(2))
    lens, nodes = (torch.full((nb,), n, dtype=torch.int32, device="cuda") for n in (T, T))
    table = torch.randperm(80, generator=g, device="cuda").int().view(nb, 20)

    def step():
        scored = dfl.token_logprobs(logits, tokens.view(nb, T, 1), top_k=5)
        outs = [dfl.tree_attn(q, k[i], v[i], table, lens, parents, num_nodes=nodes, window=w)
                for i, w in ((0, 0), (1, 40), (2, 0))]
        acc, path, nxt, best = dfl.tree_accept(logits, tokens, parents, num_nodes=nodes)
        new = dfl.tree_commit(k, v, table, lens, path, acc, num_nodes=nodes, new_lens=lens)
        assert new is lens
        return list(scored) + [x for o in outs for x in o] + [acc, path, nxt, best]

    graph = torch.cuda.CUDAGraph()
    parents.fill_(-1)
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(4):
        n = rng.integers(0, T + 1, nb)
        ctx = rng.integers(0, 20 * page - T, nb)
        table_n = np.array([[rng.integers(-1, max(1, i)) if i else -1 for i in range(T)] for _ in range(nb)], np.int32)
        lens0 = torch.tensor(np.where(n > 0, ctx + n, ctx), dtype=torch.int32, device="cuda")
        nodes.copy_(torch.tensor(n, dtype=torch.int32))
        parents.copy_(torch.from_numpy(np.minimum(table_n, np.arange(T) - 1)))
        for x in (q, logits, k, v):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        best = logits.float().argmax(2).int()
        up = parents.long().clamp(min=0)
        agree = torch.rand((nb, T), generator=g, device="cuda") < 0.7
        tokens.copy_(torch.where(agree, best.gather(1, up), (best.gather(1, up) + 1) % V))
        start = k.clone(), v.clone()
        for x in got:
            x.zero_()
        lens.copy_(lens0)
        graph.replay()
        torch.cuda.synchronize()
        from_graph = [x.clone() for x in got] + [lens.clone(), k.clone(), v.clone()]
        k.copy_(start[0])
        v.copy_(start[1])
        lens.copy_(lens0)
        eager = step()
        torch.cuda.synchronize()
        assert dfl.tree_attn_error() == 0
        for a, b in zip(from_graph, list(eager) + [lens, k, v]):
            assert torch.equal(a, b)
        want = ot.tree_accept(logits.double().cpu().numpy(), tokens.cpu().numpy(), parents.cpu().numpy(), n)
        for a, b in zip(eager[-4:], want):
            np.testing.assert_array_equal(a.cpu().numpy(), b)
        for cache, old in ((k, start[0]), (v, start[1])):
            moved, new = ot.tree_commit(old.double().cpu().numpy(), table.cpu().numpy(), lens0.cpu().numpy(), want[1],
                                        want[0], n)
            assert (cache.double().cpu().numpy() == moved).all()
        np.testing.assert_array_equal(lens.cpu().numpy(), new)


# ------------------------------------------------------------------- scores that are not finite


@pytest.mark.parametrize("kernel,dtype", BOTH)
@pytest.mark.parametrize("kind", ["nan", "inf", "overflow", "lowest"])
# one range; several ranges, of few rows (several warps to a row in the join) and of many
@pytest.mark.parametrize("n,L,hq,hkv,d", [(5, 60, 4, 2, 64), (5, 3000, 4, 2, 64), (3, 9000, 2, 1, 512), (64, 3000, 32, 4, 128),
                                          (40, 2500, 16, 2, 256)])
def test_rows_of_scores_that_are_not_finite_come_out_as_nan(kernel, dtype, kind, n, L, hq, hkv, d):
    # however the keys were dealt to ranges; and no other row changes a bit
    t = Tree([n], [L], hq=hq, hkv=hkv, d=d, dtype=dtype, seed=60)
    node, head = n - 1, hq - 1
    if kind == "overflow":  # one key of the context gives a product above the largest fp32 number
        page, slot = int(t.table[0, 3 // t.page]), 3 % t.page
        t.k[page, slot] = 16.0
    if kind == "lowest":  # every key does, below the lowest
        live = torch.from_numpy(t.table[0][:-(-L // t.page)].copy()).long().cuda()
        t.k[live] = t.k[live].abs() + 4.0
    t.q[node, head] = 0.0
    want, want_lse = t.call(kernel)
    t.q[node, head] = {"nan": 0.0, "inf": 0.0, "overflow": 1e38, "lowest": -1e38}[kind]
    if kind in ("nan", "inf"):
        t.q[node, head, 3] = float(kind)
    out, lse = t.call(kernel)
    assert t.error() == 0
    assert torch.isnan(out[node, head]).all() and torch.isnan(lse[node, head])
    same = torch.ones((n, hq), dtype=torch.bool, device="cuda")
    same[node, head] = False
    assert torch.equal(out[same], want[same]) and torch.equal(lse[same], want_lse[same])
    assert torch.isfinite(out[same].float()).all() and torch.isfinite(lse[same]).all()


# ------------------------------------------------------------------------ the word of device errors


def on_device(t):
    return (torch.from_numpy(t.table).cuda(), torch.tensor(t.lens, dtype=torch.int32, device="cuda"),
            torch.from_numpy(t.parents).cuda(), torch.tensor(t.nodes, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("kernel,dtype", BOTH)
def test_an_error_outlives_a_larger_call(kernel, dtype):
    # the second call on the stream needs a larger workspace than the first
    small, large = Tree([2], [30], dtype=dtype, seed=61), Tree([64], [5000], hq=32, hkv=4, d=512, dtype=dtype, seed=62)
    small.table[0, 1] = small.k.shape[0]
    stream = torch.cuda.Stream()
    for t in (small, large):
        args = on_device(t)
        torch.cuda.synchronize()
        dfl.tree_attn(t.q, t.k, t.v, *args[:3], num_nodes=args[3], kernel=kernel, stream=stream)
    other = torch.cuda.Stream()
    assert dfl.tree_attn_error(stream=other) == 0  # another stream's calls were sound
    assert dfl.tree_attn_error(stream=stream, clear=False) == B.DEVERR_PAGE_ID
    assert dfl.tree_attn_error(stream=stream) == B.DEVERR_PAGE_ID
    assert dfl.tree_attn_error(stream=stream) == 0


@pytest.mark.parametrize("kernel,dtype", BOTH)
def test_errors_of_captured_calls_are_reported(kernel, dtype):
    # two layers in a graph, which other graphs' and eager calls run between
    t = Tree([6, 3], [100, 200], dtype=dtype, seed=63)
    args = on_device(t)
    o, l = torch.zeros_like(t.q), torch.zeros(t.q.shape[:2], device="cuda")

    def layer(q, out):
        return dfl.tree_attn(q, t.k, t.v, *args[:3], num_nodes=args[3], kernel=kernel, out=out, lse=l)

    mid = torch.zeros_like(o)
    layer(t.q, mid)
    layer(mid, o)
    torch.cuda.synchronize()
    want = o.clone()
    assert dfl.tree_attn_error() == 0
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer(t.q, mid)
            layer(mid, o)
        graphs.append(g)
    good = args[0].clone()
    for g in graphs:
        g.replay()
        assert dfl.tree_attn_error() == 0 and torch.equal(o, want)
        args[0][1, 2] = -4
        g.replay()
        args[0].copy_(good)
        graphs[0].replay()
        graphs[1].replay()
        layer(t.q, mid)
        assert dfl.tree_attn_error(clear=False) == B.DEVERR_PAGE_ID
        assert dfl.tree_attn_error() == B.DEVERR_PAGE_ID
        assert dfl.tree_attn_error() == 0
        g.replay()
        assert dfl.tree_attn_error() == 0 and torch.equal(o, want)


@pytest.mark.parametrize("kernel,dtype", BOTH)
def test_a_given_word_takes_the_errors(kernel, dtype):
    t = Tree([6, 3], [100, 200], T=6, dtype=dtype, seed=64)
    args = on_device(t)
    word, ws = torch.zeros(1, dtype=torch.int32, device="cuda"), None

    def call(**kw):
        return dfl.tree_attn(t.q, t.k, t.v, *args[:3], num_nodes=args[3], kernel=kernel, device_error=word, **kw)

    out, lse = call()
    assert word.item() == 0 and dfl.tree_attn_error() == 0
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    args[1][0] = 5
    call()
    assert word.item() == B.DEVERR_SEQ_LEN and dfl.tree_attn_error() == 0
    args[2][1, 2] = 2  # (bits add up)
    g.replay()
    torch.cuda.synchronize()
    assert word.item() == B.DEVERR_SEQ_LEN | B.DEVERR_TREE and dfl.tree_attn_error() == 0
    # beside a given workspace: its own word stays as it is, whatever it holds
    dims = dfl.make_dims(t.q, t.k, torch.from_numpy(t.table), 6)
    ws = torch.full((dfl.tree_attn_workspace_bytes(dims, 6),), 255, dtype=torch.uint8, device="cuda")
    word.zero_()
    args[1][0], args[2][1, 2] = 100, 0
    args[0][0, 0] = t.k.shape[0]
    call(workspace=ws)
    assert word.item() == B.DEVERR_PAGE_ID and (ws[:256] == 255).all()
    for bad in (torch.zeros(1, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda"),
                torch.zeros(1, dtype=torch.int32)):
        with pytest.raises(ValueError):
            dfl.tree_attn(t.q, t.k, t.v, *args[:3], num_nodes=args[3], device_error=bad)


# ------------------------------------------------------------------ rows with one likely token


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1000, 5000, 70001])
@pytest.mark.parametrize("lead", [10.0, 16.0, 25.0, 30.0, 50.0])
def test_logprobs_of_one_likely_token(dtype, V, lead):
    # The others share a mass p / (1 + p) with p = sum exp(x - lead). Their terms are added up among themselves and to
    # the 1 of the likely one once each; such an addition rounds by half a step of [1, 2), 2^-24, at most, and
    # by no more than what it adds, as leaving 1 out of it would. So ln s is off by p, or by 2^-24 an addition: 8 in
    # a thread's step, one per later step (at most 1 + V / 2048 / slices: a row alone has one), 9 in the CTA's join,
    # V / 2048 / 128 + 1 + 9 in the slices': below 32. The entropy's other part, sum p y, is off by 2^-16 of itself: terms of
    # |y| <= 80 with two roundings of the exponent (2^-17.2) and one of 2^-22, sums of few roundings.
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randint(-32, 1, (4, V), generator=g, device="cuda").float() / 8
    at = torch.tensor([0, 7, V // 2, V - 1], device="cuda")
    x[torch.arange(4, device="cuda"), at] = lead
    x = x.to(dtype)
    tokens = at.int()[:, None].contiguous()
    given, ent, z, top, lp = dfl.token_logprobs(x, tokens, top_k=2)
    wide = x.double()
    e = (wide - lead).exp()
    e[torch.arange(4, device="cuda"), at] = 0.0
    p = e.sum(1)
    y = (e * (wide - lead)).sum(1)
    ln_s = torch.log1p(p)
    lost = torch.minimum(p, torch.full_like(p, 32 * 2.0 ** -24))
    want = ln_s - y / (1 + p)
    assert ((ent.double() - want).abs() <= lost * (1 + 2.0 ** -16) + 2.0 ** -16 * want).all()
    assert ((given[:, 0].double() + ln_s).abs() <= lost * (1 + 2.0 ** -16) + 2.0 ** -20 * ln_s).all()
    assert torch.equal(top[:, 0], tokens[:, 0]) and torch.equal(lp[:, 0], given[:, 0])
    # lead / 1 + ln s, rounded once more to half a step of 64
    assert ((z.double() - lead - ln_s).abs() <= lost * (1 + 2.0 ** -16) + 2.0 ** -18).all()


@pytest.mark.parametrize("kernel,dtype", BOTH)
@pytest.mark.parametrize("hkv,d", [(1, 16), (1, 128), (2, 64)])
def test_a_cache_of_one_page_and_requests_of_one_key(kernel, dtype, hkv, d):
    # the page stride is never taken then, nor the head stride of one head
    t = Tree([3], [13], hq=2 * hkv, hkv=hkv, d=d, dtype=dtype, page=16, seed=65)
    only = int(t.table[0, 0])
    t.k, t.v = (c[only:only + 1].clone() for c in (t.k, t.v))
    t.table[0, 0] = 0
    t.check(*t.call(kernel))
    t.k, t.v = (c.as_strided(c.shape, (0,) + c.stride()[1:]) for c in (t.k, t.v))
    t.check(*t.call(kernel))
    t = Tree([1, 1, 0, 1], [1, 1, 0, 2], hq=2 * hkv, hkv=hkv, d=d, dtype=dtype, seed=66)
    t.check(*t.call(kernel))
    assert t.error() == 0
