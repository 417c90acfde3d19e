"""GPU checks of what an append reports and leaves alone."""
import numpy as np
import pytest
import torch

import speculative_decoding_block_dflash_gb300 as dfl
from speculative_decoding_block_dflash_gb300 import _binding as B
from speculative_decoding_block_dflash_gb300 import build as build_mod
from test_cache8_gpu import Append, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build_mod.build()
    dfl.load_library()


def pages_of(a, b):
    return [int(x) for x in a.table[b] if x >= 0]


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("starts,left_out", [
    ([0, 4, 100, 104], (1, 2)),    # rows that end behind the inputs, and rows that lie behind them
    ([0, 4, 8, 3000], (2,)),       # (lengths below suit 4 rows)
    ([-4, 0, 4, 8], (0,)),         # wholly before them
    ([-2, 2, 6, 10], (0,)),        # and in part
    ([0, 4, 8, 2 ** 31 - 1], (2,)),
])
def test_starts_outside_the_inputs_are_reported(starts, left_out, e4m3):
    a = Append([4, 4, 4], [10, 20, 10], e4m3=e4m3)
    a.starts = starts
    before = a.numpy()
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    a.call(device_error=word)
    assert word.item() == B.DEVERR_SEQ_LEN
    got = a.numpy()
    for b in range(3):
        pages = pages_of(a, b)
        same = [np.array_equal(x[pages], y[pages]) for x, y in zip(before[0], got[0])]
        assert all(same) if b in left_out else not any(same), b


@pytest.mark.parametrize("e4m3", [True, False])
def test_rows_behind_the_inputs_of_many_requests(e4m3):
    """The last of 700 requests claims a row that is not there; nothing else is wrong."""
    a = Append([1] * 700, [3] * 700, hkv=1, d=16, e4m3=e4m3)
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    a.call(device_error=word)
    assert word.item() == 0
    a = Append([1] * 700, [3] * 700, hkv=1, d=16, e4m3=e4m3)
    a.k, a.v = a.k[:-1], a.v[:-1]
    before = a.numpy()
    a.call(device_error=word)
    assert word.item() == B.DEVERR_SEQ_LEN
    got = a.numpy()
    assert all(np.array_equal(x[pages_of(a, 699)], y[pages_of(a, 699)]) for x, y in zip(before[0], got[0]))
    assert not any(np.array_equal(x[pages_of(a, 698)], y[pages_of(a, 698)]) for x, y in zip(before[0], got[0]))


@pytest.mark.parametrize("e4m3", [True, False])
def test_starts_that_decrease_are_reported(e4m3):
    a = Append([4, 4], [10, 20], e4m3=e4m3)
    a.starts = [4, 0, 8]
    a.lens = [30, 30]
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    a.table = np.where(a.table < 0, a.table.max(), a.table)
    a.call(device_error=word)
    assert word.item() & B.DEVERR_SEQ_LEN


def test_starts_within_the_inputs_are_not_reported():
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    for e4m3 in (True, False):
        for pad in (0, 5):
            a = Append([0, 4, 0, 7, 0], [0, 10, 3, 20, 9], e4m3=e4m3, pad=pad)
            a.call(device_error=word)
            assert word.item() == 0
        a = Append([0, 4, 0], [0, 10, 3], e4m3=e4m3)
        a.starts = [100, 100, 100, 100]  # nobody has new rows, wherever they would be
        a.call(device_error=word)
        assert word.item() == 0


@pytest.mark.parametrize("e4m3", [True, False])
def test_errors_of_calls_without_a_word_are_kept(e4m3):
    dfl.tree_attn_error()
    a = Append([4, 4], [10, 20], e4m3=e4m3)
    a.call()
    assert dfl.tree_attn_error() == 0
    a.lens[1] = 3
    a.call()
    a.table[0][0] = 10 ** 6
    a.call()
    assert dfl.tree_attn_error(clear=False) == B.DEVERR_SEQ_LEN | B.DEVERR_PAGE_ID
    assert dfl.tree_attn_error() == B.DEVERR_SEQ_LEN | B.DEVERR_PAGE_ID and dfl.tree_attn_error() == 0
    # another stream's are its own
    s = torch.cuda.Stream()
    a.call(stream=s)
    assert dfl.tree_attn_error() == 0 and dfl.tree_attn_error(stream=s) != 0
    # a given word takes them in place of the library's
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    a.call(device_error=word)
    assert word.item() != 0 and dfl.tree_attn_error() == 0


@pytest.mark.parametrize("e4m3", [True, False])
def test_errors_of_a_captured_append(e4m3):
    a = Append([4, 4], [10, 20], e4m3=e4m3)
    table, lens, starts = torch.from_numpy(a.table).cuda(), ints(a.lens), ints(a.starts)
    kw = dict(starts=starts, k_scale=a.scales[0], v_scale=a.scales[1]) if e4m3 else dict(starts=starts)
    dfl.append_kv(a.k, a.v, *a.caches, table, lens, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dfl.append_kv(a.k, a.v, *a.caches, table, lens, **kw)
    graph.replay()
    torch.cuda.synchronize()
    assert dfl.tree_attn_error() == 0
    lens[1] = 3
    graph.replay()
    torch.cuda.synchronize()
    assert dfl.tree_attn_error() == B.DEVERR_SEQ_LEN and dfl.tree_attn_error() == 0


def test_a_drafted_tree_is_committed_by_appending_again():
    """The accepted nodes' rows, appended once more behind the context, leave what an append of those alone would have: bytes, scales and
    the next step's attention."""
    g = torch.Generator(device="cuda").manual_seed(7)
    hkv, d, page, ctx = 2, 64, 16, [21, 40]
    rope = dfl.make_rope(d)
    table = torch.arange(12, dtype=torch.int32, device="cuda").flip(0).reshape(2, 6).contiguous()
    parents = [[-1, 0, 0, 1, 2, 4, 3, 1], [-1, 0, 1, 1, 2, 0, 5, 6]]
    paths = [[0, 2, 4, 5], [0, 5]]  # the accepted nodes, the bonus token first
    n = len(parents[0])

    def depth(b, i):
        return 0 if parents[b][i] < 0 else 1 + depth(b, parents[b][i])

    def rows(count):
        # magnitudes in [1/4, 4]: never in e4m3's subnormals, so that re-encoding a page loses nothing
        x = torch.rand((2, count, hkv, d), generator=g, device="cuda") * 3.75 + 0.25
        return x * (torch.randint(0, 2, x.shape, generator=g, device="cuda") * 2 - 1)

    def caches():
        c = [torch.zeros((12, page, hkv, d), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
        return c, [torch.zeros((12, hkv), device="cuda") for _ in range(2)]

    def append(where, k, v, starts, lens, positions=None):
        dfl.append_kv(k, v, *where[0], table, ints(lens), starts=ints(starts), rope=rope, positions=positions, k_scale=where[1][0],
                      v_scale=where[1][1])

    old = rows(sum(ctx))
    tree = rows(2 * n)
    tree[1] *= 8.0  # the draft's values move the pages' scales
    at = ints([c + depth(b, i) for b, c in enumerate(ctx) for i in range(n)])
    take = torch.tensor([b * n + i for b in range(2) for i in paths[b]], device="cuda")
    starts = [0, len(paths[0]), len(paths[0]) + len(paths[1])]
    lens = [c + len(x) for c, x in zip(ctx, paths)]
    drafted, plain = caches(), caches()
    for where in (drafted, plain):
        append(where, old[0], old[1], [0, ctx[0], sum(ctx)], ctx)
    append(drafted, tree[0], tree[1], [0, n, 2 * n], [c + n for c in ctx], at)
    q = torch.randn((2 * n, 4, d), generator=g, device="cuda").to(torch.bfloat16)
    full = [c + n for c in ctx]
    out, _ = dfl.cache8_attn(dfl.rope(q, at, rope), *drafted[0], *drafted[1], table, ints(full), n, parents=ints(parents))
    assert out.isfinite().all()
    for where in (drafted, plain):
        append(where, tree[0][take], tree[1][take], starts, lens)  # (a node's depth is its place behind the context)
    for b, L in enumerate(lens):
        j = torch.arange(L, device="cuda")
        pg, sl = table[b][j // page].long(), j % page
        for c, e in zip(drafted[0], plain[0]):
            assert torch.equal(c.view(torch.uint8)[pg, sl], e.view(torch.uint8)[pg, sl])
        for c, e in zip(drafted[1], plain[1]):
            assert torch.equal(c[pg], e[pg])
    step = torch.randn((2, 4, d), generator=g, device="cuda").to(torch.bfloat16)
    got, want = (dfl.cache8_attn(step, *w[0], *w[1], table, ints(lens), 1) for w in (drafted, plain))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert dfl.tree_attn_error() == 0
