"""The operators on drafted trees without a GPU: sizes of workspaces, and arguments that are refused on the host
before any CUDA call, through the C ABI and through the Python wrappers."""
import ctypes
import math

import pytest
import torch

import speculative_decoding_block_dflash_gb300 as dfl
from speculative_decoding_block_dflash_gb300 import _binding as B
from speculative_decoding_block_dflash_gb300 import build as build_mod

# Fake device addresses are only used in calls that must fail validation (see test_abi_cpu.py).
cpu_only = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer validation runs on CPU-only hosts")
FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return dfl.load_library()


def dims(**kw):
    d = B.Dims()
    vals = dict(batch=2, num_q_heads=32, num_kv_heads=4, head_dim=128, page_size=16, num_pages=64, max_pages=16,
                max_seq_len=0, dtype=B.BF16)
    vals.update(kw)
    for k, v in vals.items():
        setattr(d, k, v)
    d.kv_stride_head = kw.get("kv_stride_head", d.head_dim)
    d.kv_stride_slot = kw.get("kv_stride_slot", d.num_kv_heads * d.head_dim)
    d.kv_stride_page = kw.get("kv_stride_page", d.page_size * d.num_kv_heads * d.head_dim)
    return d


def test_constants_match_the_header():
    text = open(build_mod.INCLUDE + "/dflash_attn.h").read()
    assert f"#define DFLASH_DEVERR_TREE {B.DEVERR_TREE}u" in text
    assert "#define DFLASH_MAX_TREE_NODES 256" in text and "#define DFLASH_MAX_TOP_K 64" in text


def test_workspace_sizes(lib):
    n = lib.dflash_tree_attn_workspace_bytes
    assert n(ctypes.byref(dims()), 16) >= 256 + 8192
    for bad in (dims(head_dim=72), dims(page_size=12), dims(num_kv_heads=5), dims(batch=0), dims(dtype=7)):
        assert n(ctypes.byref(bad), 16) == 0
    assert n(ctypes.byref(dims()), 0) == 0 and n(ctypes.byref(dims()), 257) == 0 and n(None, 4) == 0
    # a query tile per node and no range to split: no room for partials is asked for
    wide = dims(num_q_heads=1024, num_kv_heads=1)
    assert n(ctypes.byref(wide), 256) < 1 << 20
    # one wave's partials bound it, however long the keys
    assert n(ctypes.byref(dims(num_pages=1 << 20, max_pages=1 << 16)), 64) < 200 << 20
    m = lib.dflash_logprobs_workspace_bytes
    assert m(1, 1000, 8) >= 65536 * 4 and m(65535, 2 ** 31 - 1, 64) > 0
    for bad in ((-1, 1000, 8), (65536, 1000, 8), (4, 0, 0), (4, 1000, 65), (4, 10, 11), (4, 1000, -1)):
        assert m(*bad) == 0
    assert lib.dflash_tree_accept_workspace_bytes() == 2 * 65536 * 8


def attn(lib, d=None, T=4, window=0, scale=0.1, kernel=0, ws=FAKE, ws_bytes=1 << 40, **ptrs):
    p = dict(q=FAKE, k=FAKE, v=FAKE, table=FAKE, lens=FAKE, parents=FAKE, nodes=FAKE, out=2 * FAKE, lse=FAKE)
    p.update(ptrs)
    d = dims() if d is None else d
    return lib.dflash_tree_attn(p["q"], p["k"], p["v"], p["table"], p["lens"], p["parents"], p["nodes"],
                                ctypes.byref(d), T, window, scale, p["out"], p["lse"], kernel, ws, ws_bytes, 0, 0)


@cpu_only
@pytest.mark.parametrize("kw,code", [
    (dict(d=dims(head_dim=72)), B.ERR_UNSUPPORTED),
    (dict(d=dims(head_dim=528)), B.ERR_INVALID_ARG),
    (dict(d=dims(page_size=20)), B.ERR_INVALID_ARG),
    (dict(d=dims(batch=0)), B.ERR_INVALID_ARG),
    (dict(d=dims(max_seq_len=10 ** 6)), B.ERR_INVALID_ARG),
    (dict(d=dims(kv_stride_slot=516)), B.ERR_INVALID_ARG),
    (dict(d=dims(kv_stride_head=64)), B.ERR_INVALID_ARG),
    (dict(T=0), B.ERR_INVALID_ARG), (dict(T=257), B.ERR_INVALID_ARG),
    (dict(window=-1), B.ERR_INVALID_ARG),
    (dict(scale=0.0), B.ERR_INVALID_ARG), (dict(scale=-1.0), B.ERR_INVALID_ARG),
    (dict(scale=math.nan), B.ERR_INVALID_ARG), (dict(scale=math.inf), B.ERR_INVALID_ARG),
    (dict(kernel=3), B.ERR_INVALID_ARG), (dict(kernel=-1), B.ERR_INVALID_ARG),
    (dict(d=dims(dtype=B.FP32), kernel=2), B.ERR_UNSUPPORTED),
    (dict(d=dims(kv_stride_slot=0), kernel=2), B.ERR_UNSUPPORTED),
    (dict(ws=None), B.ERR_WORKSPACE), (dict(ws_bytes=300), B.ERR_WORKSPACE), (dict(ws=FAKE + 16), B.ERR_WORKSPACE),
    (dict(q=None), B.ERR_INVALID_ARG), (dict(k=None), B.ERR_INVALID_ARG), (dict(v=None), B.ERR_INVALID_ARG),
    (dict(table=None), B.ERR_INVALID_ARG), (dict(lens=None), B.ERR_INVALID_ARG), (dict(parents=None), B.ERR_INVALID_ARG),
    (dict(out=None), B.ERR_INVALID_ARG), (dict(out=FAKE), B.ERR_INVALID_ARG),
    (dict(q=FAKE + 8), B.ERR_INVALID_ARG), (dict(k=FAKE + 2), B.ERR_INVALID_ARG), (dict(lens=FAKE + 1), B.ERR_INVALID_ARG),
    (dict(lse=FAKE + 2), B.ERR_INVALID_ARG), (dict(nodes=FAKE + 2), B.ERR_INVALID_ARG),
])
def test_tree_attn_refuses(lib, kw, code):
    assert attn(lib, **kw) == code
    assert lib.dflash_last_error_message()


def logprobs(lib, dtype=0, R=2, V=100, stride=100, temp=1.0, m=1, k=4, ws=FAKE, ws_bytes=1 << 40, **ptrs):
    p = dict(logits=FAKE, tokens=FAKE, lp=FAKE, z=FAKE, ent=FAKE, top=FAKE, toplp=FAKE, err=FAKE)
    p.update(ptrs)
    return lib.dflash_token_logprobs(p["logits"], dtype, R, V, stride, temp, p["tokens"], m, p["lp"], p["z"], p["ent"], k,
                                     p["top"], p["toplp"], p["err"], ws, ws_bytes, 0)


@cpu_only
@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), B.ERR_INVALID_ARG), (dict(R=-1), B.ERR_INVALID_ARG), (dict(R=65536), B.ERR_INVALID_ARG),
    (dict(V=0), B.ERR_INVALID_ARG), (dict(stride=99), B.ERR_INVALID_ARG),
    (dict(temp=0.0), B.ERR_INVALID_ARG), (dict(temp=-1.0), B.ERR_INVALID_ARG), (dict(temp=math.nan), B.ERR_INVALID_ARG),
    (dict(temp=math.inf), B.ERR_INVALID_ARG), (dict(temp=1e-31), B.ERR_INVALID_ARG),
    (dict(m=-1), B.ERR_INVALID_ARG), (dict(m=65), B.ERR_INVALID_ARG), (dict(k=-1), B.ERR_INVALID_ARG),
    (dict(k=65), B.ERR_INVALID_ARG), (dict(V=3, stride=3, k=4), B.ERR_INVALID_ARG),
    (dict(logits=None), B.ERR_INVALID_ARG), (dict(tokens=None), B.ERR_INVALID_ARG), (dict(lp=None), B.ERR_INVALID_ARG),
    (dict(top=None), B.ERR_INVALID_ARG), (dict(toplp=None), B.ERR_INVALID_ARG),
    (dict(logits=FAKE + 1), B.ERR_INVALID_ARG), (dict(dtype=1, logits=FAKE + 2), B.ERR_INVALID_ARG),
    (dict(z=FAKE + 2), B.ERR_INVALID_ARG), (dict(err=FAKE + 1), B.ERR_INVALID_ARG),
    (dict(ws=None), B.ERR_WORKSPACE), (dict(ws_bytes=1000), B.ERR_WORKSPACE), (dict(ws=FAKE + 4), B.ERR_WORKSPACE),
])
def test_token_logprobs_refuses(lib, kw, code):
    assert logprobs(lib, **kw) == code
    assert lib.dflash_last_error_message()


@cpu_only
def test_token_logprobs_of_no_rows_is_a_no_op(lib):
    assert logprobs(lib, R=0, logits=None, ws=None) == B.OK


def accept(lib, dtype=0, nb=2, T=4, V=100, stride=100, ws=FAKE, ws_bytes=1 << 40, **ptrs):
    p = dict(logits=FAKE, tokens=FAKE, parents=FAKE, nodes=None, acc=FAKE, path=FAKE, nxt=FAKE, arg=None, err=None)
    p.update(ptrs)
    return lib.dflash_tree_accept(p["logits"], dtype, nb, T, V, stride, p["tokens"], p["parents"], p["nodes"], p["acc"],
                                  p["path"], p["nxt"], p["arg"], p["err"], ws, ws_bytes, 0)


@cpu_only
@pytest.mark.parametrize("kw,code", [
    (dict(dtype=5), B.ERR_INVALID_ARG), (dict(nb=0), B.ERR_INVALID_ARG), (dict(T=0), B.ERR_INVALID_ARG),
    (dict(T=257), B.ERR_INVALID_ARG), (dict(nb=300, T=256), B.ERR_INVALID_ARG), (dict(V=0), B.ERR_INVALID_ARG),
    (dict(stride=99), B.ERR_INVALID_ARG), (dict(logits=None), B.ERR_INVALID_ARG), (dict(tokens=None), B.ERR_INVALID_ARG),
    (dict(parents=None), B.ERR_INVALID_ARG), (dict(acc=None), B.ERR_INVALID_ARG), (dict(path=None), B.ERR_INVALID_ARG),
    (dict(nxt=None), B.ERR_INVALID_ARG), (dict(arg=FAKE + 1), B.ERR_INVALID_ARG), (dict(nodes=FAKE + 2), B.ERR_INVALID_ARG),
    (dict(logits=FAKE + 1), B.ERR_INVALID_ARG),
    (dict(ws=None), B.ERR_WORKSPACE), (dict(ws_bytes=4096), B.ERR_WORKSPACE), (dict(ws=FAKE + 8), B.ERR_WORKSPACE),
])
def test_tree_accept_refuses(lib, kw, code):
    assert accept(lib, **kw) == code
    assert lib.dflash_last_error_message()


def commit(lib, d=None, T=4, layers=2, layer_stride=1 << 20, **ptrs):
    p = dict(k=FAKE, v=32 * FAKE, table=FAKE, lens=8 * FAKE, path=FAKE, acc=FAKE, nodes=None, new=16 * FAKE, err=None)
    p.update(ptrs)
    d = dims() if d is None else d
    return lib.dflash_tree_commit(p["k"], p["v"], p["table"], p["lens"], p["path"], p["acc"], p["nodes"], p["new"],
                                  ctypes.byref(d), T, layers, layer_stride, p["err"], 0)


@cpu_only
@pytest.mark.parametrize("kw,code", [
    (dict(d=dims(head_dim=72)), B.ERR_UNSUPPORTED), (dict(T=0), B.ERR_INVALID_ARG), (dict(T=257), B.ERR_INVALID_ARG),
    (dict(layers=0), B.ERR_INVALID_ARG), (dict(layers=65536), B.ERR_INVALID_ARG), (dict(layer_stride=0), B.ERR_INVALID_ARG),
    (dict(layer_stride=-8), B.ERR_INVALID_ARG), (dict(layer_stride=1001), B.ERR_INVALID_ARG),
    (dict(d=dims(kv_stride_slot=0)), B.ERR_INVALID_ARG), (dict(d=dims(kv_stride_page=0)), B.ERR_INVALID_ARG),
    (dict(k=None), B.ERR_INVALID_ARG), (dict(v=None), B.ERR_INVALID_ARG), (dict(table=None), B.ERR_INVALID_ARG),
    (dict(lens=None), B.ERR_INVALID_ARG), (dict(path=None), B.ERR_INVALID_ARG), (dict(acc=None), B.ERR_INVALID_ARG),
    (dict(k=FAKE + 8), B.ERR_INVALID_ARG), (dict(path=FAKE + 2), B.ERR_INVALID_ARG),
    (dict(v=FAKE), B.ERR_INVALID_ARG),  # one cache for both
    # new_lens may be seq_lens itself, but overlap no other input, nor seq_lens in part
    (dict(new=8 * FAKE + 4), B.ERR_INVALID_ARG), (dict(new=FAKE), B.ERR_INVALID_ARG),
    (dict(new=16 * FAKE, nodes=16 * FAKE + 4), B.ERR_INVALID_ARG),
])
def test_tree_commit_refuses(lib, kw, code):
    assert commit(lib, **kw) == code
    assert lib.dflash_last_error_message()


def test_wrappers_refuse_host_tensors_and_bad_shapes():
    i32 = dict(dtype=torch.int32)
    logits = torch.zeros(2, 4, 10)
    with pytest.raises(ValueError):
        dfl.token_logprobs(logits)
    with pytest.raises(ValueError):
        dfl.tree_accept(logits, torch.zeros(2, 4, **i32), torch.zeros(2, 4, **i32))
    k = torch.zeros(8, 16, 2, 64, dtype=torch.bfloat16)
    q = torch.zeros(2 * 4, 4, 64, dtype=torch.bfloat16)
    table, lens, par = torch.zeros(2, 4, **i32), torch.zeros(2, **i32), torch.zeros(2, 4, **i32)
    with pytest.raises(ValueError):
        dfl.tree_attn(q, k, k, table, lens, par)
    with pytest.raises(ValueError):
        dfl.tree_attn(q[:7], k, k, table, lens, par)
    with pytest.raises(ValueError):
        dfl.tree_attn(q, k, k, table, lens, par, kernel="tc_pair")
    with pytest.raises(ValueError):
        dfl.tree_commit(k, k, table, lens, torch.zeros(2, 4, **i32), torch.zeros(2, **i32))
    with pytest.raises(ValueError):
        dfl.tree_commit(k[0], k[0], table, lens, torch.zeros(2, 4, **i32), torch.zeros(2, **i32))


def test_one_stride_of_rows():
    x = torch.zeros(4, 6, 10)
    assert B._row_stride(x, 24, 10) == 10
    assert B._row_stride(x[:, :, :7], 24, 7) == 10
    assert B._row_stride(x[:, :1, :7], 4, 7) == 60
    assert B._row_stride(x[:1, ::2, :7], 3, 7) == 20
    with pytest.raises(ValueError):
        B._row_stride(x[:, :5], 20, 10)
    with pytest.raises(ValueError):
        B._row_stride(x.transpose(1, 2), 40, 6)


@cpu_only
@pytest.mark.parametrize("kw,code", [
    (dict(err=FAKE + 2), B.ERR_INVALID_ARG), (dict(err=FAKE, ws=None), B.ERR_WORKSPACE),
    (dict(err=FAKE, ws_bytes=300), B.ERR_WORKSPACE), (dict(err=None, ws=FAKE + 16), B.ERR_WORKSPACE),
    (dict(err=FAKE, q=None), B.ERR_INVALID_ARG),
])
def test_tree_attn_with_a_word_refuses(lib, kw, code):
    q, err, ws, ws_bytes = (kw.get(k, v) for k, v in (("q", FAKE), ("err", FAKE), ("ws", FAKE), ("ws_bytes", 1 << 40)))
    assert lib.dflash_tree_attn_err(q, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, ctypes.byref(dims()), 4, 0, 0.1, 2 * FAKE, FAKE,
                                    0, err, ws, ws_bytes, 0, 0) == code
    assert lib.dflash_last_error_message()


def test_shared_error_word_refuses_null(lib):
    assert lib.dflash_shared_error_word(None) == B.ERR_INVALID_ARG
    assert lib.dflash_last_error_message()
