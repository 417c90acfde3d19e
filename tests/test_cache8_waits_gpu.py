"""The bounded waits of attention over an e4m3 cache: both tensor-core kernels give up where a wait runs out, report it, and leave
a context and a workspace that work.

The bound is 1 us. Where a CTA has several pieces, the warps that split the queries wait for a piece's last scores before they take
the next piece's queries: 20 tiles of keys for the larger shapes and 90 for the smallest, 20 us or more, however fast the copies come
(the clock is read after some ten tests of a barrier, each of which suspends the warp for a while). So every such call runs out. No
GPU fault, trap or hang is involved: the kernels give up by themselves and return.
"""
import pytest
import torch

import speculative_decoding_block_dflash_gb300 as dfl
from speculative_decoding_block_dflash_gb300 import _binding as B
from speculative_decoding_block_dflash_gb300 import build as build_mod
from test_cache8_gpu import Attn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build_mod.build()
    dfl.load_library()


@pytest.mark.parametrize("T,hq,hkv,d,keys", [
    (2, 16, 8, 128, 12000),  # few rows, their parts side by side: 480 pairs, some three pieces a CTA
    (9, 32, 8, 512, 2500),   # few rows, their parts in turn
    (40, 16, 8, 128, 2500),  # many rows
])
def test_a_wait_that_runs_out(T, hq, hkv, d, keys):
    requests = 60
    t = Attn([T] * requests, [keys + 3 * b for b in range(requests)], T=T, hq=hq, hkv=hkv, d=d, seed=5)
    good = t.call("tc")
    assert t.error() == 0
    for _ in range(3):
        t.call("tc", wait_limit_us=1)
        ws = t.ws
        assert t.error() & B.DEVERR_TIMEOUT
        # the next call, on the same workspace and with the usual bound, gives the same bits
        again = t.call("tc", workspace=ws)
        t.ws = ws
        assert t.error() == 0
        assert torch.equal(good[0], again[0]) and torch.equal(good[1], again[1])
