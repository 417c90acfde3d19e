"""Layouts of rope's output, without a GPU: rows that would share elements are refused on the host, others get past that check."""
import ctypes

import pytest
import torch

import speculative_decoding_block_dflash_gb300 as dfl
from speculative_decoding_block_dflash_gb300 import _binding as B
from speculative_decoding_block_dflash_gb300 import build as build_mod

cpu_only = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer validation runs on CPU-only hosts")
FAKE = 0x10000


def call(lib, N, H, D, strides, positions=None):
    f = B.RopeFreqs(FAKE, 64, 0, 1.0)
    status = lib.dflash_rope(FAKE, 2 * FAKE, 0, N, H, D, H * D, D, *strides, positions, ctypes.byref(f), 0, 0)
    return status, lib.dflash_last_error_message().decode()


@cpu_only
@pytest.mark.parametrize("N,H,strides", [(3, 4, (128, 128)), (3, 4, (384, 128)), (3, 4, (128, 256)), (3, 4, (511, 128)),
                                         (1000, 2, (128, 999 * 128)), (2, 2, (200, 256))])
def test_rows_that_share_elements_are_refused(N, H, strides):
    build_mod.build()
    status, why = call(dfl.load_library(), N, H, 128, strides, FAKE)
    assert status == B.ERR_INVALID_ARG and "overlap" in why


@cpu_only
@pytest.mark.parametrize("N,H,strides", [(3, 4, (512, 128)), (3, 4, (128, 384)), (3, 4, (640, 160)), (1000, 2, (128, 128000)),
                                         (1, 4, (0, 128)), (3, 1, (128, 0)), (1, 1, (0, 0))])
def test_other_layouts_pass(N, H, strides):
    build_mod.build()
    status, why = call(dfl.load_library(), N, H, 128, strides)  # (refused for its positions, the next check)
    assert status == B.ERR_INVALID_ARG and "positions" in why
