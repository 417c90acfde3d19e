"""GPU checks of rotary positions under autograd: the gradient is the turn back of the result's gradient.

The bounds are test_cache8_gpu.py's: a turned dim is off by 8 u32 gain (|x| + |y|), and by its rounding to bf16.
"""
import numpy as np
import pytest
import torch

import speculative_decoding_block_dflash_gb300 as dfl
from oracle import cache8 as oc
from speculative_decoding_block_dflash_gb300 import build as build_mod
from test_cache8_gpu import U32, check_rope, inv_freq, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build_mod.build()
    dfl.load_library()


def make(N, H, D, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, gy = (torch.randn((N, H, D), generator=g, device="cuda").to(dtype) for _ in range(2))
    pos = np.random.default_rng(seed).integers(-50, 200000, N).astype(np.int32)
    return x, gy, pos, torch.from_numpy(pos).cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("N,H,D,r", [(1, 1, 64, 64), (300, 8, 128, 64), (9, 4, 30, 10), (5, 2, 512, 512)])
def test_gradient(N, H, D, r, inverse, layout, dtype):
    x, gy, pos, pos_d = make(N, H, D, dtype, seed=N)
    turn = dfl.make_rope(r, layout=layout, gain=1.25)
    want = dfl.rope(x, pos_d, turn, inverse=inverse)
    leaf = x.clone().requires_grad_()
    y = dfl.rope(leaf, pos_d, turn, inverse=inverse)
    assert y.requires_grad and torch.equal(y, want)
    y.backward(gy)
    assert torch.equal(leaf.grad, dfl.rope(gy, pos_d, turn, inverse=not inverse))
    check_rope(gy, pos, inv_freq(r), 1.25, layout, not inverse, leaf.grad)


def test_gradient_by_differences():
    x, gy, pos, pos_d = make(6, 2, 16, torch.float32, seed=9)
    turn = dfl.make_rope(12, layout="interleaved")
    leaf = x.clone().requires_grad_()
    (dfl.rope(leaf, pos_d, turn) * gy).sum().backward()
    base = dfl.rope(x, pos_d, turn).double()
    for n, h, d in [(0, 0, 0), (1, 1, 5), (2, 0, 11), (3, 1, 2), (4, 0, 7), (5, 1, 10), (5, 0, 15)]:
        z = x.clone()
        z[n, h, d] += 1.0  # the map is linear: any step will do
        diff = ((dfl.rope(z, pos_d, turn).double() - base) * gy.double()).sum().item()
        # two results of error 8 u32 (|x| + |y|), |x| + |y| < 8 here, times two |gy| < 4
        assert abs(diff - leaf.grad[n, h, d].item()) <= 2 * 2 * 4 * 8 * U32 * 8


def test_a_sums_gradient_and_strided_inputs():
    x, _, pos, pos_d = make(50, 12, 64, torch.float32, seed=1)
    turn = dfl.make_rope(32)
    rows = x.clone().requires_grad_()
    dfl.rope(rows[:, 3:8], pos_d, turn).sum().backward()  # (the gradient of a sum is one number, repeated)
    want = torch.zeros_like(x)
    want[:, 3:8] = dfl.rope(torch.ones((50, 5, 64), device="cuda"), pos_d, turn, inverse=True)
    assert torch.equal(rows.grad, want)
    heads_first = x.permute(1, 0, 2).contiguous().requires_grad_()
    g = torch.randn((12, 50, 64), device="cuda")
    dfl.rope(heads_first.permute(1, 0, 2), pos_d, turn).permute(1, 0, 2).backward(g)
    assert torch.equal(heads_first.grad, dfl.rope(g.permute(1, 0, 2), pos_d, turn, inverse=True).permute(1, 0, 2))


def test_the_gradients_gradient():
    x, gy, pos, pos_d = make(7, 2, 32, torch.float32, seed=2)
    turn = dfl.make_rope(32)
    a, b = x.clone().requires_grad_(), gy.clone().requires_grad_()
    (ga,) = torch.autograd.grad(dfl.rope(a, pos_d, turn), a, b, create_graph=True)
    (gb,) = torch.autograd.grad(ga, b, torch.ones_like(ga))
    assert torch.equal(gb, dfl.rope(torch.ones_like(x), pos_d, turn))


def test_what_is_not_recorded():
    x, gy, pos, pos_d = make(7, 2, 32, torch.float32, seed=3)
    turn = dfl.make_rope(32)
    leaf = x.clone().requires_grad_()
    with torch.no_grad():
        assert not dfl.rope(leaf, pos_d, turn).requires_grad
        y = torch.empty_like(x)
        assert dfl.rope(leaf, pos_d, turn, out=y) is y
    assert not dfl.rope(x, pos_d, turn).requires_grad
    for out in (torch.empty_like(x), leaf):
        with pytest.raises(ValueError):
            dfl.rope(leaf, pos_d, turn, out=out)
    assert torch.equal(leaf.detach(), x)
    y = dfl.rope(leaf, pos_d, turn)
    pos_d += 1  # what the backward pass needs has changed
    with pytest.raises(RuntimeError):
        y.backward(gy)


def test_a_stream_and_a_captured_step():
    x, gy, pos, pos_d = make(33, 5, 96, torch.float32, seed=4)
    turn = dfl.make_rope(96)
    want = dfl.rope(gy, pos_d, turn, inverse=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    leaf = x.clone().requires_grad_()
    y = dfl.rope(leaf, pos_d, turn, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    y.backward(gy)
    torch.cuda.synchronize()
    assert torch.equal(leaf.grad, want)
    del y
    leaf = x.clone().requires_grad_()
    with torch.cuda.stream(s):
        for _ in range(2):
            torch.autograd.grad(dfl.rope(leaf, pos_d, turn), leaf, gy)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        (got,) = torch.autograd.grad(dfl.rope(leaf, pos_d, turn), leaf, gy)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    gy.mul_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, dfl.rope(gy, pos_d, turn, inverse=True))


def test_a_training_step_of_a_layer():
    """Weights before the rotation get the gradient of the formula in float64."""
    g = torch.Generator(device="cuda").manual_seed(5)
    h, w = torch.randn((40, 24), generator=g, device="cuda"), torch.randn((24, 2 * 32), generator=g, device="cuda")
    gy = torch.randn((40, 2, 32), generator=g, device="cuda")
    pos, turn = ints(list(range(40))), dfl.make_rope(32)
    leaf = w.clone().requires_grad_()
    dfl.rope((h @ leaf).view(40, 2, 32), pos, turn).backward(gy)
    gx = oc.rope(gy.double().cpu().numpy(), np.arange(40), inv_freq(32), inverse=True).reshape(40, 64)
    want = h.double().cpu().numpy().T @ gx
    # a sum of 40 products: each gradient is off by 8 u32 (|x| + |y|) <= 8 u32 8, and the sum by 40 u32 of its terms' sizes
    size = np.abs(h.double().cpu().numpy()).T @ (np.abs(gx) + 8)
    assert np.all(np.abs(leaf.grad.double().cpu().numpy() - want) <= 48 * U32 * size)
