"""GPU checks of attention over an e4m3 cache whose value scales lie far apart, against float64.

With p_j the exact probabilities and w_j the value scale of key j's page, the tensor cores carry p_j w_j to 2^-9 of itself or
2^-28 of the row's largest such product M (the header says 2^-26), so that a value of magnitude up to 448 adds at most
448 2^-28 M to the error beside that; a weight may be lost below 2^-62 of the largest, L 2^-62 in all; a scale of up to 2^-126 counts
as 2^-40, so that a value of such a page is off by up to 448 2^-40, whatever its bytes. The other bounds are those of
test_cache8_gpu.py: ds for a score, which changes every p by a factor within exp(+-2 ds), a rounding to bf16, fp32 sums.
"""
import math

import numpy as np
import pytest
import torch

import speculative_decoding_block_dflash_gb300 as dfl
from speculative_decoding_block_dflash_gb300 import build as build_mod
from test_cache8_gpu import E4M3, KERNELS, U16, U16H, U32, Attn, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build_mod.build()
    dfl.load_library()


def check(t, out, lse, kernel):
    tc = kernel == "tc"
    for b, (n, L) in enumerate(zip(t.queries, t.lens)):
        if n == 0:
            continue
        keys, values, w = t.request(b)
        vis = t.visible(b)
        q = t.q[b * t.T:b * t.T + n].double().cpu().numpy()
        got, got_l = (x[b * t.T:b * t.T + n].double().cpu().numpy() for x in (out, lse))
        for i in range(n):
            for h in range(t.hq):
                g = h // (t.hq // t.hkv)
                k, v, wj = keys[vis[i], g], values[vis[i], g], w[vis[i], g]
                s = t.scale * (k @ q[i, h])
                e = np.exp(s - s.max())
                p = e / e.sum()
                size = t.scale * (np.abs(k) @ np.abs(q[i, h])).max()
                ds = (t.d + 4) * U32 * size + 2.0 ** -17
                o, spread = p @ v, p @ np.abs(v)
                tol = U16 * np.abs(o) + 2.0 ** -133  # (bf16's least number)
                if tc:
                    ds += 2.0 ** -17 * t.scale * np.abs(q[i, h]).max() * np.abs(k).sum(axis=1).max()
                    ds += 2 * -(-t.d // 32) * 2.0 ** -21 * size
                    tol = tol + (U16H + 2.0 ** -9) * spread + L * 2.0 ** -28 * 448 * (p * wj).max()
                    tol = tol + 448 * 2.0 ** -40 * (wj <= 2.0 ** -126).any()
                tol = tol + (2 * ds + L * U32 + L * 2.0 ** -62) * spread
                err = np.abs(got[i, h] - o)
                assert np.all(err <= tol), f"request {b}, row {i}, {h}: off by {np.max(err / tol):.3g} bounds"
                l = s.max() + math.log(e.sum())
                assert abs(got_l[i, h] - l) <= ds + L * U32 + 2.0 ** -20 * (1 + abs(l)), f"request {b}, row {i}, {h}: lse"


def values_of(t, b, col, scale):
    """Value scale of a page of request b."""
    t.scales[1][int(t.table[b][col])] = scale


SHAPES = [(2, 4, 2, 128), (1, 16, 2, 64), (9, 8, 1, 512), (5, 4, 2, 256), (40, 4, 2, 128), (33, 4, 1, 64), (20, 8, 2, 256)]
FAR = [(-70, 70), (-126, 40), (-126, 50), (0, 100), (-126, 118), (-64, 0), (-40, 24), (-41, 23), (-125, -60), (60, 60), (-60, -60), (-90, -65),
       (80, 95), (-126, 60)]


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("T,hq,hkv,d", SHAPES)
def test_value_scales_far_apart(T, hq, hkv, d, kernel):
    """Small scales first, large ones first, and both in every tile of keys; scores of one size."""
    L = max(T, 300)
    for low, high in FAR:
        for order in (0, 1, 2):
            t = Attn([T], [L], T=T, hq=hq, hkv=hkv, d=d, seed=order + 1)
            cols = -(-L // t.page)
            for col in range(cols):
                second = (col * 2 >= cols, col * 2 < cols, col % 3 == 1)[order]
                values_of(t, 0, col, 2.0 ** (high if second else low))
            # (values of up to 2^8 times 2^118 are finite)
            t.caches[1].view(torch.uint8)[:] = t.caches[1].float().clamp(-128, 128).to(E4M3).view(torch.uint8)
            out, lse = t.call(kernel)
            assert t.error() == 0
            check(t, out, lse, kernel)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("T,hq,hkv,d", SHAPES)
def test_pages_without_a_scale_and_one_value(T, hq, hkv, d, kernel):
    """Scales of 0, as a page of zeros may have, beside a single page of values; and nothing but scales of 0."""
    L = max(T, 290)
    cols = -(-L // 16)
    for at in (0, 5, cols - 1):
        t = Attn([T], [L], T=T, hq=hq, hkv=hkv, d=d, seed=at)
        for col in range(cols):
            values_of(t, 0, col, 2.0 ** 10 if col == at else 0.0)
        out, lse = t.call(kernel)
        check(t, out, lse, kernel)
    t.scales[1][:] = 0.0
    out, lse = t.call(kernel)
    check(t, out, lse, kernel)
    t.caches[1].view(torch.uint8)[:] = 0
    out, lse = t.call(kernel)
    check(t, out, lse, kernel)
    assert (out == 0).all()


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("T,hq,hkv,d", SHAPES)
@pytest.mark.parametrize("low_first", [True, False])
def test_weights_that_undo_the_scales(T, hq, hkv, d, low_first, kernel):
    """Keys of small weight under large value scales: products of one size from scores that lie 70 powers of two apart."""
    L = max(T + 16, 320)
    t = Attn([T], [L], T=T, hq=hq, hkv=hkv, d=d, seed=7)
    t.q[:] = 1.0
    t.caches[0].view(torch.uint8)[:] = 0x38  # 1
    score = 70 * math.log(2) / (t.scale * d)
    for col in range(-(-L // t.page)):
        low = (col < 9) == low_first
        pg = int(t.table[0][col])
        t.scales[0][pg] = score if low else 0.0
        t.scales[1][pg] = 2.0 ** (-35 if low else 35)
    out, lse = t.call(kernel)
    check(t, out, lse, kernel)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("T,hq,hkv,d", [(1, 8, 2, 64), (40, 4, 2, 64)])
def test_split_requests_and_many_pieces(T, hq, hkv, d, kernel):
    """Far scales in some requests of many and in some pieces of a split one: what a piece keeps is its own."""
    nb = 240 if T == 1 else 120
    lens = [T + (37 * b) % 400 for b in range(nb)]
    t = Attn([T] * nb, lens, T=T, hq=hq, hkv=hkv, d=d, seed=3)
    for b in range(1, nb, 3):  # one scale throughout, far from the others'
        for col in range(-(-lens[b] // t.page)):
            values_of(t, b, col, 2.0 ** (-50 if b % 2 else 70))
    for b in range(0, nb, 3):
        for col in range(-(-lens[b] // t.page)):
            values_of(t, b, col, 2.0 ** (60 if (col + b) % 4 == 0 else -60))
    check(t, *t.call(kernel), kernel)
    t = Attn([T], [12000], T=T, hq=hq, hkv=hkv, d=d, seed=4)
    for col in range(300, 420):
        values_of(t, 0, col, 2.0 ** (-80 if col % 2 else 45))
    check(t, *t.call(kernel), kernel)
    assert t.error() == 0


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("T", [3, 40])
def test_rows_that_are_not_finite_beside_far_scales(T, kernel):
    t = Attn([T], [400], T=T, d=128, seed=1)
    for col in range(25):
        values_of(t, 0, col, 2.0 ** (70 if col == 4 else -70))
    good = t.call(kernel)
    check(t, *good, kernel)
    t.q[2, 1, 7] = math.nan
    out, lse = t.call(kernel)
    assert out[2, 1].isnan().all() and lse[2, 1].isnan()
    same = torch.ones(out.shape[:2], dtype=torch.bool, device="cuda")
    same[2, 1] = False
    assert torch.equal(out[same], good[0][same]) and torch.equal(lse[same], good[1][same])


@pytest.mark.parametrize("kernel", KERNELS)
def test_far_scales_under_masks(kernel):
    """Windows and trees: pages that some queries do not see, or nobody, have scales of their own."""
    for mask, window in (("causal", 100), ("tree", 60), ("full", 128), ("tree", 0)):
        for T in (6, 40):
            t = Attn([T, T], [500, T + 3], T=T, d=128, seed=T, mask=mask, window=window)
            for b in range(2):
                for col in range(-(-t.lens[b] // t.page)):
                    if not t.scales[1][int(t.table[b][col])].isnan().any():
                        values_of(t, b, col, 2.0 ** (-75 if col % 2 else 50))
            check(t, *t.call(kernel), kernel)
            assert t.error() == 0


def test_an_appended_infinity_has_one_meaning():
    """A page with a huge value: both kernels take its scale as it is."""
    T, hkv, d = 4, 2, 64
    t = Attn([T], [200], T=T, hq=4, hkv=hkv, d=d, seed=5)
    k, v = (torch.randn((200, hkv, d), generator=torch.Generator(device="cuda").manual_seed(i), device="cuda") for i in (1, 2))
    v[77, 0, 5] = 3e38
    table, lens = torch.from_numpy(t.table).cuda(), ints(t.lens)
    dfl.append_kv(k, v, *t.caches, table, lens, k_scale=t.scales[0], v_scale=t.scales[1])
    assert t.scales[1][int(t.table[0][77 // 16]), 0] == 2.0 ** 120
    for kernel in KERNELS:
        check(t, *t.call(kernel), kernel)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("T,hq,hkv,d", SHAPES)
@pytest.mark.parametrize("power", [116, -110])
def test_key_scales_that_undo_the_queries(T, hq, hkv, d, power, kernel):
    """Tiny queries on keys of huge scales, and the other way round: ordinary scores."""
    t = Attn([T], [max(T, 200)], T=T, hq=hq, hkv=hkv, d=d, seed=2)
    t.q *= 2.0 ** -power
    t.scales[0] *= 2.0 ** power
    out, lse = t.call(kernel)
    assert out.isfinite().all() and lse.isfinite().all()
    check(t, out, lse, kernel)
