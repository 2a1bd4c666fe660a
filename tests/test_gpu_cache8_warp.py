"""Attention over an 8-bit cache on warp tiles, which take the calls that the tensor-memory kernel does not: heads of 96,
192 and 256 channels, blocks and pages that are no multiple of 16, scales that are not positive.  The cases where it can
go wrong; error bounds are derived in serve_ref.py."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import serve_ref as ref  # noqa: E402
import speculative_decoding_verification_23_gb300 as sv  # noqa: E402
from test_gpu_serve import Case  # noqa: E402

CONFIGS = [dict(dim=128, page=16, block=8), dict(dim=96, page=16, block=16), dict(dim=256, page=24, block=24),
           dict(dim=64, page=10, block=5)]
configs = pytest.mark.parametrize("config", range(len(CONFIGS)))


@configs
@pytest.mark.parametrize("nodes,chain", [(1, True), (9, True), (40, False)])
def test_scales_of_zero(config, nodes, chain):
    Case(dtype="bf16", kv=2, group=4, ctx=[300, 0, 129], nodes=[nodes, nodes, 1], chain=chain, zero_scales=True, seed=1,
         **CONFIGS[config]).check()


@configs
@pytest.mark.parametrize("nodes", [1, 30])
def test_a_large_window_hides_nothing(config, nodes):
    c = Case(dtype="bf16", kv=2, group=4, ctx=[400, 37], nodes=[nodes, max(1, nodes // 2)], chain=False, seed=3, window=1 << 30,
             sinks=7, **CONFIGS[config])
    a = c.run()
    c.window, c.sinks = None, 0
    assert all(torch.equal(x, y) for x, y in zip(a, c.run()))


@configs
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("nodes,chain", [(2, True), (40, False)])
def test_what_a_window_hides_never_reaches(config, nodes, chain, dtype):
    """NaN in every hidden slot, under scales that are NaN where a block is hidden whole, and no pages between."""
    window, sinks, ctx = 100, 20, [1000, 250]
    c = Case(dtype=dtype, kv=2, group=4, ctx=ctx, nodes=[nodes, nodes], chain=chain, seed=9, window=window, sinks=sinks,
             **CONFIGS[config])
    page, block = c.page, c.block
    clean = [x.clone() for x in c.run()]
    for b, n in enumerate(ctx):
        for j in range(sinks, n - window):
            for x in (c.k, c.v):
                x.view(torch.uint8)[c.table[b, j // page], j % page] = 0x7f
            if j % block == 0 and j + block <= n - window:
                for s in c.scales:
                    s[c.table[b, j // page], j % page // block] = float("nan")
        for p in range(-(-sinks // page), (n - window) // page):
            c.table[b, p] = -1 if p % 2 else 1 << 30
    assert all(torch.equal(x, y) for x, y in zip(clean, c.run()))
    # NaN in a value that the first rows of request 0 see and the last ones do not
    j = 1000 - window + 1
    c.v.view(torch.uint8)[c.table[0, j // page], j % page] = 0x7f
    out, lse, _ = c.run()
    for i in range(nodes):
        tree = (np.arange(nodes) <= i) if c.mask is None else ref.bits(c.mask[i].view(np.int32), nodes)
        sees = ref.text(tree, 1000, window, sinks)[j]
        assert bool(out[i].isnan().all()) == bool(sees)
        if not sees:
            assert torch.equal(out[i], clean[0][i])
    assert torch.equal(out[nodes:], clean[0][nodes:]) and torch.equal(lse, clean[1])


@configs
@pytest.mark.parametrize("nodes", [2, 40])
def test_masks_that_leave_nothing(config, nodes):
    c = Case(dtype="fp16", kv=1, group=4, ctx=[0, 40], nodes=[nodes, nodes], chain=False, seed=4, window=30, **CONFIGS[config])
    c.mask[0] = 0
    c.mask[nodes - 1] = 0
    c.mask[nodes + 1] = 0
    c.check()
    out, lse, _ = c.run()
    assert (out[0] == 0).all() and (lse[0] == -math.inf).all()


@configs
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("nodes", [3, 40])
def test_infinities_and_nan_among_drafted_values(config, dtype, nodes):
    c = Case(dtype=dtype, kv=1, group=4, ctx=[70], nodes=[nodes], chain=True, seed=2, **CONFIGS[config])
    clean = [x.clone() for x in c.run()]
    c.v_new[1, 0, 7], c.v_new[2, 0, 9] = float("inf"), float("nan")
    out, lse, status = c.run()
    assert status.tolist() == [0] and torch.equal(lse, clean[1]) and torch.equal(out[0], clean[0][0])
    assert (out[1:, :, 7] == math.inf).all() and out[2:, :, 9].isnan().all() and not out[:2, :, 9].isnan().any()


@configs
@pytest.mark.parametrize("nodes", [2, 40])
def test_bf16_beyond_the_range_of_fp16(config, nodes):
    c = Case(dtype="bf16", kv=2, group=4, ctx=[90, 0], nodes=[nodes, nodes], chain=False, seed=6, **CONFIGS[config])
    c.q.mul_(1e-20)
    c.k_new.mul_(1e20)
    c.v_new.mul_(1e25)
    for s in c.scales:
        s.mul_(1e15)
    c.check()
    c = Case(dtype="bf16", kv=1, group=4, ctx=[33], nodes=[nodes], chain=False, seed=7, **CONFIGS[config])
    c.q.mul_(1e9)
    c.k_new.mul_(1e-9)
    c.v_new.mul_(1e-12)
    for i, s in enumerate(c.scales):
        s.mul_(1e-9 if i == 0 else 1e-12)
    c.check()


@configs
@pytest.mark.parametrize("nodes", [2, 40])
def test_bad_lengths_and_pages(config, nodes):
    c = Case(dtype="bf16", kv=2, group=4, ctx=[100, 60, 500, 32], nodes=[nodes] * 4, chain=True, seed=8, window=90, sinks=3,
             **CONFIGS[config])
    w_out, w_lse, t_out, t_lse = c.want()
    c.ctx[1] = c.table.shape[1] * c.page + 1     # past its table
    c.table[2, 480 // c.page] = c.k.shape[0]     # within the window
    out, lse, status = c.run()
    assert status.tolist() == [0, sv.SPEC_STATUS_BAD_LEN, sv.SPEC_STATUS_BAD_PAGE, 0]
    for b in (1, 2):
        assert out[b * nodes:(b + 1) * nodes].isnan().all() and lse[b * nodes:(b + 1) * nodes].isnan().all()
    # The others' bits may change: a request of a bad length has no tiles, the CTAs share the rest otherwise, and an item
    # that is cut elsewhere is added up in another order.
    for b in (0, 3):
        rows = slice(b * nodes, (b + 1) * nodes)
        assert (np.abs(ref.f64(out)[rows] - w_out[rows]) <= t_out[rows]).all()
        assert (np.abs(ref.f64(lse)[rows] - w_lse[rows]) <= t_lse[rows]).all()


@configs
@pytest.mark.parametrize("window,sinks", [(None, 0), (8000, 70)])
def test_a_long_context_is_split(config, window, sinks):
    Case(dtype="bf16", kv=1, group=2, ctx=[9000, 3], nodes=[10, 2], chain=False, window=window, sinks=sinks, seed=11,
         **CONFIGS[config]).check()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("scale", [-0.07, 0.0, -1e-30])
@pytest.mark.parametrize("nodes,chain", [(1, True), (40, False)])
@pytest.mark.parametrize("window", [None, 50])
def test_scales_of_scores_that_are_not_positive(window, nodes, chain, scale, dtype):
    c = Case(dtype=dtype, dim=128, kv=2, group=4, page=16, ctx=[300, 0, 129], nodes=[nodes, nodes, 1], chain=chain, block=16,
             window=window, sinks=3 if window else 0, seed=5)
    out, lse, status = c.run(c.args(scale=scale))
    assert status.tolist() == [0, 0, 0]
    k, v = (ref.e4m3(x.view(torch.uint8).cpu().numpy()) for x in (c.k, c.v))
    w_out, w_lse, t_out, t_lse = ref.attention(
        ref.f64(c.q), ref.f64(c.k_new), ref.f64(c.v_new), c.cu, k, v, c.page, c.table, c.ctx,
        None if c.mask is None else c.mask.view(np.int32), scale, dtype, window, c.sinks, [ref.f64(x) for x in c.scales], c.block)
    assert (np.abs(ref.f64(lse) - w_lse) <= t_lse).all() and (np.abs(ref.f64(out) - w_out) <= t_out).all()
