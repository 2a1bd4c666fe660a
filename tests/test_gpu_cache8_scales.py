"""Values under scale 0 in an 8-bit cache that are not all zeros: what commitment writes and what attention makes of it,
in both attention kernels (blocks of 8 tokens are for warp tiles)."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import speculative_decoding_verification_23_gb300 as sv  # noqa: E402
from test_gpu_serve import DEV, DT, Case, i32  # noqa: E402


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("window", [None, 100])
@pytest.mark.parametrize("block", [16, 8])
@pytest.mark.parametrize("nodes", [2, 40, 150])
@pytest.mark.parametrize("other", [False, True])
def test_nan_beside_zeros(other, nodes, block, window, dtype):
    """Values that are all 0 but for an infinity are committed under scale 0, the infinity as NaN: the rows that see it
    have NaN there, and all else is as with a 0 in its place.  `other`: whether there is an infinity among the drafted
    values too."""
    ctx, group, dim = 200, 2, 64
    # token 101 is in the window of the first rows alone
    j, channel = (101 if window else 77), 9
    c = Case(dtype=dtype, dim=dim, kv=1, group=group, page=16, ctx=[ctx], nodes=[nodes], chain=True, block=block, window=window,
             seed=nodes)
    cache = sv.make_cache8(c.k, c.v, *c.scales)
    v = torch.zeros(ctx, 1, dim, dtype=DT[dtype], device=DEV)
    v[:, 0] = torch.randn(ctx, dim, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).to(DT[dtype])
    first = j // 16 * 16
    v[first:first + 16] = 0
    if other:
        c.v_new[1, 0, 3] = float("inf")

    def commit_and_attend(x):
        v[j, 0, channel] = x
        length, status = sv.spec_cache8_commit(sv.make_cache8_commit_args(
            k_new=v, v_new=v, cu_nodes=i32([0, ctx]), path=i32([range(ctx)]), path_len=i32([ctx]), cache=cache,
            block_table=i32(c.table), ctx_len=i32([0])))
        assert length.tolist() == [ctx] and status.tolist() == [0]
        assert (c.scales[1][c.table[0, j // 16], j % 16 // block] == 0).all()
        c.k.view(torch.uint8).copy_(keys)
        return c.run()

    keys = c.k.view(torch.uint8).clone()
    c.scales[0].fill_(1 / 64)
    was = [x.clone() for x in commit_and_attend(0.0)]
    c.scales[0].fill_(1 / 64)
    out, lse, status = commit_and_attend(float("inf"))
    # the keys' scales were written alike both times
    assert status.tolist() == [0] and torch.equal(lse, was[1])
    sees = torch.tensor([window is None or j >= ctx + i + 1 - window for i in range(nodes)], device=DEV)
    assert sees.any() and (window is None or not sees.all())
    assert out[sees][..., channel].isnan().all() and not out[~sees][..., channel].isnan().any()
    rest = torch.arange(dim, device=DEV) != channel
    assert torch.equal(out[..., rest], was[0][..., rest]) and torch.equal(out[~sees], was[0][~sees])
