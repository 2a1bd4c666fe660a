"""Attention over an 8-bit cache with dozens of tiles a CTA, in segments of all lengths: each tile's keys and values
against 64 bits."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import serve_ref as ref  # noqa: E402
from test_gpu_cache8_queries import long_case  # noqa: E402
from test_gpu_serve import DEV, gen  # noqa: E402


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,group,nodes,block", [(128, 4, 20, 16), (64, 8, 11, 16), (128, 2, 63, 16), (128, 2, 129, 16),
                                                   (64, 1, 7, 16), (128, 2, 9, 8), (96, 1, 17, 16)])
def test_values_of_a_few_pages(dim, group, nodes, block, dtype):
    """Values are 0 but for one page in 30, so the bound, which is relative to what the values add up, is that of few
    keys: a tile with another's keys or values passes it by far.  Two choices of pages, of some requests and heads."""
    c = long_case(dtype, dim, group, nodes, block=block)
    full = c.v.clone()
    k = ref.e4m3(c.k.view(torch.uint8).cpu().numpy())
    q, k_new, v_new = (ref.f64(x) for x in (c.q, c.k_new, c.v_new * 0))
    c.v_new.zero_()
    scales = [ref.f64(x) for x in c.scales]
    for seed in range(2):
        keep = torch.rand(c.v.shape[0], generator=gen(seed), device=DEV) < 1 / 30
        c.v.view(torch.uint8).copy_(full.view(torch.uint8) * keep[:, None, None, None])
        v = ref.e4m3(c.v.view(torch.uint8).cpu().numpy())
        out, lse, status = c.run()
        assert status.tolist() == [0] * 12
        rng = np.random.RandomState(seed)
        for b, g in zip(rng.choice(12, 3, replace=False), rng.choice(8, 3, replace=False)):
            # the first, the last and one of the nodes between
            rows = [c.cu[b], c.cu[b] + rng.randint(nodes), c.cu[b + 1] - 1]
            for row in rows:
                # a chain of the nodes that the row sees, itself the last
                tree = ref.bits(c.mask[row].view(np.int32), nodes)
                seen = c.cu[b] + np.flatnonzero(tree)
                hq = slice(g * group, (g + 1) * group)
                mask = np.full((len(seen), (len(seen) + 31) // 32), -1, np.int32)
                one = np.zeros((len(seen), group, dim))
                one[-1] = q[row, hq]
                w = ref.attention(one, k_new[seen, g:g + 1], v_new[seen, g:g + 1], [0, len(seen)], k[:, :, g:g + 1],
                                  v[:, :, g:g + 1], 16, c.table[b:b + 1], c.ctx[b:b + 1], mask, dim ** -0.5, dtype,
                                  scales=[s[:, :, g:g + 1] for s in scales], block=block)
                w_out, w_lse, t_out, t_lse = (x[-1] for x in w)
                got = ref.f64(out[row, hq])
                assert (np.abs(got - w_out) <= t_out).all(), (np.abs(got - w_out) / t_out).max()
                assert (np.abs(ref.f64(lse[row, hq]) - w_lse) <= t_lse).all()
