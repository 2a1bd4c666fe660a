"""Queries of attention over an 8-bit cache, where a bf16 row is scaled by its largest channel: channels of very different
sizes, odd numbers of rows, and the same bits again."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from test_gpu_serve import DEV, Case, gen  # noqa: E402

SIZES = [(128, 4, 64), (64, 8, 40), (128, 2, 30), (128, 2, 60), (64, 2, 50), (64, 1, 17)]


def long_case(dtype, dim, group, nodes, kv=8, seed=4, **kw):
    rng, B = np.random.RandomState(seed), 12
    return Case(dtype=dtype, dim=dim, kv=kv, group=group, page=16, ctx=rng.randint(1000, 9000, B).tolist(), nodes=[nodes] * B,
                chain=False, seed=seed, **kw)


@pytest.mark.parametrize("dim,group,nodes", SIZES)
def test_bf16_gives_the_same_bits_again(dim, group, nodes):
    """The queries' scales among them: channels of very different sizes, and odd numbers of rows."""
    c = long_case("bf16", dim, group, nodes - 1 + nodes % 2, block=16)
    c.q[..., ::17] *= 1e4
    c.q[..., 1::17] *= 1e-9
    args = c.args()
    want = [x.clone() for x in c.run(args)]
    for _ in range(60):
        assert all(torch.equal(x, y) for x, y in zip(c.run(args), want))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("nodes,group", [(3, 1), (5, 7), (31, 3), (43, 3)])
def test_queries_whose_channels_differ_in_size(nodes, group, dim):
    """bf16 rows are scaled by their largest channel, wherever it lies; odd numbers of rows."""
    c = Case(dtype="bf16", dim=dim, kv=2, group=group, page=16, ctx=[200, 33], nodes=[nodes, nodes], chain=True, block=16, seed=3)
    at = torch.randint(0, dim, c.q.shape[:2], generator=gen(1), device=DEV)
    size = 2.0 ** torch.randint(-60, 60, c.q.shape[:2], generator=gen(2), device=DEV)
    c.q *= 2.0 ** -40
    c.q.scatter_(2, at[..., None], (size * 1e-20)[..., None].to(c.q.dtype))
    c.check()
