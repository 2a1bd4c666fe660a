"""Angles of the position rotation against 64 bits: frequencies of many turns a position, and those that are no number."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import serve_ref as ref  # noqa: E402
import speculative_decoding_verification_23_gb300 as sv  # noqa: E402
from test_gpu_serve import DEV, DT, gen, normal  # noqa: E402


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,rot,interleaved", [(64, 64, False), (128, 24, True)])
@pytest.mark.parametrize("size", [1.0, 7.3, 1000.0, 60000.0])
def test_frequencies_of_many_turns(size, dim, rot, interleaved, dtype):
    """Positions and frequencies are whole multiples of powers of two of at most 28 and 24 bits, so their product and the
    reference's angle are exact."""
    g = gen(int(size))
    x = normal(g, 50, 6, dim, dtype=DT[dtype])
    pos = torch.randint(-(1 << 28) + 1, 1 << 28, (50,), generator=g, device=DEV, dtype=torch.int32)
    freq = size * (0.5 + torch.rand(rot // 2, generator=g, device=DEV))
    freq[::3] *= -1
    y, _ = sv.spec_norm_rotate(sv.make_rotate_args(q=x, k=None, positions=pos, inv_freq=freq, interleaved=interleaved))
    want, tol = ref.rotate(ref.f64(x), None, pos.cpu().numpy(), freq.cpu().numpy(), float(np.float32(1e-6)), interleaved, dtype)
    assert (np.abs(ref.f64(y) - want) <= tol).all(), (np.abs(ref.f64(y) - want) / tol).max()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("rot", [64, 24])
def test_frequencies_that_are_no_number(rot, bad):
    """Their pairs are NaN, the others as without them."""
    g = gen(rot)
    q, k = normal(g, 40, 5, 64, dtype=torch.bfloat16), normal(g, 40, 2, 64, dtype=torch.bfloat16)
    pos = torch.arange(40, device=DEV, dtype=torch.int32)
    freq = torch.rand(rot // 2, generator=g, device=DEV)
    odd = freq.clone()
    odd[5] = bad
    want = sv.spec_norm_rotate(sv.make_rotate_args(q=q, k=k, positions=pos, inv_freq=freq))
    got = sv.spec_norm_rotate(sv.make_rotate_args(q=q, k=k, positions=pos, inv_freq=odd))
    pair = torch.zeros(64, dtype=torch.bool, device=DEV)
    pair[[5, 5 + rot // 2]] = True
    for x, y in zip(got, want):
        assert x[..., pair].isnan().all() and torch.equal(x[..., ~pair], y[..., ~pair])
