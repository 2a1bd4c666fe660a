"""Commitment to blocks of an 8-bit cache that hold tokens under scales at the lower end of fp32."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import speculative_decoding_verification_23_gb300 as sv  # noqa: E402
from test_gpu_serve import DEV, commit_args, commit_case, commit_want, same_bytes  # noqa: E402


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("new", [0.0, 1.0])
def test_scales_whose_inverse_is_infinite(new, dtype):
    """A block that holds tokens under a scale below 2^-128 keeps it where only zeros come to it, which are bytes of 0."""
    c = commit_case(dtype=dtype, layers=2, kv=2, dim=64, page=16, block=16, ctx=[5], nodes=[4], accepted=[4], seed=3, sizes=False)
    for x in (c["k_new"], c["v_new"]):
        x.mul_(new)
    for s in (c["ks"], c["vs"]):
        s.fill_(1e-40)
    page = c["table"][0, 0]
    before = c["k"].view(torch.uint8)[:, page].clone()
    want = commit_want(c) if new else None
    _, status = sv.spec_cache8_commit(commit_args(c))
    assert status.tolist() == [0]
    if new:
        assert same_bytes(c["k"], want[0][0]) and np.array_equal(c["ks"].cpu().numpy(), want[0][1])
        return
    for x, s in ((c["k"], c["ks"]), (c["v"], c["vs"])):
        assert (x.view(torch.uint8)[:, page, 5:9] & 0x7f == 0).all() and (s == torch.tensor(1e-40, device=DEV)).all()
    assert torch.equal(c["k"].view(torch.uint8)[:, page, :5], before[:, :5])
