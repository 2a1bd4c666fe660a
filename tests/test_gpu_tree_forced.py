"""Beams that are left one token each: its log-probability is 0, so a beam
keeps its score as it is, and equal scores go to the lowest beam."""
import pytest

import speculative_decoding_verification_23_gb300 as sv
from test_gpu_tree import TYPES, check_beams

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def forced(seed, B, W, V, dtype, rest):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.full((B * W, V + (-V) % 8), rest, device="cuda")
    at = torch.randint(0, V, (B * W,), generator=g, device="cuda")
    z[torch.arange(B * W, device="cuda"), at] = 12 * torch.randn(B * W, generator=g, device="cuda")
    return z.to(TYPES[dtype]), at.view(B, W).int()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rest", [-float("inf"), -3.3e38, -1e4])
@pytest.mark.parametrize("B,W,V", [(3, 5, 1), (40, 17, 1000), (5, 8, 152064), (300, 8, 300), (1, 64, 20011)])
def test_one_allowed_token_keeps_the_score(B, W, V, rest, dtype):
    z, at = forced(V + W, B, W, V, dtype, rest)
    cum = -torch.arange(W, device="cuda").div(3, rounding_mode="floor").float().expand(B, W).contiguous() / 7
    s, p, t, st = sv.spec_beam_select(sv.make_beam_args(logits=z, V=V, scores=cum, keep=W))
    assert st.tolist() == [0] * B
    assert torch.equal(s, cum)                                       # as they are, in order
    assert torch.equal(p, torch.arange(W, device="cuda").int().expand(B, W))
    assert torch.equal(t, at)
    # and beside ended beams of the same score
    ended = torch.zeros(B, W, dtype=torch.int32, device="cuda")
    ended[:, ::2] = 1
    s, p, t, st = sv.spec_beam_select(sv.make_beam_args(logits=z, V=V, scores=cum, keep=W, finished=ended, end_token=0))
    assert torch.equal(s, cum) and torch.equal(p, torch.arange(W, device="cuda").int().expand(B, W))
    assert torch.equal(t, torch.where(ended.bool(), torch.zeros_like(at), at))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_likely_token_never_gains(dtype):
    """A log-probability is at most 0, also where all but one token are far below."""
    g = torch.Generator(device="cuda").manual_seed(7)
    V = 5003
    z = torch.randn(64 * 8, V + 5, generator=g, device="cuda")
    z[torch.arange(512, device="cuda"), torch.randint(0, V, (512,), generator=g, device="cuda")] = torch.linspace(
        10, 60, 512, device="cuda")
    z = z.to(TYPES[dtype])
    cum = torch.zeros(64, 8, device="cuda")
    s = sv.spec_beam_select(sv.make_beam_args(logits=z, V=V, scores=cum, keep=8))[0]
    assert float(s.max()) <= 0
    want = torch.log_softmax(z[:, :V].double(), 1).amax(1).view(64, 8).sort(1, descending=True).values
    assert float((s[:, 0].double() - want[:, 0]).abs().max()) <= 2.0 ** -20
    check_beams(z[:64], V, -torch.rand(8, 8, generator=g, device="cuda"), 8)
