"""Beam selection of more rows than a call lists, and of rows that end."""
import pytest

import speculative_decoding_verification_23_gb300 as sv
from test_gpu_tree import TYPES, check_beams

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("B,W,keep,V,dtype", [
    (2100, 1, 3, 500, "bf16"), (300, 8, 8, 1001, "fp32"), (60, 40, 5, 20011, "bf16"), (33, 64, 64, 300, "bf16"),
])
def test_many_rows(B, W, keep, V, dtype):
    g = torch.Generator(device="cuda").manual_seed(V + keep)
    z = (3 * torch.randn(B * W, V + (-V) % 8, generator=g, device="cuda")).to(TYPES[dtype])
    z[:, V:] = float("nan")
    cum = -4 * torch.rand(B, W, generator=g, device="cuda")
    check_beams(z, V, cum, keep)
    ended = (torch.rand(B, W, generator=g, device="cuda") < 0.5).int()
    ended[1] = 1                    # a request without a row to read
    cum[2] = -float("inf")          # and one without a beam
    ended[-1] = 0
    z[ended.flatten().bool()] = float("nan")
    check_beams(z, V, cum, keep, ended, V - 1)


def test_a_request_of_many_that_has_no_number():
    g = torch.Generator(device="cuda").manual_seed(9)
    z = torch.randn(2400, 808, generator=g, device="cuda")
    z[1203, 777] = float("nan")
    cum = torch.zeros(300, 8, device="cuda")
    s, p, t, st = sv.spec_beam_select(sv.make_beam_args(logits=z, V=808, scores=cum, keep=4))
    want = [0] * 300
    want[150] = sv.SPEC_STATUS_BAD_LOGITS
    assert st.tolist() == want
    assert torch.all(torch.isneginf(s[150])) and torch.all(p[150] == -1) and torch.all(t[150] == -1)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_whose_maximum_comes_late(dtype):
    """The sum of a row is as exact where it is one logit's that stands far above those before it."""
    g = torch.Generator(device="cuda").manual_seed(21)
    V = 49488
    z = 12 * torch.randn(100, V, generator=g, device="cuda")
    z[:50] = z[:50].sort(1).values                                   # ascending
    z[50:60, V // 2:] += torch.linspace(5, 45, 10, device="cuda")[:, None]
    check_beams(z.to(TYPES[dtype]), V, -torch.rand(4, 25, generator=g, device="cuda"), 5)
