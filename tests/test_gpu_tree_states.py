"""Beams' states whose layers, requests and beams are as many."""
import pytest

import speculative_decoding_verification_23_gb300 as sv

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def test_as_many_layers_as_requests_and_beams():
    n = 4
    src = torch.arange(n ** 4, device="cuda", dtype=torch.float32).view(n, n, n, n)
    parents = torch.tensor([[3, 1, 0, 0], [1, 2, 2, 0], [0, 0, 3, 1], [2, 2, 1, 3]], dtype=torch.int32, device="cuda")
    rows = torch.arange(n, device="cuda")[:, None]
    with pytest.raises(ValueError):
        sv.make_reorder_args(parents=parents, beams=n, states=[(src, torch.empty_like(src))])
    for layered, want in ((False, src[rows, parents.long()]), (True, src[:, rows, parents.long()])):
        dst = torch.empty_like(src)
        sv.spec_beam_reorder(sv.make_reorder_args(parents=parents, beams=n, states=[(src, dst)], layered=layered))
        assert torch.equal(dst, want)
    a, b, flat = torch.empty_like(src), torch.empty_like(src), src[0]
    c = torch.empty_like(flat)
    sv.spec_beam_reorder(sv.make_reorder_args(parents=parents, beams=n, states=[(src, a), (src, b), (flat, c)],
                                              layered=[True, False, False]))
    assert torch.equal(a, src[:, rows, parents.long()]) and torch.equal(b, src[rows, parents.long()])
    assert torch.equal(c, flat[rows, parents.long()])
    with pytest.raises(ValueError):
        sv.make_reorder_args(parents=parents, beams=n, states=[(src, a)], layered=[True, False])
