"""Attention reports a bad page of a request that drafts nothing, as it does a bad length."""
import numpy as np
import pytest

import speculative_decoding_verification_23_gb300 as sv
from test_gpu_tree import Tree

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("hq,dim,page", [(28, 128, 16), (4, 64, 3), (4, 256, 16)])
def test_a_bad_page_of_a_request_without_nodes(hq, dim, page):
    t = Tree(21, [4, 0, 0, 0, 6], [100, 90, 200, 50, 300], hq, 4, dim, page)
    want = t.reference()
    t.table[1, 2] = 1 << 20
    t.table[2, 199 // page] = -1
    t.ctx[3] = -5
    out, lse, st = sv.spec_tree_attention(t.args())
    page_bad, len_bad = sv.SPEC_STATUS_BAD_PAGE, sv.SPEC_STATUS_BAD_LEN
    assert st.tolist() == [0, page_bad, page_bad, len_bad, 0]
    assert np.all(np.abs(out.double().cpu().numpy() - want[0]) <= want[2])
    assert np.all(np.abs(lse.double().cpu().numpy() - want[1]) <= want[3])


def test_no_request_has_nodes():
    t = Tree(22, [0, 0, 0], [100, 0, 40], 4, 2, 64, 16)
    t.table[2, 1] = -1
    out, lse, st = sv.spec_tree_attention(t.args())
    assert st.tolist() == [0, 0, sv.SPEC_STATUS_BAD_PAGE] and out.shape == (0, 4, 64)
