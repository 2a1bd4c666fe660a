"""The plain definitions that the GPU tests compare with, on values that can be said by hand."""
import numpy as np
import pytest

import serve_ref as ref


def test_e4m3_values_and_rounding():
    assert ref.e4m3([0x7e, 0x38, 0x01, 0x08, 0xb8]).tolist() == [448.0, 1.0, 2.0 ** -9, 2.0 ** -6, -1.0]
    assert np.isnan(ref.e4m3([0x7f, 0xff])).all()
    every = np.arange(127, dtype=np.uint8)
    assert (ref.nearest8(ref.e4m3(every)) == every).all()
    # halfway between neighbours: the even one
    assert ref.nearest8(np.array([1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -10])).tolist() == [0x38, 0x3a, 0, 2]


def test_torch_rounds_alike():
    torch = pytest.importorskip("torch")
    x = np.random.RandomState(0).randn(4000) * np.exp(2 * np.random.RandomState(1).randn(4000))
    x = np.clip(x, -448, 448).astype(np.float32)
    got = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert (got == ref.nearest8(x.astype(np.float64))).all()


@pytest.mark.parametrize("top,want", [(0.0, 0.0), (448.0, 1.0), (449.0, 2.0), (224.0, 0.5), (1e-40, 2.0 ** -126),
                                      (3.0e38, 2.0 ** 120)])
def test_scales(top, want):
    assert ref.scale_for(top) == want


def test_a_rows_own_text():
    # 5 cached tokens, 4 drafted of which 0, 1, 3 are seen: own text 0..4, 5, 6, 8
    sees = np.array([True, True, False, True])
    assert np.flatnonzero(ref.text(sees, 5, None, 0)).tolist() == [0, 1, 2, 3, 4, 5, 6, 8]
    assert np.flatnonzero(ref.text(sees, 5, 4, 0)).tolist() == [4, 5, 6, 8]
    assert np.flatnonzero(ref.text(sees, 5, 2, 1)).tolist() == [0, 6, 8]
    assert np.flatnonzero(ref.text(sees, 5, 1, 6)).tolist() == [0, 1, 2, 3, 4, 5, 8]
    assert np.flatnonzero(ref.text(sees, 5, 8, 0)).tolist() == [0, 1, 2, 3, 4, 5, 6, 8]
    assert not ref.text(np.zeros(3, bool), 0, 4, 2).any()
