"""The form of a beam's states: with an axis of layers before the request's or
without, by shapes where they tell and by the caller's word where not."""
import pytest

from speculative_decoding_verification_23_gb300 import tree

torch = pytest.importorskip("torch")


class OnDevice:
    """A CPU tensor that passes for a CUDA one: no memory is touched."""
    is_cuda = True

    def __init__(self, *shape):
        self.t = torch.zeros(shape)

    def __getattr__(self, name):
        return getattr(self.t, name)


def form(src, dst, B, W, keep, layered=None):
    s = tree._state(OnDevice(*src), OnDevice(*dst), B, W, keep, layered)
    return s.outer, s.row_bytes, s.src_outer, s.src_batch, s.src_beam, s.dst_outer, s.dst_batch, s.dst_beam


FLAT = (1, 64, 0, 256, 64, 0, 256, 64)      # [4, 4, 4, 4]: B, W, then rows of 16 floats
LAYERED = (4, 16, 256, 64, 16, 256, 64, 16)  # layers, B, W, then rows of 4 floats


def test_a_shape_of_both_forms_needs_a_word():
    with pytest.raises(ValueError, match="layered"):
        form((4, 4, 4, 4), (4, 4, 4, 4), 4, 4, 4)
    assert form((4, 4, 4, 4), (4, 4, 4, 4), 4, 4, 4, False) == FLAT
    assert form((4, 4, 4, 4), (4, 4, 4, 4), 4, 4, 4, True) == LAYERED
    with pytest.raises(ValueError, match="layered"):
        form((4, 4, 4), (4, 4, 4), 4, 4, 4)


def test_a_shape_of_one_form_needs_none():
    assert form((4, 4, 5), (4, 4, 5), 4, 4, 4)[:2] == (1, 20)
    assert form((3, 4, 4, 5), (3, 4, 4, 5), 4, 4, 4)[:2] == (3, 20)
    assert form((4, 4, 4, 5), (4, 4, 2, 5), 4, 4, 2)[:2] == (4, 20)    # two beams kept: the third axis is the beams'
    assert form((4, 4), (4, 2), 4, 4, 2)[:2] == (1, 4)


@pytest.mark.parametrize("src,dst,layered", [((4, 4, 5), (4, 4, 5), True), ((3, 4, 4, 5), (3, 4, 4, 5), False),
                                             ((3, 4, 4, 5), (2, 4, 4, 5), None), ((2, 3, 4, 4), (2, 3, 4, 4), None),
                                             ((4,), (4,), None)])
def test_other_shapes_are_refused(src, dst, layered):
    with pytest.raises(ValueError, match="axis before"):
        form(src, dst, 4, 4, 4, layered)
