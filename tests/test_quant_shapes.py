"""Shapes that the read-back of a quantised cache takes and refuses, before anything
reaches the GPU."""
import pytest
import torch

import paged_kv_cache_106_gb300 as pk
from tests.test_draft_arguments import Fake, one_gpu  # noqa: F401  (the fixture)
from tests.test_quant_refusals import _i64, _py_read


@pytest.mark.parametrize("shape", [(3, 128), (384,), (6, 64), (3, 64, 2), (3, 1, 2, 64), (4, 2, 16, 64)])
def test_rows_have_heads_and_dimensions(shape, one_gpu):  # noqa: F811
    with pytest.raises(ValueError, match="k is"):
        _py_read(k=Fake(shape))
    with pytest.raises(ValueError, match="v is"):
        _py_read(v=Fake(shape))


@pytest.mark.parametrize("shape", [(3, 2, 16, 64), (8, 1, 16, 64), (4, 16, 2, 64), (64, 2, 64), (16 * 2 * 64 * 4,)])
def test_values_go_to_blocks_like_the_keys(shape, one_gpu):  # noqa: F811
    with pytest.raises(ValueError, match="v is"):
        _py_read(out_slots=_i64(3), k=Fake((4, 2, 16, 64)), v=Fake(shape))
    with pytest.raises(pk.PagedKVError, match="misaligned"):       # more rows or blocks than needed are taken
        _py_read(out_slots=_i64(3), k=Fake((4, 2, 16, 64)), v=Fake((5, 2, 16, 64)))
    with pytest.raises(pk.PagedKVError, match="misaligned"):
        _py_read(k=Fake((5, 2, 64)), v=Fake((3, 2, 64)))


def test_as_many_as_are_read(one_gpu):  # noqa: F811
    with pytest.raises(ValueError, match="v"):
        _py_read(v=Fake((2, 2, 64)))
    with pytest.raises(ValueError, match="v"):
        _py_read(v=Fake((3, 2, 64), torch.bfloat16))
    with pytest.raises(pk.PagedKVError, match="NULL"):
        _py_read(v=None, status=None)
