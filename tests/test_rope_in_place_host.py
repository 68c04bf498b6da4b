"""q_out = q of gqa_rope_append needs the tokens of q back to back, as those of
q_out are: other strides are refused before any CUDA call."""
import pytest
import torch

from tests.test_packed_host import A, CUDA, SHAPE, rope

# (the addresses are not memory: what passes the checks must find no device)
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="a GPU is present")


@pytest.mark.parametrize("form", ["flat", "paged", "fp8"])
def test_stride_of_queries_rotated_in_place(form):
    assert rope(form, q=A, qo=A, qs=1024) == CUDA  # (no device here)
    assert rope(form, q=A, qo=A, qs=1536) == SHAPE
    assert rope(form, q=A, qo=A, qs=1536, total=1) == CUDA
    assert rope(form, q=A, qo=2 * A, qs=1536) == CUDA
