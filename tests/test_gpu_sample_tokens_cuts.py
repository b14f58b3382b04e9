"""sample_tokens where the number of CTAs that share a row changes: vocabularies next to what one, two, four and eight CTAs hold
with two of them on an SM, and next to the most that the call takes."""
import pytest

from test_gpu_sample_tokens import check, rows, settings

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [18991, 18992, 18993, 19279, 19280, 19281, 19968, 19969, 38560, 38561])
def test_many_rows_next_to_a_cut(cuda_lib, V):
    """(160 rows: more than SMs, so that the vocabulary alone decides.)"""
    l, u = rows(160, V, V)
    check(cuda_lib, l, u, **settings(160, V))


@pytest.mark.parametrize("V", [77120, 77121, 151936, 152064, 154240, 154241, 368639])
def test_long_rows_next_to_a_cut(cuda_lib, V):
    l, u = rows(40, V, V)
    check(cuda_lib, l, u, **settings(40, V))
    check(cuda_lib, l, u)
