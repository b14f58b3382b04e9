"""kv_paged_attention at the ends of its ranges: widest windows, longest caches, what a masked token or a
token of no weight may hold. Bounds as in test_gpu_kv_attention.py, whose cases and comparison are used; where one
is wider, its derivation stands at the test."""
import pytest
import torch

import attention_ref as ref
from test_gpu_kv_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, params=["few", "many"])
def kernel(request, cuda_lib):
    cuda_lib.pqe_test_set_attention_kernel({"few": 1, "many": 2}[request.param])
    yield request.param
    cuda_lib.pqe_test_set_attention_kernel(0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ms,lens", [([6, 300], [1, 200]), ([70, 3], [67, 0]), ([140], [129])])
def test_widest_window_and_more_queries_than_tokens(cuda_lib, ms, lens, d):
    """A window that stands for none, where the first queries' positions are below zero: they see nothing, the others all
    tokens up to their own."""
    c = Case(cuda_lib, ms, lens, 8, 2, d, 16, seed=d)
    c.check(window=2 ** 31 - 1)
    wide, wide_lse = c.run(window=2 ** 31 - 1)
    none, none_lse = c.run()
    assert torch.equal(wide, none) and torch.equal(wide_lse, none_lse)
