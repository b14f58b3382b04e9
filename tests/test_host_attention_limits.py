"""Limits of kv_paged_attention's lengths, and the fetching lanes' arithmetic at them. CPU only."""
import pytest

import paged_quantized_expert_gb300 as pqe
from test_host_attention_args import BAD, _attend, _cache

TILE, BLOCK = 64, 16


def test_longest_table():
    """Token counts are kept in 32 bits, some steps past the last token: 2^31 - 2^16 is the most that a table may describe."""
    lib = pqe.load()
    big = dict(page_size=1024, n_kv=1, page_stride=pqe.pqe_kv_page_bytes(1024, 1, 64))
    most = (2 ** 31 - 2 ** 16) // 1024
    assert _attend(lib, _cache(**big), max_pages=most, B=0) == 0
    for pages in (most + 1, 2 ** 21 - 1, 2 ** 21):
        assert _attend(lib, _cache(**big), max_pages=pages, B=0) == BAD


@pytest.mark.parametrize("length", [1, 1000, 2 ** 30 - 1, 2 ** 30, 2 ** 30 + 5000, 2 ** 31 - 2 ** 16])
def test_lanes_that_copy_nothing_never_look_at_the_table(length):
    """Lanes behind those that copy a tile's blocks start below zero and move with the others, a tile at a time: taken as
    unsigned, their token lies beyond every length, at the first tile as at the last."""
    tiles = -(-length // TILE)
    for steps in (0, 1, tiles - 1, tiles):
        j = -2 ** 31 + steps * TILE
        assert -2 ** 31 <= j < 0  # no wrap
        assert j % 2 ** 32 >= length
