"""Sizes of the page calls whose sums would not fit 32 bits are refused before any launch (no GPU)."""
import pytest

import gqa_decode_attention_kv_gb300 as gq
from gqa_decode_attention_kv_gb300 import build as gbuild

UNSUPPORTED, WORKSPACE = 2, 3


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gq.load()


@pytest.mark.parametrize("per_row", [False, True])
@pytest.mark.parametrize("batch,max_blocks,expect", [(1 << 20, 2048, UNSUPPORTED), (1 << 17, 1 << 14, UNSUPPORTED),
                                                     (32, (1 << 27) - 1, UNSUPPORTED), (17, (1 << 27) - 1, UNSUPPORTED),
                                                     (16, (1 << 27) - 1, WORKSPACE), (1 << 20, 2047, WORKSPACE)])
def test_reserve_over_tables_of_2_31_entries(lib, batch, max_blocks, expect, per_row):
    """A row may lack max_blocks pages, so the ranks reach batch * max_blocks. Tables below
    that go on to the next check, which finds the workspace too small here."""
    new = 0x50000 if per_row else None
    assert lib.gqa_kv_pages_reserve(0x10000, 100, 0x20000, max_blocks, 0x30000, new, 16, batch, 0x40000, 64, None,
                                    None) == expect
