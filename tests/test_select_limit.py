"""The longest sequences that pa_select_blocks takes (no GPU needed: the refusal
comes before anything else happens)."""
from __future__ import annotations

import pytest

import paged_kv_cache_14_gb300 as pa


def select(d, group, blocks, block=16, table=None):
    """A call of no sequences whose bounds allow `blocks` blocks of one."""
    return pa.load().pa_select_blocks(0x1000, 0x2000, 0x2100, 0x2200, table or blocks, 0x2300, 0, blocks * block,
                                      2 * group, 2, d, block, 1000, 4, 1, 1, 0x3000, 0x3100, pa.PA_BF16, None)


# The header's limits: every shape, and the usual one.
@pytest.mark.parametrize("d,group,limit", [(256, 128, 169984), (128, 8, 378752), (128, 1, 378752)])
@pytest.mark.parametrize("block", [16, 32])
def test_limit(d, group, limit, block):
    assert select(d, group, limit, block) == 0
    assert select(d, group, limit + 1, block) == -10
    assert select(d, group, 2 * limit, block, table=limit) == 0  # the table is the smaller bound
    assert select(d, group, 2 * limit, block, table=limit + 1) == -10


@pytest.mark.parametrize("d", range(32, 257, 32))
@pytest.mark.parametrize("group", [1, 9, 64, 128])
def test_every_shape(d, group):
    assert select(d, group, 169984) == 0
    assert select(d, group, 430000) == -10
