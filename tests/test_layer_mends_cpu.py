"""The operators around the indexer without a GPU: sizes and devices that they refuse."""
import pytest

import paged_fp8_mqa_gb300 as idx


@pytest.fixture(scope="module", autouse=True)
def lib():
    from paged_fp8_mqa_gb300 import build
    if not idx.LIB_PATH.exists():
        build.build()
    return idx.lib()


@pytest.mark.parametrize("batch,next_n,heads,kv_heads,dim,sms", [
    (2, 1, 4, 8, 128, 4),        # fewer query heads than K/V heads
    (2, 1, 1, 2, 64, 4), (2, 1, 12, 8, 128, 4), (2, 5, 8, 8, 128, 4), (4097, 1, 8, 8, 128, 4),
    (2, 1, 8192, 8, 128, 4), (2, 1, 8, 8, 192, 4), (2, 2 ** 31 - 1, 64, 1, 128, 4), (2, 1, 8, 8, 128, 1025),
    (2, 1, 8, 8, 128, -1),
])
def test_attention_workspace_of_refused_sizes(batch, next_n, heads, kv_heads, dim, sms):
    assert idx.idx_attention_workspace_bytes(batch, next_n, heads, kv_heads, dim, sms) == -1
