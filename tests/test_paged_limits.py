"""Host-side checks of the paged-cache entry points next to their limits.  No
compute call is made here (the addresses are never used)."""
import pytest

import unstructured_sparse_matmul_gb300 as usm
from test_paged_refusals import A16, UNSUPPORTED, append, attention, cache


@pytest.fixture(scope="module")
def lib():
    return usm.load()


def test_more_sequences_than_32_bits_can_walk_over(lib):
    """A walk's step past the last sequence, and the sum of two of their numbers in a
    search, stay in 32 bits up to 2^30 sequences; more are refused."""
    for n in (2**30 + 1, 2**31 - 1):
        assert append(lib, cache(num_seqs=n)) == UNSUPPORTED
        assert attention(lib, cache(num_seqs=n)) == UNSUPPORTED
        assert lib.paged_attention_workspace_bytes(6, n, 4, 2, 8, 1) == 0
    assert lib.paged_attention_workspace_bytes(6, 2**30, 4, 2, 8, 1) > 0
