"""Limits of the calls for trees of drafted tokens that the C entries refuse by themselves, before
any launch; the addresses are never read."""
import pytest

pytest.importorskip("torch")

import libbuild  # noqa: E402
from paged_kv_cache_146_gb300 import KVPool, tree_workspace_bytes  # noqa: E402

lib = libbuild.ensure_built()
A, UNSUPPORTED = 1 << 20, -8


@pytest.mark.parametrize("seqs,tokens,words,maxb,hq,hkv", [
    (1, 1, 1, 2 ** 27, 16, 64),                # 64 kv heads of 2^25 key tiles
    (4096, 1024, 32, 2 ** 16, 128, 8),         # 128 query tiles to a sequence, should one hold all rows
])
def test_trees_of_more_than_32_bits(seqs, tokens, words, maxb, hq, hkv):
    pool = KVPool(8, hkv, 64, "bf16")
    hq = max(hq, hkv)
    need = tree_workspace_bytes(tokens, hq, hkv, 64)
    assert need > 0
    assert lib.paged_tree_attention(pool.handle, A, A, A, A, A, maxb, A, A, A, words, seqs, tokens, hq, 0.1,
                                    A, need, A, None) == UNSUPPORTED


@pytest.mark.parametrize("seqs,entries", [(65536, 65536), (1, 2 ** 31 - 1)])
def test_lists_of_more_than_a_launch_takes(seqs, entries):
    pool = KVPool(8, 2, 64, "bf16")
    assert lib.kv_cache_compact(pool.handle, A, 4, A, A, A, A, seqs, entries, A, A, A, None) == UNSUPPORTED
