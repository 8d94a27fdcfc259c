"""The prefill calls' workspace: one list entry of 8 bytes for an item of two query tiles, as a plain
call has them, whatever a windowed call makes of them."""
import pytest

import libbuild

lib = libbuild.ensure_built()


def align(n):
    return -(-n // 256) * 256


@pytest.mark.parametrize("G", [1, 3, 4, 12, 16])
@pytest.mark.parametrize("S,T", [(1, 1), (1, 300), (12, 13000), (40, 40), (70, 9001), (512, 100000)])
def test_sizes(S, T, G):
    hkv = 2
    size = 256 + align((T // (2 * (128 // G)) + S + 1) * 8)
    assert lib.paged_prefill_workspace_bytes(S, T, G * hkv, hkv) == size
    for dim, maxb in ((64, 7), (128, 900)):
        staged = size + align(S * hkv * 4) + align(S * maxb * hkv * 16 * dim * 2)
        assert lib.paged_prefill_workspace_bytes_staged(S, T, G * hkv, hkv, dim, maxb) == staged
