"""Sequences whose lengths do not fit, next to good ones."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import libbuild  # noqa: E402
from paged_kv_cache_146_gb300 import (DEV_BAD_LEN, KVPool, paged_tree_attention, status_check,  # noqa: E402
                                      tree_workspace_bytes)
from serving_reference import assert_within, scale_of  # noqa: E402
from tree_reference import TreeCase, mask_words  # noqa: E402

libbuild.ensure_built()
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,dim,dtype,rows", [
    (64, 4, 128, torch.bfloat16, 400_000),     # 6.6 GB of zeros
    (8, 2, 64, torch.float16, 1_000),
    (3, 3, 64, torch.bfloat16, 33)])
def test_many_rows_of_a_bad_sequence(hq, hkv, dim, dtype, rows):
    """More drafted tokens than the mask has bits, and more than the sequence has tokens: zero rows,
    however many, and nothing else of it: not the sequences beside it, no time-out."""
    c = TreeCase([3000, 90], [8, 5], hq, hkv, dim, dtype, 1)
    pool = KVPool(c.nb, hkv, dim, "bf16" if dtype == torch.bfloat16 else "f16", device="cuda")
    pool.k_pool.copy_(c.k)
    pool.v_pool.copy_(c.v)
    few = 7                                    # of a sequence of 3 tokens
    total = 8 + rows + 5 + few + 2
    q = torch.zeros((total, hq, dim), dtype=dtype, device="cuda")
    out = torch.full_like(q, 3.0)
    mask = torch.zeros((total, 1), dtype=torch.int32)
    starts = [0, 8, 8 + rows, 13 + rows, 13 + rows + few]
    good = {0: slice(0, 8), 1: slice(8 + rows, 13 + rows)}
    own = mask_words(c.masks, 1)
    q[good[0]], q[good[1]] = c.q[:8].cuda(), c.q[8:].cuda()
    mask[good[0]], mask[good[1]] = own[:8], own[8:]
    tables = torch.stack([c.tables[0], c.tables[0], c.tables[1], c.tables[1]]).cuda()
    lens = torch.tensor([c.lens[0], c.lens[0], c.lens[1], 3], dtype=torch.int32, device="cuda")
    ws = torch.empty(tree_workspace_bytes(total, hq, hkv, dim), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    paged_tree_attention(pool, q, tables, torch.tensor(starts, dtype=torch.int32, device="cuda"), lens,
                         mask.cuda(), scale_of(dim), ws, status, out=out)
    assert status_check(status)[1] == DEV_BAD_LEN
    for s, at in good.items():
        assert_within(out[at], *c.expect(s, scale_of(dim)), f"sequence {s}")
    assert not bool(out[8:8 + rows].any()) and not bool(out[13 + rows:13 + rows + few].any())
    assert bool((out[13 + rows + few:] == 3.0).all())


def test_a_batch_of_nothing_but_bad_sequences():
    """No key tile in the whole call."""
    c = TreeCase([20] * 70, [4] * 70, 4, 2, 64, torch.float16, 2)
    pool = KVPool(c.nb, 2, 64, "f16", device="cuda")
    q, out = c.q.cuda(), torch.full(c.q.shape, 3.0, dtype=torch.float16, device="cuda")
    ws = torch.empty(tree_workspace_bytes(c.rows, 4, 2, 64), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    paged_tree_attention(pool, q, c.tables.cuda(), torch.tensor(c.starts, dtype=torch.int32, device="cuda"),
                         torch.full((70,), -1, dtype=torch.int32, device="cuda"),
                         mask_words(c.masks, 1).cuda(), 0.1, ws, status, out=out)
    assert status_check(status)[1] == DEV_BAD_LEN and not bool(out.any())
