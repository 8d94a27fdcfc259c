"""How precisely attention over drafted trees carries a softmax weight into the product with V."""
import math

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import libbuild  # noqa: E402
from paged_kv_cache_146_gb300 import (KVPool, paged_tree_attention, status_check,  # noqa: E402
                                      tree_workspace_bytes)

libbuild.ensure_built()
pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
RATIOS = [(64 + i, 127 - i // 3) for i in range(0, 60, 4)]


@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 2), (16, 1)])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("name", ["bf16", "f16"])
def test_two_tokens_that_cancel(name, dim, hq, hkv):
    """Every drafted token sees the one token of the cache, of score 0 and value c0 / 64, and itself, of
    a score of -scale and the value -c1 / 64; with scale = ln(c1 / c0) they cancel.

    The error of a weight on its way into the product is at most 2^-16 (bf16: the first part truncated,
    so the rest is below 2^-7 of the weight's power of two and loses 2^-9 of that) or 2^-22 (fp16:
    2^-10, 2^-12), 2^-22 (exp2) and 2^-23 (its argument, at most 1: the scale's product with log2 e and
    the product).  Each part is one term of the numerator, four in all, each addition may truncate by
    2^-23 of c0 / 64.  The denominator's error and the quotient's are of a value near zero."""
    n = 95
    pool = KVPool(6, hkv, dim, name, device="cuda")
    q = torch.zeros((n, hq, dim), dtype=DT[name], device="cuda")
    q[..., 0] = 1
    tables = torch.arange(6, dtype=torch.int32, device="cuda").view(1, 6)
    starts, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, n], [n + 1]))
    mask = torch.zeros((n, 3), dtype=torch.int64)
    for i in range(n):
        mask[i, i // 32] = 1 << i % 32
    mask = torch.where(mask >= 2 ** 31, mask - 2 ** 32, mask).to("cuda", torch.int32)
    ws = torch.empty(tree_workspace_bytes(n, hq, hkv, dim), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pool.k_pool.zero_()
    pool.k_pool[..., 0] = -1
    pool.k_pool[0, :, 0] = 0
    half = torch.finfo(DT[name]).eps / 2
    weight = (2.0 ** -16 if name == "bf16" else 2.0 ** -22) + 2.0 ** -22 + 2.0 ** -23
    for c0, c1 in RATIOS:
        scale = math.log(c1 / c0)
        pool.v_pool.fill_(-c1 / 64)
        pool.v_pool[0, :, 0] = c0 / 64
        got = paged_tree_attention(pool, q, tables, starts, lens, mask, scale, ws, status).double().cpu()
        w = math.exp(-float(torch.tensor(scale, dtype=torch.float32)))
        want = (c0 - w * c1) / 64 / (1 + w)
        room = (c0 / 64) * (weight + 4 * 2.0 ** -23) / (1 + w)
        worst = (got - want).abs().max().item()
        assert worst <= room + half * (abs(want) + room) + 2.0 ** -25 * 2.0 ** -7, (c0, c1, worst / room)
    assert status_check(status) == (0, 0)
