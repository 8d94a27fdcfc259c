"""Decode over keys of equal score, however large: each of them counts alike, whichever
block or warp it sits in."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_cache_146_gb300 import (KVPool, cache_write_b8, paged_decode_attention_b8,  # noqa: E402
                                      paged_decode_attention_window, paged_prefill_attention_window,
                                      prefill_workspace_bytes, status_check)
from serving_reference import Records, random_case, visible  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
WEIGHT = {"bf16": 2.0 ** -16, "f16": 2.0 ** -22, "b8_bf16": 2.0 ** -11, "b8_f16": 2.0 ** -21}


@pytest.mark.parametrize("exponent", [-8, -2, 0, 3, 8, 15, 45])
@pytest.mark.parametrize("n,window,sinks", [(300, 90, 3), (5000, 4900, 0)])
@pytest.mark.parametrize("kind", ["bf16", "f16", "b8_bf16", "b8_f16"])
def test_largest_keys_count_alike(kind, n, window, sinks, exponent):
    """Keys of six levels, the largest in every block.  A level is 2^10 in each of 64 dimensions,
    so with the scale of 1/8 scores lie 2^13 2^exponent apart: at least 2^5 (exponent -8; at -12
    it would be 2 and all levels count), so that only the largest level counts and the row is
    the mean of its V.

    The scores of equal keys are the same fp32 product and the reference is the largest
    score, so their weights are equal exactly.  What remains: a weight's rounding on its way into
    P V (WEIGHT; the sum takes it unrounded), sums and the quotient in fp32 (n terms: 2^-23 n
    of the mean of |V| would be the worst, random 2^-18), 8-bit pools' offset of 1152 steps of V,
    added 16 tokens at a time, and the result's own rounding, half a step; a level below
    leaves less than n 2^-32."""
    dtype, eight = kind.split("_")[-1], kind.startswith("b8")
    if dtype == "f16":
        exponent = min(exponent, 15)             # fp16 ends at 2^16
    unit = 2.0 ** 10
    hkv, hq, dim = 2, 4, 64
    gen = torch.Generator().manual_seed(exponent + 50)
    tables, nb = random_case(gen, [n], hkv, n // 16 + 2)
    level = torch.randint(1, 6, (nb, hkv, 16, 1), generator=gen).double()
    level[:, :, 1::5] = 6
    k = (level * unit).expand(nb, hkv, 16, dim).to(DT[dtype])
    v = torch.randn((nb, hkv, 16, dim), generator=gen).to(DT[dtype])
    q = torch.full((1, hq, dim), 2.0 ** exponent).to(DT[dtype])
    # queries a little apart from the powers of two, so that products are rounded
    q *= torch.tensor([1.0, 1.0078125, 1.2421875, 1.9921875]).view(1, 4, 1).to(DT[dtype])
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pool = KVPool(nb, hkv, dim, kind, device="cuda")
    tiny = 0.0
    if eight:
        rows = [t.permute(0, 2, 1, 3).reshape(-1, hkv, dim).contiguous().cuda() for t in (k, v)]
        cache_write_b8(pool, *rows, torch.arange(nb * 16, device="cuda"), status)
        records = Records.from_bytes(pool.kv.cpu().numpy())
        assert (records.scales[0] == records.scales[0, 0, 0]).all()
        v = torch.from_numpy(records.values(1))
        tiny = 16 * 2.0 ** -23 * 2 * 1152 * float(np.max(records.scales[1]))
        got = paged_decode_attention_b8(pool, q.cuda(), tables.cuda(), lens, 0.125, status, window=window,
                                        sinks=sinks)
    else:
        pool.k_pool.copy_(k)
        pool.v_pool.copy_(v)
        got = paged_decode_attention_window(pool, q.cuda(), tables.cuda(), lens, 0.125, window, sinks, status)
    assert status_check(status) == (0, 0)
    j = torch.tensor(visible(n, n - 1, window, sinks))
    blk, off = tables[0].long()[j // 16], j % 16
    half = torch.finfo(DT[dtype]).eps / 2
    for h in range(hq):
        top = level[blk, h // 2, off, 0] == 6
        vv = v[blk, h // 2, off].double()[top]
        want = vv.mean(0)
        room = half * want.abs() + (2 * WEIGHT[kind] + 2.0 ** -18) * vv.abs().mean(0) + tiny + n * 2.0 ** -32
        assert ((got[0, h].double().cpu() - want).abs() <= room).all(), h


@pytest.mark.parametrize("call", ["prefill", "decode"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_a_neighbour_of_huge_scores_changes_nothing(dtype, call):
    """Two heads of a kv head: the second sees keys of one score, near 2^20, and its row is the mean
    of V; the first head's scores pass 2^24 from the second key tile on.  Roundings as above (prefill:
    two bf16 parts, the first truncated, 2^-15; two fp16 parts, 2^-22)."""
    n, chunk, dim = 300, 40 if call == "prefill" else 1, 64
    gen = torch.Generator().manual_seed(6)
    tables, nb = random_case(gen, [n], 1, 20)
    dt, half = DT[dtype], torch.finfo(DT[dtype]).eps / 2
    v = torch.randn((nb, 1, 16, dim), generator=gen).to(dt)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    start = torch.tensor([0, chunk], dtype=torch.int32, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    ws = torch.empty(prefill_workspace_bytes(1, chunk, 2, 1), dtype=torch.uint8, device="cuda")
    pool = KVPool(nb, 1, dim, dtype, device="cuda")
    pool.v_pool.copy_(v)
    for factor in (1.0, 1.0078125, 1.2421875, 1.6640625, 1.9921875):
        k = torch.zeros((nb, 1, 16, dim))
        for j in range(n):
            k[tables[0, j // 16], 0, j % 16, 0] = 1.0 if j < 64 else 2.0 ** 14
        k[..., 1] = 2.0 ** 13 * 1.2421875
        q = torch.zeros((chunk, 2, dim))
        q[:, 0, 0] = 2.0 ** 15
        q[:, 1, 1] = 2.0 ** 10 * factor
        pool.k_pool.copy_(k)
        if call == "prefill":
            got = paged_prefill_attention_window(pool, q.to(dt).cuda(), tables.cuda(), start, lens, 0.1,
                                                 10 ** 6, 0, ws, status)
        else:
            got = paged_decode_attention_window(pool, q.to(dt).cuda(), tables.cuda(), lens, 0.1, 10 ** 6, 0,
                                                status)
        assert status_check(status) == (0, 0)
        for row in range(chunk):
            j = torch.arange(n - chunk + row + 1)
            vv = v[tables[0].long()[j // 16], 0, j % 16].double()
            want = vv.mean(0)
            room = half * want.abs() + (2 * (2.0 ** -15 if dtype == "bf16" else 2.0 ** -22) + 2.0 ** -18) * vv.abs().mean(0)
            assert ((got[row, 1].double().cpu() - want).abs() <= room).all(), (factor, row)
