"""The rotated append (16-bit pools) against its plain form in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_cache_146_gb300 import (DEV_BAD_POS, DEV_BAD_SLOT, KVPool, cache_write,  # noqa: E402
                                      cache_write_rope, rope_table, status_check)
from serving_reference import HALF_STEP, SUBNORMAL, assert_within, rotate  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def make(T, hq, hkv, dim, rot, dtype, seed, nb=None, block_size=16, fused=True, positions=None):
    gen = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    nb = nb or max(2, -(-T // block_size) + 2)
    pool = KVPool(nb, hkv, dim, dtype, block_size=block_size, device="cuda")
    pool.k_pool.fill_(7.0)
    pool.v_pool.fill_(7.0)
    if fused:
        qkv = torch.randn((T, (hq + 2 * hkv) * dim), generator=gen).to(dt).cuda()
        parts = qkv.split([hq * dim, hkv * dim, hkv * dim], 1)
        q, k, v = (p.view(T, -1, dim) for p in parts)
    else:
        q, k, v = (torch.randn((T, h, dim), generator=gen).to(dt).cuda() for h in (hq, hkv, hkv))
    slots = torch.randperm(nb * block_size, generator=gen)[:T]
    pos = torch.randint(0, 50, (T,), generator=gen) if positions is None else positions
    table = rope_table(max(50, int(pos.max()) + 1 if T else 1), rot)
    return pool, q, k, v, slots, pos.to(torch.int32), table


def check(pool, q, k, v, slots, pos, table, q_out, interleaved):
    dt, bs = k.dtype, pool.block_size
    for rows, got in ((q, q_out), (k, None)):
        if rows is None:
            continue
        want, mag = rotate(rows.double().cpu(), table, pos.long(), interleaved)
        if got is None:
            got = pool.k_pool[slots.cuda() // bs, :, slots.cuda() % bs]
        # two products and a sum in fp32 (3 roundings of 2^-24 of the magnitudes),
        # then one rounding to the row type
        bound = 3 * 2.0 ** -24 * mag * (1 + HALF_STEP[dt]) + HALF_STEP[dt] * want.abs() + SUBNORMAL[dt]
        assert_within(got, want, bound, "rotated rows")
        rot = table.shape[1]
        assert torch.equal(got[..., rot:], rows[..., rot:])
    assert torch.equal(pool.v_pool[slots.cuda() // bs, :, slots.cuda() % bs], v)
    # every other slot is untouched
    for p in (pool.k_pool, pool.v_pool):
        rest = p.permute(0, 2, 1, 3).reshape(-1, p.shape[1], p.shape[3]).clone()
        rest[slots.cuda()] = 7.0
        assert bool((rest == 7.0).all())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,dim,rot,hq,hkv,T", [
    ("bf16", 128, 128, 32, 8, 1), ("bf16", 128, 128, 32, 8, 65), ("f16", 64, 32, 8, 8, 333),
    ("f16", 64, 64, 10, 2, 17), ("bf16", 128, 96, 16, 1, 40), ("bf16", 128, 16, 5, 5, 3),
    ("f16", 96, 48, 6, 3, 29), ("bf16", 256, 112, 4, 2, 31)])
def test_append_matches_the_plain_form(dtype, dim, rot, hq, hkv, T, interleaved):
    pool, q, k, v, slots, pos, table = make(T, hq, hkv, dim, rot, dtype, T + dim)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = cache_write_rope(pool, k, v, pos.cuda(), table.cuda(), slots.cuda(), status, q=q,
                             interleaved=interleaved)
    assert status_check(status) == (0, 0)
    check(pool, q, k, v, slots, pos, table, q_out, interleaved)


def test_without_queries_and_with_contiguous_rows():
    pool, q, k, v, slots, pos, table = make(37, 4, 2, 64, 64, "bf16", 1, fused=False)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert cache_write_rope(pool, k, v, pos.cuda(), table.cuda(), slots.cuda(), status) is None
    assert status_check(status) == (0, 0)
    check(pool, None, k, v, slots, pos, table, None, False)


def test_other_block_sizes():
    pool, q, k, v, slots, pos, table = make(21, 4, 2, 64, 64, "f16", 2, block_size=4)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = cache_write_rope(pool, k, v, pos.cuda(), table.cuda(), slots.cuda(), status, q=q)
    assert status_check(status) == (0, 0)
    check(pool, q, k, v, slots, pos, table, out, False)


def test_position_zero_is_the_plain_write():
    """cos 1 and sin 0: the same bits as cache_write."""
    pool, q, k, v, slots, pos, table = make(50, 8, 2, 128, 128, "bf16", 3,
                                            positions=torch.zeros(50, dtype=torch.int64))
    other = KVPool(pool.num_blocks, 2, 128, "bf16", device="cuda")
    other.k_pool.fill_(7.0)
    other.v_pool.fill_(7.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = cache_write_rope(pool, k, v, pos.cuda(), table.cuda(), slots.cuda(), status, q=q)
    cache_write(other, k.contiguous(), v.contiguous(), slots.cuda(), status)
    assert status_check(status) == (0, 0)
    assert torch.equal(out, q)
    assert torch.equal(pool.k_pool, other.k_pool) and torch.equal(pool.v_pool, other.v_pool)


def test_in_place_queries_equal_the_copy():
    pool, q, k, v, slots, pos, table = make(33, 8, 2, 128, 64, "f16", 4)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (pool, k, v, pos.cuda(), table.cuda(), slots.cuda(), status)
    copy = cache_write_rope(*args, q=q, interleaved=True)
    same = cache_write_rope(*args, q=q, q_out=q, interleaved=True)
    assert same is q and torch.equal(copy, q)


def test_skipped_and_bad_tokens():
    """Negative slots are skipped silently; a slot or position out of range is
    skipped with a status bit; rows of skipped tokens stay as they were."""
    pool, q, k, v, slots, pos, table = make(12, 4, 2, 64, 64, "bf16", 5)
    last = pool.num_blocks * 16
    good = [0, 2, 4, 6, 7, 8, 9, 10]
    slots[1], slots[3], pos[5], pos[11] = -1, last, -1, table.shape[0]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = torch.full((12, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    cache_write_rope(pool, k, v, pos.cuda(), table.cuda(), slots.cuda(), status, q=q, q_out=q_out)
    assert status_check(status)[1] == DEV_BAD_SLOT | DEV_BAD_POS
    assert bool((q_out[[1, 3, 5, 11]] == 5.0).all())
    check(pool, q[good], k[good], v[good], slots[good], pos[good], table, q_out[good], False)


def test_no_tokens():
    pool, q, k, v, slots, pos, table = make(0, 4, 2, 64, 64, "bf16", 6, fused=False)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = cache_write_rope(pool, k, v, pos.cuda(), table.cuda(), slots.cuda(), status, q=q)
    assert out.shape == (0, 4, 64) and status_check(status) == (0, 0)


def test_far_positions_and_far_slots():
    """The last row of a long table, and slots whose byte offset in the pool passes 32 bits."""
    nb = 140_000
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    pool = KVPool(nb, 8, 128, "bf16", device="cuda")          # 4.6 GB each
    table = rope_table(200_000, 128, base=5e5)
    gen = torch.Generator().manual_seed(7)
    k, v = (torch.randn((3, 8, 128), generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    slots = torch.tensor([nb * 16 - 1, 70_000 * 16 + 5, 0])
    pos = torch.tensor([199_999, 131_071, 0], dtype=torch.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache_write_rope(pool, k, v, pos.cuda(), table.cuda(), slots.cuda(), status)
    assert status_check(status) == (0, 0)
    want, mag = rotate(k.double().cpu(), table, pos.long(), False)
    got = pool.k_pool[slots.cuda() // 16, :, slots.cuda() % 16]
    assert_within(got, want, 2.0 ** -22 * mag + 2.0 ** -8 * want.abs() + 2.0 ** -134)
    assert torch.equal(pool.v_pool[slots.cuda() // 16, :, slots.cuda() % 16], v)


def test_table_in_64_bits():
    t = rope_table(5000, 32, base=1e4).double()
    p, i = np.arange(5000)[:, None], np.arange(16)
    ang = p * 1e4 ** (-2.0 * i / 32)
    want = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    # one rounding to fp32 (2^-24 relative, values up to 1), and fp64 angles
    assert np.abs(t.numpy() - want).max() <= 2.0 ** -24 * 1.001


def test_captured_and_on_another_stream():
    pool, q, k, v, slots, pos, table = make(20, 8, 2, 128, 128, "bf16", 8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dpos, dtab, dslots = pos.cuda(), table.cuda(), slots.cuda()
    q_out = torch.zeros_like(q, memory_format=torch.contiguous_format)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    cache_write_rope(pool, k, v, dpos, dtab, dslots, status, q=q, q_out=q_out, stream=side)
    side.synchronize()
    check(pool, q, k, v, slots, pos, table, q_out, False)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache_write_rope(pool, k, v, dpos, dtab, dslots, status, q=q, q_out=q_out)
    q.copy_(torch.randn(q.shape, device="cuda").to(q.dtype))       # other data, same buffers
    k.mul_(2)
    graph.replay()
    assert status_check(status) == (0, 0)
    check(pool, q, k, v, slots, pos, table, q_out, False)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,dim,rot,hq,hkv,T", [
    ("bf16", 128, 128, 5, 3, 9000), ("f16", 96, 48, 7, 2, 9100), ("bf16", 256, 240, 1, 1, 11000),
    ("f16", 64, 64, 0, 3, 40000), ("bf16", 256, 256, 24, 2, 24000)])
def test_many_tokens_equal_few_at_a_time(dtype, dim, rot, hq, hkv, T, interleaved):
    """One large call gives the bits of many small ones: heads that do not divide into
    groups, more work than the grid has threads, padding and refused positions."""
    gen = torch.Generator(device="cuda").manual_seed(T)
    dt = {"bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    qkv = torch.randn((T, (hq + 2 * hkv) * dim), device="cuda", generator=gen).to(dt)
    q, k, v = (p.view(T, -1, dim) for p in qkv.split([hq * dim, hkv * dim, hkv * dim], 1))
    nb = T // 16 + 2
    slots = torch.randperm(nb * 16, device="cuda", generator=gen)[:T]
    slots[::97] = -1
    pos = torch.randint(0, 700, (T,), device="cuda", generator=gen, dtype=torch.int32)
    pos[5::1013] = 700
    table = rope_table(700, rot).cuda()
    got = []
    for step in (T, 997):
        pool = KVPool(nb, hkv, dim, dtype, device="cuda")
        for p in (pool.k_pool, pool.v_pool):
            p.fill_(7.0)
        q_out = torch.full((T, max(hq, 1), dim), 9.0, dtype=dt, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        for t in range(0, T, step):
            part = slice(t, t + step)
            cache_write_rope(pool, k[part], v[part], pos[part], table, slots[part], status,
                             interleaved=interleaved,
                             **(dict(q=q[part], q_out=q_out[part]) if hq else {}))
        assert status_check(status)[1] == DEV_BAD_POS
        got.append((pool.k_pool, pool.v_pool, q_out))
    for a, b in zip(*got):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    kept = (slots >= 0) & (pos < 700)
    assert torch.equal(got[0][1][slots[kept] // 16, :, slots[kept] % 16], v[kept])
    if hq:
        assert bool((got[0][2][~kept] == 9).all()) and not bool((got[0][2][kept] == 9).all(-1).any())
