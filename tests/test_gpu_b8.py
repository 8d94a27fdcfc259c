"""Block-scaled 8-bit pools: the append and the read-back, bit for bit against the
documented rule, and attention over them against 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_cache_146_gb300 import (DEV_BAD_BLOCK, DEV_BAD_LEN, DEV_BAD_POS, DEV_BAD_SLOT,  # noqa: E402
                                      KVPool, block_copy, cache_write_b8, cache_write_rope,
                                      dequantize_blocks, gather_blocks, paged_decode_attention_b8,
                                      rope_table, scatter_blocks, status_check)
from serving_reference import (F16_HALF_STEP, Records, assert_within, attention, random_case,  # noqa: E402
                               rotate_f32, scale_of, visible)

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def new_status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def random_pool(nb, hkv, dim, dtype, seed):
    """A pool of random records (scales of very different sizes) and its plain copy."""
    rng = np.random.default_rng(seed)
    ref = Records(nb, hkv, dim)
    ref.codes[:] = rng.integers(-127, 128, ref.codes.shape)
    ref.scales[:] = 0.02 * np.exp(rng.uniform(-3, 1, ref.scales.shape))
    pool = KVPool(nb, hkv, dim, "b8_" + dtype, device="cuda")
    pool.kv.copy_(torch.from_numpy(ref.to_bytes()))
    return pool, ref


def same_records(pool, ref, blocks=None):
    got = Records.from_bytes(pool.kv.cpu().numpy())
    sel = slice(None) if blocks is None else blocks
    assert np.array_equal(got.scales[:, sel].view(np.uint32), ref.scales[:, sel].view(np.uint32))
    assert np.array_equal(got.codes[:, sel], ref.codes[:, sel])


# -------------------------------------------------------------------------- append
@pytest.mark.parametrize("dtype,dim,hkv", [("bf16", 128, 8), ("f16", 64, 3), ("bf16", 64, 2), ("f16", 128, 1)])
def test_append_steps_bit_for_bit(dtype, dim, hkv):
    """Prompts of every length class, then single tokens that grow the scales or do not."""
    rng = np.random.default_rng(dim + hkv)
    news = [1, 15, 16, 17, 40, 3, 100]
    pool, ref = random_pool(30, hkv, dim, dtype, 1)         # what the blocks held before must not matter
    ledger = KVPool(30, hkv, dim, "b8_" + dtype, free_order=rng.permutation(30))
    tables = np.full((len(news), 12), -1, np.int32)
    lens = np.zeros(len(news), np.int32)
    for step in range(6):
        n = np.array(news if step == 0 else [1, 1, 2, 1, 1, 1, 1], np.int32)
        slots = ledger.append_slots(lens, n, tables)
        lens += n
        grow = [1.0, 0.5, 3.0, 1e-3, 40.0, 1.0][step]
        rows = [(rng.standard_normal((len(slots), hkv, dim)) * grow).astype(np.float32) for _ in range(2)]
        k, v = (torch.from_numpy(r).to(DT[dtype]) for r in rows)
        status = new_status()
        cache_write_b8(pool, k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), status)
        assert status_check(status) == (0, 0)
        for part, r in enumerate((k, v)):
            ref.append(part, r.float().numpy(), slots)
        same_records(pool, ref)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,dim,rot,hq,hkv,tokens", [
    ("bf16", 128, 128, 32, 8, 700), ("f16", 64, 32, 8, 2, 90), ("bf16", 128, 48, 6, 3, 33),
    ("bf16", 128, 128, 8, 8, 9000)])       # the last: 16 tokens to a warp
def test_rotated_append_bit_for_bit(dtype, dim, rot, hq, hkv, tokens, interleaved):
    rng = np.random.default_rng(tokens)
    news = np.array([tokens // 2, 1, tokens - tokens // 2 - 1], np.int32)
    nb = int(sum(-(-int(n) // 16) for n in news)) + 2
    pool, ref = random_pool(nb, hkv, dim, dtype, 2)
    ledger = KVPool(nb, hkv, dim, "b8_" + dtype, free_order=rng.permutation(nb))
    tables = np.full((3, nb), -1, np.int32)
    slots = ledger.append_slots(np.zeros(3, np.int32), news, tables)
    pos = np.concatenate([np.arange(n) for n in news]).astype(np.int32)
    table = rope_table(int(pos.max()) + 1, rot)
    qkv = torch.randn((tokens, (hq + 2 * hkv) * dim), generator=torch.Generator().manual_seed(3)).to(DT[dtype])
    q, k, v = (p.view(tokens, -1, dim) for p in qkv.split([hq * dim, hkv * dim, hkv * dim], 1))
    gpu = qkv.cuda()
    gq, gk, gv = (p.view(tokens, -1, dim) for p in gpu.split([hq * dim, hkv * dim, hkv * dim], 1))
    status = new_status()
    out = cache_write_rope(pool, gk, gv, torch.from_numpy(pos).cuda(), table.cuda(),
                           torch.from_numpy(slots).cuda(), status, q=gq, interleaved=interleaved)
    assert status_check(status) == (0, 0)
    ref.append(0, rotate_f32(k.float().numpy(), table, pos, interleaved), slots)
    ref.append(1, v.float().numpy(), slots)
    same_records(pool, ref)
    want = torch.from_numpy(rotate_f32(q.float().numpy(), table, pos, interleaved)).to(DT[dtype])
    assert torch.equal(out.cpu(), want)


def test_quantised_values_stay_near():
    """Half a step of the block's scale for fresh tokens, one more half step for each
    growth of the scale (the reference is the rows themselves, in 64 bits)."""
    dim, hkv = 128, 2
    pool = KVPool(2, hkv, dim, "b8_bf16", device="cuda")
    gen = torch.Generator().manual_seed(4)
    rows = torch.randn((16, hkv, dim), generator=gen).to(torch.bfloat16)
    rows[9:] *= 5
    for t in range(16):
        status = new_status()
        cache_write_b8(pool, rows[t:t + 1].cuda(), rows[t:t + 1].cuda(),
                       torch.tensor([16 + t], device="cuda"), status)
        assert status_check(status) == (0, 0)
    got = Records.from_bytes(pool.kv.cpu().numpy())
    steps = np.maximum.accumulate(np.abs(rows.double().numpy()).max(2), 0) / 127      # [16][Hkv]
    grows = np.concatenate([np.diff(steps, axis=0) > 0, np.zeros((1, hkv), bool)])
    for h in range(hkv):
        for t in range(16):
            later = [steps[u + 1, h] for u in range(t, 15) if grows[u, h]]
            bound = 0.5 * (steps[t, h] + sum(later)) * (1 + 2.0 ** -14)
            err = np.abs(got.values(0)[1, h, t] - rows[t, h].double().numpy()).max()
            assert err <= bound, (h, t, err, bound)


def test_extreme_values():
    """Infinities count as the largest bf16, NaN stores 0, tiny blocks store zeros."""
    dim = 64
    pool, ref = random_pool(4, 1, dim, "bf16", 5)
    k = torch.randn((4, 1, dim), generator=torch.Generator().manual_seed(6)).to(torch.bfloat16)
    v = torch.full((4, 1, dim), 2.0 ** -110).to(torch.bfloat16)
    k[0, 0, 3], k[0, 0, 5], k[1, 0, 7] = float("inf"), float("-inf"), float("nan")
    k[2] = 0.0
    slots = np.array([0, 16, 32, 48])
    status = new_status()
    cache_write_b8(pool, k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), status)
    assert status_check(status) == (0, 0)
    ref.append(0, k.float().numpy(), slots)
    ref.append(1, v.float().numpy(), slots)
    same_records(pool, ref)
    assert ref.codes[0, 0, 0, 0, 3] == 127 and ref.codes[0, 0, 0, 0, 5] == -127
    assert ref.codes[0, 1, 0, 0, 7] == 0 and not ref.codes[0, 2, 0, 0].any()
    assert not ref.scales[1].any()


def test_skipped_and_bad_slots():
    pool, ref = random_pool(5, 2, 128, "f16", 7)
    rows = torch.randn((8, 2, 128), generator=torch.Generator().manual_seed(8)).to(torch.float16)
    slots = np.array([16, 17, -1, 5 * 16, 33, 34, -1, 64])
    status = new_status()
    cache_write_b8(pool, rows.cuda(), rows.cuda(), torch.from_numpy(slots).cuda(), status)
    assert status_check(status)[1] == DEV_BAD_SLOT
    keep = np.where(slots >= 80, -1, slots)
    for part in range(2):
        ref.append(part, rows.float().numpy(), keep)
    same_records(pool, ref)


def test_bad_position_skips_the_token():
    pool, ref = random_pool(3, 2, 128, "bf16", 9)
    rows = torch.randn((3, 2, 128), generator=torch.Generator().manual_seed(10)).to(torch.bfloat16)
    pos = torch.tensor([0, 99, 0], dtype=torch.int32)
    slots = np.array([0, 1, 2])
    status = new_status()
    cache_write_rope(pool, rows.cuda(), rows.cuda(), pos.cuda(), rope_table(4, 128).cuda(),
                     torch.from_numpy(slots).cuda(), status)
    assert status_check(status)[1] == DEV_BAD_POS
    x = rows.float().numpy()
    for part in range(2):      # tokens 0 and 2 share the block's scale; token 1's codes stay
        ref.append(part, rows.float().numpy(), np.array([0, -1, 2]))
    same_records(pool, ref)


# ---------------------------------------------------------------- blocks moved about
@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("f16", 64)])
def test_dequantize_copy_and_swap(dtype, dim):
    hkv, nb = 3, 9
    pool, ref = random_pool(nb, hkv, dim, dtype, 11)
    ids = torch.tensor([4, 0, 8, 4], dtype=torch.int32, device="cuda")
    shape = (4, hkv, 16, dim)
    k, v = (torch.empty(shape, dtype=DT[dtype], device="cuda") for _ in range(2))
    status = new_status()
    dequantize_blocks(pool, ids, k, v, status)
    for part, got in enumerate((k, v)):
        codes, scales = ref.codes[part][[4, 0, 8, 4]], ref.scales[part][[4, 0, 8, 4]]
        want = torch.from_numpy((codes.astype(np.float32) * scales[..., None, None])).to(DT[dtype])
        assert torch.equal(got.cpu(), want)
    staging = torch.empty((2, hkv, pool.record_bytes), dtype=torch.uint8, device="cuda")
    gather_blocks(pool, ids[:2].contiguous(), staging, status)
    assert torch.equal(staging, pool.kv[ids[:2].long()])
    scatter_blocks(pool, torch.tensor([7, 1], dtype=torch.int32, device="cuda"), staging, status)
    block_copy(pool, ids[2:3].contiguous(), torch.tensor([2], dtype=torch.int32, device="cuda"), status)
    assert status_check(status) == (0, 0)
    for part in (ref.codes, ref.scales):
        part[:, 7], part[:, 1], part[:, 2] = part[:, 4].copy(), part[:, 0].copy(), part[:, 8].copy()
    same_records(pool, ref)
    k.fill_(3.0)
    dequantize_blocks(pool, torch.tensor([1, nb, -1, 2], dtype=torch.int32, device="cuda"), k, v, status)
    assert status_check(status)[1] == DEV_BAD_BLOCK
    assert bool((k[1:3] == 3.0).all()) and not bool((k[0] == 3.0).all())


# ----------------------------------------------------------------------- attention
# weights enter the P V product in one fp16 part for bf16 rows, two for fp16
WEIGHT = {"bf16": F16_HALF_STEP, "f16": F16_HALF_STEP ** 2}


def run_attention(lens, hq, hkv, dim, dtype, window, sinks, seed, maxb=None, evict=True):
    gen = torch.Generator().manual_seed(seed)
    maxb = maxb or max(-(-n // 16) for n in lens) + 1
    tables, nb = random_case(gen, lens, hkv, maxb)
    pool, ref = random_pool(nb, hkv, dim, dtype, seed)
    q = torch.randn((len(lens), hq, dim), generator=gen).to(DT[dtype])
    if window is not None and evict:      # blocks that nobody sees were given back
        for s, n in enumerate(lens):
            seen = {j // 16 for j in visible(n, n - 1, window, sinks)}
            for b in range(maxb):
                if b not in seen:
                    tables[s, b] = -1
    status = new_status()
    out = paged_decode_attention_b8(pool, q.cuda(), tables.cuda(),
                                    torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                    scale_of(dim), status, window=window, sinks=sinks)
    assert status_check(status) == (0, 0)
    kv = [torch.from_numpy(ref.values(p)) for p in range(2)]
    for s, n in enumerate(lens):
        if n == 0:
            assert not bool(out[s].any())
            continue
        j = torch.tensor(visible(n, n - 1, window or n, sinks))
        blk, off = tables[s].long()[j // 16], j % 16
        for h in range(hq):
            k, v = (x[blk, h // (hq // hkv), off] for x in kv)
            offs = (1152 * torch.from_numpy(x[:, h // (hq // hkv)]).double()[blk] for x in ref.scales)
            want, bound = attention(q[s, h].double(), k, v, scale_of(dim), DT[dtype], WEIGHT[dtype], *offs)
            assert_within(out[s, h], want, bound, f"sequence {s} ({n} tokens) head {h}")
    return out


@pytest.mark.parametrize("hq,hkv", [(4, 4), (8, 2), (16, 1), (12, 1), (10, 2), (9, 1)])
@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("f16", 128), ("bf16", 64), ("f16", 64)])
def test_attention_matches_64_bits(dtype, dim, hq, hkv):
    run_attention([1, 0, 16, 17, 15, 130, 777], hq, hkv, dim, dtype, None, 0, hq * dim)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (17, 16), (100, 33), (5000, 4),
                                          (250, 300), (64, 0)])
@pytest.mark.parametrize("dtype,dim,hq,hkv", [("bf16", 128, 8, 2), ("f16", 64, 12, 1)])
def test_attention_window(dtype, dim, hq, hkv, window, sinks):
    run_attention([1, 0, 16, 33, 100, 600, 1111], hq, hkv, dim, dtype, window, sinks, window + sinks)


def test_attention_long_and_wide_tables():
    """A long context next to short ones, in a table much wider than any of them."""
    run_attention([9001, 3, 40], 8, 2, 128, "bf16", None, 0, 21, maxb=2000)
    run_attention([9001], 4, 1, 64, "f16", None, 0, 22, maxb=600)


@pytest.mark.parametrize("seqs,hq,hkv,top", [(130, 4, 4, 1100), (45, 4, 2, 760), (600, 1, 1, 40)])
def test_attention_many_ragged_sequences(seqs, hq, hkv, top):
    """More CTAs than fit at once (longest first), odd cluster sizes, many short rows."""
    lens = [(37 * i * i + 11 * i) % top for i in range(seqs)]
    run_attention(lens, hq, hkv, 64, "bf16", None, 0, seqs, maxb=-(-top // 16) + 2)


@pytest.mark.parametrize("scale", [0.0, -0.1])
def test_attention_zero_and_negative_scale(scale):
    gen = torch.Generator().manual_seed(30)
    tables, nb = random_case(gen, [90], 1, 6)
    pool, ref = random_pool(nb, 1, 64, "f16", 31)
    q = torch.randn((1, 4, 64), generator=gen).to(torch.float16)
    status = new_status()
    out = paged_decode_attention_b8(pool, q.cuda(), tables.cuda(), torch.tensor([90], dtype=torch.int32, device="cuda"),
                                    scale, status, window=30, sinks=5)
    assert status_check(status) == (0, 0)
    j = torch.tensor(visible(90, 89, 30, 5))
    k, v = (torch.from_numpy(ref.values(p))[tables[0].long()[j // 16], 0, j % 16] for p in range(2))
    offs = [1152 * torch.from_numpy(x[:, 0]).double()[tables[0].long()[j // 16]] for x in ref.scales]
    for h in range(4):
        # the bound counts the score's size: take the scale's
        want, bound = attention(-q[0, h].double(), k, v, -scale, torch.float16, F16_HALF_STEP ** 2, *offs)
        assert_within(out[0, h], want, bound, f"head {h}")


def test_attention_scales_and_queries_of_any_size():
    """Blocks whose scales differ by 2^40, and queries far outside fp16's range."""
    dim, hkv, hq = 128, 1, 4
    lens = [200]
    gen = torch.Generator().manual_seed(23)
    tables, nb = random_case(gen, lens, hkv, 13)
    pool, ref = random_pool(nb, hkv, dim, "bf16", 24)
    ref.scales[1] *= np.exp2(np.arange(nb) * 3.0 - 20).astype(np.float32)[:, None]
    ref.scales[0] *= np.float32(2.0 ** -30)
    pool.kv.copy_(torch.from_numpy(ref.to_bytes()))
    q = (torch.randn((1, hq, dim), generator=gen) * 2.0 ** 27).to(torch.bfloat16)
    q[0, 1] *= 2.0 ** -60
    status = new_status()
    out = paged_decode_attention_b8(pool, q.cuda(), tables.cuda(),
                                    torch.tensor(lens, dtype=torch.int32, device="cuda"), 0.1, status)
    assert status_check(status) == (0, 0)
    j = torch.arange(200)
    k, v = (torch.from_numpy(ref.values(p))[tables[0].long()[j // 16], 0, j % 16] for p in range(2))
    for h in range(hq):
        offs = (1152 * torch.from_numpy(x[:, 0]).double()[tables[0].long()[j // 16]] for x in ref.scales)
        want, bound = attention(q[0, h].double(), k, v, 0.1, torch.bfloat16, F16_HALF_STEP, *offs)
        assert_within(out[0, h], want, bound, f"head {h}")


def test_bad_lengths_and_blocks_give_zero_rows():
    lens = [40, -1, 1000, 40, 40]
    gen = torch.Generator().manual_seed(25)
    tables, nb = random_case(gen, [40, 40, 40, 40, 40], 2, 4)
    pool, _ = random_pool(nb, 2, 128, "bf16", 26)
    tables[3, 1] = nb
    q = torch.randn((5, 8, 128), generator=gen).to(torch.bfloat16).cuda()
    status = new_status()
    args = (pool, q, tables.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), 0.1, status)
    out = paged_decode_attention_b8(*args)
    assert status_check(status)[1] == DEV_BAD_LEN | DEV_BAD_BLOCK
    assert not bool(out[1:4].any())
    assert bool(out[0].any()) and bool(out[4].any())
    # behind the window the same entry is not read
    lens = [40, 40, 40, 40, 40]
    out = paged_decode_attention_b8(pool, q, tables.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                    0.1, status, window=8)
    assert status_check(status) == (0, 0) and bool(out[3].any())


def test_records_past_32_bits():
    nb = 140_000                                   # 4.6 GB of records
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    pool = KVPool(nb, 8, 128, "b8_bf16", device="cuda")
    gen = torch.Generator().manual_seed(27)
    rows = torch.randn((40, 8, 128), generator=gen).to(torch.bfloat16).cuda()
    blocks = [nb - 1, 5, 70_001]
    slots = torch.tensor([b * 16 + t for b in blocks for t in range(16)][:40], device="cuda")
    status = new_status()
    cache_write_b8(pool, rows, rows, slots, status)
    small = KVPool(3, 8, 128, "b8_bf16", device="cuda")
    cache_write_b8(small, rows, rows, torch.arange(40, device="cuda"), status)
    q = torch.randn((1, 32, 128), generator=gen).to(torch.bfloat16).cuda()
    n = torch.tensor([40], dtype=torch.int32, device="cuda")
    far = paged_decode_attention_b8(pool, q, torch.tensor([blocks], dtype=torch.int32, device="cuda"), n, 0.1, status)
    near = paged_decode_attention_b8(small, q, torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda"), n, 0.1, status)
    assert status_check(status) == (0, 0)
    assert torch.equal(far, near)


def test_repeated_captured_and_concurrent_calls_agree():
    lens = [500, 33, 2000, 7]
    gen = torch.Generator().manual_seed(28)
    tables, nb = random_case(gen, lens, 2, 130)
    pool, _ = random_pool(nb, 2, 128, "bf16", 29)
    q = torch.randn((4, 8, 128), generator=gen).to(torch.bfloat16).cuda()
    status = new_status()
    args = (pool, q, tables.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), 0.1, status)
    first = paged_decode_attention_b8(*args)
    assert torch.equal(first, paged_decode_attention_b8(*args))
    graph, held = torch.cuda.CUDAGraph(), torch.zeros_like(q)
    with torch.cuda.graph(graph):
        paged_decode_attention_b8(*args, out=held)
    outs = [torch.empty_like(q) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o in zip(streams, outs):
            paged_decode_attention_b8(*args, out=o, stream=s)
        graph.replay()
    torch.cuda.synchronize()
    assert status_check(status) == (0, 0)
    for o in (*outs, held):
        assert torch.equal(first, o)


@pytest.mark.parametrize("dtype,dim,rot,hq,hkv,interleaved", [
    ("bf16", 128, 128, 4, 8, False), ("f16", 128, 64, 2, 3, True), ("f16", 64, 64, 3, 1, False),
    ("bf16", 64, 16, 0, 9, True), ("bf16", 128, 112, 5, 2, False),
    # values enough for spans of tokens
    ("f16", 128, 64, 2, 6, True), ("f16", 64, 64, 3, 11, False), ("bf16", 64, 16, 0, 13, True),
    ("bf16", 128, 112, 5, 7, False), ("f16", 128, 128, 3, 40, True)])
def test_many_tokens_with_gaps_and_odd_values(dtype, dim, rot, hq, hkv, interleaved):
    """Thousands of tokens of ragged sequences, some blocks cut short, some tokens
    refused, infinities and NaN among the values, queries turned in place."""
    rng = np.random.default_rng(dim + rot)
    prior = rng.integers(0, 40, 60).astype(np.int32)
    news = np.where(np.arange(60) % 7 == 0, 1, rng.integers(40, 110, 60)).astype(np.int32)
    nb = int(sum(-(-int(a + b) // 16) for a, b in zip(prior, news))) + 3
    pool, ref = random_pool(nb, hkv, dim, dtype, 21)
    ledger = KVPool(nb, hkv, dim, "b8_" + dtype, free_order=rng.permutation(nb))
    tables = np.full((60, 12), -1, np.int32)
    ledger.append_slots(np.zeros(60, np.int32), prior, tables)
    slots = np.asarray(ledger.append_slots(prior, news, tables)).copy()
    tokens = len(slots)
    assert tokens >= 3200
    pos = np.concatenate([np.arange(a, a + n) for a, n in zip(prior, news)]).astype(np.int32)
    table = rope_table(200, rot)
    for t in range(100, tokens, 97):                       # the rest of a block is left out
        slots[t:t + 16][slots[t:t + 16] // 16 == slots[t] // 16] = -1
    refused = [t for t in range(60, tokens - 1, 113)
               if slots[t] > 0 and slots[t] % 16 and slots[t - 1] == slots[t] - 1]
    pos[refused[::2]] = 200
    pos[refused[1::2]] = -1
    qkv = torch.randn((tokens, (hq + 2 * hkv) * dim), generator=torch.Generator().manual_seed(22)).to(DT[dtype])
    q, k, v = (p.view(tokens, -1, dim) for p in qkv.split([hq * dim, hkv * dim, hkv * dim], 1))
    for i, odd in enumerate([float("inf"), float("-inf"), float("nan")] * 4):
        k[37 + 211 * i, i % hkv, (5 * i) % dim] = odd
        v[90 + 173 * i, i % hkv, (7 * i) % dim] = odd
    gpu = qkv.cuda()
    gq, gk, gv = (p.view(tokens, -1, dim) for p in gpu.split([hq * dim, hkv * dim, hkv * dim], 1))
    status = new_status()
    dev = dict(q=gq, q_out=gq) if hq else {}
    cache_write_rope(pool, gk, gv, torch.from_numpy(pos).cuda(), table.cuda(), torch.from_numpy(slots).cuda(),
                     status, interleaved=interleaved, **dev)
    assert status_check(status)[1] == DEV_BAD_POS
    kept = slots.copy()
    kept[refused] = -1
    safe = np.where(kept < 0, 0, pos)
    with np.errstate(invalid="ignore"):
        ref.append(0, rotate_f32(k.float().numpy(), table, safe, interleaved), kept)
        ref.append(1, v.float().numpy(), kept)
    same_records(pool, ref)
    if hq:
        want = torch.from_numpy(rotate_f32(q.float().numpy(), table, safe, interleaved)).to(DT[dtype])
        want[torch.from_numpy(kept < 0)] = q[torch.from_numpy(kept < 0)]
        assert torch.equal(gq.cpu(), want)
    assert torch.equal(gk.cpu().view(torch.int16), k.contiguous().view(torch.int16))


@pytest.mark.parametrize("dtype,dim,hq,hkv,tokens", [("bf16", 128, 3, 33, 520), ("f16", 64, 2, 80, 421)])
def test_many_heads_and_one_token_per_sequence(dtype, dim, hq, hkv, tokens):
    """Enough values for spans of tokens, every token a run of its own."""
    rng = np.random.default_rng(tokens)
    nb = tokens + 5
    pool, ref = random_pool(nb, hkv, dim, dtype, 31)
    slots = (rng.permutation(nb)[:tokens] * 16 + rng.integers(0, 16, tokens)).astype(np.int64)
    slots[::41] = -1
    pos = rng.integers(0, 90, tokens).astype(np.int32)
    table = rope_table(90, dim)
    gen = torch.Generator().manual_seed(32)
    q, k, v = (torch.randn((tokens, h, dim), generator=gen).to(DT[dtype]) for h in (hq, hkv, hkv))
    status = new_status()
    out = torch.zeros_like(q).cuda()
    cache_write_rope(pool, k.cuda(), v.cuda(), torch.from_numpy(pos).cuda(), table.cuda(),
                     torch.from_numpy(slots).cuda(), status, q=q.cuda(), q_out=out)
    assert status_check(status) == (0, 0)
    ref.append(0, rotate_f32(k.float().numpy(), table, pos, False), slots)
    ref.append(1, v.float().numpy(), slots)
    same_records(pool, ref)
    want = torch.from_numpy(rotate_f32(q.float().numpy(), table, pos, False)).to(DT[dtype])
    want[torch.from_numpy(slots < 0)] = 0
    assert torch.equal(out.cpu(), want)


@pytest.mark.parametrize("dtype,dim,hkv,n", [("bf16", 128, 8, 2700), ("f16", 64, 7, 5900)])
def test_many_blocks_read_back_equal_few_at_a_time(dtype, dim, hkv, n):
    """More blocks than one round of the grid takes, some refused."""
    nb = 900
    pool = KVPool(nb, hkv, dim, "b8_" + dtype, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(n)
    pool.kv.random_(0, 256, generator=gen)
    pool.kv[:, :, 32 * dim:].view(torch.float32).uniform_(0.01, 3.0, generator=gen)
    ids = torch.randint(0, nb, (n,), device="cuda", generator=gen, dtype=torch.int32)
    ids[7::501], ids[9::501] = -1, nb
    got = []
    for step in (n, 61):
        out = [torch.full((n, hkv, 16, dim), 5.0, dtype=DT[dtype], device="cuda") for _ in "kv"]
        status = new_status()
        for i in range(0, n, step):
            dequantize_blocks(pool, ids[i:i + step], out[0][i:i + step], out[1][i:i + step], status)
        assert status_check(status)[1] == DEV_BAD_BLOCK
        got.append(out)
    for a, b in zip(*got):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    bad = (ids < 0) | (ids >= nb)
    assert bool((got[0][0][bad] == 5).all())
    # K of one block by the formula: byte - 128 times the scale, rounded once
    i = int((~bad).nonzero()[3])
    scale = pool.kv[ids[i], :, 32 * dim:].view(torch.float32)[:, 0]
    codes = Records.from_bytes(pool.kv[ids[i]:ids[i] + 1].cpu().numpy()).codes[0, 0]
    want = (torch.from_numpy(codes).float().cuda() * scale[:, None, None]).to(DT[dtype])
    assert torch.equal(got[0][0][i], want)
