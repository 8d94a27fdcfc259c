"""Attention over a sliding window with sinks, decode and chunks of a prompt,
against 64 bits; and the calls in the order a server makes them."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_cache_146_gb300 import (DEV_BAD_BLOCK, DEV_BAD_LEN, KVPool, cache_write_b8, cache_write_rope,  # noqa: E402
                                      dequantize_blocks, paged_decode_attention_b8,
                                      paged_decode_attention_window, paged_prefill_attention,
                                      paged_prefill_attention_window, prefill_workspace_bytes,
                                      rope_table, status_check)
from serving_reference import (F16_HALF_STEP, Records, assert_within, attention, random_case,  # noqa: E402
                               rotate, scale_of, visible)

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
# relative error of a weight on its way into P V: decode takes it in two parts of
# the pool's type; prefill in two bf16 parts, the first truncated, or one fp16 part
DECODE_WEIGHT = {"bf16": 2.0 ** -16, "f16": 2.0 ** -22}
PREFILL_WEIGHT = {"bf16": 2.0 ** -15, "f16": F16_HALF_STEP}


def new_status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def build(lens, first_query, hkv, dim, dtype, window, sinks, seed, maxb=None, nan_hidden=True):
    """Pools whose hidden tokens hold NaN and whose unseen blocks were given back."""
    gen = torch.Generator().manual_seed(seed)
    maxb = maxb or max(-(-n // 16) for n in lens) + 1
    tables, nb = random_case(gen, lens, hkv, maxb)
    k, v = (torch.randn((nb, hkv, 16, dim), generator=gen).to(DT[dtype]) for _ in range(2))
    if nan_hidden:
        keep = torch.zeros((nb, 16), dtype=torch.bool)
        for s, n in enumerate(lens):
            for q0 in range(first_query[s], n):
                j = torch.tensor(visible(n, q0, window, sinks))
                keep[tables[s].long()[j // 16], j % 16] = True
        for p in (k, v):
            p.permute(0, 2, 1, 3)[~keep] = float("nan")
        for s, n in enumerate(lens):
            for b in range(maxb):
                if tables[s, b] >= 0 and not keep[tables[s, b]].any():
                    tables[s, b] = -1
    pool = KVPool(nb, hkv, dim, dtype, device="cuda")
    pool.k_pool.copy_(k)
    pool.v_pool.copy_(v)
    return pool, k, v, tables, gen


def expect(q, k, v, tables, lens, first_query, rows, window, sinks, dtype, weight, got):
    """Every listed (row, sequence, position) of `got` against 64 bits."""
    hq, hkv, dim = q.shape[1], k.shape[1], q.shape[2]
    for row, s, pos in rows:
        j = torch.tensor(visible(lens[s], pos, window, sinks))
        blk, off = tables[s].long()[j // 16], j % 16
        for h in range(hq):
            kk, vv = (p[blk, h // (hq // hkv), off].double() for p in (k, v))
            want, bound = attention(q[row, h].double(), kk, vv, scale_of(dim), DT[dtype], weight)
            assert_within(got[row, h], want, bound, f"row {row} sequence {s} position {pos} head {h}")


def run_decode(lens, hq, hkv, dim, dtype, window, sinks, seed, maxb=None):
    first = [max(0, n - 1) for n in lens]
    pool, k, v, tables, gen = build(lens, first, hkv, dim, dtype, window, sinks, seed, maxb)
    q = torch.randn((len(lens), hq, dim), generator=gen).to(DT[dtype])
    status = new_status()
    out = paged_decode_attention_window(pool, q.cuda(), tables.cuda(),
                                        torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                        scale_of(dim), window, sinks, status)
    assert status_check(status) == (0, 0)
    for s, n in enumerate(lens):
        if n == 0:
            assert not bool(out[s].any())
    rows = [(s, s, n - 1) for s, n in enumerate(lens) if n]
    expect(q, k, v, tables, lens, first, rows, window, sinks, dtype, DECODE_WEIGHT[dtype], out)


@pytest.mark.parametrize("hq,hkv", [(4, 4), (8, 2), (16, 1), (12, 1), (10, 2), (9, 1)])
@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("f16", 128), ("bf16", 64), ("f16", 64)])
def test_decode_head_layouts(dtype, dim, hq, hkv):
    run_decode([1, 0, 16, 17, 130, 777], hq, hkv, dim, dtype, 100, 4, hq + dim)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 0), (16, 4), (17, 16), (33, 17), (64, 0),
                                          (100, 200), (5000, 4), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("dtype,dim,hq,hkv", [("bf16", 128, 8, 2), ("f16", 64, 12, 1)])
def test_decode_windows(dtype, dim, hq, hkv, window, sinks):
    run_decode([1, 0, 15, 16, 33, 100, 600, 1111], hq, hkv, dim, dtype, window, sinks, sinks % 97)


def test_decode_split_over_a_cluster():
    """Long windows with few heads: several CTAs per (sequence, kv head)."""
    run_decode([5003, 2, 400], 8, 1, 128, "bf16", 4000, 4, 31)
    run_decode([5003], 2, 2, 64, "f16", 2 ** 31 - 1, 0, 32, maxb=900)


def test_decode_bad_lengths_and_blocks():
    pool, k, v, tables, gen = build([40] * 5, [0] * 5, 2, 128, "bf16", 99, 0, 33, maxb=4)
    lens = [40, -1, 1000, 40, 40]
    tables[3, 1] = pool.num_blocks
    q = torch.randn((5, 8, 128), generator=gen).to(torch.bfloat16).cuda()
    status = new_status()
    dl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = paged_decode_attention_window(pool, q, tables.cuda(), dl, 0.1, 99, 0, status)
    assert status_check(status)[1] == DEV_BAD_LEN | DEV_BAD_BLOCK
    assert not bool(out[1:4].any()) and bool(out[0].any()) and bool(out[4].any())
    dl.fill_(40)
    out = paged_decode_attention_window(pool, q, tables.cuda(), dl, 0.1, 8, 0, status)
    assert status_check(status) == (0, 0) and bool(out[3].any())


def test_decode_infinite_scores():
    """A key of -inf products weighs nothing; the rest of the row is unharmed."""
    pool, k, v, tables, gen = build([20], [19], 1, 64, "f16", 99, 0, 34, maxb=2)
    q = torch.ones((1, 2, 64), dtype=torch.float16)
    k[tables[0, 0], 0, 0] = float("-inf")
    pool.k_pool.copy_(k)
    status = new_status()
    out = paged_decode_attention_window(pool, q.cuda(), tables.cuda(),
                                        torch.tensor([20], dtype=torch.int32, device="cuda"), 0.125, 99, 0, status)
    assert status_check(status) == (0, 0)
    j = torch.arange(1, 20)
    blk = tables[0].long()[j // 16]
    for h in range(2):
        want, bound = attention(q[0, h].double(), k[blk, 0, j % 16].double(), v[blk, 0, j % 16].double(),
                                0.125, torch.float16, 2.0 ** -22)
        assert_within(out[0, h], want, bound)


def test_decode_repeated_captured_and_concurrent():
    lens = [500, 33, 2000, 7]
    pool, k, v, tables, gen = build(lens, [n - 1 for n in lens], 2, 128, "bf16", 600, 4, 35)
    q = torch.randn((4, 8, 128), generator=gen).to(torch.bfloat16).cuda()
    status = new_status()
    args = (pool, q, tables.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), 0.1, 600, 4, status)
    first = paged_decode_attention_window(*args)
    graph, held = torch.cuda.CUDAGraph(), torch.zeros_like(q)
    with torch.cuda.graph(graph):
        paged_decode_attention_window(*args, out=held)
    outs = [torch.empty_like(q) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o in zip(streams, outs):
            paged_decode_attention_window(*args, out=o, stream=s)
        graph.replay()
    torch.cuda.synchronize()
    assert status_check(status) == (0, 0)
    for o in (*outs, held):
        assert torch.equal(first, o)


# ------------------------------------------------------------------------- prefill
def run_prefill(lens, chunks, hq, hkv, dim, dtype, window, sinks, seed, sample=None):
    first = [n - c for n, c in zip(lens, chunks)]
    pool, k, v, tables, gen = build(lens, first, hkv, dim, dtype, window, sinks, seed)
    T = sum(chunks)
    q = torch.randn((T, hq, dim), generator=gen).to(DT[dtype])
    start = torch.tensor([0] + list(np.cumsum(chunks)), dtype=torch.int32)
    ws = torch.empty(prefill_workspace_bytes(len(lens), T, hq, hkv), dtype=torch.uint8, device="cuda")
    status = new_status()
    out = paged_prefill_attention_window(pool, q.cuda(), tables.cuda(), start.cuda(),
                                         torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                         scale_of(dim), window, sinks, ws, status)
    assert status_check(status) == (0, 0)
    rows = [(int(start[s]) + i, s, first[s] + i) for s, c in enumerate(chunks) for i in range(c)]
    if sample:
        step = max(1, len(rows) // sample)
        rows = rows[::step] + rows[-1:]
    expect(q, k, v, tables, lens, first, rows, window, sinks, dtype, PREFILL_WEIGHT[dtype], out)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (16, 4), (63, 0), (64, 64), (65, 17), (257, 5),
                                          (130, 100), (5000, 0)])
@pytest.mark.parametrize("dtype,dim,hq,hkv", [("bf16", 128, 8, 2), ("f16", 64, 4, 4)])
def test_prefill_windows(dtype, dim, hq, hkv, window, sinks):
    run_prefill([700, 40, 1, 333], [90, 40, 1, 0], hq, hkv, dim, dtype, window, sinks, window, sample=50)


@pytest.mark.parametrize("hq,hkv", [(16, 1), (12, 1), (10, 2), (3, 3)])
@pytest.mark.parametrize("dtype,dim", [("bf16", 64), ("f16", 128)])
def test_prefill_head_layouts(dtype, dim, hq, hkv):
    run_prefill([500, 77], [60, 77], hq, hkv, dim, dtype, 100, 4, hq, sample=24)


@pytest.mark.parametrize("window,sinks", [(1, 0), (70, 4), (200, 33), (10 ** 6, 0)])
@pytest.mark.parametrize("dtype,dim,hq,hkv", [("bf16", 64, 32, 16), ("f16", 128, 20, 20)])
def test_prefill_many_items(dtype, dim, hq, hkv, window, sinks):
    """More items than SMs: two query tiles to an item, the second of some empty."""
    run_prefill([700, 400, 333, 64, 900], [300, 400, 100, 64, 130], hq, hkv, dim, dtype, window, sinks,
                window % 89, sample=16)


def test_prefill_long_chunk():
    """Many tiles per item, whole tiles hidden from the item's later rows."""
    run_prefill([4100], [600], 2, 2, 128, "bf16", 70, 4, 41, sample=40)
    run_prefill([3000, 2500], [1500, 900], 8, 2, 128, "bf16", 1024, 4, 42, sample=24)


def test_prefill_wide_window_is_the_causal_call():
    lens, chunks = [300, 64], [100, 64]
    pool, k, v, tables, gen = build(lens, [200, 0], 2, 128, "bf16", 10 ** 6, 0, 43)
    q = torch.randn((164, 8, 128), generator=gen).to(torch.bfloat16).cuda()
    start = torch.tensor([0, 100, 164], dtype=torch.int32, device="cuda")
    dl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = torch.empty(prefill_workspace_bytes(2, 164, 8, 2), dtype=torch.uint8, device="cuda")
    status = new_status()
    a = paged_prefill_attention(pool, q, tables.cuda(), start, dl, 0.1, ws, status)
    b = paged_prefill_attention_window(pool, q, tables.cuda(), start, dl, 0.1, 10 ** 6, 7, ws, status)
    assert status_check(status) == (0, 0)
    assert torch.equal(a, b)


@pytest.mark.parametrize("scale", [0.0, -0.125])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_zero_and_negative_scales(dtype, scale):
    """Scale 0 weighs every visible token alike; a negative one prefers small products."""
    lens, chunks, window, sinks = [200, 90], [140, 7], 33, 6
    first = [n - c for n, c in zip(lens, chunks)]
    pool, k, v, tables, gen = build(lens, first, 2, 64, dtype, window, sinks, 46)
    q = torch.randn((147, 4, 64), generator=gen).to(DT[dtype])
    start = torch.tensor([0, 140, 147], dtype=torch.int32, device="cuda")
    dl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = torch.empty(prefill_workspace_bytes(2, 147, 4, 2), dtype=torch.uint8, device="cuda")
    status = new_status()
    out = paged_prefill_attention_window(pool, q.cuda(), tables.cuda(), start, dl, scale, window, sinks, ws, status)
    last = q[[139, 146]].cuda()
    dec = paged_decode_attention_window(pool, last, tables.cuda(), dl, scale, window, sinks, status)
    assert status_check(status) == (0, 0)
    for row, s, pos in [(0, 0, 60), (77, 0, 137), (139, 0, 199), (146, 1, 89)]:
        j = torch.tensor(visible(lens[s], pos, window, sinks))
        blk, off = tables[s].long()[j // 16], j % 16
        for h in range(4):
            kk, vv = (p[blk, h // 2, off].double() for p in (k, v))
            want, bound = attention(-q[row, h].double(), kk, vv, -scale, DT[dtype], PREFILL_WEIGHT[dtype])
            assert_within(out[row, h], want, bound, f"row {row} head {h}")
            if row in (139, 146):
                assert_within(dec[s, h], want, bound, f"decode {s} head {h}")


def test_prefill_bad_sequences():
    pool, k, v, tables, gen = build([40, 40, 40], [0, 0, 0], 2, 64, "f16", 99, 0, 44)
    q = torch.randn((30, 4, 64), generator=gen).to(torch.float16).cuda()
    start = torch.tensor([0, 10, 20, 30], dtype=torch.int32, device="cuda")
    lens = torch.tensor([40, 5, 40], dtype=torch.int32, device="cuda")       # 5 < its chunk
    tables[2, 2] = -1
    ws = torch.empty(prefill_workspace_bytes(3, 30, 4, 2), dtype=torch.uint8, device="cuda")
    status = new_status()
    out = paged_prefill_attention_window(pool, q, tables.cuda(), start, lens, 0.1, 12, 0, ws, status)
    assert status_check(status)[1] == DEV_BAD_LEN | DEV_BAD_BLOCK
    assert bool(out[:10].any()) and not bool(out[10:].any())


# ----------------------------------------------------------- as a server calls them
@pytest.mark.parametrize("kind", ["bf16", "f16", "b8_bf16", "b8_f16"])
def test_append_then_attend(kind):
    """Prompts through the rotated append, the chunk's attention, then decode steps
    (append, attend), every output against 64 bits computed from the unrotated rows."""
    eight, dtype = kind.startswith("b8"), kind[-4:].lstrip("_")
    dt, hq, hkv, dim, rot, window, sinks = DT[dtype], 8, 2, 64, 32, 40, 3
    gen = torch.Generator().manual_seed(51)
    prompts, steps = [70, 5, 33], 4
    S, maxb, nb = 3, 8, 24
    pool = KVPool(nb, hkv, dim, kind, free_order=torch.randperm(nb, generator=gen).numpy(), device="cuda")
    if eight:
        pool.kv.fill_(0xFF)
    else:
        pool.k_pool.fill_(float("nan"))
        pool.v_pool.fill_(float("nan"))
    tables, lens = np.full((S, maxb), -1, np.int32), np.zeros(S, np.int32)
    table = rope_table(128, rot)
    status = new_status()
    past = [[torch.zeros((0, hkv, dim), dtype=torch.float64)] * 2 for _ in range(S)]
    for step in range(1 + steps):
        new = np.array(prompts if step == 0 else [1] * S, np.int32)
        slots = pool.append_slots(lens, new, tables)
        pos = np.concatenate([np.arange(a, a + n) for a, n in zip(lens, new)]).astype(np.int32)
        lens += new
        T = int(new.sum())
        qkv = torch.randn((T, (hq + 2 * hkv) * dim), generator=gen).to(dt)
        q, k, v = (p.view(T, -1, dim) for p in qkv.split([hq * dim, hkv * dim, hkv * dim], 1))
        gq, gk, gv = (p.view(T, -1, dim) for p in qkv.cuda().split([hq * dim, hkv * dim, hkv * dim], 1))
        q_rot = cache_write_rope(pool, gk, gv, torch.from_numpy(pos).cuda(), table.cuda(),
                                 torch.from_numpy(slots).cuda(), status, q=gq)
        dtab = torch.from_numpy(tables).cuda()
        dl = torch.from_numpy(lens).cuda()
        start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        if step == 0:
            ws = torch.empty(prefill_workspace_bytes(S, T, hq, hkv), dtype=torch.uint8, device="cuda")
            if eight:              # the 8-bit blocks as a 16-bit pool of the same numbering
                view = KVPool(nb, hkv, dim, dtype, device="cuda")
                dequantize_blocks(pool, torch.arange(nb, dtype=torch.int32, device="cuda"), view.k_pool,
                                  view.v_pool, status)
            out = paged_prefill_attention_window(view if eight else pool, q_rot, dtab,
                                                 torch.from_numpy(start).cuda(), dl, scale_of(dim), window,
                                                 sinks, ws, status)
        elif eight:
            out = paged_decode_attention_b8(pool, q_rot, dtab, dl, scale_of(dim), status, window=window,
                                            sinks=sinks)
        else:
            out = paged_decode_attention_window(pool, q_rot, dtab, dl, scale_of(dim), window, sinks, status)
        assert status_check(status) == (0, 0)
        kd, _ = rotate(k.double(), table, torch.from_numpy(pos).long(), False)
        qd, _ = rotate(q.double(), table, torch.from_numpy(pos).long(), False)
        for s in range(S):
            a, b = int(start[s]), int(start[s + 1])
            past[s] = [torch.cat([past[s][0], kd[a:b]]), torch.cat([past[s][1], v[a:b].double()])]
            for row in range(a, b, 7):
                p = int(pos[row])
                j = torch.tensor(visible(p + 1, p, window, sinks))
                for h in range(hq):
                    kk, vv = (x[j, h // (hq // hkv)] for x in past[s])
                    want, bound = attention(qd[row, h], kk, vv, scale_of(dim), dt, F16_HALF_STEP)
                    # what the cache rounds: a relative 2^-8 / 2^-11 of K and q, or half a step
                    # of an 8-bit block (and one more for each time its scale grew, at most
                    # the steps taken), at most 5 half steps of the largest value / 127
                    half = {torch.bfloat16: 2.0 ** -8, torch.float16: F16_HALF_STEP}[dt]
                    ek = kk.abs().max().item() / 127 * 2.5 if eight else 0.0
                    ev = vv.abs().max().item() / 127 * 2.5 if eight else 0.0
                    if eight:      # a block may also hold larger values that the window hides
                        ek, ev = (x.abs().max().item() / 127 * 2.5 for x in past[s])
                    dx = scale_of(dim) * (2 * half * (kk.abs() @ qd[row, h].abs()).max().item()
                                          + ek * qd[row, h].abs().sum().item() * (1 + half))
                    w = torch.softmax((kk @ qd[row, h]) * scale_of(dim), 0)
                    bound = bound + 2 * np.expm1(2 * dx) / 2 * (w @ vv.abs()) + ev * np.exp(2 * dx) + half * (w @ vv.abs()) * (2 if eight else 0)
                    assert_within(out[row, h], want, bound, f"step {step} row {row} head {h}")


@pytest.mark.parametrize("exponent", [0, 8, 15, 45])
@pytest.mark.parametrize("kind", ["bf16", "f16", "b8_bf16", "b8_f16"])
def test_large_scores(kind, exponent):
    """Scores of 2^16 to 2^64, exact in fp32 and far apart: only the largest visible
    keys count.  Prefill takes every key of a row against one reference, so those count
    alike and the row is the mean of their V; its roundings: a weight's on its way into
    P V (the sum takes it unrounded), the sum and the quotient in fp32 (2^-20 leaves
    room) and the result's own, half a step.  Decode's reference moves
    from block to block and the scale's product is rounded when it does: a weight is off
    by a factor of up to 2^(|score| 2^-23), so equal scores of 2^18 count alike to 2 % and
    the largest ones in any proportion, where the row is some mean of their V."""
    dtype = kind.split("_")[-1]
    if exponent > 15 and dtype == "f16":
        exponent, unit = 15, 2.0 ** 10           # fp16 ends at 2^16
    else:
        unit = 2.0 ** 12
    hkv, hq, dim, n, window, sinks, chunk = 2, 4, 64, 300, 90, 3, 150
    gen = torch.Generator().manual_seed(exponent)
    tables, nb = random_case(gen, [n], hkv, 20)
    level = torch.randint(1, 6, (nb, hkv, 16, 1), generator=gen).double()
    k = (level * unit).expand(nb, hkv, 16, dim).to(DT[dtype])
    v = torch.randn((nb, hkv, 16, dim), generator=gen).to(DT[dtype])
    q = torch.full((chunk, hq, dim), 2.0 ** exponent).to(DT[dtype])
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    status = new_status()
    pool = KVPool(nb, hkv, dim, kind, device="cuda")
    if pool.is_b8:
        slots = torch.arange(nb * 16, device="cuda")
        cache_write_b8(pool, *(t.permute(0, 2, 1, 3).reshape(-1, hkv, dim).contiguous().cuda()
                               for t in (k, v)), slots, status)
        kb, vb = torch.empty((2, nb, hkv, 16, dim), dtype=DT[dtype], device="cuda")
        dequantize_blocks(pool, torch.arange(nb, dtype=torch.int32, device="cuda"), kb, vb, status)
        outs = [(n - 1, paged_decode_attention_b8(pool, q[:1].cuda(), tables.cuda(), lens, 0.125, status,
                                                  window=window, sinks=sinks)[0])]
        v = vb.cpu()
    else:
        pool.k_pool.copy_(k)
        pool.v_pool.copy_(v)
        out = paged_decode_attention_window(pool, q[:1].cuda(), tables.cuda(), lens, 0.125, window, sinks,
                                            status)
        ws = torch.empty(prefill_workspace_bytes(1, chunk, hq, hkv), dtype=torch.uint8, device="cuda")
        start = torch.tensor([0, chunk], dtype=torch.int32, device="cuda")
        rows = paged_prefill_attention_window(pool, q.cuda(), tables.cuda(), start, lens, 0.125, window,
                                              sinks, ws, status)
        outs = [(n - 1, out[0])] + [(n - chunk + i, rows[i]) for i in range(chunk)]
    assert status_check(status) == (0, 0)
    for pos, got in outs:
        j = torch.tensor(visible(n, pos, window, sinks))
        blk, off = tables[0].long()[j // 16], j % 16
        for h in range(hq):
            lv = level[blk, h // 2, off, 0]
            top = lv == lv.max()
            vv = v[blk, h // 2, off].double()
            half = torch.finfo(DT[dtype]).eps / 2
            if got is outs[0][1]:        # decode: any mix of the largest
                lo, hi = vv[top].min(0).values, vv[top].max(0).values
                # the result's rounding and, of an 8-bit pool's V, the read-back's: half a step each
                room = 2 * half * (1 + half) * vv[top].abs().max(0).values + 1e-6
                g = got[h].double().cpu()
                assert ((g >= lo - room) & (g <= hi + room)).all(), (pos, h)
            else:
                want = vv[top].mean(0)
                room = half * want.abs() + (PREFILL_WEIGHT[dtype] + 2.0 ** -20) * vv[top].abs().max(0).values
                assert ((got[h].double().cpu() - want).abs() <= room).all(), (pos, h)


@pytest.mark.parametrize("n", [1, 31, 32, 33, 70])
def test_prefill_numbers_of_sequences(n):
    """Around the number of sequences up to which each CTA lists the items for itself;
    a third of them without a row, every seventh with a length that does not fit."""
    gen = torch.Generator().manual_seed(n)
    chunks = [0 if i % 3 == 1 else 1 + (37 * i) % 90 for i in range(n)]
    lens = [c + (i * 29) % 200 for i, c in enumerate(chunks)]
    bad = [i for i in range(n) if i % 7 == 3]
    first = [a - c for a, c in zip(lens, chunks)]
    pool, k, v, tables, gen = build(lens, first, 2, 64, "bf16", 60, 3, n)
    T = sum(chunks) + 5                                  # rows behind the last sequence
    q = torch.randn((T, 8, 64), generator=gen).to(torch.bfloat16)
    start = torch.tensor([0] + list(np.cumsum(chunks)), dtype=torch.int32)
    given = torch.tensor([(-1 if i % 2 else chunks[i] - 1) if i in bad else lens[i] for i in range(n)],
                         dtype=torch.int32)
    ws = torch.empty(prefill_workspace_bytes(n, T, 8, 2), dtype=torch.uint8, device="cuda")
    status = new_status()
    out = torch.full((T, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    paged_prefill_attention_window(pool, q.cuda(), tables.cuda(), start.cuda(), given.cuda(), scale_of(64),
                                   60, 3, ws, status, out=out)
    assert status_check(status)[1] == (DEV_BAD_LEN if bad else 0)
    assert bool((out[T - 5:] == 7).all())
    rows = []
    for s, c in enumerate(chunks):
        if s in bad:
            assert not bool(out[start[s]:start[s + 1]].any())
        elif c:
            rows += [(int(start[s]) + i, s, first[s] + i) for i in {0, c // 2, c - 1}]
    expect(q, k, v, tables, lens, first, rows, 60, 3, "bf16", PREFILL_WEIGHT["bf16"], out)
