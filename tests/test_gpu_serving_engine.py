"""The decode engine and the captured call with rotation, windows and block-scaled
pools: the same bits as the calls made one by one."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_cache_146_gb300 import (CapturedDecode, KVPool, block_copy, cache_write_b8,  # noqa: E402
                                      cache_write_rope, paged_decode_attention_b8,
                                      paged_decode_attention_window, rope_table, status_check)
from paged_kv_cache_146_gb300.engine import DecodeEngine  # noqa: E402

pytestmark = pytest.mark.gpu
S, HQ, HKV, D, MAXB, NB = 5, 8, 2, 128, 20, 80
PROMPTS = [100, 1, 16, 250, 33]
SCALE = D ** -0.5


def rows(gen, n, heads, dt):
    return torch.randn((n, heads, D), generator=gen).to(dt)


def engine(kind, window, sinks, rope=True):
    gen = torch.Generator().manual_seed(7)
    dt = torch.bfloat16 if kind.endswith("bf16") else torch.float16
    pool = KVPool(NB, HKV, D, kind, free_order=torch.randperm(NB, generator=gen).numpy(), device="cuda")
    for p in (pool.k_pool, pool.v_pool, pool.kv):
        if p is not None:
            p.fill_(0xFF if p.dtype == torch.uint8 else float("nan"))
    eng = DecodeEngine(pool, S, HQ, MAXB, SCALE, "cuda", rope=rope_table(400, 64).cuda() if rope else None,
                       rope_interleaved=True, window=window, sinks=sinks)
    T = sum(PROMPTS)
    q = rows(gen, T, HQ, dt).cuda()
    eng.prefill(rows(gen, T, HKV, dt).cuda(), rows(gen, T, HKV, dt).cuda(), PROMPTS, q_rows=q if rope else None)
    return eng, gen, dt, q


def attend(eng, q):
    dl, dt = torch.from_numpy(eng.lens).cuda(), torch.from_numpy(eng.tables).cuda()
    if eng.pool.is_b8:
        return paged_decode_attention_b8(eng.pool, q, dt, dl, SCALE, eng.status, window=eng.window, sinks=eng.sinks)
    return paged_decode_attention_window(eng.pool, q, dt, dl, SCALE, eng.window or 10 ** 6, eng.sinks, eng.status)


@pytest.mark.parametrize("kind,window,sinks,rope", [
    ("bf16", 60, 4, True), ("f16", 17, 0, False), ("b8_bf16", None, 0, True), ("b8_f16", 90, 20, True),
    ("b8_bf16", 40, 2, False)])
def test_engine_steps_equal_the_calls(kind, window, sinks, rope):
    eng, gen, dt, q_prompt = engine(kind, window, sinks, rope)
    twin, _, _, _ = engine(kind, window, sinks, rope)
    host_eng, _, _, _ = engine(kind, window, sinks, rope)
    table = rope_table(400, 64).cuda()
    host, outs, host_outs = [], [], []
    for _ in range(4):
        q, k, v = rows(gen, S, HQ, dt), rows(gen, S, HKV, dt), rows(gen, S, HKV, dt)
        host.append([x.pin_memory() for x in (q, k, v)])
        outs.append(eng.decode_step(q.cuda(), k.cuda(), v.cuda()).clone())
        # by hand, on a second pool in the same state
        slots = torch.from_numpy(twin.pool.append_slots(twin.lens, np.ones(S, np.int32), twin.tables)).cuda()
        pos = torch.from_numpy(twin.lens.copy()).cuda()
        twin.lens += 1
        gq = q.cuda()
        if rope:
            gq = cache_write_rope(twin.pool, k.cuda(), v.cuda(), pos, table, slots, twin.status, q=gq,
                                  interleaved=True)
        else:
            twin.write(k.cuda(), v.cuda(), slots)
        assert torch.equal(outs[-1], attend(twin, gq))
    for q, k, v in host:
        host_outs.append(torch.empty((S, HQ, D), dtype=dt).pin_memory())
        host_eng.decode_step_host(q, k, v, host_outs[-1])
    host_eng.join_copies()
    torch.cuda.synchronize()
    for e in (eng, twin, host_eng):
        assert e.check() == (0, 0)
    for a, b in zip(outs, host_outs):
        assert torch.equal(a.cpu(), b)
    assert not bool(torch.isnan(outs[-1]).any())


def test_prompt_queries_are_rotated_in_place():
    gen = torch.Generator().manual_seed(7)
    torch.randperm(NB, generator=gen)
    T = sum(PROMPTS)
    raw = rows(gen, T, HQ, torch.bfloat16)
    eng, _, _, q = engine("bf16", 60, 4)
    pool = KVPool(NB, HKV, D, "bf16", device="cuda")
    pos = torch.from_numpy(np.concatenate([np.arange(n) for n in PROMPTS]).astype(np.int32)).cuda()
    kv = rows(gen, T, HKV, torch.bfloat16).cuda()
    want = cache_write_rope(pool, kv, kv, pos, rope_table(400, 64).cuda(), torch.arange(T, device="cuda"),
                            eng.status, q=raw.cuda(), interleaved=True)
    assert eng.check() == (0, 0) and torch.equal(q, want)


@pytest.mark.parametrize("kind,window", [("bf16", 60), ("b8_bf16", None), ("b8_f16", 60)])
def test_captured_call_follows_its_buffers(kind, window):
    eng, gen, dt, _ = engine(kind, window, 4 if window else 0)
    q = torch.zeros((S, HQ, D), dtype=dt, device="cuda")
    tables = torch.full((S, MAXB), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(S, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    cap = CapturedDecode(eng.pool, q, tables, lens, SCALE, None, eng.status, out, window=window,
                         sinks=4 if window else 0)
    tables.copy_(torch.from_numpy(eng.tables))
    lens.copy_(torch.from_numpy(eng.lens))
    for _ in range(2):
        q.copy_(rows(gen, S, HQ, dt))
        assert torch.equal(cap.replay(), attend(eng, q))
    assert eng.check() == (0, 0)


def test_copy_on_write_of_an_8bit_tail():
    """A forked sequence copies the shared tail's record, scale and all, before it
    appends to it; the parent's values stay."""
    gen = torch.Generator().manual_seed(9)
    pool = KVPool(8, HKV, D, "b8_bf16", device="cuda")
    tables, lens = np.full((2, 4), -1, np.int32), np.array([0, 0], np.int32)
    k = rows(gen, 20, HKV, torch.bfloat16).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = pool.append_slots(lens, np.array([20, 0], np.int32), tables)
    cache_write_b8(pool, k, k, torch.from_numpy(slots).cuda(), status)
    pool.fork(tables[0], 20, tables[1])
    lens[:] = 20
    q = rows(gen, 2, HQ, torch.bfloat16).cuda()
    dl = torch.tensor([20, 20], dtype=torch.int32, device="cuda")
    before = paged_decode_attention_b8(pool, q, torch.from_numpy(tables).cuda(), dl, SCALE, status)
    slots, copies = pool.append_slots_cow(lens, np.array([0, 1], np.int32), tables)
    assert len(copies) == 1
    src, dst = (torch.from_numpy(np.ascontiguousarray(copies[:, i])).cuda() for i in range(2))
    block_copy(pool, src, dst, status)
    big = 100 * rows(gen, 1, HKV, torch.bfloat16).cuda()
    cache_write_b8(pool, big, big, torch.from_numpy(slots).cuda(), status)
    after = paged_decode_attention_b8(pool, q, torch.from_numpy(tables).cuda(), dl, SCALE, status)
    assert status_check(status) == (0, 0)
    assert torch.equal(before[0], after[0]) and not torch.equal(before[1], after[1])


def test_engine_refusals():
    q8 = KVPool(8, 2, 128, "q8_bf16", device="cuda")
    b8 = KVPool(8, 2, 128, "b8_bf16", device="cuda")
    with pytest.raises(ValueError, match="block-scaled"):
        DecodeEngine(q8, 2, 4, 4, 0.1, "cuda", window=8)
    with pytest.raises(ValueError, match="sinks without"):
        DecodeEngine(b8, 2, 4, 4, 0.1, "cuda", sinks=8)
    with pytest.raises(ValueError, match="own split"):
        DecodeEngine(b8, 2, 4, 4, 0.1, "cuda", blocks_per_split=32)
