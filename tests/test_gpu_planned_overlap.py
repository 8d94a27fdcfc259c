"""The planned decode begins with its main kernel, which clears the output rows of idle
sequences.  Behind a call that lets its successor start early (appends, windowed and
block-scaled decode, read-back) it must not do so before that call has ended: the same
bits with and without a synchronisation after every call, eager and from a graph."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import libbuild  # noqa: E402

libbuild.ensure_built()
import paged_kv_cache_146_gb300 as P  # noqa: E402
from paged_kv_cache_146_gb300.engine import DecodeEngine  # noqa: E402

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32
HQ, HKV, D, S = 8, 2, 128, 24
LONG, LONG_SEQS, MAXB = 48000, 2, 8
SCALE = D ** -0.5


class Steps:
    """A long call that leaves most SMs free, then calls whose buffers are used twice."""

    def __init__(self, sync):
        gen = torch.Generator(device="cuda").manual_seed(3)

        def randn(*shape):
            return torch.randn(shape, generator=gen, device="cuda", dtype=BF)

        self.sync = sync
        # two sequences of 3,000 blocks: few long pairs, tens of microseconds on few SMs
        nb = LONG // 16
        self.long = P.KVPool(LONG_SEQS * nb, 1, D, "bf16", device="cuda")
        self.long.k_pool.copy_(randn(*self.long.k_pool.shape))
        self.long.v_pool.copy_(randn(*self.long.v_pool.shape))
        self.long_tables = torch.arange(LONG_SEQS * nb, dtype=I32, device="cuda").view(LONG_SEQS, nb)
        self.long_lens = torch.full((LONG_SEQS,), LONG, dtype=I32, device="cuda")
        self.long_q = randn(LONG_SEQS, HQ, D)
        self.status = torch.zeros(1, dtype=I32, device="cuda")

        self.pool = P.KVPool(S * MAXB, HKV, D, "bf16", device="cuda")
        self.pool.k_pool.copy_(randn(*self.pool.k_pool.shape))
        self.pool.v_pool.copy_(randn(*self.pool.v_pool.shape))
        tables = np.arange(S * MAXB, dtype=np.int32).reshape(S, MAXB)
        lens = np.zeros(S, np.int32)
        lens[[5, 17]] = 100, 37                          # the other rows are idle
        self.plan = torch.zeros(P.decode_plan_bytes(S, HQ, HKV, D, MAXB), dtype=torch.uint8).pin_memory()
        assert P.decode_plan(self.pool, lens, tables, HQ, self.plan) == 0
        self.ws = torch.zeros(P.decode_workspace_bytes(S, HQ, HKV, D, MAXB), dtype=torch.uint8, device="cuda")
        self.ws[:len(self.plan)].copy_(self.plan)
        self.tables, self.lens = torch.from_numpy(tables).cuda(), torch.from_numpy(lens).cuda()
        self.idle = torch.from_numpy(lens == 0).cuda()
        # every sequence's last block takes the appended token
        self.slots = torch.arange(S, device="cuda") * (MAXB * 16) + MAXB * 16 - 3
        self.pos = torch.arange(S, dtype=I32, device="cuda")
        self.cos_sin = P.rope_table(64, D, device="cuda")
        self.fused = randn(S, (HQ + 2 * HKV) * D)
        self.first = self.fused.clone()
        self.q_out = torch.zeros(S, HQ, D, dtype=BF, device="cuda")
        self.all_lens = torch.full((S,), MAXB * 16, dtype=I32, device="cuda")

    def long_call(self):
        P.paged_decode_attention_window(self.long, self.long_q, self.long_tables, self.long_lens, SCALE,
                                        LONG, 0, self.status)
        self.sync()

    def append(self):
        f = self.fused
        P.cache_write_rope(self.pool, f[:, HQ * D:(HQ + HKV) * D].view(S, HKV, D),
                           f[:, (HQ + HKV) * D:].view(S, HKV, D), self.pos, self.cos_sin, self.slots,
                           self.status, q=f[:, :HQ * D].view(S, HQ, D), q_out=self.q_out)
        self.sync()

    def planned(self, out):
        P.paged_decode_attention_planned(self.pool, self.q_out, self.tables, self.lens, SCALE, 0, self.ws,
                                         self.status, out=out)
        self.sync()

    def rows_reused(self):
        """The append's rows are dropped after it, and the planned call's output lands there."""
        out = self.fused.view(-1)[:S * HQ * D].view(S, HQ, D)
        self.fused.copy_(self.first)
        self.long_call()
        self.append()
        self.planned(out)
        return [out.clone(), self.q_out.clone(), self.pool.k_pool.clone(), self.pool.v_pool.clone()]

    def out_reused(self):
        """One output buffer for a windowed call of all sequences and a planned call of few."""
        out = self.first.view(-1)[:S * HQ * D].view(S, HQ, D).clone()
        self.long_call()
        P.paged_decode_attention_window(self.pool, self.q_out, self.tables, self.all_lens, SCALE, 60, 2,
                                        self.status, out=out)
        self.sync()
        self.planned(out)
        return [out.clone()]


@pytest.mark.parametrize("what", ["rows_reused", "out_reused"])
def test_idle_rows_are_cleared_after_the_call_before(what):
    synced, eager, graphed = Steps(torch.cuda.synchronize), Steps(lambda: None), Steps(lambda: None)
    want = getattr(synced, what)()
    assert not want[0][synced.idle].any() and want[0][~synced.idle].abs().sum() > 0
    for _ in range(3):
        got = getattr(eager, what)()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        getattr(graphed, what)()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = getattr(graphed, what)()
    for _ in range(3):
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert [s.status.item() for s in (synced, eager, graphed)] == [0, 0, 0]


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_rotating_engine_without_a_window_equals_the_calls(kind):
    """An append stands right before the planned kernel in every step."""
    dt = BF if kind == "bf16" else torch.float16
    prompts, n = [100, 1, 16, 250, 33], 5
    table = P.rope_table(400, 64).cuda()

    def engine():
        gen = torch.Generator().manual_seed(7)
        pool = P.KVPool(80, HKV, D, kind, free_order=torch.randperm(80, generator=gen).numpy(), device="cuda")
        pool.k_pool.fill_(float("nan"))
        pool.v_pool.fill_(float("nan"))
        eng = DecodeEngine(pool, n, HQ, 20, SCALE, "cuda", rope=table)
        k, v = (torch.randn((sum(prompts), HKV, D), generator=gen).to(dt).cuda() for _ in "kv")
        eng.prefill(k, v, prompts)
        return eng, gen

    eng, gen = engine()
    twin, _ = engine()
    assert eng.planned
    ws = torch.empty(P.decode_workspace_bytes(n, HQ, HKV, D, 20), dtype=torch.uint8, device="cuda")
    rows = [[torch.randn((n, h, D), generator=gen).to(dt).cuda() for h in (HQ, HKV, HKV)] for _ in range(12)]
    outs = [eng.decode_step(*(x.clone() for x in r)).clone() for r in rows]     # nothing waits in between
    for (q, k, v), got in zip(rows, outs):
        slots = torch.from_numpy(twin.pool.append_slots(twin.lens, np.ones(n, np.int32), twin.tables)).cuda()
        pos = torch.from_numpy(twin.lens.copy()).cuda()
        twin.lens += 1
        gq = P.cache_write_rope(twin.pool, k, v, pos, table, slots, twin.status, q=q)
        torch.cuda.synchronize()
        want = P.paged_decode_attention(twin.pool, gq, torch.from_numpy(twin.tables).cuda(),
                                        torch.from_numpy(twin.lens.copy()).cuda(), SCALE, ws, twin.status)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    assert eng.check() == (0, 0) and twin.check() == (0, 0)
