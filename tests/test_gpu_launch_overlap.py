"""Calls that follow one another on a stream may overlap in their set-up and never in
their work: a chain of dependent calls gives, without a synchronisation between them
and from a captured graph, bit for bit what it gives with one after every call."""
import pytest

torch = pytest.importorskip("torch")

import libbuild  # noqa: E402

libbuild.ensure_built()
import paged_kv_cache_146_gb300 as P  # noqa: E402

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32
HKV, HQ, D, NB = 2, 8, 64, 96


class Chain:
    """Decode steps of S sequences, every buffer used again in each step: the row
    buffers are filled, rotated in place and appended, attended, and the answer is the
    next step's rows."""

    def __init__(self, kind, S, between):
        gen = torch.Generator(device="cuda").manual_seed(5)
        self.kind, self.S, self.between = kind, S, between
        self.pool = P.KVPool(NB * S, HKV, D, "b8_bf16" if kind == "b8" else "bf16", device="cuda")
        for t in (self.pool.kv, self.pool.k_pool, self.pool.v_pool):
            if t is not None:
                t.zero_()
        self.tables = torch.arange(NB * S, dtype=I32, device="cuda").view(S, NB)
        self.pos = torch.zeros(S, dtype=I32, device="cuda")
        self.lens = torch.zeros(S, dtype=I32, device="cuda")
        self.slots = torch.zeros(S, dtype=torch.int64, device="cuda")
        self.base = torch.arange(S, device="cuda") * (NB * 16)
        self.rows = torch.randn(S, (HQ + 2 * HKV) * D, device="cuda", generator=gen).to(BF)
        self.q = torch.zeros(S, HQ, D, dtype=BF, device="cuda")
        self.k, self.v = (torch.zeros(S, HKV, D, dtype=BF, device="cuda") for _ in "kv")
        self.out = torch.zeros(S, HQ, D, dtype=BF, device="cuda")
        self.table = P.rope_table(NB * 16, D, device="cuda")
        self.status = torch.zeros(1, dtype=I32, device="cuda")
        self.ids = torch.zeros(S, dtype=I32, device="cuda")
        self.back = [torch.zeros(S, HKV, 16, D, dtype=BF, device="cuda") for _ in "kv"]
        self.trace = torch.zeros(S, HQ, D, device="cuda")
        self.starts = torch.arange(S + 1, dtype=I32, device="cuda")
        self.ws = torch.empty(P.prefill_workspace_bytes(S, S, HQ, HKV), dtype=torch.uint8,
                              device="cuda")

    def step(self):
        f = self.between
        self.slots.copy_(self.pos + self.base)
        self.lens.copy_(self.pos + 1)
        self.q.copy_(self.rows[:, :HQ * D].view(self.S, HQ, D))
        self.k.copy_(self.rows[:, HQ * D:(HQ + HKV) * D].view(self.S, HKV, D))
        self.v.copy_(self.rows[:, (HQ + HKV) * D:].view(self.S, HKV, D))
        f()
        P.cache_write_rope(self.pool, self.k, self.v, self.pos, self.table, self.slots, self.status,
                           q=self.q, q_out=self.q)
        f()
        if self.kind == "b8":
            P.paged_decode_attention_b8(self.pool, self.q, self.tables, self.lens, 0.125,
                                        self.status, window=30, sinks=2, out=self.out)
            f()
            self.ids.copy_(self.slots // 16)
            P.dequantize_blocks(self.pool, self.ids, *self.back, self.status)
            f()
            P.cache_write_rope(self.pool, self.back[0][:, :, 3].contiguous(), self.v, self.pos,
                               self.table, self.slots, self.status)
        elif self.kind == "decode":
            P.paged_decode_attention_window(self.pool, self.q, self.tables, self.lens, 0.125, 30, 2,
                                            self.status, out=self.out)
        else:
            P.paged_prefill_attention_window(self.pool, self.q, self.tables, self.starts, self.lens,
                                             0.125, 30, 2, self.ws, self.status, out=self.out)
        f()
        # the answer becomes the next rows (written over what the calls just read)
        self.rows[:, :HQ * D].copy_(self.out.view(self.S, -1))
        self.rows[:, HQ * D:].mul_(0.5).add_(self.out.view(self.S, -1)[:, :2 * HKV * D], alpha=0.5)
        self.trace.add_(self.out)
        self.pos.add_(1)
        f()

    def result(self):
        torch.cuda.synchronize()
        assert self.status.item() == 0
        pools = [t for t in (self.pool.kv, self.pool.k_pool, self.pool.v_pool) if t is not None]
        return [self.trace, self.rows, self.q, *pools]


@pytest.mark.parametrize("S", [1, 3, 70])
@pytest.mark.parametrize("kind", ["decode", "b8", "prefill"])
def test_a_chain_of_calls(kind, S):
    steps = 45
    want = Chain(kind, S, torch.cuda.synchronize)
    for _ in range(steps):
        want.step()
    want = want.result()
    assert want[0].abs().sum() > 0

    eager = Chain(kind, S, lambda: None)
    for _ in range(steps):
        eager.step()
    graphed = Chain(kind, S, lambda: None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graphed.step()                                   # uncaptured first step
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(4):
            graphed.step()
    for _ in range((steps - 1) // 4):
        graph.replay()
    for got in (eager.result(), graphed.result()):
        for a, b in zip(got, want):
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
