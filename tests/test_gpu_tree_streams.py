"""Calls for trees of drafted tokens on a stream of their own, while work is queued on the
current one."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import libbuild  # noqa: E402
import paged_kv_cache_146_gb300 as P  # noqa: E402
from tree_reference import TreeCase, accept_path, mask_words, random_parents  # noqa: E402

libbuild.ensure_built()
pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def busy():
    """Some tens of milliseconds of ordinary work on the current stream."""
    a = torch.ones((8192, 8192), dtype=torch.bfloat16, device="cuda")
    b = torch.empty_like(a)
    for _ in range(40):
        torch.matmul(a, a, out=b)


def trees(seed, news):
    gen = torch.Generator().manual_seed(seed)
    parents = [random_parents(n, gen) for n in news]
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    tokens, targets = (torch.randint(0, 2, (starts[-1],), generator=gen) for _ in range(2))
    first = [5 * s for s in range(len(news))]
    kept, num, nxt = [-1] * starts[-1], [], []
    for s, n in enumerate(news):
        a, b = starts[s], starts[s + 1]
        path = accept_path(tokens[a:b].tolist(), parents[s], targets[a:b].tolist())
        kept[a:a + len(path)] = [first[s] + i for i in path]
        num.append(len(path))
        nxt.append(int(targets[a + path[-1]]) if path else -1)
    args = [tokens.cuda(), ints([x for p in parents for x in p]), targets.cuda(), ints(starts), ints(first)]
    return args, kept, num, nxt


@pytest.mark.parametrize("compiled", [True, False])
@pytest.mark.parametrize("as_int", [False, True])
def test_accept_makes_its_results_on_its_own_stream(as_int, compiled, monkeypatch):
    """What it makes itself is filled before its kernel, however much the current stream has to do."""
    assert P._load_torch()
    if not compiled:
        monkeypatch.setattr(P, "_fast", None)
    args, kept, num, nxt = trees(3, [40, 0, 17, 64, 200])
    status, side = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    busy()
    got = P.tree_accept(*args, status, stream=side.cuda_stream if as_int else side)
    torch.cuda.synchronize()
    assert status.item() == 0
    assert [t.tolist() for t in got] == [kept, num, nxt]


@pytest.mark.parametrize("as_int", [False, True])
def test_accept_on_the_default_stream(as_int):
    """The other way round: work is queued on a stream of the caller's, the call goes to the default one."""
    args, kept, num, nxt = trees(4, [9, 30])
    status, default = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.cuda.default_stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        busy()
        got = P.tree_accept(*args, status, stream=default.cuda_stream if as_int else default)
        torch.cuda.synchronize()
    assert status.item() == 0
    assert [t.tolist() for t in got] == [kept, num, nxt]


def plain_call(name):
    """One small call without `out`, all else made: a function of the stream."""
    kind = {"decode_b8": "b8_bf16", "decode_q8": "q8_bf16"}.get(name, "bf16")
    n = 1 if "decode" in name else 6
    c = TreeCase([70 - n], [n], 8, 2, 128, torch.bfloat16, 1)
    pool = P.KVPool(c.nb, 2, 128, kind, device="cuda")
    if pool.record_bytes:
        pool.kv.zero_()
    else:
        pool.k_pool.copy_(c.k.nan_to_num())
        pool.v_pool.copy_(c.v.nan_to_num())
    size = max(P.tree_workspace_bytes(n, 8, 2, 128), P.prefill_workspace_bytes(1, n, 8, 2),
               P.decode_workspace_bytes(1, 8, 2, 128, c.maxb))
    ws, status = torch.zeros(size, dtype=torch.uint8, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    q, tables, starts, lens = c.q.cuda(), c.tables.cuda(), ints([0, n]), ints(c.lens)
    mask, rot, pos = mask_words(c.masks, 1).cuda(), P.rope_table(100, 128, device="cuda"), ints([0] * n)
    slot = torch.arange(n, device="cuda")
    rows = torch.ones((n, 2, 128), dtype=torch.bfloat16, device="cuda")
    if name == "decode_planned":
        plan = torch.zeros(P.decode_plan_bytes(1, 8, 2, 128, c.maxb), dtype=torch.uint8)
        items = P.decode_plan(pool, np.array(c.lens, dtype=np.int32), c.tables.numpy(), 8, plan)
        ws[:plan.numel()].copy_(plan)
    calls = {
        "tree": lambda st: P.paged_tree_attention(pool, q, tables, starts, lens, mask, 0.1, ws, status, stream=st),
        "prefill": lambda st: P.paged_prefill_attention(pool, q, tables, starts, lens, 0.1, ws, status, stream=st),
        "prefill_window": lambda st: P.paged_prefill_attention_window(pool, q, tables, starts, lens, 0.1, 20, 2,
                                                                      ws, status, stream=st),
        "decode": lambda st: P.paged_decode_attention(pool, q, tables, lens, 0.1, ws, status, stream=st),
        "decode_planned": lambda st: P.paged_decode_attention_planned(pool, q, tables, lens, 0.1, items, ws,
                                                                      status, stream=st),
        "decode_window": lambda st: P.paged_decode_attention_window(pool, q, tables, lens, 0.1, 20, 2, status,
                                                                    stream=st),
        "decode_b8": lambda st: P.paged_decode_attention_b8(pool, q, tables, lens, 0.1, status, stream=st),
        "decode_q8": lambda st: P.paged_decode_attention_q8(pool, q, tables, lens, 0.1, ws, status, stream=st),
        "rope": lambda st: P.cache_write_rope(pool, rows, rows, pos, rot, slot, status, q=q, stream=st)}
    return calls[name], q, status


@pytest.mark.parametrize("name", ["tree", "prefill", "prefill_window", "decode", "decode_planned", "decode_window",
                                  "decode_b8", "decode_q8", "rope"])
def test_outputs_do_not_lie_where_queued_work_writes(name):
    """The current stream still has to write a tensor that has been let go: its memory is not given to
    a call on another stream.  And the other way: memory that the call has made is not given away
    while the current stream has yet to read it."""
    call, q, status = plain_call(name)
    want, side = call(None), torch.cuda.Stream()
    call(side)
    torch.cuda.synchronize()
    busy()
    late = torch.empty_like(q)
    late.fill_(7.0)
    del late
    got = call(side)
    torch.cuda.synchronize()
    assert status.item() == 0 and torch.equal(got, want)
    del got
    busy()
    got = call(side)
    torch.cuda.current_stream().wait_stream(side)
    copy = got.clone()
    del got
    with torch.cuda.stream(side):
        for _ in range(4):
            torch.empty_like(q).fill_(9.0)
    torch.cuda.synchronize()
    assert torch.equal(copy, want)


@pytest.mark.parametrize("name", ["tree", "accept"])
def test_a_captured_call_on_a_stream_of_its_own(name):
    """A capture that forks to the call's stream and joins it again; the results are the graph's."""
    if name == "tree":
        call, q, status = plain_call("tree")
        want = call(None)
    else:
        args, kept, num, nxt = trees(5, [30, 9, 140])
        status = torch.zeros(1, dtype=torch.int32, device="cuda")

        def call(st):
            return torch.cat([t.long() for t in P.tree_accept(*args, status, stream=st)]) if st is None else \
                P.tree_accept(*args, status, stream=st)
        want = call(None)
        assert want.tolist() == kept + num + nxt
    side, held = torch.cuda.Stream(), torch.zeros_like(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = call(side)
        torch.cuda.current_stream().wait_stream(side)
        held.copy_(got if name == "tree" else torch.cat([t.long() for t in got]))
        del got
    for _ in range(3):
        held.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert status.item() == 0 and torch.equal(held, want)
