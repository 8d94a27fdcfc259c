"""Calls for trees of drafted tokens on a stream of their own, while work is queued on the
current one."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import libbuild  # noqa: E402
import paged_kv_cache_146_gb300 as P  # noqa: E402
from tree_reference import accept_path, random_parents  # noqa: E402

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
