"""The windowed engine and blocks that no token sees any more: given back by the engine or by
its user, they change no result, and finished sequences release the rest."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_cache_146_gb300 import KVPool, PagedKVError, rope_table  # noqa: E402
from paged_kv_cache_146_gb300.engine import DecodeEngine  # noqa: E402

pytestmark = pytest.mark.gpu
S, HQ, HKV, D, MAXB = 4, 8, 2, 128, 40
PROMPTS = [300, 1, 16, 77]


def engine(kind, window, sinks, nb):
    gen = torch.Generator().manual_seed(2)
    dt = torch.bfloat16 if kind.endswith("bf16") else torch.float16
    pool = KVPool(nb, HKV, D, kind, device="cuda")
    eng = DecodeEngine(pool, S, HQ, MAXB, D ** -0.5, "cuda", rope=rope_table(700, 64).cuda(), window=window,
                       sinks=sinks)
    k, v = (torch.randn((sum(PROMPTS), HKV, D), generator=gen).to(dt).cuda() for _ in "kv")
    eng.prefill(k, v, PROMPTS)
    return eng, gen, dt


def visible_blocks(eng):
    n = 0
    for L in eng.lens.tolist():
        n += len({j // 16 for j in range(L) if j >= L - eng.window or j < eng.sinks})
    return n


@pytest.mark.parametrize("kind,window,sinks", [("bf16", 60, 4), ("f16", 17, 0), ("b8_bf16", 1, 33), ("b8_f16", 64, 16),
                                               ("bf16", 10 ** 6, 0)])
def test_blocks_behind_the_window_are_given_back(kind, window, sinks):
    keeps, gen, dt = engine(kind, window, sinks, 120)
    gives, _, _ = engine(kind, window, sinks, 120)
    given = 0
    for step in range(100):
        q, k, v = (torch.randn((S, h, D), generator=gen).to(dt).cuda() for h in (HQ, HKV, HKV))
        a = keeps.decode_step(q.clone(), k, v).clone()
        if step % 3:
            b = gives.decode_step(q.clone(), k, v).clone()
        else:                                # also between the ledger's step and the kernels
            gives.host_step()
            given += gives.release_hidden()
            b = gives.device_step(q.clone(), k, v).clone()
        assert torch.equal(a, b), step
        if step % 7 == 0:
            given += gives.release_hidden()
            assert 120 - gives.pool.num_free() == visible_blocks(gives)
    assert keeps.check() == (0, 0) and gives.check() == (0, 0)
    assert given == 0 if window > 500 else given >= 20
    assert 120 - keeps.pool.num_free() == sum(-(-n // 16) for n in keeps.lens.tolist())
    for e in (keeps, gives):
        e.release([1, 3])
        e.release([0, 2])
        assert e.pool.num_free() == 120 and not e.lens.any() and (e.tables == -1).all()


def test_a_users_own_holes():
    """A program frees the blocks itself, as the calls' documentation allows."""
    eng, _, _ = engine("bf16", 40, 2, 60)
    hole = eng.tables[0, 1:9].copy()
    torch.cuda.synchronize()
    eng.pool.free(hole)
    eng.tables[0, 1:9] = -1
    free = eng.pool.num_free()
    with pytest.raises(PagedKVError):        # the ledger itself takes no hole
        eng.pool.free(eng.tables[0, :19])
    assert eng.pool.num_free() == free
    eng.release(range(S))
    assert eng.pool.num_free() == 60


def test_without_a_window_nothing_is_hidden():
    eng, _, _ = engine("bf16", None, 0, 60)
    with pytest.raises(ValueError, match="stays visible"):
        eng.release_hidden()
    eng.tables[0, 1] = -1                    # a broken table is still refused
    with pytest.raises(PagedKVError):
        eng.release([0])
