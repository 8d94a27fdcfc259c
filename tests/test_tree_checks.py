"""Refusals of the calls for trees of drafted tokens: nothing of them reaches a GPU, so they run
on the CPU; and the plain 64-bit forms that the GPU tests compare with, against themselves."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

import libbuild  # noqa: E402
from paged_kv_cache_146_gb300 import (KVPool, PagedKVError, _native, cache_compact,  # noqa: E402
                                      paged_tree_attention, tree_accept, tree_mask,
                                      tree_workspace_bytes)
from tree_reference import (TreeCase, accept_path, compact, mask_words, path_masks,  # noqa: E402
                            random_parents)

lib = libbuild.ensure_built()
BF, I32 = torch.bfloat16, torch.int32
_kept = []


def zeros(*shape, dtype=I32):
    return torch.zeros(shape, dtype=dtype)


def pool16(dim=64, name="bf16"):
    p = KVPool(8, 2, dim, name)
    p.k_pool, p.v_pool = zeros(8, 2, 16, dim, dtype=BF), zeros(8, 2, 16, dim, dtype=BF)
    return p


def tree_args():
    return dict(q=zeros(5, 4, 64, dtype=BF), block_tables=zeros(2, 3), query_start=zeros(3),
                context_lens=zeros(2), tree_mask=zeros(5, 1), scale=0.1,
                workspace=zeros(1 << 20, dtype=torch.uint8), status=zeros(1))


@pytest.mark.parametrize("change,error,match", [
    (dict(q=zeros(5, 4, 32, dtype=BF)), ValueError, "q must be"),
    (dict(q=zeros(5, 256, dtype=BF)), ValueError, "q must be"),
    (dict(q=zeros(5, 3, 64, dtype=BF)), ValueError, "not a multiple"),
    (dict(q=zeros(5, 4, 64, dtype=torch.float16)), TypeError, "q must be bfloat16"),
    (dict(q=zeros(5, 8, 64, dtype=BF)[:, ::2]), ValueError, "q must be contiguous"),
    (dict(out=zeros(4, 4, 64, dtype=BF)), ValueError, "out must be"),
    (dict(block_tables=zeros(2)), ValueError, "block_tables"),
    (dict(block_tables=zeros(2, 3, dtype=torch.int64)), TypeError, "block_tables"),
    (dict(query_start=zeros(2)), ValueError, "query_start"),
    (dict(query_start=zeros(3, dtype=torch.int64)), TypeError, "query_start"),
    (dict(context_lens=zeros(3)), ValueError, "context_lens"),
    (dict(tree_mask=zeros(5)), ValueError, "tree_mask"),
    (dict(tree_mask=zeros(4, 1)), ValueError, "tree_mask"),
    (dict(tree_mask=zeros(5, 1, dtype=torch.int64)), TypeError, "tree_mask must be int32"),
    (dict(tree_mask=zeros(5, 2)[:, ::2]), ValueError, "tree_mask must be contiguous"),
    (dict(workspace=zeros(64)), TypeError, "workspace"),
    (dict(status=zeros(0)), TypeError, "status"),
    (dict(status=zeros(1, dtype=torch.int64)), TypeError, "status"),
    (dict(), ValueError, "CUDA tensors"),
])
def test_tree_attention_refusals(change, error, match):
    with pytest.raises(error, match=match):
        paged_tree_attention(pool16(), **{**tree_args(), **change})


def test_pools_refused():
    for name in ("q8_bf16", "b8_bf16"):
        pool = KVPool(8, 2, 128, name)
        with pytest.raises(ValueError, match="16-bit pool"):
            paged_tree_attention(pool, **tree_args())
        with pytest.raises(ValueError, match="16-bit pool"):
            cache_compact(pool, zeros(1, 1), zeros(1), zeros(2), zeros(1), zeros(1), zeros(1))
    pool = KVPool(8, 2, 64, "bf16")
    with pytest.raises(ValueError, match="no device memory"):
        paged_tree_attention(pool, **tree_args())
    with pytest.raises(ValueError, match="no device memory"):
        cache_compact(pool, zeros(1, 1), zeros(1), zeros(2), zeros(1), zeros(1), zeros(1))
    pool = pool16()
    with pytest.raises(ValueError, match="v_pool must be"):
        paged_tree_attention(pool, **tree_args(), v_pool=zeros(7, 2, 16, 64, dtype=BF))
    pool.close()
    with pytest.raises(ValueError):
        paged_tree_attention(pool, **tree_args())


def accept_args():
    return dict(tokens=zeros(5), parents=zeros(5), targets=zeros(5), query_start=zeros(3),
                first=zeros(2), status=zeros(1))


@pytest.mark.parametrize("change,error,match", [
    (dict(tokens=zeros(5, dtype=torch.int16)), TypeError, "int32 or int64"),
    (dict(tokens=zeros(5, 1)), ValueError, "tokens must be"),
    (dict(tokens=zeros(5, dtype=torch.int64)), TypeError, "targets must be int64"),
    (dict(parents=zeros(4)), ValueError, "parents must be"),
    (dict(parents=zeros(5, dtype=torch.int64)), TypeError, "parents must be int32"),
    (dict(query_start=zeros(2)), ValueError, "query_start"),
    (dict(first=zeros(3)), ValueError, "query_start"),
    (dict(kept=zeros(4)), ValueError, "kept must be"),
    (dict(num_kept=zeros(3)), ValueError, "num_kept must be"),
    (dict(next_tokens=zeros(2, dtype=torch.int64)), TypeError, "next_tokens must be int32"),
    (dict(), ValueError, "CUDA tensors"),
])
def test_accept_refusals(change, error, match):
    with pytest.raises(error, match=match):
        tree_accept(**{**accept_args(), **change})


@pytest.mark.parametrize("change,match", [
    (dict(block_tables=zeros(2)), "block_tables"), (dict(kept=zeros(3, 1)), "kept must be"),
    (dict(kept_start=zeros(2)), "kept_start must be"), (dict(num_kept=zeros(3)), "num_kept must be"),
    (dict(first=zeros(1)), "first must be"), (dict(k_pool=zeros(8, 2, 16, 32, dtype=BF)), "k_pool must be"),
    (dict(), "CUDA tensors")])
def test_compact_refusals(change, match):
    args = dict(block_tables=zeros(2, 3), kept=zeros(6), kept_start=zeros(3), num_kept=zeros(2),
                first=zeros(2), status=zeros(1))
    with pytest.raises(ValueError, match=match):
        cache_compact(pool16(), **{**args, **change})


def test_c_entries_refuse_before_any_launch():
    """Sizes, null pointers and alignment, by the C entries themselves; the addresses are never read."""
    bad, unsupported, ok = -1, -8, 0
    P = 1 << 20                                     # an aligned address that is not read

    def tree(dim=64, hq=4, words=1, S=1, T=1, maxb=1, scale=0.1, size=1 << 40, name="bf16", bs=16, **at):
        pool = KVPool(8, 2, dim, name, block_size=bs)
        _kept.append(pool)
        p = dict(out=P, q=P, k=P, v=P, tables=P, start=P, lens=P, mask=P, ws=P, status=P)
        p.update(at)
        return lib.paged_tree_attention(pool.handle, p["out"], p["q"], p["k"], p["v"], p["tables"], maxb,
                                        p["start"], p["lens"], p["mask"], words, S, T, hq, scale, p["ws"],
                                        size, p["status"], None)

    assert [tree(words=0), tree(words=33), tree(S=-1), tree(T=-1), tree(hq=0), tree(hq=3), tree(maxb=0)] == [bad] * 7
    assert [tree(scale=x) for x in (math.nan, math.inf, -math.inf)] == [bad] * 3
    assert [tree(dim=96), tree(hq=34), tree(bs=32)] == [unsupported] * 3
    assert tree(name="q8_bf16", dim=128) == bad and tree(name="b8_f16") == bad
    assert tree(S=0) == ok and tree(T=0) == ok
    for name in ("out", "q", "k", "v", "tables", "start", "lens", "mask", "ws", "status"):
        assert tree(**{name: None}) == bad and tree(**{name: P + 2}) == bad, name
    assert tree(ws=P + 128) == bad and tree(size=255) == bad
    need = tree_workspace_bytes(100, 4, 2, 64)
    assert need > 0 and tree(T=100, size=need - 1) == bad
    assert [tree_workspace_bytes(*a) for a in ((-1, 4, 2, 64), (1, 5, 2, 64), (1, 4, 2, 96), (1, 64, 2, 64))] == [0] * 4

    def accept(size=4, S=1, T=1, **at):
        p = dict(tokens=P, parents=P, targets=P, start=P, first=P, kept=P, num=P, nxt=P, status=P)
        p.update(at)
        return lib.kv_tree_accept(p["tokens"], p["parents"], p["targets"], size, p["start"], p["first"], S,
                                  T, p["kept"], p["num"], p["nxt"], p["status"], None)

    assert [accept(size=2), accept(S=-1), accept(T=-1)] == [bad] * 3 and accept(S=0) == ok
    for name in ("tokens", "parents", "targets", "start", "first", "kept", "num", "nxt", "status"):
        assert accept(**{name: None}) == bad and accept(**{name: P + 2}) == bad, name
    assert accept(size=8, tokens=P + 4) == bad

    def move(S=1, N=1, maxb=1, dim=64, name="bf16", **at):
        pool = KVPool(8, 2, dim, name)
        _kept.append(pool)
        p = dict(tables=P, kept=P, start=P, num=P, first=P, k=P, v=P, status=P)
        p.update(at)
        return lib.kv_cache_compact(pool.handle, p["tables"], maxb, p["kept"], p["start"], p["num"],
                                    p["first"], S, N, p["k"], p["v"], p["status"], None)

    assert [move(S=-1), move(N=-1), move(maxb=0), move(name="b8_bf16"), move(name="q8_f16", dim=128)] == [bad] * 5
    assert move(dim=12) == unsupported and move(S=0) == ok and move(N=0) == ok
    for name in ("tables", "kept", "start", "num", "first", "k", "v", "status"):
        assert move(**{name: None}) == bad and move(**{name: P + 2}) == bad, name


def test_error_names():
    with pytest.raises(PagedKVError, match="INVALID_ARG"):
        _native.check(lib.kv_tree_accept(None, None, None, 3, None, None, 1, 1, None, None, None, None, None))
    assert ctypes.sizeof(ctypes.c_void_p) == 8


def test_tree_mask():
    gen = torch.Generator().manual_seed(1)
    news = [0, 1, 5, 70, 33, 0, 128]
    parents = [random_parents(n, gen) for n in news]
    parents[3] = [i - 1 for i in range(70)]                 # one long chain
    parents[4][7] = -1                                      # a second root
    starts = torch.tensor([0] + news).cumsum(0).to(I32)
    flat = torch.tensor([x for p in parents for x in p] + [0, 1], dtype=I32)
    got = tree_mask(flat, starts)
    want = mask_words([m for p in parents for m in path_masks(p)] + [0, 0], 4)
    assert got.dtype == I32 and torch.equal(got, want)
    assert torch.equal(tree_mask(flat, starts, 4), want)
    assert torch.equal(tree_mask(flat[:0], torch.zeros(1, dtype=I32)), zeros(0, 1))
    for words in (0, 33):
        with pytest.raises(ValueError, match="words"):
            tree_mask(flat, starts, words)


def test_reference_forms():
    """The plain forms against simpler ones."""
    c = TreeCase([7, 0], [4, 3], 2, 1, 64, torch.float16, 2)
    for s in range(2):
        out, bound = c.expect(s, 0.125)
        k, v = c.kv(s, 0)
        for i in range(c.news[s]):
            seen, up = list(range(c.priors[s])), i
            while up >= 0:
                seen.append(c.priors[s] + up)
                up = c.parents[s][up]
            for h in range(2):
                x = (k[seen] @ c.q[c.starts[s] + i, h].double()) * 0.125
                assert torch.allclose(out[i, h], torch.softmax(x, 0) @ v[seen], rtol=1e-12, atol=1e-14)
        assert (bound < 0.01).all()
    assert accept_path([1, 2, 2, 3], [-1, 0, 0, 2], [2, 9, 3, 5]) == [0, 1]
    assert accept_path([1, 2, 4, 3], [-1, 0, 0, 2], [4, 9, 3, 5]) == [0, 2, 3] and accept_path([], [], []) == []
    pool = torch.arange(2 * 1 * 4 * 1).view(2, 1, 4, 1)
    compact(pool, [1, 0], [1, 2, 6], 0)
    assert pool.view(-1).tolist() == [0, 1, 2, 3, 5, 6, 2, 7]
