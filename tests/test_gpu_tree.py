"""Attention over trees of drafted tokens, the accepted path and moving kept tokens together,
against 64 bits; and the calls in the order that a server makes them."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import libbuild  # noqa: E402
from paged_kv_cache_146_gb300 import (DEV_BAD_BLOCK, DEV_BAD_LEN, DEV_BAD_TREE, KVPool,  # noqa: E402
                                      cache_compact, cache_write, cache_write_rope,
                                      decode_workspace_bytes, paged_decode_attention,
                                      paged_prefill_attention, paged_tree_attention,
                                      prefill_workspace_bytes, rope_table, status_check, tree_accept,
                                      tree_mask, tree_workspace_bytes)
from serving_reference import assert_within, attention, scale_of  # noqa: E402
from tree_reference import TreeCase, accept_path, compact, mask_words, path_masks, random_parents  # noqa: E402

libbuild.ensure_built()
pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def new_status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def pool_of(c, name):
    pool = KVPool(c.nb, c.hkv, c.dim, name, device="cuda")
    pool.k_pool.copy_(c.k)
    pool.v_pool.copy_(c.v)
    return pool


def workspace(c):
    size = tree_workspace_bytes(c.q.shape[0], c.hq, c.hkv, c.dim)
    return torch.randint(0, 256, (size,), dtype=torch.uint8, device="cuda")


def call(c, name, scale=None, words=None, out=None, pool=None, status=None, **kw):
    status = new_status() if status is None else status
    mask = torch.zeros((c.q.shape[0], words or c.words), dtype=torch.int32)
    mask[:c.rows] = mask_words(c.masks, words or c.words)
    got = paged_tree_attention(pool or pool_of(c, name), c.q.cuda(), c.tables.cuda(), ints(c.starts),
                               ints(c.lens), mask.cuda(), scale_of(c.dim) if scale is None else scale,
                               workspace(c), status, out=out, **kw)
    return got, status


def check(c, name, scale=None, words=None, seqs=None):
    got, status = call(c, name, scale, words)
    assert status_check(status) == (0, 0)
    for s in range(len(c.news)) if seqs is None else seqs:
        want, bound = c.expect(s, scale_of(c.dim) if scale is None else scale)
        assert_within(got[c.starts[s]:c.starts[s + 1]], want, bound, f"sequence {s}")
    return got


# ------------------------------------------------------------------------- attention
@pytest.mark.parametrize("hq,hkv", [(4, 4), (8, 2), (16, 1), (12, 1), (10, 2), (9, 3), (7, 1), (13, 1)])
@pytest.mark.parametrize("name,dim", [("bf16", 128), ("f16", 128), ("bf16", 64), ("f16", 64)])
def test_head_layouts(name, dim, hq, hkv):
    check(TreeCase([0, 1, 16, 100, 5, 300], [3, 0, 1, 17, 9, 33], hq, hkv, dim, DT[name], hq + dim), name)


@pytest.mark.parametrize("news", [[1] * 9, [2, 31, 32, 33], [64, 63, 65], [127, 128, 129, 1], [256, 200]])
@pytest.mark.parametrize("name,dim,hq,hkv", [("bf16", 128, 4, 1), ("f16", 64, 8, 4)])
def test_tree_sizes(name, dim, hq, hkv, news):
    priors = [0, 1, 15, 16, 47, 63, 64, 65, 129][:len(news)]
    check(TreeCase(priors, news, hq, hkv, dim, DT[name], len(news) + dim), name)


@pytest.mark.parametrize("prior", [0, 1, 14, 15, 16, 62, 63, 64, 65, 126, 127, 128, 129, 191, 1000])
def test_edges_of_key_tiles(prior):
    check(TreeCase([prior, prior], [2, 7], 8, 2, 128, torch.bfloat16, prior), "bf16")
    check(TreeCase([prior, prior], [1, 13], 3, 3, 64, torch.float16, prior), "f16")


def test_long_contexts_are_split():
    """Few long sequences: a sequence's keys go to many CTAs and their pieces are joined."""
    check(TreeCase([20011], [5], 4, 1, 128, torch.bfloat16, 1), "bf16")
    check(TreeCase([7003, 3, 9000], [40, 2, 33], 8, 2, 64, torch.float16, 2), "f16")
    check(TreeCase([4100], [70], 16, 2, 128, torch.bfloat16, 3), "bf16")


def test_many_ragged_sequences():
    gen = torch.Generator().manual_seed(4)
    priors = torch.randint(0, 700, (150,), generator=gen).tolist()
    news = torch.randint(0, 20, (150,), generator=gen).tolist()
    c = TreeCase(priors, news, 4, 2, 64, torch.bfloat16, 5)
    check(c, "bf16", seqs=range(0, 150, 7))


def test_more_sequences_than_threads():
    gen = torch.Generator().manual_seed(6)
    priors = torch.randint(0, 40, (1500,), generator=gen).tolist()
    news = torch.randint(0, 4, (1500,), generator=gen).tolist()
    c = TreeCase(priors, news, 2, 1, 64, torch.float16, 7)
    check(c, "f16", seqs=list(range(0, 1500, 97)) + [1499])


@pytest.mark.parametrize("name", ["bf16", "f16"])
def test_masks_that_are_no_trees(name):
    """Any bits: rows that see nothing (zero rows), not even themselves, later tokens, all."""
    gen = torch.Generator().manual_seed(8)
    news, priors = [40, 40, 3, 33], [0, 77, 0, 16]
    masks = []
    for n in news:
        for i in range(n):
            r = int(torch.randint(0, 4, (1,), generator=gen))
            bits = sum(int(b) << j for j, b in enumerate(torch.randint(0, 2, (n,), generator=gen)))
            masks.append([0, bits, (1 << n) - 1, 1 << int(torch.randint(0, n, (1,), generator=gen))][r])
    c = TreeCase(priors, news, 8, 2, 128, DT[name], 9, masks=masks)
    got = check(c, name)
    none = [r for r in range(c.rows) if masks[r] == 0 and (r < 40 or 80 <= r < 83)]
    assert none and not bool(got[none].any())


def test_bits_past_the_tree_count_for_nothing():
    c = TreeCase([50, 3, 0], [5, 31, 33], 4, 2, 64, torch.bfloat16, 10)
    got = check(c, "bf16", words=4)
    c.masks = [m | ~((1 << n) - 1) for m, n in zip(c.masks, [n for n in c.news for _ in range(n)])]
    again, status = call(c, "bf16", words=4)
    assert status_check(status) == (0, 0) and torch.equal(got, again)


@pytest.mark.parametrize("name,dim", [("bf16", 128), ("f16", 64)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_hidden_values_reach_nothing(name, dim, value):
    """A drafted token of odd values reaches the rows that see it and no other."""
    c = TreeCase([0, 30, 100], [9, 40, 20], 8, 2, dim, DT[name], 11)
    clean = check(c, name)
    for s, i in ((0, 4), (1, 17), (1, 33), (2, 0)):
        pos = c.priors[s] + i
        b, o = int(c.tables[s, pos // 16]), pos % 16
        c.v[b, :, o, 5] = value
        c.v[b, :, o, dim - 1] = -value
        if value != value:
            c.k[b, :, o] = value
    got, status = call(c, name)
    assert status_check(status) == (0, 0)
    for s, odd in ((0, [4]), (1, [17, 33]), (2, [0])):
        n = c.news[s]
        rows = torch.arange(c.starts[s], c.starts[s + 1])
        hit = torch.tensor([any(c.masks[r] >> i & 1 for i in odd) for r in rows.tolist()])
        assert hit.any() and (s == 2 or not hit.all())
        assert torch.equal(got[rows[~hit]], clean[rows[~hit]])
        hurt = got[rows[hit]].float().cpu()
        if value != value:
            assert hurt.isnan().all()
            continue
        both = torch.tensor([sum(c.masks[r] >> i & 1 for i in odd) for r in rows[hit].tolist()])
        assert (hurt[..., 5] == value).all() and (hurt[..., dim - 1] == -value).all() and n and both.all()
        rest = torch.ones(dim, dtype=torch.bool)
        rest[[5, dim - 1]] = False
        assert torch.equal(hurt[..., rest], clean[rows[hit]].float().cpu()[..., rest])


def test_infinite_keys():
    """A key of -inf products weighs nothing: the row is that of the other keys."""
    c = TreeCase([20], [3], 2, 1, 64, torch.float16, 12)
    c.q = torch.ones_like(c.q)
    c.k[c.tables[0, 0], 0, 0] = float("-inf")
    got, status = call(c, "f16", 0.125)
    assert status_check(status) == (0, 0)
    k, v = c.kv(0, 0)
    for i in range(3):
        seen = c.sees(0)[i].nonzero()[1:, 0]
        want, bound = attention(torch.ones(64, dtype=torch.float64), k[seen], v[seen], 0.125, torch.float16,
                                2.0 ** -22)
        assert_within(got[i], want.expand(2, -1), bound.expand(2, -1), f"row {i}")


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
@pytest.mark.parametrize("name", ["bf16", "f16"])
def test_scales(name, scale):
    check(TreeCase([0, 40, 200], [5, 40, 9], 4, 1, 128, DT[name], 13), name, scale=scale)


@pytest.mark.parametrize("name", ["bf16", "f16"])
def test_weights_far_below_a_dominant_key(name):
    """5,000 tokens of 2^-19 behind one dominant key of zero values: their part is the result."""
    c = TreeCase([5000, 70], [3, 3], 2, 1, 64, DT[name], 14)
    c.q = torch.zeros_like(c.q)
    c.q[..., 0] = 1.0
    for s in range(2):
        j = torch.arange(c.lens[s])
        blk = c.tables[s].long()[j // 16]
        c.k[blk, 0, j % 16] = 0.0
        at = int(c.tables[s, 1]), 4
        c.k[at[0], 0, at[1], 0] = 13.25
        c.v[at[0], 0, at[1]] = 0.0
        c.v[blk, 0, j % 16] = c.v[blk, 0, j % 16].abs()
    check(c, name, scale=1.0)


@pytest.mark.parametrize("size", [2.0 ** 10, 2.0 ** 14])
def test_huge_equal_scores(size):
    """Keys that agree weigh alike, whatever the scores' size."""
    c = TreeCase([700], [4], 2, 1, 64, torch.bfloat16, 15)
    j = torch.arange(704)
    blk = c.tables[0].long()[j // 16]
    c.k[blk, 0, j % 16] = size
    c.q = torch.full_like(c.q, size)
    for sign in (1.0, -1.0):
        got, status = call(c, "bf16", sign)
        assert status_check(status) == (0, 0)
        v = c.v[blk, 0, j % 16].double()
        want = (c.sees(0).double() @ v) / c.sees(0).double().sum(-1, keepdim=True)
        bound = 2.0 ** -8 * want.abs() + 2.0 ** -14 * v.abs().mean(0) + 1e-30
        assert_within(got, want[:, None].expand(-1, 2, -1), bound[:, None].expand(-1, 2, -1))


def test_a_chain_is_the_causal_call():
    """A tree without branches is a chunk of a prompt."""
    c = TreeCase([100, 0, 333], [17, 40, 5], 8, 2, 128, torch.bfloat16, 16,
                 masks=[m for n in (17, 40, 5) for m in path_masks([i - 1 for i in range(n)])])
    got = check(c, "bf16")
    pool, status = pool_of(c, "bf16"), new_status()
    pool.v_pool.nan_to_num_()
    ws = torch.empty(prefill_workspace_bytes(3, c.rows, 8, 2), dtype=torch.uint8, device="cuda")
    want = paged_prefill_attention(pool, c.q.cuda(), c.tables.cuda(), ints(c.starts), ints(c.lens),
                                   scale_of(128), ws, status)
    assert status_check(status) == (0, 0)
    # both within a half step and little more of the same value
    assert ((got.float() - want.float()).abs() <= 2.0 ** -7 * want.float().abs() + 2.0 ** -13).all()


def test_bad_sequences_get_zero_rows():
    c = TreeCase([40] * 6, [4] * 6, 8, 2, 128, torch.bfloat16, 17)
    good, _ = call(c, "bf16")
    lens = list(c.lens)
    c.lens = [44, 3, 10 ** 6, -5, 44, 44]
    c.tables[4, 2] = c.nb
    got, status = call(c, "bf16")
    assert status_check(status)[1] == DEV_BAD_LEN | DEV_BAD_BLOCK
    assert torch.equal(got[:4], good[:4]) and not bool(got[4:20].any()) and torch.equal(got[20:], good[20:])
    # one bad block among many: the whole sequence is zero, also where its keys were split
    c = TreeCase([9000, 9000], [4, 4], 8, 2, 128, torch.bfloat16, 18)
    good, _ = call(c, "bf16")
    c.tables[0, 300] = -1
    got, status = call(c, "bf16")
    assert status_check(status)[1] == DEV_BAD_BLOCK
    assert not bool(got[:4].any()) and torch.equal(got[4:], good[4:])
    # more drafted tokens than the mask has bits
    c = TreeCase([9, 9], [40, 4], 2, 2, 64, torch.float16, 19)
    c.lens, keep = list(c.lens), c.masks
    c.masks = [m & 0xffffffff for m in keep]
    got, status = call(c, "f16", words=1)
    assert status_check(status)[1] == DEV_BAD_LEN and not bool(got[:40].any()) and bool(got[40:].any())
    assert lens


def test_bad_row_ranges():
    c = TreeCase([40] * 4, [4] * 4, 2, 1, 64, torch.float16, 20)
    good, _ = call(c, "f16")
    c.starts = [0, 4, 2, 12, 99]
    out = torch.full_like(good, 7.0)
    got, status = call(c, "f16", out=out)
    assert status_check(status)[1] == DEV_BAD_LEN and torch.equal(got[:2], good[:2])
    assert (got[12:] == 7.0).all()


def test_rows_of_no_sequence_stay():
    c = TreeCase([33, 5], [6, 3], 4, 2, 64, torch.bfloat16, 21, spare=5)
    out = torch.full((14, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    got, status = call(c, "bf16", out=out)
    assert status_check(status) == (0, 0) and got is out and (out[9:] == 3.0).all()
    want, bound = c.expect(1, scale_of(64))
    assert_within(out[6:9], want, bound)


def test_empty_calls():
    c = TreeCase([5, 9], [0, 0], 4, 2, 64, torch.bfloat16, 22, spare=1)
    out = torch.full((1, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    got, status = call(c, "bf16", out=out)
    assert status_check(status) == (0, 0) and (got == 3.0).all()
    c.q = c.q[:0]
    got, status = call(c, "bf16")
    assert status_check(status) == (0, 0) and got.shape == (0, 4, 64)


def test_repeated_captured_and_concurrent():
    c = TreeCase([5000, 33, 2000, 7], [16, 1, 40, 3], 8, 2, 128, torch.bfloat16, 23)
    pool, status = pool_of(c, "bf16"), new_status()
    args = (pool, c.q.cuda(), c.tables.cuda(), ints(c.starts), ints(c.lens),
            mask_words(c.masks, c.words).cuda(), 0.1)
    first = paged_tree_attention(*args, workspace(c), status)
    held, spaces = torch.zeros_like(first), [workspace(c) for _ in range(3)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        paged_tree_attention(*args, spaces[0], status, out=held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        paged_tree_attention(*args, spaces[0], status, out=held)
    held.zero_()
    outs = [torch.empty_like(first) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, o, w in zip(streams, outs, spaces[1:]):
            paged_tree_attention(*args, w, status, out=o, stream=st)
        graph.replay()
    torch.cuda.synchronize()
    assert status_check(status) == (0, 0)
    for o in (held, *outs):
        assert torch.equal(o, first)


def test_two_graphs_share_a_workspace():
    """Graphs that run one after the other may share it."""
    c = [TreeCase([3000 + 50 * i, 9], [8, 5], 8, 2, 128, torch.bfloat16, 24 + i) for i in range(2)]
    ws, status, graphs, outs, want = workspace(c[0]), new_status(), [], [], []
    for x in c:
        args = (pool_of(x, "bf16"), x.q.cuda(), x.tables.cuda(), ints(x.starts), ints(x.lens),
                mask_words(x.masks, x.words).cuda(), 0.1, ws, status)
        want.append(paged_tree_attention(*args))
        outs.append(torch.zeros_like(want[-1]))
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            paged_tree_attention(*args, out=outs[-1])
        graphs[-1].args = args
    for _ in range(3):
        for g in graphs:
            g.replay()
    assert status_check(status) == (0, 0)
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_pool_beyond_32_bits():
    """Blocks past 2^31 elements of the pool."""
    c = TreeCase([200], [9], 16, 8, 128, torch.bfloat16, 26)
    nb = 2 ** 31 // (8 * 16 * 128) + 64
    pool = KVPool(nb, 8, 128, "bf16", device="cuda")
    shift = nb - c.nb
    pool.k_pool[shift:] = c.k.cuda()
    pool.v_pool[shift:] = c.v.cuda()
    c.tables = torch.where(c.tables >= 0, c.tables + shift, c.tables)
    got, status = call(c, "bf16", pool=pool)
    assert status_check(status) == (0, 0)
    c.tables -= shift
    want, bound = c.expect(0, scale_of(128))
    assert_within(got, want, bound)
    c.tables += shift
    kept = [200, 203, 207]
    cache_compact(pool, c.tables.cuda(), ints(kept), ints([0, 3]), ints([3]), ints([200]), status)
    assert status_check(status) == (0, 0)
    for mine, ref in ((pool.k_pool, c.k), (pool.v_pool, c.v)):
        compact(ref, (c.tables[0] - shift).tolist(), kept, 200)
        assert torch.equal(mine[shift:].cpu().view(torch.int16), ref.view(torch.int16))


# ---------------------------------------------------------------------- accepted path
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("news", [[1], [7], [0, 3, 1, 0], [64, 33, 32, 31, 5], [400, 2, 129] * 30])
def test_accept(dtype, news):
    gen = torch.Generator().manual_seed(len(news))
    parents = [random_parents(n, gen) for n in news]
    total = sum(news)
    tokens = torch.randint(0, 3, (total,), generator=gen)      # few values: long paths and ties
    targets = torch.randint(0, 3, (total,), generator=gen)
    big = 2 ** 33 if dtype == torch.int64 else 2 ** 30
    tokens, targets = tokens + big, targets + big
    first = torch.randint(0, 5000, (len(news),), generator=gen).tolist()
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    status = new_status()
    kept = torch.full((total + 2,), 9, dtype=torch.int32, device="cuda")
    pad = torch.zeros(2, dtype=torch.int64)
    flat = [x for p in parents for x in p] + [0, 0]
    got = tree_accept(torch.cat([tokens, pad]).to("cuda", dtype), ints(flat),
                      torch.cat([targets, pad]).to("cuda", dtype), ints(starts), ints(first), status,
                      kept=kept)
    assert status_check(status) == (0, 0) and got[0] is kept and got[2].dtype == dtype
    assert kept[total:].tolist() == [9, 9]
    for s, n in enumerate(news):
        a, b = starts[s], starts[s + 1]
        path = accept_path(tokens[a:b].tolist(), parents[s], targets[a:b].tolist())
        assert kept[a:b].tolist() == [first[s] + i for i in path] + [-1] * (n - len(path))
        assert got[1][s].item() == len(path)
        assert got[2][s].item() == (targets[a + path[-1]].item() if path else -1)


def test_accept_bad_trees():
    """Wrong parents, positions and ranges: such a sequence keeps nothing, its neighbours theirs."""
    parents = [-1, 0, 1] + [-1, 1, 0] + [0, 0, 1] + [-1, -2, 0] + [-1, 0, 3] + [-1, -1, 0] + [-1, 0, 1]
    ones = torch.ones(21, dtype=torch.int32, device="cuda")
    first = [5, 5, 5, 5, 5, 5, 2 ** 31 - 3]
    status = new_status()
    kept, num, nxt = tree_accept(ones, ints(parents), ones, ints(list(range(0, 22, 3))), ints(first), status)
    assert status_check(status)[1] == DEV_BAD_TREE | DEV_BAD_LEN
    assert num.tolist() == [3, 0, 0, 0, 0, 2, 0] and nxt.tolist() == [1, -1, -1, -1, -1, 1, -1]
    assert kept.tolist() == [5, 6, 7] + [-1] * 12 + [5, 7, -1] + [-1] * 3
    kept, num, nxt = tree_accept(ones, ints(parents), ones, ints([0, 3, 2, 40]), ints([0, 0, -1]), status)
    assert status_check(status)[1] & DEV_BAD_LEN and num.tolist() == [3, 0, 0]
    kept, num, nxt = tree_accept(ones[:0], ints([]), ones[:0], ints([0, 0, 0]), ints([4, 4]), status)
    assert status_check(status) == (0, 0) and num.tolist() == [0, 0] and nxt.tolist() == [-1, -1]


# ------------------------------------------------------------------------ moving tokens
def compact_case(lens, hkv, dim, dtype, seed, bs=16):
    gen = torch.Generator().manual_seed(seed)
    nbs = [-(-n // bs) for n in lens]
    nb, maxb = sum(nbs) + 2, max(nbs) + 1
    perm = torch.randperm(nb, generator=gen).tolist()
    tables = torch.full((len(lens), maxb), -1, dtype=torch.int32)
    for s, n in enumerate(nbs):
        for b in range(n):
            tables[s, b] = perm.pop()
    k, v = (torch.randint(-2 ** 15, 2 ** 15, (nb, hkv, bs, dim), generator=gen).to(torch.int16)
            for _ in range(2))
    return gen, nb, tables, k, v


def run_compact(tables, k, v, kept, first, name, starts=None, num=None, bs=16):
    """kept: a list per sequence.  The pools after the call and the status word."""
    nb, hkv, _, dim = k.shape
    pool = KVPool(nb, hkv, dim, name, block_size=bs, device="cuda")
    pool.k_pool.view(torch.int16).copy_(k)
    pool.v_pool.view(torch.int16).copy_(v)
    if starts is None:
        starts = [0]
        for x in kept:
            starts.append(starts[-1] + len(x))
    status = new_status()
    cache_compact(pool, tables.cuda(), ints([p for x in kept for p in x]), ints(starts),
                  ints([len(x) for x in kept] if num is None else num), ints(first), status)
    word = status_check(status)[1]
    return pool.k_pool.view(torch.int16).cpu(), pool.v_pool.view(torch.int16).cpu(), word


@pytest.mark.parametrize("name,hkv,dim,bs", [("bf16", 8, 128, 16), ("f16", 1, 64, 16), ("bf16", 3, 96, 16),
                                             ("f16", 2, 256, 16), ("bf16", 2, 8, 16), ("f16", 2, 64, 5),
                                             ("bf16", 1, 128, 32), ("bf16", 1, 400, 16)])
def test_compact(name, hkv, dim, bs):
    lens = [1, 40, 700, 3000, 16, 333]
    gen, nb, tables, k, v = compact_case(lens, hkv, dim, name, dim + bs, bs)
    kept, first = [], []
    for s, n in enumerate(lens):
        some = torch.randperm(n, generator=gen)[:max(1, n // (1 + s % 3))].sort().values.tolist()
        kept.append(some)
        first.append(int(torch.randint(0, some[0] + 1, (1,), generator=gen)))
    kept[4] = []
    got_k, got_v, word = run_compact(tables, k, v, kept, first, name, bs=bs)
    assert word == 0
    for got, ref in ((got_k, k), (got_v, v)):
        for s in range(len(lens)):
            compact(ref, tables[s].tolist(), kept[s], first[s])
        assert torch.equal(got, ref)


@pytest.mark.parametrize("drop", [[0], [1], [15, 16, 17], list(range(0, 900, 2)), list(range(1, 899))])
def test_compact_shifts(drop):
    """Short and long shifts: a destination is a source of earlier tokens."""
    gen, nb, tables, k, v = compact_case([900], 2, 64, "bf16", len(drop))
    gone = set(drop)
    kept = [[p for p in range(900) if p not in gone]]
    got_k, got_v, word = run_compact(tables, k, v, kept, [0], "bf16")
    assert word == 0
    for got, ref in ((got_k, k), (got_v, v)):
        compact(ref, tables[0].tolist(), kept[0], 0)
        assert torch.equal(got, ref)


def test_compact_bad_lists():
    lens = [100] * 9
    gen, nb, tables, k, v = compact_case(lens, 2, 64, "bf16", 3)
    kept = [[3, 5, 9]] * 9
    kept[1] = [3, 9, 9, 20]            # does not rise: the first two move
    kept[2] = [3, 2, 9]                # the first moves
    kept[3] = [1, 5, 9]                # below its destination: nothing moves
    kept[4] = [3, 5, 16 * tables.shape[1]]     # outside the row
    kept[7] = [-4, 5, 9]
    first = [2, 2, 2, 2, 2, -1, 2, 2, 2]
    num = [len(x) for x in kept]
    num[6] = 4                         # more than its entries
    tables[8, 0] = nb + 5
    got_k, got_v, word = run_compact(tables, k, v, kept, first, "bf16", num=num)
    assert word == DEV_BAD_LEN | DEV_BAD_TREE | DEV_BAD_BLOCK
    moved = {0: [3, 5, 9], 1: [3, 9], 2: [3], 4: [3, 5]}
    for got, ref in ((got_k, k), (got_v, v)):
        for s, x in moved.items():
            compact(ref, tables[s].tolist(), x, 2)
        assert torch.equal(got, ref)
    # row ranges that do not fit
    for starts in ([0, 5, 2], [0, 2, 7], [-1, 3, 6]):
        gen, nb, tables, k, v = compact_case([50, 50], 1, 64, "f16", 4)
        got_k, got_v, word = run_compact(tables, k, v, [[3, 4, 5], [6, 7, 8]], [0, 0], "f16",
                                         starts=starts, num=[9, 9])
        assert word == DEV_BAD_LEN and torch.equal(got_k, k) and torch.equal(got_v, v)


def test_compact_long_list_with_a_bad_end():
    """What stands before the first bad position has moved, nothing behind it."""
    gen, nb, tables, k, v = compact_case([9000], 1, 128, "bf16", 5)
    kept = list(range(1, 9000, 2))
    broken = kept[:4000] + [kept[4000] - 2] + kept[4001:]
    got_k, got_v, word = run_compact(tables, k, v, [broken], [0], "bf16")
    assert word == DEV_BAD_TREE
    for got, ref in ((got_k, k), (got_v, v)):
        compact(ref, tables[0].tolist(), kept[:4000], 0)
        assert torch.equal(got, ref)


# ------------------------------------------------------------------- a run of them together
@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("name,hq,hkv,dim", [("bf16", 8, 2, 128), ("f16", 4, 4, 64)])
def test_steps_of_a_server(name, hq, hkv, dim, graph):
    """Append the drafted tokens rotated by their depth, attend, take the path, move it
    together: after several steps the cache holds what appending the path's tokens one by one
    leaves, bit for bit, and decode attention over it gives the same."""
    S, steps, width = 3, 4, 11
    gen = torch.Generator().manual_seed(dim)
    pool, plain = (KVPool(64, hkv, dim, name, device="cuda") for _ in range(2))
    status, table = new_status(), rope_table(400, dim, device="cuda")
    maxb = 8
    tables, own = (torch.full((S, maxb), -1, dtype=torch.int32).numpy() for _ in range(2))
    lens = [5, 33, 0]

    def rows(n, h):
        return torch.randn((n, h, dim), generator=gen).to(DT[name]).cuda()

    for s, n in enumerate(lens):
        if n:
            k, v = rows(n, hkv), rows(n, hkv)
            for p, t in ((pool, tables), (plain, own)):
                slots = p.append_slots([0], [n], t[s:s + 1])
                cache_write_rope(p, k, v, ints(list(range(n))), table, torch.from_numpy(slots).cuda(), status)
    for step in range(steps):
        news = [width, 1, 7]
        parents = [random_parents(n, gen) for n in news]
        depth = []
        for p in parents:
            d = []
            for up in p:
                d.append(d[up] + 1 if up >= 0 else 0)
            depth += d
        total = sum(news)
        starts = ints([0, news[0], news[0] + news[1], total])
        first, after = ints(lens), [a + b for a, b in zip(lens, news)]
        slots = torch.from_numpy(pool.append_slots(lens, news, tables)).cuda()
        q, k, v = rows(total, hq), rows(total, hkv), rows(total, hkv)
        base = [lens[s] for s in range(S) for _ in range(news[s])]
        pos = ints([b + d for b, d in zip(base, depth)])
        flat = ints([x for p in parents for x in p])
        tokens = torch.randint(0, 2, (total,), generator=gen).cuda()
        targets = torch.randint(0, 2, (total,), generator=gen).cuda()
        d_tables, d_lens = torch.from_numpy(tables).cuda(), ints(after)
        mask = tree_mask(flat, starts, 1)
        ws = torch.empty(tree_workspace_bytes(total, hq, hkv, dim), dtype=torch.uint8, device="cuda")
        out = torch.empty_like(q)
        kept = torch.empty(total, dtype=torch.int32, device="cuda")
        num, nxt = torch.empty(S, dtype=torch.int32, device="cuda"), torch.empty_like(tokens[:S])
        q_rot = torch.empty_like(q)

        def chain():
            cache_write_rope(pool, k, v, pos, table, slots, status, q=q, q_out=q_rot)
            paged_tree_attention(pool, q_rot, d_tables, starts, d_lens, mask, scale_of(dim), ws, status,
                                 out=out)
            tree_accept(tokens, flat, targets, starts, first, status, kept=kept, num_kept=num,
                        next_tokens=nxt)
            cache_compact(pool, d_tables, kept, starts, num, first, status)

        if graph:
            # (the first run sets kernels up; the replay below starts from the same cache)
            k0, v0 = pool.k_pool.clone(), pool.v_pool.clone()
            chain()
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                chain()
            pool.k_pool.copy_(k0)
            pool.v_pool.copy_(v0)
            g.replay()
        else:
            chain()
        assert status_check(status) == (0, 0)
        # one token after the other, each attending to its path: the plain way
        at = 0
        for s, n in enumerate(news):
            path = accept_path(tokens[at:at + n].tolist(), parents[s], targets[at:at + n].tolist())
            assert kept[at:at + len(path)].tolist() == [lens[s] + i for i in path] and num[s] == len(path)
            for i in path:
                slot = plain.append_slots([lens[s]], [1], own[s:s + 1])
                r = at + i
                qr = cache_write_rope(plain, k[r:r + 1], v[r:r + 1], ints([lens[s]]), table,
                                      torch.from_numpy(slot).cuda(), status, q=q[r:r + 1])
                lens[s] += 1
                dws = torch.empty(decode_workspace_bytes(1, hq, hkv, dim, maxb), dtype=torch.uint8,
                                  device="cuda")
                one = paged_decode_attention(plain, qr, torch.from_numpy(own[s:s + 1]).cuda(),
                                             ints([lens[s]]), scale_of(dim), dws, status)
                assert torch.allclose(out[r].float(), one[0].float(), rtol=2.0 ** -6, atol=2.0 ** -9)
            at += n
            # the ledger takes back the blocks behind the path
            nb, old = -(-lens[s] // 16), -(-after[s] // 16)
            if old > nb:
                pool.free(tables[s, nb:old])
                tables[s, nb:old] = -1
        assert status_check(status) == (0, 0)
        for s in range(S):
            j = torch.arange(lens[s])
            a, b = (torch.from_numpy(t[s]).long()[j // 16] for t in (tables, own))
            for x, y in ((pool.k_pool, plain.k_pool), (pool.v_pool, plain.v_pool)):
                assert torch.equal(x[a, :, j % 16], y[b, :, j % 16])
        assert pool.num_free() == plain.num_free()


def test_other_device_stream_and_strided_masks():
    """Tensors on the current device, the call on another stream than the current one."""
    c = TreeCase([64], [8], 4, 1, 64, torch.bfloat16, 27)
    st = torch.cuda.Stream()
    pool, status = pool_of(c, "bf16"), new_status()
    torch.cuda.synchronize()
    got, _ = call(c, "bf16", pool=pool, status=status)
    torch.cuda.synchronize()
    out = torch.empty_like(got)
    args = (pool, c.q.cuda(), c.tables.cuda(), ints(c.starts), ints(c.lens),
            mask_words(c.masks, 1).cuda(), scale_of(64), workspace(c), status)
    torch.cuda.synchronize()
    paged_tree_attention(*args, out=out, stream=st)
    st.synchronize()
    assert torch.equal(out, got)


def test_cache_write_then_attend():
    """The plain append beside the rotated one."""
    c = TreeCase([0], [20], 4, 2, 64, torch.float16, 28)
    pool, status = KVPool(c.nb, 2, 64, "f16", device="cuda"), new_status()
    j = torch.arange(20)
    slots = c.tables[0].long()[j // 16] * 16 + j % 16
    blk = c.tables[0].long()[j // 16]
    cache_write(pool, c.k[blk, :, j % 16].cuda(), c.v[blk, :, j % 16].cuda(), slots.cuda(), status)
    got, _ = call(c, "f16", pool=pool, status=status)
    assert status_check(status) == (0, 0)
    want, bound = c.expect(0, scale_of(64))
    assert_within(got, want, bound)
