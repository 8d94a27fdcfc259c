"""Trees of drafted tokens at the ends of their ranges: the largest trees, odd values where keys
are split, scales out of the ordinary, lists of every size; and the compiled argument checks of
these calls against the binding's own."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import libbuild  # noqa: E402

libbuild.ensure_built()
import paged_kv_cache_146_gb300 as P  # noqa: E402
from paged_kv_cache_146_gb300 import status_check  # noqa: E402
from serving_reference import assert_within, scale_of  # noqa: E402
from test_gpu_tree import (DT, call, check, compact_case, ints, new_status, pool_of, run_compact,  # noqa: E402
                           workspace)
from tree_reference import TreeCase, compact, mask_words, random_parents  # noqa: E402

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32


# ------------------------------------------------------------------------- attention
@pytest.mark.parametrize("name,dim,hq,hkv", [("bf16", 64, 2, 1), ("f16", 128, 3, 3)])
def test_the_largest_trees(name, dim, hq, hkv):
    """1,024 drafted tokens, masks of 32 words over 17 key tiles."""
    check(TreeCase([40, 0, 700], [1024, 700, 993], hq, hkv, dim, DT[name], dim), name, seqs=[0, 2])


@pytest.mark.parametrize("spread", [1, 33, 40])
def test_many_query_tiles_of_many_sequences(spread):
    """Query tiles of 8 tokens, up to 5 of them, in more sequences than a warp has lanes."""
    gen = torch.Generator().manual_seed(spread)
    news = [int(x) for x in torch.randint(1, spread + 1, (70,), generator=gen)]
    priors = [int(x) for x in torch.randint(0, 200, (70,), generator=gen)]
    news[3] = news[69] = spread
    c = TreeCase(priors, news, 16, 1, 64, BF, spread)
    check(c, "bf16", seqs=[0, 3, 20, 31, 32, 33, 63, 64, 69])


@pytest.mark.parametrize("tokens", [1, 2, 3, 5, 9, 40])
def test_calls_of_less_work_than_ctas(tokens):
    """Ranges of one key tile, and fewer of them than the GPU could take."""
    check(TreeCase([64 * tokens], [tokens], 4, 2, 128, BF, tokens), "bf16")
    check(TreeCase([5] * tokens, [1] * tokens, 4, 1, 64, torch.float16, tokens), "f16")


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_odd_values_in_split_keys(value):
    """Drafted tokens over several key tiles and pieces; K and V behind the end are NaN anyway."""
    c = TreeCase([3000, 1, 9001], [130, 200, 7], 8, 2, 128, BF, 31)
    clean = check(c, "bf16", seqs=[0, 2])
    odd = {0: [5, 60, 100, 129], 1: [3, 64, 150], 2: [6]}
    for s, nodes in odd.items():
        for i in nodes:
            pos = c.priors[s] + i
            c.v[int(c.tables[s, pos // 16]), :, pos % 16, 77] = value
    got, status = call(c, "bf16")
    assert status_check(status) == (0, 0)
    for s, nodes in odd.items():
        for r in range(c.starts[s], c.starts[s + 1]):
            hit = any(c.masks[r] >> i & 1 for i in nodes)
            want = clean[r].float()
            if hit:
                want[:, 77] = value
            assert torch.equal(torch.nan_to_num(got[r].float(), 1e30, 2e30, -2e30),
                               torch.nan_to_num(want, 1e30, 2e30, -2e30)), (s, r)


@pytest.mark.parametrize("name", ["bf16", "f16"])
@pytest.mark.parametrize("scale", [-0.2, 1e-40, -1e-40])
def test_scales_of_split_keys(name, scale):
    """A negative scale, and ones below the normal numbers: all weigh alike."""
    check(TreeCase([6000, 3], [20, 40], 8, 2, 64, DT[name], 32), name, scale=scale)


@pytest.mark.parametrize("scale", [3e38, -3e38])
def test_the_largest_scale_picks_a_key(scale):
    """Products of small whole numbers are exact; the one extreme key takes all the weight."""
    c = TreeCase([500, 0], [6, 3], 4, 2, 128, BF, 33)
    c.q = torch.zeros_like(c.q)
    c.q[..., 0] = 1.0
    c.k.nan_to_num_().clamp_(-2, 2).round_()
    for s, L in enumerate(c.lens):
        at = c.priors[s]                                   # the root: all nodes see it
        c.k[int(c.tables[s, at // 16]), :, at % 16, 0] = 5.0 if scale > 0 else -5.0
    got, status = call(c, "bf16", scale=scale)
    assert status_check(status) == (0, 0)
    for s in range(2):
        at = c.priors[s]
        v = c.v[int(c.tables[s, at // 16]), :, at % 16].repeat_interleave(2, 0)
        assert torch.equal(got[c.starts[s]:c.starts[s + 1]].cpu(), v.expand(c.news[s], -1, -1))


def test_the_output_may_be_the_queries():
    c = TreeCase([900, 3, 40], [30, 5, 64], 8, 2, 128, BF, 34)
    want, _ = call(c, "bf16")
    q, status = c.q.cuda(), new_status()
    P.paged_tree_attention(pool_of(c, "bf16"), q, c.tables.cuda(), ints(c.starts), ints(c.lens),
                           mask_words(c.masks, c.words).cuda(), scale_of(128), workspace(c), status, out=q)
    assert status_check(status) == (0, 0) and torch.equal(q, want)


def test_a_sequence_twice():
    """Two rows of the table with the same blocks: the same results."""
    c = TreeCase([700, 700], [9, 9], 8, 2, 64, torch.float16, 35)
    c.tables[1] = c.tables[0]
    c.q[9:] = c.q[:9]
    c.masks[9:] = c.masks[:9]
    got, status = call(c, "f16")
    assert status_check(status) == (0, 0)
    for s in range(2):
        want, bound = c.expect(s, scale_of(64))
        assert_within(got[9 * s:9 * s + 9], want, bound)


# ------------------------------------------------------------------------ moving tokens
@pytest.mark.parametrize("seqs,hkv,dim,lo,hi", [
    (64, 8, 64, 1, 100),           # short lists
    (100, 4, 128, 200, 700),       # long lists, a CTA to a row
    (20, 4, 128, 900, 2500),       # rows shared among CTAs
    (2, 1, 64, 4000, 5000),        # few sequences
    (1, 8, 128, 961, 961), (1, 1, 256, 3900, 3900), (3, 40, 64, 130, 2000), (1, 2, 8, 9000, 9000),
    (7, 1, 4096, 3, 60), (2, 1, 16384, 40, 70)])       # rows of more chunks than a CTA has threads
def test_lists_of_every_size(seqs, hkv, dim, lo, hi):
    gen = torch.Generator().manual_seed(seqs + dim)
    lens = [int(x) for x in torch.randint(lo, hi + 1, (seqs,), generator=gen)]
    gen, nb, tables, k, v = compact_case(lens, hkv, dim, "bf16", seqs)
    kept, first = [], []
    for s, n in enumerate(lens):
        part = (0.1, 0.5, 0.9, 1.0)[s % 4] if seqs > 1 else 0.98
        some = torch.randperm(n, generator=gen)[:max(1, int(n * part))].sort().values.tolist()
        kept.append(some)
        first.append(min(some[0], s % 3))
    got_k, got_v, word = run_compact(tables, k, v, kept, first, "bf16")
    assert word == 0
    for got, ref in ((got_k, k), (got_v, v)):
        for s in range(seqs):
            compact(ref, tables[s].tolist(), kept[s], first[s])
        assert torch.equal(got, ref)


@pytest.mark.parametrize("hkv,dim", [(8, 128), (6, 96), (8, 64), (5, 256), (6, 136)])
def test_long_lists_of_uneven_lengths(hkv, dim):
    """Rows shared by length: an empty list, one that does not fit, one with a bad position."""
    gen, nb, tables, k, v = compact_case([40, 6000, 900, 2500, 900, 30, 4100, 1000, 1200], hkv, dim, "f16", dim)
    kept, first = [], [0, 3, 0, 7, 2, 0, 0, 1, 5]
    for n, part, lo in zip((40, 6000, 900, 2500, 900, 30, 4100, 1000, 1200),
                           (1.0, 0.98, 0.5, 0.4, 0.0, 0.5, 0.97, 0.3, 0.5), first):
        some = torch.randperm(n - lo, generator=gen)[:int((n - lo) * part)] + lo
        kept.append(some.sort().values.tolist())
    num = [len(x) for x in kept]
    num[5] = -1                                            # does not fit
    kept[6][3000] = kept[6][2999]                          # does not rise
    got_k, got_v, word = run_compact(tables, k, v, kept, first, "f16", num=num)
    assert word == P.DEV_BAD_LEN | P.DEV_BAD_TREE
    moved = [x if s not in (5, 6) else x[:3000] if s == 6 else [] for s, x in enumerate(kept)]
    for got, ref in ((got_k, k), (got_v, v)):
        for s, x in enumerate(moved):
            compact(ref, tables[s].tolist(), x, first[s])
        assert torch.equal(got, ref)


def test_tokens_that_stay_and_tokens_of_no_one():
    """Nothing moves where positions equal their destinations; entries behind num_kept are not read."""
    gen, nb, tables, k, v = compact_case([300, 300], 2, 128, "bf16", 41)
    kept = [list(range(40)) + [-7] * 8, [5, 6] + [99999999] * 46]
    got_k, got_v, word = run_compact(tables, k, v, kept, [0, 5], "bf16", num=[40, 2])
    assert word == 0 and torch.equal(got_k, k) and torch.equal(got_v, v)


# --------------------------------------------------------- compiled checks of the arguments
def tree_data():
    gen = torch.Generator().manual_seed(51)
    c = TreeCase([70, 5, 0], [9, 20, 3], 8, 2, 64, BF, 51)
    parents = [x for p in c.parents for x in p]
    tokens, targets = (torch.randint(0, 2, (c.rows,), generator=gen) for _ in range(2))
    # K and V of a row that a table does not name are NaN: plain numbers, so that pools compare
    c.k.nan_to_num_()
    c.v.nan_to_num_()
    return dict(c=c, q=c.q.cuda(), tables=c.tables.cuda(), starts=ints(c.starts), lens=ints(c.lens),
                mask=mask_words(c.masks, c.words).cuda(), ws=workspace(c), parents=ints(parents),
                tokens=tokens.cuda(), targets=targets.cuda(), first=ints(c.priors),
                kept=ints([70, 73] + [-1] * 7 + [5, 9, 11] + [-1] * 17 + [1, 2, -1]),
                num=ints([2, 3, 2]))


def one_call(name, d, stream=None):
    """One call on a fresh pool; everything that it wrote."""
    pool, status = pool_of(d["c"], "bf16"), new_status()
    torch.cuda.synchronize()
    if name == "tree":
        res = [P.paged_tree_attention(pool, d["q"], d["tables"], d["starts"], d["lens"], d["mask"], 0.125,
                                      d["ws"], status, stream=stream)]
    elif name == "accept":
        res = list(P.tree_accept(d["tokens"], d["parents"], d["targets"], d["starts"], d["first"], status,
                                 stream=stream))
    else:
        P.cache_compact(pool, d["tables"], d["kept"], d["starts"], d["num"], d["first"], status, stream=stream)
        res = [pool.k_pool, pool.v_pool]
    torch.cuda.synchronize()
    return [*res, status]


class Noted:
    """The module of compiled checks with the answers of its calls noted."""

    def __init__(self, fast):
        self._fast, self.answers = fast, []

    def __getattr__(self, name):
        fn = getattr(self._fast, name)

        def noted(*args):
            self.answers.append(fn(*args))
            return self.answers[-1]
        return noted


@pytest.mark.parametrize("name", ["tree", "accept", "compact"])
def test_both_checks_make_the_same_call(name, monkeypatch):
    assert P._load_torch() and P._fast is not None, "_fastcall.so is not built"
    d, noted, side = tree_data(), Noted(P._fast), torch.cuda.Stream()
    monkeypatch.setattr(P, "_fast", noted)
    results = [one_call(name, d), one_call(name, d, side), one_call(name, d, side.cuda_stream)]
    assert noted.answers == [0, 0, 0]
    monkeypatch.setattr(P, "_fast", None)
    own = one_call(name, d)
    assert own[-1].item() == 0
    for other in results:
        assert len(other) == len(own)
        for a, b in zip(other, own):
            assert a.dtype == b.dtype and torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("name,key,change,error", [
    ("tree", "q", lambda t: t.float(), TypeError),
    ("tree", "q", lambda t: t.cpu(), ValueError),
    ("tree", "q", lambda t: t[:, :3], ValueError),
    ("tree", "q", lambda t: t[:, ::2], ValueError),
    ("tree", "tables", lambda t: t[:2], ValueError),
    ("tree", "tables", lambda t: t.long(), TypeError),
    ("tree", "starts", lambda t: t[:3], ValueError),
    ("tree", "lens", lambda t: t.cpu(), ValueError),
    ("tree", "mask", lambda t: t[:-1], ValueError),
    ("tree", "mask", lambda t: t.long(), TypeError),
    ("tree", "mask", lambda t: t[:, 0], ValueError),
    ("tree", "ws", lambda t: t.int(), TypeError),
    ("accept", "tokens", lambda t: t.short(), TypeError),
    ("accept", "targets", lambda t: t.int(), TypeError),
    ("accept", "parents", lambda t: t[:-1], ValueError),
    ("accept", "starts", lambda t: t[1:], ValueError),
    ("accept", "first", lambda t: t.cpu(), ValueError),
    ("compact", "kept", lambda t: t.long(), TypeError),
    ("compact", "kept", lambda t: t[::2], ValueError),
    ("compact", "starts", lambda t: t[1:], ValueError),
    ("compact", "num", lambda t: t[:2], ValueError),
    ("compact", "first", lambda t: t.long(), TypeError),
    ("compact", "tables", lambda t: t.t().contiguous().t(), ValueError)])
def test_a_check_that_fails_is_named_by_the_binding(name, key, change, error, monkeypatch):
    d, noted = tree_data(), Noted(P._fast)
    bad = dict(d, **{key: change(d[key])})
    messages = []
    for fast, answers in ((noted, [None]), (None, [None])):
        monkeypatch.setattr(P, "_fast", fast)
        with pytest.raises(error) as e:
            one_call(name, bad)
        messages.append(str(e.value))
        assert noted.answers == answers
    assert messages[0] == messages[1]


def test_a_small_workspace_is_refused():
    d = tree_data()
    d["ws"] = d["ws"][:-1]
    with pytest.raises(P.PagedKVError, match="INVALID_ARG"):
        one_call("tree", d)


def test_parents_of_long_chains():
    """tree_mask on the device, up to 32 words."""
    gen = torch.Generator().manual_seed(52)
    news = [1024, 0, 700, 1]
    parents = [random_parents(n, gen, 2) for n in news]
    parents[2] = [i - 1 for i in range(700)]
    starts = torch.tensor([0] + news).cumsum(0).to(I32)
    flat = torch.tensor([x for p in parents for x in p], dtype=I32)
    assert torch.equal(P.tree_mask(flat.cuda(), starts.cuda(), 32).cpu(), P.tree_mask(flat, starts, 32))


FIRST_CALL = """
import sys
sys.path[:0] = [{tests!r}, {root!r}]
import torch
import paged_kv_cache_146_gb300 as P
from test_gpu_tree_ranges import one_call, tree_data
import test_gpu_tree_ranges as R
d = tree_data()
pool, status = R.pool_of(d["c"], "bf16"), R.new_status()
out = torch.zeros_like(d["q"])
kept, num, nxt = torch.zeros_like(d["kept"]), torch.zeros_like(d["num"]), torch.zeros_like(d["tokens"][:3])
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    P.paged_tree_attention(pool, d["q"], d["tables"], d["starts"], d["lens"], d["mask"], 0.125, d["ws"], status,
                           out=out)
    P.tree_accept(d["tokens"], d["parents"], d["targets"], d["starts"], d["first"], status, kept=kept,
                  num_kept=num, next_tokens=nxt)
    P.cache_compact(pool, d["tables"], d["kept"], d["starts"], d["num"], d["first"], status)
assert not out.any() and not num.any()
graph.replay()
torch.cuda.synchronize()
mine = [out, kept, num, nxt, pool.k_pool, pool.v_pool]
want = one_call("tree", d)[:1] + one_call("accept", d)[:3] + one_call("compact", d)[:2]
assert status.item() == 0
for a, b in zip(mine, want):
    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
print("captured")
"""


def test_the_first_calls_of_a_process_are_captured(tmp_path):
    """Nothing that a kernel's first launch needs stands in a capture's way."""
    import os
    import subprocess
    import sys
    tests = os.path.dirname(os.path.abspath(__file__))
    script = tmp_path / "first.py"
    script.write_text(FIRST_CALL.format(tests=tests, root=os.path.dirname(tests)))
    run = subprocess.run([sys.executable, str(script)], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and run.stdout.strip().endswith("captured"), run.stdout + run.stderr
