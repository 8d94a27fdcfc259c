"""Sums over long contexts: what the rounding of many additions takes off a result."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import libbuild  # noqa: E402
from paged_kv_cache_146_gb300 import (KVPool, paged_tree_attention, status_check,  # noqa: E402
                                      tree_workspace_bytes)

libbuild.ensure_built()
pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def run(name, dim, priors, news, group, rise=0.0, seed=0):
    """Sequences that share one cache of positive values, one kv head; scores within +-1 and a rise along
    the keys.  Drafted token i of a sequence sees the cache and itself."""
    dt, longest = DT[name], max(p + n for p, n in zip(priors, news))
    gen = torch.Generator(device="cuda").manual_seed(seed)
    nb, S, T = -(-longest // 16), len(priors), sum(news)
    pool = KVPool(nb, 1, dim, name, device="cuda")
    k = torch.randn((nb, 1, 16, dim), generator=gen, device="cuda") * 0.1
    k[..., 0] = (torch.arange(nb * 16, device="cuda") / (nb * 16)).view(nb, 1, 16)
    pool.k_pool.copy_(k)
    pool.v_pool.copy_(torch.randn((nb, 1, 16, dim), generator=gen, device="cuda").abs() + 0.5)
    q = torch.randn((T, group, dim), generator=gen, device="cuda")
    q[..., 0] = rise
    q = q.to(dt)
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    words = -(-max(news) // 32)
    mask = torch.zeros((T, words), dtype=torch.int64)
    for s, n in enumerate(news):
        for i in range(n):
            mask[starts[s] + i, i // 32] = 1 << i % 32
    mask = torch.where(mask >= 2 ** 31, mask - 2 ** 32, mask).to("cuda", torch.int32)
    lens = torch.tensor([p + n for p, n in zip(priors, news)], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.randint(0, 256, (tree_workspace_bytes(T, group, 1, dim),), dtype=torch.uint8, device="cuda")
    tables = torch.arange(nb, dtype=torch.int32, device="cuda").expand(S, nb).contiguous()
    got = paged_tree_attention(pool, q, tables, torch.tensor(starts, dtype=torch.int32, device="cuda"), lens, mask,
                               1.0, ws, status)
    assert status_check(status) == (0, 0)
    return got, pool, q, starts


def check(name, dim, priors, news, group, rise=0.0, seqs=None):
    """Relative to a result of positive terms: a tile is eight matrix instructions (four steps of 16
    keys, two parts), each of which may truncate its products' sum and its addition to O by 2^-23; O
    takes at most 128 tiles, 2^-12 in all.  Sums of the moved ones and of the weights round by 2^-24
    for each tile or less.  Weights, in numerator and denominator: 2^-16 (bf16 parts) or 2^-22 (fp16), 2^-20
    (exponent and argument), and the error of a score, whose dim / 16 instructions may truncate twice
    each by 2^-23 of the sum of |q k|.  Then the result's half step."""
    got, pool, q, starts = run(name, dim, priors, news, group, rise)
    keys = pool.k_pool.view(-1, dim).double(), pool.v_pool.view(-1, dim).double()
    for s in range(len(priors)) if seqs is None else seqs:
        p, n = priors[s], news[s]
        for i in range(n):
            j = torch.arange(p + 1, device="cuda")
            j[-1] = p + i
            k, v = (t[j] for t in keys)
            x = q[starts[s] + i].double() @ k.T
            want = torch.softmax(x, -1) @ v
            score = (q[starts[s] + i].double().abs() @ k.abs().T).max().item()
            assert score <= 32
            weight = (2.0 ** -16 if name == "bf16" else 2.0 ** -22) + 2.0 ** -20 + dim * 2.0 ** -23 * score / 8
            rel = 2.0 ** -12 + (p / 64 + 64) * 2.0 ** -24 + 2 * weight + torch.finfo(DT[name]).eps / 2
            worst = (got[starts[s] + i].double() / want - 1).abs().max().item()
            assert worst <= rel, (s, i, worst, rel)


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
def test_whole_long_contexts(name, dim):
    """As many sequences as CTAs, each goes through 131,072 tokens by itself."""
    check(name, dim, [131071] * 304, [1] * 304, 1, seqs=[0, 151, 303])


@pytest.mark.parametrize("name,dim,group", [("f16", 128, 4), ("bf16", 128, 4), ("f16", 64, 16), ("bf16", 64, 3)])
def test_long_and_short_contexts_in_turn(name, dim, group):
    """Sums that are moved, pieces of cut sequences and short sequences in the same CTAs; the largest
    score rises along the keys (2^5.8), so references move between the sums."""
    priors = [(8191, 40000, 30, 8192, 8193, 16400, 0, 66000)[s % 8] for s in range(120)]
    news = [(1, 2, 5, 1, 3, 1, 2, 1)[s % 8] for s in range(120)]
    check(name, dim, priors, news, group, rise=4.0, seqs=list(range(16, 24)) + [119])


@pytest.mark.parametrize("name", ["f16", "bf16"])
def test_few_very_long_contexts(name):
    """Every piece of a cut sequence holds a moved sum."""
    check(name, 128, [600000, 450001], [2, 1], 8)
    check(name, 64, [300000], [40], 8, rise=4.0)


@pytest.mark.parametrize("name", ["f16", "bf16"])
def test_results_do_not_vary(name):
    """Moved sums are added in one order, whatever the workspace held."""
    priors = [(20000, 70, 12000, 9000)[s % 4] for s in range(90)]
    args = (name, 128, priors, [1 + s % 3 for s in range(90)], 4, 4.0)
    first = run(*args)[0]
    for _ in range(4):
        assert torch.equal(run(*args)[0], first)
