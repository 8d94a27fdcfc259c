"""Cases of the operators that decode with a tree of drafted tokens, and their plain forms.

A small model drafts a tree of likely next tokens, the large model looks at all of them in
one step, and the path that it agrees with is kept.  The operators:

  tree     attention of each sequence's drafted tokens: a drafted token sees the sequence's
           cache and those drafted tokens that its bit mask names (itself and the tokens
           before it on its path).  The drafted tokens' K and V stand in the cache behind
           the sequence's own, in the tree's order.
  accept   walks each tree down from its root as long as some child holds the token that
           the large model answered with; gives the path's positions in the cache.
  compact  moves the cache's kept tokens together: the path behind the sequence's own
           tokens, or what a policy of leaving out tokens keeps of a whole cache.

`listed` and `draw` give the cases, `prepare` their inputs, `run` one pass (plain torch, or
the library's calls where `own` is set), `work` what a pass cannot do without, and `exact`
the results in 64 bits.
"""
import math

import torch

own = False

BS = 16                                  # tokens per block
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
TOKENS = {"int32": torch.int32, "int64": torch.int64}
WORDS = 31991                            # token ids of a vocabulary


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # one conversation with a small model, a handful of drafted tokens: latency
        dict(name="tree one", kind="tree", type="f16", hq=8, hkv=2, dim=64, seqs=1, new_lo=7,
             new_hi=7, prior_lo=530, prior_hi=530),
        # a few conversations, trees of different sizes
        dict(name="tree few", kind="tree", type="bf16", hq=32, hkv=8, dim=128, seqs=4, new_lo=9,
             new_hi=31, prior_lo=200, prior_hi=4000),
        # an ordinary batch, some sequences with hardly anything drafted
        dict(name="tree batch", kind="tree", type="bf16", hq=32, hkv=8, dim=128, seqs=48, new_lo=1,
             new_hi=25, prior_lo=17, prior_hi=6001),
        # a full server: many long contexts, trees of a fixed size
        dict(name="tree long batch", kind="tree", type="bf16", hq=32, hkv=8, dim=128, seqs=96,
             new_lo=16, new_hi=16, prior_lo=1000, prior_hi=16384),
        # wide trees
        dict(name="tree wide", kind="tree", type="bf16", hq=32, hkv=8, dim=128, seqs=24, new_lo=64,
             new_hi=64, prior_lo=500, prior_hi=8192),
        # a model with as many kv heads as query heads, ragged
        dict(name="tree many heads", kind="tree", type="f16", hq=40, hkv=40, dim=128, seqs=20,
             new_lo=3, new_hi=33, prior_lo=5, prior_hi=2500),
        # the answer to one small tree: latency
        dict(name="accept one", kind="accept", tokens="int64", seqs=1, new_lo=7, new_hi=7),
        # the answers to the trees of a full server
        dict(name="accept batch", kind="accept", tokens="int64", seqs=256, new_lo=21, new_hi=64),
        # the accepted paths of a full server's trees
        dict(name="compact paths", kind="compact", type="bf16", hkv=8, dim=128, seqs=96, new_lo=16,
             new_hi=16, kept_lo=1, kept_hi=6, prior=900, whole=False),
        # a small cache that keeps a third of its tokens
        dict(name="compact one", kind="compact", type="f16", hkv=2, dim=64, seqs=1, new_lo=911,
             new_hi=911, kept_lo=301, kept_hi=301, prior=0, whole=True),
        # long caches that keep about half of their tokens
        dict(name="compact caches", kind="compact", type="bf16", hkv=8, dim=128, seqs=9,
             new_lo=2000, new_hi=16384, kept_lo=1000, kept_hi=8000, prior=0, whole=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["tree", "tree", "tree", "accept", "compact", "compact"])
    if kind == "accept":
        hi = _log_int(rng, 1, 128)
        return dict(kind=kind, tokens=rng.choice(["int32", "int64"]), seqs=_log_int(rng, 1, 256),
                    new_lo=rng.randint(1, hi), new_hi=hi)
    hq, hkv = rng.choice([(32, 8), (8, 2), (8, 8), (16, 1), (10, 2), (40, 40), (12, 1), (6, 3)])
    case = dict(kind=kind, type=rng.choice(["bf16", "f16"]), dim=rng.choice([64, 128]), hkv=hkv)
    if kind == "compact":
        if rng.random() < 0.5:
            hi = _log_int(rng, 2, 128)
            case.update(seqs=_log_int(rng, 1, 128), new_lo=rng.randint(1, hi), new_hi=hi,
                        prior=_log_int(rng, 1, 500), whole=False)
        else:
            hi = _log_int(rng, 40, 16384)
            case.update(seqs=_log_int(rng, 1, max(1, 100_000 // hi)), new_lo=rng.randint(20, hi),
                        new_hi=hi, prior=0, whole=True)
            case["seqs"] = max(1, case["seqs"] * 8 // max(8, hkv))
        high = rng.randint(1, hi)
        return dict(case, kept_lo=rng.randint(1, high), kept_hi=high)
    case.update(hq=hq, seqs=_log_int(rng, 1, 96), new_hi=_log_int(rng, 1, 128))
    case["new_lo"] = rng.randint(1, case["new_hi"])
    # keys of the whole batch, and products of the padded plain form, at most
    most = min(700_000 * 8 // max(8, hkv) // case["seqs"],
               300_000_000 // (case["seqs"] * hq * case["new_hi"]))
    case["prior_hi"] = min(_log_int(rng, 1, 30000), max(1, most))
    case["prior_lo"] = rng.randint(0, case["prior_hi"])
    return case


# ----------------------------------------------------------- sizes that a case stands for
def _spread(n, lo, hi, phase):
    """n whole numbers spread over lo .. hi (fixed by the case, as `work` counts with them)."""
    return [lo + int(round((hi - lo) * ((i * 0.6180339887498949 + phase) % 1.0))) for i in range(n)]


def _news(case):
    """Drafted tokens of each sequence (compact, whole caches: all tokens)."""
    return _spread(case["seqs"], case["new_lo"], case["new_hi"], 0.9)


def _priors(case):
    """Tokens before the drafted ones."""
    if case["kind"] == "tree":
        return _spread(case["seqs"], case["prior_lo"], case["prior_hi"], 0.37)
    return _spread(case["seqs"], 0, case.get("prior", 900), 0.37)


def _kept(case):
    return [min(k, n) for k, n in zip(_spread(case["seqs"], case["kept_lo"], case["kept_hi"], 0.2),
                                      _news(case))]


# ------------------------------------------------------------------------------ inputs
def _starts(counts):
    starts = [0]
    for n in counts:
        starts.append(starts[-1] + n)
    return starts


def _random_trees(news, cpu):
    """Parents of every sequence's drafted tokens (-1: the root, which comes first); a parent
    comes before its children.  Trees as drafting leaves them: a trunk with branches."""
    draws = torch.rand(sum(news), generator=cpu).tolist()
    parents = []
    for n in news:
        for i in range(n):
            back = 1 + int(4 * draws[len(parents)] ** 3 * min(i, 3)) if i else 0
            parents.append(max(0, i - back) if i else -1)
    return parents


def _masks(news, parents, words):
    """Bit j of a drafted token's words: it sees drafted token j of its sequence."""
    rows, at = [], 0
    for n in news:
        seen = []
        for i in range(n):
            seen.append((seen[parents[at + i]] if i else 0) | 1 << i)
        at += n
        rows += [[(m >> 32 * w) & 0xffffffff for w in range(words)] for m in seen]
    return torch.tensor(rows, dtype=torch.int64).to(torch.int32)


def _prepare_accept(case, seed):
    cpu = torch.Generator()
    cpu.manual_seed(seed)
    news, dt = _news(case), TOKENS[case["tokens"]]
    total, starts = sum(news), _starts(news)
    parents = _random_trees(news, cpu)
    tokens = torch.randint(0, WORDS, (total,), generator=cpu)
    targets = torch.randint(0, WORDS, (total,), generator=cpu)
    # the large model agrees with some child of most tokens (one after the other: several
    # children of one token, the last one counts)
    at = [s for s, n in zip(starts, news) for _ in range(n)]
    agrees, answer = torch.rand(total, generator=cpu).tolist(), tokens.tolist()
    chosen = {at[i] + parents[i]: answer[i] for i in torch.randperm(total, generator=cpu).tolist()
              if parents[i] >= 0 and agrees[i] < 0.9}
    if chosen:
        targets[list(chosen)] = torch.tensor(list(chosen.values()))
    return dict(case=case, tokens=tokens.to(DEV, dt), targets=targets.to(DEV, dt),
                parents=torch.tensor(parents, dtype=torch.int32, device=DEV),
                starts=torch.tensor(starts, dtype=torch.int32, device=DEV),
                first=torch.tensor(_priors(case), dtype=torch.int32, device=DEV),
                kept=torch.empty(total, dtype=torch.int32, device=DEV),
                num_kept=torch.empty(len(news), dtype=torch.int32, device=DEV),
                next=torch.empty(len(news), dtype=dt, device=DEV),
                status=torch.zeros(1, dtype=torch.int32, device=DEV))


def prepare(case, seed):
    if case["kind"] == "accept":
        return _prepare_accept(case, seed)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    cpu = torch.Generator()
    cpu.manual_seed(seed)
    dt, hkv, dim, kind, seqs = TYPES[case["type"]], case["hkv"], case["dim"], case["kind"], case["seqs"]
    news, priors = _news(case), _priors(case)
    lens = [p + n for p, n in zip(priors, news)]
    blocks = [-(-n // BS) for n in lens]
    nb, maxb = sum(blocks) + 3, max(blocks) + 2
    ids = torch.randperm(nb, generator=gen, device=DEV).to(torch.int32)[:sum(blocks)].cpu()
    tables = torch.full((seqs, maxb), -1, dtype=torch.int32)
    for s, (b, at) in enumerate(zip(blocks, _starts(blocks))):
        tables[s, :b] = ids[at:at + b]
    shape = (nb, hkv, BS, dim)
    st = dict(case=case, scale=1.0 / math.sqrt(dim), tables=tables.to(DEV),
              lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
              first=torch.tensor(priors, dtype=torch.int32, device=DEV),
              k_pool=torch.randn(shape, generator=gen, device=DEV, dtype=dt),
              v_pool=torch.randn(shape, generator=gen, device=DEV, dtype=dt),
              status=torch.zeros(1, dtype=torch.int32, device=DEV))
    if kind == "tree":
        total = sum(news)
        words = -(-max(news) // 32)
        st["q"] = torch.randn((total, case["hq"], dim), generator=gen, device=DEV, dtype=dt)
        st["out"] = torch.empty_like(st["q"])
        st["starts"] = torch.tensor(_starts(news), dtype=torch.int32, device=DEV)
        st["mask"] = _masks(news, _random_trees(news, cpu), words).to(DEV)
    else:
        # kept positions of each sequence in order; a path begins with the tree's root, a cache
        # of which tokens are left out keeps its first one
        kept = torch.full((sum(news),), -1, dtype=torch.int32)
        for n, k, p, at in zip(news, _kept(case), priors, _starts(news)):
            some = 1 + torch.randperm(n - 1, generator=cpu)[:k - 1].sort().values
            kept[at] = p
            kept[at + 1:at + k] = p + some.to(torch.int32)
        st["kept"] = kept.to(DEV)
        st["starts"] = torch.tensor(_starts(news), dtype=torch.int32, device=DEV)
        st["num_kept"] = torch.tensor(_kept(case), dtype=torch.int32, device=DEV)
    if own:                                # the pool's ledger, and a workspace, as a program keeps them
        import paged_kv_cache_146_gb300 as pkv
        st["pool"] = pkv.KVPool(nb, hkv, dim, case["type"])
        if kind == "tree":
            size = pkv.tree_workspace_bytes(total, case["hq"], hkv, dim)
            st["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    return st


# ------------------------------------------------------------------- a pass, plain form
def _run_tree(st):
    case = st["case"]
    seqs, hq, hkv, dim, most = case["seqs"], case["hq"], case["hkv"], case["dim"], case["new_hi"]
    start, lens, first = st["starts"].long(), st["lens"].long(), st["first"].long()
    i = torch.arange(most, device=DEV)
    row = (start[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)              # [S][C]
    j = torch.arange(case["prior_hi"] + most, device=DEV)
    jj = torch.minimum(j[None], lens[:, None] - 1)
    block = torch.gather(st["tables"].long(), 1, jj // BS)
    k = st["k_pool"][block, :, jj % BS].float()                               # [S][n][Hkv][dim]
    v = st["v_pool"][block, :, jj % BS].float()
    q = st["q"][row].float().view(seqs, most, hkv, hq // hkv, dim).permute(0, 2, 3, 1, 4)
    x = torch.matmul(q.reshape(seqs, hkv, -1, dim), k.permute(0, 2, 3, 1)) * st["scale"]
    x = x.view(seqs, hkv, hq // hkv, most, -1)
    # bits of the drafted tokens: [S][C][n]
    d = (j[None] - first[:, None]).clamp(0, 32 * st["mask"].shape[1] - 1)     # [S][n]
    word = torch.gather(st["mask"][row].long(), 2, (d // 32)[:, None].expand(-1, most, -1))
    see = ((word >> (d % 32)[:, None]) & 1).bool() & (j[None] < lens[:, None])[:, None]
    see = (see | (j[None] < first[:, None])[:, None])[:, None, None]
    x = x.masked_fill_(~see, -math.inf)
    p = torch.exp_(x.sub_(x.amax(-1, keepdim=True).clamp(min=-1e30)))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(seqs, hkv, -1, j.numel()), v.transpose(1, 2))
    o = o.view(seqs, hkv, -1, most, dim) / total
    t = torch.arange(st["q"].shape[0], device=DEV)
    s = torch.searchsorted(start, t, right=True) - 1
    return o.permute(0, 3, 1, 2, 4)[s, t - start[s]].reshape(-1, hq, dim).to(st["q"].dtype)


def _run_accept(st):
    start, parents = st["starts"].long(), st["parents"].long()
    total = parents.numel()
    t = torch.arange(total, device=DEV)
    s = torch.searchsorted(start, t, right=True) - 1
    root = t == start[s]
    up = torch.where(parents >= 0, start[s] + parents, t)                     # the parent's row
    same = (st["tokens"] == st["targets"][up]) & (parents >= 0)
    lowest = torch.full((total,), total, device=DEV)
    lowest = lowest.scatter_reduce(0, up, torch.where(same, t, total), "amin")
    on_path = (same & (lowest[up] == t)) | root
    # a token is kept when it and all those above it agree: twice as far up each time
    for _ in range(max(1, st["case"]["new_hi"] - 1).bit_length()):
        on_path = on_path & on_path[up]
        up = up[up]
    count = torch.cumsum(on_path, 0)
    before = count[start[:-1]] - on_path[start[:-1]].long()
    num = count[start[1:] - 1] - before
    place = torch.where(on_path, start[s] + count - 1 - before[s], total)
    kept = torch.full((total + 1,), -1, device=DEV)
    kept[place] = st["first"].long()[s] + t - start[s]
    kept[total] = -1
    last = torch.zeros_like(num).scatter_reduce(0, s, torch.where(on_path, t, 0), "amax")
    st["kept"].copy_(kept[:total])
    st["num_kept"].copy_(num)
    st["next"].copy_(st["targets"][last])
    return st["kept"], st["num_kept"], st["next"]


def _run_compact(st):
    start, kept = st["starts"].long(), st["kept"].long()
    t = torch.arange(kept.numel(), device=DEV)
    s = torch.searchsorted(start, t, right=True) - 1
    i = t - start[s]
    moved = i < st["num_kept"][s]
    s, src, dst = s[moved], kept[moved], (st["first"].long()[s] + i)[moved]
    tables = st["tables"].long()
    for pool in (st["k_pool"], st["v_pool"]):
        pool[tables[s, dst // BS], :, dst % BS] = pool[tables[s, src // BS], :, src % BS]
    return st["k_pool"], st["v_pool"]


# ---------------------------------------------------------- a pass, the library's calls
def _run_own(st):
    import paged_kv_cache_146_gb300 as pkv
    kind = st["case"]["kind"]
    if kind == "tree":
        return pkv.paged_tree_attention(st["pool"], st["q"], st["tables"], st["starts"], st["lens"],
                                        st["mask"], st["scale"], st["workspace"], st["status"],
                                        out=st["out"], k_pool=st["k_pool"], v_pool=st["v_pool"])
    if kind == "accept":
        return pkv.tree_accept(st["tokens"], st["parents"], st["targets"], st["starts"], st["first"],
                               st["status"], kept=st["kept"], num_kept=st["num_kept"],
                               next_tokens=st["next"])
    pkv.cache_compact(st["pool"], st["tables"], st["kept"], st["starts"], st["num_kept"],
                      st["first"], st["status"], k_pool=st["k_pool"], v_pool=st["v_pool"])
    return st["k_pool"], st["v_pool"]


def run(st):
    if own:
        return _run_own(st)
    return {"tree": _run_tree, "accept": _run_accept, "compact": _run_compact}[st["case"]["kind"]](st)


# ------------------------------------------------------------------- what a pass must do
def work(case):
    news, seqs = _news(case), case["seqs"]
    total = sum(news)
    if case["kind"] == "accept":
        size = 8 if case["tokens"] == "int64" else 4
        # the trees in, the positions out, lengths and the next tokens
        return {"bytes": total * (2 * size + 8) + seqs * (12 + size), "flops": total}
    hkv, dim = case["hkv"], case["dim"]
    if case["kind"] == "compact":
        moved = sum(k - 1 for k in _kept(case))                 # a first token stays
        return {"bytes": moved * 2 * (2 * hkv * dim * 2) + 4 * sum(_kept(case)) + 12 * seqs,
                "flops": 0}
    hq, priors = case["hq"], _priors(case)
    keys = sum(priors) + total
    tables = 4 * sum(-(-(p + n) // BS) for p, n in zip(priors, news))
    pairs = sum(n * (p + 1) for p, n in zip(priors, news))      # the cache and the token itself
    return {"bytes": keys * 4 * hkv * dim + 2 * total * hq * dim * 2 + tables
            + total * 4 * -(-max(news) // 32) + 8 * seqs, "flops": 4 * pairs * hq * dim}


# ------------------------------------------------------------------ results in 64 bits
def _exact_tree(case, st):
    hq, hkv, dim = case["hq"], case["hkv"], case["dim"]
    group, out, row = hq // hkv, torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV), 0
    for s, (n, prior) in enumerate(zip(_news(case), _priors(case))):
        length = prior + n
        blocks = st["tables"][s, :-(-length // BS)].long()
        k, v = (p[blocks].transpose(0, 1).reshape(hkv, -1, dim)[:, :length].double()
                for p in (st["k_pool"], st["v_pool"]))
        bits = st["mask"][row:row + n].tolist()
        hide = torch.zeros((n, length), dtype=torch.bool)
        for i in range(n):
            for j in range(n):
                hide[i, prior + j] = not (bits[i][j // 32] >> (j % 32)) & 1
        hide = hide.to(DEV)
        for h in range(hq):
            x = (st["q"][row:row + n, h].double() @ k[h // group].T) * st["scale"]
            w = torch.softmax(x.masked_fill(hide, -math.inf), -1)
            out[row:row + n, h] = w @ v[h // group]
        row += n
    return out


def _exact_accept(case, st):
    tokens, targets, parents = (st[x].tolist() for x in ("tokens", "targets", "parents"))
    kept, nums, nexts, at = [], [], [], 0
    for n, prior in zip(_news(case), _priors(case)):
        path, found = [0], True
        while found:
            found = False
            for i in range(path[-1] + 1, n):
                if parents[at + i] == path[-1] and tokens[at + i] == targets[at + path[-1]]:
                    path.append(i)
                    found = True
                    break
        kept += [prior + i for i in path] + [-1] * (n - len(path))
        nums.append(len(path))
        nexts.append(targets[at + path[-1]])
        at += n
    return tuple(torch.tensor(x, dtype=st[y].dtype) for x, y in
                 ((kept, "kept"), (nums, "num_kept"), (nexts, "next")))


def _exact_compact(case, st):
    pools, at = [st[x].double() for x in ("k_pool", "v_pool")], 0
    for s, (n, k, prior) in enumerate(zip(_news(case), _kept(case), _priors(case))):
        slots = (st["tables"][s].long()[:, None] * BS + torch.arange(BS, device=DEV)).view(-1)
        src = slots[st["kept"][at:at + k].long()]
        dst = slots[prior:prior + k]
        for pool in pools:
            for h in range(case["hkv"]):
                rows = pool[src // BS, h, src % BS].clone()
                pool[dst // BS, h, dst % BS] = rows
        at += n
    return tuple(pools)


def exact(case, seed):
    st = prepare(case, seed)
    return {"tree": _exact_tree, "accept": _exact_accept, "compact": _exact_compact}[case["kind"]](case, st)
