"""Plain 64-bit forms of attention over trees of drafted tokens, of the accepted path and of
moving kept tokens together, with bounds on what the kernels' roundings can add.  CPU only;
nothing of the library is used."""
import torch

from serving_reference import HALF_STEP, SUBNORMAL, random_case

# relative error of a weight on its way into P V: two bf16 parts, the first truncated
# (remainder below 2^-7 of the weight, its rounding 2^-8 of that), or two fp16 parts
WEIGHT = {torch.bfloat16: 2.0 ** -15, torch.float16: 2.0 ** -22}


def path_masks(parents):
    """Whole numbers of one tree: bit j of entry i, node i sees node j."""
    seen = []
    for i, up in enumerate(parents):
        seen.append((seen[up] if up >= 0 else 0) | 1 << i)
    return seen


def random_parents(n, gen, branch=3):
    if n == 0:
        return []
    back = torch.randint(1, branch + 1, (n,), generator=gen).tolist()
    return [-1] + [max(0, i - back[i]) for i in range(1, n)]


def mask_words(rows, words):
    """Whole numbers -> int32 [T][words]."""
    t = torch.tensor([[(m >> 32 * w) & 0xffffffff for w in range(words)] for m in rows],
                     dtype=torch.int64).view(len(rows), words)
    return t.to(torch.int32)


class TreeCase:
    """Pools, tables and drafted tokens of sequences with `priors` tokens and `news` drafted
    ones; `masks`: whole numbers per row (default: random trees).  Blocks lie anywhere; what no
    sequence holds (the ends of last blocks among it) is NaN."""

    def __init__(self, priors, news, hq, hkv, dim, dtype, seed, masks=None, words=None, spare=0):
        self.gen = gen = torch.Generator().manual_seed(seed)
        self.priors, self.news, self.hq, self.hkv, self.dim, self.dtype = priors, news, hq, hkv, dim, dtype
        self.lens = [p + n for p, n in zip(priors, news)]
        self.maxb = max([-(-n // 16) for n in self.lens] + [0]) + 1
        self.tables, self.nb = random_case(gen, self.lens, hkv, self.maxb)
        self.k, self.v = (torch.randn((self.nb, hkv, 16, dim), generator=gen).to(dtype) for _ in range(2))
        held = torch.zeros((self.nb, 16), dtype=torch.bool)
        for s, n in enumerate(self.lens):
            j = torch.arange(n)
            held[self.tables[s].long()[j // 16], j % 16] = True
        for p in (self.k, self.v):
            p.permute(0, 2, 1, 3)[~held] = float("nan")
        self.starts = [0]
        for n in news:
            self.starts.append(self.starts[-1] + n)
        self.rows = self.starts[-1]
        self.parents = [random_parents(n, gen) for n in news]
        self.masks = masks if masks is not None else [m for p in self.parents for m in path_masks(p)]
        self.words = words or max(1, -(-max(news + [0]) // 32))
        self.q = torch.randn((self.rows + spare, hq, dim), generator=gen).to(dtype)

    def sees(self, s):
        """[n][L]: what the drafted tokens of sequence s see."""
        n, prior = self.news[s], self.priors[s]
        see = torch.ones((n, prior + n), dtype=torch.bool)
        for i in range(n):
            m = self.masks[self.starts[s] + i]
            see[i, prior:] = torch.tensor([(m >> d) & 1 for d in range(n)], dtype=torch.bool)
        return see

    def kv(self, s, g):
        j = torch.arange(self.lens[s])
        blk = self.tables[s].long()[j // 16]
        return (p[blk, g, j % 16].double() for p in (self.k, self.v))

    def expect(self, s, scale, q=None):
        """Results of sequence s, [n][Hq][D], and the bounds on a kernel's error.

        The output is sum p v / sum p.  A weight's relative error is at most WEIGHT (its parts)
        + 2^-20 (exponent, its argument, the joining of pieces) + the error of its score: products
        of two 16-bit values are exact in fp32, and a chain of D fp32 additions that may truncate
        is off by at most D 2^-23 times the sum of magnitudes.  Numerator and denominator then move
        by that much of sum p |v| and sum p; weights below fp16's normal range add 2^-25 |v| each
        (the largest weight is at least 1).  Sums of n weights or products that may truncate add n
        2^-23 at most, and the tiles are summed one after the other, 64 keys at a time.  Last, one
        rounding to the output type."""
        q = self.q if q is None else q
        n, group = self.news[s], self.hq // self.hkv
        out = torch.zeros((n, self.hq, self.dim), dtype=torch.float64)
        bound = torch.zeros_like(out)
        see = self.sees(s)
        steps = self.lens[s] / 64 + 64
        for g in range(self.hkv):
            k, v = self.kv(s, g)
            for h in range(g * group, (g + 1) * group):
                qq = q[self.starts[s]:self.starts[s] + n, h].double()
                x = ((qq @ k.T) * scale).masked_fill(~see, float("-inf"))
                p = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-1e300))
                p = p.masked_fill(~see, 0.0)
                total = p.sum(-1, keepdim=True)
                empty = total == 0
                total = torch.where(empty, 1.0, total)
                o = (p @ v) / total
                score = (abs(scale) * (qq.abs() @ k.abs().T)).masked_fill(~see, 0.0).amax(-1, keepdim=True)
                rel = WEIGHT[self.dtype] + 2.0 ** -20 + (self.dim * score + steps) * 2.0 ** -23
                tiny = 2.0 ** -25 * (see.double() @ v.abs()) / total
                out[:, h] = o
                bound[:, h] = (2 * rel * (p @ v.abs()) / total + tiny + HALF_STEP[self.dtype] * o.abs()
                               + SUBNORMAL[self.dtype])
        return out, bound


def accept_path(tokens, parents, targets):
    """Nodes of one tree that are kept, root first."""
    if not parents:
        return []
    path, found = [0], True
    while found:
        found = False
        for i in range(len(parents)):
            if parents[i] == path[-1] and tokens[i] == targets[path[-1]]:
                path.append(i)
                found = True
                break
    return path


def compact(pool, table, kept, first):
    """pool [nb][Hkv][bs][D] of which one sequence's `kept` positions move to first, first + 1, ...;
    all are read before the first is written."""
    bs = pool.shape[2]
    rows = [pool[table[p // bs], :, p % bs].clone() for p in kept]
    for i, r in enumerate(rows):
        pool[table[(first + i) // bs], :, (first + i) % bs] = r
