"""Cases of the serving operators around the paged cache, and their plain forms.

The operators:

  append   K and V of new tokens go to their slots in a paged cache, K (and the queries
           beside it) rotated by the tokens' positions on the way; 16-bit pools, and 8-bit
           pools with one scale for each block of tokens and kv head.
  decode8  single-token attention over such an 8-bit cache.
  window   single-token attention over the last `window` tokens and the first `sinks` tokens
           of each sequence (16-bit and 8-bit pools), and the same for chunks of a prompt
           (16-bit pools).

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


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a mid-sized batch: one token per sequence, queries, keys and values
        # as slices of one fused projection, batch padded to a fixed size
        dict(name="append step", kind="append", type="bf16", hq=32, hkv=8, dim=128, rot=128,
             pairs="halves", seqs=57, new_lo=1, new_hi=1, prior=4000, pad=7),
        # ragged prompts of a smaller model: half of each head rotated, neighbouring pairs
        dict(name="append prompts", kind="append", type="f16", hq=8, hkv=8, dim=64, rot=32,
             pairs="neighbours", seqs=13, new_lo=37, new_hi=1900, prior=700, pad=0),
        # a decode step into an 8-bit cache: every token lands inside a block that is partly full
        dict(name="append step 8-bit", kind="append8", type="bf16", hq=32, hkv=8, dim=128, rot=128,
             pairs="halves", seqs=203, new_lo=1, new_hi=1, prior=2500, pad=0),
        # long prompts into an 8-bit cache
        dict(name="append prompts 8-bit", kind="append8", type="bf16", hq=32, hkv=8, dim=128,
             rot=128, pairs="halves", seqs=9, new_lo=500, new_hi=3500, prior=40, pad=0),
        # one short conversation with a small model: latency
        dict(name="8-bit one sequence", kind="decode8", type="f16", hq=8, hkv=2, dim=64, seqs=1,
             len_lo=777, len_hi=777, window=0, sinks=0),
        # an ordinary batch of ragged contexts
        dict(name="8-bit batch", kind="decode8", type="bf16", hq=32, hkv=8, dim=128, seqs=48,
             len_lo=17, len_hi=6001, window=0, sinks=0),
        # a full server: many long contexts
        dict(name="8-bit long batch", kind="decode8", type="bf16", hq=32, hkv=8, dim=128, seqs=160,
             len_lo=1000, len_hi=16384, window=0, sinks=0),
        # an 8-bit cache whose blocks behind the window were given back
        dict(name="8-bit window", kind="decode8", type="bf16", hq=40, hkv=40, dim=128, seqs=64,
             len_lo=3, len_hi=9000, window=1024, sinks=4),
        # few sequences and a narrow window: latency
        dict(name="window few", kind="window", type="bf16", hq=32, hkv=8, dim=128, seqs=3,
             len_lo=90, len_hi=5000, window=128, sinks=4),
        # a large batch far behind its window, the blocks in between given back
        dict(name="window batch", kind="window", type="bf16", hq=32, hkv=8, dim=128, seqs=256,
             len_lo=40, len_hi=16000, window=1024, sinks=4),
        # one chunk of a small model's prompt, odd window
        dict(name="window chunk", kind="prefill", type="f16", hq=8, hkv=8, dim=64, seqs=1,
             new_lo=300, new_hi=300, prior=1811, window=257, sinks=5),
        # chunked prefill of a batch of long prompts
        dict(name="window prompts", kind="prefill", type="bf16", hq=32, hkv=8, dim=128, seqs=12,
             new_lo=100, new_hi=2048, prior=4000, window=1024, sinks=4),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["append", "append8", "decode8", "decode8", "window", "window", "prefill"])
    dim = rng.choice([64, 128])
    hq, hkv = rng.choice([(32, 8), (8, 2), (8, 8), (16, 1), (10, 2), (40, 40), (12, 1), (6, 3)])
    case = dict(kind=kind, type=rng.choice(["bf16", "f16"]), hq=hq, hkv=hkv, dim=dim)
    if kind in ("append", "append8"):
        case["rot"] = rng.choice([r for r in (16, 32, 64, 96, 128) if r <= dim])
        case["pairs"] = rng.choice(["halves", "neighbours"])
        if rng.random() < 0.5:
            case.update(seqs=_log_int(rng, 1, 512), new_lo=1, new_hi=1)
        else:
            case.update(seqs=_log_int(rng, 1, 12), new_lo=_log_int(rng, 1, 40),
                        new_hi=_log_int(rng, 41, 1500))
        case.update(prior=_log_int(rng, 1, 3000), pad=rng.choice([0, 0, 5]))
        return case
    if kind == "prefill":
        case.update(seqs=_log_int(rng, 1, 8), new_lo=_log_int(rng, 1, 100),
                    new_hi=_log_int(rng, 101, 1600), prior=_log_int(rng, 1, 4000),
                    window=_log_int(rng, 16, 1500), sinks=rng.choice([0, 1, 4, 19, 64]))
        return case
    tokens = 700_000 // max(1, hkv // 8)               # over the whole batch, at most
    case["seqs"] = _log_int(rng, 1, 300)
    hi = min(_log_int(rng, 30, 30000), max(30, tokens // case["seqs"]))
    case.update(len_lo=rng.randint(1, max(1, hi // 2)), len_hi=hi, window=0, sinks=0)
    if kind == "window" or rng.random() < 0.3:
        case.update(window=_log_int(rng, 1, 4096), sinks=rng.choice([0, 1, 4, 16, 33]))
    return case


# ----------------------------------------------------------- sizes that a case stands for
def _spread(n, lo, hi, phase):
    """n whole numbers spread over lo .. hi (fixed by the case, as `work` counts with them)."""
    return [lo + int(round((hi - lo) * ((i * 0.6180339887498949 + phase) % 1.0))) for i in range(n)]


def _news(case):
    return _spread(case["seqs"], case["new_lo"], case["new_hi"], 0.9)


def _priors(case):
    return _spread(case["seqs"], 0, case["prior"], 0.37)


def _lens(case):
    if case["kind"] in ("append", "append8", "prefill"):
        return [p + n for p, n in zip(_priors(case), _news(case))]
    return _spread(case["seqs"], case["len_lo"], case["len_hi"], 0.9)


def _first_query(case):
    """Position of each sequence's first query."""
    if case["kind"] == "prefill":
        return _priors(case)
    return [n - 1 for n in _lens(case)]


def _visible_blocks(case):
    """Per sequence the logical blocks that the call may read or write."""
    out = []
    for n, q0 in zip(_lens(case), _first_query(case)):
        nb = -(-n // BS)
        if case.get("window"):
            first = max(0, q0 - case["window"] + 1) // BS
            out.append([b for b in range(nb) if b * BS < case["sinks"] or b >= first])
        else:
            out.append(list(range(nb)))
    return out


# ------------------------------------------------------------------------------ inputs
def _record_index(dim, device):
    """Byte of (token, dimension) within the K or V codes of an 8-bit record."""
    t = torch.arange(BS, device=device)[:, None]
    d = torch.arange(dim, device=device)[None, :]
    line = t * dim // 128
    chunk = (d // 16) ^ (4 * (t & 1)) ^ (2 * ((t >> 1) & 3))
    return line * 128 + chunk * 16 + d % 16


def _random_records(nb, hkv, dim, gen):
    """An 8-bit pool's records as quantised normal values leave them."""
    kv = torch.zeros((nb, hkv, 32 * dim + 32), dtype=torch.uint8, device=DEV)
    codes = torch.randn((nb, hkv, 32 * dim), generator=gen, device=DEV, dtype=torch.float16)
    kv[:, :, :32 * dim] = codes.mul_(36).round_().clamp_(-127, 127).add_(128).to(torch.uint8)
    scales = torch.rand((nb, hkv, 2), generator=gen, device=DEV) * 0.03 + 0.01
    kv[:, :, 32 * dim:32 * dim + 8] = scales.view(torch.uint8).reshape(nb, hkv, 8)
    return kv


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt, hq, hkv, dim, kind = TYPES[case["type"]], case["hq"], case["hkv"], case["dim"], case["kind"]
    lens, seqs = _lens(case), case["seqs"]
    vis = _visible_blocks(case)
    used = sum(len(v) for v in vis)
    nb = used + 3
    maxb = max(-(-n // BS) for n in lens) + 2
    ids = torch.randperm(nb, generator=gen, device=DEV).to(torch.int32)[:used].cpu()
    tables = torch.full((seqs, maxb), -1, dtype=torch.int32)
    rows = torch.tensor([s for s, v in enumerate(vis) for _ in v])
    cols = torch.tensor([b for v in vis for b in v])
    tables[rows, cols] = ids
    st = dict(case=case, scale=1.0 / math.sqrt(dim), tables=tables.to(DEV),
              lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
              status=torch.zeros(1, dtype=torch.int32, device=DEV))
    eight = kind in ("append8", "decode8")
    if eight:
        st["kv"] = _random_records(nb, hkv, dim, gen)
        st["byte"] = _record_index(dim, DEV)
    else:
        shape = (nb, hkv, BS, dim)
        st["k_pool"] = torch.randn(shape, generator=gen, device=DEV, dtype=dt)
        st["v_pool"] = torch.randn(shape, generator=gen, device=DEV, dtype=dt)
    if kind in ("append", "append8"):
        news, priors = _news(case), _priors(case)
        tokens = sum(news)
        total = tokens + case["pad"]
        seq = torch.tensor([s for s, n in enumerate(news) for _ in range(n)])
        pos = torch.tensor([p + i for p, n in zip(priors, news) for i in range(n)])
        block = tables[seq, pos // BS].long()
        slots = torch.full((total,), -1, dtype=torch.int64)
        slots[:tokens] = block * BS + pos % BS
        positions = torch.zeros(total, dtype=torch.int32)
        positions[:tokens] = pos
        half = case["rot"] // 2
        freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
        angle = torch.arange(max(lens) + 1, dtype=torch.float64)[:, None] * freq
        st["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32).to(DEV)
        qkv = torch.randn((total, (hq + 2 * hkv) * dim), generator=gen, device=DEV, dtype=dt)
        st["q"] = qkv[:, :hq * dim].view(total, hq, dim)
        st["k"] = qkv[:, hq * dim:(hq + hkv) * dim].view(total, hkv, dim)
        st["v"] = qkv[:, (hq + hkv) * dim:].view(total, hkv, dim)
        st["q_out"] = torch.zeros((total, hq, dim), device=DEV, dtype=dt)
        st["slots"], st["positions"], st["tokens"] = slots.to(DEV), positions.to(DEV), tokens
        if eight:
            touched = torch.unique(block).to(torch.int32).to(DEV)
            st["touched"] = touched
            shape = (touched.numel(), hkv, BS, dim)
            st["k_out"], st["v_out"] = (torch.empty(shape, device=DEV, dtype=dt) for _ in range(2))
    else:
        total = seqs
        if kind == "prefill":
            starts = [0]
            for n in _news(case):
                starts.append(starts[-1] + n)
            total = starts[-1]
            st["query_start"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
        st["q"] = torch.randn((total, hq, dim), generator=gen, device=DEV, dtype=dt)
        st["out"] = torch.empty_like(st["q"])
    if own:                                # the pool's ledger, and a workspace, as a program keeps them
        import paged_kv_cache_146_gb300 as pkv
        name = ("b8_" if eight else "") + case["type"]
        st["pool"] = pkv.KVPool(nb, hkv, dim, name)
        if kind == "prefill":
            size = pkv.prefill_workspace_bytes(seqs, total, hq, hkv)
            st["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    return st


# ------------------------------------------------------------------- a pass, plain form
def _rotate(x, cos_sin, pairs):
    half = cos_sin.shape[1] // 2
    c, s = cos_sin[:, None, :half], cos_sin[:, None, half:]
    x = x.float()
    if pairs == "halves":
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * c - b * s, b * c + a * s], -1)
    else:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _codes(kv, dim, byte, part):
    """Codes [n][Hkv][16][dim] (fp32) and scales [n][Hkv] of records, part 0 = K, 1 = V."""
    codes = kv[..., 16 * dim * part:16 * dim * (part + 1)][..., byte].float() - 128
    scales = kv[..., 32 * dim:32 * dim + 8].contiguous().view(torch.float32)[..., part]
    return codes, scales


def _values(kv, dim, byte, part):
    codes, scales = _codes(kv, dim, byte, part)
    return codes * scales[:, :, None, None]


def _append8(kv, part, x, slots, touched, byte):
    """Rows x [T][Hkv][dim] (fp32) into the records `touched`: a block's scale covers the largest
    value it holds; when it grows, the codes before the new tokens are rounded to the new scale."""
    dim = x.shape[-1]
    rec = kv[touched.long()]
    codes, scale = _codes(rec, dim, byte, part)
    which = torch.searchsorted(touched.long(), slots // BS)
    n, hkv = scale.shape
    amax = torch.zeros((n, hkv), device=x.device)
    amax = amax.scatter_reduce(0, which[:, None].expand(-1, hkv), x.abs().amax(-1), "amax")
    first = torch.full((n,), BS, device=x.device)
    first = first.scatter_reduce(0, which, slots % BS, "amin")
    amax = torch.where(amax < 2.0 ** -100, 0.0, amax)
    old = torch.where(first[:, None] > 0, scale, 0.0)
    new = torch.maximum(old, amax * (1.0 / 127.0))
    grow = (new > old)[:, :, None, None]
    before = (torch.arange(BS, device=x.device) < first[:, None])[:, None, :, None]
    ratio = torch.where(new > 0, old / new, 0.0)[:, :, None, None]
    codes = torch.where(grow & before, torch.round(codes * ratio), codes)
    inverse = torch.where(new > 0, 1.0 / new, 0.0)
    codes[which, :, slots % BS] = torch.round(x * inverse[which][:, :, None]).clamp(-127, 127)
    flat = torch.empty((n, hkv, BS * dim), dtype=torch.uint8, device=x.device)
    flat[..., byte.reshape(-1)] = (codes + 128).to(torch.uint8).reshape(n, hkv, -1)
    rec[..., 16 * dim * part:16 * dim * (part + 1)] = flat
    at = 32 * dim + 4 * part
    rec[..., at:at + 4] = new[..., None].contiguous().view(torch.uint8)
    kv[touched.long()] = rec


def _run_append(st):
    case, n, dt = st["case"], st["tokens"], st["q"].dtype
    turns = st["cos_sin"][st["positions"][:n].long()]
    slots = st["slots"][:n]
    st["q_out"][:n] = _rotate(st["q"][:n], turns, case["pairs"]).to(dt)
    k = _rotate(st["k"][:n], turns, case["pairs"])
    if case["kind"] == "append":
        st["k_pool"][slots // BS, :, slots % BS] = k.to(dt)
        st["v_pool"][slots // BS, :, slots % BS] = st["v"][:n]
        return st["q_out"], st["k_pool"], st["v_pool"]
    touched = st["touched"]
    _append8(st["kv"], 0, k, slots, touched, st["byte"])
    _append8(st["kv"], 1, st["v"][:n].float(), slots, touched, st["byte"])
    st["k_out"].copy_(_values(st["kv"][touched.long()], case["dim"], st["byte"], 0))
    st["v_out"].copy_(_values(st["kv"][touched.long()], case["dim"], st["byte"], 1))
    return st["q_out"], st["k_out"], st["v_out"]


def _gather(st, j, part):
    """K (part 0) or V of positions j [S][n] as fp32 [S][n][Hkv][dim]."""
    block = torch.gather(st["tables"].long(), 1, j // BS).clamp(min=0)
    if "kv" not in st:
        return (st["v_pool"] if part else st["k_pool"])[block, :, j % BS].float()
    dim, kv = st["case"]["dim"], st["kv"]
    heads = torch.arange(kv.shape[1], device=kv.device)
    at = st["byte"][j % BS][:, :, None] + 16 * dim * part
    codes = kv[block[:, :, None, None], heads[:, None], at].float() - 128
    scales = kv[..., 32 * dim:32 * dim + 8].contiguous().view(torch.float32)[..., part]
    return codes * scales[block][..., None]


def _positions(st):
    """Visible positions [S][n] of each sequence's last token, and which of them count."""
    case, lens = st["case"], st["lens"].long()[:, None]
    if not case["window"]:
        j = torch.arange(case["len_hi"], device=DEV)[None, :].expand(case["seqs"], -1)
        return torch.minimum(j, lens - 1), j < lens
    sinks = torch.arange(case["sinks"], device=DEV)[None, :]
    low = (lens - case["window"]).clamp(min=0)
    wide = torch.arange(min(case["window"], case["len_hi"]), device=DEV)[None, :] + low
    j = torch.cat([sinks.expand(case["seqs"], -1), wide], 1)
    ok = torch.cat([sinks < torch.minimum(low, lens), wide < lens], 1)
    return torch.minimum(j, lens - 1), ok


def _run_decode(st):
    case = st["case"]
    hkv, dim = case["hkv"], case["dim"]
    j, ok = _positions(st)
    q = st["q"].float().view(case["seqs"], hkv, -1, dim)
    k = _gather(st, j, 0)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * st["scale"]
    x = x.masked_fill(~ok[:, None, None], -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    v = _gather(st, j, 1).masked_fill(~ok[:, :, None, None], 0.0)
    o = torch.matmul(p, v.transpose(1, 2)) / p.sum(-1, keepdim=True)
    return o.reshape(case["seqs"], -1, dim).to(st["q"].dtype)


def _run_prefill(st):
    case = st["case"]
    seqs, hq, hkv, dim = case["seqs"], case["hq"], case["hkv"], case["dim"]
    start, lens = st["query_start"].long(), st["lens"].long()
    most = case["new_hi"]
    i = torch.arange(most, device=DEV)
    row = (start[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
    pos = lens[:, None] - (start[1:] - start[:-1])[:, None] + i               # [S][C]
    j = torch.arange(case["prior"] + most, device=DEV)
    jj = torch.minimum(j[None], lens[:, None] - 1)
    q = st["q"].float()[row].view(seqs, most, hkv, hq // hkv, dim).permute(0, 2, 3, 1, 4)
    q = q.reshape(seqs, hkv, -1, dim)
    x = torch.matmul(q, _gather(st, jj, 0).permute(0, 2, 3, 1)) * st["scale"]
    x = x.view(seqs, hkv, hq // hkv, most, -1)
    see = (j <= pos[..., None]) & ((j > pos[..., None] - case["window"]) | (j < case["sinks"]))
    see = (see & (j < lens[:, None, None]))[:, None, None]
    x = x.masked_fill_(~see, -math.inf)
    p = torch.exp_(x.sub_(x.amax(-1, keepdim=True).clamp(min=-1e30)))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(seqs, hkv, -1, j.numel()), _gather(st, jj, 1).transpose(1, 2))
    o = o.view(seqs, hkv, -1, most, dim) / total
    t = torch.arange(st["q"].shape[0], device=DEV)
    s = torch.searchsorted(start, t, right=True) - 1
    return o.permute(0, 3, 1, 2, 4)[s, t - start[s]].reshape(-1, hq, dim).to(st["q"].dtype)


# ---------------------------------------------------------- a pass, the library's calls
def _run_own(st):
    import paged_kv_cache_146_gb300 as pkv
    case = st["case"]
    if case["kind"] in ("append", "append8"):
        eight = case["kind"] == "append8"
        pools = dict(kv=st["kv"]) if eight else dict(k_pool=st["k_pool"], v_pool=st["v_pool"])
        pkv.cache_write_rope(st["pool"], st["k"], st["v"], st["positions"], st["cos_sin"],
                             st["slots"], st["status"], q=st["q"], q_out=st["q_out"],
                             interleaved=case["pairs"] == "neighbours", **pools)
        if not eight:
            return st["q_out"], st["k_pool"], st["v_pool"]
        pkv.dequantize_blocks(st["pool"], st["touched"], st["k_out"], st["v_out"], st["status"],
                              kv=st["kv"])
        return st["q_out"], st["k_out"], st["v_out"]
    if case["kind"] == "decode8":
        return pkv.paged_decode_attention_b8(st["pool"], st["q"], st["tables"], st["lens"],
                                             st["scale"], st["status"],
                                             window=case["window"] or None, sinks=case["sinks"],
                                             out=st["out"], kv=st["kv"])
    if case["kind"] == "window":
        return pkv.paged_decode_attention_window(st["pool"], st["q"], st["tables"], st["lens"],
                                                 st["scale"], case["window"], case["sinks"],
                                                 st["status"], out=st["out"], k_pool=st["k_pool"],
                                                 v_pool=st["v_pool"])
    return pkv.paged_prefill_attention_window(st["pool"], st["q"], st["tables"], st["query_start"],
                                              st["lens"], st["scale"], case["window"],
                                              case["sinks"], st["workspace"], st["status"],
                                              out=st["out"], k_pool=st["k_pool"],
                                              v_pool=st["v_pool"])


def run(st):
    if own:
        return _run_own(st)
    kind = st["case"]["kind"]
    if kind in ("append", "append8"):
        return _run_append(st)
    return _run_prefill(st) if kind == "prefill" else _run_decode(st)


# ------------------------------------------------------------------- what a pass must do
def work(case):
    hq, hkv, dim, kind = case["hq"], case["hkv"], case["dim"], case["kind"]
    if kind in ("append", "append8"):
        t = sum(_news(case))
        ends = list(zip(_priors(case), _lens(case)))
        size = t * (2 * hq * dim * 2 + 2 * hkv * dim * 2 + case["rot"] * 4 + 12)
        if kind == "append":
            return {"bytes": size + t * 2 * hkv * dim * 2, "flops": 6 * t * (hq + hkv) * dim}
        blocks = sum(-(-n // BS) - p // BS for p, n in ends)
        # codes of the new tokens and the scales; then the blocks read back as 16-bit values
        size += t * 2 * hkv * dim + blocks * hkv * 16
        size += blocks * hkv * (32 * dim + 8 + 2 * BS * dim * 2)
        return {"bytes": size, "flops": 12 * t * (hq + hkv) * dim}
    lens, first = _lens(case), _first_query(case)
    pairs = keys = 0
    for n, q0 in zip(lens, first):
        if not case["window"]:
            pairs, keys = pairs + n, keys + n
            continue
        w, sinks = case["window"], case["sinks"]
        for p in range(q0, n):
            pairs += min(p + 1, w + min(sinks, max(0, p + 1 - w)))
        low = max(0, q0 - w + 1)
        keys += n - low + min(sinks, low)
    # 8-bit blocks also hold two fp32 scales per head
    per_key = 2 * hkv * dim + hkv / 2 if kind == "decode8" else 4 * hkv * dim
    rows = sum(_news(case)) if kind == "prefill" else case["seqs"]
    table = 4 * sum(len(v) for v in _visible_blocks(case))
    return {"bytes": keys * per_key + 2 * rows * hq * dim * 2 + table + 4 * case["seqs"],
            "flops": 4 * pairs * hq * dim}


# ------------------------------------------------------------------ results in 64 bits
def _exact_cache(st, part):
    """All blocks' K or V in 64 bits, [nb][Hkv][16][dim]; records are decoded byte by byte."""
    if "kv" not in st:
        return (st["v_pool"] if part else st["k_pool"]).double()
    dim, kv = st["case"]["dim"], st["kv"]
    scales = kv[:, :, 32 * dim + 4 * part:32 * dim + 4 * part + 4].contiguous().view(torch.float32)
    out = torch.empty((kv.shape[0], kv.shape[1], BS, dim), dtype=torch.float64, device=DEV)
    for t in range(BS):
        for c in range(dim // 16):
            place = c ^ (4 * (t % 2)) ^ (2 * (t // 2 % 4))
            at = 16 * dim * part + t * dim // 128 * 128 + 16 * place
            out[:, :, t, 16 * c:16 * c + 16] = kv[:, :, at:at + 16].double() - 128
    return out * scales.double()[..., None]


def _exact_rotation(x, pos, cos_sin, rot, pairs):
    y = x.double().clone()
    half = rot // 2
    i = torch.arange(half, device=DEV)
    one, two = (i, i + half) if pairs == "halves" else (2 * i, 2 * i + 1)
    c = cos_sin[pos][:, None, :half].double()
    s = cos_sin[pos][:, None, half:].double()
    a, b = x.double()[..., one], x.double()[..., two]
    y[..., one], y[..., two] = c * a - s * b, s * a + c * b
    return y


def _exact_append(case, st):
    n = st["tokens"]
    pos, slots = st["positions"][:n].long(), st["slots"][:n]
    q_out = st["q_out"].double()
    q_out[:n] = _exact_rotation(st["q"][:n], pos, st["cos_sin"], case["rot"], case["pairs"])
    k = _exact_rotation(st["k"][:n], pos, st["cos_sin"], case["rot"], case["pairs"])
    v = st["v"][:n].double()
    if case["kind"] == "append":
        pools = [st["k_pool"].double(), st["v_pool"].double()]
        for pool, rows in zip(pools, (k, v)):
            for h in range(case["hkv"]):
                pool[slots // BS, h, slots % BS] = rows[:, h]
        return (q_out, *pools)
    tokens_of = {}
    for t, slot in enumerate(slots.tolist()):
        tokens_of.setdefault(slot // BS, []).append((slot % BS, t))
    outs, dim = [], case["dim"]
    for part, rows in enumerate((k, v)):
        cache = _exact_cache(st, part)
        at = 32 * dim + 4 * part
        scales = st["kv"][:, :, at:at + 4].contiguous().view(torch.float32)[..., 0].double()
        blocks = []
        for b in st["touched"].tolist():
            offs, ts = zip(*tokens_of[b])
            first = min(offs)
            fresh = rows[list(ts)].transpose(0, 1)                        # [Hkv][n][dim]
            need = fresh.abs().amax((1, 2)) / 127
            old = scales[b] if first else torch.zeros_like(need)
            scale = torch.maximum(old, need)[:, None, None]
            codes = torch.round(cache[b] / scales[b][:, None, None])
            if first:
                earlier = torch.round(codes[:, :first] * (old[:, None, None] / scale))
                codes[:, :first] = torch.where(scale > old[:, None, None], earlier, codes[:, :first])
            codes[:, list(offs)] = torch.round(fresh / scale).clamp(-127, 127)
            blocks.append(codes * scale)
        outs.append(torch.stack(blocks))
    return (q_out, *outs)


def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] in ("append", "append8"):
        return _exact_append(case, st)
    hq, hkv, dim = case["hq"], case["hkv"], case["dim"]
    lens, first = _lens(case), _first_query(case)
    out, row = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV), 0
    for s, (n, q0) in enumerate(zip(lens, first)):
        rows = n - q0
        sees = torch.arange(n, device=DEV)
        if case["window"]:
            low = max(0, q0 - case["window"] + 1)
            sees = sees[(sees >= low) | (sees < case["sinks"])]
        blocks = st["tables"][s].long()[torch.unique(sees // BS)]
        place = torch.searchsorted(torch.unique(sees // BS), sees // BS)
        part = dict(st)
        for name in ("kv", "k_pool", "v_pool"):
            if name in st:
                part[name] = st[name][blocks]
        k, v = (_exact_cache(part, i)[place, :, sees % BS] for i in range(2))   # [n][Hkv][dim]
        at = torch.arange(q0, n, device=DEV)[:, None]
        hide = sees[None] > at
        if case["window"]:
            hide |= (sees[None] <= at - case["window"]) & (sees[None] >= case["sinks"])
        for h in range(hkv):
            q = st["q"][row:row + rows, h * (hq // hkv):(h + 1) * (hq // hkv)].double()
            x = (q @ k[:, h].T) * st["scale"]                                   # [rows][G][n]
            w = torch.softmax(x.masked_fill(hide[:, None], -math.inf), -1)
            out[row:row + rows, h * (hq // hkv):(h + 1) * (hq // hkv)] = w @ v[:, h]
        row += rows
    return out
