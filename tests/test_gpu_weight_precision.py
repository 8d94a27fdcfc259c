"""How precisely the attention calls carry a softmax weight into the product with V."""
import math

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_cache_146_gb300 import (KVPool, paged_decode_attention_b8,  # noqa: E402
                                      paged_decode_attention_window, paged_prefill_attention_window,
                                      prefill_workspace_bytes, status_check)
from serving_reference import Records  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
HKV, NB = 2, 6                               # the pool is one sequence of 96 tokens


def cancelling(kind, dim, c0, c1):
    """A pool whose even tokens have score 0 and value c0 / 64, the odd ones a score of -scale and
    the value -c1 / 64; with a window of two and scale = ln(c1 / c0) they cancel."""
    pool = KVPool(NB, HKV, dim, kind, device="cuda")
    if pool.is_b8:
        r = Records(NB, HKV, dim)
        r.scales[:] = 2.0 ** -6
        r.codes[0, :, :, 1::2, 0] = -64
        r.codes[1, :, :, 0::2], r.codes[1, :, :, 1::2] = c0, -c1
        pool.kv.copy_(torch.from_numpy(r.to_bytes()))
    else:
        pool.k_pool.zero_()
        pool.k_pool[:, :, 1::2, 0] = -1
        pool.v_pool[:, :, 0::2], pool.v_pool[:, :, 1::2] = c0 / 64, -c1 / 64
    return pool


def query(rows, hq, dim, dt):
    q = torch.zeros((rows, hq, dim), dtype=dt, device="cuda")
    q[..., 0] = 1
    return q


def check(out, c0, c1, scale, weight):
    """The error of a weight is at most `weight` (its way into the product) + 2^-22 (exp2) + 2^-23
    (its argument: the scale's product with log2 e) + 2^-22 (joining two warps' sums); the sums of
    up to three products and the quotient add 5 2^-24; in all 2^-20 beside `weight`.  The result's
    rounding is of a value near zero."""
    w = math.exp(-float(torch.tensor(scale, dtype=torch.float32)))
    room = (c0 / 64) * (weight + 2.0 ** -20) / (1 + w)
    want = (c0 - w * c1) / 64 / (1 + w)
    half = torch.finfo(out.dtype).eps / 2
    tiny = torch.finfo(out.dtype).smallest_normal * torch.finfo(out.dtype).eps / 2
    worst = (out.double().cpu() - want).abs().max().item()
    assert worst <= room + half * (abs(want) + room) + tiny, (c0, c1, worst / room)


RATIOS = [(64 + i, 127 - i // 3) for i in range(0, 60, 4)]


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("hq", [4, 24])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_8bit_decode(dtype, dim, hq):
    """Two fp16 parts: 2^-22."""
    lens = torch.arange(2, 96, dtype=torch.int32, device="cuda")
    tables = torch.arange(NB, dtype=torch.int32, device="cuda").repeat(len(lens), 1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for c0, c1 in RATIOS:
        pool = cancelling("b8_" + dtype, dim, c0, c1)
        scale = math.log(c1 / c0)
        out = paged_decode_attention_b8(pool, query(len(lens), hq, dim, DT[dtype]), tables, lens, scale,
                                        status, window=2)
        check(out, c0, c1, scale, 2.0 ** -22)
    assert status_check(status) == (0, 0)


@pytest.mark.parametrize("dim,hq", [(64, 4), (128, 8), (128, 24)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_16bit_decode(dtype, dim, hq):
    """Three bf16 parts (half a step is 2^-8, so 2^-24) or two fp16 parts (2^-22)."""
    lens = torch.arange(2, 96, dtype=torch.int32, device="cuda")
    tables = torch.arange(NB, dtype=torch.int32, device="cuda").repeat(len(lens), 1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for c0, c1 in RATIOS:
        pool = cancelling(dtype, dim, c0, c1)
        scale = math.log(c1 / c0)
        out = paged_decode_attention_window(pool, query(len(lens), hq, dim, DT[dtype]), tables, lens, scale,
                                            2, 0, status)
        check(out, c0, c1, scale, 2.0 ** -24 if dtype == "bf16" else 2.0 ** -22)
    assert status_check(status) == (0, 0)


def prefill(pool, q, tables, lens, scale, window):
    """One chunk a sequence, of equal size."""
    seqs, rows, hq = len(lens), q.shape[0], q.shape[1]
    start = torch.arange(seqs + 1, dtype=torch.int32, device="cuda") * (rows // seqs)
    ws = torch.empty(prefill_workspace_bytes(seqs, rows, hq, HKV), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = paged_prefill_attention_window(pool, q, tables, start, lens, scale, window, 0, ws, status)
    assert status_check(status) == (0, 0)
    return out


@pytest.mark.parametrize("dim,hq", [(64, 2), (64, 8), (128, 8), (128, 24)])
@pytest.mark.parametrize("seqs", [1, 70])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_prefill(dtype, seqs, dim, hq):
    """Two parts: in bf16 the first truncated (2^-7) and the remainder rounded (2^-8), 2^-15, the
    causal call's own; in fp16 both rounded, 2^-22."""
    lens = torch.full((seqs,), 96, dtype=torch.int32, device="cuda")
    tables = torch.arange(NB, dtype=torch.int32, device="cuda").repeat(seqs, 1)
    for c0, c1 in RATIOS:
        pool = cancelling(dtype, dim, c0, c1)
        scale = math.log(c1 / c0)
        out = prefill(pool, query(seqs * 95, hq, dim, DT[dtype]), tables, lens, scale, 2)
        check(out, c0, c1, scale, 2.0 ** -15 if dtype == "bf16" else 2.0 ** -22)


# ------------------------------------------------------------- a few dominant tokens
def dominated(kind, dim, n, first):
    """A pool of one sequence of n tokens: the first ones have score 0 and value 0, the others a
    score of -1 times the scale and the value 1."""
    nb = -(-n // 16)
    pool = KVPool(nb, HKV, dim, kind, device="cuda")
    late = (torch.arange(nb * 16) >= first).view(nb, 1, 16)
    if pool.is_b8:
        r = Records(nb, HKV, dim)
        r.scales[:] = 2.0 ** -6
        r.codes[0, :, :, :, 0] = torch.where(late, -64, 0).numpy()
        r.codes[1] = torch.where(late, 64, 0)[..., None].numpy()
        pool.kv.copy_(torch.from_numpy(r.to_bytes()))
    else:
        pool.k_pool.zero_()
        pool.k_pool[..., 0] = torch.where(late, -1.0, 0.0).to(pool.k_pool)
        pool.v_pool.copy_(torch.where(late, 1.0, 0.0)[..., None].expand_as(pool.v_pool))
    return pool, nb


def check_dominated(out, n, first, bits, scale, weight, late):
    """n - first equal weights of 2^-bits against one.  Numerator and denominator are off by the
    error of a weight (`weight` and 2^-20, see `check`), the numerator also by what fp16 cannot
    hold of the late weights (`late`: with the largest weight 2^8 and a step of 2^-24 at the
    small end, 2^-25 2^-8 2^bits) and by the sums' own error (some hundred additions a warp:
    2^-16)."""
    w = math.exp(-float(torch.tensor(scale, dtype=torch.float32))) * (n - first)
    want = w / (first + w)
    rel = 2 * (weight + 2.0 ** -20) + late + 2.0 ** -16 + torch.finfo(out.dtype).eps / 2
    worst = (out.double().cpu() / want - 1).abs().max().item()
    assert worst <= rel, (bits, worst / rel)


@pytest.mark.parametrize("kind,dim,hq", [("bf16", 128, 8), ("f16", 64, 4), ("f16", 128, 24), ("b8_bf16", 128, 8),
                                         ("b8_f16", 64, 24)])
@pytest.mark.parametrize("n", [1000, 24000])
def test_decode_far_below_a_few_tokens(kind, dim, hq, n):
    """The dominant tokens sit among the late ones' blocks of one warp, and alone in others'."""
    dt = DT[kind.split("_")[-1]]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    pool, nb = dominated(kind, dim, n, 1)
    tables = torch.arange(nb, dtype=torch.int32, device="cuda").view(1, nb)
    for bits in (19.0, 20.37, 21.5, 22.0):
        scale = bits * math.log(2.0)
        q = query(1, hq, dim, dt)
        if pool.is_b8:
            out = paged_decode_attention_b8(pool, q, tables, lens, scale, status)
        else:
            out = paged_decode_attention_window(pool, q, tables, lens, scale, n, 0, status)
        half = kind != "bf16"                        # weights become fp16
        check_dominated(out, n, 1, bits, scale, 2.0 ** -22 if half else 2.0 ** -24,
                        2.0 ** (bits - 33) if half else 0.0)
    assert status_check(status) == (0, 0)


@pytest.mark.parametrize("dim,hq", [(64, 4), (128, 8), (128, 24)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n,rows", [(1000, 60), (6000, 300)])
def test_prefill_far_below_a_few_tokens(dtype, dim, hq, n, rows):
    """A row has one reference for all its keys, so a dominant sink stands against every late one.
    With the largest weight 2^7, what fp16 cannot hold of a weight of 2^-bits is 2^-25 2^-7 2^bits of
    it; sums of n products in order round to n 2^-24 at worst, most of it in the same direction."""
    pool, nb = dominated(dtype, dim, n, 1)
    tables = torch.arange(nb, dtype=torch.int32, device="cuda").view(1, nb)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    for bits in (18.0, 19.37, 20.5, 21.0):
        scale = bits * math.log(2.0)
        out = prefill(pool, query(rows, hq, dim, DT[dtype]), tables, lens, scale, n)
        w = math.exp(-float(torch.tensor(scale, dtype=torch.float32)))
        late = torch.arange(n - rows, n, dtype=torch.float64) * w      # the query itself is late
        want = (late / (1 + late))[:, None, None]
        rel = (2 * ((2.0 ** -22 if dtype == "f16" else 2.0 ** -15) + 2.0 ** -20) + n * 2.0 ** -24
               + (2.0 ** (bits - 32) if dtype == "f16" else 0.0) + torch.finfo(DT[dtype]).eps / 2)
        # (an output of 2^-11 and up is a normal number of either type)
        worst = (out.double().cpu() / want - 1).abs().max().item()
        assert worst <= rel, (bits, worst / rel)
