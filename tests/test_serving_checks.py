"""Refusals of the rotated append, the block-scaled 8-bit calls and the windowed
calls: nothing of them reaches a GPU, so they run on the CPU; and the plain 64-bit
forms that the GPU tests compare with, against themselves."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import libbuild  # noqa: E402
from paged_kv_cache_146_gb300 import (KVPool, PagedKVError, _native, cache_write, cache_write_b8,  # noqa: E402
                                      cache_write_q8, cache_write_rope, dequantize_blocks,
                                      gather_blocks, kv_pool_bytes, paged_decode_attention,
                                      paged_decode_attention_b8, paged_decode_attention_window,
                                      paged_prefill_attention_window, rope_table)
from serving_reference import Records, rotate, rotate_f32  # noqa: E402

lib = libbuild.ensure_built()
BF = torch.bfloat16
_kept = []


def handle(pool):
    """The ledger's handle, kept alive to the end of the run."""
    _kept.append(pool)
    return pool.handle


def pool16(dim=64):
    p = KVPool(8, 2, dim, "bf16")
    p.k_pool = torch.zeros((8, 2, 16, dim), dtype=BF)
    p.v_pool = torch.zeros((8, 2, 16, dim), dtype=BF)
    return p


def pool8(dim=64):
    p = KVPool(8, 2, dim, "b8_bf16")
    p.kv = torch.zeros((8, 2, 32 * dim + 32), dtype=torch.uint8)
    return p


def append_args(T=3):
    return dict(k_new=torch.zeros((T, 2, 64), dtype=BF), v_new=torch.zeros((T, 2, 64), dtype=BF),
                positions=torch.zeros(T, dtype=torch.int32), cos_sin=rope_table(4, 32),
                slot_mapping=torch.zeros(T, dtype=torch.int64), status=torch.zeros(1, dtype=torch.int32),
                q=torch.zeros((T, 4, 64), dtype=BF))


@pytest.mark.parametrize("change,error,match", [
    (dict(k_new=torch.zeros((3, 2, 32), dtype=BF)), ValueError, r"k_new must be \[3, 2, 64\]"),
    (dict(k_new=torch.zeros((3, 2, 64))), TypeError, "k_new must be bfloat16"),
    (dict(v_new=torch.zeros((2, 2, 64), dtype=BF)), ValueError, "v_new must be"),
    (dict(v_new=torch.zeros((2, 3, 64), dtype=BF).transpose(0, 1)), ValueError, "heads of a token"),
    (dict(k_new=torch.zeros((1, 2, 64), dtype=BF).expand(3, 2, 64)), ValueError, "token stride"),
    (dict(k_new=torch.zeros((3, 132), dtype=BF)[:, :128].view(3, 2, 64)), ValueError, "token stride"),
    (dict(q=torch.zeros((3, 4, 32), dtype=BF)), ValueError, "q must be"),
    (dict(q=torch.zeros((3, 256), dtype=BF)), ValueError, "q must be"),
    (dict(q=None, q_out=torch.zeros((3, 4, 64), dtype=BF)), ValueError, "q_out without q"),
    (dict(q_out=torch.zeros((3, 2, 64), dtype=BF)), ValueError, "q_out must be"),
    (dict(positions=torch.zeros(3, dtype=torch.int64)), TypeError, "positions must be int32"),
    (dict(positions=torch.zeros(2, dtype=torch.int32)), ValueError, "positions must be"),
    (dict(slot_mapping=torch.zeros(3, dtype=torch.int32)), TypeError, "slot_mapping must be int64"),
    (dict(slot_mapping=torch.zeros((3, 1), dtype=torch.int64)), ValueError, "slot_mapping must be"),
    (dict(cos_sin=torch.zeros((4, 32), dtype=torch.float64)), TypeError, "cos_sin must be float32"),
    (dict(cos_sin=torch.zeros(32)), ValueError, "cos_sin must be"),
    (dict(cos_sin=torch.zeros((4, 64))[:, :32]), ValueError, "cos_sin must be contiguous"),
    (dict(status=torch.zeros(1)), TypeError, "status must be an int32"),
    (dict(k_pool=torch.zeros((8, 2, 16, 32), dtype=BF)), ValueError, "k_pool must be"),
    (dict(), ValueError, "must be CUDA tensors"),
])
def test_append_refusals(change, error, match):
    args = append_args()
    args.update(change)
    with pytest.raises(error, match=match):
        cache_write_rope(pool16(), **args)


def test_append_refuses_overlapping_queries():
    buf = torch.zeros((3, 512), dtype=BF)
    args = append_args()
    args.update(q=buf[:, :256].view(3, 4, 64), q_out=buf.view(-1)[:768].view(3, 4, 64))
    with pytest.raises(ValueError, match="same token stride"):
        cache_write_rope(pool16(), **args)


def test_append_takes_no_pool_with_a_scale_per_32_values():
    p = KVPool(8, 2, 128, "q8_bf16")
    T = 3
    args = append_args()
    for name, h in (("k_new", 2), ("v_new", 2), ("q", 4)):
        args[name] = torch.zeros((T, h, 128), dtype=BF)
    with pytest.raises(ValueError, match="16-bit and block-scaled"):
        cache_write_rope(p, **args)


@pytest.mark.parametrize("rot,rows,code", [(8, 4, -1), (0, 4, -1), (128, 4, -1), (24, 4, -8), (32, 0, -1)])
def test_append_table_shapes_in_the_library(rot, rows, code):
    """The library's own checks, with addresses that are never read."""
    p = pool16()
    a = ctypes.c_void_p(4096)
    rc = lib.kv_cache_write_rope(p.handle, a, 256, a, 256, 4, a, 128, a, 128, a, a, rows, rot, 0, a, 3, a, a,
                                 a, None)
    assert rc == code


@pytest.mark.parametrize("name,args", [
    ("stride", (0, 0, 0, 0, 0, 4096, 127, 4096, 128)), ("odd stride", (0, 0, 0, 0, 0, 4096, 132, 4096, 128)),
    ("alignment", (0, 0, 0, 0, 0, 4104, 128, 4096, 128)), ("no q_out", (0, 0, 4096, 256, 4, 4096, 128, 4096, 128)),
    ("q heads", (0, 0, 0, 0, -1, 4096, 128, 4096, 128))])
def test_append_rows_in_the_library(name, args):
    qo, qos, q, qs, hq, k, ks, v, vs = args
    a = 4096
    rc = lib.kv_cache_write_rope(handle(pool16()), qo, qos, q, qs, hq, k, ks, v, vs, a, a, 4, 32, 0, a, 3, a, a, a,
                                 None)
    assert rc == -1, name


def test_b8_refusals():
    p, rows = pool8(), torch.zeros((3, 2, 64), dtype=BF)
    slots, status = torch.zeros(3, dtype=torch.int64), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="block-scaled"):
        cache_write_b8(pool16(), rows, rows, slots, status)
    with pytest.raises(ValueError, match="k_new must be contiguous"):
        cache_write_b8(p, torch.zeros((3, 256), dtype=BF)[:, :128].view(3, 2, 64), rows, slots, status)
    with pytest.raises(ValueError, match="kv must be"):
        cache_write_b8(p, rows, rows, slots, status, kv=p.kv[:7])
    with pytest.raises(ValueError, match="CUDA tensors"):
        cache_write_b8(p, rows, rows, slots, status)
    out = torch.zeros((2, 2, 16, 64), dtype=BF)
    with pytest.raises(ValueError, match="block-scaled"):
        dequantize_blocks(pool16(), torch.zeros(2, dtype=torch.int32), out, out, status)
    with pytest.raises(TypeError, match="ids must be int32"):
        dequantize_blocks(p, torch.zeros(2, dtype=torch.int64), out, out, status)
    with pytest.raises(ValueError, match="v_out must be"):
        dequantize_blocks(p, torch.zeros(2, dtype=torch.int32), out, out[:1], status)
    with pytest.raises(ValueError, match="staging holds fewer"):
        gather_blocks(p, torch.zeros(2, dtype=torch.int32), torch.zeros(2080 * 3, dtype=torch.uint8), status)
    # the calls for the other pools take none of these records
    with pytest.raises(PagedKVError, match="INVALID_ARG"):
        _native.check(lib.kv_cache_write(p.handle, 4096, 4096, 4096, 3, 4096, 4096, 4096, None))
    with pytest.raises(PagedKVError, match="INVALID_ARG"):
        _native.check(lib.kv_cache_write_q8(p.handle, 4096, 4096, 4096, 3, 4096, 4096, None))
    for call in (cache_write, cache_write_q8):
        with pytest.raises((ValueError, TypeError, AttributeError)):
            call(p, rows, rows, slots, status)


def test_b8_sizes():
    assert kv_pool_bytes(10, 16, 3, 128, "b8_bf16") == 10 * 3 * 4128
    assert kv_pool_bytes(10, 16, 3, 64, "b8_f16") == 10 * 3 * 2080
    assert kv_pool_bytes(10, 16, 3, 96, "b8_f16") == 0 and kv_pool_bytes(10, 8, 3, 64, "b8_f16") == 0
    assert KVPool(4, 2, 128, "b8_f16").record_bytes == 4128
    odd = KVPool(4, 2, 96, "b8_f16")
    assert lib.kv_cache_write_b8(odd.handle, 4096, 4096, 4096, 3, 4096, 4096, None) == -8
    assert lib.kv_dequantize_blocks(odd.handle, 4096, 1, 4096, 4096, 4096, 4096, None) == -8
    assert lib.paged_decode_attention_b8(odd.handle, 4096, 4096, 4096, 4096, 4, 4096, 1, 4, 0.1, 0, 0, 4096, None) == -8


def attention_args(S=2, hq=4, dim=64):
    return (torch.zeros((S, hq, dim), dtype=BF), torch.zeros((S, 3), dtype=torch.int32),
            torch.ones(S, dtype=torch.int32))


@pytest.mark.parametrize("window,sinks", [(0, 0), (-1, 0), (4, -1), (2 ** 31, 0), (4, 2 ** 31)])
def test_window_ranges(window, sinks):
    q, tables, lens = attention_args()
    status = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="window >= 1"):
        paged_decode_attention_window(pool16(), q, tables, lens, 0.1, window, sinks, status)
    with pytest.raises(ValueError, match="window >= 1"):
        paged_decode_attention_b8(pool8(), q, tables, lens, 0.1, status, window=window, sinks=sinks)
    with pytest.raises(ValueError, match="window >= 1"):
        paged_prefill_attention_window(pool16(), q, tables, torch.zeros(3, dtype=torch.int32), lens, 0.1,
                                       window, sinks, torch.zeros(4096, dtype=torch.uint8), status)
    if window < 2 ** 31 and sinks < 2 ** 31:
        assert lib.paged_decode_attention_window(handle(pool16()), 4096, 4096, 4096, 4096, 4096, 3, 4096, 2, 4, 0.1,
                                                 window, sinks, 4096, None) == -1


@pytest.mark.parametrize("which", ["window", "b8", "prefill"])
def test_attention_refusals(which):
    status = torch.zeros(1, dtype=torch.int32)
    ws = torch.zeros(4096, dtype=torch.uint8)
    start = torch.tensor([0, 1, 2], dtype=torch.int32)

    def call(q, tables, lens, out=None, pool=None):
        if which == "window":
            return paged_decode_attention_window(pool or pool16(), q, tables, lens, 0.1, 8, 2, status, out=out)
        if which == "b8":
            return paged_decode_attention_b8(pool or pool8(), q, tables, lens, 0.1, status, out=out)
        return paged_prefill_attention_window(pool or pool16(), q, tables, start, lens, 0.1, 8, 2, ws, status,
                                              out=out)

    q, tables, lens = attention_args()
    with pytest.raises(ValueError, match=r"q must be \[n\]\[h\]\[64\]"):
        call(q[..., :32].contiguous(), tables, lens)
    with pytest.raises(ValueError, match="not a multiple"):
        call(q[:, :3].contiguous(), tables, lens)
    with pytest.raises(ValueError, match="q must be contiguous"):
        call(torch.zeros((2, 64, 4), dtype=BF).transpose(1, 2), tables, lens)
    with pytest.raises(TypeError, match="q must be bfloat16"):
        call(q.half(), tables, lens)
    with pytest.raises(ValueError, match="out must be"):
        call(q, tables, lens, out=q[:1])
    with pytest.raises(TypeError, match="block_tables must be int32"):
        call(q, tables.long(), lens)
    with pytest.raises(ValueError, match="context_lens must be"):
        call(q, tables, lens[:1])
    with pytest.raises(ValueError, match="16-bit pool|block-scaled"):
        call(q, tables, lens, pool=pool16() if which == "b8" else pool8())
    with pytest.raises(ValueError, match="CUDA tensors"):
        call(q, tables, lens)
    if which == "b8":
        with pytest.raises(ValueError, match="sinks without a window"):
            paged_decode_attention_b8(pool8(), q, tables, lens, 0.1, status, sinks=2)


def test_attention_shapes_in_the_library():
    p = pool16()
    a = 4096
    call = lib.paged_decode_attention_window
    assert call(p.handle, a, a, a, a, a, 3, a, 2, 34, 0.1, 8, 0, a, None) == -8         # G = 17
    assert call(p.handle, a, a, a, a, a, 3, a, 2, 5, 0.1, 8, 0, a, None) == -1          # heads
    assert call(p.handle, a, a, a, a, a, 0, a, 2, 4, 0.1, 8, 0, a, None) == -1          # table width
    assert call(p.handle, a, a, a, a, a, 3, a, 2, 4, float("nan"), 8, 0, a, None) == -1
    assert call(p.handle, a, 4104, a, a, a, 3, a, 2, 4, 0.1, 8, 0, a, None) == -1       # alignment
    assert call(p.handle, a, None, a, a, a, 3, a, 2, 4, 0.1, 8, 0, a, None) == -1
    assert call(p.handle, a, a, a, a, a, 3, a, 0, 4, 0.1, 8, 0, a, None) == 0           # no sequences
    assert call(p.handle, a, a, a, a, a, 2 ** 30, a, 2, 4, 0.1, 8, 0, a, None) == -8    # lengths past 32 bits
    assert call(handle(pool8()), a, a, a, a, a, 3, a, 2, 4, 0.1, 8, 0, a, None) == -1
    assert call(handle(KVPool(8, 2, 96, "bf16")), a, a, a, a, a, 3, a, 2, 4, 0.1, 8, 0, a, None) == -8
    assert call(handle(KVPool(8, 2, 64, "bf16", block_size=8)), a, a, a, a, a, 3, a, 2, 4, 0.1, 8, 0, a, None) == -8
    q8 = lib.paged_decode_attention_b8
    assert q8(p.handle, a, a, a, a, 3, a, 2, 4, 0.1, 0, 0, a, None) == -1
    assert q8(handle(pool8()), a, a, a, a, 3, a, 2, 4, 0.1, -1, 0, a, None) == -1
    assert q8(handle(pool8()), a, a, a, a, 3, a, 0, 4, 0.1, 0, 0, a, None) == 0


def test_existing_decode_refuses_the_records():
    q, tables, lens = attention_args()
    status, ws = torch.zeros(1, dtype=torch.int32), torch.zeros(1 << 16, dtype=torch.uint8)
    with pytest.raises((ValueError, PagedKVError)):
        paged_decode_attention(pool8(), q, tables, lens, 0.1, ws, status)


# ------------------------------------------------------------- the plain forms
def test_record_bytes_round_trip():
    rng = np.random.default_rng(0)
    for dim in (64, 128):
        r = Records(3, 2, dim)
        r.codes[:] = rng.integers(-127, 128, r.codes.shape)
        r.scales[:] = rng.random(r.scales.shape)
        back = Records.from_bytes(r.to_bytes())
        assert np.array_equal(back.codes, r.codes) and np.array_equal(back.scales, r.scales)
        # the chunk rule covers every byte of a slab once
        assert len({(t * dim // 128 * 128 + 16 * (j ^ (4 * (t % 2)) ^ (2 * (t // 2 % 4))))
                    for t in range(16) for j in range(dim // 16)}) == dim


def test_plain_append_keeps_values_within_half_a_step():
    rng = np.random.default_rng(1)
    r = Records(2, 1, 64)
    rows = rng.standard_normal((16, 1, 64)).astype(np.float32)
    r.append(0, rows, np.arange(16))
    err = np.abs(r.values(0)[0, 0] - rows[:, 0].astype(np.float64)).max()
    assert err <= 0.5 * r.scales[0, 0, 0] * (1 + 2.0 ** -14)
    assert r.scales[0, 0, 0] == np.float32(np.abs(rows).max() * np.float32(1 / 127))


@pytest.mark.parametrize("interleaved", [False, True])
def test_plain_rotation_turns_by_the_angle(interleaved):
    table = rope_table(9, 32)
    x = torch.randn((9, 2, 64), generator=torch.Generator().manual_seed(0)).double()
    y, _ = rotate(x, table, torch.arange(9), interleaved)
    assert torch.allclose(y[..., :32].norm(dim=-1), x[..., :32].norm(dim=-1), rtol=1e-6)
    assert torch.equal(y[..., 32:], x[..., 32:]) and torch.equal(y[0], x[0])
    # scores depend on the distance alone
    a, b = x[:1].expand(9, 2, 64), x[1:2].expand(9, 2, 64)
    ra, _ = rotate(a.clone(), table, torch.arange(9), interleaved)
    rb, _ = rotate(b.clone(), table, torch.arange(9), interleaved)
    d = [(ra[i] * rb[j]).sum() for i, j in ((2, 0), (5, 3), (8, 6))]
    assert max(d) - min(d) < 1e-5
    z = rotate_f32(x.float().numpy(), table, np.arange(9), interleaved)
    assert np.abs(z - y.numpy()).max() < 1e-6
