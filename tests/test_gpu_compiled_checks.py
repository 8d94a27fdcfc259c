"""The compiled argument checks (_fastcall) against the binding's own: the same
results bit for bit, and nothing called where a check does not hold."""
import pytest

torch = pytest.importorskip("torch")

import libbuild  # noqa: E402

libbuild.ensure_built()
import paged_kv_cache_146_gb300 as P  # noqa: E402

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32
NB, HKV, HQ, D, T, S = 24, 2, 8, 64, 5, 3


@pytest.fixture(scope="module")
def data():
    assert P._load_torch() and P._fast is not None, "_fastcall.so is not built"
    gen = torch.Generator(device="cuda").manual_seed(11)

    def rand(*shape):
        return torch.randn(*shape, device="cuda", generator=gen).to(BF)

    fused = rand(T, (HQ + 2 * HKV) * D)
    d = dict(
        q_rows=fused[:, :HQ * D].unflatten(1, (HQ, D)),
        k_rows=fused[:, HQ * D:(HQ + HKV) * D].unflatten(1, (HKV, D)),
        v_rows=fused[:, (HQ + HKV) * D:].unflatten(1, (HKV, D)),
        positions=torch.tensor([3, 40, 0, 7, 63], dtype=I32, device="cuda"),
        slots=torch.tensor([5, 17, -1, 300, 33], dtype=torch.int64, device="cuda"),
        table=P.rope_table(64, 32, device="cuda"),
        q=rand(S, HQ, D), pre=rand(T, HQ, D), k=rand(NB, HKV, 16, D), v=rand(NB, HKV, 16, D),
        tables=torch.arange(S * 4, dtype=I32, device="cuda").view(S, 4) + 1,
        lens=torch.tensor([0, 17, 64], dtype=I32, device="cuda"),
        starts=torch.tensor([0, 0, 1, T], dtype=I32, device="cuda"),
        ids=torch.tensor([2, 1, 9], dtype=I32, device="cuda"))
    return d


def pool16(d):
    p = P.KVPool(NB, HKV, D, "bf16", device="cuda")
    p.k_pool.copy_(d["k"])
    p.v_pool.copy_(d["v"])
    return p


def pool8(d):
    p = P.KVPool(NB, HKV, D, "b8_bf16", device="cuda")
    p.kv.zero_()
    slots = torch.arange(NB * 16, dtype=torch.int64, device="cuda")
    flat = [d[n].transpose(1, 2).reshape(NB * 16, HKV, D).contiguous() for n in ("k", "v")]
    P.cache_write_b8(p, *flat, slots, torch.zeros(1, dtype=I32, device="cuda"))
    return p


def call(name, d, stream=None):
    """One call of the framework on fresh pools; everything that it wrote."""
    status = torch.zeros(1, dtype=I32, device="cuda")
    window = dict(window=9, sinks=2, status=status, stream=stream)
    if name in ("append", "append b8"):
        pool = pool16(d) if name == "append" else pool8(d)
        torch.cuda.synchronize()
        q = P.cache_write_rope(pool, d["k_rows"], d["v_rows"], d["positions"], d["table"], d["slots"],
                               status, q=d["q_rows"], stream=stream,
                               q_out=torch.zeros(d["q_rows"].shape, dtype=BF, device="cuda"))
        torch.cuda.synchronize()
        return [q, status] + ([pool.kv] if pool.is_b8 else [pool.k_pool, pool.v_pool])
    if name == "append without queries":
        pool = pool16(d)
        torch.cuda.synchronize()
        assert P.cache_write_rope(pool, d["k_rows"], d["v_rows"], d["positions"], d["table"],
                                  d["slots"], status, interleaved=True, stream=stream) is None
        torch.cuda.synchronize()
        return [pool.k_pool, pool.v_pool, status]
    if name == "decode":
        pool = pool16(d)
        torch.cuda.synchronize()
        out = P.paged_decode_attention_window(pool, d["q"], d["tables"], d["lens"], 0.125, **window)
    elif name == "decode b8":
        pool = pool8(d)
        torch.cuda.synchronize()
        out = P.paged_decode_attention_b8(pool, d["q"], d["tables"], d["lens"], 0.125, **window)
    elif name == "prefill":
        pool = pool16(d)
        ws = torch.empty(P.prefill_workspace_bytes(S, T, HQ, HKV), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        out = P.paged_prefill_attention_window(pool, d["pre"], d["tables"], d["starts"], d["lens"],
                                               0.125, 9, 2, ws, status, stream=stream)
    else:
        pool = pool8(d)
        out = tuple(torch.zeros(len(d["ids"]), HKV, 16, D, dtype=BF, device="cuda") for _ in "kv")
        torch.cuda.synchronize()
        P.dequantize_blocks(pool, d["ids"], *out, status, stream=stream)
    torch.cuda.synchronize()
    return [*(out if isinstance(out, tuple) else (out,)), status]


CALLS = ("append", "append b8", "append without queries", "decode", "decode b8", "prefill",
         "dequantize")


class Counted:
    """_fastcall with the answers of its calls noted."""

    def __init__(self, fast):
        self._fast, self.answers = fast, []

    def __getattr__(self, name):
        fn = getattr(self._fast, name)

        def noted(*args):
            self.answers.append(fn(*args))
            return self.answers[-1]
        return noted


@pytest.mark.parametrize("name", CALLS)
def test_both_checks_make_the_same_call(name, data, monkeypatch):
    counted = Counted(P._fast)
    monkeypatch.setattr(P, "_fast", counted)
    fast = call(name, data)
    side = torch.cuda.Stream()
    on_object, on_handle = call(name, data, side), call(name, data, side.cuda_stream)
    assert counted.answers == [0, 0, 0]
    monkeypatch.setattr(P, "_fast", None)
    own = call(name, data)
    for other in (fast, on_object, on_handle):
        assert len(other) == len(own)
        for a, b in zip(other, own):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("name,key,change,error", [
    ("decode", "q", lambda t: t.float(), TypeError),
    ("decode", "q", lambda t: t[:, :3], ValueError),
    ("decode", "q", lambda t: t.cpu(), ValueError),
    ("decode", "tables", lambda t: t.t().contiguous().t(), ValueError),
    ("decode", "tables", lambda t: t[:2], ValueError),
    ("decode", "lens", lambda t: t.long(), TypeError),
    ("decode", "lens", lambda t: t.cpu(), ValueError),
    ("decode b8", "lens", lambda t: t[:2], ValueError),
    ("decode b8", "tables", lambda t: t.long(), TypeError),
    ("prefill", "starts", lambda t: t[:3], ValueError),
    ("prefill", "pre", lambda t: t.half(), TypeError),
    ("append", "k_rows", lambda t: t.transpose(0, 1).contiguous().transpose(0, 1), ValueError),
    ("append", "v_rows", lambda t: t[:4], ValueError),
    ("append", "q_rows", lambda t: t[..., :32], ValueError),
    ("append", "positions", lambda t: t.long(), TypeError),
    ("append", "table", lambda t: t.double(), TypeError),
    ("append", "slots", lambda t: t.int(), TypeError),
    ("append b8", "slots", lambda t: t.repeat_interleave(2)[::2], ValueError),
    ("dequantize", "ids", lambda t: t.long(), TypeError),
    ("dequantize", "ids", lambda t: t.repeat_interleave(2)[::2], ValueError)])
def test_a_check_that_fails_is_named_by_the_binding(name, key, change, error, data, monkeypatch):
    counted = Counted(P._fast)
    monkeypatch.setattr(P, "_fast", counted)
    bad = dict(data, **{key: change(data[key])})
    with pytest.raises(error) as first:
        call(name, bad)
    assert counted.answers == [None]
    monkeypatch.setattr(P, "_fast", None)
    with pytest.raises(error) as second:
        call(name, bad)
    assert str(first.value) == str(second.value)


def test_errors_of_the_library_are_raised(data, monkeypatch):
    counted = Counted(P._fast)
    monkeypatch.setattr(P, "_fast", counted)
    with pytest.raises(P.PagedKVError):
        call("append", dict(data, table=data["table"][:, :24].contiguous()))
    assert len(counted.answers) == 1 and counted.answers[0] not in (0, None)


def test_a_closed_pool_is_refused(data):
    pool = pool16(data)
    pool.close()
    status = torch.zeros(1, dtype=I32, device="cuda")
    with pytest.raises(Exception):
        P.paged_decode_attention_window(pool, data["q"], data["tables"], data["lens"], 0.125, 9, 2,
                                        status)


def test_threads_and_streams(data):
    """Calls from several threads at once, each on its own stream and pool."""
    import threading
    want = call("decode", data)[0]
    pool, got, errors = pool16(data), [None] * 4, []
    torch.cuda.synchronize()

    def work(i):
        try:
            status = torch.zeros(1, dtype=I32, device="cuda")
            stream = torch.cuda.Stream()
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                for _ in range(50):
                    got[i] = P.paged_decode_attention_window(pool, data["q"], data["tables"],
                                                             data["lens"], 0.125, 9, 2, status)
            stream.synchronize()
        except Exception as e:                       # shown by the assertion below
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for out in got:
        assert torch.equal(out, want)
