"""Windowed prefill with the workspace that the sizing call gives, and with room for an entry to every
query tile: the same result, whichever way the items are cut."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_cache_146_gb300 import (KVPool, PagedKVError, paged_prefill_attention,  # noqa: E402
                                      paged_prefill_attention_window, prefill_workspace_bytes, status_check)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seqs,chunk,hq", [(33, 1, 4), (40, 5, 16), (60, 17, 16), (60, 20, 12)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_item_lists_of_either_size(dtype, seqs, chunk, hq):
    """More sequences than a CTA lists for itself and few enough items for one query tile each."""
    dt = {"bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    gen = torch.Generator(device="cuda").manual_seed(seqs)
    nb, dim = 9, 64
    pool = KVPool(seqs * nb, 1, dim, dtype, device="cuda")
    for p in (pool.k_pool, pool.v_pool):
        p.copy_(torch.randn(p.shape, generator=gen, device="cuda"))
    tables = torch.arange(seqs * nb, dtype=torch.int32, device="cuda").view(seqs, nb)
    q = torch.randn((seqs * chunk, hq, dim), generator=gen, device="cuda").to(dt)
    lens = torch.randint(chunk, nb * 16 + 1, (seqs,), generator=gen, device="cuda", dtype=torch.int32)
    start = torch.arange(seqs + 1, dtype=torch.int32, device="cuda") * chunk
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    size = prefill_workspace_bytes(seqs, seqs * chunk, hq, 1)
    guard = 4096
    outs = []
    for room in (size, size + guard // 2):
        ws = torch.full((size + guard,), 0x5A, dtype=torch.uint8, device="cuda")
        outs.append(paged_prefill_attention_window(pool, q, tables, start, lens, 0.125, 50, 3, ws[:room],
                                                   status))
        assert (ws[room:] == 0x5A).all()
    # a window that hides nothing, against the plain call with the same workspace
    ws = torch.full((size + guard,), 0x5A, dtype=torch.uint8, device="cuda")
    wide = paged_prefill_attention_window(pool, q, tables, start, lens, 0.125, 10 ** 6, 0, ws[:size], status)
    plain = paged_prefill_attention(pool, q, tables, start, lens, 0.125, ws[:size], status)
    assert (ws[size:] == 0x5A).all() and status_check(status) == (0, 0)
    assert torch.equal(outs[0], outs[1])
    if dtype == "bf16":                      # (fp16: two parts of a weight against one)
        assert torch.equal(wide, plain)
    for call in (lambda: paged_prefill_attention_window(pool, q, tables, start, lens, 0.125, 50, 3,
                                                        ws[:size - 256], status),
                 lambda: paged_prefill_attention(pool, q, tables, start, lens, 0.125, ws[:size - 256], status)):
        with pytest.raises(PagedKVError):
            call()
