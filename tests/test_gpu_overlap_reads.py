"""A read-back right behind an append sees the codes and scales that the append left,
although both may be set up while the calls before them run: the same bits as with a
synchronisation after every call."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import libbuild  # noqa: E402

libbuild.ensure_built()
import paged_kv_cache_146_gb300 as P  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("blocks,hkv", [(1, 1), (12, 2), (90, 8)])
@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("f16", 64)])
def test_read_back_between_appends(dtype, dim, blocks, hkv):
    """Token after token goes to every block, each larger than the one before, so that every
    append raises every scale; the whole pool is read back before and after each."""
    dt = {"bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    gen = torch.Generator(device="cuda").manual_seed(blocks)
    rows = [torch.randn((blocks, hkv, dim), generator=gen, device="cuda").to(dt) * (1.3 ** t)
            for t in range(16)]
    table = P.rope_table(16, dim, device="cuda")
    ids = torch.arange(blocks, dtype=torch.int32, device="cuda")
    slots = [torch.arange(blocks, device="cuda") * 16 + t for t in range(16)]
    pos = [torch.full((blocks,), t, dtype=torch.int32, device="cuda") for t in range(16)]

    def run(sync):
        pool = P.KVPool(blocks, hkv, dim, "b8_" + dtype, device="cuda")
        pool.kv.zero_()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        back = [torch.empty((2, blocks, hkv, 16, dim), device="cuda", dtype=dt) for _ in range(32)]
        torch.cuda.synchronize()
        for t in range(16):
            for k, after in enumerate((False, True)):
                if after:
                    P.cache_write_rope(pool, rows[t], rows[t], pos[t], table, slots[t], status)
                    sync()
                P.dequantize_blocks(pool, ids, *back[2 * t + k], status)
                sync()
        torch.cuda.synchronize()
        assert status.item() == 0
        return back

    want = run(torch.cuda.synchronize)
    assert want[-1].abs().sum() > 0
    for _ in range(4):
        assert all(torch.equal(a, b) for a, b in zip(run(lambda: None), want))
