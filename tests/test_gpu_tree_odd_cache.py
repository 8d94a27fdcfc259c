"""Infinities and NaN in V of the tokens before the drafted ones, which every row sees."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import libbuild  # noqa: E402
from paged_kv_cache_146_gb300 import (KVPool, paged_tree_attention, status_check,  # noqa: E402
                                      tree_workspace_bytes)
from tree_reference import TreeCase, mask_words  # noqa: E402

libbuild.ensure_built()
pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def call(c, name, scale):
    pool = KVPool(c.nb, c.hkv, c.dim, name, device="cuda")
    pool.k_pool.copy_(c.k)
    pool.v_pool.copy_(c.v)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(tree_workspace_bytes(c.rows, c.hq, c.hkv, c.dim), dtype=torch.uint8, device="cuda")
    got = paged_tree_attention(pool, c.q.cuda(), c.tables.cuda(),
                               torch.tensor(c.starts, dtype=torch.int32, device="cuda"),
                               torch.tensor(c.lens, dtype=torch.int32, device="cuda"),
                               mask_words(c.masks, c.words).cuda(), scale, ws, status)
    assert status_check(status) == (0, 0)
    return got.float().cpu()


def put(c, s, pos, d, value):
    c.v[c.tables[s, pos // 16].long(), :, pos % 16, d] = value


@pytest.mark.parametrize("name,dim", [("bf16", 128), ("f16", 128), ("bf16", 64), ("f16", 64)])
@pytest.mark.parametrize("prior", [192, 2000, 40000])
def test_an_infinity_of_the_cache(name, dim, prior):
    """One in each dimension, of another token each, of ordinary weights: the row's result is that
    infinity in every dimension, whatever the weights' last bits."""
    c = TreeCase([prior, 70], [7, 40], 8, 2, dim, DT[name], prior)
    gen = torch.Generator().manual_seed(prior)
    signs = torch.randint(0, 2, (dim,), generator=gen) * 2 - 1
    at = torch.randint(0, prior, (dim,), generator=gen)
    at[:64], at[-1] = torch.arange(64), prior - 1
    for d in range(dim):
        put(c, 0, int(at[d]), d, float("inf") * int(signs[d]))
    got = call(c, name, 0.02)                    # scores within +-1: weights within 2^-3 of each other
    assert torch.equal(got[:7], (signs * float("inf")).expand(7, 8, dim))
    assert bool(got[7:].isfinite().all())


@pytest.mark.parametrize("name", ["bf16", "f16"])
@pytest.mark.parametrize("pos", [0, 63, 64, 500, 699])
def test_an_infinity_of_the_token_that_weighs_most(name, pos):
    """Its weight is one, which the first part holds; others weigh down to 2^-7 of it."""
    c = TreeCase([700], [5], 8, 2, 128, DT[name], 3)
    c.q = torch.zeros_like(c.q)
    c.q[..., 0] = 1.0
    c.k[..., 0] = torch.rand(c.k[..., 0].shape, generator=c.gen).to(c.k)
    c.k[c.tables[0, pos // 16].long(), :, pos % 16, 0] = 2.0
    clean = call(c, name, 2.0)                   # e^-4 = 2^-5.8 at least
    put(c, 0, pos, 3, float("inf"))
    put(c, 0, pos, 9, -float("inf"))
    put(c, 0, (pos + 100) % 700, 20, float("inf"))
    put(c, 0, (pos + 300) % 700, 21, float("nan"))
    got = call(c, name, 2.0)
    assert bool((got[..., 3] == float("inf")).all()) and bool((got[..., 9] == -float("inf")).all())
    assert bool((got[..., 20] == float("inf")).all()) and bool(got[..., 21].isnan().all())
    rest = torch.ones(128, dtype=torch.bool)
    rest[[3, 9, 20, 21]] = False
    assert torch.equal(got[..., rest], clean[..., rest])


@pytest.mark.parametrize("name", ["bf16", "f16"])
def test_two_infinities_of_unlike_signs(name):
    c = TreeCase([300], [3], 4, 1, 64, DT[name], 4)
    put(c, 0, 10, 5, float("inf"))
    put(c, 0, 200, 5, -float("inf"))
    put(c, 0, 10, 6, float("inf"))
    put(c, 0, 200, 6, float("inf"))
    got = call(c, name, 0.02)
    assert bool(got[..., 5].isnan().all()) and bool((got[..., 6] == float("inf")).all())
