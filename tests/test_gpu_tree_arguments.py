"""Arguments of the calls for trees of drafted tokens that lie elsewhere than they should: strided
ones and ones of the host are refused by name, offset ones are taken."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import libbuild  # noqa: E402
import paged_kv_cache_146_gb300 as P  # noqa: E402
from serving_reference import assert_within, scale_of  # noqa: E402
from tree_reference import TreeCase, mask_words  # noqa: E402

libbuild.ensure_built()
pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def arguments():
    c = TreeCase([70, 3], [12, 40], 8, 2, 128, torch.bfloat16, 4)
    c.k.nan_to_num_()
    c.v.nan_to_num_()
    pool = P.KVPool(c.nb, 2, 128, "bf16", device="cuda")
    pool.k_pool.copy_(c.k)
    pool.v_pool.copy_(c.v)
    ws = torch.empty(P.tree_workspace_bytes(c.rows, 8, 2, 128), dtype=torch.uint8, device="cuda")
    tokens = torch.arange(c.rows, device="cuda") % 2
    return c, pool, {
        "tree": dict(q=c.q.cuda(), block_tables=c.tables.cuda(), query_start=ints(c.starts),
                     context_lens=ints(c.lens), tree_mask=mask_words(c.masks, c.words).cuda(), workspace=ws,
                     out=torch.empty(c.q.shape, dtype=torch.bfloat16, device="cuda")),
        "accept": dict(tokens=tokens, parents=ints([x for p in c.parents for x in p]), targets=tokens.flip(0),
                       query_start=ints(c.starts), first=ints(c.priors), kept=ints([0] * c.rows),
                       num_kept=ints([0, 0]), next_tokens=tokens[:2].clone()),
        "compact": dict(block_tables=c.tables.cuda(), kept=ints([70, 73, 3, 9]), kept_start=ints([0, 2, 4]),
                        num_kept=ints([2, 2]), first=ints(c.priors))}


def call(name, pool, args, status):
    if name == "tree":
        return P.paged_tree_attention(pool, scale=scale_of(128), status=status, **args)
    if name == "accept":
        return P.tree_accept(status=status, **args)
    return P.cache_compact(pool, status=status, **args)


NAMES = [(n, a) for n, names in (
    ("tree", "q block_tables query_start context_lens tree_mask out"),
    ("accept", "tokens parents targets query_start first kept num_kept next_tokens"),
    ("compact", "block_tables kept kept_start num_kept first")) for a in names.split()]


@pytest.mark.parametrize("compiled", [True, False])
@pytest.mark.parametrize("name,arg", NAMES)
def test_strided_and_host_tensors_are_refused(name, arg, compiled, monkeypatch):
    assert P._load_torch()
    if not compiled:
        monkeypatch.setattr(P, "_fast", None)
    _, pool, args = arguments()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = pool.k_pool.clone()
    t = args[name][arg]
    apart = torch.stack([t, t], -1)[..., 0]      # every other element
    assert apart.shape == t.shape and not apart.is_contiguous()
    for bad in (apart, t.cpu()):
        with pytest.raises(ValueError):
            call(name, pool, dict(args[name], **{arg: bad}), status)
    torch.cuda.synchronize()
    assert status.item() == 0 and torch.equal(pool.k_pool, before)


def test_offset_tensors_are_taken():
    """Tensors that begin inside another one: 4-byte offsets of the lists, 16-byte ones of the rows."""
    c, pool, args = arguments()

    def inside(t, lead):
        whole = torch.zeros(t.numel() + lead, dtype=t.dtype, device="cuda")
        whole[lead:] = t.reshape(-1)
        return whole[lead:].view(t.shape)

    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    tree = {k: v if k == "workspace" else inside(v, 8 if k in ("q", "out") else 1) for k, v in args["tree"].items()}
    got = call("tree", pool, tree, status)
    assert P.status_check(status) == (0, 0)
    for s in range(2):
        assert_within(got[c.starts[s]:c.starts[s + 1]], *c.expect(s, scale_of(128)), f"sequence {s}")
    plain = call("accept", pool, args["accept"], status)
    other = call("accept", pool, {k: inside(v, 1) for k, v in args["accept"].items()}, status)
    assert P.status_check(status) == (0, 0)
    for a, b in zip(plain, other):
        assert torch.equal(a, b)


def test_a_token_that_stays_needs_no_block():
    """Only tokens that move are looked up: blocks outside the pool are reported for them alone."""
    _, pool, args = arguments()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = pool.k_pool.clone()
    args = args["compact"]
    args["block_tables"][:] = -1
    args["kept"], args["first"] = ints([16, 17, 5, 6]), ints([16, 5])
    call("compact", pool, args, status)
    assert P.status_check(status) == (0, 0)
    args["kept"] = ints([16, 18, 5, 6])
    call("compact", pool, args, status)
    assert P.status_check(status)[1] == P.DEV_BAD_BLOCK and torch.equal(pool.k_pool, before)
