"""Bounded waits of the kernel of drafted trees, read from its source: a wait that runs out (or is
told to stop) ends for all lanes of a warp at once.  Running into one on a GPU would hang it."""
import os
import re

SOURCE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "paged_kv_cache_146_gb300", "csrc",
                      "paged_tree.cu")


def statements(text):
    text = re.sub(r"//[^\n]*", "", text)
    return [" ".join(s.split()) for s in re.split(r"[;{}]", text)]


def test_every_wait_is_voted_on():
    """Each lane polls the barrier, the stop flag and the clock by itself, so lanes may disagree; the
    answer counts only once the warp has voted, in the same statement or the next one."""
    with open(SOURCE) as f:
        code = statements(f.read())
    waits = [i for i, s in enumerate(code) if "mbar_wait(" in s]
    assert waits
    for i in waits:
        voted = re.search(r"__all_sync\(kFull, mbar_wait\(", code[i])
        assigned = re.search(r"\bok = mbar_wait\(", code[i]) and code[i + 1] == "ok = __all_sync(kFull, ok)"
        assert voted or assigned, code[i]


def test_no_barrier_is_polled_without_a_limit():
    """`mbar_try_wait` stands in loops that look at the clock."""
    with open(SOURCE) as f:
        code = statements(f.read())
    polls = [i for i, s in enumerate(code) if "mbar_try_wait(" in s]
    for i in polls:
        assert "while" in code[i] and any("kTimeoutNs" in s for s in code[i:i + 3]), code[i]


def test_a_cta_that_gives_up_leaves_nothing_to_join():
    """The joining kernel goes by what every CTA left in the workspace, so one that ends without a plan
    leaves an empty range there, after the kernels before it have ended."""
    with open(SOURCE) as f:
        code = statements(f.read())
    start = next(i for i, s in enumerate(code) if "& 1023u" in s)
    end = next(i for i in range(start, len(code)) if code[i] == "return")
    waited = code.index("griddep_wait()", start, end)
    assert any(s.startswith("p.ranges[blockIdx.x] = make_int4(0, 0, 0, 0)") for s in code[waited:end])


def test_warps_without_rows_take_every_phase():
    """A barrier tells even phases from odd ones only.  A softmax warp that has no rows, and waits only
    for the last product of an item, could take the end of the last but two for it; so it waits for each
    tile's, as the others do."""
    with open(SOURCE) as f:
        code = statements(f.read())
    start = next(i for i, s in enumerate(code) if s.startswith("if (!busy)") or s == "if (!busy)")
    end = code.index("continue", start)
    assert any("reach(&o_full[b ^ 1u], ((kt - 1) >> 1) & 1u)" in s for s in code[start:end])
