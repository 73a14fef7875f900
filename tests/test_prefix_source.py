"""What the kernels of shared pages and shared prefixes promise in an order that no run can show:
read from their sources."""
import os
import re

import pytest

import block_sparse_long_quest_gb300 as kt

CSRC = os.path.join(os.path.dirname(kt.__file__), "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())  # without comments


def kernels(name):
    """(name, body) of every kernel of a file."""
    text = source(name)
    for m in re.finditer(r"__global__", text):
        at = text.index("{", m.start())
        head = text[m.start():at]
        yield re.findall(r"(\w+)\(const __grid_constant__", head)[0], text[at:text.index("\n}\n", at)]


# members of the parameters that point to what an earlier kernel may have written
POINTERS = r"\bp\.(q|k_scale|v_scale|table|seq_lens|cu|prefix|out|status|head|items_a|items_b|cost_a|" \
           r"cost_b|q_rows|seqs|parts|stats|lens|blocks|refs|list|list2|a|b|moves|num_moves|new_table|" \
           r"new_refs|base)\b"


@pytest.mark.parametrize("name", ["pages.cu", "prefix.cu"])
def test_nothing_is_read_before_the_wait(name):
    """These kernels start before the one ahead of them has ended; what that one and its predecessors
    have written is visible behind the kernel's own wait only."""
    found = list(kernels(name))
    assert len(found) == {"pages.cu": 5, "prefix.cu": 3}[name]
    for kernel, body in found:
        before = body[:body.index("griddep_wait();")]
        assert not re.search(POINTERS, before), kernel
        assert "load_" not in before and "__ldcg" not in before, kernel


def attend_body():
    return dict(kernels("prefix.cu"))["attend_kernel"]


def test_probabilities_are_stored_again_behind_a_wait():
    """Stores to tensor memory are asynchronous and not ordered among themselves: a row's second pass
    waits for those of the first one, whose columns it writes again."""
    loop = attend_body()
    loop = loop[loop.index("for (int round = 0;; ++round)"):]
    loop = loop[:loop.index("if (round > 0) break;")]
    wait = loop.index("if (round > 0) tmem_wait_st();")
    assert wait < loop.index("row_exp<") and "row_exp<" not in loop[:wait]


def test_every_arrival_of_the_rows_is_behind_a_fence():
    """The tensor cores write columns that row warps have read: each path to an arrival on p_full goes
    through a fence for the warp's own loads and stores of tensor memory."""
    body = attend_body()
    arrivals = [m.start() for m in re.finditer(r"mbar_arrive\(p_full", body)]
    assert len(arrivals) == 2
    for at, since in zip(arrivals, ("if (quarter < q0", "tmem_wait_st();\n        tc_fence")):
        begin = body.rindex(since, 0, at)
        assert "tc_fence_before();" in body[begin:at]
        assert not re.search(r"tmem_ld|row_exp|row_max", body[begin:at])


def test_a_cache_is_prepared_by_itself():
    """Whether the registers that the compiler took suffice is asked of the kernel that is launched,
    as an inequality (its bounds are static assertions beside it)."""
    text = source("prefix.cu")
    launch = text[text.index("cudaError_t launch_prefix("):]
    assert "a.k_scale ? prepare<true>() : prepare<false>()" in launch
    assert "attr.numRegs !=" not in text and "registers_ok(attr.numRegs)" in text


def test_the_simulated_barriers_have_the_kernels_sizes():
    """test_prefix_barriers models the rings, the runs and who arrives on what: sizes and counts of
    arrivals are those of the source."""
    import random

    import test_prefix_barriers as sim
    text = source("prefix.cu")
    value = lambda name: int(re.search(r"constexpr int %s = (\d+);" % name, text)[1])  # noqa: E731
    assert value("UNITS") == sim.UNITS and value("STEPS_AHEAD") == sim.STEPS_AHEAD
    assert value("SLOTS") == 2 and value("SOFT_WARPS") == 8
    for f8 in (0, 1):
        k = sim.Kernel(random.Random(1), [1], (128, 1), [[], []], bool(f8))
        for name, n in (("entries", k.entries), ("codes", k.codes)):
            assert int(re.search(r"%s = F8 \? (\d+) : (\d+);" % name, text)[2 - f8]) == n
        init = dict(re.findall(r"mbar_init\((\w+) \+ 8 \* i, ([^)]+)\);", text))
        count = {"empty": "2", "full": "F8 ? 4 : 1", "code_full": "1", "code_empty": "4", "s_full": "1",
                 "p_full": "SOFT_WARPS / SLOTS", "o_full": "1", "q_full": "1", "q_done": "1"}
        assert init == count
        bars = dict(empty=k.empty, full=k.full[0], code_full=k.code_full, code_empty=k.code_empty,
                    s_full=k.s_full, p_full=k.p_full, o_full=k.o_full, q_full=k.q_full[0],
                    q_done=k.q_done[0])
        for name, c in count.items():
            want = {"F8 ? 4 : 1": 4 if f8 else 1, "SOFT_WARPS / SLOTS": 4}.get(c) or int(c)
            assert all(b.count == want for b in bars[name]), name
