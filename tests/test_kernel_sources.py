"""Rules that the kernels' inline assembly keeps, checked in the sources: what the
compiler may do to a statement shows in no run of the build at hand."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_quantized_mixture_b200", "csrc")


def statements():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))):
        with open(path) as f:
            text = f.read()
        for m in re.finditer(r"\basm(\s+volatile)?\s*\((.*?)\)\s*;", text, re.S):
            code = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', m.group(2)))
            yield f"{os.path.basename(path)}:{text.count(chr(10), 0, m.start()) + 1}", bool(m.group(1)), code


def test_there_are_statements():
    assert len(list(statements())) > 50


def test_collectives_are_volatile():
    """A collective that names lanes in a mask must stay where it is written: moved
    into a branch that some of them do not take, it would wait for them."""
    found = [(at, code) for at, volatile, code in statements() if re.search(r"\.sync\b|barrier\.|\bbar\.", code) and not volatile]
    assert not found


def test_tensor_memory_loads_end_with_their_wait():
    """The load writes its registers until the wait; as a statement of its own, the
    wait would not keep what reads them behind it."""
    found = [(at, code) for at, _, code in statements() if "tcgen05.ld" in code and "tcgen05.wait::ld" not in code.split("tcgen05.ld")[-1]]
    assert not found
