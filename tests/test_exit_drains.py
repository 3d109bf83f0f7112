"""No arrival may be in flight to a thread block that has left: the next block on the
SM keeps its own barriers at the same addresses. Every mbarrier that a tensor-core commit
arrives on is therefore drained in the kernel that commits to it, read here from the
sources: that the MMAs of a commit have retired does not say that the arrivals of
earlier commits, on other barriers, have landed.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weight_only_int4_gb300", "csrc")


def kernels(name):
    """(name, body) of the kernels of a source file, comments taken out."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    for part in re.split(r"\b__global__\b", text)[1:]:
        yield re.search(r"\b(\w+_kernel)\s*\(", part).group(1), part


def barriers(args, before):
    """Barriers that the arguments of a call name, themselves or by a variable, last defined in the code before it."""
    found = set(re.findall(r"bars->(\w+)", args))
    for variable in re.findall(r"\b[a-z]\w*\b", args):
        definitions = re.findall(r"\b%s\s*=\s*(smem_u32\([^;]*?bars->[^;]*?)[,;]\s" % variable, before)
        if definitions:
            found.add(re.search(r"bars->(\w+)", definitions[-1]).group(1))
    return found


def calls(function, body):
    """Arguments of the calls of a function whose name starts so, and the code before each."""
    for m in re.finditer(r"\b%s\w*\(" % function, body):
        depth, at = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(body[at], 0)
            at += 1
        yield body[m.end():at - 1], body[:m.start()]


def committed_and_drained(body):
    committed = set().union(*(barriers(*a) for a in calls("umma_commit", body)))
    drained = set().union(*(barriers(*a) for a in calls("drain_ring", body)))
    return committed, drained


@pytest.mark.parametrize("source,names", [("int8_matmul.cu", {"tiles_kernel", "pair_kernel"}),
                                          ("mx_matmul.cu", {"rows_kernel", "pair_kernel"}),
                                          ("gemm.cu", {"gemm_kernel"}), ("gemm_skinny.cu", {"gemm_skinny_kernel"})])
def test_stages(source, names):
    seen = set()
    for name, body in kernels(source):
        committed, drained = committed_and_drained(body)
        if not committed:
            continue
        seen.add(name)
        assert {"drain", "tfull"} < committed
        assert committed <= drained, (name, committed - drained)
    assert seen == names


def test_every_source_that_commits():
    named = {n for n in os.listdir(CSRC) if n.endswith(".cu") and "umma_commit" in open(os.path.join(CSRC, n)).read()}
    assert named == {"int8_matmul.cu", "mx_matmul.cu", "gemm.cu", "gemm_skinny.cu"}
