"""Which kernels are launched with programmatic stream serialization, read from
the sources: the decode GEMV and the few-row GEMM alone. A queue that had the
attribute on the MXFP4 quantisation and on the product's cluster kernel stopped
making progress, so none of the kernels that take quantised activations or
experts has it, nor asks for an early start of the kernel after it."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weight_only_int4_gb300", "csrc")
PROGRAMMATIC = {"gemv.cu", "gemm_skinny.cu"}


def code(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(CSRC) if f.endswith(".cu")))
def test_programmatic_launches(name):
    found = re.findall(r"cudaLaunchAttributeProgrammatic\w+|griddep_\w+", code(name))
    assert bool(found) == (name in PROGRAMMATIC), (name, found)
