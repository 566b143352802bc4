"""Kernels that start while the one before them ends (programmatic dependent
launch): an input may be read only after griddep_wait, and a load may be moved
by the compiler (CUDA's cache-hinted bf16 load is no volatile statement) unless
its pointer has come through after_wait.  The sources of the gated delta rule
and of the group norm are read for it (CPU)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(__file__), "..", "delta_rule_linear_dpfp_gb300", "csrc")
FILES = sorted(os.path.basename(f) for p in ("fw_gated*.cu", "fw_group_norm.cu") for f in glob.glob(os.path.join(CSRC, p)))


def functions(text):
    """(name, parameters, body) of the device functions that wait for the kernel before."""
    for m in re.finditer(r"\n(?:__global__|FW_DEV) void(?: __launch_bounds__\([^\n]*\))?\s+(\w+)\(([^{};]*)\) \{\n(.*?)\n\}\n", text, re.S):
        if "griddep_wait()" in m[3]:
            yield m[1], m[2], m[3]


def unordered(text):
    """Inputs that such a function names and does not pass through after_wait behind its first wait."""
    found = []
    for name, params, body in functions(text):
        start, rest = body.split("griddep_wait()", 1)
        for p in re.findall(r"const (?:T|float|bf|__nv_bfloat16) \*__restrict__ (\w+)", params):
            early = re.sub(r"l2_prefetch\([^;]*;|//[^\n]*", "", start)
            if re.search(rf"after_wait\({p}\)", rest) is None or re.search(rf"(?<![.\w]){p}\b(?! *=)", early):
                found.append((name, p))
    return found


def test_the_functions_are_found():
    names = {n for f in FILES for n, _, _ in functions(open(os.path.join(CSRC, f)).read())}
    assert names >= {"gated_prep_kernel", "gated_walk_kernel", "gated_reverse_kernel", "gated_grad_kernel", "gated_tc_prep_kernel",
                     "walk", "gated_tc_grad_kernel", "gated_decode_kernel", "group_norm_kernel", "group_norm_backward_kernel"}


@pytest.mark.parametrize("name", FILES)
def test_inputs_are_read_behind_the_wait(name):
    assert unordered(open(os.path.join(CSRC, name)).read()) == []


def test_lengths_too():
    text = open(os.path.join(CSRC, "fw_gated_tiles.cuh")).read()
    assert "__ldcg(after_wait(a.lengths) + b)" in text


def test_a_missing_one_is_seen():
    text = "\n__global__ void kern(const T *__restrict__ x, const T *__restrict__ y) {\n    griddep_wait();\n    y = after_wait(y);\n}\n"
    assert unordered(text) == [("kern", "x")]
