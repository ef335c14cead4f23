"""Rules of the kernels that may be launched with programmatic serialization, read from their sources (a race cannot be
shown by a test that is sure to meet it)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gemm_uq_gb300", "csrc")


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())                    # without comments


def _kernels(name):
    """{name: source from the kernel's name to the end of its body} of the __global__ functions of a file."""
    text, out = _source(name), {}
    for m in re.finditer(r"__global__\s+void[^;{]*?\b(\w+_kernel)\s*\(", text):
        depth, i = 0, text.index("{", m.end())
        for j in range(i, len(text)):
            depth += (text[j] == "{") - (text[j] == "}")
            if depth == 0:
                break
        out[m.group(1)] = text[m.start():j + 1]
    return out


EARLY = [("uq_mx_quant.cu", "quantize_mx_kernel"), ("uq_mx_gemm.cu", "mx_gemm_kernel"), ("uq_mx_gemm.cu", "mx_gemm_pair_kernel")]


def test_the_early_kernels_are_all():
    """Every kernel of the microscaled and routing sources that waits for its predecessor is in the list above."""
    waits = {(f, k) for f in ("uq_mx_quant.cu", "uq_mx_gemm.cu", "uq_moe.cu") for k, body in _kernels(f).items()
             if "griddepcontrol.wait" in body or "after_prior_work" in body}
    assert waits == set(EARLY)


@pytest.mark.parametrize("file,kernel", EARLY)
def test_no_read_only_loads_of_what_a_predecessor_may_write(file, kernel):
    """Such a kernel is resident while the one before still writes its inputs: no load of them may take the read-only
    path, which __ldg asks for and const __restrict__ pointers allow."""
    body = _kernels(file)[kernel]
    assert "__ldg(" not in body and "__restrict__" not in body
    for shared in ("uq_mx.cuh", "uq_mx_quant.cuh", "uq_mx_gemm.cu"):
        parts = _source(shared)
        for k in _kernels(shared).values():
            parts = parts.replace(k, "")
        assert "__ldg(" not in parts and "__restrict__" not in parts, shared


@pytest.mark.parametrize("kernel", [k for f, k in EARLY if f == "uq_mx_gemm.cu"])
def test_products_let_dependents_go_after_their_own_wait(kernel):
    """The next kernel requests its weights before it waits, so it may start only once all work before this product is
    complete: the trigger follows the product's wait, in the same warp."""
    text, trigger = _source("uq_mx_gemm.cu"), "griddepcontrol.launch_dependents"
    assert text.count(trigger) == 1 and trigger not in _kernels("uq_mx_gemm.cu")[kernel]
    helper = text[text.index("void launch_dependents("):]
    helper = helper[:helper.index("}")]
    assert 0 <= helper.find("after_prior_work(a);") < helper.index(trigger)
    assert _kernels("uq_mx_gemm.cu")[kernel].count("launch_dependents(a)") == 1


def test_only_a_products_own_quantizer_lets_dependents_go():
    body = _kernels("uq_mx_quant.cu")["quantize_mx_kernel"]
    assert body.count("griddepcontrol.launch_dependents") == 1
    assert re.search(r"if \(early\) asm volatile\(\"griddepcontrol\.launch_dependents;", body)
