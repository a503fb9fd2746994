"""Kernels launched early (programmatic dependent launch, launch_next) wait for
the kernel before them, unconditionally and before they touch memory: read from
the sources, as no run shows it reliably."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_moe_layer_expert_b200", "csrc")


def text(path):
    with open(path) as f:
        return re.sub(r"//[^\n]*", "", f.read())


SOURCES = {os.path.basename(p): text(p) for p in sorted(glob.glob(os.path.join(CSRC, "*.cu")))}
EARLY = sorted({(f, k) for f, s in SOURCES.items() for k in re.findall(r"launch_next\(\s*(\w+)", s)})


def body(src, name):
    """The braces of the function definition `name`, and what stands in its parameter list."""
    for m in re.finditer(r"\b%s\s*\(" % name, src):
        depth, i = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(src[i], 0)
            i += 1
        params = src[m.end():i - 1]
        j = i
        while src[j].isspace():
            j += 1
        if src[j] != "{":
            continue
        depth, k = 1, j + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(src[k], 0)
            k += 1
        return params, src[j + 1:k - 1]
    raise AssertionError(name)


MEMORY = r"tma_load_\dd|bulk_load|ld_\w+\(|\ba\.off\[|\bpart\[|__ldcg|reinterpret_cast<const (float|int)4"


def waits_first(src, name):
    params, b = body(src, name)
    if "predecessor_done" not in b:  # a kernel that hands over to a function for its share: each of them waits
        called = re.findall(r"\b(\w+_pair)\(", b)
        assert called, f"{name} never waits"
        return [r for c in set(called) for r in waits_first(src, c)]
    at = b.index("predecessor_done")
    # at the top level of the body, not under a condition
    head = b[:at]
    assert head.count("{") == head.count("}"), f"{name} waits inside a block"
    assert not re.search(r"\b(if|else)\b[^;{}]*$", head), f"{name} waits under a condition"
    assert not re.search(MEMORY, re.sub(r"\[&\][^{]*\{.*?\};", "", head, flags=re.S)), f"{name} reads before it waits"
    return [(name, params, b)]


def test_there_are_some():
    assert {k for _, k in EARLY} >= {"norm_dw_join_kernel", "balance_join_kernel", "dwr_join_kernel", "router_dx_kernel",
                                     "router_dwr_kernel"}


@pytest.mark.parametrize("file,kernel", EARLY)
def test_early_kernels_wait(file, kernel):
    waits_first(SOURCES[file], kernel)


@pytest.mark.parametrize("file,kernel", EARLY)
def test_early_kernels_do_not_read_as_if_read_only(file, kernel):
    """Their inputs are written while they are already under way."""
    for name, params, b in waits_first(SOURCES[file], kernel):
        assert not re.search(r"const [^,]*__restrict__", params), name
        assert "__ldg(" not in b, name
