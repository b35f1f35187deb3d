"""Every kernel of the row operators waits for the launch before it, whatever its grid,
before it reads or writes global memory: only what the launch before it (and all that
that one waited for) wrote is then visible to it.

Read off the sources: a missing wait shows on a GPU only where the timing is right for it."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "tile_size_decision_gb300", "csrc")
FILES = ["route_sm103a.cu", "layernorm_sm103a.cu", "clip_sm103a.cu", "norm_sm103a.cu", "row_ops.cuh"]


def text_of(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def closing(text, at):
    """Where the brace that opens at `at` is closed."""
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == "{") - (text[i] == "}")
        if depth == 0:
            return i
    raise AssertionError("an open brace")


def kernels(text):
    """Name, parameters and body of every kernel."""
    for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\([^\n]*\)\s+)?(\w+)\(([^)]*)\)\s*\{", text):
        open_at = m.end() - 1
        yield m[1], m[2], text[open_at + 1:closing(text, open_at)]


def pointer_fields(text, struct):
    m = re.search(r"struct (?:alignas\(\d+\) )?%s\s*\{" % struct, text)
    return re.findall(r"\*\s*(\w+)\s*;", text[m.end():closing(text, m.end() - 1)]) if m else []


def before_the_wait(body):
    """What a kernel does before it has waited: up to the first wait that stands as a
    statement of its own in the outermost block."""
    for m in re.finditer(r"ptx::grid_dependency_wait\(\);", body):
        ahead = body[:m.start()]
        if ahead.count("{") == ahead.count("}") and re.search(r"[;{}]\s*$|^\s*$", ahead):
            return ahead
    return body


ALL = [(f, *k) for f in FILES for k in kernels(text_of(f))]


def test_the_kernels_are_found():
    names = [k[1] for k in ALL]
    assert len(names) >= 20 and len(set(names)) == len(names)
    assert {"sort_place_kernel", "layernorm_odd_ring_kernel", "scale_kernel", "rmsnorm_grad_kernel",
            "reduce_partials_kernel"} <= set(names)


@pytest.mark.parametrize("file,name,params,body", ALL, ids=[k[1] for k in ALL])
def test_a_kernel_waits_before_it_touches_memory(file, name, params, body):
    ahead = before_the_wait(body)
    assert ahead != body, "no wait on every path"
    text = text_of("row_ops.cuh") + text_of(file)
    for kind, arg in re.findall(r"(\w+)(?:<\w+>)?[\s&]+(\w+)\s*(?:,|$)", params):
        if kind in ("int", "float", "int64_t"):
            continue
        for field in pointer_fields(text, kind):
            assert not re.search(r"\b%s\.%s\b" % (arg, field), ahead), field
        # The arguments handed on whole: the function may read anything.
        assert not re.search(r"[(,]\s*%s\s*[,)]" % arg, ahead), arg
    for arg in re.findall(r"\*\s*(\w+)", params):
        assert not re.search(r"\b%s\b" % arg, ahead), arg
