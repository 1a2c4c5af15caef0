"""The order of the operators' kernels, read from their source (no GPU).

They are launched before the kernels ahead of them have ended (programmatic dependent launch), and PTX makes
what those wrote visible only to a kernel that waits itself.  So every kernel waits, on every path, and none lets
the next one in before it has.
"""
import os
import re

import pytest

import zero_sharded_mixed_03_gb300 as Z

CSRC = os.path.join(os.path.dirname(os.path.abspath(Z.__file__)), "csrc")
FILES = ("zero_linear.cu", "zero_norm.cu", "zero_adamw.cu")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def kernels(text):
    """(name, body) of every __global__ function."""
    for m in re.finditer(r"__global__", text):
        at = text.index("{", m.end())
        name = re.findall(r"(\w+)\s*\(", re.sub(r"__launch_bounds__\(.*?\)\s*(?=\w)|__cluster_dims__\(.*?\)", "", text[m.end():at]))
        depth, end = 0, at
        while True:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
            if depth == 0:
                break
        yield name[0] if name else "?", text[at:end]


@pytest.mark.parametrize("name", FILES)
def test_every_kernel_waits_for_itself(name):
    text = source(name)
    seen = list(kernels(text))
    assert seen
    for kernel, body in seen:
        lines = [x.strip() for x in body.splitlines()]
        at = [i for i, x in enumerate(lines) if "after_earlier_work" in x]
        assert len(at) == 1 and lines[at[0]] == "after_earlier_work();", kernel
        # in the function's own block, whatever branch ran before
        before = "\n".join(lines[:at[0]])
        assert before.count("{") - before.count("}") == 1, kernel
        previous = [x for x in lines[:at[0]] if x][-1]
        assert previous[-1] in ";{}" and not re.match(r"(if|else|for|while)\b.*[^;{}]$", previous), kernel
    assert "griddepcontrol" not in text


def test_the_next_launch_is_let_in_after_the_wait():
    text = source("zero_device.cuh")
    assert re.findall(r"griddepcontrol\.\w+", text) == ["griddepcontrol.wait", "griddepcontrol.launch_dependents"]
    body = text[text.index("after_earlier_work"):]
    assert body.index("griddepcontrol.wait") < body.index("griddepcontrol.launch_dependents") < body.index("}")


def test_constant_loads_are_of_constants():
    """__ldg is for what no other kernel writes while this one lives, and it lives before the one ahead of it ends:
    the optimizer's table of blocks is, as its bind waits; a norm's weights and a layer's operands are not."""
    for name in FILES:
        text = source(name)
        found = [m.start() for m in re.finditer(r"__ldg|ld\.global\.nc|__restrict__", text)]
        if name == "zero_adamw.cu":
            at = text.index("AdamBlock block_at(")
            assert all(at < f < text.index("}", at) for f in found)
        else:
            assert not found, name
