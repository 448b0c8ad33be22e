"""Kernels that are launched to overlap the launch before them (csrc/kernels.h, launch_overlapped), read as source: what that
launch writes is no read-only argument of theirs, and is read past the first-level cache.

A `const T* __restrict__` argument tells the compiler that nothing writes there while the kernel runs, so it may move a load of
it above the wait for the launch before. Arguments that an earlier kernel of the same call writes are therefore plain pointers,
read by __ldcg or by asynchronous copies behind the wait."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sliding_window_attention_chunked_b200", "csrc")


def _balanced(text, at):
    """The end of the bracket that opens at text[at]."""
    pair = {"(": ")", "{": "}"}[text[at]]
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == text[at]) - (text[i] == pair)
        if depth == 0:
            return i
    raise AssertionError("unbalanced")


def kernels(text):
    """name -> (arguments, body) of the kernels in a source file, comments taken out."""
    text = re.sub(r"//[^\n]*", "", text)
    found = {}
    for m in re.finditer(r"__global__ void(?: __launch_bounds__)?", text):
        at = m.end()
        if text[at] == "(":
            at = _balanced(text, at) + 1
        name = re.compile(r"\s*(\w+)\s*\(").match(text, at)
        end = _balanced(text, name.end() - 1)
        body = text.index("{", end)
        found[name.group(1)] = ([a.strip() for a in text[name.end():end].split(",")], text[body:_balanced(text, body) + 1])
    return found


def faults(text):
    """What is wrong with the overlapped kernels of a source file."""
    ks = kernels(text)
    name_of = lambda arg: re.search(r"(\w+)$", arg).group(1)
    found = []
    for at in re.finditer(r"launch_overlapped\(\s*(\w+)", text):
        k = at.group(1)
        if k not in ks:
            continue  # the definition of launch_overlapped itself
        args, body = ks[k]
        # the kernels that the host function has launched so far, and what they write
        host = text[text.rfind("\n}\n", 0, at.start()) + 1:at.start()]
        before = re.findall(r"(\w+)(?:<[^<>]*>)?<<<", host) + re.findall(r"launch_overlapped\(\s*(\w+)", host)
        written = {name_of(a) for b in before if b in ks for a in ks[b][0] if "*" in a and "const " not in a}
        for a in args:
            n = name_of(a)
            if "*" not in a or n not in written:
                continue
            if "__restrict__" in a:
                found.append(f"{k}: {n} is restricted")
            if re.search(rf"(?<![&\w.]){n}\[[^\]]*\](?!\s*=[^=])", body):
                found.append(f"{k}: {n} is read by a plain load")
    return found


FILES = [f for f in sorted(os.listdir(CSRC)) if f.endswith((".cu", ".cuh")) and "launch_overlapped(" in open(os.path.join(CSRC, f)).read()]


def test_there_are_overlapped_launches():
    assert len(FILES) >= 5


@pytest.mark.parametrize("name", FILES)
def test_overlapped_kernels_read_what_the_launch_before_writes_past_the_cache(name):
    assert faults(open(os.path.join(CSRC, name)).read()) == []


def test_the_check_catches_both_mistakes():
    text = """__global__ void other(const float* __restrict__ x, float* __restrict__ w) { w[0] = x[0]; }
__global__ void first(const float* __restrict__ x, float* __restrict__ y) { y[0] = x[0]; }
__global__ void __launch_bounds__(NT, D + E <= 8 ? 3 : 1)
second(const float* __restrict__ x, const float* __restrict__ w, ARG y, float* __restrict__ z) { z[0] = x[0] + w[0] + READ; }
void before() {
    other<<<1, 1>>>(x, w);
}
void go() {
    first<<<1, 1>>>(x, y);
    launch_overlapped(second, 1, 1, x, w, y, z);
}
"""
    assert faults(text.replace("ARG", "const float*").replace("READ", "__ldcg(y + 1)")) == []
    assert faults(text.replace("ARG", "const float* __restrict__").replace("READ", "__ldcg(y + 1)")) == ["second: y is restricted"]
    assert faults(text.replace("ARG", "const float*").replace("READ", "y[3]")) == ["second: y is read by a plain load"]
