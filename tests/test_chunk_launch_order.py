"""Programmatic launches of the chunk kernels: a kernel launched while the one before it in the stream still
runs waits for that one on every path, an early way out too.  Otherwise work queued behind it could run
while the first kernel still writes.  Read from the sources: the order is one of instructions, and a
run only shows it by luck."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_sparse_long_kap_b200", "csrc")


def _body(name):
    for f in sorted(os.listdir(CSRC)):
        text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, f)).read())
        m = re.search(r"__global__[^;{]*?\b" + name + r"\s*\([^{;]*\)\s*\{", text)
        if m:
            depth, i = 1, m.end()
            while depth:
                depth += {"{": 1, "}": -1}.get(text[i], 0)
                i += 1
            return text[m.end():i - 1]
    raise AssertionError(name)


def _dependents():
    """Kernels that a launch_pdl call names."""
    text = open(os.path.join(CSRC, "cosa.cu")).read()
    calls = re.findall(r"launch_pdl\(([^;]*);", text)
    names = {n for c in calls for n in re.findall(r"\b(\w+_kernel)\b", c)}
    if any(re.match(r"kern\b", c) for c in calls):
        names.add("chunk_attn_kernel")
    return sorted(names)


def test_the_dependent_kernels_are_these():
    assert _dependents() == ["chunk_attn_kernel", "chunk_combine_kernel", "evict_gather_kernel"]


@pytest.mark.parametrize("name", ["chunk_attn_kernel", "chunk_combine_kernel", "evict_gather_kernel"])
def test_a_dependent_kernel_waits_before_its_first_way_out(name):
    body = _body(name)
    # (returns of lambdas hand back a value)
    first = re.search(r"\breturn\s*;", body)
    wait = body.find("pdl_wait()")
    assert wait >= 0 and (first is None or wait < first.start())
    # and again where the early way out is not taken
    assert first is None or body.count("pdl_wait()") >= (2 if name == "chunk_attn_kernel" else 1)


def test_the_mass_loaders_allow_for_the_work_they_are_ahead_of():
    """A slot of theirs comes free after whole pairs of key blocks, not after one hand-off: a limit that
    does not grow with the chunk's tiles would end a long one as a timeout."""
    body = _body("attn_mass_kernel")
    waits = re.findall(r"(\w+)\(b_[kq]empty\(s\), [^;{]*?, (.*?)\) *[?)]", body)
    assert [w[0] for w in waits] == ["wait_long", "wait_long"]
    assert "most_tiles" in waits[0][1] and "share" in waits[1][1]
    assert re.search(r"tmo \+ \d+ull \* steps", body)
