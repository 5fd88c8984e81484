"""Kernels that may start before the kernel in front of them has ended: read in
the sources that none of them takes the non-coherent load path, whose data must
not be written while a kernel lives (and here is, by the kernel in front)."""
import os
import re

from conftest import ROOT

CSRC = os.path.join(ROOT, "fully_sharded_unit_gb300", "csrc")
NON_COHERENT = re.compile(r"\b__ldg\s*\(|ld\.global(\.\w+)*\.nc\b|__restrict__|__restrict\b")


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_no_kernel_that_starts_early_reads_non_coherently():
    sources = {n: _code(n) for n in sorted(os.listdir(CSRC)) if n.endswith((".cu", ".cuh", ".hpp"))}
    early = [n for n, s in sources.items() if "starts_early(" in s]
    assert {"few.cu", "linear.cu", "norm.cu", "act8.cu"} <= set(early)
    for n in early + ["epilogue.cuh"]:      # block_device.cuh is among them: it defines the call
        found = NON_COHERENT.findall(sources[n])
        assert not found, (n, found)


def test_every_kernel_of_these_sources_waits_before_it_touches_memory():
    for n in ("few.cu", "linear.cu", "norm.cu", "act8.cu"):
        s = _code(n)
        kernels = [m.start() for m in re.finditer(r"__global__", s)]
        for a, b in zip(kernels, kernels[1:] + [len(s)]):
            body = s[a:b]
            assert re.search(r"starts_early\(\);\s*after_previous\(\);", body), (n, body[:120])
