"""The plans of products (csrc/product_plan.hpp), asked of a small host program."""
import functools
import os
import shutil
import subprocess
import tempfile

from conftest import ROOT

CLUSTERS = 76          # pairs of SMs: those of a whole GB300


@functools.lru_cache(maxsize=None)
def _program():
    cxx = shutil.which("g++") or shutil.which("c++")
    assert cxx, "a C++ compiler is needed"
    exe = os.path.join(tempfile.mkdtemp(prefix="product_plan_"), "product_plan")
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-I", os.path.join(ROOT, "fully_sharded_unit_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "product_plan.cpp"), "-o", exe], check=True)
    return exe


class Plan(dict):
    __getattr__ = dict.__getitem__

    @property
    def tiles(self):
        return self.tiles_m * self.tiles_n

    @property
    def shared(self):
        """Tiles that several clusters share along k."""
        return self.tiles - self.whole

    @property
    def deepest(self):
        return self.ks if self.whole else -(-self.ks // self.parts)

    @property
    def slices(self):
        return -(-self.deepest // self.slice)


def plans(products, clusters=CLUSTERS):
    """``products``: (M, N, K, a_trans, b_trans, sums), sums 0 for a BF16 result, 1
    for an F32 one, 2 for an 8-bit checkpoint."""
    text = "".join("%d %d %d %d %d %d %d\n" % (*(int(v) for v in p), clusters) for p in products)
    out = subprocess.run([_program()], input=text, capture_output=True, text=True, check=True).stdout
    return [Plan((k, int(v)) for k, v in (f.split("=") for f in line.split())) for line in out.splitlines()]


def of(kind, T, I, O, layout, sums):
    """The plan of one of the linear layer's products."""
    io = layout == "in_out"
    p = {"forward": (T, O, I, 0, io, sums), "grad_input": (T, I, O, 0, not io, sums),
         "grad_weight": ((I, O) if io else (O, I)) + (T, 1, 1, sums)}[kind]
    return plans([p])[0]


# Products (M, N, K) whose plans take every path of the product kernels between
# them; tests/test_product_plan.py says which and holds them to it.
PRODUCTS = [
    (2500, 2608, 264), (2500, 2600, 264), (2501, 2603, 265),          # rounds of tiles, more than one band
    (4096, 5120, 256), (4864, 5120, 320),                             # wide tiles, four chunks to a warp
    (512, 512, 16384), (520, 520, 16384), (513, 515, 16385),          # every tile shared along k
    (2600, 2608, 20000), (2600, 2600, 20000), (2601, 2603, 20001),    # one accumulator, long sums, some tiles shared
    (2048, 3200, 17000), (2600, 2608, 1400), (2600, 2600, 1400), (2601, 2603, 1401),   # two accumulators and slices
    (200, 30000, 264), (201, 30001, 265),                             # swapped, rounds
    (200, 512, 16384), (201, 515, 16385),                             # swapped and shared
    (200, 20000, 17000), (250, 19456, 17000),                         # swapped, long sums
]
