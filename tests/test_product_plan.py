"""How products are cut (csrc/product_plan.hpp), asked on the host: what any plan
has to keep to, and that the shapes which the GPU tests take reach every path."""
import random

from plan_harness import CLUSTERS, PRODUCTS, of, plans

UNCUT = 0x40000000


def _sound(q, p, clusters):
    M, N, K = q[:3]
    rows, cols = (N, M) if p.swapped else (M, N)
    assert p.bn in range(32, 257, 32) and p.tiles_m * 256 >= rows > (p.tiles_m - 1) * 256 and p.tiles_n * p.bn >= cols > (p.tiles_n - 1) * p.bn
    assert p.ks == -(-K // 64) and 1 <= p.parts <= max(1, p.ks // 4)
    assert p.units == p.whole + p.shared * p.parts and p.shared >= 0 and (p.parts > 1 or p.shared == 0)
    assert p.shared * p.parts <= clusters                       # the workspace has room for one part to a cluster
    assert 2 <= p.stages <= 10 and p.stages * (128 * 64 * 2 + p.stage_b) <= 6 * 256 * 64 * 2
    assert p.stage_b % 1024 == 0 and p.stage_b >= p.bn // 2 * 64 * 2
    # tensor memory: the accumulators, and the running sums where there are any
    sliced = p.deepest > p.slice
    assert p.two in (0, 1) and p.buffer >= p.bn
    assert (p.running + p.bn if sliced or not p.two else (p.two * p.buffer + p.bn)) <= 512
    assert p.running >= p.buffer * (1 + p.two)
    longest = (256, 12, max(4, min(12, int(K ** 0.5 / 4))))[q[5]]
    assert p.deepest <= longest and p.slice == UNCUT or p.slice <= longest and p.slices == -(-p.deepest // longest)
    assert p.two or not q[5]


def test_any_plan_is_sound():
    rng = random.Random(1)
    size = lambda hi: int(2 ** rng.uniform(0, hi))  # noqa: E731
    asked = [(size(15), size(15), size(19), rng.random() < 0.3, rng.random() < 0.5, rng.randrange(3)) for _ in range(4000)]
    asked += [(*p, a, b, e) for p in PRODUCTS for a, b in ((0, 0), (0, 1), (1, 1)) for e in (0, 1, 2)]
    for clusters in (CLUSTERS, 70, 1):
        for q, p in zip(asked, plans(asked, clusters)):
            _sound(q, p, clusters)


def test_the_shapes_of_the_gpu_tests_reach_every_path():
    """forward and grad_input call both orders of B's memory, with every type of
    result; what each of them has to have met."""
    asked = [(*p, 0, b, e) for p in PRODUCTS for b in (0, 1) for e in (0, 1, 2)]
    met = list(zip(asked, plans(asked)))
    have = lambda f: [q for q, p in met if f(q, p)]  # noqa: E731
    alignment = lambda q: 0 if q[1] % 8 else 2 if q[1] % 16 == 0 else 1  # noqa: E731
    for vec in (0, 1, 2):                      # of the epilogue's rows
        for f in (lambda p: p.shared > 0, lambda p: p.whole > 2 * CLUSTERS and p.slice == UNCUT and p.two, lambda p: not p.two and p.slices > 1,
                  lambda p: p.two and p.slices > 1, lambda p: p.tiles_m > 8 and p.whole > CLUSTERS):
            assert have(lambda q, p: not p.swapped and alignment(q) == vec and f(p)), (vec, f)
    for f in (lambda p: p.shared > 0, lambda p: p.whole > CLUSTERS, lambda p: not p.two, lambda p: p.two and p.slices > 1):
        assert have(lambda q, p: p.swapped and f(p))
    for b in (0, 1):
        assert have(lambda q, p: p.by_rows == b and not p.swapped and p.bn > 128) and have(lambda q, p: p.by_rows == b and p.bn == 256)
    assert have(lambda q, p: p.whole > 0 and p.shared > 0) and have(lambda q, p: p.whole == 0 and p.slices > 1 and p.parts > 1)
    assert have(lambda q, p: p.by_rows and p.stage_b == 2 * 64 * 64 * 2 and p.bn % 128)         # a second box, in part


def test_a_plan_by_layer():
    p = of("grad_input", 4096, 5120, 1280, "in_out", 0)
    assert p.by_rows == 0 and p.ks == 20
    assert of("grad_weight", 4096, 1280, 5120, "in_out", 1).by_rows == 1
    assert of("forward", 40, 64, 520, "in_out", 0).swapped and not of("grad_weight", 4096, 40, 520, "in_out", 0).swapped
