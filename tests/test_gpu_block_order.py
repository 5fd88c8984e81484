"""Block operators one after another on buffers that are written again while the
next call is already waiting to start: the bits of the same calls with the GPU
waited for after each."""
import pytest
import torch

from fully_sharded_unit_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from conftest import library
    library()


@pytest.mark.parametrize("tokens,d,o,pad", [(1, 256, 512, 0), (3, 40, 72, 0), (8, 1280, 640, 0), (2, 129, 40, 1), (40, 129, 129, 1)])
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
def test_reused_buffers_are_read_as_last_written(tokens, d, o, pad, layout):
    """norm into n, product of n into y, norm of y into m, product of m into n's
    width, 100 times; n, y and m stay the same buffers, and so does the weight,
    which is written anew (a copy) before every product."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(tokens * d)
    normal = lambda *s: torch.empty(s, device="cuda").normal_(generator=gen).to(BF)  # noqa: E731
    cut = lambda rows, cols: torch.empty((rows, cols + pad), dtype=BF, device="cuda")[:, :cols]  # noqa: E731
    shape = lambda a, b: (a, b) if layout == "in_out" else (b, a)  # noqa: E731
    up, down = [normal(*shape(d, o)) for _ in range(2)], [normal(*shape(o, d)) for _ in range(2)]
    gd, go, x0 = normal(d), normal(o), normal(tokens, d)
    c = B.Compute(B.fsdp_linear_workspace_bytes(tokens, d, o, weight_aligned=False))

    def run(wait):
        n, y, m = cut(tokens, d), cut(tokens, o), cut(tokens, o)
        w, v = torch.empty_like(up[0]), torch.empty_like(down[0])
        x = x0.clone()
        mean, rstd = torch.empty(tokens, device="cuda"), torch.empty(tokens, device="cuda")
        kept = []
        for i in range(100):
            w.copy_(up[i & 1])
            v.copy_(down[i & 1])
            for call in (lambda: c.layer_norm_forward(x, gd, gd, 1e-5, n, mean, rstd),
                         lambda: c.linear_forward(n, w, y, weight_layout=layout),
                         lambda: c.layer_norm_forward(y, go, go, 1e-5, m, mean, rstd),
                         lambda: c.linear_forward(m, v, x, residual=x, weight_layout=layout)):
                call()
                if wait:
                    torch.cuda.synchronize()
            kept.append((n.clone(), y.clone(), m.clone(), x.clone()))
        torch.cuda.synchronize()
        return kept

    for i, (a, b) in enumerate(zip(run(True), run(False))):
        for u, w in zip(a, b):
            assert torch.equal(u.view(torch.int16) if u.is_contiguous() else u, w.view(torch.int16) if w.is_contiguous() else w), i
    assert c.status() == 0
    c.close()
