"""The residual stream updated where it lies: out may be residual itself."""
import pytest
import torch

from block_harness import Guarded
from fully_sharded_unit_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


# a chunk to a thread, the ring (three chunks to a thread, two blocks to a row), passes over rows past 49152 columns
@pytest.mark.parametrize("rows,cols,pad", [(7, 40, 0), (5, 1283, 2), (1300, 1280, 0), (320, 12288, 0), (320, 12304, 8), (3, 20488, 0), (3, 49992, 0), (4, 70001, 3)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("block", [True, False])
def test_out_is_residual(rows, cols, pad, dtype, block):
    from conftest import library
    library()
    g = torch.Generator(device="cuda").manual_seed(rows)
    h, o = (torch.empty((rows, cols), device="cuda").normal_(generator=g) for _ in range(2))
    o = Guarded(rows, cols, dtype, pad, offset=pad % 3, like=o).t
    w = [torch.empty(cols, device="cuda").normal_(1.0, 0.2, generator=g).to(BF) for _ in range(3)]
    c = B.Compute(0)
    got = []
    for same in (False, True):
        x = Guarded(rows, cols, dtype, pad, offset=pad % 3, like=h)
        s = x if same else Guarded(rows, cols, dtype, pad, offset=pad % 3)
        y, r1, r2 = torch.empty((rows, cols), dtype=dtype, device="cuda"), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        kw = dict(block=o, post_gamma=w[0], gate=w[1], post_rstd=r2) if block else {}
        c.residual_norm_forward(x.t, s.t, residual_scale=0.75, y=y, gamma=w[2], rstd=r1, **kw)
        x.check(), s.check()
        got.append([s.t.clone(), y, r1] + ([r2] if block else []))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    c.close()
