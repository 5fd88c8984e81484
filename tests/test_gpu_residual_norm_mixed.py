"""The residual stream in F32 beside a block in BF16: what each matrix gives is the all-F32 call's, rounded to its type."""
import pytest
import torch

from fully_sharded_unit_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("rows,cols", [(1, 8), (9, 40), (700, 1280), (33, 1283), (5, 20488), (3, 49992), (2, 70001)])
@pytest.mark.parametrize("params", [BF, F32])
def test_every_matrix_has_its_own_type(rows, cols, params):
    from conftest import library
    library()
    g = torch.Generator(device="cuda").manual_seed(cols)
    n = lambda *s, t=F32: torch.empty(s, device="cuda").normal_(generator=g).to(t)  # noqa: E731
    h, o, dy, dout = n(rows, cols), n(rows, cols, t=BF), n(rows, cols, t=BF), n(rows, cols)
    w = [n(cols, t=params) for _ in range(3)]
    c = B.Compute(B.fsdp_residual_norm_workspace_bytes(rows, cols))
    got = []
    for block in (BF, F32):      # y, dy, dblock and the block's result in this type, the rest in F32
        out, y, dh, db = (torch.empty((rows, cols), dtype=t, device="cuda") for t in (F32, block, F32, block))
        r1, r2, v = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), [torch.empty(cols, device="cuda") for _ in range(3)]
        c.residual_norm_forward(h, out, block=o.to(block), post_gamma=w[0], gate=w[1], residual_scale=0.9, y=y, gamma=w[2], rstd=r1, post_rstd=r2)
        c.residual_norm_backward(dy.to(block), dout, out, o.to(block), dh, db, gamma=w[2], rstd=r1, dgamma=v[0], post_gamma=w[0], post_rstd=r2, dpost_gamma=v[1],
                                 gate=w[1], dgate=v[2], residual_scale=0.9)
        got.append((out, y.to(BF), r1, r2, dh, db.to(BF), *v))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert all(bool(torch.isfinite(t).all()) for t in got[0])
    c.close()
