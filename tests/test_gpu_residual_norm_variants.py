"""Every kernel of the residual norm at rows enough to reach it, on 16-byte boundaries and off them: chunks to a thread,
groups to a block, clusters, vectors in shared memory or registers.  Checks and bounds are those of test_gpu_residual_norm."""
import pytest
import torch

import test_gpu_residual_norm as R
from residual_norm_rows import Aligned

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from conftest import library
    library()


def _both(rows, cols, dtype, params, post, gate, grads=F32, out=None, **kw):
    i, c, s, rstd, post_rstd = R._check(rows, cols, dtype, params, post, gate, 0, out=out, **kw)
    R._check_backward(i, c, s, rstd, post_rstd, params, grads, out or dtype, 0, **{k: v for k, v in kw.items() if k.startswith("has")})
    c.close()


VECTORS = [(BF, True, True), (BF, True, False), (F32, True, True), (BF, False, True), (F32, False, False)]


# forward: one, two and three chunks to a thread, 1 to 15 groups to a block, clusters of two to eight.  Backward: groups up to
# 4096 columns, rows held from 4104 to 12288 (two and three chunks; BF16 vectors), clusters beyond and where vectors are floats
@pytest.mark.parametrize("rows,cols", [(1, 8), (5, 40), (1, 5120), (3, 9000), (2, 12288), (2, 12304), (5000, 128), (1300, 1280), (700, 2048), (320, 4096), (160, 4104), (160, 5120), (320, 6144), (320, 7168), (160, 8192),
                                       (160, 8200), (320, 12288), (160, 12304), (160, 20480), (80, 33008), (40, 49152)])
@pytest.mark.parametrize("params,post,gate", VECTORS)
def test_rows_on_boundaries(monkeypatch, rows, cols, params, post, gate):
    monkeypatch.setattr(R, "Guarded", Aligned)
    _both(rows, cols, BF, params, post, gate)


@pytest.mark.parametrize("rows,cols", [(5000, 129), (1300, 1283), (320, 4099), (320, 6150), (320, 7169), (160, 8195), (320, 12289), (160, 12299), (160, 20483), (80, 33001)])
@pytest.mark.parametrize("params,post,gate", VECTORS[1:4])
def test_rows_that_start_anywhere(rows, cols, params, post, gate):
    _both(rows, cols, BF, params, post, gate)


@pytest.mark.parametrize("rows,cols", [(1300, 1280), (160, 5120), (160, 12288)])
@pytest.mark.parametrize("kw", [dict(dtype=F32), dict(dtype=F32, out=BF), dict(dtype=BF, out=F32), dict(dtype=BF, mixed=True), dict(dtype=BF, has_block=False), dict(dtype=BF, grads=BF)])
def test_types_and_absences_on_boundaries(monkeypatch, rows, cols, kw):
    monkeypatch.setattr(R, "Guarded", Aligned)
    kw = dict(kw)
    block = kw.get("has_block", True)
    _both(rows, cols, kw.pop("dtype"), BF, block, block, **kw)


@pytest.mark.parametrize("rows,cols", [(5000, 128), (1300, 1280), (320, 4096), (160, 5120), (320, 7168), (320, 12288), (160, 12304), (1300, 1283), (320, 5121), (60, 33001)])
def test_values_that_are_not_finite(rows, cols):
    """They stay in their rows, and in the columns' sums; a row's other group, block or cluster does not meet them."""
    i = R._inputs(rows, cols, BF, BF, True, True, 0)
    h, o, dy, dout = ((i[k].t if cols % 8 else i[k].t.clone()) for k in ("h", "o", "dy", "dout"))
    c = R._compute(rows, cols)
    h[1, 5], o[3, 7], dy[5, 2], dout[rows - 1, cols - 1] = float("inf"), float("nan"), float("nan"), float("-inf")
    s, y, dh, db = (torch.empty_like(h) for _ in range(4))
    r1, r2, g = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), [torch.empty(cols, device="cuda") for _ in range(3)]
    c.residual_norm_forward(h, s, block=o, post_gamma=i["post"], gate=i["gate"], y=y, gamma=i["gamma"], eps=R.EPS, rstd=r1, post_rstd=r2)
    rest = torch.ones(rows, dtype=torch.bool, device="cuda")
    rest[[1, 3]] = False
    assert bool(torch.isfinite(y[rest].float()).all()) and bool(torch.isfinite(s[rest].float()).all()) and bool(torch.isnan(y[3]).all())
    assert bool(torch.isnan(y[1, 5])) and not bool(y[1, :5].any()) and not bool(y[1, 6:].any()) and torch.isinf(s[1]).sum() == 1
    c.residual_norm_backward(dy, dout, s, o, dh, db, gamma=i["gamma"], rstd=r1, dgamma=g[0], post_gamma=i["post"], post_rstd=r2, dpost_gamma=g[1],
                             gate=i["gate"], dgate=g[2])
    rest[[5, rows - 1]] = False
    assert bool(torch.isfinite(dh[rest].float()).all()) and bool(torch.isfinite(db[rest].float()).all())
    assert bool(torch.isnan(dh[3]).all()) and bool(torch.isnan(dh[5]).all()) and bool(torch.isnan(db[5]).all())
    assert bool(torch.isinf(dh[rows - 1]).sum() == 1) and bool(torch.isfinite(dh[rows - 1, :cols - 1].float()).all())
    assert bool(torch.isnan(g[1]).all()) and bool(torch.isnan(g[2]).all())     # every column meets row 5's t
    c.close()
