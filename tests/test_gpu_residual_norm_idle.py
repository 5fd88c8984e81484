"""Widths whose chunks of eight columns do not fill a row's threads: what lies in shared memory behind
a row's end (here NaN, of the calls before) is in no result.  The checks and their bounds are those of
test_gpu_residual_norm, on rows that start on 16-byte boundaries."""
import pytest
import torch

import test_gpu_residual_norm as R
from fully_sharded_unit_gb300 import binding as B
from residual_norm_rows import Aligned

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from conftest import library
    library()


class _Poisoned:
    """A handle whose calls come right behind a backward pass of NaN, which leaves NaN in the ring, in the vectors'
    places and where the column sums are joined."""

    def __init__(self, rows, cols, width=4096):
        self.c = B.Compute(max(B.fsdp_residual_norm_workspace_bytes(rows, cols), B.fsdp_residual_norm_workspace_bytes(1300, width)))

        def nan(*shape, dtype=BF):
            return torch.full(shape, float("nan"), dtype=dtype, device="cuda")

        self.x, self.w, self.r, self.g = [nan(1300, width) for _ in range(6)], nan(width), nan(1300, dtype=F32), [nan(width) for _ in range(3)]

    def _poison(self):
        x, w, r, g = self.x, self.w, self.r, self.g
        self.c.residual_norm_backward(x[0], x[1], x[2], x[3], x[4], x[5], gamma=w, rstd=r, dgamma=g[0], post_gamma=w, post_rstd=r,
                                      dpost_gamma=g[1], gate=w, dgate=g[2])

    def residual_norm_forward(self, *a, **k):
        self._poison()
        self.c.residual_norm_forward(*a, **k)

    def residual_norm_backward(self, *a, **k):
        self._poison()
        self.c.residual_norm_backward(*a, **k)

    def close(self):
        self.c.close()


# rows enough for the forward pass to walk them in a ring as well; 6160 to 12304 columns have two or three chunks to a
# thread, or two blocks to a row
@pytest.mark.parametrize("rows,cols", [(5000, 64), (5000, 128), (4000, 320), (1000, 1600), (700, 2880), (320, 6160), (320, 9000), (320, 12304), (3, 40)])
@pytest.mark.parametrize("params,post,gate", [(BF, True, True), (F32, True, False), (BF, False, True), (F32, False, False)])
def test_places_past_a_rows_end(monkeypatch, rows, cols, params, post, gate):
    monkeypatch.setattr(R, "Guarded", Aligned)
    monkeypatch.setattr(R, "_compute", _Poisoned)
    i, c, s, rstd, post_rstd = R._check(rows, cols, BF, params, post, gate, 0)
    R._check_backward(i, c, s, rstd, post_rstd, params, F32, BF, 0)
    c.close()


@pytest.mark.parametrize("rows,cols", [(5000, 64), (5000, 128), (4000, 320), (1000, 1600), (700, 2880), (320, 6160)])
def test_again_and_again(monkeypatch, rows, cols):
    """Ordinary values: each call finds the column sums of the one before."""
    monkeypatch.setattr(R, "Guarded", Aligned)
    i, c, s, rstd, post_rstd = R._check(rows, cols, BF, BF, True, True, 0)
    dh, db, g = Aligned(rows, cols, BF), Aligned(rows, cols, BF), [torch.empty(cols, device="cuda") for _ in range(3)]
    first = None
    for _ in range(20):
        c.residual_norm_backward(i["dy"].t, i["dout"].t, s.t, i["o"].t, dh.t, db.t, gamma=i["gamma"], rstd=rstd, dgamma=g[0], post_gamma=i["post"],
                                 post_rstd=post_rstd, dpost_gamma=g[1], gate=i["gate"], dgate=g[2], residual_scale=0.75)
        got = [v.clone() for v in (dh.t, db.t, *g)]
        assert all(bool(torch.isfinite(v).all()) for v in got)
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(got, first))
    c.close()
