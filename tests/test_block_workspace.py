"""Workspace for weights that are pieces of a longer buffer: widths do not say
where a row begins."""
import pytest
import torch

from fully_sharded_unit_gb300 import binding as B

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from conftest import library
    library()


def test_the_weight_itself_is_looked_at():
    flat = torch.empty(72 * 200 + 64, dtype=BF)
    flat = flat[-(flat.data_ptr() // 2) % 8:]                 # from a 16-byte boundary
    aligned = B.fsdp_linear_workspace_bytes(100, 72, 200, weight_aligned=True)
    room = B.fsdp_linear_workspace_bytes(100, 72, 200, weight_aligned=False)
    assert room > aligned
    for offset in range(17):
        w = flat[offset:offset + 72 * 200]
        want = aligned if offset % 8 == 0 else room
        for view in (w.view(72, 200), w.view(200, 72)):
            assert B.fsdp_linear_workspace_bytes(100, 72, 200, weight_aligned=view) == want
            assert B.fsdp_linear_workspace_bytes(100, 72, 200, weight_aligned=[flat[:14400].view(72, 200), view]) == want
    assert B.fsdp_linear_workspace_bytes(100, 72, 200, weight_aligned=flat[:14400].view(72, 200)[:, :64]) == aligned
    assert B.fsdp_linear_workspace_bytes(100, 64, 64, weight_aligned=flat[:64 * 68].view(64, 68)[:, :64]) > \
        B.fsdp_linear_workspace_bytes(100, 64, 64, weight_aligned=True)


@pytest.mark.gpu
@pytest.mark.parametrize("offset", [0, 1, 4, 8])
def test_a_handle_sized_by_the_weight_serves_it(offset):
    T, i, o = 40, 64, 72
    gen = torch.Generator(device="cuda")
    gen.manual_seed(offset)
    normal = lambda *s: torch.empty(s, device="cuda").normal_(generator=gen).to(BF)  # noqa: E731
    w = normal(offset + i * o)[offset:].view(i, o)
    x, dy, y, dx = normal(T, i), normal(T, o), normal(T, o), normal(T, i)
    c = B.Compute(B.fsdp_linear_workspace_bytes(T, i, o, weight_aligned=w))
    c.linear_forward(x, w, y)
    c.linear_grad_input(dy, w, dx)
    c.linear_grad_weight(x, dy, torch.empty((i, o), device="cuda"))
    assert c.status() == 0
    c.close()
    for got, want in ((y, x.double() @ w.double()), (dx, dy.double() @ w.double().t())):
        assert (got.double() - want).norm() <= 2.0 ** -8 * want.norm()


def test_sizes_whose_bytes_do_not_fit_are_refused():
    """Each width is below 2^31 - 512, but a matrix of two of them has more bytes
    than 63 bits hold; a workspace of a negative or a wrapped size helps nobody."""
    top = (1 << 31) - 513
    for sizes in ((top, top, 8), (top, 8, top), (8, top, top), (top, top, top)):
        for aligned in (True, False):
            with pytest.raises(B.FsdpError) as e:
                B.fsdp_linear_workspace_bytes(*sizes, weight_aligned=aligned)
            assert e.value.code == B.FSDP_E_INVALID_ARG
    most = B.fsdp_linear_workspace_bytes(1 << 28, 1 << 30, 1 << 30, weight_aligned=False)
    assert most > (1 << 59) + (1 << 59) + (1 << 61)
