"""What a compute handle keeps between calls, beside products of a few tokens,
which run without staged tiles and without workspace."""
import pytest
import torch

from fully_sharded_unit_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from conftest import library
    library()


def _normal(seed, *shape):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.empty(shape, device="cuda").normal_(generator=gen).to(BF)


def _code(f):
    with pytest.raises(B.FsdpError) as e:
        f()
    return e.value.code


def test_a_withheld_copy_is_that_of_the_next_staged_product():
    """Products of a few tokens, of none, and refused calls between arming and the
    staged product do not disarm it."""
    c = B.Compute(B.fsdp_linear_workspace_bytes(512, 256, 512))
    x, w = _normal(1, 512, 256), _normal(2, 256, 512)
    y, again = (torch.empty((512, 512), dtype=BF, device="cuda") for _ in range(2))
    c.linear_forward(x, w, y)
    assert c.status() == 0
    c.set_wait_limit(0.02, withhold_next=1)
    c.linear_forward(x[:1], w, again[:1])
    c.linear_grad_input(y[:8], w, torch.empty((8, 256), dtype=BF, device="cuda"))
    c.linear_forward(x[:0], w, again[:0])
    c.linear_grad_weight(x[:0], y[:0], torch.empty((256, 512), device="cuda"))
    assert _code(lambda: c.linear_forward(x, w[:, :511], again)) == B.FSDP_E_INVALID_ARG
    assert c.status() == 0
    c.linear_forward(x, w, again)
    assert c.status() == B.FSDP_KSTATUS_WAIT_TIMEOUT
    c.set_wait_limit()
    c.linear_forward(x, w, again)
    assert c.status() == 0 and torch.equal(y, again)
    c.close()


@pytest.mark.parametrize("tokens", [1, 2, 8])
@pytest.mark.parametrize("i,o", [(64, 128), (129, 40), (1280, 640)])
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
def test_a_few_tokens_need_no_workspace(tokens, i, o, layout):
    """Aligned or not: the same bits from a handle that has none as from one that
    has more than enough."""
    none, plenty = B.Compute(0), B.Compute(64 << 20)
    x, dy = _normal(i, tokens, i), _normal(o, tokens, o)
    w = _normal(7, i * o + 1)[1:].view((i, o) if layout == "in_out" else (o, i))
    got = []
    for c in (none, plenty):
        y, dx = torch.empty_like(dy), torch.empty_like(x)
        c.linear_forward(x, w, y, weight_layout=layout)
        c.linear_grad_input(dy, w, dx, weight_layout=layout)
        assert c.status() == 0
        got.append((y, dx))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    more = _normal(8, 9, i)
    assert _code(lambda: none.linear_forward(more, w, torch.empty((9, o), dtype=BF, device="cuda"), weight_layout=layout)) == B.FSDP_E_CAPACITY
    none.close()
    plenty.close()
