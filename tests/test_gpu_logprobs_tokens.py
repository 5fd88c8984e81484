"""Tokens outside the vocabulary in the calls that give gradients."""
import pytest
import torch

from fully_sharded_unit_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_a_token_outside_the_vocabulary_with_the_entropys_gradient_alone(dtype, out):
    """The loss takes tokens whatever gradients are given: one that does not exist makes its row of dlogits NaN."""
    from conftest import library
    library()
    c = B.Compute(0)
    z = torch.randn((5, 100), device="cuda").to(dtype)
    t = torch.tensor([3, 100, 2 ** 40, -1, 99], device="cuda")
    lp, dz, b = torch.empty(5, device="cuda"), torch.empty((5, 100), dtype=out, device="cuda"), torch.ones(5, device="cuda")
    for a in (None, torch.zeros(5, device="cuda"), torch.ones(5, device="cuda")):
        c.token_logprobs_loss(z, t, lp, dz, dlogprob=a, dentropy=b)
        assert torch.isnan(lp).tolist() == [False, True, True, False, False]
        assert torch.isnan(dz).all(dim=1).tolist() == torch.isnan(dz).any(dim=1).tolist() == [False, True, True, False, False]
        assert c.status() == B.FSDP_KSTATUS_BAD_TOKEN and c.status() == 0
    # the backward pass looks at tokens only where a gradient goes through them
    st, h = torch.empty((5, 2), device="cuda"), torch.empty(5, device="cuda")
    c.token_logprobs_forward(z, None, None, entropy=h, stats=st)
    c.token_logprobs_backward(z, t, st, dz, entropy=h, dentropy=b)
    assert bool(torch.isfinite(dz).all()) and c.status() == 0
    c.close()
