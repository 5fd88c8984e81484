"""AdamW over tensors: constants of a tensor that are no numbers in fp32 are refused before anything is enqueued."""
import pytest
import torch

from fully_sharded_unit_gb300 import binding as B

HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)


@pytest.mark.gpu
def test_scaled_constants():
    from conftest import library
    library()
    c = B.Compute(0)
    p, g, m, v = (torch.ones(40, device="cuda") for _ in range(4))

    def step(lr_scale=1.0, decay_scale=1.0, **hp):
        c.adamw_tensors(B.AdamWTensors([p], [g], [m], [v], lr_scale=[lr_scale], decay_scale=[decay_scale]), dict(HP, **hp), 1)

    for kw in (dict(lr=0.0, weight_decay=1e300, decay_scale=1e300),         # 0 times infinity
               dict(lr=1e20, weight_decay=1e20), dict(lr=1.0, lr_scale=1e25, decay_scale=1e20),      # decay past fp32
               dict(lr=1e38, beta1=0.999, lr_scale=3.0), dict(lr=1e39)):    # lr / (1 - beta1^t) past fp32
        with pytest.raises(B.FsdpError) as e:
            step(**kw)
        assert e.value.code == B.FSDP_E_INVALID_ARG and "finite" in str(e.value), kw
    assert all(bool((t == 1).all()) for t in (p, g, m, v))
    step(lr=0.0, weight_decay=1e30, decay_scale=1e30)
    assert bool((p == 1).all())
    step()
    assert bool((p != 1).all()) and bool(torch.isfinite(p).all())
    c.close()
