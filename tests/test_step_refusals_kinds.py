"""What is no tensor where one is expected: an error of the binding's, not of Python's."""
import pytest
import torch

from fully_sharded_unit_gb300 import binding as B

HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)


def _refused(f):
    with pytest.raises(B.FsdpError) as e:
        f()
    assert e.value.code == B.FSDP_E_INVALID_ARG


def test_numbers_for_scale_and_skip():
    from conftest import library
    library()
    none = B.AdamWTensors([], [], [], [])
    for kw in (dict(grad_scale=0.5), dict(skip=1), dict(skip=False), dict(grad_scale=[1.0])):
        _refused(lambda: B.fsdp_adamw_tensors(B.ComputeHandle(), none, HP, 1, **kw))


@pytest.mark.gpu
def test_lists_for_alternatives():
    from conftest import library
    library()
    c = B.Compute(0)
    z = torch.zeros((4, 8), device="cuda")
    tt, tl = torch.zeros((4, 3), dtype=torch.int64, device="cuda"), torch.zeros((4, 3), device="cuda")
    for kw in (dict(top_tokens=tt.tolist(), top_logprobs=tl), dict(top_tokens=tt, top_logprobs=tl.tolist()), dict(top_tokens=None, top_logprobs=tl), dict(top_tokens=3, top_logprobs=tl)):
        _refused(lambda: c.token_logprobs_forward(z, None, None, **kw))
    c.close()
