"""Block operators: what needs no GPU.  Sizes of checkpoints and workspaces, and
refusals that come before any CUDA call."""
import ctypes

import pytest

from fully_sharded_unit_gb300 import binding as B


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from conftest import library
    library()


def _code(f):
    with pytest.raises(B.FsdpError) as e:
        f()
    return e.value.code


@pytest.mark.parametrize("cols,ld,groups", [(1, 32, 1), (31, 32, 1), (32, 32, 1), (33, 64, 2), (12288, 12288, 384)])
def test_checkpoint_sizes(cols, ld, groups):
    assert B.fsdp_act8_layout(7, cols) == (ld, groups)


def test_workspace_grows_with_every_size():
    base = B.fsdp_linear_workspace_bytes(100, 72, 200)
    assert base < B.fsdp_linear_workspace_bytes(101, 72, 200)
    assert base < B.fsdp_linear_workspace_bytes(100, 80, 200)
    assert base < B.fsdp_linear_workspace_bytes(100, 72, 208)
    assert base + 72 * 200 * 2 <= B.fsdp_linear_workspace_bytes(100, 72, 200, weight_aligned=False)
    assert B.fsdp_linear_workspace_bytes(0, 8, 8) > 0
    assert B.fsdp_layer_norm_workspace_bytes(0, 8) == 0
    assert B.fsdp_layer_norm_workspace_bytes(10, 64) < B.fsdp_layer_norm_workspace_bytes(11, 64)


def test_bad_sizes_are_refused():
    bad = B.FSDP_E_INVALID_ARG
    assert _code(lambda: B.fsdp_act8_layout(-1, 8)) == bad
    assert _code(lambda: B.fsdp_act8_layout(1, 0)) == bad
    assert _code(lambda: B.fsdp_layer_norm_workspace_bytes(1, 0)) == bad
    assert _code(lambda: B.fsdp_layer_norm_workspace_bytes(-1, 8)) == bad
    assert _code(lambda: B.fsdp_linear_workspace_bytes(1, 0, 8)) == bad
    assert _code(lambda: B.fsdp_linear_workspace_bytes(1, 8, 1 << 31)) == bad
    lib = B.lib()
    assert lib.fsdp_linear_workspace_bytes(1, 8, 8, 1, None) == bad
    assert lib.fsdp_layer_norm_workspace_bytes(1, 8, None) == bad


def test_null_handles_are_refused():
    lib, bad = B.lib(), B.FSDP_E_INVALID_ARG
    f = ctypes.c_int32()
    assert lib.fsdp_compute_destroy(None) == B.FSDP_OK
    assert lib.fsdp_compute_create(-1, None, ctypes.byref(ctypes.c_void_p())) == bad
    assert lib.fsdp_compute_create(0, None, None) == bad
    assert lib.fsdp_compute_status(None, ctypes.byref(f), None) == bad
    assert lib.fsdp_compute_set_wait_limit(None, 1.0, 0) == bad
    assert lib.fsdp_layer_norm_forward(None, None, None, None, 0, 1e-5, None, None, None, None, None) == bad
    assert lib.fsdp_layer_norm_backward(None, None, None, None, 0, None, None, None, None, None, None, 0, 0, None) == bad
    assert lib.fsdp_linear_forward(None, None, None, 0, None, 0, 0, None, None, None, None) == bad
    assert lib.fsdp_linear_grad_input(None, None, None, 0, 0, None, None, None, None) == bad
    assert lib.fsdp_linear_grad_weight(None, None, None, 0, None, None, 0, None) == bad
    assert lib.fsdp_act8_pack(None, None, None, None) == bad
    assert lib.fsdp_act8_unpack(None, None, 0, None, None) == bad
    assert "null" in B.fsdp_last_error()


def test_allocator_without_both_functions_is_refused():
    one = B.Allocator(B._ALLOC_FN(lambda n, ctx: None), B._FREE_FN(0), None)
    assert _code(lambda: B.fsdp_compute_create(0, one)) == B.FSDP_E_INVALID_ARG
