"""Refusals of the linear layers' entry points: on the host, before anything
is enqueued (CPU only)."""
import ctypes as C

import pytest
import torch

import routing_capacity_dispatch_amd as rcd
from routing_capacity_dispatch_amd import abi

FAKE = 0x100000
OK, INV, UNS, WS = abi.MOE_OK, abi.MOE_ERR_INVALID_ARG, abi.MOE_ERR_UNSUPPORTED, abi.MOE_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    return abi.load()


def args(**over):
    f = dict(M=100, N=48, K=32, x=FAKE, ldx=32, w=FAKE, ldw=32, bias=FAKE, residual=FAKE, ldr=48, y=FAKE, ldy=48,
             pre=FAKE, ldp=48, act=2, bias_dtype=0, out_dtype=1, reserved=0)
    return abi.MoeLinearArgs(**{**f, **over})


def grad(**over):
    f = dict(M=100, N=48, K=32, dy=FAKE, lddy=48, pre=FAKE, ldp=48, x=FAKE, ldx=32, w=FAKE, ldw=32, dx=FAKE, lddx=32,
             dw=FAKE, lddw=32, db=FAKE, act=2, dy_dtype=1, reserved=0)
    return abi.MoeLinearGrad(**{**f, **over})


def test_struct_layouts_match_header():
    assert C.sizeof(abi.MoeLinearArgs) == 14 * 8 + 4 * 4
    assert C.sizeof(abi.MoeLinearGrad) == 16 * 8 + 4 * 4  # three int32 and padding


@pytest.mark.parametrize("over,status", [
    (dict(M=-1), INV), (dict(N=-1), INV), (dict(K=-1), INV), (dict(ldx=31), INV), (dict(ldw=31), INV),
    (dict(ldy=47), INV), (dict(ldr=47), INV), (dict(ldp=47), INV), (dict(act=-1), INV), (dict(act=4), INV),
    (dict(bias_dtype=2), INV), (dict(out_dtype=2), INV), (dict(out_dtype=-1), INV), (dict(reserved=1), INV),
    (dict(x=FAKE + 1), INV), (dict(w=FAKE + 1), INV), (dict(bias=FAKE + 2), INV), (dict(y=FAKE + 1), INV),
    (dict(residual=FAKE + 1), INV), (dict(pre=FAKE + 1), INV),
    (dict(M=(1 << 30) + 1), UNS), (dict(N=(1 << 22) + 1, ldy=(1 << 22) + 1), UNS), (dict(ldx=(1 << 22) + 1), UNS),
    (dict(M=1 << 30, N=1 << 20, ldy=1 << 20, ldr=1 << 20, ldp=1 << 20), UNS)])
def test_linear_refusals(lib, over, status):
    n = C.c_size_t(0)
    assert lib.moe_linear_ws_bytes(C.byref(args(**over)), C.byref(n)) == status
    assert lib.moe_linear(C.byref(args(**over)), FAKE, 1 << 30, None) == status


def test_linear_null_and_workspace(lib):
    n = C.c_size_t(7)
    assert lib.moe_linear_ws_bytes(None, C.byref(n)) == INV and lib.moe_linear(None, None, 0, None) == INV
    assert lib.moe_linear_ws_bytes(C.byref(args()), None) == INV
    for f in ("x", "w", "y"):
        assert lib.moe_linear(C.byref(args(**{f: None})), FAKE, 1 << 30, None) == INV
    # nothing to do: no pointer is looked at
    assert lib.moe_linear(C.byref(args(M=0, x=None, w=None, y=None)), None, 0, None) == OK
    assert lib.moe_linear(C.byref(args(N=0, x=None, w=None, y=None)), None, 0, None) == OK
    # few rows or a small product: none needed; many whose rows do not start or end on 16 bytes: copies; a long K shared: sums
    big = dict(M=4096, N=4096, ldy=4096, ldr=4096, ldp=4096)
    for over, some in ((dict(M=16, N=1 << 20, K=31, ldy=1 << 20, ldr=1 << 20, ldp=1 << 20), False), (dict(M=100, K=31), False), (big, False), (dict(big, K=31), True),
                       (dict(big, ldx=36), True), (dict(big, w=FAKE + 2), True),
                       (dict(M=100, K=32768, ldx=32768, ldw=32768), True)):
        a = args(**over)
        assert lib.moe_linear_ws_bytes(C.byref(a), C.byref(n)) == OK and (n.value > 0) == some, over
        if some:
            for ws, size in ((None, n.value), (FAKE + 16, n.value), (FAKE, n.value - 1)):
                assert lib.moe_linear(C.byref(a), ws, size, None) == WS


@pytest.mark.parametrize("over,status", [
    (dict(M=-1), INV), (dict(lddy=47), INV), (dict(ldp=47), INV), (dict(ldx=31), INV), (dict(ldw=31), INV),
    (dict(lddx=31), INV), (dict(lddw=31), INV), (dict(act=4), INV), (dict(dy_dtype=2), INV), (dict(reserved=1), INV),
    (dict(dy=FAKE + 1), INV), (dict(pre=FAKE + 1), INV), (dict(dx=FAKE + 1), INV), (dict(db=FAKE + 2), INV),
    (dict(dy=FAKE + 2, dy_dtype=0), INV), (dict(M=2097121), UNS), (dict(lddy=(1 << 22) + 1), UNS)])
def test_linear_backward_refusals(lib, over, status):
    n = C.c_size_t(0)
    assert lib.moe_linear_backward_ws_bytes(C.byref(grad(**over)), C.byref(n)) == status
    assert lib.moe_linear_backward(C.byref(grad(**over)), FAKE, 1 << 30, None) == status


def test_linear_backward_null_and_workspace(lib):
    n = C.c_size_t(0)
    assert lib.moe_linear_backward(None, None, 0, None) == INV
    assert lib.moe_linear_backward_ws_bytes(C.byref(grad()), None) == INV
    for f in ("dy", "pre", "x", "w"):
        assert lib.moe_linear_backward(C.byref(grad(**{f: None})), FAKE, 1 << 30, None) == INV
    a = grad()
    assert lib.moe_linear_backward_ws_bytes(C.byref(a), C.byref(n)) == OK and n.value > 0
    for ws, size in ((None, n.value), (FAKE + 16, n.value), (FAKE, n.value - 1)):
        assert lib.moe_linear_backward(C.byref(a), ws, size, None) == WS
    # nothing asked for, nothing to do
    assert lib.moe_linear_backward(C.byref(grad(dx=None, dw=None, db=None, dy=None, pre=None)), None, 0, None) == OK


def test_binding_refusals():
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(3, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="act"):
        rcd.linear(x, w, act="tanh")
    with pytest.raises(ValueError, match="on a GPU"):
        rcd.linear(x, w)
    with pytest.raises(ValueError, match="two-dimensional"):
        rcd.linear(x[0], w)
    with pytest.raises(ValueError, match="out_dtype"):
        rcd.linear(x, w, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="on a GPU"):
        rcd.linear_backward(x, x, w)
