"""Refusals of moe_orthogonalize: on the host, before anything is enqueued
(CPU only)."""
import ctypes as C

import pytest
import torch

import routing_capacity_dispatch_amd as rcd
from routing_capacity_dispatch_amd import abi

FAKE = 0x100000
OK, INV, UNS, WS = abi.MOE_OK, abi.MOE_ERR_INVALID_ARG, abi.MOE_ERR_UNSUPPORTED, abi.MOE_ERR_WORKSPACE
USUAL = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module")
def lib():
    return abi.load()


def args(coeffs=USUAL, steps=5, **over):
    co = (C.c_float * (3 * max(steps, 1)))(*(list(coeffs) * max(steps, 1)))
    f = dict(batch=2, M=40, N=24, g=FAKE, ldg=24, stride_g=960, out=FAKE, ldo=24, stride_o=960,
             coeffs=C.cast(co, C.POINTER(C.c_float)), steps=steps, dtype=1, eps=1e-7, scale=1.0, reserved=0)
    return abi.MoeOrthoArgs(**{**f, **over}), co


def test_struct_layout_matches_header():
    assert C.sizeof(abi.MoeOrthoArgs) == 10 * 8 + 5 * 4 + 4


@pytest.mark.parametrize("over,status", [
    (dict(batch=-1), INV), (dict(M=-1), INV), (dict(N=-1), INV), (dict(ldg=23), INV), (dict(ldo=23), INV),
    (dict(stride_g=959), INV), (dict(stride_o=959), INV), (dict(steps=0), INV), (dict(steps=65), INV),
    (dict(dtype=2), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(scale=float("inf")), INV),
    (dict(reserved=1), INV), (dict(coeffs=None), INV), (dict(g=FAKE + 1), INV), (dict(out=FAKE + 1), INV),
    (dict(M=65537), UNS), (dict(N=65537, ldg=65537, ldo=65537), UNS), (dict(ldg=(1 << 30) + 1), UNS),
    (dict(batch=1 << 31), UNS)])
def test_refusals(lib, over, status):
    n = C.c_size_t(0)
    if over.get("steps") == 65:
        a, keep = args(steps=65)
    elif "steps" in over:
        a, keep = args()
        a.steps = over["steps"]
    else:
        a, keep = args()
        for k, v in over.items():
            setattr(a, k, v)
    assert lib.moe_orthogonalize_ws_bytes(C.byref(a), C.byref(n)) == status
    assert lib.moe_orthogonalize(C.byref(a), FAKE, 1 << 40, None) == status


@pytest.mark.parametrize("coeffs,steps,status", [
    (USUAL, 64, OK), ((1.5, -0.5, 0.0), 30, OK), ((1.875, -1.25, 0.375), 30, OK), ((0.0, 0.0, 0.0), 3, OK),
    ((1.0, 0.0, 0.0), 5, OK), ((2.0, 0.0, 0.0), 19, OK), ((2.0, 0.0, 0.0), 40, UNS), ((3.0, 3.0, 3.0), 5, UNS),
    ((float("nan"), 0.0, 0.0), 1, INV), ((1.0, float("inf"), 0.0), 1, INV)])
def test_coefficients(lib, coeffs, steps, status):
    n = C.c_size_t(0)
    a, keep = args(coeffs, steps)
    assert lib.moe_orthogonalize_ws_bytes(C.byref(a), C.byref(n)) == status


def test_null_and_workspace(lib):
    n = C.c_size_t(0)
    assert lib.moe_orthogonalize(None, FAKE, 1 << 30, None) == INV
    a, keep = args()
    assert lib.moe_orthogonalize_ws_bytes(C.byref(a), None) == INV
    assert lib.moe_orthogonalize_ws_bytes(C.byref(a), C.byref(n)) == OK and n.value > 0
    for ws, size in ((None, n.value), (FAKE + 16, n.value), (FAKE, n.value - 1)):
        assert lib.moe_orthogonalize(C.byref(a), ws, size, None) == WS
    for f in ("g", "out"):
        a, keep = args(**{f: None})
        assert lib.moe_orthogonalize(C.byref(a), FAKE, 1 << 40, None) == INV
    for f in ("batch", "M", "N"):
        a, keep = args(**{f: 0, "g": None, "out": None})
        assert lib.moe_orthogonalize(C.byref(a), None, 0, None) == OK
    # the workspace stops growing with the batch
    sizes = []
    for batch in (1, 4, 1 << 14, 1 << 20):
        a, keep = args(batch=batch)
        assert lib.moe_orthogonalize_ws_bytes(C.byref(a), C.byref(n)) == OK
        sizes.append(n.value)
    assert sizes[0] < sizes[1] < sizes[2] == sizes[3]


def test_binding_refusals():
    with pytest.raises(ValueError, match="on a GPU"):
        rcd.orthogonalize(torch.zeros(4, 4))
    with pytest.raises(ValueError, match="coeffs"):
        rcd._coefficients(((1.0, 2.0, 3.0),) * 3, 4)
    for bad in ((), (1.0, 2.0), ((1.0, 2.0, 3.0), 4.0)):
        with pytest.raises(ValueError, match="coeffs"):
            rcd._coefficients(bad, 2)
