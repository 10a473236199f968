"""Linear layers whose launches would pass 2^32 threads are refused on the host,
before anything is enqueued (CPU only)."""
import ctypes as C

import pytest

from routing_capacity_dispatch_amd import abi
from test_linear_abi import FAKE, OK, UNS, WS, args, grad

WIDE = dict(ldy=1 << 22, ldr=1 << 22, ldp=1 << 22)


@pytest.fixture(scope="module")
def lib():
    return abi.load()


# 2^35 values of x: copied where rows or their ends are off 16 bytes
@pytest.mark.parametrize("over,status", [
    (dict(M=1 << 23, K=4089, ldx=4096, ldw=4096), UNS), (dict(M=1 << 23, K=4096, ldx=4097, ldw=4096), UNS),
    (dict(M=1 << 23, K=4096, ldx=4096, ldw=4096, x=FAKE + 2), UNS),
    (dict(M=(1 << 23) - 1024, K=4089, ldx=4096, ldw=4096), WS), (dict(M=1 << 23, K=4096, ldx=4096, ldw=4097), WS),
    (dict(M=128, N=1 << 22, K=8185, ldx=8192, ldw=8192, **WIDE), UNS),
    (dict(M=128, N=1 << 22, K=8177, ldx=8192, ldw=8192, **WIDE), WS),
    (dict(M=1 << 23, N=1 << 10, K=4081, ldx=4096, ldw=4096, **WIDE), WS)])
def test_forward(lib, over, status):
    n = C.c_size_t(0)
    a = args(**over)
    assert lib.moe_linear_ws_bytes(C.byref(a), C.byref(n)) == (OK if status == WS else status)
    assert lib.moe_linear(C.byref(a), None, 0, None) == status


@pytest.mark.parametrize("over,status", [
    (dict(M=1 << 20, K=1 << 15, ldx=(1 << 15) + 1), UNS), (dict(M=(1 << 20) - 1024, K=1 << 15, ldx=(1 << 15) + 1), WS),
    (dict(M=1 << 20, K=1 << 15, ldx=(1 << 15) + 1, dw=None), WS),
    # dx and dw in one launch, each alone below the limit
    (dict(M=1 << 15, N=1 << 15, K=1 << 21, lddy=1 << 15, ldp=1 << 15), UNS),
    (dict(M=1 << 15, N=1 << 15, K=1 << 21, lddy=1 << 15, ldp=1 << 15, dw=None), WS),
    (dict(M=1 << 15, N=1 << 15, K=1 << 21, lddy=1 << 15, ldp=1 << 15, dx=None), WS),
    (dict(M=1 << 14, N=1 << 15, K=1 << 21, lddy=1 << 15, ldp=1 << 15), WS)])
def test_backward(lib, over, status):
    K = over["K"]
    f = {**dict(ldx=K, ldw=K, lddx=K, lddw=K), **over}
    n = C.c_size_t(0)
    a = grad(**f)
    assert lib.moe_linear_backward_ws_bytes(C.byref(a), C.byref(n)) == (OK if status == WS else status)
    assert lib.moe_linear_backward(C.byref(a), None, 0, None) == status
