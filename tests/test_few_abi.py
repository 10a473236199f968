"""Refusals of moe_forward_few: on the host, before anything is enqueued (CPU only)."""
import ctypes as C

import pytest
import torch

import routing_capacity_dispatch_amd as rcd
from routing_capacity_dispatch_amd import abi

FAKE = 0x100000
OK, INV, UNS, WS = abi.MOE_OK, abi.MOE_ERR_INVALID_ARG, abi.MOE_ERR_UNSUPPORTED, abi.MOE_ERR_WORKSPACE
NAMES = [n for n, _ in abi.MoeWeights._fields_]


@pytest.fixture(scope="module")
def lib():
    return abi.load()


def cfg(T=4, D=128, L=64, E=10, k=3, F=192, S=2, Fs=64, **kw):
    return rcd.make_config(T, D, L, E, 1, k, F, S, Fs, 1, **kw)


def call(lib, c, w="all", x=FAKE, r=FAKE, y=FAKE, lo=FAKE, ti=FAKE, ga=FAKE, ws=FAKE, size=1 << 40):
    w = abi.MoeWeights(**{n: FAKE for n in NAMES}) if w == "all" else w
    return lib.moe_forward_few(c and C.byref(c), w and C.byref(w), x, r, y, lo, ti, ga, ws, size, None)


@pytest.mark.parametrize("c,status", [
    (None, INV), (cfg(T=-1), INV), (cfg(T=17), UNS), (cfg(k=11), INV), (cfg(D=100), UNS), (cfg(L=96), UNS),
    (cfg(F=32), UNS), (cfg(Fs=32), UNS), (cfg(S=4), UNS), (cfg(E=1025, k=1), UNS), (cfg(E=100, k=65), UNS),
    (cfg(dtype="f32"), UNS), (cfg(S=0, Fs=0), WS), (cfg(), WS), (cfg(T=16, E=1024, k=64), WS)])
def test_configs(lib, c, status):
    n = C.c_size_t(0)
    assert lib.moe_forward_few_ws_bytes(c and C.byref(c), C.byref(n)) == (OK if status == WS else status)
    # a valid call goes on to its workspace, and no further
    assert call(lib, c, ws=None) == status
    if status == WS:
        assert n.value > 0 and call(lib, c, size=n.value - 1) == WS and call(lib, c, ws=FAKE + 16) == WS
        assert lib.moe_forward_few_ws_bytes(C.byref(c), None) == INV


def test_pointers(lib):
    c = cfg()
    assert call(lib, c, w=None) == INV
    for n in NAMES:
        for bad in (None, FAKE + 2):
            w = abi.MoeWeights(**{m: (bad if m == n else FAKE) for m in NAMES})
            want = WS if n == "router_bias" and bad is None else INV
            assert call(lib, c, w=w, ws=None) == want, n
            if n.startswith("ws_"):
                assert call(lib, cfg(S=0, Fs=0), w=w, ws=None) == WS
    for over in (dict(x=None), dict(y=None), dict(x=FAKE + 8), dict(y=FAKE + 8), dict(r=FAKE + 8), dict(lo=FAKE + 2),
                 dict(ti=FAKE + 1), dict(ga=FAKE + 3)):
        assert call(lib, c, **over, ws=None) == INV, over
    assert call(lib, c, r=None, lo=None, ti=None, ga=None, ws=None) == WS
    assert call(lib, cfg(T=0), x=None, y=None, r=None, ws=None) == OK


def test_binding_refusals():
    with pytest.raises(rcd.MoeError, match="UNSUPPORTED"):
        rcd.ForwardFew(cfg(T=17), {}, torch.device("cuda", 0))
    with pytest.raises(ValueError, match="w_latent"):
        rcd.ForwardFew(cfg(), {"w_latent": torch.zeros(64, 128, dtype=torch.bfloat16)}, torch.device("cuda", 0))
