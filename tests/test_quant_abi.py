"""Refusals of the scored-routing and e4m3 entry points: on the host, before
anything is enqueued (CPU only)."""
import ctypes as C

import pytest
import torch

import routing_capacity_dispatch_amd as rcd
from routing_capacity_dispatch_amd import abi

FAKE, NUL = C.c_void_p(0x100000), None
OK, INV, UNS, WS = abi.MOE_OK, abi.MOE_ERR_INVALID_ARG, abi.MOE_ERR_UNSUPPORTED, abi.MOE_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    return abi.load()


def test_struct_layouts_match_header():
    assert C.sizeof(abi.MoeScoring) == 7 * 4
    assert C.sizeof(abi.MoeQuantGemm) == 13 * 8 + 4 * 4
    assert C.sizeof(abi.MoeQuantExperts) == 6 * 8


@pytest.mark.parametrize("field,value,status", [
    ("score", 2, INV), ("score", -1, INV), ("n_groups", 0, INV), ("n_groups", 5, INV), ("top_groups", 0, INV),
    ("top_groups", 9, INV), ("group_top", 0, INV), ("group_top", 3, INV), ("renormalise", 2, INV),
    ("scale", float("inf"), INV), ("scale", float("nan"), INV), ("reserved", 1, INV)])
def test_scoring_refusals(lib, field, value, status):
    cfg = rcd.make_config(10, 64, 64, 384, 1, 8, 64)
    sc = rcd.scoring("sigmoid", 8, 4)
    setattr(sc, field, value)
    assert lib.moe_route_scored(C.byref(cfg), C.byref(sc), FAKE, NUL, FAKE, FAKE, NUL) == status
    assert lib.moe_route_scored_backward(C.byref(cfg), C.byref(sc), FAKE, FAKE, FAKE, FAKE, NUL) == status


def test_route_scored_refusals(lib):
    sc = rcd.scoring("sigmoid")

    def fwd(cfg, s, *p):
        return lib.moe_route_scored(cfg and C.byref(cfg), s and C.byref(s), *p, NUL)
    cfg = rcd.make_config(10, 64, 64, 64, 1, 8, 64)
    assert fwd(None, sc, FAKE, NUL, FAKE, FAKE) == INV and fwd(cfg, None, FAKE, NUL, FAKE, FAKE) == INV
    for i in (0, 2, 3):
        p = [FAKE, NUL, FAKE, FAKE]
        p[i] = NUL
        assert fwd(cfg, sc, *p) == INV
    for i in range(4):
        p = [FAKE] * 4
        p[i] = NUL
        assert lib.moe_route_scored_backward(C.byref(cfg), C.byref(sc), *p, NUL) == INV
    assert fwd(rcd.make_config(10, 64, 64, 64, 1, 65, 64), sc, FAKE, NUL, FAKE, FAKE) == UNS
    assert fwd(rcd.make_config(10, 64, 64, 8, 1, 9, 64), sc, FAKE, NUL, FAKE, FAKE) == INV
    assert fwd(rcd.make_config(10, 64, 64, 2048, 1, 8, 64), sc, FAKE, NUL, FAKE, FAKE) == UNS
    assert fwd(rcd.make_config(-1, 64, 64, 64, 1, 8, 64), sc, FAKE, NUL, FAKE, FAKE) == INV
    # two groups of 4 hold fewer than 9 experts; 128 groups
    assert fwd(rcd.make_config(10, 64, 64, 64, 1, 9, 64), rcd.scoring("sigmoid", 16, 2), FAKE, NUL, FAKE, FAKE) == INV
    assert fwd(rcd.make_config(10, 64, 64, 256, 1, 8, 64), rcd.scoring("sigmoid", 128, 64), FAKE, NUL, FAKE, FAKE) == UNS
    assert fwd(rcd.make_config(0, 64, 64, 64, 1, 8, 64), sc, NUL, NUL, NUL, NUL) == OK


def test_quantize_refusals(lib):
    def q(rows=4, cols=256, x=FAKE, ld=256, dt=abi.MOE_BF16, block=1, tr=0, out=FAKE, s=FAKE):
        return lib.moe_quantize(rows, cols, x, ld, dt, block, tr, out, s, NUL)
    assert q(rows=-1) == INV and q(cols=-1) == INV and q(ld=255) == INV and q(dt=2) == INV and q(block=64) == INV
    assert q(tr=2) == INV and q(x=NUL) == INV and q(out=NUL) == INV and q(s=NUL) == INV
    assert q(x=C.c_void_p(0x100001)) == INV and q(x=C.c_void_p(0x100002), dt=abi.MOE_F32) == INV
    assert q(out=C.c_void_p(0x100008)) == INV and q(s=C.c_void_p(0x100002)) == INV
    assert q(rows=(1 << 30) + 1) == UNS and q(rows=1 << 20, cols=1 << 20, ld=1 << 20) == UNS
    assert q(rows=0, x=NUL, out=NUL, s=NUL) == OK and q(cols=0, x=NUL, out=NUL, s=NUL) == OK


def gemm(**kw):
    f = dict(M=64, N=96, K=256, a=0x100000, lda=256, a_scale=0x100000, a_scale_ld=64, b=0x100000, ldb=256,
             b_scale=0x100000, b_scale_ld=2, c=0x100000, ldc=96, b_block_rows=128, out_dtype=abi.MOE_BF16, reserved=0)
    f.update(kw)
    return abi.MoeQuantGemm(**f)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), INV), (dict(N=-1), INV), (dict(K=-128), INV), (dict(K=100), INV), (dict(lda=128), INV),
    (dict(ldb=240), INV), (dict(lda=264), UNS), (dict(ldb=264), UNS), (dict(a_scale_ld=63), INV), (dict(b_scale_ld=1), INV),
    (dict(b_block_rows=1), INV), (dict(b_block_rows=64), INV), (dict(ldc=95), INV), (dict(out_dtype=2), INV),
    (dict(reserved=1), INV), (dict(a=0), INV), (dict(b=0), INV), (dict(c=0), INV), (dict(a_scale=0), INV),
    (dict(b_scale=0), INV), (dict(a=0x100008), INV), (dict(b=0x100001), INV), (dict(c=0x100001), INV),
    (dict(c=0x100002, out_dtype=abi.MOE_F32), INV), (dict(a_scale=0x100002), INV),
    (dict(K=1 << 24, lda=1 << 24, ldb=1 << 24, b_scale_ld=1 << 17), UNS), (dict(lda=1 << 24), UNS),
    (dict(M=1 << 20, a_scale_ld=1 << 20, N=1 << 20, ldc=1 << 20), UNS),
    (dict(M=(1 << 30) + 1, a_scale_ld=1 << 31), UNS)])
def test_gemm_refusals(lib, kw, status):
    assert lib.moe_gemm_quant(C.byref(gemm(**kw)), FAKE, 1 << 40, NUL) == status


def test_gemm_workspace(lib):
    n = C.c_size_t(0)
    assert lib.moe_gemm_quant_ws_bytes(None, C.byref(n)) == INV
    assert lib.moe_gemm_quant_ws_bytes(C.byref(gemm()), None) == INV
    assert lib.moe_gemm_quant(None, FAKE, 0, NUL) == INV
    # few tiles, a long K: shared K needs a workspace
    g = gemm(M=128, N=256, K=8192, lda=8192, ldb=8192, a_scale_ld=128, b_scale_ld=64, ldc=256)
    assert lib.moe_gemm_quant_ws_bytes(C.byref(g), C.byref(n)) == OK and n.value > 0 and n.value % 256 == 0
    assert lib.moe_gemm_quant(C.byref(g), NUL, 0, NUL) == WS
    assert lib.moe_gemm_quant(C.byref(g), FAKE, n.value - 1, NUL) == WS
    assert lib.moe_gemm_quant(C.byref(g), C.c_void_p(0x100010), n.value, NUL) == WS
    assert lib.moe_gemm_quant(C.byref(gemm(M=0, a=0, c=0)), NUL, 0, NUL) == OK
    assert lib.moe_gemm_quant(C.byref(gemm(N=0, b=0, c=0)), NUL, 0, NUL) == OK


def test_experts_refusals(lib):
    def call(cfg, xs=FAKE, off=FAKE, w=None, out=FAKE, ws=FAKE, n=1 << 40):
        w = w or abi.MoeQuantExperts(*([0x100000] * 6))
        return lib.moe_experts_dropless_quant(C.byref(cfg), xs, off, C.byref(w), out, ws, n, NUL)
    cfg = rcd.make_config(64, 64, 256, 8, 1, 2, 128)
    n = rcd.experts_dropless_quant_ws_bytes(cfg)
    assert n % 256 == 0 and n >= 128 * (256 + 128 + 8 + 4)
    assert call(cfg, off=NUL) == INV and call(cfg, xs=NUL) == INV and call(cfg, out=NUL) == INV
    for i in range(6):
        p = [0x100000] * 6
        p[i] = 0
        assert call(cfg, w=abi.MoeQuantExperts(*p)) == INV
    assert call(cfg, w=abi.MoeQuantExperts(0x100008, *([0x100000] * 5))) == INV
    assert call(cfg, ws=NUL) == WS and call(cfg, n=n - 1) == WS and call(cfg, ws=C.c_void_p(0x100080)) == WS
    assert call(rcd.make_config(64, 64, 192, 8, 1, 2, 128)) == UNS
    assert call(rcd.make_config(64, 64, 256, 8, 1, 2, 64)) == UNS
    assert call(rcd.make_config(64, 64, 256, 8, 1, 2, 128, dtype="f32")) == UNS
    assert call(rcd.make_config(64, 64, 256, 8, 1, 0, 128)) == INV
    assert call(rcd.make_config(0, 64, 256, 8, 1, 2, 128), xs=NUL, out=NUL, ws=NUL, n=0) == OK
    assert lib.moe_experts_dropless_quant(C.byref(cfg), FAKE, FAKE, None, FAKE, FAKE, n, NUL) == INV
    assert lib.moe_experts_dropless_quant_ws_bytes(C.byref(cfg), None) == INV


def test_binding_refuses_tensors_the_kernels_cannot_take():
    # checked before a pointer is taken: CPU tensors are enough
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    for bad in (x, x.double(), x[0]):
        with pytest.raises(ValueError):
            rcd.quantize(bad)
    cfg = rcd.make_config(4, 64, 64, 16, 1, 2, 64)
    with pytest.raises(ValueError):
        rcd.route_scored(cfg, rcd.scoring(), torch.zeros((4, 16)))
    with pytest.raises(ValueError):
        rcd.scoring("relu")
    q = torch.zeros((4, 256), dtype=torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        rcd.gemm_quant(q, torch.zeros((2, 4)), q, torch.zeros((1, 2)))
    with pytest.raises(ValueError):
        rcd.experts_dropless_quant(rcd.make_config(4, 64, 128, 4, 1, 1, 128), x, None, None, None, None)


def test_forward_quant_refusals(lib):
    assert C.sizeof(abi.MoeQuantWeights) == 16 * 8
    sc = rcd.scoring("sigmoid", 4, 2)

    def call(cfg, scoring=sc, w=None, x=FAKE, y=FAKE, taps=None, ws=FAKE, n=1 << 40):
        w = w or weights()
        return lib.moe_forward_dropless_quant(C.byref(cfg), scoring and C.byref(scoring), C.byref(w), x, y,
                                              taps and C.byref(taps), NUL, ws, n, NUL)

    def weights(**kw):
        w = abi.MoeQuantWeights(experts=abi.MoeQuantExperts(*([0x100000] * 6)))
        for name, _ in w._fields_:
            if name != "experts":
                setattr(w, name, kw.get(name, 0x100000))
        return w
    shape = dict(T=64, d_model=256, d_latent=128, n_experts=16, n_pools=1, top_k=2, d_ff=128, n_shared=2, d_ff_shared=128)
    cfg = rcd.make_config(**shape)
    n = C.c_size_t(0)
    assert lib.moe_forward_dropless_quant_ws_bytes(C.byref(cfg), C.byref(n)) == OK and n.value % 256 == 0
    # quantised x and the joined operand, the dispatched rows and the experts' outputs among it
    assert n.value >= 64 * 256 + 64 * 384 + 2 * 128 * 128 * 2
    assert lib.moe_forward_dropless_quant_ws_bytes(C.byref(cfg), None) == INV
    for name in ("q_latent", "s_latent", "w_router", "q_output", "s_output", "q_shared_gate", "s_shared_up"):
        assert call(cfg, w=weights(**{name: 0})) == INV, name
    assert call(cfg, w=weights(q_output=0x100008)) == INV
    assert call(cfg, scoring=None) == INV and call(cfg, x=NUL) == INV and call(cfg, y=C.c_void_p(0x100002)) == INV
    assert call(cfg, taps=abi.MoeDroplessTaps(z=0x100008)) == INV
    assert call(cfg, ws=NUL) == WS and call(cfg, n=n.value - 1) == WS and call(cfg, ws=C.c_void_p(0x100010)) == WS
    for field, value, status in (("d_model", 320, UNS), ("d_latent", 192, UNS), ("d_ff_shared", 64, UNS),
                                 ("n_experts", 18, UNS), ("top_k", 17, INV)):
        bad = rcd.make_config(**{**shape, field: value})
        assert call(bad, scoring=rcd.scoring("sigmoid")) == status, field
    assert call(rcd.make_config(**shape, dtype="f32")) == UNS


def test_more_threads_than_a_launch_has(lib):
    # one column in 2^30 rows: 2^25 workgroups of 32 rows; 2^26 tokens of 64 threads
    for rows in (1 << 30, (1 << 29) - 31):
        assert lib.moe_quantize(rows, 1, FAKE, 1, abi.MOE_BF16, 1, 0, FAKE, FAKE, NUL) == UNS
    sc = rcd.scoring("sigmoid")
    cfg = rcd.make_config((1 << 26) - 3, 64, 64, 1, 1, 1, 64)
    assert lib.moe_route_scored(C.byref(cfg), C.byref(sc), FAKE, NUL, FAKE, FAKE, NUL) == UNS
    assert lib.moe_route_scored_backward(C.byref(cfg), C.byref(sc), FAKE, FAKE, FAKE, FAKE, NUL) == UNS
