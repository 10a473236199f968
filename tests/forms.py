"""Which kernels a call of the linear layers or of orthogonalize takes, by the
library's own rule on the host (nothing is enqueued, no GPU needed)."""
import ctypes as C

from routing_capacity_dispatch_amd import abi

TILES = {1: "big", 2: "small", 3: "mid", 4: "deep", 5: "stream"}
FAKE = 0x100000


def _ask(name, args, kind):
    f = getattr(abi.load(), name)
    f.restype, f.argtypes = C.c_int, [C.POINTER(kind)]
    bits = f(C.byref(args))
    assert bits >= 0
    return bits


def linear(M, N, K, shift=(0, 0), pad=(0, 0)):
    """x and w start `shift` values past 16 bytes, their rows are K + `pad` values apart."""
    b = _ask("moe_linear_form", abi.MoeLinearArgs(
        M, N, K, FAKE + 2 * shift[0], K + pad[0], FAKE + 2 * shift[1], K + pad[1], None, None, 0, FAKE, N, None, 0, 0, 1, 1,
        0), abi.MoeLinearArgs)
    return " ".join([TILES[b & 7]] + [w for i, w in ((3, "registers"), (4, "copy-x"), (5, "copy-w"), (6, "shared"))
                                      if b >> i & 1])


def backward(M, N, K, act="silu", fp32=False, shift=(0, 0), pad=(0, 0), dx=True, dw=True, pad_dy=0):
    """Likewise; dy starts on 16 bytes."""
    b = _ask("moe_linear_backward_form", abi.MoeLinearGrad(
        M, N, K, FAKE, N + pad_dy, FAKE, N, FAKE + 2 * shift[0], K + pad[0], FAKE + 2 * shift[1], K + pad[1],
        FAKE if dx else None, K, FAKE if dw else None, K, FAKE, abi.ACTS[act], 0 if fp32 else 1, 0), abi.MoeLinearGrad)
    return " ".join([TILES[b & 7]] + [w for i, w in ((3, "registers"), (4, "copy-x"), (5, "copy-w"), (6, "shared-dw"),
                                                     (7, "shared-dx"), (8, "d")) if b >> i & 1])


def orthogonalize(B, M, N):
    """Tiles of A and B, of X, and 'split' with both fp16 numbers in the products."""
    co = (C.c_float * 3)(1.5, -0.5, 0.0)
    b = _ask("moe_orthogonalize_form", abi.MoeOrthoArgs(
        B, M, N, FAKE, N, M * N, FAKE, N, M * N, C.cast(co, C.POINTER(C.c_float)), 1, 0, 0.0, 1.0, 0), abi.MoeOrthoArgs)
    return " ".join([TILES[b & 7], TILES[b >> 3 & 7]] + ["split"] * (b >> 6 & 1))

# Sizes that the tests of the kernels rely on, with the form that they take (test_forms.py holds them to it).
# x and w: (shift, pad) of each.
ALIGNED, ODD = (0, 8), (1, 3)
LINEAR = [
    ("stream", (13, 700, 900), ODD, ODD), ("stream", (190, 200, 136), ALIGNED, ALIGNED),
    ("deep", (50, 6200, 512), ALIGNED, ALIGNED), ("deep registers", (50, 6203, 517), ODD, ODD),
    ("deep registers", (70, 6200, 512), ALIGNED, ODD),
    ("deep shared", (100, 300, 9000), ALIGNED, ALIGNED), ("deep registers shared", (101, 299, 9001), ODD, ODD),
    ("mid", (1500, 1700, 200), ALIGNED, ALIGNED), ("mid copy-x copy-w", (1501, 1699, 203), ODD, ODD),
    ("mid copy-x", (1500, 1700, 200), ODD, ALIGNED), ("mid copy-w", (1500, 1700, 200), ALIGNED, ODD),
    ("mid shared", (1500, 1300, 8000), ALIGNED, ALIGNED), ("mid copy-x copy-w shared", (1499, 1301, 8005), ALIGNED, ODD),
    ("small", (3000, 2100, 200), ALIGNED, ALIGNED), ("small copy-x copy-w", (3001, 2099, 203), ODD, ODD),
    ("small copy-w", (3000, 2100, 200), ALIGNED, ODD),
    ("small shared", (2000, 2100, 8000), ALIGNED, ALIGNED), ("small copy-x copy-w shared", (2001, 2101, 8007), ODD, ODD),
    ("big", (3500, 3601, 200), ALIGNED, ALIGNED), ("big copy-x copy-w", (3501, 3599, 203), ODD, ODD),
    ("big copy-x", (3500, 3601, 200), ODD, ALIGNED), ("big shared", (5100, 2550, 32760), ALIGNED, ALIGNED)]
# act, dy in fp32, (M, N, K), x and w, values between dy's rows
BACKWARD = [
    ("deep d", "gelu", True, (1000, 300, 264), ALIGNED, ALIGNED, 0),
    ("deep", "none", False, (264, 600, 1000), ALIGNED, ALIGNED, 8),
    ("deep registers d", "silu", False, (400, 299, 263), ODD, ODD, 3),
    ("deep registers", "none", False, (400, 304, 263), ODD, ALIGNED, 8),
    ("deep shared-dw d", "relu", True, (1500, 300, 400), ALIGNED, ALIGNED, 0),
    ("deep registers shared-dw d", "silu", False, (2001, 131, 262), ODD, ODD, 5),
    ("deep registers shared-dw", "none", False, (3000, 200, 300), ODD, ODD, 0),
    ("deep registers shared-dx d", "gelu", True, (500, 3001, 299), ODD, ODD, 0),
    ("mid shared-dw d", "silu", False, (2000, 700, 1008), ALIGNED, ALIGNED, 0),
    ("mid shared-dw", "none", False, (2000, 704, 1008), ALIGNED, ALIGNED, 0),
    ("mid copy-x copy-w d", "relu", True, (900, 1101, 1300), ODD, ODD, 0),
    ("mid copy-x shared-dw d", "gelu", False, (2000, 700, 1008), ODD, ALIGNED, 1),
    ("small d", "silu", False, (2048, 2048, 2048), ALIGNED, ALIGNED, 0),
    ("small", "none", False, (2050, 2056, 2040), ALIGNED, ALIGNED, 8),
    ("small copy-x copy-w shared-dw d", "gelu", True, (2000, 1601, 1700), ODD, ODD, 0),
    ("small copy-x copy-w shared-dw d", "none", False, (20000, 255, 257), ODD, ODD, 0),
    ("big d", "silu", False, (1024, 1280, 5632), ALIGNED, ALIGNED, 0),
    ("big", "none", False, (1024, 1280, 5632), ALIGNED, ALIGNED, 0),
    ("big copy-x copy-w d", "gelu", True, (1000, 1279, 5601), ODD, ODD, 0),
    ("big shared-dw d", "relu", False, (7000, 2041, 3576), ALIGNED, ALIGNED, 0),
    ("big copy-w shared-dw", "none", False, (6999, 2040, 3584), ALIGNED, ODD, 8)]
ORTHOGONALIZE = [
    ("deep deep split", (3, 200, 700)), ("deep mid split", (20, 200, 500)), ("mid small split", (50, 200, 300)),
    ("small small split", (100, 300, 200)), ("deep deep", (2, 700, 800)), ("deep mid", (3, 1000, 1100)),
    ("deep mid", (3, 1100, 1000)), ("mid mid", (1, 2000, 2000)), ("mid small", (6, 1000, 1000)),
    ("small small", (64, 512, 513)), ("small big", (64, 1020, 1030)), ("small big", (64, 1030, 1020)),
    ("big small", (7, 2000, 2040)), ("big big", (7, 2000, 2300)), ("big big", (7, 2300, 2000)),
    ("small big", (8, 2048, 4096)), ("small big", (9, 4090, 2000))]
