"""Newton-Schulz iteration that moves a matrix's singular values near 1
(moe_orthogonalize), in fp64: from its definition, and once more with the
roundings that the GPU's arithmetic makes."""
import numpy as np

USUAL = (3.4445, -4.7750, 2.0315)


def start(g, eps):
    x = np.asarray(g, dtype=np.float64)
    x = x.T if x.shape[0] > x.shape[1] else x
    n = np.sqrt((x * x).sum()) + eps
    return x / n if n > 0 else np.zeros_like(x)


def exact(g, steps=5, coeffs=USUAL, eps=1e-7, scale=1.0):
    x = start(g, eps)
    for a, b, c in (coeffs if isinstance(coeffs[0], tuple) else [coeffs] * steps):
        p = x @ x.T
        x = a * x + (b * p + c * (p @ p)) @ x
    return scale * (x.T if np.shape(g)[0] > np.shape(g)[1] else x)


def by_singular_values(g, steps=5, coeffs=USUAL, eps=1e-7, scale=1.0):
    """The same through the singular value decomposition."""
    x = np.asarray(g, dtype=np.float64)
    u, s, v = np.linalg.svd(x, full_matrices=False)
    s = s / (np.sqrt((x * x).sum()) + eps)
    for a, b, c in (coeffs if isinstance(coeffs[0], tuple) else [coeffs] * steps):
        s = a * s + b * s ** 3 + c * s ** 5
    return scale * (u * s) @ v


def fp16(x):
    """x in fp16, scaled by the power of two that takes its largest value to half of fp16's range."""
    most = np.abs(x).max()
    e = int(np.floor(np.log2(32768.0 / most))) if most > 0 else 0
    return np.ldexp(np.ldexp(x, e).astype(np.float16).astype(np.float64), -e)


def held(x):
    h = fp16(x)
    return h + fp16(x - h)


def weights_of_low(coeffs):
    """The share of B's diagonal that X's second number is given in every step: 1 over the most that the later steps
    multiply a singular value by."""
    m, gains = 1.0, []
    for a, b, c in coeffs:
        t = np.linspace(0.0, m * m, 20001)
        p = np.abs(a + b * t + c * t * t)
        gains.append(p.max())
        m = (np.sqrt(t) * p).max() * (1 + 1 / 64)
    return [1 / max(np.prod(gains[k + 1:]), 1.0) for k in range(len(gains))]


def emulated(g, steps=5, coeffs=USUAL, eps=1e-7, scale=1.0):
    """X in two fp16 numbers; the products take the first (both where the
    smaller side is below 256), and A and B off their diagonals, in fp16; sums
    exact."""
    x = held(start(g, eps))
    split = min(x.shape) < 256
    coeffs = coeffs if isinstance(coeffs[0], tuple) else [coeffs] * steps
    for (a, b, c), w in zip(coeffs, [1.0] * len(coeffs) if split else weights_of_low(coeffs)):
        h = fp16(x)
        low = fp16(x - h) if split else np.zeros_like(x)
        p = h @ h.T + h @ low.T + low @ h.T
        d = np.diag(p).copy()
        r = fp16(p - np.diag(d))
        p2 = r @ r + (d[:, None] + d[None]) * r + np.diag(d * d)
        q = b * (r + np.diag(d)) + c * p2
        e = np.diag(q).copy()
        x = (a + e[:, None]) * h + (a + w * e[:, None]) * (x - h) + fp16(q - np.diag(e)) @ (h + low)
        x = held(x)
    return scale * (x.T if np.shape(g)[0] > np.shape(g)[1] else x)
