"""Pins of the e4m3 block oracle (CPU only)."""
import numpy as np
import torch

from oracle import block_quant as bq


def test_magnitudes_are_torchs():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    assert np.array_equal(t, bq.DECODE, equal_nan=True)


def test_rounding_of_every_midpoint_and_its_neighbours():
    m = bq.MAGNITUDES
    mid = (m[1:] + m[:-1]) / 2
    even = np.where(np.arange(1, 127) % 2 == 0, m[1:], m[:-1])
    assert np.array_equal(bq.round_e4m3(mid), even)
    assert np.array_equal(bq.round_e4m3(-mid), -even)
    assert np.array_equal(bq.round_e4m3(np.nextafter(mid, 1e9)), m[1:])
    assert np.array_equal(bq.round_e4m3(np.nextafter(mid, 0)), m[:-1])
    assert np.array_equal(bq.round_e4m3(m), m)


def test_blocks_scales_and_padding():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((130, 200))
    q, s = bq.quantize(x)
    assert q.shape == (130, 256) and s.shape == (130, 2) and (q[:, 200:] == 0).all()
    assert np.allclose(s[7, 1], np.abs(x[7, 128:]).max() / 448)
    q, s = bq.quantize(x, 128)
    assert s.shape == (2, 2) and np.allclose(s[1, 0], np.abs(x[128:, :128]).max() / 448)
    assert np.abs(q).max() == 448
    qt, st = bq.quantize(x, 128, transpose=True)  # the transpose of square blocks is the transposed result
    assert qt.shape == (200, 256) and np.array_equal(qt[:, :130], q[:, :200].T) and np.array_equal(st, s.T)
    v = bq.values(*bq.quantize(x), 1)[:, :200]
    # half a step of 2^-3 of a normal value's power of two, or half the smallest subnormal step
    amax = np.repeat(np.abs(np.pad(x, ((0, 0), (0, 56)))).reshape(130, 2, 128).max(2), 128, 1)[:, :200]
    assert (np.abs(v - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * amax / 448)).all()


def test_zero_and_tiny_blocks():
    q, s = bq.quantize(np.zeros((2, 128)))
    assert (q == 0).all() and (s == bq.TINY / 448).all()
    q, _ = bq.quantize(np.full((1, 128), 2.0 ** -120))
    assert (q == 0).all()
