"""The sizes that stand for a kernel in the GPU tests take that kernel (CPU
only): a change of the rules that moves one fails here."""
import pytest

import forms


@pytest.mark.parametrize("form,size,x,w", forms.LINEAR)
def test_linear(form, size, x, w):
    assert forms.linear(*size, shift=(x[0], w[0]), pad=(x[1], w[1])) == form


@pytest.mark.parametrize("form,act,fp32,size,x,w,pad_dy", forms.BACKWARD)
def test_backward(form, act, fp32, size, x, w, pad_dy):
    assert forms.backward(*size, act=act, fp32=fp32, shift=(x[0], w[0]), pad=(x[1], w[1]), pad_dy=pad_dy) == form


@pytest.mark.parametrize("form,size", forms.ORTHOGONALIZE)
def test_orthogonalize(form, size):
    assert forms.orthogonalize(*size) == form


def test_every_tile_is_there():
    for table in (forms.LINEAR, forms.BACKWARD):
        kinds = {c[0].split()[0] for c in table}
        assert kinds >= {"deep", "mid", "small", "big"}
        assert {c[0].split()[0] for c in table if "shared" in c[0]} >= {"deep", "mid", "small", "big"}
    for i in (0, 1):
        assert {c[0].split()[i] for c in forms.ORTHOGONALIZE} == {"deep", "mid", "small", "big"}
