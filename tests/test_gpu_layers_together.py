"""Linear layers, the dropless branch, orthogonalised updates and the form for
a few tokens together, as a training step and the decoding step after it use
them."""
import numpy as np
import pytest
import torch

import routing_capacity_dispatch_amd as rcd
from gpu_common import dev, say
from oracle import newton_schulz as ns
from test_gpu_few import np64, verify, weights

pytestmark = pytest.mark.gpu


def test_train_then_decode():
    d = dev()
    T, D, L, E, k, F = 96, 320, 256, 8, 2, 256
    w = {n: t.to(d) for n, t in weights(D, L, E, F, 0, 0, 1).items()}
    gen = torch.Generator().manual_seed(2)
    x = torch.randn((T, D), generator=gen).to(torch.bfloat16).to(d)
    dy = torch.randn((T, D), generator=gen).to(torch.bfloat16).to(d)
    cfg = rcd.make_config(T, D, L, E, 1, k, F, 0, 0, 1)
    say("train", T, D, L, E, k, F)
    # forward: latent layer, router layer in fp32, dropless experts, up-projection added to the input
    z = rcd.linear(x, w["w_latent"])
    logits = rcd.linear(z, w["w_router"], out_dtype=torch.float32)
    idx, gates = rcd.route(cfg, logits, w["router_bias"])
    sent = rcd.dispatch_dropless(cfg, idx, z)
    o = rcd.experts_dropless(cfg, sent["xs"], sent["expert_offsets"], w["w_gate"], w["w_up"], w["w_down"])
    lat = rcd.combine_dropless(cfg, o, sent["row_of"], gates)
    y = rcd.linear(lat, w["w_up_proj"], residual=x)
    # the same layer in one call
    whole, _, _ = rcd.forward_dropless(cfg, w, x)
    a, b = (y.double() - x.double()), whole.double()
    assert float(((a - b).abs().amax(1) / b.abs().amax(1)).max()) <= 2e-2 + 2.0 ** -6
    # backward
    dlat, dup, _ = rcd.linear_backward(dy, lat, w["w_up_proj"], bias=False)
    dg, do = rcd.combine_backward_dropless(cfg, o, sent["row_of"], gates, dlat)
    dxs, dw = rcd.experts_backward_dropless(cfg, sent["xs"], sent["expert_offsets"], w["w_gate"], w["w_up"],
                                            w["w_down"], do)
    dz = rcd.dispatch_backward_dropless(cfg, sent["row_of"], dxs)
    dl = rcd.route_backward(cfg, idx, gates, dg)
    dzr, drouter, _ = rcd.linear_backward(dl, z, w["w_router"], bias=False)
    dx, dlatent, _ = rcd.linear_backward((dz.float() + dzr.float()).to(torch.bfloat16), x, w["w_latent"], bias=False)
    grads = dict(w_up_proj=dup, w_gate=dw[0], w_up=dw[1], w_down=dw[2], w_router=drouter, w_latent=dlatent)
    # the dense layers' gradients against 64 bits, from the same incoming ones
    for got, l, r in ((dup, dy, lat), (dlatent, (dz.float() + dzr.float()).to(torch.bfloat16), x)):
        ref = np64(l).T @ np64(r)
        tol = (T + 8) * 2.0 ** -24 * (np.abs(np64(l)).T @ np.abs(np64(r)))
        assert (np.abs(np64(got) - ref) <= tol + 2.0 ** -8 * (np.abs(ref) + tol)).all()
    # update: orthogonalised, in one call for all experts of a kind
    new = dict(w)
    for n, g in grads.items():
        up = rcd.orthogonalize(g, scale=0.2)
        mats = g if g.dim() == 3 else g[None]
        for i in (0, len(mats) - 1):
            ref = ns.exact(np64(mats[i]), scale=0.2)
            got = np64(up if g.dim() == 2 else up[i])
            norm = np.linalg.norm(ref)
            assert np.linalg.norm(got - ref) <= (2.9e-3 + 2.0 ** -8) * norm, n
        new[n] = (w[n].float() - 0.1 * up.float()).to(torch.bfloat16)
    assert not torch.equal(new["w_gate"], w["w_gate"])
    # decode four tokens with the new weights
    few = rcd.ForwardFew(rcd.make_config(4, D, L, E, 1, k, F, 0, 0, 1), new, d, taps=True)
    few(x[:4], x[:4])
    torch.cuda.synchronize()
    verify(few, {n: t.cpu() for n, t in new.items()}, x[:4].cpu(), x[:4].cpu(), 4, E, k, 0)
