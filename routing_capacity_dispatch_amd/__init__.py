"""Pooled-wave capacity-dispatch MoE branch (forward, and the backward of its
routed path) for MI355X / gfx950.

Thin torch binding over the C ABI in include/moe.h (libmoe.so).  torch only
provides device memory and the current stream; every step of the branch runs
in the HIP kernels of the library.  The same names as the C entry points:
route, dispatch, experts, combine, forward, their *_backward transposes and
BackwardRouted (moe_backward_routed), plus make_config / plan; and the layers
around it: linear and linear_backward, orthogonalize (the update made of a
weight's gradient) and ForwardFew (at most 16 tokens).
"""
from __future__ import annotations

import ctypes as C
import functools
from typing import Dict, Optional

import torch

from . import abi

__all__ = ["make_config", "plan", "route", "dispatch", "experts", "combine", "forward",
           "dispatch_dropless", "experts_dropless", "combine_dropless", "forward_dropless",
           "combine_backward", "experts_backward", "dispatch_backward", "route_backward",
           "combine_backward_dropless", "experts_backward_dropless", "dispatch_backward_dropless",
           "BackwardRouted", "scoring", "route_scored", "route_scored_backward", "quantize", "gemm_quant",
           "experts_dropless_quant", "quantize_weights", "ForwardDroplessQuant", "linear", "linear_backward",
           "orthogonalize", "ForwardFew", "library", "MoeError"]

MoeError = abi.MoeError
_DT = {"f32": abi.MOE_F32, "bf16": abi.MOE_BF16, torch.float32: abi.MOE_F32,
       torch.bfloat16: abi.MOE_BF16}


def library():
    return abi.load()


def make_config(T, d_model, d_latent, n_experts, n_pools, top_k, d_ff, n_shared=0,
                d_ff_shared=0, n_waves=3, dtype="bf16", send_cap=(11, 10), recv_cap=(23, 20),
                cap_send_rows=0, cap_recv_rows=0) -> abi.MoeConfig:
    # in the order of the fields
    return abi.MoeConfig(T, d_model, d_latent, n_experts, n_pools, top_k, d_ff, n_shared, d_ff_shared, n_waves,
                         send_cap[0], send_cap[1], recv_cap[0], recv_cap[1], cap_send_rows, cap_recv_rows, _DT[dtype], 0)


def config_of(w, **over) -> abi.MoeConfig:
    """Config from any object with the workload attribute names."""
    f = dict(T=w.T, d_model=w.d_model, d_latent=w.d_latent, n_experts=w.n_experts,
             n_pools=w.n_pools, top_k=w.top_k, d_ff=w.d_ff, n_shared=w.n_shared,
             d_ff_shared=w.d_ff_shared, n_waves=w.n_waves, dtype=w.dtype,
             send_cap=tuple(w.send_cap), recv_cap=tuple(w.recv_cap),
             cap_send_rows=getattr(w, "cap_send_rows", 0),
             cap_recv_rows=getattr(w, "cap_recv_rows", 0))
    f.update(over)
    return make_config(**f)


def plan(cfg: abi.MoeConfig) -> Dict[str, int]:
    p = abi.MoePlan()
    abi.check("moe_make_plan", library().moe_make_plan(C.byref(cfg), C.byref(p)))
    return p.as_dict()


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(device=None):
    return C.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _tdt(cfg):
    return torch.bfloat16 if cfg.dtype == abi.MOE_BF16 else torch.float32


def _ws(nbytes, device):
    # 256-byte aligned: torch's caching allocator returns 512-byte aligned blocks
    t = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
    assert t.data_ptr() % 256 == 0
    return t


def route(cfg, logits: torch.Tensor, bias: Optional[torch.Tensor] = None, out=None):
    T, k = cfg.T, cfg.top_k
    dev = logits.device
    topk = out["topk_idx"] if out else torch.empty((T, k), dtype=torch.int32, device=dev)
    gates = out["gates"] if out else torch.empty((T, k), dtype=torch.float32, device=dev)
    abi.check("moe_route", library().moe_route(
        C.byref(cfg), _ptr(logits), _ptr(bias), _ptr(topk), _ptr(gates), _stream(dev)))
    return topk, gates


def router_bias_ws_bytes(cfg, n_bins: int) -> int:
    n = C.c_size_t(0)
    abi.check("moe_router_bias_ws_bytes", library().moe_router_bias_ws_bytes(C.byref(cfg), n_bins, C.byref(n)))
    return int(n.value)


def router_bias_update(cfg, logits: torch.Tensor, n_bins: int, with_hist: bool = False, ws=None, out=None):
    """Next step's zero-mean router bias [E] fp32 from this step's logits
    [T][E] fp32 (moe_router_bias_update).  With with_hist, also the
    per-expert counts [E][n_bins] int32 and ranges [E][2] fp32."""
    dev = logits.device
    E = cfg.n_experts
    bias = out if out is not None else torch.empty(E, dtype=torch.float32, device=dev)
    hist = torch.empty((E, n_bins), dtype=torch.int32, device=dev) if with_hist else None
    lohi = torch.empty((E, 2), dtype=torch.float32, device=dev) if with_hist else None
    if ws is None:
        ws = _ws(router_bias_ws_bytes(cfg, n_bins), dev)
    abi.check("moe_router_bias_update", library().moe_router_bias_update(
        C.byref(cfg), _ptr(logits), n_bins, _ptr(bias), _ptr(hist), _ptr(lohi), _ptr(ws), ws.numel(),
        _stream(dev)))
    return (bias, hist, lohi) if with_hist else bias


class RouterBias:
    """moe_router_bias_update with its workspace and output allocated once:
    call it with each step's logits [T][E] fp32; it returns the next step's
    bias [E] fp32 (the same tensor every call)."""

    def __init__(self, cfg, n_bins: int, device):
        self.cfg, self.n_bins = cfg, n_bins
        self.ws = _ws(router_bias_ws_bytes(cfg, n_bins), device)
        self.bias = torch.empty(cfg.n_experts, dtype=torch.float32, device=device)

    def __call__(self, logits: torch.Tensor):
        return router_bias_update(self.cfg, logits, self.n_bins, ws=self.ws, out=self.bias)

    def profiled(self, logits: torch.Tensor, events):
        arr = (C.c_void_p * len(events))(*[C.c_void_p(e.cuda_event) for e in events])
        abi.check("moe_router_bias_update_profiled", library().moe_router_bias_update_profiled(
            C.byref(self.cfg), _ptr(logits), self.n_bins, _ptr(self.bias), None, None, _ptr(self.ws),
            self.ws.numel(), _stream(logits.device), arr, len(events)))
        return self.bias


def router_bias_stage_count() -> int:
    return library().moe_router_bias_stage_count()


def dispatch(cfg, topk_idx: torch.Tensor, z: torch.Tensor) -> Dict[str, torch.Tensor]:
    p = plan(cfg)
    dev = z.device
    T, k, W, P, E = cfg.T, cfg.top_k, cfg.n_waves, cfg.n_pools, cfg.n_experts
    out = dict(
        pools=torch.empty(p["pools_bytes"], dtype=torch.uint8, device=dev),
        pool_slot=torch.empty((T, k), dtype=torch.int32, device=dev),
        recv_slot=torch.empty((T, k), dtype=torch.int32, device=dev),
        bank_rows=torch.full((W, E, max(p["cap_recv"], 0)), -1, dtype=torch.int32, device=dev),
        pool_count=torch.empty((W, P), dtype=torch.int32, device=dev),
        expert_count=torch.empty((W, E), dtype=torch.int32, device=dev),
        counts=torch.empty(3, dtype=torch.int64, device=dev),
    )
    ws = _ws(p["dispatch_ws_bytes"], dev)
    abi.check("moe_dispatch", library().moe_dispatch(
        C.byref(cfg), _ptr(topk_idx), _ptr(z), _ptr(out["pools"]), _ptr(out["pool_slot"]),
        _ptr(out["recv_slot"]), _ptr(out["bank_rows"]), _ptr(out["pool_count"]),
        _ptr(out["expert_count"]), _ptr(out["counts"]), _ptr(ws), ws.numel(), _stream(dev)))
    out["plan"] = p
    return out


def dispatch_noalloc(cfg, topk_idx: torch.Tensor, z: torch.Tensor, out: Dict[str, torch.Tensor]):
    """moe_dispatch_noalloc into caller-provided outputs (the dict that
    dispatch() returns, or one shaped like it); allocates nothing."""
    abi.check("moe_dispatch_noalloc", library().moe_dispatch_noalloc(
        C.byref(cfg), _ptr(topk_idx), _ptr(z), _ptr(out["pools"]), _ptr(out["pool_slot"]),
        _ptr(out["recv_slot"]), _ptr(out["bank_rows"]), _ptr(out["pool_count"]),
        _ptr(out["expert_count"]), _ptr(out["counts"]), _stream(z.device)))
    return out


def dispatch_noalloc_scratch_bytes() -> int:
    return library().moe_dispatch_noalloc_scratch_bytes()


def pool_views(cfg, pools: torch.Tensor):
    """(rows [W, P, C_send, L], ids [W, P, C_send]) views of a pools buffer."""
    p = plan(cfg)
    W, P = cfg.n_waves, cfg.n_pools
    cs, blk = p["cap_send"], p["pool_block_bytes"]
    if cs == 0:
        return (torch.empty((W, P, 0, cfg.d_latent), dtype=_tdt(cfg), device=pools.device),
                torch.empty((W, P, 0), dtype=torch.int32, device=pools.device))
    b = pools.view(W, P, blk)
    rows = b[:, :, :p["ids_offset"]].view(_tdt(cfg)).view(W, P, cs, cfg.d_latent)
    ids = b[:, :, p["ids_offset"]:p["ids_offset"] + 4 * cs].view(torch.int32).view(W, P, cs)
    return rows, ids


def experts(cfg, pools, bank_rows, expert_count, w_gate, w_up, w_down, expert_out=None):
    p = plan(cfg)
    dev = pools.device
    if expert_out is None:
        expert_out = torch.empty(p["expert_out_bytes"], dtype=torch.uint8, device=dev)
    ws = _ws(p["experts_ws_bytes"], dev)
    abi.check("moe_experts", library().moe_experts(
        C.byref(cfg), _ptr(pools), _ptr(bank_rows), _ptr(expert_count), _ptr(w_gate),
        _ptr(w_up), _ptr(w_down), _ptr(expert_out), _ptr(ws), ws.numel(), _stream(dev)))
    return expert_out


def expert_out_view(cfg, expert_out: torch.Tensor):
    p = plan(cfg)
    n = cfg.n_waves * cfg.n_pools * p["cap_send"] * cfg.d_latent
    return expert_out.view(_tdt(cfg))[:n].view(cfg.n_waves, cfg.n_pools, p["cap_send"],
                                                 cfg.d_latent)


def combine(cfg, expert_out, topk_idx, pool_slot, recv_slot, gates, y_latent=None):
    dev = expert_out.device
    if y_latent is None:
        y_latent = torch.empty((cfg.T, cfg.d_latent), dtype=_tdt(cfg), device=dev)
    abi.check("moe_combine", library().moe_combine(
        C.byref(cfg), _ptr(expert_out), _ptr(topk_idx), _ptr(pool_slot), _ptr(recv_slot),
        _ptr(gates), _ptr(y_latent), _stream(dev)))
    return y_latent


class Forward:
    """Reusable forward call: weights, workspace and outputs bound once, so a
    timed loop only enqueues kernels."""

    def __init__(self, cfg, weights: Dict[str, torch.Tensor], device, taps=False):
        self.cfg = cfg
        self.p = plan(cfg)
        self.w = weights
        self.wstruct = abi.MoeWeights(**{n: _ptr(weights.get(n)) for n, _ in
                                         abi.MoeWeights._fields_})
        self.ws = _ws(self.p["forward_ws_bytes"], device)
        self.y = torch.empty((cfg.T, cfg.d_model), dtype=_tdt(cfg), device=device)
        self.counts = torch.empty(3, dtype=torch.int64, device=device)
        self.taps = None
        self.tap_t = {}
        if taps:
            T, k, E, W, P, L = cfg.T, cfg.top_k, cfg.n_experts, cfg.n_waves, cfg.n_pools, cfg.d_latent
            dt = _tdt(cfg)
            i32 = dict(dtype=torch.int32, device=device)
            self.tap_t = dict(
                logits=torch.empty((T, E), dtype=torch.float32, device=device),
                topk_idx=torch.empty((T, k), **i32),
                gates=torch.empty((T, k), dtype=torch.float32, device=device),
                pool_slot=torch.empty((T, k), **i32),
                recv_slot=torch.empty((T, k), **i32),
                pool_count=torch.empty((W, P), **i32),
                expert_count=torch.empty((W, E), **i32),
                bank_rows=torch.full((W, E, self.p["cap_recv"]), -1, **i32),
                z=torch.empty((T, L), dtype=dt, device=device),
                pools=torch.empty(self.p["pools_bytes"], dtype=torch.uint8, device=device),
                expert_out=torch.empty(self.p["expert_out_bytes"], dtype=torch.uint8, device=device),
                y_latent=torch.empty((T, L), dtype=dt, device=device),
            )
            self.taps = abi.MoeTaps(**{n: _ptr(t) for n, t in self.tap_t.items()})

    def __call__(self, x: torch.Tensor):
        lib = library()
        abi.check("moe_forward", lib.moe_forward(
            C.byref(self.cfg), C.byref(self.wstruct), _ptr(x), _ptr(self.y),
            C.byref(self.taps) if self.taps is not None else None, _ptr(self.counts),
            _ptr(self.ws), self.ws.numel(), _stream(x.device)))
        return self.y

    def profiled(self, x: torch.Tensor, events):
        """As __call__, recording torch.cuda.Event objects (enable_timing) at
        the stage boundaries on the current stream: len(events) ==
        stage count + 1."""
        lib = library()
        arr = (C.c_void_p * len(events))(*[C.c_void_p(e.cuda_event) for e in events])
        abi.check("moe_forward_profiled", lib.moe_forward_profiled(
            C.byref(self.cfg), C.byref(self.wstruct), _ptr(x), _ptr(self.y),
            C.byref(self.taps) if self.taps is not None else None, _ptr(self.counts),
            _ptr(self.ws), self.ws.numel(), _stream(x.device), arr, len(events)))
        return self.y


def stage_count() -> int:
    return library().moe_forward_stage_count()


def forward(cfg, weights: Dict[str, torch.Tensor], x: torch.Tensor, taps=False):
    """One forward call; returns (y, counts, taps-dict)."""
    f = Forward(cfg, weights, x.device, taps=taps)
    y = f(x)
    return y, f.counts, f.tap_t


# ---------------------------------------------------------------- dropless


def dispatch_dropless(cfg, topk_idx: torch.Tensor, z: torch.Tensor) -> Dict[str, torch.Tensor]:
    """Rows ordered by expert: xs [T*k, L], row_of [T, k], expert_offsets [E+1]."""
    p = plan(cfg)
    dev = z.device
    T, k, E = cfg.T, cfg.top_k, cfg.n_experts
    out = dict(
        xs=torch.empty((p["dropless_rows"], cfg.d_latent), dtype=_tdt(cfg), device=dev),
        row_of=torch.empty((T, k), dtype=torch.int32, device=dev),
        expert_offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
        counts=torch.empty(3, dtype=torch.int64, device=dev),
    )
    ws = _ws(p["dropless_dispatch_ws_bytes"], dev)
    abi.check("moe_dispatch_dropless", library().moe_dispatch_dropless(
        C.byref(cfg), _ptr(topk_idx), _ptr(z), _ptr(out["xs"]), _ptr(out["row_of"]),
        _ptr(out["expert_offsets"]), _ptr(out["counts"]), _ptr(ws), ws.numel(), _stream(dev)))
    out["plan"] = p
    return out


def experts_dropless(cfg, xs, expert_offsets, w_gate, w_up, w_down, expert_out=None):
    p = plan(cfg)
    dev = xs.device
    if expert_out is None:
        expert_out = torch.empty((p["dropless_rows"], cfg.d_latent), dtype=_tdt(cfg), device=dev)
    ws = _ws(p["dropless_experts_ws_bytes"], dev)
    abi.check("moe_experts_dropless", library().moe_experts_dropless(
        C.byref(cfg), _ptr(xs), _ptr(expert_offsets), _ptr(w_gate), _ptr(w_up), _ptr(w_down),
        _ptr(expert_out), _ptr(ws), ws.numel(), _stream(dev)))
    return expert_out


def combine_dropless(cfg, expert_out, row_of, gates, y_latent=None):
    dev = expert_out.device
    if y_latent is None:
        y_latent = torch.empty((cfg.T, cfg.d_latent), dtype=_tdt(cfg), device=dev)
    abi.check("moe_combine_dropless", library().moe_combine_dropless(
        C.byref(cfg), _ptr(expert_out), _ptr(row_of), _ptr(gates), _ptr(y_latent), _stream(dev)))
    return y_latent


class ForwardDropless:
    """Reusable dropless forward call (weights, workspace and outputs bound once).
    For at most 16 tokens ForwardFew is faster."""

    def __init__(self, cfg, weights: Dict[str, torch.Tensor], device, taps=False):
        self.cfg = cfg
        self.p = plan(cfg)
        self.w = weights
        self.wstruct = abi.MoeWeights(**{n: _ptr(weights.get(n)) for n, _ in
                                         abi.MoeWeights._fields_})
        self.ws = _ws(self.p["dropless_forward_ws_bytes"], device)
        self.y = torch.empty((cfg.T, cfg.d_model), dtype=_tdt(cfg), device=device)
        self.counts = torch.empty(3, dtype=torch.int64, device=device)
        self.taps = None
        self.tap_t = {}
        if taps:
            T, k, E, L = cfg.T, cfg.top_k, cfg.n_experts, cfg.d_latent
            n = self.p["dropless_rows"]
            dt = _tdt(cfg)
            i32 = dict(dtype=torch.int32, device=device)
            self.tap_t = dict(
                logits=torch.empty((T, E), dtype=torch.float32, device=device),
                topk_idx=torch.empty((T, k), **i32),
                gates=torch.empty((T, k), dtype=torch.float32, device=device),
                row_of=torch.empty((T, k), **i32),
                expert_offsets=torch.empty(E + 1, **i32),
                z=torch.empty((T, L), dtype=dt, device=device),
                xs=torch.empty((n, L), dtype=dt, device=device),
                expert_out=torch.empty((n, L), dtype=dt, device=device),
                y_latent=torch.empty((T, L), dtype=dt, device=device),
            )
            self.taps = abi.MoeDroplessTaps(**{n_: _ptr(t) for n_, t in self.tap_t.items()})

    def _taps_arg(self):
        return C.byref(self.taps) if self.taps is not None else None

    def __call__(self, x: torch.Tensor):
        abi.check("moe_forward_dropless", library().moe_forward_dropless(
            C.byref(self.cfg), C.byref(self.wstruct), _ptr(x), _ptr(self.y), self._taps_arg(),
            _ptr(self.counts), _ptr(self.ws), self.ws.numel(), _stream(x.device)))
        return self.y

    def profiled(self, x: torch.Tensor, events):
        arr = (C.c_void_p * len(events))(*[C.c_void_p(e.cuda_event) for e in events])
        abi.check("moe_forward_dropless_profiled", library().moe_forward_dropless_profiled(
            C.byref(self.cfg), C.byref(self.wstruct), _ptr(x), _ptr(self.y), self._taps_arg(),
            _ptr(self.counts), _ptr(self.ws), self.ws.numel(), _stream(x.device), arr,
            len(events)))
        return self.y


def dropless_stage_count() -> int:
    return library().moe_forward_dropless_stage_count()


def forward_dropless(cfg, weights: Dict[str, torch.Tensor], x: torch.Tensor, taps=False):
    """One dropless forward call; returns (y, counts, taps-dict)."""
    f = ForwardDropless(cfg, weights, x.device, taps=taps)
    y = f(x)
    return y, f.counts, f.tap_t


# ---------------------------------------------------------------- backward
def combine_backward(cfg, expert_out, topk_idx, pool_slot, recv_slot, gates, dy_latent,
                     d_gates=None, d_expert_out=None):
    """(d_gates [T, k] fp32, d_expert_out bytes) = transpose of combine."""
    p = plan(cfg)
    dev = dy_latent.device
    if d_gates is None:
        d_gates = torch.empty((cfg.T, cfg.top_k), dtype=torch.float32, device=dev)
    if d_expert_out is None:
        d_expert_out = torch.empty(p["expert_out_bytes"], dtype=torch.uint8, device=dev)
    abi.check("moe_combine_backward", library().moe_combine_backward(
        C.byref(cfg), _ptr(expert_out), _ptr(topk_idx), _ptr(pool_slot), _ptr(recv_slot),
        _ptr(gates), _ptr(dy_latent), _ptr(d_gates), _ptr(d_expert_out), _stream(dev)))
    return d_gates, d_expert_out


def experts_backward(cfg, pools, bank_rows, expert_count, w_gate, w_up, w_down, d_expert_out,
                     d_pool_rows=None, dw=None):
    """(d_pool_rows bytes, (dw_gate, dw_up, dw_down)) = transpose of experts."""
    p = plan(cfg)
    dev = pools.device
    if d_pool_rows is None:
        d_pool_rows = torch.empty(p["expert_out_bytes"], dtype=torch.uint8, device=dev)
    if dw is None:
        dw = (torch.empty_like(w_gate), torch.empty_like(w_up), torch.empty_like(w_down))
    ws = _ws(p["experts_bwd_ws_bytes"], dev)
    abi.check("moe_experts_backward", library().moe_experts_backward(
        C.byref(cfg), _ptr(pools), _ptr(bank_rows), _ptr(expert_count), _ptr(w_gate), _ptr(w_up),
        _ptr(w_down), _ptr(d_expert_out), _ptr(d_pool_rows), _ptr(dw[0]), _ptr(dw[1]),
        _ptr(dw[2]), _ptr(ws), ws.numel(), _stream(dev)))
    return d_pool_rows, dw


def dispatch_backward(cfg, topk_idx, pool_slot, recv_slot, d_pool_rows, dz=None):
    """dz [T, L] = transpose of dispatch (sum over a token's kept rows)."""
    dev = d_pool_rows.device
    if dz is None:
        dz = torch.empty((cfg.T, cfg.d_latent), dtype=_tdt(cfg), device=dev)
    abi.check("moe_dispatch_backward", library().moe_dispatch_backward(
        C.byref(cfg), _ptr(topk_idx), _ptr(pool_slot), _ptr(recv_slot), _ptr(d_pool_rows),
        _ptr(dz), _stream(dev)))
    return dz


def route_backward(cfg, topk_idx, gates, d_gates, d_logits=None):
    """d_logits [T, E] fp32 = transpose of the gate softmax."""
    dev = gates.device
    if d_logits is None:
        d_logits = torch.empty((cfg.T, cfg.n_experts), dtype=torch.float32, device=dev)
    abi.check("moe_route_backward", library().moe_route_backward(
        C.byref(cfg), _ptr(topk_idx), _ptr(gates), _ptr(d_gates), _ptr(d_logits), _stream(dev)))
    return d_logits


class BackwardRouted:
    """Reusable routed-path backward bound to a Forward (or ForwardDropless)
    built with taps=True: its saved routing, rows and expert outputs feed the
    gradient (moe_backward_routed, or moe_backward_dropless)."""

    def __init__(self, fwd):
        if fwd.taps is None:
            raise ValueError("the forward must keep its taps (taps=True)")
        cfg, dev = fwd.cfg, fwd.y.device
        self.cfg, self.fwd = cfg, fwd
        self.p = fwd.p
        self.dropless = isinstance(fwd, ForwardDropless)
        self.ws = _ws(self.p["dropless_backward_ws_bytes" if self.dropless else "backward_ws_bytes"], dev)
        self.dz = torch.empty((cfg.T, cfg.d_latent), dtype=_tdt(cfg), device=dev)
        self.d_logits = torch.empty((cfg.T, cfg.n_experts), dtype=torch.float32, device=dev)
        w = fwd.w
        self.dw = (torch.empty_like(w["w_gate"]), torch.empty_like(w["w_up"]),
                   torch.empty_like(w["w_down"]))

    def _args(self, dy_latent):
        return (C.byref(self.cfg), C.byref(self.fwd.wstruct), C.byref(self.fwd.taps),
                _ptr(dy_latent), _ptr(self.dz), _ptr(self.d_logits), _ptr(self.dw[0]),
                _ptr(self.dw[1]), _ptr(self.dw[2]), _ptr(self.ws), self.ws.numel(),
                _stream(dy_latent.device))

    def __call__(self, dy_latent: torch.Tensor):
        name = "moe_backward_dropless" if self.dropless else "moe_backward_routed"
        abi.check(name, getattr(library(), name)(*self._args(dy_latent)))
        return self.dz, self.d_logits, self.dw

    def profiled(self, dy_latent: torch.Tensor, events):
        arr = (C.c_void_p * len(events))(*[C.c_void_p(e.cuda_event) for e in events])
        name = "moe_backward_dropless_profiled" if self.dropless else "moe_backward_routed_profiled"
        abi.check(name, getattr(library(), name)(*self._args(dy_latent), arr, len(events)))
        return self.dz, self.d_logits, self.dw


def backward_stage_count() -> int:
    return library().moe_backward_routed_stage_count()


def combine_backward_dropless(cfg, expert_out, row_of, gates, dy_latent, d_gates=None,
                              d_expert_out=None):
    """(d_gates [T, k] fp32, d_expert_out [T*k, L]) = transpose of combine_dropless."""
    dev = dy_latent.device
    if d_gates is None:
        d_gates = torch.empty((cfg.T, cfg.top_k), dtype=torch.float32, device=dev)
    if d_expert_out is None:
        d_expert_out = torch.empty_like(expert_out)
    abi.check("moe_combine_backward_dropless", library().moe_combine_backward_dropless(
        C.byref(cfg), _ptr(expert_out), _ptr(row_of), _ptr(gates), _ptr(dy_latent), _ptr(d_gates),
        _ptr(d_expert_out), _stream(dev)))
    return d_gates, d_expert_out


def experts_backward_dropless(cfg, xs, expert_offsets, w_gate, w_up, w_down, d_expert_out,
                              d_xs=None, dw=None):
    """(d_xs [T*k, L], (dw_gate, dw_up, dw_down)) = transpose of experts_dropless."""
    p = plan(cfg)
    dev = xs.device
    if d_xs is None:
        d_xs = torch.empty_like(xs)
    if dw is None:
        dw = (torch.empty_like(w_gate), torch.empty_like(w_up), torch.empty_like(w_down))
    ws = _ws(p["dropless_experts_bwd_ws_bytes"], dev)
    abi.check("moe_experts_backward_dropless", library().moe_experts_backward_dropless(
        C.byref(cfg), _ptr(xs), _ptr(expert_offsets), _ptr(w_gate), _ptr(w_up), _ptr(w_down),
        _ptr(d_expert_out), _ptr(d_xs), _ptr(dw[0]), _ptr(dw[1]), _ptr(dw[2]), _ptr(ws),
        ws.numel(), _stream(dev)))
    return d_xs, dw


def dispatch_backward_dropless(cfg, row_of, d_xs, dz=None):
    """dz [T, L] = transpose of dispatch_dropless."""
    dev = d_xs.device
    if dz is None:
        dz = torch.empty((cfg.T, cfg.d_latent), dtype=_tdt(cfg), device=dev)
    abi.check("moe_dispatch_backward_dropless", library().moe_dispatch_backward_dropless(
        C.byref(cfg), _ptr(row_of), _ptr(d_xs), _ptr(dz), _stream(dev)))
    return dz


# ---------------------------------------------------------- scored routing
def _check(ok, what):
    if not ok:
        raise ValueError(what)


def _rows(t, shape, dtype, what, dev=None):
    """A contiguous device tensor of this shape and type (the entry points take plain pointers)."""
    if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.shape == shape and t.is_contiguous()
            and t.is_cuda and (dev is None or t.device == dev)):
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)}"
                         + (f" on {dev}" if dev is not None else " on a GPU"))
    return t


def _new(rows, cols, dtype, dev):
    """A new contiguous [rows, cols] (empty_strided returns sooner than empty)."""
    return torch.empty_strided((rows, cols), (max(cols, 1), 1), dtype=dtype, device=dev)


def _workspace(ws, nbytes, dev):
    """The caller's workspace (bytes on the tensors' device), or a new one."""
    if ws is None:
        return _ws(nbytes, dev)
    if not (ws.dtype == torch.uint8 and ws.device == dev and ws.is_contiguous()):
        raise ValueError(f"ws must be a contiguous uint8 tensor on {dev}")
    return ws


# raw handle of the current stream of a device: torch's own accessor where it
# has one (a Stream object costs a microsecond per call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


# index of the current device: likewise (valid once a tensor is on a GPU)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _status(name, dev, *args):
    """Status of a C entry point called on the tensors' device (made current for
    the call where it is not) and its current stream."""
    index = dev.index
    prev = _current_device()
    if prev == index:
        return getattr(abi.load(), name)(*args, _raw_stream(index))
    torch.cuda.set_device(index)
    try:
        return getattr(abi.load(), name)(*args, _raw_stream(index))
    finally:
        torch.cuda.set_device(prev)


def _launch(name, dev, *args):
    """The same, raising its error."""
    status = _status(name, dev, *args)
    if status:
        raise MoeError(name, status)


def scoring(score="sigmoid", n_groups=1, top_groups=1, group_top=2, renormalise=True, scale=1.0) -> abi.MoeScoring:
    """How route_scored makes scores, limits groups and scales gates (moe_scoring)."""
    _check(score in ("sigmoid", "softmax"), "score is 'sigmoid' or 'softmax'")
    return abi.MoeScoring(abi.MOE_SCORE_SIGMOID if score == "sigmoid" else abi.MOE_SCORE_SOFTMAX, n_groups, top_groups,
                          group_top, int(bool(renormalise)), scale, 0)


def route_scored(cfg, sc: abi.MoeScoring, logits: torch.Tensor, bias: Optional[torch.Tensor] = None, out=None):
    """(topk_idx [T, k] int32, gates [T, k] fp32) by scores (moe_route_scored)."""
    T, k, E = cfg.T, cfg.top_k, cfg.n_experts
    dev = _rows(logits, (T, E), torch.float32, "logits").device
    if bias is not None:
        _rows(bias, (E,), torch.float32, "bias", dev)
    topk = _new(T, k, torch.int32, dev) if out is None else \
        _rows(out["topk_idx"], (T, k), torch.int32, "out['topk_idx']", dev)
    gates = _new(T, k, torch.float32, dev) if out is None else \
        _rows(out["gates"], (T, k), torch.float32, "out['gates']", dev)
    _launch("moe_route_scored", dev, C.byref(cfg), C.byref(sc), logits.data_ptr(),
            None if bias is None else bias.data_ptr(), topk.data_ptr(), gates.data_ptr())
    return topk, gates


def route_scored_backward(cfg, sc: abi.MoeScoring, logits, topk_idx, d_gates, d_logits=None):
    """d_logits [T, E] fp32 = transpose of route_scored's gates for the selection made."""
    T, k, E = cfg.T, cfg.top_k, cfg.n_experts
    dev = _rows(logits, (T, E), torch.float32, "logits").device
    _rows(topk_idx, (T, k), torch.int32, "topk_idx", dev)
    _rows(d_gates, (T, k), torch.float32, "d_gates", dev)
    d_logits = torch.empty_like(logits) if d_logits is None else \
        _rows(d_logits, (T, E), torch.float32, "d_logits", dev)
    _launch("moe_route_scored_backward", dev, C.byref(cfg), C.byref(sc), logits.data_ptr(), topk_idx.data_ptr(),
            d_gates.data_ptr(), d_logits.data_ptr())
    return d_logits


# ------------------------------------------------------- block-scaled e4m3
def quantize(x: torch.Tensor, block_rows: int = 1, transpose: bool = False, out=None):
    """(q, scales) of x [rows, cols] (bf16 or fp32; rows may be strided) in
    e4m3 with one fp32 scale for 1 x 128 or 128 x 128 blocks (moe_quantize).
    With transpose, of x^T.  q [R, K padded to 128]; scales [K/128, R], or
    [R/128, K/128] for 128 x 128 blocks."""
    _check(isinstance(x, torch.Tensor) and x.dim() == 2 and x.is_cuda and x.dtype in (torch.bfloat16, torch.float32),
           "x must be a two-dimensional bf16 or fp32 tensor on a GPU")
    _check(x.shape[1] <= 1 or x.stride(1) == 1, "the columns of x must be contiguous")
    _check(block_rows in (1, 128), "block_rows is 1 or 128")
    rows, cols = x.shape
    ld = x.stride(0) if rows > 1 else cols
    _check(ld >= cols, "the rows of x must not overlap")
    R, K = (cols, rows) if transpose else (rows, cols)
    kb = -(-K // 128)
    dev = x.device
    qs, ss = (R, kb * 128), ((kb, R) if block_rows == 1 else (-(-R // 128), kb))
    q = _new(*qs, torch.float8_e4m3fn, dev) if out is None else \
        _rows(out[0], qs, torch.float8_e4m3fn, "out[0]", dev)
    s = _new(*ss, torch.float32, dev) if out is None else \
        _rows(out[1], ss, torch.float32, "out[1]", dev)
    _launch("moe_quantize", dev, rows, cols, x.data_ptr(), ld, _DT[x.dtype], block_rows, int(transpose), q.data_ptr(),
            s.data_ptr())
    return q, s


def _operand(q, what, dev=None):
    if not (isinstance(q, torch.Tensor) and q.dim() == 2 and q.is_cuda and q.dtype == torch.float8_e4m3fn
            and (dev is None or q.device == dev) and (q.shape[1] <= 1 or q.stride(1) == 1)):
        raise ValueError(f"{what} must be a two-dimensional e4m3 tensor with contiguous columns on one GPU")
    return q.stride(0) if q.shape[0] > 1 and q.shape[1] > 0 else q.shape[1]


def _scale_ld(s, shape, what, dev):
    if not (isinstance(s, torch.Tensor) and s.dtype == torch.float32 and s.shape == shape and s.device == dev
            and (shape[1] <= 1 or s.stride(1) == 1)):
        raise ValueError(f"{what} must be an fp32 tensor of shape {shape} with contiguous columns")
    return s.stride(0) if shape[0] > 1 else max(shape[1], 1)


def gemm_quant(a, a_scales, b, b_scales, block_rows: int = 128, out_dtype=torch.bfloat16, out=None, ws=None):
    """C [M, N] = A B^T of e4m3 operands with block scales (moe_gemm_quant):
    a [M, K] with a_scales [K/128, M]; b [N, K] with b_scales [N/128, K/128]
    (block_rows 128) or [K/128, N] (block_rows 1).  Rows may be strided (a
    slice of a larger batch); C is bf16 or fp32."""
    lda = _operand(a, "a")
    dev = a.device
    ldb = _operand(b, "b", dev)
    (M, K), N = a.shape, b.shape[0]
    _check(b.shape[1] == K and K % 128 == 0, "a and b must have the same K, a multiple of 128")
    _check(block_rows in (1, 128), "block_rows is 1 or 128")
    _check(out_dtype in (torch.bfloat16, torch.float32), "out_dtype is bfloat16 or float32")
    kb = K // 128
    sa = _scale_ld(a_scales, (kb, M), "a_scales", dev)
    sb = _scale_ld(b_scales, (kb, N) if block_rows == 1 else (-(-N // 128), kb), "b_scales", dev)
    if out is None:
        out = _new(M, N, out_dtype, dev)
    else:
        _check(out.shape == (M, N) and out.dtype == out_dtype and out.device == dev
               and (N <= 1 or out.stride(1) == 1) and (M <= 1 or out.stride(0) >= N),
               "out must be a tensor of C's shape and type with contiguous columns")
    g = abi.MoeQuantGemm(M, N, K, a.data_ptr(), lda, a_scales.data_ptr(), sa, b.data_ptr(), ldb, b_scales.data_ptr(),
                         sb, out.data_ptr(), out.stride(0) if M > 1 else N, block_rows, _DT[out_dtype], 0)
    lib = library()
    n = C.c_size_t(0)
    abi.check("moe_gemm_quant_ws_bytes", lib.moe_gemm_quant_ws_bytes(C.byref(g), C.byref(n)))
    if n.value:
        ws = _workspace(ws, n.value, dev)
        _launch("moe_gemm_quant", dev, C.byref(g), ws.data_ptr(), ws.numel())
    else:
        _launch("moe_gemm_quant", dev, C.byref(g), None, 0)
    return out


def _quant_experts(cfg, w_gate, w_up, w_down, dev):
    E, L, F = cfg.n_experts, cfg.d_latent, cfg.d_ff
    f = {}
    for name, (q, s), r, c in (("gate", w_gate, F, L), ("up", w_up, F, L), ("down", w_down, L, F)):
        f["q_" + name] = _rows(q, (E, r, c), torch.float8_e4m3fn, f"w_{name}[0]", dev).data_ptr()
        f["s_" + name] = _rows(s, (E, r // 128, c // 128), torch.float32, f"w_{name}[1]", dev).data_ptr()
    return abi.MoeQuantExperts(**f)


def experts_dropless_quant_ws_bytes(cfg) -> int:
    n = C.c_size_t(0)
    abi.check("moe_experts_dropless_quant_ws_bytes",
              library().moe_experts_dropless_quant_ws_bytes(C.byref(cfg), C.byref(n)))
    return int(n.value)


def experts_dropless_quant(cfg, xs, expert_offsets, w_gate, w_up, w_down, expert_out=None, ws=None):
    """experts_dropless with e4m3 weights (moe_experts_dropless_quant): each
    weight a (q [E, out, in], scales [E, out/128, in/128]) pair."""
    n, L = cfg.T * cfg.top_k, cfg.d_latent
    nbytes = experts_dropless_quant_ws_bytes(cfg)
    dev = _rows(xs, (n, L), torch.bfloat16, "xs").device
    _rows(expert_offsets, (cfg.n_experts + 1,), torch.int32, "expert_offsets", dev)
    w = _quant_experts(cfg, w_gate, w_up, w_down, dev)
    expert_out = torch.empty_like(xs) if expert_out is None else \
        _rows(expert_out, (n, L), torch.bfloat16, "expert_out", dev)
    ws = _workspace(ws, nbytes, dev)
    _launch("moe_experts_dropless_quant", dev, C.byref(cfg), xs.data_ptr(), expert_offsets.data_ptr(), C.byref(w),
            expert_out.data_ptr(), ws.data_ptr(), ws.numel())
    return expert_out


def quantize_weights(cfg, weights: Dict[str, torch.Tensor]) -> Dict:
    """The weights of a branch (bf16 or fp32, the names of Forward's) in the
    form ForwardDroplessQuant takes: (q, scales) pairs in 128 x 128 blocks,
    the up-projection and the shared down-projections side by side as
    w_output; the router stays bf16."""
    def blocks(w):
        _check(w.shape[-1] % 128 == 0 and w.shape[-2] % 128 == 0, "the weights' sizes must be multiples of 128")
        q, s = quantize(w.reshape(-1, w.shape[-1]), 128)
        return q.view(w.shape), s.view(*w.shape[:-2], w.shape[-2] // 128, w.shape[-1] // 128)
    out = {n: blocks(weights[n]) for n in ("w_latent", "w_gate", "w_up", "w_down")}
    cols = [weights["w_up_proj"]]
    if cfg.n_shared:
        out.update({n: blocks(weights[n]) for n in ("ws_gate", "ws_up")})
        cols += list(weights["ws_down"])
    out["w_output"] = blocks(torch.cat(cols, dim=1).contiguous())
    out["w_router"] = weights["w_router"].to(torch.bfloat16)
    out["router_bias"] = weights.get("router_bias")
    return out


class ForwardDroplessQuant:
    """Reusable dropless forward in e4m3 with scored routing
    (moe_forward_dropless_quant): weights (quantize_weights), workspace and
    outputs bound once."""

    def __init__(self, cfg, sc: abi.MoeScoring, weights: Dict, device, taps=False):
        device = torch.device(device)
        if device.index is None:
            device = torch.device(device.type, torch.cuda.current_device())
        self.cfg, self.sc, self.w, self.p = cfg, sc, weights, plan(cfg)
        n = C.c_size_t(0)
        abi.check("moe_forward_dropless_quant_ws_bytes",
                  library().moe_forward_dropless_quant_ws_bytes(C.byref(cfg), C.byref(n)))
        T, D, L, E, k = cfg.T, cfg.d_model, cfg.d_latent, cfg.n_experts, cfg.top_k
        S, Fs = cfg.n_shared, cfg.d_ff_shared
        W = L + S * Fs

        def pair(name, shape):
            q, s = weights[name]
            return (_rows(q, shape, torch.float8_e4m3fn, name + "[0]", device).data_ptr(),
                    _rows(s, (*shape[:-2], shape[-2] // 128, shape[-1] // 128), torch.float32, name + "[1]",
                          device).data_ptr())
        f = dict(w_router=_rows(weights["w_router"], (E, L), torch.bfloat16, "w_router", device).data_ptr(),
                 experts=_quant_experts(cfg, weights["w_gate"], weights["w_up"], weights["w_down"], device))
        if weights.get("router_bias") is not None:
            f["router_bias"] = _rows(weights["router_bias"], (E,), torch.float32, "router_bias", device).data_ptr()
        f["q_latent"], f["s_latent"] = pair("w_latent", (L, D))
        f["q_output"], f["s_output"] = pair("w_output", (D, W))
        if S:
            f["q_shared_gate"], f["s_shared_gate"] = pair("ws_gate", (S, Fs, D))
            f["q_shared_up"], f["s_shared_up"] = pair("ws_up", (S, Fs, D))
        self.wstruct = abi.MoeQuantWeights(**f)
        self.ws = _ws(n.value, device)
        self.y = torch.empty((T, D), dtype=torch.bfloat16, device=device)
        self.counts = torch.empty(3, dtype=torch.int64, device=device)
        self.taps, self.tap_t = None, {}
        if taps:
            rows = self.p["dropless_rows"]
            i32, bf = dict(dtype=torch.int32, device=device), dict(dtype=torch.bfloat16, device=device)
            self.tap_t = dict(
                logits=torch.empty((T, E), dtype=torch.float32, device=device), topk_idx=torch.empty((T, k), **i32),
                gates=torch.empty((T, k), dtype=torch.float32, device=device), row_of=torch.empty((T, k), **i32),
                expert_offsets=torch.empty(E + 1, **i32), z=torch.empty((T, L), **bf), xs=torch.empty((rows, L), **bf),
                expert_out=torch.empty((rows, L), **bf), y_latent=torch.empty((T, L), **bf))
            self.taps = abi.MoeDroplessTaps(**{m: t.data_ptr() for m, t in self.tap_t.items()})

    def __call__(self, x: torch.Tensor):
        cfg = self.cfg
        _rows(x, (cfg.T, cfg.d_model), torch.bfloat16, "x", self.y.device)
        _launch("moe_forward_dropless_quant", self.y.device, C.byref(cfg), C.byref(self.sc), C.byref(self.wstruct),
                x.data_ptr(), self.y.data_ptr(), C.byref(self.taps) if self.taps is not None else None,
                self.counts.data_ptr(), self.ws.data_ptr(), self.ws.numel())
        return self.y


# ------------------------------------------------------------- linear layers
def _matrix(t, shape, dtypes, what, dev=None):
    """Leading dimension of a two-dimensional tensor of this shape with contiguous columns (rows may be strided)."""
    if isinstance(t, torch.Tensor) and t.shape == shape and t.dtype in dtypes and \
            (t.is_cuda if dev is None else t.device == dev):
        ld, one = t.stride()
        rows, cols = shape
        if (one == 1 or cols <= 1) and (ld >= cols or rows <= 1):
            return ld if rows > 1 else max(cols, 1)
    raise ValueError(f"{what} must be a {' or '.join(str(d) for d in dtypes)} tensor of shape {tuple(shape)} with "
                     f"contiguous columns" + (f" on {dev}" if dev is not None else " on a GPU"))


def _with_workspace(name, dev, args, ws, likely=True):
    """Call `name`(args, workspace) with the caller's workspace, or a new one of
    the size asked for.  likely: whether one is asked for mostly; else the call is
    made without first."""
    ref = C.byref(args)
    if ws is None and not likely:
        status = _status(name, dev, ref, None, 0)
        if status != abi.MOE_ERR_WORKSPACE:
            if status:
                raise MoeError(name, status)
            return
    n = C.c_size_t(0)
    abi.check(name + "_ws_bytes", getattr(abi.load(), name + "_ws_bytes")(ref, C.byref(n)))
    if ws is None and n.value == 0:
        return _launch(name, dev, ref, None, 0)
    ws = _workspace(ws, n.value, dev)
    _launch(name, dev, ref, ws.data_ptr(), ws.numel())


_BF16 = (torch.bfloat16,)
_FLOATS = (torch.bfloat16, torch.float32)


def linear(x, w, bias=None, act: str = "none", residual=None, out_dtype=torch.bfloat16, save_pre: bool = False,
           out=None, ws=None):
    """y [M, N] = act(x w^T + bias) + residual (moe_linear): x [M, K] and w
    [N, K] bf16, bias [N] bf16 or fp32, residual and y of out_dtype (bf16 or
    fp32); residual may be out.  With save_pre, (y, the pre-activation in
    bf16), which linear_backward takes.  Rows may be strided."""
    _check(act in abi.ACTS, "act is 'none', 'relu', 'silu' or 'gelu'")
    _check(isinstance(x, torch.Tensor) and x.dim() == 2 and isinstance(w, torch.Tensor) and w.dim() == 2,
           "x and w must be two-dimensional tensors")
    _check(out_dtype in _FLOATS, "out_dtype is bfloat16 or float32")
    (M, K), N = x.shape, w.shape[0]
    ldx = _matrix(x, (M, K), _BF16, "x")
    dev = x.device
    ldw = _matrix(w, (N, K), _BF16, "w", dev)
    if bias is not None and not (isinstance(bias, torch.Tensor) and bias.shape == (N,) and bias.dtype in _FLOATS
                                 and bias.device == dev and bias.is_contiguous()):
        raise ValueError(f"bias must be a contiguous bf16 or fp32 tensor of shape ({N},) on {dev}")
    ldr = _matrix(residual, (M, N), (out_dtype,), "residual", dev) if residual is not None else 0
    if out is None:
        out, ldy = _new(M, N, out_dtype, dev), max(N, 1)
    else:
        ldy = _matrix(out, (M, N), (out_dtype,), "out", dev)
    pre = _new(M, N, torch.bfloat16, dev) if save_pre else None
    a = abi.MoeLinearArgs(M, N, K, x.data_ptr(), ldx, w.data_ptr(), ldw, None if bias is None else bias.data_ptr(),
                          None if residual is None else residual.data_ptr(), ldr, out.data_ptr(), ldy,
                          None if pre is None else pre.data_ptr(), max(N, 1), abi.ACTS[act],
                          abi.MOE_F32 if bias is not None and bias.dtype == torch.float32 else abi.MOE_BF16,
                          _DT[out_dtype], 0)
    _with_workspace("moe_linear", dev, a, ws, likely=False)
    return (out, pre) if save_pre else out


def linear_backward(dy, x, w, pre=None, act: str = "none", bias: bool = True, need_dx: bool = True,
                    need_dw: bool = True, dx=None, dw=None, db=None, ws=None):
    """(dx [M, K] bf16, dw [N, K] bf16, db [N] fp32) of linear for dy [M, N]
    (bf16 or fp32) and the pre-activation it kept (moe_linear_backward); None
    in the place of what need_dx, need_dw and bias leave out.  The residual's
    gradient is dy."""
    _check(act in abi.ACTS, "act is 'none', 'relu', 'silu' or 'gelu'")
    _check(isinstance(x, torch.Tensor) and x.dim() == 2 and isinstance(w, torch.Tensor) and w.dim() == 2,
           "x and w must be two-dimensional tensors")
    (M, K), N = x.shape, w.shape[0]
    ldx = _matrix(x, (M, K), _BF16, "x")
    dev = x.device
    ldw = _matrix(w, (N, K), _BF16, "w", dev)
    lddy = _matrix(dy, (M, N), _FLOATS, "dy", dev)
    _check(act == "none" or pre is not None, "the pre-activation is needed")
    ldp = _matrix(pre, (M, N), _BF16, "pre", dev) if act != "none" else 0

    def out(t, rows, what):
        t = _new(rows, K, torch.bfloat16, dev) if t is None else t
        return t, _matrix(t, (rows, K), _BF16, what, dev)
    dx, lddx = out(dx, M, "dx") if need_dx else (None, 0)
    dw, lddw = out(dw, N, "dw") if need_dw else (None, 0)
    if not bias:
        db = None
    elif db is None:
        db = torch.empty(N, dtype=torch.float32, device=dev)
    else:
        _rows(db, (N,), torch.float32, "db", dev)
    a = abi.MoeLinearGrad(M, N, K, dy.data_ptr(), lddy, pre.data_ptr() if ldp else None, ldp, x.data_ptr(), ldx,
                          w.data_ptr(), ldw, None if dx is None else dx.data_ptr(), lddx,
                          None if dw is None else dw.data_ptr(), lddw, None if db is None else db.data_ptr(),
                          abi.ACTS[act], _DT[dy.dtype], 0)
    _with_workspace("moe_linear_backward", dev, a, ws)
    return dx, dw, db


# --------------------------------------------------- orthogonalised updates
_COEFFS = "coeffs is (a, b, c), or one of them for each step"


@functools.lru_cache(maxsize=64)
def _coefficient_array(coeffs, steps):
    rows = list(coeffs) if any(isinstance(c, tuple) for c in coeffs) else [coeffs] * steps
    _check(len(rows) == steps and all(isinstance(r, tuple) and len(r) == 3 for r in rows), _COEFFS)
    return (C.c_float * (3 * steps))(*[v for r in rows for v in r])


def _coefficients(coeffs, steps):
    """[steps][3] fp32 on the host of one (a, b, c), or of one for each step.
    What is kept between calls is kept for their values: any number is read anew."""
    try:
        values = tuple(tuple(map(float, c)) if isinstance(c, (list, tuple)) else float(c) for c in coeffs)
    except (TypeError, ValueError, RuntimeError):
        raise ValueError(_COEFFS) from None
    return _coefficient_array(values, steps)


def _batch(t, what):
    """(leading dimension, stride between matrices) of a [B, M, N] tensor with contiguous columns."""
    B, M, N = t.shape
    ld = t.stride(1) if M > 1 else max(N, 1)
    stride = t.stride(0) if B > 1 else M * ld
    _check((N <= 1 or t.stride(2) == 1) and ld >= N and (B <= 1 or M == 0 or stride >= (M - 1) * ld + N),
           f"{what} must have contiguous columns and matrices that do not overlap")
    return ld, stride


def orthogonalize(g, steps: int = 5, coeffs=(3.4445, -4.7750, 2.0315), eps: float = 1e-7, scale: float = 1.0, out=None,
                  ws=None):
    """scale times the Newton-Schulz iterate of g [M, N] or [B, M, N] (bf16 or
    fp32; rows and matrices may be strided) in bf16 (moe_orthogonalize): the
    update of a weight whose singular values lie near 1.  coeffs: (a, b, c)
    for every step, or a sequence of them, one for each."""
    _check(isinstance(g, torch.Tensor) and g.dim() in (2, 3) and g.is_cuda and g.dtype in _FLOATS,
           "g must be a two- or three-dimensional bf16 or fp32 tensor on a GPU")
    dev = g.device
    if out is None:
        out = torch.empty(g.shape, dtype=torch.bfloat16, device=dev)
    else:
        _check(isinstance(out, torch.Tensor) and out.shape == g.shape and out.dtype == torch.bfloat16
               and out.device == dev, f"out must be a bf16 tensor of g's shape on {dev}")
    g3, o3 = (g, out) if g.dim() == 3 else (g[None], out[None])
    B, M, N = g3.shape
    ldg, sg = _batch(g3, "g")
    ldo, so = _batch(o3, "out")
    _check(1 <= steps <= 64, "steps is 1 to 64")
    co = _coefficients(coeffs, steps)
    a = abi.MoeOrthoArgs(B, M, N, g.data_ptr(), ldg, sg, out.data_ptr(), ldo, so, co, steps, _DT[g.dtype], eps, scale, 0)
    _with_workspace("moe_orthogonalize", dev, a, ws)
    return out


# ------------------------------------------------------- a few tokens
class ForwardFew:
    """Reusable dropless forward for at most 16 tokens (moe_forward_few): the
    weights of ForwardDropless, workspace and outputs bound once.  One call at a
    time: calls on two streams need an object each."""

    def __init__(self, cfg, weights: Dict[str, torch.Tensor], device, taps=False):
        device = torch.device(device)
        if device.index is None:
            device = torch.device(device.type, torch.cuda.current_device())
        self.cfg, self.w = cfg, weights
        n = C.c_size_t(0)
        abi.check("moe_forward_few_ws_bytes", library().moe_forward_few_ws_bytes(C.byref(cfg), C.byref(n)))
        T, D, L, E, k, F = cfg.T, cfg.d_model, cfg.d_latent, cfg.n_experts, cfg.top_k, cfg.d_ff
        shapes = dict(w_latent=(L, D), w_router=(E, L), w_gate=(E, F, L), w_up=(E, F, L), w_down=(E, L, F),
                      w_up_proj=(D, L))
        if cfg.n_shared:
            S, Fs = cfg.n_shared, cfg.d_ff_shared
            shapes.update(ws_gate=(S, Fs, D), ws_up=(S, Fs, D), ws_down=(S, D, Fs))
        f = {m: _rows(weights[m], shape, torch.bfloat16, m, device).data_ptr() for m, shape in shapes.items()}
        if weights.get("router_bias") is not None:
            f["router_bias"] = _rows(weights["router_bias"], (E,), torch.float32, "router_bias", device).data_ptr()
        self.wstruct = abi.MoeWeights(**f)
        self.ws = _ws(n.value, device)
        self.y = torch.empty((T, D), dtype=torch.bfloat16, device=device)
        self.tap_t = {}
        if taps:
            self.tap_t = dict(logits=torch.empty((T, E), dtype=torch.float32, device=device),
                              topk_idx=torch.empty((T, k), dtype=torch.int32, device=device),
                              gates=torch.empty((T, k), dtype=torch.float32, device=device))
        self._tail = (self.y.data_ptr(), *((self.tap_t[m].data_ptr() if taps else None)
                                           for m in ("logits", "topk_idx", "gates")),
                      self.ws.data_ptr(), self.ws.numel())

    def __call__(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None):
        cfg, dev = self.cfg, self.y.device
        _rows(x, (cfg.T, cfg.d_model), torch.bfloat16, "x", dev)
        if residual is not None:
            _rows(residual, (cfg.T, cfg.d_model), torch.bfloat16, "residual", dev)
        _launch("moe_forward_few", dev, C.byref(cfg), C.byref(self.wstruct), x.data_ptr(),
                None if residual is None else residual.data_ptr(), *self._tail)
        return self.y
