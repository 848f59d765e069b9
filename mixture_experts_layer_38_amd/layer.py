"""Device-resident MoE layer on top of the C ABI.

torch provides the device memory (weights, workspace, outputs) and the stream;
every step of the forward pass runs in libmoe.so through `moe_forward`.
"""
from __future__ import annotations

import numpy as np

from . import (MoEProblem, i8_weights, moe_aux_loss, moe_bias_update, moe_combine, moe_combine_backward,
               moe_dispatch, moe_dispatch_workspace_size, moe_expert_ffn_backward,
               moe_expert_ffn_backward_workspace_size, moe_expert_ffn_train,
               moe_expert_ffn_train_workspace_size, moe_forward, moe_forward_i8,
               moe_forward_i8_workspace_size, moe_quantize_rows, moe_route, moe_route_backward,
               moe_route_backward_workspace_size, moe_route_workspace_size, moe_workspace_size, problem)
from .configs import MoEConfig


def to_device(a: np.ndarray, dtype: str, device="cuda"):
    """Host array (float32, or bf16 bit patterns as uint16) -> torch tensor."""
    import torch
    if dtype == "bf16":
        t = torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).view(torch.bfloat16)
    else:
        t = torch.from_numpy(np.ascontiguousarray(a, np.float32))
    return t.to(device)


def to_host(t, dtype: str) -> np.ndarray:
    """torch tensor -> float32 array, or uint16 bit patterns for bf16."""
    import torch
    t = t.detach().cpu()
    if t.dtype == torch.bfloat16:
        return t.view(torch.int16).numpy().view(np.uint16)
    return t.numpy()


class MoELayer:
    """One MoE layer with its weights resident in HBM."""

    def __init__(self, T: int, d: int, E: int, K: int, F: int, dtype: str, w_router, w1, w3, w2,
                 capacity: int = -1, device="cuda", flags: int = 0):
        import torch
        self.T, self.d, self.E, self.K, self.F = T, d, E, K, F
        self.dtype = dtype
        self.capacity = capacity
        self.device = device
        self.w_router, self.w1, self.w3, self.w2 = w_router, w1, w3, w2
        self.torch_dtype = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.flags = flags
        self.p: MoEProblem = problem(T, d, E, K, F, dtype, capacity, flags)
        self.ws = torch.empty(moe_workspace_size(self.p), dtype=torch.uint8, device=device)

    @classmethod
    def from_host(cls, cfg: MoEConfig, inputs: dict, device="cuda", T: int | None = None,
                  flags: int = 0):
        dt = cfg.dtype
        return cls(cfg.T if T is None else T, cfg.d, cfg.E, cfg.K, cfg.F, dt,
                   to_device(inputs["w_router"], dt, device), to_device(inputs["w1"], dt, device),
                   to_device(inputs["w3"], dt, device), to_device(inputs["w2"], dt, device),
                   cfg.capacity, device, flags)

    def alloc_debug(self, losses: bool = False) -> dict:
        """Device buffers for every optional output of moe_forward; with
        losses, also the two router regularisers (z_loss, aux_topk)."""
        import torch
        T, E, K = self.T, self.E, self.K
        dev = self.device
        f32, i32 = torch.float32, torch.int32
        extra = {}
        if losses:
            extra = {"z_loss": torch.full((1,), -1.0, dtype=f32, device=dev),
                     "aux_topk": torch.full((1,), -1.0, dtype=f32, device=dev)}
        return extra | {
            "logits": torch.empty((T, E), dtype=f32, device=dev),
            "probs": torch.empty((T, E), dtype=f32, device=dev),
            "prob_sum": torch.empty((E,), dtype=f32, device=dev),
            "topk_ids": torch.empty((T, K), dtype=i32, device=dev),
            "topk_w": torch.empty((T, K), dtype=f32, device=dev),
            "counts": torch.empty((E,), dtype=i32, device=dev),
            "kept": torch.empty((E,), dtype=i32, device=dev),
            "offsets": torch.empty((E + 1,), dtype=i32, device=dev),
            "assign_row": torch.empty((T * K,), dtype=i32, device=dev),
            "row_assign": torch.empty((T * K,), dtype=i32, device=dev),
        }

    def forward(self, x, logit_bias=None, y=None, dbg: dict | None = None, stream=None):
        import torch
        if y is None:
            y = torch.empty((self.T, self.d), dtype=self.torch_dtype, device=self.device)
        moe_forward(self.p, x, self.w_router, self.w1, self.w3, self.w2, logit_bias, y, self.ws,
                    dbg, stream)
        return y

    def aux_loss(self, counts, prob_sum, out=None, stream=None):
        import torch
        if out is None:
            out = torch.empty((1,), dtype=torch.float32, device=self.device)
        moe_aux_loss(self.p, counts, prob_sum, out, stream)
        return out

    def bias_update(self, counts, alpha: float, bias, stream=None):
        moe_bias_update(self.p, counts, alpha, bias, stream)
        return bias

    # ---- training: forward and backward as step calls --------------------------
    def _train_ws(self):
        """One workspace for every training step call (they run one after another)."""
        import torch
        if getattr(self, "train_ws", None) is None:
            p = self.p
            size = max(moe_route_workspace_size(p), moe_dispatch_workspace_size(p),
                       moe_expert_ffn_train_workspace_size(p), moe_expert_ffn_backward_workspace_size(p),
                       moe_route_backward_workspace_size(p))
            self.train_ws = torch.empty(size, dtype=torch.uint8, device=self.device)
        return self.train_ws

    def forward_train(self, x, logit_bias=None):
        """The layer's output, and what backward() needs: (y, saved).  Runs on torch's current
        stream, which also owns the buffers allocated here."""
        import torch
        p, ws, dev, dt = self.p, self._train_ws(), self.device, self.torch_dtype
        T, K, E, d, F = self.T, self.K, self.E, self.d, self.F
        f32, i32, n = torch.float32, torch.int32, self.T * self.K
        new = lambda *shape, dtype=dt: torch.empty(shape, dtype=dtype, device=dev)  # noqa: E731
        s = {"x": x, "logit_bias": logit_bias, "logits": new(T, E, dtype=f32), "topk_ids": new(T, K, dtype=i32),
             "topk_w": new(T, K, dtype=f32), "counts": new(E, dtype=i32), "offsets": new(E + 1, dtype=i32),
             "assign_row": new(n, dtype=i32), "x_perm": new(n, d), "gate": new(n, F), "up": new(n, F),
             "h": new(n, d), "prob_sum": new(E, dtype=f32)}
        moe_route(p, x, self.w_router, logit_bias, s["logits"], None, s["prob_sum"], s["topk_ids"], s["topk_w"], ws)
        moe_dispatch(p, s["topk_ids"], x, s["counts"], new(E, dtype=i32), s["offsets"], s["assign_row"],
                     new(n, dtype=i32), s["x_perm"], ws)
        moe_expert_ffn_train(p, s["x_perm"], s["offsets"], self.w1, self.w3, self.w2, s["gate"], s["up"], s["h"], ws)
        y = new(T, d)
        moe_combine(p, s["h"], s["assign_row"], s["topk_w"], y)
        return y, s

    def backward(self, dy, saved, d_aux: float = 0.0, d_z: float = 0.0) -> dict:
        """Gradients of the layer from dy = d(loss)/dy: dx, dw_router, dw1, dw3, dw2 (and dlogits).
        d_aux, d_z: gradients of the loss with respect to the load-balancing loss and the z-loss."""
        import torch
        p, ws, s, dev, dt = self.p, self._train_ws(), saved, self.device, self.torch_dtype
        new = lambda *shape, dtype=dt: torch.empty(shape, dtype=dtype, device=dev)  # noqa: E731
        dh, dw = new(self.T * self.K, self.d), new(self.T, self.K, dtype=torch.float32)
        moe_combine_backward(p, dy, s["h"], s["assign_row"], s["topk_w"], dh, dw)
        g = {k: torch.empty_like(getattr(self, k[1:])) for k in ("dw1", "dw3", "dw2", "dw_router")}
        dx_perm = new(self.T * self.K, self.d)
        moe_expert_ffn_backward(p, s["x_perm"], s["offsets"], self.w1, self.w3, self.w2, s["gate"], s["up"], dh,
                                dx_perm, g["dw1"], g["dw3"], g["dw2"], ws)
        g["dx"], g["dlogits"] = new(self.T, self.d), new(self.T, self.E, dtype=torch.float32)
        moe_route_backward(p, s["x"], self.w_router, s["logit_bias"], s["logits"], s["topk_ids"], s["topk_w"], dw,
                           s["counts"], d_aux, d_z, dx_perm, s["assign_row"], g["dlogits"], g["dx"], g["dw_router"],
                           ws)
        return g

    # ---- 8-bit experts -------------------------------------------------------------
    def quantized(self) -> "MoELayerI8":
        """The same layer on 8-bit expert weights."""
        return MoELayerI8(self)


class MoELayerI8:
    """A bf16 layer whose experts run on 8-bit weights, quantised once from it."""

    def __init__(self, layer: MoELayer):
        import torch
        self.p, self.T, self.d, self.device = layer.p, layer.T, layer.d, layer.device
        self.w_router = layer.w_router
        self.ws = torch.empty(moe_forward_i8_workspace_size(self.p), dtype=torch.uint8, device=self.device)
        parts = []
        for w in (layer.w1, layer.w3, layer.w2):
            q = torch.empty_like(w, dtype=torch.int8)
            scale = torch.empty(w.shape[:-1], dtype=torch.float32, device=w.device)
            moe_quantize_rows(w, q, scale)
            parts += [q, scale]
        self.weights = i8_weights(*parts)

    def forward(self, x, logit_bias=None, y=None, dbg: dict | None = None, stream=None):
        import torch
        if y is None:
            y = torch.empty((self.T, self.d), dtype=torch.bfloat16, device=self.device)
        moe_forward_i8(self.p, x, self.w_router, self.weights, logit_bias, y, self.ws, dbg, stream)
        return y
