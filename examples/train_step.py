"""Train one pre-norm MoE layer, y = x + MoE(norm(x)), on a synthetic target.

Every kernel of the step is the library's: layer norm, router, dispatch, expert
FFNs, combine, and the gradient of each; torch holds the memory, forms the loss
(the mean squared distance to the target plus the load-balancing loss) and
takes the optimiser's step on fp32 master weights.  The target is a second
layer with weights of its own, so the loss can fall.

    python examples/train_step.py                      # bf16, 30 steps
    python examples/train_step.py --dtype f32 --n 256 --d 128 --d-ff 256
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_synth  # noqa: E402
from mixture_experts_layer_moe_gb300 import moe  # noqa: E402

_DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


class MoEBlock:
    """The layer's parameters, and the buffers of one step (allocated once)."""

    def __init__(self, cfg: moe_synth.MoEConfig, seed: int, aux_weight: float = 0.01):
        self.cfg, self.aux_weight = cfg, aux_weight
        n, d, F, E, k = cfg.n, cfg.d, cfg.d_ff, cfg.E, cfg.k
        P, dt = n * k, _DTYPE[cfg.act_dtype]
        g = torch.Generator(device="cuda").manual_seed(seed)
        shapes = dict(gamma=(d,), beta=(d,), Wg=(E, d), bias=(E,), W1=(E, F, d), W3=(E, F, d),
                      W2=(E, d, F))
        self.master = {}
        for name, shape in shapes.items():
            t = torch.randn(shape, generator=g, device="cuda") * shape[-1] ** -0.5
            if name in ("gamma", "beta", "bias"):
                t.fill_(1.0 if name == "gamma" else 0.0)
            self.master[name] = t
        # bf16 copies of the parameters (the router's bias stays fp32)
        self.p = {name: t.to(torch.float32 if name == "bias" else dt).clone()
                  for name, t in self.master.items()}
        self.grad = {name: torch.empty_like(t) for name, t in self.p.items()}
        for name in ("gamma", "beta"):
            self.grad[name] = torch.empty(d, device="cuda")      # summed in fp32
        self.w = moe.make_weights(self.p)
        self.expert_grads = moe.make_expert_grads(self.grad)
        self.ws = moe.alloc_train_workspace(cfg)
        self.norm_ws = torch.empty(max(256, moe.moe_layernorm_workspace_size(n, d, cfg.act_dtype)),
                                   dtype=torch.uint8, device="cuda")
        new = lambda *s, dtype=dt: torch.empty(*s, dtype=dtype, device="cuda")
        f32, i32 = torch.float32, torch.int32
        self.xn, self.y = new(n, d), new(n, d)
        self.mean, self.rstd = new(n, dtype=f32), new(n, dtype=f32)
        self.idx, self.gate, self.probs = new(n, k, dtype=i32), new(n, k, dtype=f32), new(n, E, dtype=f32)
        self.counts, self.offsets = new(E, dtype=i32), new(E + 1, dtype=i32)
        self.perm, self.inv_perm = new(P, dtype=i32), new(P, dtype=i32)
        self.x_perm, self.y_perm = new(P, d), new(P, d)
        self.g, self.u, self.h = new(P, F), new(P, F), new(P, F)
        self.Pm, self.f, self.aux = new(E, dtype=f32), new(E, dtype=f32), new(4, dtype=f32)
        self.dy_perm, self.dx_perm, self.dgate = new(P, d), new(P, d), new(n, k, dtype=f32)
        self.dxn, self.dx = new(n, d), new(n, d)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        """x + MoE(norm(x)); keeps what backward() reads.  self.aux[0]: the balancing loss."""
        cfg, ws = self.cfg, self.ws
        moe.moe_layernorm(x, self.p["gamma"], self.p["beta"], self.xn, self.mean, self.rstd)
        moe.moe_route(cfg, self.xn, self.w, self.idx, self.gate, self.probs, ws)
        moe.moe_route_stats(cfg, self.probs, self.idx, self.aux_weight, self.Pm, self.f, self.aux[:1],
                            ws)
        moe.moe_dispatch(cfg, self.idx, self.xn, self.counts, self.offsets, self.perm, self.inv_perm,
                         self.x_perm, ws)
        moe.moe_expert_ffn_train(cfg, self.x_perm, self.offsets, self.w, self.g, self.u, self.h,
                                 self.y_perm, ws)
        moe.moe_combine(cfg, self.y_perm, self.inv_perm, self.gate, None, self.y, ws)
        return x + self.y

    def backward(self, x: torch.Tensor, dout: torch.Tensor) -> torch.Tensor:
        """Gradients of every parameter (self.grad) and of x, from the output's gradient."""
        cfg, ws, grad = self.cfg, self.ws, self.grad
        moe.moe_combine_backward(cfg, dout, self.y_perm, self.inv_perm, self.gate, self.dy_perm,
                                 self.dgate, ws)
        moe.moe_expert_ffn_backward(cfg, self.x_perm, self.offsets, self.w, self.g, self.u, self.h,
                                    self.dy_perm, self.dx_perm, self.expert_grads, ws)
        moe.moe_route_backward(cfg, self.xn, self.w, self.probs, self.idx, self.gate, self.dgate,
                               self.f, self.aux_weight, self.inv_perm, self.dx_perm, self.dxn,
                               grad["Wg"], grad["bias"], ws)
        moe.moe_layernorm_backward(x, self.p["gamma"], self.mean, self.rstd, self.dxn, self.dx,
                                   grad["gamma"], grad["beta"], self.norm_ws)
        return dout + self.dx

    def step(self, lr: float):
        for name, t in self.master.items():
            t.sub_(self.grad[name].float(), alpha=lr)
            self.p[name].copy_(t)


def train(cfg: moe_synth.MoEConfig, steps: int, lr: float, seed: int = 0) -> list[float]:
    """The loss of each step."""
    block, teacher = MoEBlock(cfg, seed), MoEBlock(cfg, seed + 1)
    g = torch.Generator(device="cuda").manual_seed(seed + 2)
    x = torch.randn(cfg.n, cfg.d, generator=g, device="cuda").to(_DTYPE[cfg.act_dtype])
    target = teacher.forward(x).float()
    losses = []
    for _ in range(steps):
        err = block.forward(x).float() - target
        losses.append(float(err.square().mean() / 2 + block.aux[0]))
        # the loss of a token is its own distance: gradients of order one
        block.backward(x, err.to(x.dtype))
        block.step(lr / cfg.n)
        for b in (block, teacher):
            st, detail = moe.moe_status_check(b.ws)
            if st != 0:
                raise RuntimeError(f"device status {moe.status_string(st)} ({detail})")
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("n", 2048), ("d", 512), ("d-ff", 1024), ("experts", 8), ("top-k", 2),
                          ("steps", 30)):
        ap.add_argument("--" + name, type=int, default=default)
    ap.add_argument("--lr", type=float, default=0.3)
    ap.add_argument("--dtype", choices=sorted(_DTYPE), default="bf16")
    ap.add_argument("--gate", choices=("renorm", "top_prob"), default="renorm")
    a = ap.parse_args()
    cfg = moe_synth.MoEConfig("train", a.n, a.d, a.d_ff, a.experts, a.top_k, a.dtype, a.dtype, a.gate,
                              "swiglu")
    for i, loss in enumerate(train(cfg, a.steps, a.lr)):
        print(f"step {i:3d}  loss {loss:.5f}")


if __name__ == "__main__":
    main()
