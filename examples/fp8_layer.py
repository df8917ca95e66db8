"""A linear layer behind an RMS norm, trained with 8-bit forward and input-gradient
products and a 16-bit weight gradient.

One optimizer step over several micro-batches:

  forward    rmsnorm: h = x + residual, its norm in bf16 (kept for the weight
             gradient) and in e4m3 codes with a scale per 128 columns;
             linear_fp8: Y = X W^T from the codes and the quantised weight
  backward   quantize_b128: the loss gradient's codes; dgrad_fp8: dX = dY W from
             the same quantised weight; rmsnorm_backward: through the norm;
             wgrad_accumulate: the exact fp32 sum of dY^T X (bf16 operands)
  step       grad_norm over the accumulators, adamw_clip with the coefficient it
             left on the device, quantize_b128 of the new weight

Run `python examples/fp8_layer.py` on a GB300: it fits a random teacher and prints
the loss and the gradient norm.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from weight_gradient_gemm_gb300 import forge  # noqa: E402

EPS = 1e-5


class Fp8Layer:
    """Y = rmsnorm(x + residual) W^T, with everything a step keeps between calls."""

    def __init__(self, d_in: int, d_out: int, bt: int, device="cuda", seed: int = 0):
        g = torch.Generator(device=device).manual_seed(seed)
        f32 = dict(dtype=torch.float32, device=device)
        b16 = dict(dtype=torch.bfloat16, device=device)
        self.bt, self.d_in, self.d_out, self.step_count = bt, d_in, d_out, 0
        self.W = (torch.randn((d_out, d_in), generator=g, device=device) * d_in ** -0.5).bfloat16()
        self.gain = torch.ones(d_in, **f32)
        self.m, self.v, _, _ = forge.alloc_moments(d_out, d_in, forge.MOM_FP32, device)
        # the weight as the 8-bit products read it
        self.Wq, self.Ws = forge.alloc_b128(d_out, d_in, 128, device)
        forge.quantize_b128(self.W, self.Wq, self.Ws, block_rows=128)
        # activations of one micro-batch
        self.h, self.X = torch.empty((bt, d_in), **b16), torch.empty((bt, d_in), **b16)
        self.Xq, self.Xs = forge.alloc_b128(bt, d_in, 1, device)
        self.rstd = torch.empty(bt, **f32)
        self.Y = torch.empty((bt, d_out), **b16)
        self.dYq, self.dYs = forge.alloc_b128(bt, d_out, 1, device)
        self.dX, self.dh = torch.empty((bt, d_in), **b16), torch.empty((bt, d_in), **b16)
        # gradients of a step
        self.dW = torch.empty((d_out, d_in), **f32)
        self.dgain = torch.empty(d_in, **f32)
        self.dgain_sum = torch.zeros(d_in, **f32)
        self.clip = torch.empty(2, **f32)     # the norm and the coefficient
        self.workspace = torch.empty(
            max(forge.rmsnorm_backward_workspace_bytes(bt, d_in),
                forge.grad_norm_workspace_bytes(2), 16), dtype=torch.uint8, device=device)
        self.micro = 0

    def forward(self, x: torch.Tensor, residual: torch.Tensor) -> torch.Tensor:
        forge.rmsnorm(x, self.gain, eps=EPS, residual=residual, sum_out=self.h, y=self.X,
                      codes=self.Xq, scales=self.Xs, rstd=self.rstd)
        forge.linear_fp8(self.Xq, self.Xs, self.Wq, self.Ws, self.Y)
        return self.Y

    def backward(self, dY: torch.Tensor, dsum=None) -> torch.Tensor:
        """The gradient of x (and of the residual); the weight's and the gain's are
        added to the step's sums."""
        forge.quantize_b128(dY, self.dYq, self.dYs)
        forge.dgrad_fp8(self.dYq, self.dYs, self.Wq, self.Ws, self.dX)
        forge.rmsnorm_backward(self.dX, self.h, self.gain, self.rstd, self.dh, self.dgain,
                               dsum=dsum, workspace=self.workspace)
        self.dgain_sum += self.dgain
        forge.wgrad_accumulate(self.X, dY, self.dW, 1.0 if self.micro else 0.0)
        self.micro += 1
        return self.dh

    def step(self, lr: float, max_norm: float = 1.0) -> torch.Tensor:
        """Clips by the global norm, steps the weight and the gain, quantises the
        weight again.  Returns the norm and the coefficient (on the device)."""
        self.step_count += 1
        forge.grad_norm([self.dW, self.dgain_sum], max_norm, self.clip, workspace=self.workspace)
        forge.adamw_clip(self.dW, self.W, self.m, self.v, self.clip, lr=lr, beta1=0.9, beta2=0.95,
                         eps=1e-8, weight_decay=0.0, step=self.step_count)
        self.gain -= lr * self.clip[1] * self.dgain_sum
        forge.quantize_b128(self.W, self.Wq, self.Ws, block_rows=128)
        self.dgain_sum.zero_()
        self.micro = 0
        return self.clip


def train(steps: int = 40, bt: int = 512, d_in: int = 1024, d_out: int = 1536,
          micro_batches: int = 2, lr: float = 2e-3, seed: int = 0):
    """Fits a random linear teacher of the normalised input; the losses by step."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed + 1)
    teacher = (torch.randn((d_out, d_in), generator=g, device=dev) * d_in ** -0.5).bfloat16()
    layer = Fp8Layer(d_in, d_out, bt, dev, seed)
    batches = []
    for _ in range(micro_batches):
        x = torch.randn((bt, d_in), generator=g, device=dev).bfloat16()
        r = torch.randn((bt, d_in), generator=g, device=dev).bfloat16()
        h = x.float() + r.float()
        y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
        batches.append((x, r, y @ teacher.float().t()))
    losses, norms = [], []
    for _ in range(steps):
        loss = torch.zeros((), device=dev)
        for x, r, target in batches:
            diff = layer.forward(x, r).float() - target
            loss += diff.square().mean() / micro_batches
            layer.backward((diff * (2.0 / (diff.numel() * micro_batches))).bfloat16())
        norms.append(layer.step(lr)[0].clone())
        losses.append(loss)
    if forge.device_error() != 0:
        raise RuntimeError("a kernel reported an error")
    return [float(v) for v in losses], [float(v) for v in norms]


if __name__ == "__main__":
    loss, norm = train()
    for i in range(0, len(loss), 5):
        print(f"step {i:3d}  loss {loss[i]:.5f}  gradient norm {norm[i]:.5f}")
    print(f"last      loss {loss[-1]:.5f}")
