"""Trains a pre-norm MLP block with FP8 linear layers, then serves it in int8.

    y = x + relu(norm(x) W1^T)^2 W2^T

Training, on bf16 activations with fp32 master weights: layer norm forward and
backward, both linear layers in block-scaled FP8 (forward, dgrad and wgrad),
and one AdamW step over all four tensors with E4M3 moments.  Serving: the two
weights quantized to int8 once (a scale per output channel), activations per
token, both products in int8; a few tokens or a whole prompt take the same
calls.

    python examples/norm_mlp.py [--steps 60]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_precision_quant_amd as fq  # noqa: E402


class Block:
    def __init__(self, hidden, inner, device="cuda:0", seed=0):
        g = torch.Generator().manual_seed(seed)
        self.gamma = torch.ones(hidden, device=device)
        self.beta = torch.zeros(hidden, device=device)
        self.w1 = (torch.randn(inner, hidden, generator=g) / hidden ** 0.5).to(device)
        self.w2 = (0.5 * torch.randn(hidden, inner, generator=g) / inner ** 0.5).to(device)

    def parameters(self):
        return [self.gamma, self.beta, self.w1, self.w2]


def _linear(x, w):
    """x w^T in FP8, and what its backward pass reads: x by columns, w's codes."""
    qx, sx, qxT, sxT = fq.fp8_quant_transpose(x)
    qw, sw = fq.fp8_quant_blockwise(w, fq.BLOCK_128x128)
    y = fq.fp8_gemm_blockscaled(qx, sx, fq.ROW_1x128, qw, sw, fq.BLOCK_128x128, fq.B_NK)
    return y, (qxT, sxT, qw, sw)


def _linear_backward(dy, saved):
    """(dx in bf16, dw in fp32)"""
    qxT, sxT, qw, sw = saved
    qdy, sdy, qdyT, sdyT = fq.fp8_quant_transpose(dy)
    dx = fq.fp8_gemm_blockscaled(qdy, sdy, fq.ROW_1x128, qw, sw, fq.BLOCK_128x128, fq.B_KN)
    dw = fq.fp8_gemm_blockscaled(qdyT, sdyT, fq.ROW_1x128, qxT, sxT, fq.ROW_1x128, fq.B_NK, out_dtype=torch.float32)
    return dx, dw


def train_step(block, plan, x, target, step, lr=3e-3):
    """One step on the mean squared error; returns the loss (on the GPU)."""
    n, mean, rstd = fq.fp8q_layer_norm_forward(x, block.gamma, block.beta)
    h, saved1 = _linear(n, block.w1)
    r = h.float().relu()
    a = (r * r).to(torch.bfloat16)
    o, saved2 = _linear(a, block.w2)
    d = x.float() + o.float() - target.float()
    loss = (d * d).mean()
    do = (2 / d.numel() * d).to(torch.bfloat16)
    da, dw2 = _linear_backward(do, saved2)
    dh = (2 * r * da.float()).to(torch.bfloat16)
    dn, dw1 = _linear_backward(dh, saved1)
    _, dgamma, dbeta = fq.fp8q_layer_norm_backward(dn, x, mean, rstd, block.gamma)
    fq.fp8q_adamw_multi_step(plan, [dgamma, dbeta, dw1, dw2], lr=lr, weight_decay=0.01, step=step)
    return loss


class Int8Block:
    """A trained block with its weights in int8."""

    def __init__(self, block):
        self.gamma, self.beta = block.gamma, block.beta
        self.w1, self.s1 = fq.fp8q_int8_quant_rows(block.w1)
        self.w2, self.s2 = fq.fp8q_int8_quant_rows(block.w2)

    def __call__(self, x):
        n, _, _ = fq.fp8q_layer_norm_forward(x, self.gamma, self.beta)
        h = fq.fp8q_int8_gemm(*fq.fp8q_int8_quant_rows(n), self.w1, self.s1)
        r = h.relu()
        o = fq.fp8q_int8_gemm(*fq.fp8q_int8_quant_rows(r * r), self.w2, self.s2)
        return x + o


def reference(block, x):
    """The block in fp32."""
    x = x.float()
    c = x - x.mean(1, keepdim=True)
    n = c * torch.rsqrt(c.square().mean(1, keepdim=True) + 1e-5) * block.gamma + block.beta
    return x + (n @ block.w1.t()).relu().square() @ block.w2.t()


def main(steps=60, tokens=1024, hidden=512, inner=2048, device="cuda:0"):
    """Trains towards another block's outputs; returns (first loss, last loss, errors of int8 serving by tokens)."""
    teacher, block = Block(hidden, inner, device, seed=1), Block(hidden, inner, device, seed=2)
    plan = fq.fp8q_adamw_plan(block.parameters(), fq.STATE_E4M3)
    g = torch.Generator(device=device).manual_seed(3)
    losses = []
    for step in range(1, steps + 1):
        x = torch.randn(tokens, hidden, device=device, generator=g).to(torch.bfloat16)
        losses.append(train_step(block, plan, x, reference(teacher, x).to(torch.bfloat16), step))
    losses = torch.stack(losses).tolist()
    served, errors = Int8Block(block), {}
    for m in (1, 17, tokens):
        x = torch.randn(m, hidden, device=device, generator=g).to(torch.bfloat16)
        want = reference(block, x) - x.float()
        errors[m] = ((served(x).float() - x.float() - want).norm() / want.norm()).item()
    return losses[0], losses[-1], errors


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    first, last, errors = main(ap.parse_args().steps)
    print("loss %.4f -> %.4f" % (first, last))
    for m, e in errors.items():
        print("int8 serving of %d token(s): error %.4f of the block's output" % (m, e))
