"""A gated MLP block trained with MXFP4 weights and MXFP8 activations, and served.

    y   = rmsnorm(x) w_norm           -> E4M3 codes           (rmsnorm_mx)
    gu  = y W_up^T                    E4M3 x E2M1             (mxfp4_scaled_gemm)
    h   = silu(g) u                   -> E4M3 codes           (swiglu_mx)
    out = x + h W_down^T              E4M3 x E2M1             (mxfp4_scaled_gemm)

The backward pass keeps x, gu, y and h as 8-bit codes.  Data gradients are E5M2 x E2M1
products with the transposed weights; weight gradients are E5M2 x E4M3 products over the
tokens, whose activation operand is turned from the kept codes (requantize_mx_t).  The
weights are fp32 masters, quantized again after each update (gradients pass straight
through the quantization).

    python examples/gated_mlp.py [--tokens 500 --hidden 512 --inner 1408 --steps 30]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mx_block_scaled_x128_amd as mx  # noqa: E402

EPS = 1e-6


class GatedMLP:
    """hidden and inner sizes are multiples of 128 (the K of the products)."""

    def __init__(self, hidden, inner, device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)

        def weight(rows, cols):
            return torch.randn(rows, cols, generator=gen, device=device) * cols ** -0.5
        self.norm = torch.ones(hidden, device=device)
        self.up, self.down = weight(2 * inner, hidden), weight(hidden, inner)
        self.quantize()

    def quantize(self):
        """The weights' codes in both orientations: along the inputs for the forward product,
        along the outputs for the data gradient's."""
        self.up_q, self.down_q = mx.quantize_mxfp4(self.up), mx.quantize_mxfp4(self.down)
        self.up_t = mx.quantize_mx_t(self.up, mx.E2M1, mx.RULE_FLOOR)
        self.down_t = mx.quantize_mx_t(self.down, mx.E2M1, mx.RULE_FLOOR)

    def forward(self, x, keep=True):
        """out [tokens][hidden] in bf16 for x of that shape and, with keep, what backward needs."""
        y, ys, norm_kept = mx.rmsnorm_mx(x, self.norm, EPS, keep=keep)
        gu = mx.mxfp4_scaled_gemm(y, ys, mx.E4M3, *self.up_q, out_dtype=torch.bfloat16)
        h, hs, act_kept = mx.swiglu_mx(gu, keep=keep)
        out = mx.mxfp4_scaled_gemm(h, hs, mx.E4M3, *self.down_q, out_dtype=torch.bfloat16)
        return x + out, ((y, ys), norm_kept, (h, hs), act_kept) if keep else None

    @staticmethod
    def _weight_grad(grad, codes, scales):
        """grad^T activations over the tokens (filled up to a multiple of 128 with zeros)."""
        g, gs = mx.quantize_mx_t(grad, mx.E5M2)
        a, a_s = mx.requantize_mx_t(codes, scales, mx.E4M3)
        return mx.mx_scaled_gemm(g, gs, mx.E5M2, a, a_s, mx.E4M3)

    @staticmethod
    def _data_grad(grad, weight_t):
        q, s, _ = mx.quantize_mx(grad, mx.E5M2, mx.RULE_CEIL, counts=False)
        return mx.mxfp4_scaled_gemm(q, s, mx.E5M2, *weight_t, out_dtype=torch.bfloat16)

    def backward(self, kept, dout):
        """dx and the gradients of norm, up and down; dout [tokens][hidden] in bf16."""
        y, norm_kept, h, act_kept = kept
        ddown = self._weight_grad(dout, *h)
        dgu = mx.swiglu_mx_backward(act_kept, self._data_grad(dout, self.down_t))
        dup = self._weight_grad(dgu, *y)
        dx, dnorm = mx.rmsnorm_mx_backward(norm_kept, self.norm, self._data_grad(dgu, self.up_t))
        return dout + dx, {"norm": dnorm, "up": dup, "down": ddown}

    def update(self, grads, rate):
        for name, g in grads.items():
            getattr(self, name).sub_(g, alpha=rate)
        self.quantize()


def reference(mlp, x, dout):
    """The same block in fp32 with torch's own gradients."""
    x, norm, up, down = (t.detach().float().clone().requires_grad_(True) for t in (x, mlp.norm, mlp.up, mlp.down))
    y = x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * norm
    g, u = (y @ up.t()).chunk(2, dim=1)
    out = x + (torch.nn.functional.silu(g) * u) @ down.t()
    out.backward(dout.float())
    return out.detach(), x.grad, {"norm": norm.grad, "up": up.grad, "down": down.grad}


def cosine(a, b):
    return torch.nn.functional.cosine_similarity(a.float().flatten(), b.float().flatten(), dim=0).item()


def train(tokens, hidden, inner, steps, rate=2.0, seed=0):
    """Losses of fitting a teacher block of the same shape, and the block."""
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    teacher, mlp = GatedMLP(hidden, inner, seed=seed + 2), GatedMLP(hidden, inner, seed=seed + 3)
    x = torch.randn(tokens, hidden, generator=gen, device="cuda").bfloat16()
    target = teacher.forward(x, keep=False)[0]
    losses = []
    for _ in range(steps):
        out, kept = mlp.forward(x)
        diff = (out - target).float()
        losses.append(diff.square().mean().item())
        _, grads = mlp.backward(kept, (diff * (2 / tokens)).bfloat16())
        mlp.update(grads, rate / hidden)
    return losses, mlp


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 500), ("hidden", 512), ("inner", 1408), ("steps", 30)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    losses, mlp = train(a.tokens, a.hidden, a.inner, a.steps)
    for i in range(0, len(losses), max(1, len(losses) // 10)):
        print("step %3d  loss %.5f" % (i, losses[i]))
    x = torch.randn(a.tokens, a.hidden, device="cuda").bfloat16()
    out, kept = mlp.forward(x)
    dout = torch.randn(a.tokens, a.hidden, device="cuda").mul_(1e-3).bfloat16()
    dx, grads = mlp.backward(kept, dout)
    ref, ref_dx, ref_grads = reference(mlp, x, dout)
    print("cosine with fp32: out %.4f  dx %.4f  " % (cosine(out, ref), cosine(dx, ref_dx))
          + "  ".join("d%s %.4f" % (k, cosine(grads[k], ref_grads[k])) for k in grads))
    (y, ys), n, (h, hs), k = kept
    held = sum(t.numel() * t.element_size() for t in (y, ys, n.codes, n.scales, n.rstd, h, hs, k.codes, k.scales))
    print("kept for the backward pass: %.1f KB, in bf16 %.1f KB"
          % (held / 1e3, 2 * (y.numel() + n.codes.numel() + h.numel() + k.codes.numel()) / 1e3))
    token = mlp.forward(x[:1], keep=False)[0]
    print("one token served: cosine with the batch's row %.4f" % cosine(token, out[:1]))


if __name__ == "__main__":
    main()
