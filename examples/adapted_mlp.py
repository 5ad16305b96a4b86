"""A gated MLP block with frozen MXFP4 weights, tuned through low-rank adapters and its norm,
and served to requests with adapters of their own.

    y   = layernorm(x) w + b                     -> E4M3 codes       (layernorm_mx)
    gu  = y W_up^T + (y A_up^T) B_up^T           E4M3 x E2M1         (mxfp4_adapted_gemm)
    h   = silu(g) u                              -> E4M3 codes       (swiglu_mx)
    out = x + h W_down^T + (h A_down^T) B_down^T                     (mxfp4_adapted_gemm)

The weights are quantized once, in both orientations.  Each row of x names its adapter (or
none), so that one call serves a batch of requests, and one backward pass gives the gradients
of all adapters whose rows it holds.  Data gradients are the same adapted products with the
transposed weight and adapters, on the gradient as E5M2 codes; those codes and the kept ones
are what the adapters' gradients are taken from (adapter_grad_mx).

    python examples/adapted_mlp.py [--tokens 500 --hidden 512 --inner 1408 --rank 16 --adapters 3]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mx_block_scaled_x128_amd as mx  # noqa: E402

EPS = 1e-5


class Adapted:
    """A frozen linear layer [out][in] and its adapters; sizes are multiples of 128, the rank of 8."""

    def __init__(self, weight, adapters, rank, gen):
        self.q = mx.quantize_mxfp4(weight)
        self.q_t = mx.quantize_mx_t(weight, mx.E2M1, mx.RULE_FLOOR)
        rows, cols = weight.shape
        self.down = torch.randn(adapters, rank, cols, generator=gen, device=weight.device).mul_(cols ** -0.5)
        self.up = torch.randn(adapters, rows, rank, generator=gen, device=weight.device).mul_(0.1 * rank ** -0.5)
        self.alpha = torch.ones(adapters, device=weight.device)
        self.cast()

    def cast(self):
        """The adapters as the kernels take them, bf16 copies of the fp32 masters."""
        self.down_16, self.up_16 = self.down.bfloat16(), self.up.bfloat16()

    def forward(self, x, ids):
        """(out in bf16, the adapters' projection) for x = (codes, scales)."""
        return mx.mxfp4_adapted_gemm(*x, mx.E4M3, *self.q, self.down_16, self.up_16, ids, self.alpha,
                                     out_dtype=torch.bfloat16)

    def backward(self, x, p, ids, grad):
        """(dx, {down, up}) from what forward took and gave and the output's gradient in bf16."""
        g, gs, _ = mx.quantize_mx(grad, mx.E5M2, mx.RULE_CEIL, counts=False)
        up_t, down_t = self.up_16.transpose(1, 2).contiguous(), self.down_16.transpose(1, 2).contiguous()
        dx, u = mx.mxfp4_adapted_gemm(g, gs, mx.E5M2, *self.q_t, up_t, down_t, ids, self.alpha, out_dtype=torch.bfloat16)
        n = len(self.alpha)
        return dx, {"down": mx.adapter_grad_mx(u, *x, mx.E4M3, ids, n),
                    "up": mx.adapter_grad_mx(p, g, gs, mx.E5M2, ids, n, transposed=True)}


class AdaptedMLP:
    def __init__(self, hidden, inner, adapters, rank, device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)

        def weight(rows, cols):
            return torch.randn(rows, cols, generator=gen, device=device) * cols ** -0.5
        self.w = torch.randn(hidden, generator=gen, device=device).mul_(0.1).add_(1)
        self.b = torch.randn(hidden, generator=gen, device=device).mul_(0.1)
        self.up = Adapted(weight(2 * inner, hidden), adapters, rank, gen)
        self.down = Adapted(weight(hidden, inner), adapters, rank, gen)

    def forward(self, x, ids, keep=True):
        """out [tokens][hidden] in bf16 and, with keep, what backward needs; ids [tokens] int32."""
        y, ys, norm = mx.layernorm_mx(x, self.w, self.b, EPS, keep=keep)
        gu, p_up = self.up.forward((y, ys), ids)
        h, hs, act = mx.swiglu_mx(gu, keep=keep)
        out, p_down = self.down.forward((h, hs), ids)
        return x + out, ((y, ys), norm, p_up, (h, hs), act, p_down, ids) if keep else None

    def backward(self, kept, dout):
        """dx and the gradients of w, b and the adapters; dout [tokens][hidden] in bf16."""
        y, norm, p_up, h, act, p_down, ids = kept
        dh, down = self.down.backward(h, p_down, ids, dout)
        dy, up = self.up.backward(y, p_up, ids, mx.swiglu_mx_backward(act, dh))
        dx, dw, db = mx.layernorm_mx_backward(norm, self.w, dy)
        return dout + dx, {"w": dw, "b": db, "up.down": up["down"], "up.up": up["up"], "down.down": down["down"],
                           "down.up": down["up"]}

    def parameters(self):
        return {"w": self.w, "b": self.b, "up.down": self.up.down, "up.up": self.up.up, "down.down": self.down.down,
                "down.up": self.down.up}

    def update(self, grads, rate):
        for name, value in self.parameters().items():
            value.sub_(grads[name], alpha=rate)
        self.up.cast()
        self.down.cast()


def reference(mlp, x, ids, dout):
    """The same block in fp32, its weights' codes as they are, with torch's own gradients."""
    p = {k: v.detach().clone().requires_grad_(True) for k, v in mlp.parameters().items()}
    x = x.detach().float().requires_grad_(True)

    def linear(z, layer, name):
        out = z @ mx.dequantize_mx(*layer.q, mx.E2M1).t()
        for a in range(len(layer.alpha)):
            own = (ids == a).float()[:, None]
            out = out + own * ((z @ p[name + ".down"][a].t()) @ p[name + ".up"][a].t())
        return out
    y = torch.nn.functional.layer_norm(x, x.shape[1:], p["w"], p["b"], EPS)
    g, u = linear(y, mlp.up, "up").chunk(2, dim=1)
    out = x + linear(torch.nn.functional.silu(g) * u, mlp.down, "down")
    out.backward(dout.float())
    return out.detach(), x.grad, {k: v.grad for k, v in p.items()}


def cosine(a, b):
    return torch.nn.functional.cosine_similarity(a.float().flatten(), b.float().flatten(), dim=0).item()


def sequences(tokens, adapters, device="cuda"):
    """ids of as many sequences as adapters and one without, behind each other."""
    return (torch.arange(tokens, device=device) * (adapters + 1) // tokens - 1).int()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 500), ("hidden", 512), ("inner", 1408), ("rank", 16), ("adapters", 3), ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    mlp = AdaptedMLP(a.hidden, a.inner, a.adapters, a.rank)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(a.tokens, a.hidden, generator=gen, device="cuda").bfloat16()
    dout = torch.randn(a.tokens, a.hidden, generator=gen, device="cuda").mul_(1e-3).bfloat16()
    ids = sequences(a.tokens, a.adapters)
    out, kept = mlp.forward(x, ids)
    dx, grads = mlp.backward(kept, dout)
    ref, ref_dx, ref_grads = reference(mlp, x, ids, dout)
    print("cosine with fp32: out %.4f  dx %.4f  " % (cosine(out, ref), cosine(dx, ref_dx))
          + "  ".join("%s %.4f" % (k, cosine(grads[k], ref_grads[k])) for k in grads))
    target = AdaptedMLP(a.hidden, a.inner, a.adapters, a.rank, seed=0)
    target.update({k: torch.randn_like(v) * v.std() for k, v in target.parameters().items()}, 0.5)
    goal = target.forward(x, ids, keep=False)[0]
    for step in range(a.steps):
        out, kept = mlp.forward(x, ids)
        diff = (out - goal).float()
        if step % max(1, a.steps // 5) == 0:
            print("step %3d  loss %.5f" % (step, diff.square().mean().item()))
        mlp.update(mlp.backward(kept, (diff * (2 / a.tokens)).bfloat16())[1], 0.05)
    every = max(1, a.tokens // 8)
    served = mlp.forward(x[::every], ids[::every].contiguous(), keep=False)[0]
    print("%d requests served, cosine with the same rows of the whole %.4f"
          % (len(served), cosine(served, mlp.forward(x, ids, keep=False)[0][::every])))


if __name__ == "__main__":
    main()
