"""One training step of a pre-norm MLP block that keeps its activations in 8 bits.

    out = x + relu(norm(x) W1^T) W2^T

The forward pass keeps three activations for the backward pass, each as an
8-bit checkpoint (33/32 bytes an element): the norm's input, saved by the norm
itself in the same pass, and the inputs of both layers.  The backward pass
reads the checkpoints: the weight gradients are delta^T a from them, the
norm's backward takes its input from one.  The two weight gradients are then
encoded to FP8 payloads, as they would go to the other workers, and decoded.

    python examples/mlp_block_step.py [--tokens 16384 --width 1536 --hidden 6144]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


class Block:
    def __init__(self, width, hidden, tokens, kind="layer", fmt="e4m3", device="cuda", seed=0):
        import fac_whitening_amd as fw
        self.fw, self.kind, self.tokens = fw, kind, tokens
        g = torch.Generator(device=device).manual_seed(seed)

        def param(m, d):
            return (torch.randn(m, d, generator=g, device=device) * d ** -0.5).bfloat16()

        self.w1, self.w2 = param(hidden, width), param(width, hidden)
        self.gamma = torch.ones(width, dtype=torch.bfloat16, device=device)
        self.beta = torch.zeros(width, dtype=torch.bfloat16, device=device) if kind == "layer" else None
        # kept from step to step: checkpoints, the gradients, and the layers' codecs
        self.ck_x = fw.ActCheckpoint(tokens, width, fmt, device=device)
        self.ck_y = fw.ActCheckpoint(tokens, width, fmt, device=device)
        self.ck_h = fw.ActCheckpoint(tokens, hidden, fmt, device=device)
        self.dw1 = torch.empty(hidden, width, device=device)
        self.dw2 = torch.empty(width, hidden, device=device)
        self.codec1, self.codec2 = (fw.Layer(*w.shape, "euclid", device=device) for w in (self.w1, self.w2))

    def forward(self, x):
        fw = self.fw
        y, self.mean, self.rstd = fw.norm_forward(x, self.gamma, self.beta, kind=self.kind, ckpt=self.ck_x)
        self.ck_y.save(y)
        h = torch.relu_(y @ self.w1.t())
        self.ck_h.save(h)
        return torch.addmm(x, h, self.w2.t())

    def backward(self, dout):
        """Gradients of the block's input, the norm's parameters and both weights."""
        fw, alpha = self.fw, 1.0 / self.tokens
        fw.weight_grad(dout, self.ck_h, alpha, out=self.dw2)
        # a hidden unit is live where its stored value is positive
        dh = (dout @ self.w2) * (self.ck_h.restore(torch.bfloat16) > 0)
        fw.weight_grad(dh, self.ck_y, alpha, out=self.dw1)
        dx, dgamma, dbeta = fw.norm_backward(dh @ self.w1, self.ck_x, self.mean, self.rstd, self.gamma, kind=self.kind)
        return {"dx": dx.add_(dout), "dgamma": dgamma, "dbeta": dbeta, "dw1": self.dw1, "dw2": self.dw2}

    def exchange(self):
        """Both weight gradients through the FP8 codec, with one worker."""
        out = []
        for codec, g in ((self.codec1, self.dw1), (self.codec2, self.dw2)):
            codes, scales = codec.encode(g)
            out.append(codec.decode_reduce(codes.unsqueeze(0), scales.unsqueeze(0)))
        return out

    def kept_bytes(self):
        return sum(c.nbytes() for c in (self.ck_x, self.ck_y, self.ck_h))


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=16384)
    ap.add_argument("--width", type=int, default=1536)
    ap.add_argument("--hidden", type=int, default=6144)
    ap.add_argument("--kind", choices=["layer", "rms"], default="layer")
    a = ap.parse_args()
    b = Block(a.width, a.hidden, a.tokens, a.kind)
    x = torch.randn(a.tokens, a.width, device="cuda").bfloat16()
    dout = (0.1 * torch.randn(a.tokens, a.width, device="cuda")).bfloat16()

    def step():
        out = b.forward(x)
        grads = b.backward(dout)
        return out, grads, b.exchange()

    step()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(10):
        out, grads, mean = step()
    end.record()
    torch.cuda.synchronize()
    print(f"step {start.elapsed_time(end) / 10:.3f} ms, activations kept {b.kept_bytes() / 1e6:.1f} MB "
          f"({2 * a.tokens * (2 * a.width + a.hidden) / 1e6:.1f} MB in bf16)")
    for name, g, m in (("dw1", grads["dw1"], mean[0]), ("dw2", grads["dw2"], mean[1])):
        print(f"{name}: norm {g.norm().item():.4g}, payload off by {((m - g).norm() / g.norm()).item():.4f}")


if __name__ == "__main__":
    main()
