"""One training step of a pre-norm gated MLP block with dropout.

    h = drop(act(y Wg^T) (y Wu^T)),  y = norm(x),  out = x + drop(h Wd^T)

Both projections are halves of one matrix, so one weight gradient makes both.
Neither dropout stores a mask: the backward pass draws it again from the same
seeds and the step's number.  The down projection's input is kept as an 8-bit
checkpoint, saved by the gated block itself; the norm's output is kept whole.
The weight gradients are then encoded to FP8 payloads, as they would go to the
other workers, and decoded.

    python examples/gated_block_step.py [--tokens 16384 --width 1536 --hidden 6144]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


class GatedBlock:
    def __init__(self, width, hidden, tokens, act="silu", p=0.1, fmt="e4m3", device="cuda", seed=0):
        import fac_whitening_amd as fw
        self.fw, self.act, self.tokens, self.hidden = fw, act, tokens, hidden
        g = torch.Generator(device=device).manual_seed(seed)

        def param(m, d):
            return (torch.randn(m, d, generator=g, device=device) * d ** -0.5).bfloat16()

        self.w1, self.w2 = param(2 * hidden, width), param(width, hidden)     # gate above up; down
        self.gamma = torch.ones(width, dtype=torch.bfloat16, device=device)
        # the step's number, counted on the device: a captured step draws anew at each replay
        self.step = torch.zeros(1, dtype=torch.int64, device=device)
        self.drop_h = fw.Dropout(p, seed=2 * seed + 1, counter=self.step)
        self.drop_o = fw.Dropout(p, seed=2 * seed + 2, counter=self.step)
        # kept from step to step
        self.ck_h = fw.ActCheckpoint(tokens, hidden, fmt, device=device)
        self.dgu = torch.empty(tokens, 2 * hidden, dtype=torch.bfloat16, device=device)
        self.dw1 = torch.empty(2 * hidden, width, device=device)
        self.dw2 = torch.empty(width, hidden, device=device)
        self.codec1, self.codec2 = (fw.Layer(*w.shape, "euclid", device=device) for w in (self.w1, self.w2))

    def forward(self, x):
        fw, f = self.fw, self.hidden
        self.x = x
        self.y, _, self.rstd = fw.norm_forward(x, self.gamma, kind="rms")
        h, self.gate, self.up = fw.glu_forward(self.y, self.w1[:f], self.w1[f:], act=self.act, keep=True,
                                               drop=self.drop_h, ckpt=self.ck_h)
        return fw.dropout_forward(h @ self.w2.t(), self.drop_o, residual=x)

    def backward(self, dout):
        """Gradients of the block's input, the norm's weight and both matrices."""
        fw, f, alpha = self.fw, self.hidden, 1.0 / self.tokens
        do = fw.dropout_backward(dout, self.drop_o)
        fw.weight_grad(do, self.ck_h, alpha, out=self.dw2)
        dy, _, _ = fw.glu_backward(do @ self.w2, self.gate, self.up, self.w1[:f], self.w1[f:], act=self.act,
                                   drop=self.drop_h, dgate=self.dgu[:, :f], dup=self.dgu[:, f:])
        fw.weight_grad(self.dgu, self.y, alpha, out=self.dw1)
        dx, dgamma, _ = fw.norm_backward(dy, self.x, None, self.rstd, self.gamma, kind="rms")
        self.step.add_(1)
        return {"dx": dx.add_(dout), "dgamma": dgamma, "dw1": self.dw1, "dw2": self.dw2}

    def exchange(self):
        """Both weight gradients through the FP8 codec, with one worker."""
        out = []
        for codec, g in ((self.codec1, self.dw1), (self.codec2, self.dw2)):
            codes, scales = codec.encode(g)
            out.append(codec.decode_reduce(codes.unsqueeze(0), scales.unsqueeze(0)))
        return out


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=16384)
    ap.add_argument("--width", type=int, default=1536)
    ap.add_argument("--hidden", type=int, default=6144)
    ap.add_argument("--act", choices=["silu", "gelu", "gelu_tanh", "relu", "sigmoid"], default="silu")
    ap.add_argument("--dropout", type=float, default=0.1)
    a = ap.parse_args()
    b = GatedBlock(a.width, a.hidden, a.tokens, a.act, a.dropout)
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
    print(f"step {start.elapsed_time(end) / 10:.3f} ms")
    for name, g, m in (("dw1", grads["dw1"], mean[0]), ("dw2", grads["dw2"], mean[1])):
        print(f"{name}: norm {g.norm().item():.4g}, payload off by {((m - g).norm() / g.norm()).item():.4f}")


if __name__ == "__main__":
    main()
